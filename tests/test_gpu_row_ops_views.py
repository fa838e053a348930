"""Row-wise operators on views with several leading dimensions whose rows lie apart (GPU)."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def _swg():
    import swiglu_ffn_backward_gb300 as swg
    return swg


def _rn(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda")


def _padded(shape, pad, seed=1, dtype=torch.bfloat16):
    """[..., V] inside rows of V + pad, the pad NaN; the whole buffer as well."""
    buf = torch.full((*shape[:-1], shape[-1] + pad), float("nan"), dtype=dtype, device="cuda")
    buf[..., : shape[-1]] = _rn(seed, *shape).to(dtype)
    return buf[..., : shape[-1]], buf


def _copies(call):
    """Bytes that a call allocates beyond what it returns, at its peak."""
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    out = call()
    torch.cuda.synchronize()
    peak = torch.cuda.max_memory_allocated() - before
    kept = torch.cuda.memory_allocated() - before
    return out, peak - kept


VIEWS = [((2, 3, 1000), 24), ((2, 1, 3, 777), 11), ((5, 1, 2048), 8), ((1, 4, 333), 3)]


@pytest.mark.parametrize("shape,pad", VIEWS, ids=lambda v: str(v))
def test_gradient_over_padded_logits(shape, pad):
    swg = _swg()
    z, buf = _padded(shape, pad)
    lead, V = shape[:-1], shape[-1]
    t = (torch.arange(z[..., 0].numel(), device="cuda") * 37 % V).view(lead)
    dl = _rn(2, *lead)
    dense = z.contiguous()
    st = swg.token_logprobs_fwd(dense, t)["stats"]
    want = swg.token_logprobs_bwd(dl, dense, t, st)
    got = swg.token_logprobs_bwd(dl, z, t, st, dlogits=z)
    assert got.data_ptr() == buf.data_ptr() and got.shape == z.shape
    torch.testing.assert_close(got, want, rtol=0, atol=0)
    assert buf[..., V:].isnan().all()


@pytest.mark.parametrize("shape,pad", VIEWS, ids=lambda v: str(v))
def test_distillation_over_padded_logits(shape, pad):
    swg = _swg()
    lead, V = shape[:-1], shape[-1]
    ids = torch.rand(shape, device="cuda", generator=torch.Generator("cuda").manual_seed(5)).topk(6, dim=-1).indices
    tl, w = _rn(3, *lead, 6), _rn(4, *lead)
    rows = lambda buf: buf.view(-1, V + pad)[:, :V]  # noqa: E731  (the same memory in two dimensions)
    flat = (ids.view(-1, 6), tl.view(-1, 6), w.view(-1))
    want = swg.distill_fwd_bwd(rows(_padded(shape, pad)[1]), flat[0], flat[1], flat[2])
    z, buf = _padded(shape, pad)
    out = swg.distill_fwd_bwd(z, ids, tl, w, out={"dlogits": z})
    assert out["dlogits"].data_ptr() == buf.data_ptr() and out["dlogits"].shape == z.shape
    assert torch.equal(rows(buf), want["dlogits"]) and buf[..., V:].isnan().all()
    assert torch.equal(out["loss"].view(-1), want["loss"]) and out["loss"].shape == lead
    z, buf = _padded(shape, pad)
    alone = swg.distill_bwd(flat[2], rows(_padded(shape, pad)[1]), flat[0], flat[1], want["stats"])
    got = swg.distill_bwd(w, z, ids, tl, want["stats"], dlogits=z)
    assert got.data_ptr() == buf.data_ptr()
    assert torch.equal(rows(buf), alone) and buf[..., V:].isnan().all()


def test_views_are_not_copied():
    swg = _swg()
    z, _ = _padded((2, 3, 100000), 96)
    t = torch.zeros((2, 3), dtype=torch.int64, device="cuda")
    dense = swg.token_logprobs_fwd(z.contiguous(), t, top_k=3)
    for view in (z, z[:, 1:2], z[1:], z[:1, :2]):
        out, extra = _copies(lambda: swg.token_logprobs_fwd(view, t[: view.shape[0], : view.shape[1]], top_k=3))
        assert extra < 100000
    out, extra = _copies(lambda: swg.token_logprobs_fwd(z, t, top_k=3))
    assert all(torch.equal(out[k], dense[k]) for k in dense)
    x, _ = _padded((4, 5, 4096), 64, seed=7)
    r, _ = _padded((4, 5, 4096), 64, seed=8)
    want = swg.layer_norm_fwd(x.contiguous(), residual=r.contiguous())
    out, extra = _copies(lambda: swg.layer_norm_fwd(x, residual=r))
    assert extra < 4096 and all(torch.equal(out[k], want[k]) for k in want)
    dy, _ = _padded((4, 5, 4096), 32, seed=9)
    got, wantb = swg.layer_norm_bwd(dy, x, want["stats"]), swg.layer_norm_bwd(dy.contiguous(), x.contiguous(), want["stats"])
    assert all(torch.equal(a, b) for a, b in zip(got, wantb))


def test_views_without_one_distance_are_copied():
    # rows at two distances, a shared row in one dimension only, elements apart
    swg = _swg()
    base = _rn(1, 4, 6, 96).bfloat16()
    for x in (base[:, :4], base[::2], base[:, :1].expand(4, 6, 96), base.transpose(0, 1), base[..., ::2],
              base[:1, :1].expand(4, 6, 96), base[:1].expand(4, 6, 96)):
        d = x.contiguous()
        t = torch.zeros(d.shape[:-1], dtype=torch.int64, device="cuda")
        a, b = swg.token_logprobs_fwd(x, t, top_k=2), swg.token_logprobs_fwd(d, t, top_k=2)
        assert all(torch.equal(a[k], b[k]) for k in a)
        a, b = swg.layer_norm_fwd(x, residual=d), swg.layer_norm_fwd(d, residual=x)
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_gradients_are_not_written_to_shared_or_scattered_rows():
    swg = _swg()
    z = _rn(1, 4, 6, 96)
    t = torch.zeros((4, 6), dtype=torch.int64, device="cuda")
    st = swg.token_logprobs_fwd(z, t)["stats"]
    dl = _rn(2, 4, 6)
    wide = torch.empty((4, 12, 96), device="cuda")
    for bad in (torch.empty((1, 6, 96), device="cuda").expand(4, 6, 96), wide[:, :6], torch.empty((4, 6, 192), device="cuda")[..., ::2],
                torch.empty((6, 4, 96), device="cuda").transpose(0, 1), torch.empty((4, 6, 97), device="cuda")):
        with pytest.raises(ValueError):
            swg.token_logprobs_bwd(dl, z, t, st, dlogits=bad)
