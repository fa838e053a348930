"""Log probabilities of given tokens, entropy, top alternatives and their gradient against the
fp64 oracle (GPU)."""

import numpy as np
import pytest
import torch

import oracle

from ._guard import check_all, guarded
from ._row_ops import DTYPES, EXP, LAYOUTS, NAME, SUM, check, f64, strided

pytestmark = pytest.mark.gpu


def _swg():
    import swiglu_ffn_backward_gb300 as swg
    return swg


def _inputs(T, V, dtype, seed, masked=False, scale=3.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    z = (torch.randn((T, V), generator=g, device="cuda") * scale).to(dtype)
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    if masked:
        r = torch.arange(T, device="cuda")
        drop = torch.rand((T, V), generator=g, device="cuda") > 0.1
        z.masked_fill_(drop & (r % 3 == 0).unsqueeze(1), float("-inf"))
        z[r % 5 == 1, V // 2:] = torch.finfo(dtype).min
        z[r % 7 == 2] = float("-inf")
        z[r % 7 == 3] = torch.finfo(dtype).min  # every logit the lowest value: a uniform distribution
        z[r % 11 == 4, : V - 1] = float("-inf")  # one token left
        t[r % 6 == 5] = -100
    return z, t, torch.randn(T, generator=g, device="cuda"), torch.randn(T, generator=g, device="cuda")


def _errors(z, tau):
    """Per row: s, |d| (0 where masked), the expected |d| and the relative error of s."""
    m, s, lp, p = oracle.row_softmax(z, tau)
    with np.errstate(invalid="ignore"):
        d = np.where(np.isneginf(z) | np.isnan(z), 0.0, np.abs(z - np.where(np.isfinite(m), m, 0.0)[:, None]) / tau)
        ed = np.nansum(np.where(p > 0, p * d, 0.0), axis=1)
    return s, lp, p, d, ed, SUM + EXP + 2.0 ** -22 * ed


def _check_fwd(z, t, out, k, tau, ignore=-100):
    z = f64(z)
    ref = oracle.token_logprobs_fwd(z, None if t is None else t.cpu().numpy(), k, tau, ignore)
    s, lp, p, d, ed, serr = _errors(z, tau)
    ls = np.abs(np.log(np.where(s > 0, s, 1.0)))
    f32 = torch.float32
    check("max", out["stats"][:, 0], ref["stats"][:, 0], f32, 0.0)
    check("sum", out["stats"][:, 1], ref["stats"][:, 1], f32, np.nan_to_num(serr * s))
    check("entropy", out["entropy"], ref["entropy"], f32, np.nan_to_num(2 * serr * (1 + ed) + 2.0 ** -22 * (ls + ed)))
    base = np.nan_to_num(serr + 2.0 ** -22 * ls)
    if t is not None:
        at = np.clip(t.cpu().numpy(), 0, z.shape[1] - 1)
        check("logp", out["logp"], _f32_range(ref["logp"]), f32, base + 2.0 ** -22 * d[np.arange(len(at)), at])
    if k:
        np.testing.assert_array_equal(out["top_idx"].cpu().numpy().reshape(-1, k), ref["top_idx"])
        dk = np.take_along_axis(d, ref["top_idx"], axis=1)
        check("top_logp", out["top_logp"], _f32_range(ref["top_logp"]), f32, base[:, None] + 2.0 ** -22 * dk)


def _f32_range(v):
    """fp64 values as fp32 stores them: below its range they are -inf."""
    with np.errstate(over="ignore"):
        return np.where(np.isfinite(np.asarray(v, np.float32)), v, np.asarray(v, np.float32).astype(np.float64))


def _check_bwd(z, t, dl, de, got, dtype, tau):
    zz, dl = f64(z), f64(dl)
    de = None if de is None else f64(de)
    tt = None if t is None else t.cpu().numpy()
    ref = oracle.token_logprobs_bwd(zz, tt, tau, dlogp=dl, dentropy=de)
    s, lp, p, d, ed, serr = _errors(zz, tau)
    perr = serr[:, None] + EXP + 2.0 ** -22 * d + 2.0 ** -21
    part = np.abs(dl)[:, None] * (p * perr)
    if de is not None:
        size = np.where(p > 0, np.abs(np.where(p > 0, lp, 0.0)), 0.0) + ed[:, None] + np.abs(np.log(np.where(s > 0, s, 1)))[:, None]
        part = part + np.abs(de)[:, None] * p * (size * (perr + 2.0 ** -21) + 2 * serr[:, None])
    if tt is not None:
        hit = np.zeros_like(zz)
        hit[np.arange(len(tt)), np.clip(tt, 0, zz.shape[1] - 1)] = np.abs(dl)
        part = part + 2.0 ** -22 * hit
    check("dlogits", got, ref, dtype, np.nan_to_num(part / tau))


def _run(T, V, dtype, k=0, tau=1.0, masked=False, layout="dense", seed=1, index=torch.int64, entropy=True):
    swg = _swg()
    z, t, dl, de = _inputs(T, V, dtype, seed, masked)
    zl, t = strided(z, layout), t.to(index)
    out = swg.token_logprobs_fwd(zl, t, top_k=min(k, V), temperature=tau)
    _check_fwd(z, t, out, min(k, V), tau)
    de = de if entropy else None
    got = swg.token_logprobs_bwd(dl, zl, t, out["stats"], dentropy=de, entropy=out["entropy"] if entropy else None,
                                 temperature=tau)
    _check_bwd(z, t, dl, de, got, dtype, tau)


SHAPES = [(1, 1), (3, 2), (2, 7), (5, 33), (4, 256), (7, 1000), (3, 4097), (40, 8192), (2, 32768), (3, 50001),
          (1, 131072), (2, 160001), (1, 300007), (400, 515), (700, 2048)]


@pytest.mark.parametrize("dtype", DTYPES, ids=NAME.get)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes(shape, dtype):
    _run(*shape, dtype, k=20)
    _run(*shape, dtype, k=32, tau=0.7, masked=True, index=torch.int32, seed=2)


# more rows than there are blocks on the device, so that each takes several: blocks of few and of many warps
MANY = [(3001, 2048, torch.bfloat16), (1501, 8191, torch.float32), (1001, 32768, torch.float16),
        (951, 40001, torch.bfloat16), (501, 50001, torch.float16), (401, 100000, torch.bfloat16)]


@pytest.mark.parametrize("shape", MANY, ids=lambda s: "x".join(map(str, s[:2])) + "-" + NAME[s[2]])
def test_many_rows(shape):
    _run(*shape, k=20, tau=0.7, masked=True, seed=21)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", DTYPES, ids=NAME.get)
def test_layouts(dtype, layout):
    for V in (64, 1001, 9000, 40007):
        _run(13, V, dtype, k=3, tau=2.0, masked=True, layout=layout, entropy=False)


@pytest.mark.parametrize("k", [1, 2, 5, 31, 32])
def test_top_k_with_many_ties(k):
    # a handful of distinct values: the order among equal logits is the index's
    swg = _swg()
    g = torch.Generator(device="cuda")
    g.manual_seed(k)
    for T, V in ((6, 40), (5, 3000), (3, 70001), (2, 200000)):
        z = torch.randint(-2, 3, (T, V), generator=g, device="cuda").to(torch.bfloat16)
        z[0] = 1.5
        z[1] = torch.where(z[1] == 0, -0.0, z[1])  # -0 and +0 are equal
        z[1] = torch.where((z[1] == 0) & (torch.arange(V, device="cuda") % 2 == 0), 0.0, z[1].float()).to(z.dtype)
        _check_fwd(z, None, swg.token_logprobs_fwd(z, top_k=k), k, 1.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=NAME.get)
def test_top_k_of_ordered_and_clustered_rows(dtype):
    # the best logits side by side, in one lane's share, at either end, or the whole row in order
    swg = _swg()
    V = 65536 + 24
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    z = torch.randn((8, V), generator=g, device="cuda")
    ramp = torch.arange(V, device="cuda", dtype=torch.float32) / V
    z[0], z[1] = ramp, -ramp
    z[2, 1000:1064] += 50
    z[3, torch.arange(0, V, 2048, device="cuda")] += 50     # far apart, one thread's share
    z[4, :40] += 50
    z[5, -40:] += 50
    z[6, torch.arange(0, V, 8, device="cuda")] += 50        # thousands of good ones, regularly
    z[7, : V // 4] += 50
    _check_fwd(z.to(dtype), None, swg.token_logprobs_fwd(z.to(dtype), top_k=32), 32, 1.0)


def test_nan_and_inf():
    swg = _swg()
    for V in (37, 3000, 100001):
        z, t, dl, de = _inputs(6, V, torch.float32, 4)
        z[1, V // 2], z[2, 0], z[3, V - 1] = float("nan"), float("inf"), float("nan")
        z[3, : V - 1] = float("-inf")
        out = swg.token_logprobs_fwd(z, t, top_k=3)
        g = swg.token_logprobs_bwd(dl, z, t, out["stats"], dentropy=de, entropy=out["entropy"])
        for r in (1, 2, 3):
            assert out["logp"][r].isnan() and out["entropy"][r].isnan() and g[r].isnan().all()
            assert out["top_logp"][r].isnan().any()
        assert out["top_idx"][2, 0] == 0 and out["top_idx"][3].tolist() == [0, 1, 2]
        order = torch.where(z[1].isnan(), float("-inf"), z[1]).topk(3).indices
        assert out["top_idx"][1].tolist() == order.tolist()
        fine = [0, 4, 5]
        sub = {k: v[fine] for k, v in out.items()}
        _check_fwd(z[fine], t[fine], sub, 3, 1.0)
        _check_bwd(z[fine], t[fine], dl[fine], de[fine], g[fine], torch.float32, 1.0)


def test_targets_ignored_absent_and_outside():
    swg = _swg()
    z, t, dl, _ = _inputs(5, 600, torch.float16, 5)
    t[0], t[1], t[2] = 7, 600, -1
    out = swg.token_logprobs_fwd(z, t, ignore_index=7)
    assert out["logp"][0] == 0 and out["logp"][1].isnan() and out["logp"][2].isnan()
    g = swg.token_logprobs_bwd(dl, z, t, out["stats"], ignore_index=7)
    assert not g[0].any() and g[1].isnan().all() and g[2].isnan().all()
    _check_bwd(z[3:], t[3:], dl[3:], None, g[3:], torch.float16, 1.0)
    out = swg.token_logprobs_fwd(z)
    assert set(out) == {"entropy", "stats"}
    # the entropy's gradient alone
    de = torch.randn(5, device="cuda")
    g = swg.token_logprobs_bwd(None, z, None, out["stats"], dentropy=de, entropy=out["entropy"])
    _check_bwd(z, None, torch.zeros(5), de, g, torch.float16, 1.0)


def test_gradient_by_differences():
    swg = _swg()
    z, t, dl, de = _inputs(4, 40, torch.float32, 6, scale=1.0)
    f = lambda z: float((lambda o: (o["logp"].double() * dl + o["entropy"].double() * de).sum())(  # noqa: E731
        swg.token_logprobs_fwd(z, t, temperature=0.8)))
    out = swg.token_logprobs_fwd(z, t, temperature=0.8)
    g = swg.token_logprobs_bwd(dl, z, t, out["stats"], dentropy=de, entropy=out["entropy"], temperature=0.8)
    e = 2.0 ** -7
    for seed in range(3):
        v = torch.sign(torch.randn(z.shape, generator=torch.Generator().manual_seed(seed))).cuda()
        diff = (f(z + e * v) - f(z - e * v)) / (2 * e)
        # truncation e^2 / 6 times third derivatives of order 10 a row, and the forward's fp32 error over e
        assert abs(diff - float((g.double() * v).sum())) <= 4 * 10 * e * e + 8 * 2.0 ** -20 / e


def test_in_place_and_guarded():
    swg = _swg()
    for V, dtype in ((4096, torch.bfloat16), (30001, torch.float16), (999, torch.float32), (140000, torch.bfloat16)):
        z, t, dl, de = _inputs(9, V, dtype, 7)
        gs = dict(logp=guarded((9,), torch.float32), entropy=guarded((9,), torch.float32),
                  stats=guarded((9, 2), torch.float32), top_logp=guarded((9, 5), torch.float32),
                  top_idx=guarded((9, 5), torch.int64), dlogits=guarded((9, V), dtype))
        out = swg.token_logprobs_fwd(z, t, top_k=5, out={k: v.t for k, v in gs.items() if k != "dlogits"})
        args = dict(dentropy=de, entropy=out["entropy"])
        got = swg.token_logprobs_bwd(dl, z, t, out["stats"], dlogits=gs["dlogits"].t, **args)
        torch.cuda.synchronize()
        check_all(gs)
        _check_fwd(z, t, out, 5, 1.0)
        _check_bwd(z, t, dl, de, got, dtype, 1.0)
        zi = strided(z, "padded")
        same = swg.token_logprobs_bwd(dl, zi, t, out["stats"], dlogits=zi, **args)
        assert same.data_ptr() == zi.data_ptr() and torch.equal(same, got)
        # another alignment for the output than for the logits
        shifted = strided(torch.zeros_like(z), "shifted")
        assert torch.equal(swg.token_logprobs_bwd(dl, z, t, out["stats"], dlogits=shifted, **args), got)


def test_shared_row_and_leading_dimensions():
    swg = _swg()
    z, t, _, _ = _inputs(1, 5000, torch.bfloat16, 8)
    t = torch.tensor([0, 5, 4999, 17], device="cuda")
    out = swg.token_logprobs_fwd(z.expand(4, 5000), t, top_k=4)
    _check_fwd(z.expand(4, 5000), t, out, 4, 1.0)
    zz = z.expand(4, 5000).contiguous().view(2, 2, 5000)
    o2 = swg.token_logprobs_fwd(zz, t.view(2, 2), top_k=4)
    assert o2["logp"].shape == (2, 2) and o2["top_idx"].shape == (2, 2, 4)
    assert torch.equal(o2["logp"].view(-1), out["logp"])


def test_offsets_past_32_bits():
    swg = _swg()
    T, V = 33000, 65544
    z = torch.empty((T, V), dtype=torch.bfloat16, device="cuda").normal_(0, 3, generator=torch.Generator("cuda").manual_seed(1))
    assert z.numel() > 2 ** 31
    t = torch.arange(T, device="cuda") % V
    out = swg.token_logprobs_fwd(z, t, top_k=2)
    dl = torch.ones(T, device="cuda")
    rows = [0, 32763, 32764, T - 1]
    sub = {k: v[rows] for k, v in out.items()}
    zr = z[rows].clone()
    _check_fwd(zr, t[rows], sub, 2, 1.0)
    g = swg.token_logprobs_bwd(dl, z, t, out["stats"], dlogits=z)
    _check_bwd(zr, t[rows], dl[rows], None, g[rows], torch.bfloat16, 1.0)


def test_reproducible_on_another_stream():
    swg = _swg()
    z, t, dl, de = _inputs(300, 20011, torch.bfloat16, 9)
    a = swg.token_logprobs_fwd(z, t, top_k=8)
    ga = swg.token_logprobs_bwd(dl, z, t, a["stats"], dentropy=de, entropy=a["entropy"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = swg.token_logprobs_fwd(z, t, top_k=8, stream=s)
    gb = swg.token_logprobs_bwd(dl, z, t, b["stats"], dentropy=de, entropy=b["entropy"], stream=s)
    s.synchronize()
    assert all(torch.equal(a[k], b[k]) for k in a) and torch.equal(ga, gb)


def test_empty_and_refusals():
    swg = _swg()
    z = torch.zeros((0, 50), device="cuda")
    out = swg.token_logprobs_fwd(z, torch.zeros(0, dtype=torch.int64, device="cuda"), top_k=3)
    assert out["top_idx"].shape == (0, 3) and out["logp"].shape == (0,)
    z, t, dl, _ = _inputs(4, 50, torch.bfloat16, 1)
    with pytest.raises(swg.SwgError):
        swg.token_logprobs_fwd(z, t, top_k=33)
    with pytest.raises(swg.SwgError):
        swg.token_logprobs_fwd(z[:, :4], t, top_k=5)
    for tau in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(swg.SwgError):
            swg.token_logprobs_fwd(z, t, temperature=tau)
    with pytest.raises(ValueError):
        swg.token_logprobs_fwd(z, t[:3])
    with pytest.raises(ValueError):
        swg.token_logprobs_fwd(z, t.float())
    with pytest.raises(TypeError):
        swg.token_logprobs_fwd(z.double(), t)
    stats = torch.zeros((4, 2), device="cuda")
    with pytest.raises(ValueError):
        swg.token_logprobs_bwd(dl, z, t, stats, dlogits=torch.empty((4, 49), dtype=z.dtype, device="cuda"))
    with pytest.raises(swg.SwgError):  # the gradient over part of the logits
        swg.token_logprobs_bwd(dl, z[:, :40], t, stats, dlogits=z[:, 5:45])
    with pytest.raises(swg.SwgError):  # targets without dlogp
        swg.token_logprobs_bwd(None, z, t, stats)
    with pytest.raises(swg.SwgError):  # dentropy without the entropy
        swg.token_logprobs_bwd(dl, z, t, stats, dentropy=dl)
