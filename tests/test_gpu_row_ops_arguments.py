"""Shapes of the row-wise operators' tensors: what a call takes, and what it refuses because the elements would
be read in another order than the caller's (GPU: the binding looks at CUDA tensors only)."""

import pytest
import torch

pytestmark = pytest.mark.gpu
B, S, V, K = 3, 5, 70, 4


def _swg():
    import swiglu_ffn_backward_gb300 as swg
    return swg


def _data():
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    t = dict(z=rn(B, S, V), dl=rn(B, S), de=rn(B, S), w=rn(B, S), tl=rn(B, S, K), x=rn(B, S, 16), dy=rn(B, S, 16))
    t["t"] = torch.randint(0, V, (B, S), generator=g, device="cuda")
    t["ids"] = torch.rand((B, S, V), generator=g, device="cuda").topk(K, dim=-1).indices
    swg = _swg()
    t["lp"] = swg.token_logprobs_fwd(t["z"], t["t"])
    t["kd"] = swg.distill_fwd(t["z"], t["ids"], t["tl"])
    t["ln"] = swg.layer_norm_fwd(t["x"])
    return swg, t


def _turned(a):
    """a's elements in a dense tensor whose first two dimensions are exchanged."""
    return a.transpose(0, 1).contiguous()


def test_tensors_of_another_order_are_refused():
    swg, t = _data()
    e, st = t["lp"]["entropy"], t["lp"]["stats"]
    flat = lambda a: a.reshape(B * S, *a.shape[2:])  # noqa: E731
    z2, ids2, tl2 = flat(t["z"]), flat(t["ids"]), flat(t["tl"])
    out = lambda name, a: {name: torch.empty_like(a)}  # noqa: E731
    calls = {
        "targets": lambda: swg.token_logprobs_fwd(t["z"], _turned(t["t"])),
        "targets of the gradient": lambda: swg.token_logprobs_bwd(t["dl"], t["z"], _turned(t["t"]), st),
        "dlogp": lambda: swg.token_logprobs_bwd(_turned(t["dl"]), t["z"], t["t"], st),
        "dentropy": lambda: swg.token_logprobs_bwd(t["dl"], t["z"], t["t"], st, dentropy=_turned(t["de"]), entropy=e),
        "entropy": lambda: swg.token_logprobs_bwd(t["dl"], t["z"], t["t"], st, dentropy=t["de"], entropy=_turned(e)),
        "stats": lambda: swg.token_logprobs_bwd(t["dl"], t["z"], t["t"], _turned(st)),
        "teacher_logits": lambda: swg.distill_fwd(z2, ids2, _turned(tl2)),
        "teacher_logits of three dimensions": lambda: swg.distill_fwd(t["z"], t["ids"], _turned(t["tl"])),
        "weight": lambda: swg.distill_fwd_bwd(t["z"], t["ids"], t["tl"], _turned(t["w"])),
        "weight of the gradient": lambda: swg.distill_bwd(_turned(t["w"]), t["z"], t["ids"], t["tl"], t["kd"]["stats"]),
        "stats of the gradient": lambda: swg.distill_bwd(t["w"], t["z"], t["ids"], t["tl"], _turned(t["kd"]["stats"])),
        "layer norm's stats": lambda: swg.layer_norm_bwd(t["dy"], t["x"], _turned(t["ln"]["stats"])),
        "logp as output": lambda: swg.token_logprobs_fwd(t["z"], t["t"], out=out("logp", _turned(t["t"]).float())),
        "top_idx as output": lambda: swg.token_logprobs_fwd(
            t["z"], top_k=K, out={"top_idx": torch.empty((B, K, S), dtype=torch.int64, device="cuda")}),
        "loss as output": lambda: swg.distill_fwd(t["z"], t["ids"], t["tl"], out=out("loss", _turned(t["w"]))),
        "stats as output": lambda: swg.layer_norm_fwd(t["x"], out=out("stats", _turned(t["ln"]["stats"]))),
        "y as output": lambda: swg.layer_norm_fwd(t["x"], out=out("y", _turned(t["x"]))),
        "dx": lambda: swg.layer_norm_bwd(t["dy"], t["x"], t["ln"]["stats"], dx=torch.empty_like(_turned(t["x"]))),
    }
    taken = []
    for name, call in calls.items():
        try:
            call()
            taken.append(name)
        except ValueError:
            pass
    assert not taken


def test_tensors_of_the_same_order_are_taken():
    # rows in one dimension or in the logits' own, dimensions of one anywhere, everything in one dimension
    swg, t = _data()
    n = B * S
    st, e = t["lp"]["stats"], t["lp"]["entropy"]
    want = swg.token_logprobs_bwd(t["dl"], t["z"], t["t"], st, dentropy=t["de"], entropy=e)
    forms = (lambda a: a.reshape(n), lambda a: a.reshape(B, S, 1), lambda a: a.reshape(1, B, S), lambda a: a.reshape(n, 1))
    for f in forms:
        assert torch.equal(swg.token_logprobs_fwd(t["z"], f(t["t"]))["logp"], t["lp"]["logp"])
        for z in (t["z"], t["z"].reshape(n, V)):
            for s in (st, st.view(B, S, 2), st.view(-1)):
                got = swg.token_logprobs_bwd(f(t["dl"]), z, f(t["t"]), s, dentropy=f(t["de"]), entropy=f(e))
                assert torch.equal(got.view_as(want), want)
    # rows counted in one dimension beside tensors in two
    z2 = t["z"].reshape(n, V)
    assert torch.equal(swg.token_logprobs_fwd(z2, t["t"])["logp"].view(B, S), t["lp"]["logp"])
    want = swg.distill_fwd_bwd(t["z"], t["ids"], t["tl"], t["w"])
    for tl in (t["tl"], t["tl"].view(n, K), t["tl"].view(B, S, 1, K), t["tl"].view(-1)):
        for w in [f(t["w"]) for f in forms]:
            got = swg.distill_fwd_bwd(t["z"], t["ids"], tl, w)
            assert all(torch.equal(got[k], want[k]) for k in want)
    got = swg.distill_fwd_bwd(z2, t["ids"].view(n, K), t["tl"], t["w"])
    assert torch.equal(got["dlogits"].view_as(t["z"]), want["dlogits"])
    wantb = swg.layer_norm_bwd(t["dy"], t["x"], t["ln"]["stats"])
    got = swg.layer_norm_bwd(t["dy"], t["x"], t["ln"]["stats"].view(B, S, 2), dx=torch.empty((n, 16), device="cuda"))
    assert torch.equal(got[0].view(B, S, 16), wantb[0])
    # the weights of a norm over several dimensions taken as one
    gam = 1 + torch.rand(4, 4, device="cuda")
    assert torch.equal(swg.layer_norm_fwd(t["x"], gam)["y"], swg.layer_norm_fwd(t["x"], gam.view(16))["y"])
