"""A transformer block's feed-forward half out of the library's calls, as they are used together: the norm and residual at
its junctions, SwiGLU, the down projection; its gradients against fp64 autograd on the same formulas, a captured
training step, and the answer for single tokens (GPU)."""

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _swg():
    import swiglu_ffn_backward_gb300 as swg
    return swg


def _params(cols, hidden, B, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return {"w_g": (rn(cols, hidden) / cols ** 0.5).to(BF16), "w_fc": (rn(cols, hidden) / cols ** 0.5).to(BF16),
            "w_out": (rn(hidden, cols) / hidden ** 0.5).to(BF16), "b_out": (0.1 * rn(cols)).to(BF16),
            "w_up": (rn(cols, hidden) / cols ** 0.5).to(BF16), "b_up": 0.1 * rn(hidden),
            "w_down": (rn(hidden, cols) / hidden ** 0.5).to(BF16),
            "g0": 1 + 0.1 * rn(cols), "g1": 1 + 0.1 * rn(cols), "g2": 1 + 0.1 * rn(cols), "g3": 1 + 0.1 * rn(cols),
            "gate": (1 + 0.3 * rn(B, 1, cols)).to(BF16)}


ALPHA = 0.9


def forward(swg, p, u, r, stream=None):
    """u [B, S, cols] (the block before), r its residual stream: y and what the backward needs. A junction with a gate for
    each sequence, a SwiGLU block, a junction without one, a GELU block whose projection adds the stream itself."""
    lead = u.shape[:-1]
    n1 = swg.block_norm_fwd(u, r, p["g0"], p["g1"], p["gate"], alpha=ALPHA, stream=stream)
    f = swg.swiglu_fwd(n1["y"].view(-1, u.shape[-1]), p["w_g"], p["w_fc"], stream=stream)
    down = swg.linear_fwd(f["y"].view(*lead, -1), p["w_out"], p["b_out"], stream=stream)["y"]
    n2 = swg.block_norm_fwd(down, n1["h"], p["g2"], p["g3"], stream=stream)
    up = swg.linear_fwd(n2["y"], p["w_up"], p["b_up"], act="gelu", save_z=True, stream=stream)
    y = swg.linear_fwd(up["y"], p["w_down"], residual=n2["h"], stream=stream)["y"]
    return y, (u, n1, f, down, n2, up)


def backward(swg, p, saved, dy):
    u, n1, f, down, n2, up = saved
    lead, flat = u.shape[:-1], lambda t: t.reshape(-1, t.shape[-1])
    b3 = swg.linear_bwd(dy, up["y"], p["w_down"], bias=False)
    b2 = swg.linear_bwd(b3["dx"], n2["y"], p["w_up"], z=up["z"], act="gelu", db_dtype=torch.float32)
    j2 = swg.block_norm_bwd(b2["dx"], dy, down, n2["h"], n2["stats"], gamma_post=p["g2"], gamma_pre=p["g3"])
    b1 = swg.linear_bwd(j2["du"], f["y"].view(*lead, -1), p["w_out"])
    ffn = swg.swiglu_bwd(flat(n1["y"]), p["w_g"], p["w_fc"], flat(b1["dx"]), f["g"], f["fc"], return_dg=False)
    j1 = swg.block_norm_bwd(ffn["dx"].view(u.shape), j2["dresidual"], u, n1["h"], n1["stats"], gamma_post=p["g0"],
                            gamma_pre=p["g1"], gate=p["gate"], alpha=ALPHA)
    return {"w_down": b3["dw"], "w_up": b2["dw"], "b_up": b2["db"], "g2": j2["dgamma_post"], "g3": j2["dgamma_pre"],
            "w_out": b1["dw"], "b_out": b1["db"], "w_g": ffn["dw_g"], "w_fc": ffn["dw_fc"], "g0": j1["dgamma_post"],
            "g1": j1["dgamma_pre"], "gate": j1["dgate"], "u": j1["du"], "r": j1["dresidual"]}


def _exact(p, u, r, dy=None):
    q = {k: v.double().requires_grad_() for k, v in {**p, "u": u, "r": r}.items()}
    norm = lambda t, g: t * torch.rsqrt(t.square().mean(dim=-1, keepdim=True) + 1e-6) * g  # noqa: E731
    h = ALPHA * q["r"] + q["gate"] * norm(q["u"], q["g0"])
    x = norm(h, q["g1"])
    down = (torch.nn.functional.silu(x @ q["w_g"]) * (x @ q["w_fc"])) @ q["w_out"] + q["b_out"]
    h = h + norm(down, q["g2"])
    y = torch.nn.functional.gelu(norm(h, q["g3"]) @ q["w_up"] + q["b_up"]) @ q["w_down"] + h
    if dy is not None:
        y.backward(dy.double())
    return y.detach(), {k: v.grad for k, v in q.items()}


def _inputs(B, S, cols, seed=3):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [torch.randn((B, S, cols), generator=g, device="cuda").to(BF16) for _ in range(3)]


def _rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("B,S,cols,hidden", [(2, 3, 64, 128), (3, 130, 136, 264), (4, 1000, 512, 1024)])
def test_training_step(B, S, cols, hidden):
    swg = _swg()
    p, (u, r, dy) = _params(cols, hidden, B), _inputs(B, S, cols)
    want, grads = _exact(p, u, r, dy)
    y, saved = forward(swg, p, u, r)
    got = backward(swg, p, saved, dy)
    swg.swg_check()
    # some fifteen tensors on the way are rounded to bf16, at most 2^-8 relative each: in the norm below 15 2^-8 < 2^-4
    assert _rel(y, want) <= 2.0 ** -4
    assert set(got) == set(grads)
    for k, v in grads.items():
        assert got[k].shape == v.shape and _rel(got[k], v) <= 2.0 ** -4, k


def test_captured_step_beside_an_eager_one():
    # a captured forward and backward, replayed on new inputs, with an eager step between the replays
    swg = _swg()
    B, S, cols, hidden = 2, 70, 136, 264
    p, (u, r, dy) = _params(cols, hidden, B), _inputs(B, S, cols)
    backward(swg, p, forward(swg, p, u, r)[1], dy)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, saved = forward(swg, p, u, r)
        got = backward(swg, p, saved, dy)
    for seed in (5, 6):
        for t, v in zip((u, r, dy), _inputs(B, S, cols, seed)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        ey, esaved = forward(swg, p, u, r)
        want = backward(swg, p, esaved, dy)
        assert torch.equal(y, ey) and all(torch.equal(got[k], want[k]) for k in want)


def test_two_streams_at_once():
    # the same calls on two streams, each with its own memory, give what one stream gives
    swg = _swg()
    B, S, cols, hidden = 2, 500, 512, 1024
    p = _params(cols, hidden, B)
    sets = [_inputs(B, S, cols, seed) for seed in (7, 8)]
    want = [forward(swg, p, u, r)[0] for u, r, _ in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = [forward(swg, p, u, r, stream=s)[0] for (u, r, _), s in zip(sets, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_single_tokens_match_the_batch():
    # each token alone: other kernels, the same function (every tensor on the way rounds differently at ties only)
    swg = _swg()
    B, S, cols, hidden = 1, 5, 512, 1024
    p, (u, r, _) = _params(cols, hidden, B), _inputs(B, S, cols)
    want, _ = _exact(p, u, r)
    for i in range(S):
        y = forward(swg, p, u[:, i:i + 1], r[:, i:i + 1])[0]
        assert _rel(y, want[:, i:i + 1]) <= 2.0 ** -4
