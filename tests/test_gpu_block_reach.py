"""The linear layer and the norms between blocks where offsets pass 32 bits, and with values that are not finite (GPU).
Behind 2^31 elements only the last rows hold a gradient, so that they alone make the sums over the rows."""

import pytest
import torch

from ._block import ACTS, check_linear_bwd, check_linear_fwd, check_norm_bwd, check_norm_fwd, linear_inputs, norm_inputs

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _swg():
    import swiglu_ffn_backward_gb300 as swg
    return swg


def _behind(tail, M, fill=None):
    """[M, n] whose last rows are `tail`, the others zeros or copies of one row."""
    t = torch.zeros(M, tail.shape[1], dtype=tail.dtype, device="cuda")
    if fill is not None:
        t[:] = fill
    t[-tail.shape[0]:] = tail
    return t


def test_linear_far_rows():
    swg, M, last = _swg(), 270001, 100
    t = linear_inputs(last, 64, 8192, BF16, seed=61)
    x = _behind(t["x"], M, t["x"][0])
    out = swg.linear_fwd(x, t["w"], t["b"], act="gelu", save_z=True)
    check_linear_fwd(t, {k: v[-last:] for k, v in out.items()}, BF16, "gelu", t["b"])
    assert torch.equal(out["y"][0], out["y"][M // 2])
    z, dy = out["z"], _behind(t["dy"], M)
    t["z"] = z[-last:].clone()
    del out
    got = swg.linear_bwd(dy, x, t["w"], z=z, act="gelu")
    assert not got["dx"][:-last].any()
    got["dx"] = got["dx"][-last:]
    check_linear_bwd(t, got, BF16, "gelu")
    swg.swg_check()


@pytest.mark.parametrize("gates", [0, 2])
def test_norm_far_rows(gates):
    swg, M, N, last = _swg(), 540002, 4096, 64
    t = norm_inputs(last, N, BF16, F32, 1 if gates else 0, F32)
    gate = None if not gates else torch.cat([torch.full_like(t["gate"], 0.5)] * (gates - 1) + [t["gate"]])
    u, r = _behind(t["u"], M, t["u"][0]), _behind(t["residual"], M, t["residual"][0])
    kw = dict(gamma_post=t["gamma_post"], gamma_pre=t["gamma_pre"], gate=gate)
    out = swg.block_norm_fwd(u, r, **kw)
    check_norm_fwd(t, {k: v[-last:] for k, v in out.items()}, BF16)
    assert torch.equal(out["y"][0], out["y"][M // 2 - 1])
    del r, out["y"]
    got = swg.block_norm_bwd(_behind(t["dy"], M), _behind(t["dh"], M), u, out["h"], out["stats"], **kw)
    for k in ("du", "dresidual"):
        assert not got[k][:-last].any()
        got[k] = got[k][-last:]
    if gates:
        assert not got["dgate"][0].any()
        got["dgate"] = got["dgate"][1:]
    check_norm_bwd(t, out["h"][-last:], out["stats"][-last:], got, BF16, F32, F32)
    swg.swg_check()


# results of the kernel for few rows and of the one on CTA pairs
@pytest.mark.parametrize("M,K,N", [(5, 64, 136), (3000, 64, 1032)])
@pytest.mark.parametrize("act", ACTS)
def test_linear_not_finite(M, K, N, act):
    swg, t = _swg(), linear_inputs(M, K, N, BF16, seed=63)
    b = t["b"].float()
    b[3], b[N - 2] = float("inf"), float("nan")
    x = t["x"].clone()
    x[M - 2] = float("nan")
    y = swg.linear_fwd(x, t["w"], b, act=act)["y"]
    want = swg.linear_fwd(t["x"], t["w"], t["b"].float(), act=act)["y"]
    rows = torch.arange(M, device="cuda") != M - 2
    cols = torch.ones(N, dtype=torch.bool, device="cuda")
    cols[3] = cols[N - 2] = False
    assert torch.equal(y[rows][:, cols], want[rows][:, cols])
    assert torch.isposinf(y[rows, 3]).all()
    assert torch.isnan(y[rows, N - 2]).all() and torch.isnan(y[M - 2]).all()


@pytest.mark.parametrize("M,N", [(6, 1001), (2000, 4096), (600, 4001)])
def test_norm_not_finite(M, N):
    # a row of NaN or infinity leaves the other rows as they are
    swg, t = _swg(), norm_inputs(M, N, BF16, F32, 0)
    args = dict(gamma_post=t["gamma_post"], gamma_pre=t["gamma_pre"])
    bad = {k: t[k].clone() for k in ("u", "residual")}
    bad["u"][1, 5], bad["residual"][M - 2, N - 1] = float("nan"), float("inf")
    rows = torch.ones(M, dtype=torch.bool, device="cuda")
    rows[1] = rows[M - 2] = False
    a, c = (swg.block_norm_fwd(v["u"], v["residual"], **args) for v in (t, bad))
    for k in ("h", "y"):
        assert torch.equal(a[k][rows], c[k][rows])
    assert torch.isnan(c["y"][1]).all() and torch.isnan(c["y"][M - 2, N - 1])
    ga, gc = (swg.block_norm_bwd(t["dy"], t["dh"], v["u"], o["h"], o["stats"], params=False, **args)
              for v, o in ((t, a), (bad, c)))
    for k in ("du", "dresidual"):
        assert torch.equal(ga[k][rows], gc[k][rows])
    assert torch.isnan(gc["du"][1]).all()
    swg.swg_check()
