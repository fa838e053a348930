"""Layer norm forward and backward against the fp64 oracle (GPU)."""

import numpy as np
import pytest
import torch

import oracle

from ._guard import check_all, guarded, workspace
from ._row_ops import DTYPES, LAYOUTS, NAME, SUM, check, f64, strided

pytestmark = pytest.mark.gpu
EPS = 1e-5


def _swg():
    import swiglu_ffn_backward_gb300 as swg
    return swg


def _inputs(M, N, dtype, wdtype, seed, shift=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = (rn(M, N) * (0.5 + torch.rand((M, 1), generator=g, device="cuda")) + shift * rn(M, 1)).to(dtype)
    return dict(x=x, residual=rn(M, N).to(dtype), dy=rn(M, N).to(dtype), dh=rn(M, N).to(dtype),
                gamma=(1 + 0.3 * rn(N)).to(wdtype), beta=(0.2 * rn(N)).to(wdtype))


def _check_fwd(t, out, dtype, gamma=True, beta=True, residual=False, eps=EPS):
    ga, be = (t["gamma"] if gamma else None), (t["beta"] if beta else None)
    y, mu, rstd, h = oracle.layer_norm_fwd(f64(t["x"]), None if ga is None else f64(ga), None if be is None else f64(be),
                                           eps, f64(t["residual"]) if residual else None, NAME[dtype])
    if residual:
        np.testing.assert_array_equal(f64(out["h"]), h)
    top = np.abs(h).max(axis=1)
    stats = f64(out["stats"])
    check("mean", out["stats"][:, 0], mu, torch.float32, SUM * top)
    # rstd: relative error half of the variance's; the mean's error enters squared, and as 2^-24 of h
    var_err = 2 * SUM + (SUM * top * rstd) ** 2 + 2.0 ** -22 * top * rstd
    check("rstd", out["stats"][:, 1], rstd, torch.float32, rstd * var_err)
    xhat = (h - mu[:, None]) * rstd[:, None]
    g = np.ones(h.shape[1]) if ga is None else np.abs(f64(ga))
    part = g * ((SUM * top * rstd)[:, None] + np.abs(xhat) * (var_err[:, None] + 2.0 ** -22)) + 2.0 ** -23 * np.abs(y)
    if be is not None:
        part = part + 2.0 ** -23 * np.abs(f64(be))
    check("y", out["y"], y, dtype, part)
    return stats


def _check_bwd(t, h, stats, got, dtype, wdtype, gamma=True, dh=False):
    dx, dgamma, dbeta = got
    h, dy, st = f64(h), f64(t["dy"]), f64(stats)
    ga = f64(t["gamma"]) if gamma else None
    rdx, rdg, rdb = oracle.layer_norm_bwd(dy, h, st[:, 0], st[:, 1], ga, f64(t["dh"]) if dh else None)
    g = np.abs(dy if ga is None else dy * ga)
    xhat = np.abs((h - st[:, :1]) * st[:, 1:])
    xerr = 2.0 ** -23 * (np.abs(h) + np.abs(st[:, :1])) * st[:, 1:]  # of x_hat, from its difference
    mg, mgx = g.mean(axis=1, keepdims=True), (g * (xhat + xerr)).mean(axis=1, keepdims=True)
    part = st[:, 1:] * (2.0 ** -22 * g + SUM * mg + (SUM + 2.0 ** -22) * (xhat + xerr) * mgx + xerr * mgx
                        + xhat * (g * xerr).mean(axis=1, keepdims=True)) + 2.0 ** -23 * np.abs(rdx)
    if dh:
        part = part + 2.0 ** -23 * np.abs(f64(t["dh"]))
    check("dx", dx, rdx, dtype, part)
    if dgamma is not None:
        check("dgamma", dgamma, rdg, wdtype, (np.abs(dy) * (SUM * xhat + 2 * xerr)).sum(axis=0))
        check("dbeta", dbeta, rdb, wdtype, SUM * np.abs(dy).sum(axis=0))


def _run(M, N, dtype, wdtype, seed=3, layout="dense", gamma=True, beta=True, residual=False, dh=False, params=True):
    swg = _swg()
    t = _inputs(M, N, dtype, wdtype, seed)
    lay = {k: strided(t[k], layout) for k in ("x", "residual", "dy", "dh")}
    out = swg.layer_norm_fwd(lay["x"], t["gamma"] if gamma else None, t["beta"] if beta else None, eps=EPS,
                             residual=lay["residual"] if residual else None)
    assert ("h" in out) == residual
    _check_fwd(t, out, dtype, gamma, beta, residual)
    h = out["h"] if residual else lay["x"]
    got = swg.layer_norm_bwd(lay["dy"], h, out["stats"], gamma=t["gamma"] if gamma else None,
                             dh=lay["dh"] if dh else None, params=params)
    assert (got[1] is None) == (not params)
    _check_bwd(t, h, out["stats"], got, dtype, wdtype if gamma else dtype, gamma, dh)


SHAPES = [(1, 1), (3, 2), (1, 4096), (2, 7), (33, 100), (5, 1001), (257, 64), (300, 512), (19, 1024), (65, 2048),
          (7, 5000), (6, 8192), (9, 12288), (3, 16384), (2, 40000), (2, 65544), (1200, 8), (4000, 33)]


@pytest.mark.parametrize("dtype", DTYPES, ids=NAME.get)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes(shape, dtype):
    _run(*shape, dtype, dtype)
    _run(*shape, dtype, torch.float32, residual=True, dh=True, seed=4)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", DTYPES, ids=NAME.get)
def test_layouts(dtype, layout):
    for N in (96, 101, 1026, 4100):
        _run(37, N, dtype, torch.float32, layout=layout, residual=True, dh=True)
        _run(37, N, dtype, dtype, layout=layout)


@pytest.mark.parametrize("dtype", DTYPES, ids=NAME.get)
def test_optional_parts(dtype):
    for gamma, beta in ((False, False), (True, False), (False, True)):
        _run(21, 264, dtype, dtype, gamma=gamma, beta=beta)
        _run(21, 264, dtype, dtype, gamma=gamma, beta=beta, residual=True, dh=True, params=False)


def test_many_rows():
    _run(60000, 64, torch.bfloat16, torch.float32, residual=True, dh=True)
    _run(9001, 512, torch.bfloat16, torch.bfloat16)


# rows that begin and end inside 16 bytes, more of them than groups of threads: every group has several
RAGGED = [(20011, 61), (9003, 127), (5002, 250), (5001, 1001), (2003, 2047), (1501, 4001), (701, 8181), (401, 8191),
          (331, 9001), (301, 16381)]


@pytest.mark.parametrize("dtype", DTYPES, ids=NAME.get)
@pytest.mark.parametrize("shape", RAGGED, ids=lambda s: "x".join(map(str, s)))
def test_ragged_rows(shape, dtype):
    _run(*shape, dtype, torch.float32, residual=True, dh=True, seed=12)
    _run(*shape, dtype, dtype, seed=13)


# rows that a cluster of two to eight blocks shares, several rows each; the last one is too long for that
@pytest.mark.parametrize("dtype", DTYPES, ids=NAME.get)
@pytest.mark.parametrize("shape", [(601, 8200), (401, 12288), (261, 20480), (171, 32768), (91, 65536), (61, 32777),
                                   (101, 32761), (51, 16377), (20, 70001)], ids=lambda s: "x".join(map(str, s)))
def test_shared_rows(shape, dtype):
    _run(*shape, dtype, torch.float32, residual=True, dh=True, seed=17)
    _run(*shape, dtype, dtype, seed=18, layout="padded")


@pytest.mark.parametrize("N", [61, 1001, 4001, 8195])
def test_nan_at_a_ragged_end_stays_in_its_row(N):
    # the 16 bytes around a row's ends belong to its neighbours as well
    swg = _swg()
    for dtype in DTYPES:
        t = _inputs(9, N, dtype, torch.float32, 14)
        clean = swg.layer_norm_fwd(t["x"], t["gamma"], t["beta"], residual=t["residual"])
        dclean = swg.layer_norm_bwd(t["dy"], clean["h"], clean["stats"], gamma=t["gamma"])[0]
        t["x"][2, 0], t["x"][2, N - 1], t["residual"][5, 0], t["residual"][5, N - 1] = (float("nan"),) * 4
        out = swg.layer_norm_fwd(t["x"], t["gamma"], t["beta"], residual=t["residual"])
        h = clean["h"].clone()
        h[2, 0], h[2, N - 1], t["dy"][5, 0], t["dy"][5, N - 1] = (float("inf"),) * 4
        dx = swg.layer_norm_bwd(t["dy"], h, clean["stats"], gamma=t["gamma"])[0]
        rows = [r for r in range(9) if r not in (2, 5)]
        assert torch.equal(out["y"][rows], clean["y"][rows]) and torch.equal(out["h"][rows], clean["h"][rows])
        assert torch.equal(dx[rows], dclean[rows])
        assert out["y"][2].isnan().all() and out["y"][5].isnan().all()
        assert not dx[2].isfinite().all() and not dx[5].isfinite().all()


def test_weights_and_rows_off_16_bytes():
    # outputs on 16 bytes, inputs and weights not, and the other way round
    swg = _swg()
    for dtype in DTYPES:
        for N in (96, 1000, 1003):
            t = _inputs(700, N, dtype, dtype, 15)
            off = {}
            for k, v in t.items():
                off[k] = torch.empty(v.numel() + 1, dtype=v.dtype, device="cuda")[1:].view(v.shape).copy_(v)
            for a in (off, {**t, "gamma": off["gamma"], "beta": off["beta"]}, {**off, "x": t["x"]}):
                out = swg.layer_norm_fwd(a["x"], a["gamma"], a["beta"], eps=EPS, residual=a["residual"])
                _check_fwd(t, out, dtype, residual=True)
                got = swg.layer_norm_bwd(a["dy"], out["h"], out["stats"], gamma=a["gamma"], dh=a["dh"])
                _check_bwd(t, out["h"], out["stats"], got, dtype, dtype, dh=True)
            spare = {k: torch.empty(700 * N + 1, dtype=dtype, device="cuda")[1:].view(700, N) for k in ("y", "h", "dx")}
            stats = torch.empty((700, 2), device="cuda")
            out = swg.layer_norm_fwd(t["x"], t["gamma"], t["beta"], eps=EPS, residual=t["residual"],
                                     out={"y": spare["y"], "h": spare["h"], "stats": stats})
            _check_fwd(t, out, dtype, residual=True)
            _check_bwd(t, out["h"], stats, swg.layer_norm_bwd(t["dy"], out["h"], stats, gamma=t["gamma"], dh=t["dh"],
                                                              dx=spare["dx"]), dtype, dtype, dh=True)


def test_leading_dimensions_and_shared_rows():
    swg = _swg()
    t = _inputs(12, 72, torch.bfloat16, torch.float32, 5)
    out = swg.layer_norm_fwd(t["x"].view(3, 4, 72), t["gamma"], t["beta"])
    assert out["y"].shape == (3, 4, 72) and out["stats"].shape == (12, 2)
    _check_fwd(t, out, torch.bfloat16)
    # one gradient row shared by all rows (an expanded tensor)
    t["dy"] = t["dy"][:1].expand(12, 72)
    _check_bwd(t, t["x"], out["stats"], swg.layer_norm_bwd(t["dy"], t["x"], out["stats"], gamma=t["gamma"]),
               torch.bfloat16, torch.float32)
    x1 = t["x"][0]  # one dimension
    assert torch.equal(swg.layer_norm_fwd(x1, t["gamma"], t["beta"])["y"], out["y"].view(12, 72)[0])


def test_large_mean_and_constant_rows():
    # rows far from zero keep their spread (the variance is of centred values); a constant row gives beta
    swg = _swg()
    t = _inputs(16, 1024, torch.float32, torch.float32, 6)
    t["x"] += 300.0
    t["x"][3] = 7.25
    out = swg.layer_norm_fwd(t["x"], t["gamma"], t["beta"])
    _check_fwd(t, out, torch.float32)
    assert torch.equal(out["y"][3], t["beta"])


def test_nan_and_inf_stay_in_their_rows():
    swg = _swg()
    t = _inputs(9, 520, torch.bfloat16, torch.float32, 7)
    clean = swg.layer_norm_fwd(t["x"], t["gamma"], t["beta"])
    dclean = swg.layer_norm_bwd(t["dy"], t["x"], clean["stats"], gamma=t["gamma"])[0]
    t["x"][2, 17], t["x"][5, 500] = float("nan"), float("inf")
    out = swg.layer_norm_fwd(t["x"], t["gamma"], t["beta"])
    dx, dgamma, dbeta = swg.layer_norm_bwd(t["dy"], t["x"], out["stats"], gamma=t["gamma"])
    rows = [r for r in range(9) if r not in (2, 5)]
    assert torch.equal(out["y"][rows], clean["y"][rows]) and torch.equal(dx[rows], dclean[rows])
    assert out["y"][2].isnan().all() and dx[2].isnan().all() and out["y"][5].isnan().all()
    assert dgamma.isnan().all() and not dbeta.isnan().any()


def test_gradient_by_differences():
    # directional difference of the library's own fp32 forward: the loss is sum(y dy), h moves along v
    swg = _swg()
    t = _inputs(4, 96, torch.float32, torch.float32, 8)
    loss = lambda x, g, b: float((swg.layer_norm_fwd(x, g, b)["y"].double() * t["dy"].double()).sum())  # noqa: E731
    out = swg.layer_norm_fwd(t["x"], t["gamma"], t["beta"])
    dx, dgamma, dbeta = swg.layer_norm_bwd(t["dy"], t["x"], out["stats"], gamma=t["gamma"])
    e = 2.0 ** -7
    for name, grad in (("x", dx), ("gamma", dgamma), ("beta", dbeta)):
        v = torch.sign(t["dh"][0, :96] if name != "x" else t["dh"])
        args = lambda s: [t[k] + s * e * v if k == name else t[k] for k in ("x", "gamma", "beta")]  # noqa: E731
        diff = (loss(*args(1)) - loss(*args(-1))) / (2 * e)
        want = float((grad.double() * v.double()).sum())
        # truncation e^2/6 of a third derivative of order (rows cols)^(1/2) 10, and fp32 forward error / e
        assert abs(diff - want) <= e * e * 10 * 20 + 384 * 2.0 ** -22 * 4 / e, (name, diff, want)


def test_reproducible_and_guarded():
    swg = _swg()
    for M, N, dtype in ((33, 1000, torch.bfloat16), (7, 1003, torch.float16), (501, 128, torch.float32)):
        t = _inputs(M, N, dtype, torch.float32, 9)
        gs = dict(y=guarded((M, N), dtype), h=guarded((M, N), dtype), stats=guarded((M, 2), torch.float32),
                  dx=guarded((M, N), dtype), dgamma=guarded((N,), torch.float32), dbeta=guarded((N,), torch.float32),
                  ws=workspace(swg.layer_norm_bwd_workspace_size(M, N)))
        out = swg.layer_norm_fwd(t["x"], t["gamma"], t["beta"], residual=t["residual"],
                                 out={k: gs[k].t for k in ("y", "h", "stats")})
        got = swg.layer_norm_bwd(t["dy"], out["h"], out["stats"], gamma=t["gamma"], dh=t["dh"], dx=gs["dx"].t,
                                 dgamma=gs["dgamma"].t, dbeta=gs["dbeta"].t, workspace=gs["ws"].t)
        torch.cuda.synchronize()
        check_all(gs)
        assert out["y"].data_ptr() == gs["y"].t.data_ptr() and got[0].data_ptr() == gs["dx"].t.data_ptr()
        again = swg.layer_norm_bwd(t["dy"], out["h"], out["stats"], gamma=t["gamma"], dh=t["dh"])
        assert all(torch.equal(a, b) for a, b in zip(got, again))
        _check_fwd(t, out, dtype, residual=True)
        _check_bwd(t, out["h"], out["stats"], got, dtype, torch.float32, dh=True)


def test_empty():
    swg = _swg()
    x = torch.empty((0, 16), dtype=torch.bfloat16, device="cuda")
    out = swg.layer_norm_fwd(x, residual=x)
    assert out["y"].shape == (0, 16) and out["h"].shape == (0, 16) and out["stats"].shape == (0, 2)
    dx, dgamma, dbeta = swg.layer_norm_bwd(x, x, out["stats"])
    assert dx.shape == (0, 16) and not dgamma.any() and not dbeta.any()
    assert swg.layer_norm_fwd(torch.empty((3, 0), device="cuda"))["y"].shape == (3, 0)


@pytest.mark.parametrize("M,N", [(264000, 8192), (2150000, 1001)], ids=["whole", "ragged"])
def test_offsets_past_32_bits(M, N):
    swg = _swg()
    assert M * N > 2 ** 31
    g = torch.Generator(device="cuda")
    g.manual_seed(12)
    x = torch.empty((M, N), dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g)
    t = _inputs(1, N, torch.bfloat16, torch.float32, 13)
    out = swg.layer_norm_fwd(x, t["gamma"], t["beta"], eps=EPS, residual=x)
    dx = swg.layer_norm_bwd(x, out["h"], out["stats"], gamma=t["gamma"], params=False)[0]
    rows = [0, 1, M // 2, M - 2, M - 1]
    few = dict(x=x[rows], residual=x[rows], dy=x[rows], gamma=t["gamma"], beta=t["beta"])
    small = {k: v[rows] for k, v in out.items()}
    _check_fwd(few, small, torch.bfloat16, residual=True)
    _check_bwd(few, small["h"], small["stats"], (dx[rows], None, None), torch.bfloat16, torch.float32)


def test_on_another_stream():
    swg = _swg()
    t = _inputs(2000, 1024, torch.bfloat16, torch.float32, 10)
    want = swg.layer_norm_fwd(t["x"], t["gamma"], t["beta"])
    wantb = swg.layer_norm_bwd(t["dy"], t["x"], want["stats"], gamma=t["gamma"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for st in (s, s.cuda_stream):
        out = swg.layer_norm_fwd(strided(t["x"], "transposed"), t["gamma"], t["beta"], stream=st)
        got = swg.layer_norm_bwd(t["dy"], t["x"], out["stats"], gamma=t["gamma"], stream=st)
        s.synchronize()
        assert torch.equal(out["y"], want["y"]) and all(torch.equal(a, b) for a, b in zip(got, wantb))


def test_in_a_graph():
    swg = _swg()
    t = _inputs(64, 512, torch.bfloat16, torch.float32, 11)
    out = {"y": torch.empty_like(t["x"]), "stats": torch.empty((64, 2), device="cuda")}
    ws = torch.empty(swg.layer_norm_bwd_workspace_size(64, 512), dtype=torch.uint8, device="cuda")
    grads = dict(dx=torch.empty_like(t["x"]), dgamma=torch.empty_like(t["gamma"]), dbeta=torch.empty_like(t["gamma"]))

    def step():
        swg.layer_norm_fwd(t["x"], t["gamma"], t["beta"], out=out)
        swg.layer_norm_bwd(t["dy"], t["x"], out["stats"], gamma=t["gamma"], workspace=ws, **grads)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    t["x"].mul_(2.0)
    g.replay()
    torch.cuda.synchronize()
    _check_fwd(t, out, torch.bfloat16)
    _check_bwd(t, t["x"], out["stats"], (grads["dx"], grads["dgamma"], grads["dbeta"]), torch.bfloat16, torch.float32)


def test_refusals():
    swg = _swg()
    x = torch.zeros((4, 8), dtype=torch.bfloat16, device="cuda")
    st = torch.zeros((4, 2), device="cuda")
    with pytest.raises(TypeError):
        swg.layer_norm_fwd(x.int())
    with pytest.raises(ValueError):
        swg.layer_norm_fwd(x, residual=x[:2])
    with pytest.raises(ValueError):
        swg.layer_norm_fwd(x, gamma=torch.zeros(8, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        swg.layer_norm_fwd(x, gamma=x[0], beta=torch.zeros(8, device="cuda"))
    with pytest.raises(ValueError):
        swg.layer_norm_fwd(x, gamma=torch.zeros(7, device="cuda"))
    with pytest.raises(swg.SwgError):
        swg.layer_norm_fwd(x, eps=-1.0)
    with pytest.raises(swg.SwgError):  # y over x
        swg.layer_norm_fwd(x, out={"y": x})
    with pytest.raises(ValueError):
        swg.layer_norm_bwd(x, x, st[:3])
    with pytest.raises(ValueError):
        swg.layer_norm_bwd(x[:, :4], x, st)
    with pytest.raises(swg.SwgError):  # a short workspace
        swg.layer_norm_bwd(x, x, st, workspace=torch.empty(4, dtype=torch.uint8, device="cuda"))
