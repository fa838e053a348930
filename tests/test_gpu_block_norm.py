"""The norms between blocks, forward and backward, against the fp64 oracle (GPU)."""

import itertools

import pytest
import torch

from ._block import check_norm_bwd, check_norm_fwd, norm_inputs
from ._guard import check_all, guarded, workspace
from ._row_ops import DTYPES, LAYOUTS, strided

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _swg():
    import swiglu_ffn_backward_gb300 as swg
    return swg


def _run(M, N, dtype, wdtype, gates, gdtype=None, residual=True, alpha=1.0, post=True, pre=True, dh=True, params=True,
         layout="dense", seed=5, eps=1e-6):
    swg = _swg()
    t = norm_inputs(M, N, dtype, wdtype, gates, gdtype, seed)
    lay = {k: strided(t[k], layout) for k in ("u", "residual", "dy", "dh")}
    kw = dict(gamma_post=t["gamma_post"] if post else None, gamma_pre=t["gamma_pre"] if pre else None, gate=t["gate"],
              alpha=alpha, post=post, pre=pre)
    out = swg.block_norm_fwd(lay["u"], lay["residual"] if residual else None, eps=eps, **kw)
    check_norm_fwd(t, out, dtype, residual, alpha, eps, post, pre)
    h = out.get("h")
    got = swg.block_norm_bwd(lay["dy"] if pre else None, lay["dh"] if dh else None, lay["u"], h, out["stats"],
                             residual=residual, params=params, **kw)
    check_norm_bwd(t, t["u"] if h is None else h, out["stats"], got, dtype, wdtype, gdtype or dtype, residual, alpha,
                   post, pre, dh, params)
    swg.swg_check()
    return t, out, got


# rows of a few vectors to many, whole and ragged
SIZES = [(1, 8), (1, 4096), (3, 1), (5, 7), (7, 64), (64, 100), (130, 256), (257, 1001), (31, 2048), (33, 4096),
         (12, 5001), (9, 8192), (6, 12288), (5, 20000), (4, 16383), (2, 40000), (2, 70001)]


@pytest.mark.parametrize("M,N", SIZES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_sizes(M, N, dtype):
    _run(M, N, dtype, F32 if M % 2 else dtype, gates=1)
    _run(M, N, dtype, dtype, gates=M, alpha=0.7)


@pytest.mark.parametrize("gates", [0, 1, 2, 8, 30, 240])
@pytest.mark.parametrize("N", [72, 520, 515])
@pytest.mark.parametrize("dtype,gdtype", [(BF16, BF16), (F16, F32), (F32, F32)])
def test_gates(gates, N, dtype, gdtype):
    _run(240, N, dtype, dtype, gates, gdtype, alpha=0.5)


PARTS = [(g, r, p, q, dh) for g, r, p, q, dh in itertools.product((0, 1, 5, 20), (True, False), (True, False), (True, False),
                                                               (True, False)) if (p or q) and (q or dh)]


@pytest.mark.parametrize("gates,residual,post,pre,dh", PARTS)
def test_parts(gates, residual, post, pre, dh):
    # every combination of what may be absent
    for N, dtype in ((264, BF16), (37, F32)):
        _run(20, N, dtype, F32, gates, residual=residual, post=post, pre=pre, dh=dh, alpha=0.8 if residual else 1.0)


def test_without_parameter_gradients_and_gammas():
    swg = _swg()
    _run(50, 136, BF16, BF16, 5, params=False)
    t = norm_inputs(50, 136, BF16, BF16, 5)
    ones = {k: torch.ones_like(t[k]) for k in ("gamma_post", "gamma_pre")}
    a = swg.block_norm_fwd(t["u"], t["residual"], gate=t["gate"])
    b = swg.block_norm_fwd(t["u"], t["residual"], gate=t["gate"], **ones)
    assert all(torch.equal(a[k], b[k]) for k in b)
    ga = swg.block_norm_bwd(t["dy"], t["dh"], t["u"], a["h"], a["stats"], gate=t["gate"])
    gb = swg.block_norm_bwd(t["dy"], t["dh"], t["u"], a["h"], a["stats"], gate=t["gate"], **ones)
    assert all(torch.equal(ga[k], gb[k]) for k in gb)


def test_plain_norm():
    # neither a norm before it, a residual nor a gate: h is u itself, which is neither copied nor returned
    swg, t = _swg(), norm_inputs(33, 520, BF16, F32, 0)
    out = swg.block_norm_fwd(t["u"], gamma_pre=t["gamma_pre"], post=False)
    assert set(out) == {"y", "stats"}
    got = swg.block_norm_bwd(t["dy"], None, t["u"], None, out["stats"], gamma_pre=t["gamma_pre"], post=False,
                             residual=False)
    assert set(got) == {"du", "dgamma_pre"}
    # with a residual and nothing else both gradients are the same tensor
    out = swg.block_norm_fwd(t["u"], t["residual"], gamma_pre=t["gamma_pre"], post=False)
    got = swg.block_norm_bwd(t["dy"], t["dh"], t["u"], out["h"], out["stats"], gamma_pre=t["gamma_pre"], post=False)
    assert got["du"] is got["dresidual"]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("N", [64, 264, 101])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layouts(layout, N, dtype):
    _run(48, N, dtype, dtype, 6, layout=layout)


def test_leading_shapes_and_gate_shapes():
    swg = _swg()
    B, S, N = 3, 4, 72
    t = norm_inputs(B * S, N, BF16, BF16, B)
    kw = dict(gamma_post=t["gamma_post"], gamma_pre=t["gamma_pre"])
    want = swg.block_norm_fwd(t["u"], t["residual"], gate=t["gate"], **kw)
    wantb = swg.block_norm_bwd(t["dy"], t["dh"], t["u"], want["h"], want["stats"], gate=t["gate"], **kw)
    v = {k: t[k].view(B, S, N) for k in ("u", "residual", "dy", "dh")}
    for gate in (t["gate"], t["gate"].view(B, 1, N), t["gate"].t().contiguous().t()):
        out = swg.block_norm_fwd(v["u"], v["residual"], gate=gate, **kw)
        assert out["y"].shape == (B, S, N) and torch.equal(out["y"].view(-1, N), want["y"])
        got = swg.block_norm_bwd(v["dy"], v["dh"], v["u"], out["h"], out["stats"], gate=gate, **kw)
        assert got["dgate"].shape == gate.shape
        assert all(torch.equal(got[k].reshape(wantb[k].shape), wantb[k]) for k in wantb)
    # one gate for all rows, in the forms of a vector and of a row; one for each row
    one = swg.block_norm_fwd(v["u"], v["residual"], gate=t["gate"][0], **kw)["y"]
    assert torch.equal(one, swg.block_norm_fwd(v["u"], v["residual"], gate=t["gate"][:1].view(1, 1, N), **kw)["y"])
    each = torch.repeat_interleave(t["gate"], S, dim=0)
    for gate in (each, each.view(B, S, N)):
        assert torch.equal(swg.block_norm_fwd(v["u"], v["residual"], gate=gate, **kw)["y"].view(-1, N), want["y"])
    # rows with one shared residual
    shared = t["residual"][:1].expand(B * S, N)
    a = swg.block_norm_fwd(t["u"], shared, gate=t["gate"], **kw)
    b = swg.block_norm_fwd(t["u"], shared.contiguous(), gate=t["gate"], **kw)
    assert all(torch.equal(a[k], b[k]) for k in a)
    # a single vector
    a = swg.block_norm_fwd(t["u"][0], t["residual"][0], gate=t["gate"][0], **kw)
    assert a["y"].shape == (N,) and torch.equal(a["y"], want["y"][0])


@pytest.mark.parametrize("M,N,gates,dtype", [(37, 264, 37, BF16), (40, 101, 4, F16), (3, 9000, 1, F32), (70, 65, 0, BF16)])
def test_nothing_outside_the_outputs(M, N, gates, dtype):
    swg, t = _swg(), norm_inputs(M, N, dtype, F32, gates)
    kw = dict(gamma_post=t["gamma_post"], gamma_pre=t["gamma_pre"], gate=t["gate"])
    for shift in (0, 1):
        g = {"h": guarded((M, N), dtype, offset_elems=shift), "y": guarded((M, N), dtype, offset_elems=shift),
             "stats": guarded((M, 2), F32)}
        out = swg.block_norm_fwd(t["u"], t["residual"], out={k: v.t for k, v in g.items()}, **kw)
        check_all(g)
        check_norm_fwd(t, out, dtype)
        g = {"du": guarded((M, N), dtype, offset_elems=shift), "dresidual": guarded((M, N), dtype, offset_elems=shift),
             "dgamma_post": guarded((N,), F32), "dgamma_pre": guarded((N,), F32),
             "ws": workspace(swg.block_norm_bwd_workspace_size(M, N, gates))}
        if gates:
            g["dgate"] = guarded((gates, N), dtype)
        got = swg.block_norm_bwd(t["dy"], t["dh"], t["u"], out["h"], out["stats"], workspace=g["ws"].t,
                                 out={k: v.t for k, v in g.items() if k != "ws"}, **kw)
        check_all(g)
        check_norm_bwd(t, out["h"], out["stats"], got, dtype, F32, dtype)


@pytest.mark.parametrize("M,N,gates", [(60000, 64, 0), (60000, 64, 3), (33000, 72, 16500), (20011, 33, 1), (4099, 1024, 0)])
def test_many_rows(M, N, gates):
    _run(M, N, BF16, F32, gates)


# many whole rows: their loads go through a ring in shared memory, for groups of one warp to clusters of eight blocks
@pytest.mark.parametrize("M,N,dtype", [(20011, 264, BF16), (40000, 132, F32), (9001, 512, F16), (2003, 4096, BF16), (1200, 2048, F32),
                                       (900, 5120, BF16), (1801, 8192, F16), (700, 12288, BF16), (640, 12288, F32), (300, 32768, BF16)])
@pytest.mark.parametrize("gates", ["none", "one", "some", "rows"])
def test_ring(M, N, dtype, gates):
    divisor = next(d for d in (7, 5, 3, 2, 1) if M % d == 0)
    G = {"none": 0, "one": 1, "some": divisor if divisor > 1 else 1, "rows": M}[gates]
    _run(M, N, dtype, F32 if gates == "one" else dtype, G, F32 if gates != "some" else dtype, alpha=0.9)


@pytest.mark.parametrize("residual,post,pre,dh", [(False, True, True, True), (True, False, True, True), (True, True, False, True),
                                                  (True, True, True, False), (False, False, True, False)])
@pytest.mark.parametrize("gates", [0, 4, 2400])
def test_ring_parts(residual, post, pre, dh, gates):
    _run(2400, 4096, BF16, BF16, gates, residual=residual, post=post, pre=pre, dh=dh)
    _run(2400, 8192, F16, F32, gates, residual=residual, post=post, pre=pre, dh=dh)


# ragged rows take the ring where all tensors' rows lie on the same offsets within 16 bytes
@pytest.mark.parametrize("M,N,dtype", [(20011, 265, BF16), (40000, 133, F32), (9001, 515, F16), (2003, 4001, BF16), (1200, 2047, F32),
                                       (1801, 8190, F16), (700, 12289, BF16), (640, 10001, F32), (301, 32700, BF16)])
@pytest.mark.parametrize("gates", ["none", "some", "rows"])
def test_ragged_ring(M, N, dtype, gates):
    divisor = next(d for d in (7, 5, 3, 2, 1) if M % d == 0)
    G = {"none": 0, "some": divisor, "rows": M}[gates]
    _run(M, N, dtype, F32 if gates == "some" else dtype, G, dtype, alpha=0.9)


@pytest.mark.parametrize("residual,post,pre,dh", [(False, True, True, True), (True, False, True, True), (True, True, False, True),
                                                  (True, True, True, False), (False, False, True, False)])
def test_ragged_ring_parts(residual, post, pre, dh):
    for gates in (0, 4, 2400):
        _run(2400, 4003, BF16, F32, gates, residual=residual, post=post, pre=pre, dh=dh)


def test_ragged_ring_stays_inside():
    # every tensor begins and ends inside 16 bytes, between others' bytes, which are NaN: nothing outside it is written
    # and nothing of its neighbours enters
    swg = _swg()
    for M, N, dtype in ((2003, 4001, BF16), (1200, 2047, F32)):
        t = norm_inputs(M, N, dtype, F32, M)
        pad = {}
        for k in ("u", "residual", "dy", "dh", "gate"):
            pad[k] = guarded(t[k].shape, dtype, offset_elems=1)
            pad[k].raw.fill_(0xFF)
            pad[k].t.copy_(t[k])
        kw = dict(gamma_post=t["gamma_post"], gamma_pre=t["gamma_pre"], gate=pad["gate"].t)
        g = {k: guarded((M, N), dtype, offset_elems=1) for k in ("h", "y")}
        out = swg.block_norm_fwd(pad["u"].t, pad["residual"].t, out={k: v.t for k, v in g.items()}, **kw)
        check_all(g)
        check_norm_fwd(t, out, dtype)
        gb = {k: guarded((M, N), dtype, offset_elems=1) for k in ("du", "dresidual", "dgate")}
        gb["ws"] = workspace(swg.block_norm_bwd_workspace_size(M, N, M))
        got = swg.block_norm_bwd(pad["dy"].t, pad["dh"].t, pad["u"].t, out["h"], out["stats"], workspace=gb["ws"].t,
                                 out={k: v.t for k, v in gb.items() if k != "ws"}, **kw)
        check_all(gb)
        check_norm_bwd(t, out["h"], out["stats"], got, dtype, F32, dtype)


def test_ring_layouts():
    for layout in ("padded", "dense"):
        _run(2003, 4096, BF16, BF16, 1, layout=layout)
    swg, t = _swg(), norm_inputs(3000, 4096, BF16, F32, 3)
    a = swg.block_norm_fwd(t["u"], t["residual"][:1].expand(3000, 4096), gate=t["gate"])
    b = swg.block_norm_fwd(t["u"], t["residual"][:1].expand(3000, 4096).contiguous(), gate=t["gate"])
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_like_rows_do_not_drift():
    # parameter gradients of equal rows: in one chain of fp32 additions like terms are rounded the same way
    swg, M, N = _swg(), 200000, 64
    t = norm_inputs(1, N, F32, F32, 1, seed=8)
    big = {k: t[k].expand(M, N).contiguous() for k in ("u", "residual", "dy", "dh")}
    kw = dict(gamma_post=t["gamma_post"], gamma_pre=t["gamma_pre"], gate=t["gate"])
    out = swg.block_norm_fwd(big["u"], big["residual"], **kw)
    got = swg.block_norm_bwd(big["dy"], big["dh"], big["u"], out["h"], out["stats"], **kw)
    one = swg.block_norm_bwd(t["dy"], t["dh"], t["u"], out["h"][:1], out["stats"][:1], **kw)
    for k in ("dgamma_post", "dgamma_pre", "dgate"):
        want = one[k].double().flatten() * M
        assert float(((got[k].double().flatten() - want) / want).abs().max()) <= 2.0 ** -16


def test_empty():
    swg = _swg()
    e = lambda *s: torch.empty(s, device="cuda", dtype=BF16)  # noqa: E731
    out = swg.block_norm_fwd(e(0, 16), e(0, 16))
    assert out["y"].shape == (0, 16) and out["stats"].shape == (0, 2)
    got = swg.block_norm_bwd(e(0, 16), None, e(0, 16), e(0, 16), out["stats"],
                             gate=torch.ones((4, 16), device="cuda", dtype=BF16))
    assert got["dgate"].shape == (4, 16)
    assert not any(got[k].any() for k in ("dgamma_post", "dgamma_pre", "dgate"))
    assert swg.block_norm_fwd(e(3, 0), e(3, 0))["y"].shape == (3, 0)


def test_rows_of_zeros_and_non_finite_rows():
    swg, t = _swg(), norm_inputs(40, 136, BF16, F32, 0)
    kw = dict(gamma_post=t["gamma_post"], gamma_pre=t["gamma_pre"])
    clean = swg.block_norm_fwd(t["u"], t["residual"], **kw)
    cleanb = swg.block_norm_bwd(t["dy"], t["dh"], t["u"], clean["h"], clean["stats"], **kw)
    t["u"][2], t["residual"][2] = 0, 0
    t["u"][7, 3], t["residual"][11, 0] = float("nan"), float("inf")
    out = swg.block_norm_fwd(t["u"], t["residual"], **kw)
    assert not out["y"][2].any() and torch.isnan(out["y"][7]).all()
    assert float(out["stats"][2, 0]) == pytest.approx(1e3) and float(out["stats"][2, 1]) == pytest.approx(1e3)
    got = swg.block_norm_bwd(t["dy"], t["dh"], t["u"], out["h"], out["stats"], params=False, **kw)
    assert torch.isfinite(got["du"][2]).all() and torch.isnan(got["du"][7]).all()
    keep = [r for r in range(40) if r not in (2, 7, 11)]
    assert torch.equal(out["y"][keep], clean["y"][keep])
    assert torch.equal(got["du"][keep], cleanb["du"][keep])


@pytest.mark.parametrize("M,N,dtype", [(300, 264, BF16), (300, 101, F32), (20, 9000, BF16), (3000, 4096, BF16),
                                       (800, 12288, BF16), (3000, 4001, BF16)])
def test_same_bits_every_time(M, N, dtype):
    swg, t = _swg(), norm_inputs(M, N, dtype, F32, 4)
    kw = dict(gamma_post=t["gamma_post"], gamma_pre=t["gamma_pre"], gate=t["gate"])
    a, b = (swg.block_norm_fwd(t["u"], t["residual"], **kw) for _ in range(2))
    assert all(torch.equal(a[k], b[k]) for k in a)
    c, d = (swg.block_norm_bwd(t["dy"], t["dh"], t["u"], a["h"], a["stats"], **kw) for _ in range(2))
    assert all(torch.equal(c[k], d[k]) for k in c)


def test_streams_and_graphs():
    swg, t = _swg(), norm_inputs(96, 264, BF16, F32, 4)
    kw = dict(gamma_post=t["gamma_post"], gamma_pre=t["gamma_pre"], gate=t["gate"])
    want = swg.block_norm_fwd(t["u"], t["residual"], **kw)
    back = swg.block_norm_bwd(t["dy"], t["dh"], t["u"], want["h"], want["stats"], **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = swg.block_norm_fwd(t["u"], t["residual"], stream=s, **kw)
    gotb = swg.block_norm_bwd(t["dy"], t["dh"], t["u"], got["h"], got["stats"], stream=s, **kw)
    s.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want) and all(torch.equal(gotb[k], back[k]) for k in back)
    out, outb = {k: torch.zeros_like(v) for k, v in want.items()}, {k: torch.zeros_like(v) for k, v in back.items()}
    ws = torch.empty(swg.block_norm_bwd_workspace_size(96, 264, 4), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        swg.block_norm_fwd(t["u"], t["residual"], out=out, **kw)
        swg.block_norm_bwd(t["dy"], t["dh"], t["u"], out["h"], out["stats"], out=outb, workspace=ws, **kw)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], want[k]) for k in want) and all(torch.equal(outb[k], back[k]) for k in back)
        for v in (*out.values(), *outb.values()):
            v.zero_()


def test_refusals():
    swg, t = _swg(), norm_inputs(12, 16, BF16, F32, 3)
    u, r, g = t["u"], t["residual"], t["gate"]
    st = swg.block_norm_fwd(u, r)["stats"]
    u3 = u.view(3, 4, 16)
    for call in (lambda: swg.block_norm_fwd(u, r.float()), lambda: swg.block_norm_fwd(u, r[:4]),
                 lambda: swg.block_norm_fwd(u, r, gamma_post=t["gamma_post"], post=False),
                 lambda: swg.block_norm_fwd(u, r, gamma_pre=t["gamma_pre"], pre=False),
                 lambda: swg.block_norm_fwd(u, r, gamma_post=t["gamma_post"], gamma_pre=t["gamma_pre"].bfloat16()),
                 lambda: swg.block_norm_fwd(u, r, gate=g[:, :8]), lambda: swg.block_norm_fwd(u, r, gate=g.half()),
                 lambda: swg.block_norm_fwd(u, r, gate=torch.ones((5, 16), device="cuda", dtype=BF16)),
                 # a gate for each position of a sequence is none for runs of rows
                 lambda: swg.block_norm_fwd(u3, r.view(3, 4, 16), gate=torch.ones((1, 4, 16), device="cuda", dtype=BF16)),
                 lambda: swg.block_norm_fwd(u3, r.view(3, 4, 16), gate=torch.ones((4, 16), device="cuda", dtype=BF16)),
                 lambda: swg.block_norm_bwd(t["dy"], None, u, r, st[:3]),
                 lambda: swg.block_norm_fwd(u, r, out={"y": torch.empty((16, 12), device="cuda", dtype=BF16)})):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: swg.block_norm_fwd(u.cpu(), r), lambda: swg.block_norm_fwd(u, r, gate=g.cpu()),
                 lambda: swg.block_norm_fwd(u.long(), r), lambda: swg.block_norm_bwd(None, t["dh"], u, r, st),
                 lambda: swg.block_norm_bwd(t["dy"], None, u, None, st), lambda: swg.block_norm_bwd(None, None, u, None, st, pre=False)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: swg.block_norm_fwd(u, r, post=False, pre=False), lambda: swg.block_norm_fwd(u, r, eps=-1.0),
                 lambda: swg.block_norm_fwd(u, r, alpha=float("nan")), lambda: swg.block_norm_fwd(u, r, out={"y": r}),
                 lambda: swg.block_norm_bwd(t["dy"], None, u, r, st, out={"du": t["dy"]}),
                 lambda: swg.block_norm_bwd(t["dy"], None, u, r, st, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(swg.SwgError):
            call()
    swg.swg_check()
