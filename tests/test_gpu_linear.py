"""The linear layer with its epilogue, forward and backward, against the fp64 oracle (GPU)."""

import pytest
import torch

from ._block import ACTS, check_linear_bwd, check_linear_fwd, f64, linear_inputs
from ._guard import check_all, guarded, workspace

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _swg():
    import swiglu_ffn_backward_gb300 as swg
    return swg


# one token to some tiles of rows; widths below a tile, of whole tiles, and between
SHAPES = [(1, 8, 8), (1, 2048, 136), (2, 264, 1032), (17, 64, 128), (33, 520, 264), (64, 128, 256), (65, 72, 200),
          (127, 512, 8), (130, 8, 512), (256, 320, 384), (257, 512, 1024), (300, 1032, 136), (1000, 136, 72),
          (2049, 64, 64)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_forward(M, K, N, dtype):
    swg, t = _swg(), linear_inputs(M, K, N, dtype)
    out = swg.linear_fwd(t["x"], t["w"])
    check_linear_fwd(t, out, dtype, None)
    out = swg.linear_fwd(t["x"], t["w"], t["b"], act="silu", residual=t["residual"], save_z=True)
    check_linear_fwd(t, out, dtype, "silu", t["b"], t["residual"])
    swg.swg_check()


@pytest.mark.parametrize("M,K,N", [(5, 72, 136), (130, 264, 264), (700, 136, 328)])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias,residual,save_z", [(True, False, True), (False, True, False), (True, True, True),
                                                  (False, False, True)])
def test_epilogues(M, K, N, act, bias, residual, save_z):
    swg, t = _swg(), linear_inputs(M, K, N, BF16, seed=7)
    b = t["b"].float() if bias and M == 130 else t["b"]
    out = swg.linear_fwd(t["x"], t["w"], b if bias else None, act=act, residual=t["residual"] if residual else None,
                         save_z=save_z)
    assert set(out) == ({"y", "z"} if save_z else {"y"})
    check_linear_fwd(t, out, BF16, act, b if bias else None, t["residual"] if residual else None)


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_backward(M, K, N, dtype):
    swg, t = _swg(), linear_inputs(M, K, N, dtype, seed=9)
    check_linear_bwd(t, swg.linear_bwd(t["dy"], t["x"], t["w"]), dtype, None)
    check_linear_bwd(t, swg.linear_bwd(t["dy"], t["x"], t["w"], z=t["z"], act="gelu", db_dtype=F32), dtype, "gelu",
                     db_dtype=F32)
    swg.swg_check()


# results of many tiles, which go to the kernel on CTA pairs: whole tiles and ragged ones, several waves, bands; the last
# one in wide tiles
LARGE = [(8192, 512, 1024), (8100, 264, 2056), (5001, 1032, 1528), (20000, 64, 264), (2600, 72, 8008), (300, 200, 40008),
         (2000, 9000, 4000)]


@pytest.mark.parametrize("M,K,N", LARGE)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_large_forward(M, K, N, dtype):
    swg, t = _swg(), linear_inputs(M, K, N, dtype, seed=33)
    check_linear_fwd(t, swg.linear_fwd(t["x"], t["w"]), dtype, None)
    out = swg.linear_fwd(t["x"], t["w"], t["b"].float(), act="gelu", residual=t["residual"], save_z=True)
    check_linear_fwd(t, out, dtype, "gelu", t["b"].float(), t["residual"])
    r = t["residual"].clone()
    again = swg.linear_fwd(t["x"], t["w"], t["b"].float(), act="gelu", residual=r, out={"y": r})["y"]
    assert torch.equal(again, out["y"])
    swg.swg_check()


@pytest.mark.parametrize("M,K,N", [(8192, 512, 1024), (5001, 1032, 1528), (2600, 8008, 72), (9000, 2056, 264), (70000, 512, 520), (70000, 1000, 1000),
                                   (2000, 4000, 4104)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_large_backward(M, K, N, dtype):
    swg, t = _swg(), linear_inputs(M, K, N, dtype, seed=35)
    check_linear_bwd(t, swg.linear_bwd(t["dy"], t["x"], t["w"], z=t["z"], act="silu"), dtype, "silu")
    g = {"dx": guarded((M, K), dtype), "dw": guarded((K, N), dtype), "db": guarded((N,), dtype),
         "ws": workspace(swg.linear_bwd_workspace_size(M, K, N))}
    g["dw"].t.fill_(0.5)
    g["db"].t.fill_(-0.25)
    got = swg.linear_bwd(t["dy"], t["x"], t["w"], accumulate=True, workspace=g["ws"].t,
                         out={k: g[k].t for k in ("dx", "dw", "db")})
    check_all(g)
    check_linear_bwd(t, got, dtype, None, old={"dw": 0.5, "db": -0.25})
    swg.swg_check()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,K,N", [(3, 136, 72), (515, 200, 392), (2500, 64, 72)])
def test_backward_activations(M, K, N, act):
    swg, t = _swg(), linear_inputs(M, K, N, F16, seed=11)
    check_linear_bwd(t, swg.linear_bwd(t["dy"], t["x"], t["w"], z=t["z"], act=act), F16, act)


def test_backward_parts():
    swg, t = _swg(), linear_inputs(200, 136, 264, BF16, seed=13)
    whole = swg.linear_bwd(t["dy"], t["x"], t["w"], z=t["z"], act="silu")
    for kw, names in ((dict(need_dx=False), {"dw", "db"}), (dict(need_dw=False), {"dx", "db"}), (dict(bias=False), {"dx", "dw"}),
                      (dict(need_dx=False, need_dw=False), {"db"}), (dict(need_dx=False, bias=False), {"dw"})):
        x = None if kw.get("need_dw") is False else t["x"]
        w = None if kw.get("need_dx") is False else t["w"]
        got = swg.linear_bwd(t["dy"], x, w, z=t["z"], act="silu", **kw)
        assert set(got) == names
        assert all(torch.equal(got[k], whole[k]) for k in names)


@pytest.mark.parametrize("M", [40, 900, 40000])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_accumulate(M, dtype):
    swg, t = _swg(), linear_inputs(M, 72, 136, dtype, seed=15)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    for db_dtype in (dtype, F32):
        out = {"dw": torch.randn((72, 136), generator=g, device="cuda").to(dtype),
               "db": torch.randn(136, generator=g, device="cuda").to(db_dtype)}
        old = {k: f64(v) for k, v in out.items()}
        got = swg.linear_bwd(t["dy"], t["x"], t["w"], z=t["z"], act="hardswish", accumulate=True, out=out)
        assert got["dw"] is out["dw"] and got["db"] is out["db"]
        check_linear_bwd(t, got, dtype, "hardswish", old=old, db_dtype=db_dtype)


def test_long_reduction():
    # a weight gradient over many rows, of a small and of a wide layer
    swg = _swg()
    for M, K, N in ((70001, 64, 72), (33000, 264, 520)):
        t = linear_inputs(M, K, N, BF16, seed=17)
        check_linear_bwd(t, swg.linear_bwd(t["dy"], t["x"], t["w"]), BF16, None)


def test_like_terms_do_not_drift():
    # db of equal rows: the fp32 sums of n like terms in one chain would be off by up to n / 2 ulp
    swg = _swg()
    dy = torch.full((300000, 8), 0.1001, device="cuda").bfloat16()
    got = swg.linear_bwd(dy, None, None, need_dx=False, need_dw=False, db_dtype=F32)["db"]
    want = float(dy[0, 0].double()) * 300000
    assert float((got.double() - want).abs().max()) <= 2.0 ** -17 * want


def test_far_tails_of_gelu():
    # x Phi(x) keeps its relative accuracy where 1 + erf would cancel (bias alone: a zero input)
    swg = _swg()
    b = torch.linspace(-12, 6, 1024, device="cuda")
    x, w = torch.zeros((1, 8), device="cuda", dtype=BF16), torch.zeros((8, 1024), device="cuda", dtype=BF16)
    y = swg.linear_fwd(x, w, b, act="gelu")["y"][0].double()
    want = 0.5 * b.double() * torch.special.erfc(-b.double() * 0.5 ** 0.5)
    assert float(((y - want) / want).abs()[b != 0].max()) <= 2.0 ** -8 + 2.0 ** -15


def test_non_finite_values_stay_in_their_rows():
    swg, t = _swg(), linear_inputs(140, 72, 136, BF16, seed=19)
    clean = swg.linear_fwd(t["x"], t["w"], t["b"], residual=t["residual"])["y"]
    t["x"][3, 5], t["x"][70, 0], t["residual"][139, 7] = float("nan"), float("inf"), float("-inf")
    y = swg.linear_fwd(t["x"], t["w"], t["b"], residual=t["residual"])["y"]
    assert torch.isnan(y[3]).all() and not torch.isfinite(y[70]).any() and y[139, 7] == float("-inf")
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[3], keep[70], keep[139, 7] = False, False, False
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("M,K,N", [(3, 72, 136), (300, 264, 136)])
def test_views(M, K, N):
    # rows apart, rows that no 16-byte vector starts at, transposed, expanded, and leading dimensions
    swg, t = _swg(), linear_inputs(M, K, N, BF16, seed=21)
    want = swg.linear_fwd(t["x"], t["w"], t["b"], residual=t["residual"])["y"]
    back = swg.linear_bwd(t["dy"], t["x"], t["w"])

    def apart(v, by):
        b = torch.full((v.shape[0], v.shape[1] + by), float("nan"), dtype=v.dtype, device="cuda")
        b[:, :v.shape[1]] = v
        return b[:, :v.shape[1]]

    for f in (lambda v: apart(v, 8), lambda v: apart(v, 3), lambda v: v.t().contiguous().t()):
        x, r, dy = f(t["x"]), f(t["residual"]), f(t["dy"])
        assert torch.equal(swg.linear_fwd(x, f(t["w"]), t["b"], residual=r)["y"], want)
        got = swg.linear_bwd(dy, x, f(t["w"]))
        assert all(torch.equal(got[k], back[k]) for k in back)
    x3 = t["x"].view(1, M, 1, K)
    y3 = swg.linear_fwd(x3, t["w"], t["b"], residual=t["residual"].view(1, M, 1, N))["y"]
    assert y3.shape == (1, M, 1, N) and torch.equal(y3.view(M, N), want)
    got = swg.linear_bwd(t["dy"].view(1, M, 1, N), x3, t["w"])
    assert got["dx"].shape == x3.shape and torch.equal(got["dx"].view(M, K), back["dx"])
    one = swg.linear_fwd(t["x"][:1].expand(M, K), t["w"])["y"]
    assert torch.equal(one, one[:1].expand(M, N))
    assert torch.equal(swg.linear_fwd(t["x"][0], t["w"])["y"], one[0])


@pytest.mark.parametrize("M", [1, 70, 600])
def test_residual_in_place(M):
    swg, t = _swg(), linear_inputs(M, 136, 264, BF16, seed=23)
    want = swg.linear_fwd(t["x"], t["w"], t["b"], act="silu", residual=t["residual"])["y"]
    r = t["residual"].clone()
    out = swg.linear_fwd(t["x"], t["w"], t["b"], act="silu", residual=r, out={"y": r})
    assert out["y"] is r and torch.equal(r, want)


@pytest.mark.parametrize("M,K,N", [(1, 72, 136), (129, 136, 72), (515, 264, 200)])
def test_nothing_outside_the_outputs(M, K, N):
    swg, t = _swg(), linear_inputs(M, K, N, BF16, seed=25)
    g = {"y": guarded((M, N), BF16), "z": guarded((M, N), BF16)}
    out = swg.linear_fwd(t["x"], t["w"], t["b"], act="gelu", residual=t["residual"], save_z=True,
                         out={k: v.t for k, v in g.items()})
    check_all(g)
    check_linear_fwd(t, out, BF16, "gelu", t["b"], t["residual"])
    g = {"dx": guarded((M, K), BF16), "dw": guarded((K, N), BF16), "db": guarded((N,), BF16),
         "ws": workspace(swg.linear_bwd_workspace_size(M, K, N, "gelu"))}
    out = swg.linear_bwd(t["dy"], t["x"], t["w"], z=t["z"], act="gelu", workspace=g["ws"].t,
                         out={k: g[k].t for k in ("dx", "dw", "db")})
    check_all(g)
    check_linear_bwd(t, out, BF16, "gelu")


def test_empty():
    swg = _swg()
    e = lambda *s: torch.empty(s, device="cuda", dtype=BF16)  # noqa: E731
    w = torch.ones((16, 24), device="cuda", dtype=BF16)
    assert swg.linear_fwd(e(0, 16), w)["y"].shape == (0, 24)
    got = swg.linear_bwd(e(0, 24), e(0, 16), w)
    assert got["dx"].shape == (0, 16) and not got["dw"].any() and not got["db"].any()
    keep = {"dw": torch.ones_like(w), "db": torch.ones(24, device="cuda", dtype=BF16)}
    swg.linear_bwd(e(0, 24), e(0, 16), w, accumulate=True, out=keep)
    assert bool((keep["dw"] == 1).all()) and bool((keep["db"] == 1).all())


def test_same_bits_every_time():
    swg, t = _swg(), linear_inputs(3000, 264, 392, BF16, seed=27)
    for f in (lambda: swg.linear_fwd(t["x"], t["w"], t["b"], act="gelu", save_z=True),
              lambda: swg.linear_bwd(t["dy"], t["x"], t["w"], z=t["z"], act="gelu")):
        a, b = f(), f()
        assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("M", [1, 400])
def test_streams_and_graphs(M):
    swg, t = _swg(), linear_inputs(M, 264, 392, BF16, seed=29)
    want = swg.linear_fwd(t["x"], t["w"], t["b"], act="silu", save_z=True)
    back = swg.linear_bwd(t["dy"], t["x"], t["w"], z=t["z"], act="silu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = swg.linear_fwd(t["x"], t["w"], t["b"], act="silu", save_z=True, stream=s)
    gotb = swg.linear_bwd(t["dy"], t["x"], t["w"], z=t["z"], act="silu", stream=s)
    s.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want) and all(torch.equal(gotb[k], back[k]) for k in back)
    out, outb = {k: torch.zeros_like(v) for k, v in want.items()}, {k: torch.zeros_like(v) for k, v in back.items()}
    ws = torch.empty(swg.linear_bwd_workspace_size(M, 264, 392, "silu"), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        swg.linear_fwd(t["x"], t["w"], t["b"], act="silu", save_z=True, out=out)
        swg.linear_bwd(t["dy"], t["x"], t["w"], z=t["z"], act="silu", out=outb, workspace=ws)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], want[k]) for k in want) and all(torch.equal(outb[k], back[k]) for k in back)
        for v in (*out.values(), *outb.values()):
            v.zero_()


def test_refusals():
    swg, t = _swg(), linear_inputs(4, 16, 24, BF16, seed=31)
    x, w, b, dy, z, r = (t[k] for k in ("x", "w", "b", "dy", "z", "residual"))
    for call in (lambda: swg.linear_fwd(x.float(), w), lambda: swg.linear_fwd(x, w.cpu()),
                 lambda: swg.linear_fwd(x, w, b.cpu()), lambda: swg.linear_bwd(dy, x, w, db_dtype=F16)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: swg.linear_fwd(x, w.half()), lambda: swg.linear_fwd(x, w[:8]), lambda: swg.linear_fwd(x, w, b[:8]),
                 lambda: swg.linear_fwd(x, w, b.half()), lambda: swg.linear_fwd(x, w, act="relu"),
                 lambda: swg.linear_fwd(x, w, residual=x), lambda: swg.linear_fwd(x, w, residual=r.half()),
                 lambda: swg.linear_fwd(x, w, out={"y": torch.empty((4, 16), device="cuda", dtype=BF16)}),
                 lambda: swg.linear_bwd(dy, x, w, act="silu"), lambda: swg.linear_bwd(dy, x[:2], w),
                 lambda: swg.linear_bwd(dy, x, w[:8]), lambda: swg.linear_bwd(dy, x, w, accumulate=True),
                 lambda: swg.linear_bwd(dy, x, w, z=z.half(), act="silu"), lambda: swg.linear_bwd(dy, None, w),
                 lambda: swg.linear_bwd(dy, x, w, out={"dw": torch.empty((16, 24), device="cuda")})):
        with pytest.raises(ValueError):
            call()
    odd = torch.zeros((4, 12), device="cuda", dtype=BF16)
    for call in (lambda: swg.linear_fwd(odd, torch.zeros((12, 16), device="cuda", dtype=BF16)),
                 lambda: swg.linear_fwd(x, torch.zeros((16, 20), device="cuda", dtype=BF16)),
                 lambda: swg.linear_fwd(x[:, :0], w[:0]),
                 lambda: swg.linear_fwd(x, w, out={"y": torch.empty(97, device="cuda", dtype=BF16)[1:].view(4, 24)}),
                 lambda: swg.linear_bwd(dy, x, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(swg.SwgError):
            call()
    buf = torch.zeros((8, 24), device="cuda", dtype=BF16)
    with pytest.raises(swg.SwgError):  # a residual that overlaps y without being it
        swg.linear_fwd(x, w, residual=buf[1:5], out={"y": buf[:4]})
    swg.swg_check()


# the column sums of up to 512 rows by one cluster, of more by a second launch; added to what is there
@pytest.mark.parametrize("M", [1, 8, 9, 63, 65, 500, 512, 513])
@pytest.mark.parametrize("N", [8, 264, 1032])
@pytest.mark.parametrize("act", [None, "gelu"])
def test_bias_gradient(M, N, act):
    swg, t = _swg(), linear_inputs(M, 16, N, BF16, seed=71)
    for db_dtype in (BF16, F32):
        g = {"db": guarded((N,), db_dtype), "ws": workspace(swg.linear_bwd_workspace_size(M, 16, N, act))}
        kw = dict(z=t["z"], act=act, need_dx=False, need_dw=False, workspace=g["ws"].t, out={"db": g["db"].t})
        got = swg.linear_bwd(t["dy"], t["x"], t["w"], db_dtype=db_dtype, **kw)
        check_linear_bwd(t, got, BF16, act, db_dtype=db_dtype)
        old = f64(g["db"].t)
        got = swg.linear_bwd(t["dy"], t["x"], t["w"], accumulate=True, db_dtype=db_dtype, **kw)
        check_linear_bwd(t, got, BF16, act, old={"db": old}, db_dtype=db_dtype)
        swg.swg_check()
        check_all(g)
