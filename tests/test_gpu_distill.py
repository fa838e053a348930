"""Distillation from a teacher's top logits, forward and backward, against the fp64 oracle (GPU)."""

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


def _inputs(T, V, K, dtype, seed, masked=False, tdtype=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    z = (rn(T, V) * 3).to(dtype)
    ids = torch.rand((T, V), generator=g, device="cuda").topk(min(K, V), dim=1).indices
    if K > V:
        ids = torch.cat([ids, torch.full((T, K - V), -1, device="cuda")], dim=1)
    tl = (rn(T, K) * 2).sort(dim=1, descending=True).values.to(tdtype or dtype)
    w = torch.rand(T, generator=g, device="cuda") - 0.3
    if masked:
        r = torch.arange(T, device="cuda")
        ids[r % 3 == 1, K // 2:] = -1
        ids[r % 5 == 2] = V
        tl[r % 7 == 3, 0] = float("-inf")
        tl[r % 7 == 4] = float("-inf")
        ids[r % 4 == 3, -1] = ids[r % 4 == 3, 0]  # an id twice
        w[r % 6 == 5] = 0
        z[r % 9 == 7, V // 3:] = torch.finfo(dtype).min
        z[r % 11 == 8] = float("-inf")
        if T > 10:
            z[10, ids[10].clamp(0, V - 1)[0]] = float("-inf")
    return z, ids, tl, w


def _check(z, ids, tl, w, out, dtype, tau, dlogits=None):
    zz, ii, tt = f64(z), ids.cpu().numpy(), f64(tl)
    V = zz.shape[1]
    m, s, lp, p = oracle.row_softmax(zz, tau)
    q, lq = oracle.teacher_probs(ii, tt, V, tau)
    with np.errstate(invalid="ignore"):
        d = np.where(np.isneginf(zz), 0.0, np.abs(zz - np.where(np.isfinite(m), m, 0.0)[:, None]) / tau)
    serr = SUM + EXP + 2.0 ** -22 * (p * d).sum(axis=1)
    ls = np.abs(np.log(np.where(s > 0, s, 1.0)))
    lqa = np.where(q > 0, np.abs(lq), 0.0)
    qerr = SUM + EXP + 2.0 ** -21 * (1 + lqa.max(axis=1, keepdims=True))
    f32 = torch.float32
    if out is not None:
        loss, _, _ = oracle.distill_fwd(zz, ii, tt, tau)
        check("max", out["stats"][:, 0], m, f32, 0.0)
        check("sum", out["stats"][:, 1], s, f32, serr * s)
        dk = np.take_along_axis(d, np.clip(ii, 0, V - 1), axis=1)
        size = lqa + dk + ls[:, None]
        with np.errstate(over="ignore"):
            loss = np.where(np.isfinite(loss.astype(np.float32)), loss, loss.astype(np.float32))
        check("loss", out["loss"], loss, f32, (q * ((qerr + SUM + 2.0 ** -21) * size + qerr + serr[:, None])).sum(axis=1))
    if dlogits is not None:
        ref = oracle.distill_bwd(f64(w), zz, ii, tt, tau)
        part = p * (serr[:, None] + EXP + 2.0 ** -22 * d + 2.0 ** -21)
        qd = np.zeros_like(part)
        for k in range(ii.shape[1]):
            ok = (ii[:, k] >= 0) & (ii[:, k] < V)
            np.add.at(qd, (np.nonzero(ok)[0], ii[ok, k]), q[ok, k])
        part = part + qd * (qerr + 2.0 ** -21)
        check("dlogits", dlogits, ref, dtype, np.abs(f64(w))[:, None] / tau * part)


def _run(T, V, K, dtype, tau=1.0, masked=False, layout="dense", index=torch.int64, tdtype=None, seed=1):
    swg = _swg()
    z, ids, tl, w = _inputs(T, V, K, dtype, seed, masked, tdtype)
    zl, ids = strided(z, layout), ids.to(index)
    out = swg.distill_fwd(zl, ids, tl, temperature=tau)
    _check(z, ids, tl, w, out, dtype, tau)
    _check(z, ids, tl, w, None, dtype, tau, swg.distill_bwd(w, zl, ids, tl, out["stats"], temperature=tau))
    both = swg.distill_fwd_bwd(zl, ids, tl, w, temperature=tau)
    _check(z, ids, tl, w, both, dtype, tau, both["dlogits"])


SHAPES = [(1, 1, 1), (3, 2, 2), (5, 33, 8), (12, 1000, 20), (3, 4097, 64), (40, 8192, 128), (23, 50001, 50),
          (1, 131072, 64), (12, 131072, 20), (2, 300007, 30), (400, 515, 7), (2, 600, 1024), (4, 40, 64)]


@pytest.mark.parametrize("dtype", DTYPES, ids=NAME.get)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes(shape, dtype):
    _run(*shape, dtype)
    _run(*shape, dtype, tau=2.0, masked=True, index=torch.int32, tdtype=torch.float32, seed=2)


# more rows than there are clusters of blocks on the device, so that each takes several: rows of one block (of
# few and of many warps) and of two, four and eight, and more entries than are loaded ahead
MANY = [(2001, 1000, 20, torch.bfloat16), (1501, 8000, 64, torch.float16), (1000, 4100, 128, torch.float32),
        (701, 20000, 40, torch.bfloat16), (401, 50001, 50, torch.float16), (201, 131072, 64, torch.bfloat16),
        (151, 131075, 20, torch.float32), (601, 3001, 300, torch.bfloat16), (301, 12000, 700, torch.float16),
        (161, 40001, 1024, torch.bfloat16)]


@pytest.mark.parametrize("shape", MANY, ids=lambda s: "x".join(map(str, s[:3])) + "-" + NAME[s[3]])
def test_many_rows(shape):
    _run(*shape, tau=0.7, masked=True, seed=21)


@pytest.mark.parametrize("K", [9, 64, 200, 1024])
def test_ids_that_come_again(K):
    # every id several times, in one lane's entries and across lanes; absent ones in between
    for T, V, dtype in ((900, 3000, torch.bfloat16), (300, 40001, torch.float32)):
        z, ids, tl, w = _inputs(T, V, min(K, V), dtype, 22)
        g = torch.Generator(device="cuda")
        g.manual_seed(23)
        some = torch.randint(-1, V + 1, (T, max(2, K // 5)), generator=g, device="cuda")
        ids = some.gather(1, torch.randint(0, some.shape[1], (T, K), generator=g, device="cuda"))
        ids[: T // 3] = ids[: T // 3, :1]  # one id only
        out = _swg().distill_fwd_bwd(z, ids, tl, w)
        _check(z, ids, tl, w, out, dtype, 1.0, out["dlogits"])
        _check(z, ids, tl, w, None, dtype, 1.0, _swg().distill_bwd(w, z, ids, tl, out["stats"]))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", DTYPES, ids=NAME.get)
def test_layouts(dtype, layout):
    for V in (64, 1001, 9000, 40007):
        _run(13, V, 16, dtype, tau=0.7, masked=True, layout=layout)


@pytest.mark.parametrize("tdtype", DTYPES, ids=NAME.get)
def test_teacher_types(tdtype):
    _run(15, 3000, 12, torch.bfloat16, tdtype=tdtype, masked=True)


def test_student_equal_to_the_teacher():
    swg = _swg()
    z = torch.randn((6, 64), device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    ids = torch.stack([torch.randperm(64) for _ in range(6)]).cuda()
    out = swg.distill_fwd_bwd(z, ids, z.gather(1, ids), torch.ones(6, device="cuda"))
    assert out["loss"].abs().max() < 2.0 ** -18 and out["dlogits"].abs().max() < 2.0 ** -20


def test_weight_zero_hides_a_row():
    # a padding row's gradient is 0 whatever the row holds
    swg = _swg()
    z, ids, tl, w = _inputs(6, 900, 9, torch.float32, 3)
    z[2, 5], z[4] = float("nan"), float("inf")
    w[2] = w[4] = 0
    out = swg.distill_fwd_bwd(z, ids, tl, w)
    assert not out["dlogits"][2].any() and not out["dlogits"][4].any() and out["loss"][2].isnan()
    g = swg.distill_bwd(w, z, ids, tl, out["stats"])
    assert not g[2].any() and not g[4].any()
    w[2] = 1
    assert swg.distill_fwd_bwd(z, ids, tl, w)["dlogits"][2].isnan().all()
    fine = [0, 1, 3, 5]
    _check(z[fine], ids[fine], tl[fine], w[fine], {k: out[k][fine] for k in ("loss", "stats")}, torch.float32, 1.0,
           out["dlogits"][fine])


def test_gradient_by_differences():
    swg = _swg()
    z, ids, tl, w = _inputs(4, 50, 8, torch.float32, 4)
    z /= 3
    f = lambda z: float((swg.distill_fwd(z, ids, tl, temperature=1.5)["loss"].double() * w).sum())  # noqa: E731
    g = swg.distill_fwd_bwd(z, ids, tl, w, temperature=1.5)["dlogits"]
    e = 2.0 ** -7
    for seed in range(3):
        v = torch.sign(torch.randn(z.shape, generator=torch.Generator().manual_seed(seed))).cuda()
        diff = (f(z + e * v) - f(z - e * v)) / (2 * e)
        # truncation e^2 / 6 times a third derivative of order 10 a row, and the forward's fp32 error over e
        assert abs(diff - float((g.double() * v).sum())) <= 4 * 10 * e * e + 8 * 2.0 ** -20 / e


def test_in_place_and_guarded():
    swg = _swg()
    for V, dtype in ((4096, torch.bfloat16), (30001, torch.float16), (999, torch.float32), (140000, torch.bfloat16),
                     (500003, torch.float32)):
        z, ids, tl, w = _inputs(9, V, 33, dtype, 5)
        ids[:, 0], ids[:, 1] = 0, V - 1  # the row's ends
        gs = dict(loss=guarded((9,), torch.float32), stats=guarded((9, 2), torch.float32), dlogits=guarded((9, V), dtype))
        out = swg.distill_fwd_bwd(z, ids, tl, w, out={k: v.t for k, v in gs.items()})
        torch.cuda.synchronize()
        check_all(gs)
        _check(z, ids, tl, w, out, dtype, 1.0, out["dlogits"])
        want = out["dlogits"].clone()
        gs["dlogits"].t.zero_()
        _check(z, ids, tl, w, None, dtype, 1.0, swg.distill_bwd(w, z, ids, tl, out["stats"], dlogits=gs["dlogits"].t))
        check_all(gs)
        for layout in ("padded", "dense"):
            zi, zj = strided(z, layout).clone(memory_format=torch.preserve_format), strided(z, layout)
            if layout == "dense":
                zj = zj.clone()
            same = swg.distill_fwd_bwd(zj, ids, tl, w, out={"dlogits": zj})
            assert same["dlogits"].data_ptr() == zj.data_ptr()
            _check(z, ids, tl, w, same, dtype, 1.0, same["dlogits"])
            g = swg.distill_bwd(w, zi, ids, tl, out["stats"], dlogits=zi)
            _check(z, ids, tl, w, None, dtype, 1.0, g)
        shifted = strided(torch.zeros_like(z), "shifted")
        assert torch.equal(swg.distill_fwd_bwd(z, ids, tl, w, out={"dlogits": shifted})["dlogits"], want)


def test_offsets_past_32_bits():
    swg = _swg()
    T, V = 33000, 65544
    z = torch.empty((T, V), dtype=torch.bfloat16, device="cuda").normal_(0, 3, generator=torch.Generator("cuda").manual_seed(1))
    ids = (torch.arange(T, device="cuda").unsqueeze(1) * 7 + torch.arange(4, device="cuda") * 1000) % V
    tl = torch.randn((T, 4), device="cuda")
    w = torch.ones(T, device="cuda")
    rows = [0, 32763, 32764, T - 1]
    zr = z[rows].clone()
    out = swg.distill_fwd_bwd(z, ids, tl, w, out={"dlogits": z})
    _check(zr, ids[rows], tl[rows], w[rows], {k: out[k][rows] for k in ("loss", "stats")}, torch.bfloat16, 1.0,
           out["dlogits"][rows])


def test_reproducible_on_another_stream():
    swg = _swg()
    z, ids, tl, w = _inputs(300, 20011, 40, torch.bfloat16, 6)
    ids[:, 5] = ids[:, 3]
    a = swg.distill_fwd_bwd(z, ids, tl, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = swg.distill_fwd_bwd(z, ids, tl, w, stream=s)
    f = swg.distill_fwd(z, ids, tl, stream=s)
    g = swg.distill_bwd(w, z, ids, tl, b["stats"], stream=s)
    s.synchronize()
    assert all(torch.equal(a[k], b[k]) for k in a)
    _check(z, ids, tl, w, f, torch.bfloat16, 1.0, g)


def test_empty_and_refusals():
    swg = _swg()
    z, ids, tl, w = _inputs(4, 50, 6, torch.bfloat16, 1)
    out = swg.distill_fwd_bwd(z[:0], ids[:0], tl[:0], w[:0])
    assert out["loss"].shape == (0,) and out["dlogits"].shape == (0, 50)
    with pytest.raises(ValueError):
        swg.distill_fwd(z, ids[:3], tl)
    with pytest.raises(ValueError):
        swg.distill_fwd(z, ids, tl[:, :5])
    with pytest.raises(ValueError):
        swg.distill_fwd(z, ids.float(), tl)
    with pytest.raises(ValueError):
        swg.distill_fwd_bwd(z, ids, tl, w.double())
    with pytest.raises(swg.SwgError):
        swg.distill_fwd(z, ids[:, :0], tl[:, :0])
    with pytest.raises(swg.SwgError):
        swg.distill_fwd(z, ids, tl, temperature=0.0)
    with pytest.raises(swg.SwgError):
        swg.distill_fwd(z, ids.repeat(1, 200), tl.repeat(1, 200))
    with pytest.raises(swg.SwgError):  # missing weight
        swg.distill_fwd_bwd(z, ids, tl, None)
    with pytest.raises(swg.SwgError):  # the gradient over part of the logits
        swg.distill_fwd_bwd(z[:, :40], ids % 40, tl, w, out={"dlogits": z[:, 5:45]})
