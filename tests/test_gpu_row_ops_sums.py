"""Long sums of the row-wise operators (GPU): terms that are all alike, whose roundings go the same way, so that an
accumulator that takes them one after the other is off by its length. The bounds are those of _row_ops.py, which
hold for some 100 terms in sequence. Rows are shared (a stride of 0), so that many of them take no memory."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle

from ._row_ops import EXP, SUM, check, f64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _swg():
    import swiglu_ffn_backward_gb300 as swg
    return swg


# one group of threads a block and two, several small ones, ragged rows, rows shared by a cluster, and rows read again
ROWS = [(264000, 8192, BF16), (264000, 4096, BF16), (200000, 4096, F32), (2150000, 64, BF16), (2150000, 200, F32),
        (300000, 4001, BF16), (300000, 1001, F32), (60000, 12288, BF16), (60000, 16381, F32), (20000, 70001, BF16)]


@pytest.mark.parametrize("M,N,dtype", ROWS, ids=lambda v: str(v).replace("torch.", ""))
def test_weight_gradients_of_many_like_rows(M, N, dtype):
    swg = _swg()
    g = torch.Generator(device="cuda")
    g.manual_seed(41)
    x = torch.randn((1, N), generator=g, device="cuda").to(dtype)
    dy = torch.full((1, N), 1 / 3, device="cuda").to(dtype)
    gamma = torch.ones(N, device="cuda")
    st = swg.layer_norm_fwd(x, gamma)["stats"]
    _, dgamma, dbeta = swg.layer_norm_bwd(dy.expand(M, N), x.expand(M, N), st.expand(M, 2), gamma=gamma)
    h, d, s = f64(x), f64(dy), f64(st)
    xhat = (h - s[:, :1]) * s[:, 1:]
    xerr = 2.0 ** -23 * (np.abs(h) + np.abs(s[:, :1])) * s[:, 1:]
    check("dgamma", dgamma, M * (d * xhat)[0], F32, M * (np.abs(d) * (SUM * np.abs(xhat) + 2 * xerr))[0])
    check("dbeta", dbeta, M * d[0], F32, SUM * M * np.abs(d[0]))


# every number of threads that a group may have, with more rows than it takes in one sequence
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["float32", "bfloat16"])
@pytest.mark.parametrize("shift", [0, 3], ids=["whole", "ragged"])
def test_weight_gradients_of_many_rows_by_any_group(dtype, shift):
    swg = _swg()
    g = torch.Generator(device="cuda")
    g.manual_seed(42)
    vec = 16 // dtype.itemsize
    for n in (4, 12, 30, 40, 90, 150, 200, 250, 300, 370, 440, 500, 560, 630, 700, 760, 820, 890, 950, 1000, 1010):
        N = n * vec + shift
        M = min(45000, 2 ** 30 // N) if n > 100 else 400000
        x = torch.randn((1, N), generator=g, device="cuda").to(dtype)
        dy = torch.randn((1, N), generator=g, device="cuda").to(dtype)
        st = swg.layer_norm_fwd(x)["stats"]
        dx, dgamma, dbeta = swg.layer_norm_bwd(dy.expand(M, N), x.expand(M, N), st.expand(M, 2),
                                               gamma=torch.ones(N, device="cuda"))
        h, d, s = f64(x), f64(dy), f64(st)
        xhat = (h - s[:, :1]) * s[:, 1:]
        xerr = 2.0 ** -23 * (np.abs(h) + np.abs(s[:, :1])) * s[:, 1:]
        check(f"dgamma {N}", dgamma, M * (d * xhat)[0], F32, M * (np.abs(d) * (SUM * np.abs(xhat) + 2 * xerr))[0])
        check(f"dbeta {N}", dbeta, M * d[0], F32, SUM * M * np.abs(d[0]))
        assert torch.equal(dx[M - 1], dx[0]) and torch.equal(dx[M // 2], dx[0]) or shift


FIRST_CALL = """
import torch
import swiglu_ffn_backward_gb300 as swg
N = {n}
x = torch.randn((1, N), device="cuda").bfloat16()
st = swg.layer_norm_fwd(x)["stats"]
swg.layer_norm_bwd(x.expand(60000, N), x.expand(60000, N), st.expand(60000, 2))
torch.cuda.synchronize()
"""


@pytest.mark.parametrize("n", [2960, 2965, 2500, 8000])
def test_first_call_of_a_process_with_many_rows(n):
    # the sums' place in shared memory is just what a kernel has without asking (2960, 2965), or more
    subprocess.run([sys.executable, "-c", FIRST_CALL.format(n=n)], check=True, cwd=ROOT, timeout=200)


# a row's first logits are 0, its largest, the others the background, so that every warp of a block has met the
# maximum before the terms that are all alike; 2^-x of a background is no short fraction
BACKGROUND = (-0.3125, -0.75, -1.0, -1.375, -2.25)
FIRST = 17000


def _like_rows(V, dtype):
    """[len(BACKGROUND), V] logits; the sums s of exp(z) and sum p |z| in fp64."""
    z = torch.tensor(BACKGROUND, device="cuda").unsqueeze(1).repeat(1, V).to(dtype)
    z[:, :FIRST] = 0
    e = np.exp(np.asarray(BACKGROUND))
    s = FIRST + (V - FIRST) * e
    return z, s, (V - FIRST) * e * -np.asarray(BACKGROUND) / s


@pytest.mark.parametrize("T,V,dtype", [(1000, 32768, BF16), (1000, 131072, BF16), (1000, 262144, BF16), (1000, 262147, F32),
                                       (1000, 2000003, BF16), (200, 2000003, BF16), (1, 4000003, F32)],
                         ids=lambda v: str(v).replace("torch.", ""))
def test_distillation_of_like_logits(T, V, dtype):
    swg = _swg()
    z, s, ed = _like_rows(V, dtype)
    ids, tl = torch.full((T, 1), V - 1, device="cuda"), torch.zeros((T, 1), device="cuda")
    for r in range(len(BACKGROUND)):
        out = swg.distill_fwd(z[r: r + 1].expand(T, V), ids, tl)
        rel = SUM + EXP + 2.0 ** -22 * ed[r]
        check("sum", out["stats"][:, 1], np.full(T, s[r]), F32, rel * s[r])
        loss = np.log(s[r]) - BACKGROUND[r]
        check("loss", out["loss"], np.full(T, loss), F32, rel + 2.0 ** -22 * (np.log(s[r]) + 3))


@pytest.mark.parametrize("T,V,dtype", [(1000, 51000, BF16), (1000, 25500, F32), (200, 131072, BF16), (200, 1000003, BF16),
                                       (200, 1000003, F32), (1, 4000003, BF16)], ids=lambda v: str(v).replace("torch.", ""))
def test_log_probabilities_of_like_logits(T, V, dtype):
    swg = _swg()
    z, s, ed = _like_rows(V, dtype)
    t = torch.full((T,), V - 1, device="cuda")
    for r in range(len(BACKGROUND)):
        out = swg.token_logprobs_fwd(z[r: r + 1].expand(T, V), t, top_k=2)
        rel, ls = SUM + EXP + 2.0 ** -22 * ed[r], np.log(s[r])
        check("sum", out["stats"][:, 1], np.full(T, s[r]), F32, rel * s[r])
        check("logp", out["logp"], np.full(T, BACKGROUND[r] - ls), F32, rel + 2.0 ** -22 * (ls + 3))
        check("entropy", out["entropy"], np.full(T, ls + ed[r]), F32, 2 * rel * (1 + ed[r]) + 2.0 ** -22 * (ls + ed[r]))
        assert (out["top_idx"] == torch.tensor([0, 1], device="cuda")).all()


@pytest.mark.parametrize("N,dtype", [(300007, BF16), (4000003, F32), (4000003, BF16)],
                         ids=lambda v: str(v).replace("torch.", ""))
def test_layer_norm_of_long_like_rows(N, dtype):
    # rows read again: a constant with a few other elements, and a gradient that is all alike
    swg = _swg()
    x = torch.full((3, N), 0.45, device="cuda")
    x[0, ::1000], x[1] = 0.5, 0.1
    x[1, ::7] = 0.15
    x[2] += torch.randn(N, generator=torch.Generator("cuda").manual_seed(2), device="cuda")
    x = x.to(dtype)
    out = swg.layer_norm_fwd(x)
    y, mu, rstd, h = oracle.layer_norm_fwd(f64(x), None, None, 1e-5)
    top = np.abs(h).max(axis=1)
    check("mean", out["stats"][:, 0], mu, F32, SUM * top)
    var_err = 2 * SUM + (SUM * top * rstd) ** 2 + 2.0 ** -22 * top * rstd
    check("rstd", out["stats"][:, 1], rstd, F32, rstd * var_err)
    dy = torch.full((1, N), 0.1, device="cuda").to(dtype).expand(3, N)
    dx, _, dbeta = swg.layer_norm_bwd(dy, x, out["stats"])
    st, d = f64(out["stats"]), f64(dy)
    rdx, _, rdb = oracle.layer_norm_bwd(d, h, st[:, 0], st[:, 1], None)
    xhat = np.abs((h - st[:, :1]) * st[:, 1:])
    xerr = 2.0 ** -23 * (np.abs(h) + np.abs(st[:, :1])) * st[:, 1:]
    mg, mgx = d.mean(axis=1, keepdims=True), (d * (xhat + xerr)).mean(axis=1, keepdims=True)
    part = st[:, 1:] * (2.0 ** -22 * d + SUM * mg + (SUM + 2.0 ** -22) * (xhat + xerr) * mgx + xerr * mgx
                        + xhat * (d * xerr).mean(axis=1, keepdims=True)) + 2.0 ** -23 * np.abs(rdx)
    check("dx", dx, rdx, dtype, part)
    check("dbeta", dbeta, rdb, dtype, SUM * np.abs(d).sum(axis=0))


@pytest.mark.parametrize("N", [520, 70001, 300007])
def test_infinite_and_nan_elements_of_long_rows(N):
    swg = _swg()
    x = torch.randn((5, N), generator=torch.Generator("cuda").manual_seed(3), device="cuda")
    clean = swg.layer_norm_fwd(x)
    x[0, N // 2], x[1, 7], x[2, N - 1], x[3, 0], x[3, N - 1] = (float(v) for v in ("inf", "-inf", "nan", "inf", "-inf"))
    out = swg.layer_norm_fwd(x)
    mean = out["stats"][:, 0].tolist()
    assert mean[0] == float("inf") and mean[1] == float("-inf") and mean[2] != mean[2] and mean[3] != mean[3]
    assert out["y"][:4].isnan().all() and torch.equal(out["y"][4], clean["y"][4])
