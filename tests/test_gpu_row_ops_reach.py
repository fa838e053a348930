"""Rows that reach the less common branches of the vocabulary kernels (GPU): the search for the best alternatives where
a thread's table holds several stages a group, ties among them, rings that wrap within a row, and gradients written
over padded logits."""

import numpy as np
import pytest
import torch

import oracle

from ._row_ops import EXP, SUM, check, f64, strided

pytestmark = pytest.mark.gpu
BF16, F32, F16 = torch.bfloat16, torch.float32, torch.float16


def _swg():
    import swiglu_ffn_backward_gb300 as swg
    return swg


def _check_rows(z, out, k, rows):
    """The rows' statistics and their best logits by a stable sort: descending, equal ones by the lower index."""
    sub = f64(z[rows])
    m, s, lp, p = oracle.row_softmax(sub, 1.0)
    with np.errstate(invalid="ignore"):
        ed = np.where(p > 0, p * np.where(np.isfinite(sub), m[:, None] - sub, 0.0), 0.0).sum(axis=1)
    check("max", out["stats"][rows, 0], m, F32, 0.0)
    check("sum", out["stats"][rows, 1], s, F32, (SUM + EXP + 2.0 ** -22 * ed) * s)
    order = np.argsort(-sub, axis=1, kind="stable")[:, :k]
    np.testing.assert_array_equal(out["top_idx"][rows].cpu().numpy(), order)


# four warps and 16; one, two and more stages a group; fp32 above 32768 columns, 16-bit above 131072
@pytest.mark.parametrize("T,V,dtype", [(1000, 20001, F32), (950, 25500, F32), (300, 50001, F32), (200, 140001, BF16),
                                       (160, 262147, F16), (3, 300007, F32), (1, 1000003, BF16)],
                         ids=lambda v: str(v).replace("torch.", ""))
def test_ties_across_stages(T, V, dtype):
    swg = _swg()
    g = torch.Generator("cuda").manual_seed(81)
    z = torch.randint(-3, 3, (T, V), generator=g, device="cuda").to(dtype)
    if T > 3:
        z[1] = 1.5                                       # all equal
        z[2] = torch.arange(V, device="cuda") // 4096    # the best at the end, in runs that are equal
        z[3] = -(torch.arange(V, device="cuda") // 4096)
        z[T - 2] = float("-inf")
        z[T - 2, V - 5:] = 2.0                           # fewer than wanted
        z[T - 1, torch.arange(0, V, 512, device="cuda")] = 7.0
    rows = sorted({0, min(1, T - 1), min(2, T - 1), min(3, T - 1), T // 2, max(T - 2, 0), T - 1})
    for k in (1, 5, 32):
        _check_rows(z, swg.token_logprobs_fwd(z, top_k=k), k, rows)


@pytest.mark.parametrize("T,V,dtype", [(1000, 20001, F32), (300, 50001, F32), (200, 140001, BF16), (160, 262147, F16)],
                         ids=lambda v: str(v).replace("torch.", ""))
def test_random_rows_with_masks_across_stages(T, V, dtype):
    swg = _swg()
    g = torch.Generator("cuda").manual_seed(82)
    z = (torch.randn((T, V), generator=g, device="cuda") * 3).to(dtype)
    z[::3].masked_fill_(torch.rand(z[::3].shape, generator=g, device="cuda") > 0.05, float("-inf"))
    z[1::7, V // 2:] = torch.finfo(dtype).min
    z[5::50] = float("-inf")
    rows = [0, 1, 2, 3, 5, 8, T // 2, T - 2, T - 1]
    _check_rows(z, swg.token_logprobs_fwd(z, top_k=32), 32, rows)


# six stages of four warps hold 24576 16-bit logits: longer rows wrap the ring within a row
@pytest.mark.parametrize("T,V,dtype", [(1000, 32768, BF16), (1000, 50001, BF16), (1500, 131072, F16), (950, 40003, F32)],
                         ids=lambda v: str(v).replace("torch.", ""))
def test_distillation_loss_of_many_long_rows(T, V, dtype):
    swg = _swg()
    g = torch.Generator("cuda").manual_seed(83)
    z = (torch.randn((T, V), generator=g, device="cuda") * 2).to(dtype)
    drop = torch.rand((T // 4 + 1, V), generator=g, device="cuda") > 0.1
    z[::4].masked_fill_(drop[: z[::4].shape[0]], float("-inf"))
    ids = torch.randint(0, V, (T, 40), generator=g, device="cuda")
    ids[:, 3] = ids[:, 2]
    ids[::9, 5] = -1
    tl = torch.randn((T, 40), generator=g, device="cuda")
    out = swg.distill_fwd(z, ids, tl, temperature=1.5)
    rows = [0, 1, 4, 7, 8, 9, T // 2, T - 2, T - 1]
    zz = f64(z[rows])
    loss, m, s = oracle.distill_fwd(zz, ids[rows].cpu().numpy(), f64(tl[rows]), 1.5)
    check("max", out["stats"][rows, 0], m, F32, 0.0)
    check("sum", out["stats"][rows, 1], s, F32, (SUM + EXP + 2.0 ** -22 * 10) * s)
    # q, ln q and ln p are each off by some SUM and EXP; the terms are of the size of ln s and of d
    check("loss", out["loss"][rows], loss, F32, np.where(np.isfinite(loss), 4 * (SUM + EXP) * (1 + np.log(s) + 20), 0.0))


@pytest.mark.parametrize("V,dtype", [(4096, BF16), (30001, F16), (999, F32), (140000, BF16)],
                         ids=lambda v: str(v).replace("torch.", ""))
def test_gradients_over_padded_logits(V, dtype):
    swg = _swg()
    g = torch.Generator("cuda").manual_seed(84)
    T, K = 9, 33
    z = (torch.randn((T, V), generator=g, device="cuda") * 3).to(dtype)
    ids = torch.rand((T, V), generator=g, device="cuda").topk(K, dim=1).indices
    ids[:, 0], ids[:, 1] = 0, V - 1
    tl, w = torch.randn((T, K), generator=g, device="cuda"), torch.rand(T, generator=g, device="cuda")
    ref = oracle.distill_bwd(f64(w), f64(z), ids.cpu().numpy(), f64(tl), 1.0)
    scale = np.abs(f64(w))[:, None]
    st = swg.distill_fwd(z, ids, tl)["stats"]
    for alone in (True, False):
        zi = strided(z, "padded")
        assert zi.stride(0) > V
        pad = zi.as_strided((T - 1, zi.stride(0) - V), (zi.stride(0), 1), V)  # between the rows
        assert pad.isnan().all()
        if alone:
            got = swg.distill_bwd(w, zi, ids, tl, st, dlogits=zi)
        else:
            got = swg.distill_fwd_bwd(zi, ids, tl, w, out={"dlogits": zi})["dlogits"]
        assert got.data_ptr() == zi.data_ptr() and pad.isnan().all()
        check("dlogits", got, ref, dtype, 4 * (SUM + EXP + 2.0 ** -20) * scale)
