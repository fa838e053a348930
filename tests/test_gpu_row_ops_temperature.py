"""Temperatures at the ends of the range that the row-wise operators take (GPU)."""

import numpy as np
import pytest
import torch

import oracle

from ._row_ops import f64

pytestmark = pytest.mark.gpu


# the smallest whose reciprocal is in range (both are subnormal numbers), ordinary ones, the largest
@pytest.mark.parametrize("tau", [3.4e-39, 4.2e-39, 1e-38, 1e-20, 1e20, 3e38])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_extreme_temperatures(tau, dtype):
    import swiglu_ffn_backward_gb300 as swg
    tau = float(np.float32(tau))
    T, V, K = 5, 3000, 7
    g = torch.Generator("cuda").manual_seed(61)
    z = torch.randn((T, V), generator=g, device="cuda").to(dtype)
    ids = torch.rand((T, V), generator=g, device="cuda").topk(K, dim=1).indices
    tl = torch.randn((T, K), generator=g, device="cuda")
    # student and teacher agree on the best token; in row 1 two entries are equally good, in row 2 all logits are equal
    r = torch.arange(T, device="cuda")
    z[r, ids[:, 0]], tl[:, 0] = 9.0, 9.0
    z[1, ids[1, 1]], tl[1, 1] = 9.0, 9.0
    z[2], tl[2] = 0.0, 0.0
    w = torch.full((T,), tau, device="cuda")  # the gradient's factor 1 / tau leaves the range of fp32 otherwise
    loss, m, s = oracle.distill_fwd(f64(z), ids.cpu().numpy(), f64(tl), tau)
    ref = oracle.distill_bwd(f64(w), f64(z), ids.cpu().numpy(), f64(tl), tau)
    out = swg.distill_fwd_bwd(z, ids, tl, w, temperature=tau)
    alone = swg.distill_bwd(w, z, ids, tl, swg.distill_fwd(z, ids, tl, temperature=tau)["stats"], temperature=tau)
    np.testing.assert_allclose(f64(out["loss"]), loss, rtol=2.0 ** -16, atol=2.0 ** -16)
    np.testing.assert_allclose(f64(out["stats"]), np.stack([m, s], axis=1), rtol=2.0 ** -16)
    for d in (out["dlogits"], alone):
        np.testing.assert_allclose(f64(d), ref, rtol=2.0 ** -7, atol=2.0 ** -14)
    lp = swg.token_logprobs_fwd(z, ids[:, 0], top_k=3, temperature=tau)
    lref = oracle.token_logprobs_fwd(f64(z), ids[:, 0].cpu().numpy(), 3, tau)
    np.testing.assert_allclose(f64(lp["logp"]), lref["logp"], rtol=2.0 ** -16, atol=2.0 ** -16)
    np.testing.assert_allclose(f64(lp["entropy"]), lref["entropy"], rtol=2.0 ** -16, atol=2.0 ** -16)
    np.testing.assert_array_equal(lp["top_idx"].cpu().numpy(), lref["top_idx"])
