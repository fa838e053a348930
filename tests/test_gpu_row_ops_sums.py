"""Long sums of the row-wise operators (GPU): terms that are all alike, whose roundings go the same way, so that an
accumulator that takes them one after the other is off by its length. The bounds are those of _row_ops.py, which
hold for some 100 terms in sequence. Rows are shared (a stride of 0), so that many of them take no memory."""

import numpy as np
import pytest
import torch

from ._row_ops import SUM, check, f64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


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
