"""The norms between blocks at the edges of what the kernels plan for: outputs that lie on their elements' alignment only, as
slices of a flat buffer do, and rows that do not fill the chunks whose column sums are taken together (GPU)."""

import pytest
import torch

from ._block import check_norm_bwd, norm_inputs
from ._guard import check_all, guarded, workspace

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _swg():
    import swiglu_ffn_backward_gb300 as swg
    return swg


# a gate for each row, fp32: sizes of the rings (blocks by themselves, clusters), of rows in registers, shared rows and
# rows of any length, with every other tensor on a 16-byte boundary
@pytest.mark.parametrize("M,N,dtype", [(10000, 132, F32), (2500, 1024, F32), (1300, 4096, BF16), (10000, 264, F16), (700, 8192, F32),
                                       (700, 12288, BF16), (40, 1024, F32), (40, 264, BF16), (50, 64, BF16), (9, 12288, F32),
                                       (9, 16384, BF16), (3, 70000, F32)])
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_gradient_of_an_fp32_gate_for_each_row(M, N, dtype, shift):
    swg, t = _swg(), norm_inputs(M, N, dtype, F32, M, F32)
    kw = dict(gamma_post=t["gamma_post"], gamma_pre=t["gamma_pre"], gate=t["gate"])
    out = swg.block_norm_fwd(t["u"], t["residual"], **kw)
    g = {"dgate": guarded((M, N), F32, offset_elems=shift), "du": guarded((M, N), dtype)}
    got = swg.block_norm_bwd(t["dy"], t["dh"], t["u"], out["h"], out["stats"], out={k: v.t for k, v in g.items()}, **kw)
    swg.swg_check()
    check_all(g)
    check_norm_bwd(t, out["h"], out["stats"], got, dtype, F32, F32)


@pytest.mark.parametrize("dtype,gdtype", [(BF16, BF16), (BF16, F32), (F32, F32)])
def test_gradient_of_a_shared_gate(dtype, gdtype):
    # its elements are stored one by one
    swg, t = _swg(), norm_inputs(2400, 4096, dtype, F32, 6, gdtype)
    kw = dict(gamma_post=t["gamma_post"], gamma_pre=t["gamma_pre"], gate=t["gate"])
    out = swg.block_norm_fwd(t["u"], t["residual"], **kw)
    want = swg.block_norm_bwd(t["dy"], t["dh"], t["u"], out["h"], out["stats"], **kw)
    g = {"dgate": guarded((6, 4096), gdtype, offset_elems=1)}
    got = swg.block_norm_bwd(t["dy"], t["dh"], t["u"], out["h"], out["stats"], out={"dgate": g["dgate"].t}, **kw)
    swg.swg_check()
    check_all(g)
    assert all(torch.equal(got[k], want[k]) for k in want)


# ragged rows in rings whose chunks are not all of one length, or have no rows: one gate row for all, and gate rows of fewer
# rows than there are offsets within 16 bytes
@pytest.mark.parametrize("M,N,gates,dtype,gdtype", [(60001, 515, 1, BF16, F32), (20000, 1001, 10000, BF16, BF16),
                                                    (21000, 515, 7000, F16, F32), (9800, 2047, 1400, F32, F32)])
def test_gates_of_chunks_without_rows(M, N, gates, dtype, gdtype):
    swg, t = _swg(), norm_inputs(M, N, dtype, F32, gates, gdtype)
    kw = dict(gamma_post=t["gamma_post"], gamma_pre=t["gamma_pre"], gate=t["gate"])
    out = swg.block_norm_fwd(t["u"], t["residual"], **kw)
    ws = workspace(swg.block_norm_bwd_workspace_size(M, N, gates))
    got = swg.block_norm_bwd(t["dy"], t["dh"], t["u"], out["h"], out["stats"], workspace=ws.t, **kw)
    swg.swg_check()
    ws.check("workspace")
    check_norm_bwd(t, out["h"], out["stats"], got, dtype, F32, gdtype)
