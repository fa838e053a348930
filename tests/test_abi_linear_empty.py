"""The linear layer's backward without input columns at the C ABI: K = 0, for the bias's gradient alone (fake,
never-dereferenced addresses: every case returns before any CUDA call)."""

import pytest

FAKE, STEP = 0x7f0000000000, 0x10000000


@pytest.fixture(scope="module")
def b():
    from swiglu_ffn_backward_gb300 import _binding
    return _binding


@pytest.mark.parametrize("act", ["SWG_ACT_NONE", "gelu"])
@pytest.mark.parametrize("M", [4, 5000])
def test_the_size_that_is_asked_for_is_enough(b, act, M):
    # a workspace of the query's size is not refused: the call goes on to what is checked behind it
    act = b.SWG_ACT_NONE if act == "SWG_ACT_NONE" else b.SWG_ACT[act]
    need = b.lib.linear_bwd_workspace_size(M, 0, 24, act)
    assert 0 < need <= b.lib.linear_bwd_workspace_size(M, 8, 24, act)
    dy, z, db, ws = (FAKE + i * STEP for i in range(4))
    call = lambda ws, size: b.lib.linear_bwd(dy, None, None, z, None, None, db, M, 0, 24, 24, 0, act, 0, b.SWG_BF16,  # noqa: E731
                                             b.SWG_BF16, ws, size, None)
    assert call(ws, need - 1) == b.SWG_ERR_WORKSPACE
    assert call(db, need) == b.SWG_ERR_PARAM_INVALID  # a workspace of enough bytes, over the output


@pytest.mark.gpu
def test_gradient_of_the_bias():
    import torch
    import swiglu_ffn_backward_gb300 as swg
    dy = torch.randn((700, 24), device="cuda").bfloat16()
    x, w = torch.empty((700, 0), device="cuda", dtype=dy.dtype), torch.empty((0, 24), device="cuda", dtype=dy.dtype)
    got = swg.linear_bwd(dy, x, w)
    assert got["dx"].shape == (700, 0) and got["dw"].shape == (0, 24)
    assert torch.equal(got["db"], swg.linear_bwd(dy, None, None, need_dx=False, need_dw=False)["db"])
    swg.swg_check()
