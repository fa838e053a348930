"""Argument checks of the linear layer and of the norms between blocks at the C ABI (fake, never-dereferenced
addresses: every case returns before any CUDA call)."""

import pytest

FAKE = 0x7f0000000000
STEP = 0x10000000


@pytest.fixture(scope="module")
def b():
    from swiglu_ffn_backward_gb300 import _binding
    return _binding


def _p(n):
    return [FAKE + i * STEP for i in range(n)]


def _with(args, change):
    args = list(args)
    for i, v in change.items():
        args[i] = v
    return args


def test_linear_fwd(b):
    f = b.lib.linear_fwd  # x w b residual y z M K N ldx ldr act dtype bdtype stream
    ok = _p(6) + [4, 16, 24, 16, 24, b.SWG_ACT_NONE, b.SWG_BF16, b.SWG_F32, None]
    x, w, bias, res, y, z = ok[:6]
    for change in ({6: -1}, {7: -8}, {8: -8}, {9: 8}, {10: 16}, {11: 3}, {11: -1}, {12: b.SWG_F32}, {12: 7},
                   {13: b.SWG_F16}, {4: x}, {4: w + 32}, {4: bias}, {5: y + 64}, {5: res}, {4: res + 16},
                   {4: res, 10: 32}):
        assert f(*_with(ok, change)) == b.SWG_ERR_PARAM_INVALID, change
    for i in (0, 1, 4):
        assert f(*_with(ok, {i: None})) == b.SWG_ERR_NULLPTR, i
    for change in ({7: 0}, {7: 12}, {8: 20}, {9: 20}, {10: 28}, {0: x + 8}, {1: w + 2}, {2: bias + 4}, {3: res + 8},
                   {4: y + 8}, {5: z + 2}, {6: 2 ** 31}, {7: 2 ** 31, 9: 2 ** 31}, {9: 2 ** 41}):
        assert f(*_with(ok, change)) == b.SWG_ERR_UNSUPPORTED, change
    assert f(*([None] * 6), 0, 16, 24, 16, 24, 0, b.SWG_F16, b.SWG_F16, None) == b.SWG_OK
    assert f(*([None] * 6), 4, 16, 0, 16, 24, 0, b.SWG_F16, b.SWG_F16, None) == b.SWG_OK


def test_linear_bwd(b):
    f = b.lib.linear_bwd  # dy x w z dx dw db M K N lddy ldx act flags dtype bdtype ws bytes stream
    need = b.lib.linear_bwd_workspace_size(4, 16, 24, 1)
    assert need > b.lib.linear_bwd_workspace_size(4, 16, 24, b.SWG_ACT_NONE) > 0
    assert b.lib.linear_bwd_workspace_size(0, 16, 24, 1) == 0 and b.lib.linear_bwd_workspace_size(4, 12, 24, 1) == 0
    ok = _p(7) + [4, 16, 24, 24, 16, 1, 0, b.SWG_F16, b.SWG_F16, FAKE + 9 * STEP, need, None]
    dy, x, w, z, dx, dw, db = ok[:7]
    for change in ({7: -1}, {8: -8}, {9: -8}, {10: 16}, {11: 8}, {12: 5}, {13: 1}, {13: b.SWG_ACCUMULATE | 4},
                   {14: b.SWG_F32}, {15: b.SWG_BF16}, {4: dy}, {5: w}, {5: x + 16}, {6: dw + 16}, {6: z}, {16: dx},
                   {16: w}):
        assert f(*_with(ok, change)) == b.SWG_ERR_PARAM_INVALID, change
    for i in (0, 1, 2, 3):
        assert f(*_with(ok, {i: None})) == b.SWG_ERR_NULLPTR, i
    for change in ({16: None}, {17: need - 1}):
        assert f(*_with(ok, change)) == b.SWG_ERR_WORKSPACE, change
    for change in ({8: 12}, {9: 20}, {10: 28}, {11: 20}, {0: dy + 8}, {4: dx + 8}, {6: db + 2}, {16: ok[16] + 8}):
        assert f(*_with(ok, change)) == b.SWG_ERR_UNSUPPORTED, change
    nothing = _with(ok, {4: None, 5: None, 6: None})
    assert f(*nothing) == b.SWG_OK


def test_block_norm_fwd(b):
    # u residual gamma_post gamma_pre gate h y stats M N G ldu ldr alpha eps flags dtype wdtype gdtype stream
    f = b.lib.block_norm_fwd
    both = b.SWG_NORM_POST | b.SWG_NORM_PRE
    ok = _p(8) + [4, 16, 2, 16, 16, 1.0, 1e-6, both, b.SWG_BF16, b.SWG_F32, b.SWG_BF16, None]
    u, res, gp, gn, gate, h, y, st = ok[:8]
    for change in ({8: -1}, {9: -1}, {10: -1}, {10: 3}, {10: 0}, {11: 15}, {12: 15}, {13: float("nan")},
                   {13: float("inf")}, {14: -1.0}, {14: float("nan")}, {15: 0}, {15: 4 | both}, {16: 3},
                   {17: b.SWG_F16}, {18: b.SWG_F16}, {15: b.SWG_NORM_POST}, {15: b.SWG_NORM_PRE}, {5: None},
                   {5: u}, {6: res + 32}, {7: y}, {6: gate}, {5: gp},
                   {1: None, 2: None, 4: None, 10: 0, 15: b.SWG_NORM_PRE},            # the plain norm has no h
                   {3: None, 15: b.SWG_NORM_POST}):                                   # no y without its norm
        assert f(*_with(ok, change)) == b.SWG_ERR_PARAM_INVALID, change
    for i in (0, 4, 6, 7):
        assert f(*_with(ok, {i: None})) == b.SWG_ERR_NULLPTR, i
    for change in ({0: u + 1}, {2: gp + 2}, {4: gate + 1}, {5: h + 1}, {7: st + 2}, {8: 2 ** 31}, {11: 2 ** 50},
                   {9: 2 ** 31, 11: 2 ** 31, 12: 2 ** 31}):
        assert f(*_with(ok, change)) == b.SWG_ERR_UNSUPPORTED, change
    assert f(*([None] * 8), 0, 16, 2, 16, 16, 1.0, 1e-6, both, 0, 0, 0, None) == b.SWG_OK
    assert f(*([None] * 8), 4, 0, 2, 0, 0, 1.0, 1e-6, both, 0, 0, 0, None) == b.SWG_OK


def test_block_norm_bwd(b):
    # dy dh u h stats gamma_post gamma_pre gate du dres dgamma_post dgamma_pre dgate M N G lddy lddh ldu ldh alpha flags
    # dtype wdtype gdtype ws bytes stream
    f = b.lib.block_norm_bwd
    both = b.SWG_NORM_POST | b.SWG_NORM_PRE
    size = b.lib.block_norm_bwd_workspace_size
    need = size(4, 16, 2)
    assert need > 0 and size(0, 16, 0) == 0 and size(4, 16, 3) == 0 and size(-1, 16, 0) == 0
    ok = _p(13) + [4, 16, 2, 16, 16, 16, 16, 1.0, both, b.SWG_F16, b.SWG_F32, b.SWG_F16, FAKE + 15 * STEP, need, None]
    dy, dh, u, h, st, gp, gn, gate, du, dres, dgp, dgn, dgate = ok[:13]
    for change in ({13: -1}, {14: -1}, {15: 3}, {15: 0}, {16: 8}, {17: 8}, {18: 8}, {19: 8}, {20: float("inf")},
                   {21: 0}, {21: 8}, {22: 3}, {23: b.SWG_BF16}, {24: b.SWG_BF16}, {21: b.SWG_NORM_POST},
                   {21: b.SWG_NORM_PRE}, {8: dy}, {9: dh}, {9: du + 16}, {12: gate}, {25: u}, {25: dgn}):
        assert f(*_with(ok, change)) == b.SWG_ERR_PARAM_INVALID, change
    for i in (0, 2, 3, 4, 7, 8):
        assert f(*_with(ok, {i: None})) == b.SWG_ERR_NULLPTR, i
    only_post = {0: None, 3: None, 6: None, 11: None, 21: b.SWG_NORM_POST, 1: None}
    assert f(*_with(ok, only_post)) == b.SWG_ERR_NULLPTR  # dh is the only gradient then
    for change in ({25: None}, {26: need - 1}, {25: ok[25] + 8}):
        assert f(*_with(ok, change)) == b.SWG_ERR_WORKSPACE, change
    for change in ({0: dy + 1}, {5: gp + 2}, {8: du + 1}, {12: dgate + 1}, {13: 2 ** 31}, {18: 2 ** 50}):
        assert f(*_with(ok, change)) == b.SWG_ERR_UNSUPPORTED, change
    assert f(*([None] * 13), 0, 16, 0, 16, 16, 16, 16, 1.0, both, 0, 0, 0, None, 0, None) == b.SWG_OK


def test_kernels_can_be_armed(b):
    for kernel in (b.SWG_INJECT_LINEAR_SPLIT, b.SWG_INJECT_LINEAR, b.SWG_INJECT_BLOCK_NORM_FWD,
                   b.SWG_INJECT_BLOCK_NORM_BWD):
        assert b.lib.swg_inject_stall(kernel, 3, 1 << 20) == b.SWG_OK
        assert b.lib.swg_inject_stall(kernel, -1, 1 << 20) == b.SWG_ERR_PARAM_INVALID
    assert b.lib.swg_inject_stall(0, 0, 0) == b.SWG_OK


def test_binding_requires_cuda_tensors(b):
    import torch
    t, w = torch.zeros(4, 8, dtype=torch.float16), torch.zeros(8, 16, dtype=torch.float16)
    for call in (lambda: b.linear_fwd(t, w), lambda: b.linear_bwd(t, t, w), lambda: b.block_norm_fwd(t),
                 lambda: b.block_norm_bwd(t, t, t, t, t)):
        with pytest.raises(TypeError):
            call()
