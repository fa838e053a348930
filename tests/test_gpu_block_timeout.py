"""The timeout path of the bounded waits of the linear layer and of the norms between blocks: a producer that stops, or
a block that sends no sums (armed on the host by swg_inject_stall), lets the waits of the next launch run out. The status, guard bands around the outputs and the same call afterwards."""

import pytest
import torch

from ._block import check_linear_bwd, check_linear_fwd, check_norm_bwd, check_norm_fwd, linear_inputs, norm_inputs
from ._guard import check_all, guarded

pytestmark = pytest.mark.gpu
LIMIT = 1 << 20  # cycles, about half a millisecond
BF16 = torch.bfloat16


def _swg():
    import swiglu_ffn_backward_gb300 as swg
    return swg


def _expect_timeout(swg):
    status = None
    try:
        swg.swg_check()
    except swg.SwgError as e:  # not kept: its traceback would hold the test's tensors
        status = e.status
    assert status == 6  # SWG_ERR_TIMEOUT
    swg.swg_check()  # the status word was cleared


# few rows by clusters of eight blocks, with rings that wrap, and rows by blocks on their own
@pytest.mark.parametrize("M,K,N,entry", [(1, 4096, 256, 0), (1, 4096, 256, 2), (40, 16384, 128, 7), (256, 16384, 256, 5),
                                         (200, 512, 128, 0)])
def test_split_forward(M, K, N, entry):
    swg, t = _swg(), linear_inputs(M, K, N, BF16)
    g = {"y": guarded((M, N), BF16)}
    swg.swg_inject_stall(swg.SWG_INJECT_LINEAR_SPLIT, entry, LIMIT)
    swg.linear_fwd(t["x"], t["w"], out={"y": g["y"].t})
    _expect_timeout(swg)
    check_all(g)
    check_linear_fwd(t, swg.linear_fwd(t["x"], t["w"], out={"y": g["y"].t}), BF16, None)
    swg.swg_check()
    check_all(g)


@pytest.mark.parametrize("entry", [0, 3])
def test_split_backward(entry):
    # the armed launch is the first of the call, that of dw
    swg, t = _swg(), linear_inputs(4096, 128, 256, BF16)
    swg.swg_inject_stall(swg.SWG_INJECT_LINEAR_SPLIT, entry, LIMIT)
    swg.linear_bwd(t["dy"], t["x"], t["w"])
    _expect_timeout(swg)
    check_linear_bwd(t, swg.linear_bwd(t["dy"], t["x"], t["w"]), BF16, None)
    swg.swg_check()


@pytest.mark.parametrize("entry", [0, 1, 7, 20])
@pytest.mark.parametrize("residual", [False, True])
def test_pair_forward(entry, residual):
    # 128 tiles of sixteen blocks on 76 pairs, a ring of five stages: entry 7 follows a wait for a released slot, entry 20
    # lies in a pair's second tile
    swg, t = _swg(), linear_inputs(8192, 1024, 1024, BF16)
    r = t["residual"] if residual else None
    g = {"y": guarded((8192, 1024), BF16)}
    swg.swg_inject_stall(swg.SWG_INJECT_LINEAR, entry, LIMIT)
    swg.linear_fwd(t["x"], t["w"], residual=r, out={"y": g["y"].t})
    _expect_timeout(swg)
    check_all(g)
    check_linear_fwd(t, swg.linear_fwd(t["x"], t["w"], residual=r, out={"y": g["y"].t}), BF16, None, None, r)
    swg.swg_check()
    check_all(g)


@pytest.mark.parametrize("entry,residual", [(0, False), (3, True), (40, False)])
def test_wide_pair_forward(entry, residual):
    # wide tiles: 141 blocks of 64, a ring of four stages
    swg, t = _swg(), linear_inputs(2000, 9000, 4000, BF16)
    r = t["residual"] if residual else None
    g = {"y": guarded((2000, 4000), BF16)}
    swg.swg_inject_stall(swg.SWG_INJECT_LINEAR, entry, LIMIT)
    swg.linear_fwd(t["x"], t["w"], residual=r, out={"y": g["y"].t})
    _expect_timeout(swg)
    check_all(g)
    check_linear_fwd(t, swg.linear_fwd(t["x"], t["w"], residual=r, out={"y": g["y"].t}), BF16, None, None, r)
    swg.swg_check()
    check_all(g)


@pytest.mark.parametrize("entry", [0, 40])
def test_pair_backward(entry):
    # the armed launch is that of dw, cut into parts
    swg, t = _swg(), linear_inputs(70000, 512, 1024, BF16)
    swg.swg_inject_stall(swg.SWG_INJECT_LINEAR, entry, LIMIT)
    swg.linear_bwd(t["dy"], t["x"], t["w"])
    _expect_timeout(swg)
    check_linear_bwd(t, swg.linear_bwd(t["dy"], t["x"], t["w"]), BF16, None)
    swg.swg_check()


# rows shared by three to eight blocks, whole and ragged; many rows in rings, by blocks on their own (the entry is a
# ring's then) and by clusters
@pytest.mark.parametrize("M,N,row", [(30, 12288, 0), (30, 12288, 7), (9, 32768, 3), (12, 20001, 0), (12, 20001, 5),
                                     (2400, 4096, 0), (2400, 4096, 3), (2400, 4096, 5), (21000, 512, 2), (699, 12288, 200)])
def test_block_norm(M, N, row):
    swg, t = _swg(), norm_inputs(M, N, BF16, torch.float32, 3)
    kw = dict(gamma_post=t["gamma_post"], gamma_pre=t["gamma_pre"], gate=t["gate"])
    g = {"h": guarded((M, N), BF16), "y": guarded((M, N), BF16), "stats": guarded((M, 2), torch.float32)}
    swg.swg_inject_stall(swg.SWG_INJECT_BLOCK_NORM_FWD, row, LIMIT)
    swg.block_norm_fwd(t["u"], t["residual"], out={k: v.t for k, v in g.items()}, **kw)
    _expect_timeout(swg)
    check_all(g)
    out = swg.block_norm_fwd(t["u"], t["residual"], out={k: v.t for k, v in g.items()}, **kw)
    check_norm_fwd(t, out, BF16)
    gb = {"du": guarded((M, N), BF16), "dresidual": guarded((M, N), BF16), "dgamma_pre": guarded((N,), torch.float32)}
    swg.swg_inject_stall(swg.SWG_INJECT_BLOCK_NORM_BWD, row, LIMIT)
    args = (t["dy"], t["dh"], t["u"], out["h"], out["stats"])
    swg.block_norm_bwd(*args, out={k: v.t for k, v in gb.items()}, **kw)
    _expect_timeout(swg)
    check_all(gb)
    got = swg.block_norm_bwd(*args, out={k: v.t for k, v in gb.items()}, **kw)
    check_norm_bwd(t, out["h"], out["stats"], got, BF16, torch.float32, BF16)
    check_all(gb)
    swg.swg_check()
