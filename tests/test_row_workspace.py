"""The workspace of layer norm's backward: as much as is written, and no more than a few rows of column sums for each
SM. The sizes are host arithmetic (no GPU); the GPU test runs calls on guarded workspaces of exactly that size."""

import pytest
import torch

from ._guard import check_all, guarded, workspace


def _size(M, N):
    from swiglu_ffn_backward_gb300 import _binding as b
    return b.lib.layer_norm_bwd_workspace_size(M, N)


def test_sizes_follow_what_is_written():
    row = lambda N: 2 * 4 * N  # noqa: E731  (dgamma's and dbeta's sums)
    for M in (1, 40, 63):
        for N in (1, 8, 1000, 4096, 9001, 70001):
            assert _size(M, N) == M * row(N)
    assert _size(16384, 4096) <= 2.2 * 152 * row(4096)
    assert _size(16384, 8192) <= 2.2 * 152 * row(8192)
    assert _size(3000, 12288) <= 112 * row(12288)       # clusters of three blocks
    assert _size(3000, 65536) == 64 * row(65536)
    assert _size(3000, 70001) == _size(10 ** 6, 70001) == 64 * row(70001)
    assert _size(2 ** 30, 2 ** 30) == 64 * row(2 ** 30)
    last = 1024
    for N in (8, 256, 257, 1000, 8192, 8193, 12288, 20000, 65536, 65537, 10 ** 6):
        rows = _size(10 ** 6, N) // row(N)
        assert 64 <= rows <= last
        last = rows


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(100000, 8), (30000, 61), (20000, 256), (302, 4096), (303, 4001), (5000, 264),
                                 (5000, 4096), (3000, 8192), (3000, 8185), (500, 8200), (500, 12288), (300, 32768),
                                 (300, 65536), (200, 65537), (100, 70001)], ids=lambda v: str(v))
def test_calls_stay_inside(M, N, dtype):
    import swiglu_ffn_backward_gb300 as swg
    g = torch.Generator("cuda").manual_seed(71)
    x, dy = (torch.randn((M, N), generator=g, device="cuda").to(dtype) for _ in range(2))
    st = swg.layer_norm_fwd(x)["stats"]
    gs = dict(ws=workspace(_size(M, N)), dx=guarded((M, N), dtype), dgamma=guarded((N,), dtype),
              dbeta=guarded((N,), dtype))
    swg.layer_norm_bwd(dy, x, st, dx=gs["dx"].t, dgamma=gs["dgamma"].t, dbeta=gs["dbeta"].t, workspace=gs["ws"].t)
    torch.cuda.synchronize()
    check_all(gs)
    want = dy.double().sum(dim=0)
    bound = 2.0 ** -16 * dy.double().abs().sum(dim=0) + (2.0 ** -8 if dtype is torch.bfloat16 else 0.0) * want.abs()
    assert ((gs["dbeta"].t.double() - want).abs() <= bound).all()
