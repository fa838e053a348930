"""The linear layer's weight gradient over many rows of factors of one sign (GPU).

The tensor cores cut off what an addition to an accumulator leaves below fp32. For factors of one sign the running sum
grows evenly, so that n additions lose at most n / 2 2^-23 of it. One addition is made for every four rows (the slope that
long chains show), and an accumulator takes 32768 rows: 4096 2^-23 = 2^-11, beside the rounding of the output and the fp32
sums of the parts (64 in sequence, twice: 2^-17)."""

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


# few columns, where the reduction is all there is to share out, and more tiles than pairs of SMs, which are not cut for that
@pytest.mark.parametrize("M,K,N", [(4194304, 64, 64), (1048576, 128, 72), (4000000, 8, 136), (400000, 1536, 1792)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_like_terms_do_not_drift(M, K, N, dtype):
    import swiglu_ffn_backward_gb300 as swg
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty((M, K), device="cuda", dtype=dtype).uniform_(0.05, 0.15, generator=g)
    dy = torch.empty((M, N), device="cuda", dtype=dtype).uniform_(0.005, 0.015, generator=g)
    got = swg.linear_bwd(dy, x, None, need_dx=False, bias=False)["dw"]
    swg.swg_check()
    cols = min(N, 64)
    want = torch.zeros((K, cols), device="cuda", dtype=torch.float64)
    for r in range(0, M, 65536):
        want += x[r:r + 65536].double().t() @ dy[r:r + 65536, :cols].double()
    err = float(((got[:, :cols].double() - want) / want).abs().max())
    assert err <= torch.finfo(dtype).eps / 2 + 2.0 ** -11 + 2.0 ** -17
    # and added to what is there
    old = torch.full_like(got, 3.0)
    added = swg.linear_bwd(dy, x, None, need_dx=False, bias=False, accumulate=True, out={"dw": old})["dw"]
    err = float(((added[:, :cols].double() - 3.0 - want) / (want + 3.0)).abs().max())
    assert err <= torch.finfo(dtype).eps / 2 + 2.0 ** -11 + 2.0 ** -17
