"""The linear layer's inputs off a 16-byte boundary, as parameters in one flat buffer are: all are taken alike (GPU)."""

import pytest
import torch

from ._block import linear_inputs

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _shifted(t, by):
    """t's values in a dense tensor `by` elements behind a 16-byte boundary."""
    buf = torch.zeros(t.numel() + by, dtype=t.dtype, device="cuda")
    buf[by:] = t.flatten()
    got = buf[by:].view(t.shape)
    assert got.data_ptr() % 16 and got.is_contiguous()
    return got


@pytest.mark.parametrize("name", ["x", "w", "b", "b in fp32", "residual", "dy", "z"])
@pytest.mark.parametrize("M", [3, 600])
def test_an_input_off_the_boundary(name, M):
    import swiglu_ffn_backward_gb300 as swg
    t = linear_inputs(M, 72, 136, BF16, seed=81)
    if name == "b in fp32":
        name, t["b"] = "b", t["b"].float()
    fwd = lambda: swg.linear_fwd(t["x"], t["w"], t["b"], act="gelu", residual=t["residual"], save_z=True)  # noqa: E731
    bwd = lambda: swg.linear_bwd(t["dy"], t["x"], t["w"], z=t["z"], act="gelu")  # noqa: E731
    want, back = fwd(), bwd()
    t[name] = _shifted(t[name], 1)
    got, gback = fwd(), bwd()
    assert all(torch.equal(got[k], want[k]) for k in want) and all(torch.equal(gback[k], back[k]) for k in back)
    # and on a stream of its own: the copy is made there
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    on = swg.linear_fwd(t["x"], t["w"], t["b"], act="gelu", residual=t["residual"], save_z=True, stream=s)
    s.synchronize()
    assert all(torch.equal(on[k], want[k]) for k in want)
    swg.swg_check()


def test_an_output_off_the_boundary_is_refused():
    import swiglu_ffn_backward_gb300 as swg
    t = linear_inputs(4, 16, 24, BF16, seed=83)
    with pytest.raises(swg.SwgError):
        swg.linear_fwd(t["x"], t["w"], out={"y": torch.empty(97, device="cuda", dtype=BF16)[1:].view(4, 24)})
    with pytest.raises(swg.SwgError):
        swg.linear_bwd(t["dy"], t["x"], t["w"], out={"dw": torch.empty(16 * 24 + 1, device="cuda", dtype=BF16)[1:].view(16, 24)})
    swg.swg_check()
