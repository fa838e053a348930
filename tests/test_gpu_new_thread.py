"""Calls from a host thread that has made no CUDA call before (a server's worker, a thread that prefetches): the kernels
whose operands come by tensor maps, with every output given, so that the call is the thread's first (GPU)."""

import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _swg():
    import swiglu_ffn_backward_gb300 as swg
    return swg


def _in_new_thread(call):
    """The result of a call in a thread of its own."""
    got = []

    def run():
        try:
            got.append((call(), None))
        except Exception as e:  # handed to the caller's thread
            got.append((None, f"{type(e).__name__}: {e}"))

    torch.cuda.synchronize()
    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    out, error = got[0]
    assert error is None, error
    return out


def _inputs(M, K, N):
    g = torch.Generator(device="cuda").manual_seed(41)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF16)  # noqa: E731
    return dict(x=rn(M, K), w=rn(K, N) * K ** -0.5, w2=rn(K, N) * K ** -0.5, dy=rn(M, N))


# results of the kernel for few rows and of the one on CTA pairs
@pytest.mark.parametrize("M,K,N", [(200, 64, 128), (8192, 512, 1024)])
def test_linear(M, K, N):
    swg, t = _swg(), _inputs(M, K, N)
    want = swg.linear_fwd(t["x"], t["w"])
    out = {"y": torch.empty_like(want["y"])}
    assert torch.equal(_in_new_thread(lambda: swg.linear_fwd(t["x"], t["w"], out=out))["y"], want["y"])
    want = swg.linear_bwd(t["dy"], t["x"], t["w"])
    out = {k: torch.empty_like(v) for k, v in want.items()}
    ws = torch.empty(swg.linear_bwd_workspace_size(M, K, N), dtype=torch.uint8, device="cuda")
    got = _in_new_thread(lambda: swg.linear_bwd(t["dy"], t["x"], t["w"], out=out, workspace=ws))
    assert all(torch.equal(got[k], want[k]) for k in want)
    # without bias and activation the first launch is that of dw
    got = _in_new_thread(lambda: swg.linear_bwd(t["dy"], t["x"], t["w"], bias=False, out=out, workspace=ws))
    assert all(torch.equal(got[k], want[k]) for k in got)
    swg.swg_check()


def test_swiglu():
    swg, t = _swg(), _inputs(200, 64, 128)
    want = swg.swiglu_fwd(t["x"], t["w"], t["w2"])
    out = {k: torch.empty_like(v) for k, v in want.items()}
    got = _in_new_thread(lambda: swg.swiglu_fwd(t["x"], t["w"], t["w2"], out=out))
    assert all(torch.equal(got[k], want[k]) for k in want)
    for fused in (False, True):
        args = (t["x"], t["w"], t["w2"], t["dy"], want["g"], want["fc"])
        back = swg.swiglu_bwd(*args, fused=fused)
        got = _in_new_thread(lambda: swg.swiglu_bwd(*args, fused=fused))
        assert all(torch.equal(got[k], back[k]) for k in back)
    swg.swg_check()


def test_current_device_stays():
    # the thread's device stays what it was
    swg, t = _swg(), _inputs(200, 64, 128)
    y = torch.empty((200, 128), dtype=BF16, device="cuda")

    def call():
        before = torch.cuda.current_device()
        swg.linear_fwd(t["x"], t["w"], out={"y": y})
        return before == torch.cuda.current_device()

    assert _in_new_thread(call)
