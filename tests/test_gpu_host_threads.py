"""Calls from several host threads at once whose plans want different amounts of shared memory of the same kernel: all are
launched, with the results of the same calls one after the other (GPU). The threads are C++ ones, so that nothing but the
library orders them."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F32 = torch.bfloat16, torch.float32
THREADS, CALLS = 8, 8000

PROGRAM = r"""
#include <atomic>
#include <thread>
#include <vector>
#include "swiglu_bwd.h"
template <typename F>
static int run(int threads, int calls, F call) {
  std::atomic<int> failed{0};
  std::vector<std::thread> all;
  for (int i = 0; i < threads; ++i)
    all.emplace_back([&, i] {
      for (int n = 0; n < calls; ++n) failed += call(i) != SWG_OK;
    });
  for (auto& t : all) t.join();
  return failed;
}
extern "C" int linear(decltype(&linear_fwd) f, void** x, void** w, void** y, const int64_t* M, int64_t K, int64_t N,
                      void** streams, int threads, int calls) {
  return run(threads, calls, [&](int i) {
    return f(x[i], w[i], nullptr, nullptr, y[i], nullptr, M[i], K, N, K, N, SWG_ACT_NONE, SWG_BF16, SWG_BF16,
             reinterpret_cast<swg_stream_t>(streams[i]));
  });
}
extern "C" int norm(decltype(&block_norm_fwd) f, void** u, void** h, void** y, void** stats, const int64_t* M,
                    const int64_t* N, void** streams, int threads, int calls) {
  return run(threads, calls, [&](int i) {
    return f(u[i], u[i], nullptr, nullptr, nullptr, h[i], y[i], static_cast<float*>(stats[i]), M[i], N[i], 0, N[i], N[i], 1.0f,
             1e-6f, SWG_NORM_POST | SWG_NORM_PRE, SWG_BF16, SWG_BF16, SWG_BF16, reinterpret_cast<swg_stream_t>(streams[i]));
  });
}
"""


@pytest.fixture(scope="module")
def callers(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("threads")
    (d / "threads.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O2", "-shared", "-fPIC", "-pthread", "-I", os.path.join(ROOT, "include"),
                    str(d / "threads.cpp"), "-o", str(d / "threads.so")], check=True)
    return ctypes.CDLL(str(d / "threads.so"))


def _lib():
    from swiglu_ffn_backward_gb300 import _binding as b
    return b.lib


def _pointers(tensors):
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


def _sizes(v):
    return (ctypes.c_int64 * len(v))(*v)


def _streams(n):
    s = [torch.cuda.Stream() for _ in range(n)]
    return s, (ctypes.c_void_p * n)(*[t.cuda_stream for t in s])


def test_linear_of_few_rows(callers):
    # rings of 177 to 193 KB
    import swiglu_ffn_backward_gb300 as swg
    g = torch.Generator(device="cuda").manual_seed(3)
    rows, K, N = [1, 100, 77, 100] * (THREADS // 4), 512, 8192
    x = [torch.randn((m, K), generator=g, device="cuda").to(BF16) for m in rows]
    w = [torch.randn((K, N), generator=g, device="cuda").to(BF16) for _ in rows]
    y = [torch.empty((m, N), device="cuda", dtype=BF16) for m in rows]
    keep, streams = _streams(THREADS)
    torch.cuda.synchronize()
    fn = ctypes.cast(_lib().linear_fwd, ctypes.c_void_p)
    failed = callers.linear(fn, _pointers(x), _pointers(w), _pointers(y), _sizes(rows), ctypes.c_int64(K), ctypes.c_int64(N),
                            streams, THREADS, CALLS)
    torch.cuda.synchronize()
    assert failed == 0
    assert all(torch.equal(y[i], swg.linear_fwd(x[i], w[i])["y"]) for i in range(THREADS))
    swg.swg_check()


def test_norms_of_many_rows(callers):
    # rings of 70 to 98 KB a block
    import swiglu_ffn_backward_gb300 as swg
    g = torch.Generator(device="cuda").manual_seed(4)
    shapes = [(2400, 4096), (2800, 3584), (3900, 2560), (2800, 3584)] * (THREADS // 4)
    u = [torch.randn(s, generator=g, device="cuda").to(BF16) for s in shapes]
    h, y = ([torch.empty_like(t) for t in u] for _ in range(2))
    stats = [torch.empty((s[0], 2), device="cuda", dtype=F32) for s in shapes]
    keep, streams = _streams(THREADS)
    torch.cuda.synchronize()
    fn = ctypes.cast(_lib().block_norm_fwd, ctypes.c_void_p)
    failed = callers.norm(fn, _pointers(u), _pointers(h), _pointers(y), _pointers(stats), _sizes([s[0] for s in shapes]),
                          _sizes([s[1] for s in shapes]), streams, THREADS, CALLS // 4)
    torch.cuda.synchronize()
    assert failed == 0
    for i in range(THREADS):
        want = swg.block_norm_fwd(u[i], u[i])
        assert torch.equal(h[i], want["h"]) and torch.equal(y[i], want["y"]) and torch.equal(stats[i], want["stats"])
    swg.swg_check()
