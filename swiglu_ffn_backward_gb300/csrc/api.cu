// C ABI of the library (declared in include/swiglu_bwd.h): argument checks,
// workspace layout and kernel dispatch. No device memory is allocated here.
//
// Error model after the two-phase aclnn interface described in "SwishGrad in
// CANN ops-nn: principle, implementation and the aclnnSwishBackward guide",
// section 3.3 (null pointer -> its own code; unsupported dtype, mismatched
// dtype or shape -> invalid parameter) and section 3.5 (empty tensors
// short-circuit with no launch; a missing beta means 1.0).
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "../../include/swiglu_bwd.h"
#include "swg_launch.h"

namespace {

using swg::WPlan;

constexpr int64_t kMaxDim = 0x7fffffffLL;  // TMA coordinates are 32-bit

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};
inline Range rng(const void* p, int64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Range{a, a + static_cast<uintptr_t>(bytes)};
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

// true if any output range overlaps another output or any input range
bool any_overlap(const Range* outs, int nout, const Range* ins, int nin) {
  for (int i = 0; i < nout; ++i) {
    for (int j = i + 1; j < nout; ++j)
      if (overlap(outs[i], outs[j])) return true;
    for (int j = 0; j < nin; ++j)
      if (overlap(outs[i], ins[j])) return true;
  }
  return false;
}

// current device must be sm_103 (the kernels are built for sm_103a only)
swg_status check_device() {
  static std::mutex mu;
  static int known[64] = {0};  // 0 unknown, 1 ok, 2 not ok
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SWG_ERR_CUDA;
  if (dev < 0 || dev >= 64) return SWG_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lk(mu);
  if (known[dev] == 0) {
    int maj = 0, min = 0;
    if (cudaDeviceGetAttribute(&maj, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&min, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
      return SWG_ERR_CUDA;
    known[dev] = (maj == 10 && min == 3) ? 1 : 2;
  }
  return known[dev] == 1 ? SWG_OK : SWG_ERR_UNSUPPORTED;
}

inline swg_status cuda_status(cudaError_t e) { return e == cudaSuccess ? SWG_OK : SWG_ERR_CUDA; }

inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

swg_status check_shape(int64_t M, int64_t K, int64_t N) {
  if (M < 0 || K < 0 || N < 0) return SWG_ERR_PARAM_INVALID;
  if (M > kMaxDim || K > kMaxDim || N > kMaxDim) return SWG_ERR_UNSUPPORTED;
  if ((K % 8) != 0 || (N % 8) != 0) return SWG_ERR_UNSUPPORTED;
  return SWG_OK;
}

// zero-fill a bf16 buffer of n elements (used for sums over zero rows)
swg_status zero_bf16(void* p, int64_t n, cudaStream_t st) {
  if (n <= 0) return SWG_OK;
  return cuda_status(cudaMemsetAsync(p, 0, static_cast<size_t>(n) * 2, st));
}

}  // namespace

extern "C" {

const char* swg_status_string(swg_status s) {
  switch (s) {
    case SWG_OK: return "SWG_OK";
    case SWG_ERR_NULLPTR: return "SWG_ERR_NULLPTR: a required pointer is NULL";
    case SWG_ERR_PARAM_INVALID: return "SWG_ERR_PARAM_INVALID: invalid dtype, size or overlapping buffers";
    case SWG_ERR_UNSUPPORTED:
      return "SWG_ERR_UNSUPPORTED: K/N not a multiple of 8, misaligned pointer or device is not sm_103";
    case SWG_ERR_WORKSPACE: return "SWG_ERR_WORKSPACE: workspace missing or smaller than the query";
    case SWG_ERR_CUDA: return "SWG_ERR_CUDA: a CUDA call or kernel launch failed";
    case SWG_ERR_TIMEOUT: return "SWG_ERR_TIMEOUT: a kernel gave up waiting on a pipeline barrier";
  }
  return "SWG_ERR_?: unknown status";
}

swg_status swg_inject_stall(swg_inject_kernel kernel, int64_t entry, int64_t wait_limit_cycles) {
  if (kernel == SWG_INJECT_NONE) {
    swg::arm_injection(0, -1, 0);
    return SWG_OK;
  }
  if (kernel != SWG_INJECT_X_GEMM && kernel != SWG_INJECT_FUSED_X && kernel != SWG_INJECT_FUSED_W &&
      kernel != SWG_INJECT_FWD && kernel != SWG_INJECT_LAYER_NORM_FWD && kernel != SWG_INJECT_LAYER_NORM_BWD &&
      kernel != SWG_INJECT_TOKEN_LOGPROBS && kernel != SWG_INJECT_DISTILL && kernel != SWG_INJECT_LINEAR_SPLIT &&
      kernel != SWG_INJECT_LINEAR && kernel != SWG_INJECT_BLOCK_NORM_FWD && kernel != SWG_INJECT_BLOCK_NORM_BWD)
    return SWG_ERR_PARAM_INVALID;
  if (entry < 0 || wait_limit_cycles < 1024) return SWG_ERR_PARAM_INVALID;
  swg::arm_injection(static_cast<int>(kernel), entry, static_cast<long long>(wait_limit_cycles));
  return SWG_OK;
}

swg_status swg_check(swg_stream_t stream) {
  uint32_t v = 0;
  cudaError_t e = swg::read_and_clear_status(&v, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return SWG_ERR_CUDA;
  return v != 0 ? SWG_ERR_TIMEOUT : SWG_OK;
}

// ---------------------------------------------------------------- SwishGrad
// shared argument checks of the element-wise gradients (swish_grad, act_grad)
swg_status check_elementwise(const void* grad, const void* x, void* grad_x, int64_t n, swg_dtype dtype) {
  if (n < 0 || (dtype != SWG_F32 && dtype != SWG_F16 && dtype != SWG_BF16)) return SWG_ERR_PARAM_INVALID;
  if (n == 0) return SWG_OK;  // empty tensors may carry NULL data pointers
  if (grad == nullptr || x == nullptr || grad_x == nullptr) return SWG_ERR_NULLPTR;
  const int64_t es = dtype == SWG_F32 ? 4 : 2;
  const uintptr_t mask = static_cast<uintptr_t>(es - 1);
  if ((reinterpret_cast<uintptr_t>(grad) & mask) || (reinterpret_cast<uintptr_t>(x) & mask) ||
      (reinterpret_cast<uintptr_t>(grad_x) & mask))
    return SWG_ERR_UNSUPPORTED;
  // grad_x may alias grad or x exactly, but must not partially overlap either
  const Range o = rng(grad_x, n * es), a = rng(grad, n * es), b = rng(x, n * es);
  if ((overlap(o, a) && o.lo != a.lo) || (overlap(o, b) && o.lo != b.lo)) return SWG_ERR_PARAM_INVALID;
  return SWG_OK;
}

swg_status act_grad(const void* grad, const void* x, swg_act act, void* grad_x, int64_t n, swg_dtype dtype,
                    swg_stream_t stream) {
  if (act != SWG_ACT_SILU && act != SWG_ACT_GELU && act != SWG_ACT_HARDSWISH) return SWG_ERR_PARAM_INVALID;
  swg_status st = check_elementwise(grad, x, grad_x, n, dtype);
  if (st != SWG_OK || n == 0) return st;
  st = check_device();
  if (st != SWG_OK) return st;
  return cuda_status(swg::launch_act_grad(grad, x, static_cast<int>(act), grad_x, n, static_cast<int>(dtype),
                                          reinterpret_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------- GroupNorm backward
size_t group_norm_bwd_workspace_size(int64_t N, int64_t C, int64_t HxW, int64_t G) {
  if (N <= 0 || C <= 0 || HxW <= 0 || G <= 0 || C % G != 0) return 0;
  return swg::gn_workspace_bytes(N, C, G);
}

swg_status group_norm_bwd(const void* dy, const void* x, const void* gamma, void* dx, void* dgamma, void* dbeta,
                          int64_t N, int64_t C, int64_t HxW, int64_t G, float eps, swg_dtype dtype,
                          void* workspace, size_t workspace_bytes, swg_stream_t stream) {
  if (dtype != SWG_F32 && dtype != SWG_F16 && dtype != SWG_BF16) return SWG_ERR_PARAM_INVALID;
  if (N < 0 || C < 0 || HxW < 0 || G < 1 || C % G != 0 || !(eps >= 0.0f)) return SWG_ERR_PARAM_INVALID;
  // sizes: every index fits 64 bits (N C HxW elements, and their bytes, below 2^60); the grid of
  // N G clusters of up to 8 CTAs stays below 2^31 blocks
  if (N > kMaxDim || C > kMaxDim || HxW > (int64_t(1) << 40) || N * G >= (int64_t(1) << 28))
    return SWG_ERR_UNSUPPORTED;
  if (N > 0 && C > 0 && HxW > ((int64_t(1) << 60) / N) / C) return SWG_ERR_UNSUPPORTED;
  const int64_t es = dtype == SWG_F32 ? 4 : 2;
  const int64_t n = N * C * HxW;
  const bool params = dgamma != nullptr || dbeta != nullptr;
  const uintptr_t mask = static_cast<uintptr_t>(es - 1);
  auto misaligned = [&](const void* p) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; };
  if (misaligned(dy) || misaligned(x) || misaligned(gamma) || misaligned(dx) || misaligned(dgamma) ||
      misaligned(dbeta))
    return SWG_ERR_UNSUPPORTED;
  if (n > 0 && (dy == nullptr || x == nullptr || dx == nullptr)) return SWG_ERR_NULLPTR;
  const Range outs[3] = {rng(dx, n * es), rng(dgamma, dgamma ? C * es : 0), rng(dbeta, dbeta ? C * es : 0)};
  const Range ins[3] = {rng(dy, n * es), rng(x, n * es), rng(gamma, gamma ? C * es : 0)};
  if (any_overlap(outs, 3, ins, 3)) return SWG_ERR_PARAM_INVALID;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (n == 0) {
    if (C == 0 || !params) return SWG_OK;
    swg_status s = check_device();
    if (s != SWG_OK) return s;
    if (dgamma != nullptr && cudaMemsetAsync(dgamma, 0, static_cast<size_t>(C * es), st) != cudaSuccess)
      return SWG_ERR_CUDA;
    if (dbeta != nullptr && cudaMemsetAsync(dbeta, 0, static_cast<size_t>(C * es), st) != cudaSuccess)
      return SWG_ERR_CUDA;
    return SWG_OK;
  }
  if (params && (workspace == nullptr || !aligned16(workspace) ||
                 workspace_bytes < swg::gn_workspace_bytes(N, C, G)))
    return SWG_ERR_WORKSPACE;
  swg_status s = check_device();
  if (s != SWG_OK) return s;
  return cuda_status(swg::launch_group_norm_bwd(dy, x, gamma, dx, dgamma, dbeta, N, C, HxW, G, eps,
                                                static_cast<int>(dtype), params ? workspace : nullptr, st));
}

swg_status swish_grad(const void* grad, const void* x, const float* scale, void* grad_x, int64_t n,
                      swg_dtype dtype, swg_stream_t stream) {
  swg_status st = check_elementwise(grad, x, grad_x, n, dtype);
  if (st != SWG_OK || n == 0) return st;
  st = check_device();
  if (st != SWG_OK) return st;
  const float beta = scale != nullptr ? *scale : 1.0f;
  return cuda_status(swg::launch_swish_grad(grad, x, beta, grad_x, n, static_cast<int>(dtype),
                                            reinterpret_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------- b stage
size_t swiglu_bwd_b_workspace_size(int64_t M, int64_t N) {
  if (M <= 0 || N <= 0) return 0;
  return swg::b_workspace_bytes(M, N);
}

swg_status swiglu_bwd_b(const void* dy, const void* g, const void* fc, void* dg, void* dfc, void* db_g,
                        void* db_fc, int64_t M, int64_t N, void* workspace, size_t workspace_bytes,
                        swg_stream_t stream) {
  swg_status st = check_shape(M, 8, N);
  if (st != SWG_OK) return st;
  if (N == 0) return SWG_OK;
  // [M,N] tensors may be NULL when M == 0 (empty); [1,N] outputs are required
  if (!db_g || !db_fc || (M > 0 && (!dy || !g || !fc || !dg || !dfc))) return SWG_ERR_NULLPTR;
  const void* all[] = {dy, g, fc, dg, dfc, db_g, db_fc};
  for (const void* p : all)
    if (!aligned16(p)) return SWG_ERR_UNSUPPORTED;
  const int64_t mn = M * N * 2;
  const Range outs[] = {rng(dg, mn), rng(dfc, mn), rng(db_g, N * 2), rng(db_fc, N * 2)};
  const Range ins[] = {rng(dy, mn), rng(g, mn), rng(fc, mn)};
  if (any_overlap(outs, 4, ins, 3)) return SWG_ERR_PARAM_INVALID;
  st = check_device();
  if (st != SWG_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {
    st = zero_bf16(db_g, N, s);
    return st != SWG_OK ? st : zero_bf16(db_fc, N, s);
  }
  const size_t need = swg::b_workspace_bytes(M, N);
  if (workspace == nullptr || workspace_bytes < need) return SWG_ERR_WORKSPACE;
  if (!aligned16(workspace)) return SWG_ERR_UNSUPPORTED;
  const Range w = rng(workspace, static_cast<int64_t>(need));
  if (any_overlap(&w, 1, outs, 4) || any_overlap(&w, 1, ins, 3)) return SWG_ERR_PARAM_INVALID;
  return cuda_status(swg::launch_b_stage(
      static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(g), static_cast<const uint16_t*>(fc),
      static_cast<uint16_t*>(dg), static_cast<uint16_t*>(dfc), static_cast<uint16_t*>(db_g),
      static_cast<uint16_t*>(db_fc), M, N, workspace, s));
}

// ---------------------------------------------------------------- w stage
size_t swiglu_bwd_w_workspace_size(int64_t M, int64_t K, int64_t N) {
  if (M <= 0 || K <= 0 || N <= 0) return 0;
  return swg::w_plan(M, K, N, swg::device_sm_count()).ws_bytes;
}

swg_status swiglu_bwd_w(const void* x, const void* dg, const void* dfc, void* dw_g, void* dw_fc, int64_t M,
                        int64_t K, int64_t N, void* workspace, size_t workspace_bytes, swg_stream_t stream) {
  swg_status st = check_shape(M, K, N);
  if (st != SWG_OK) return st;
  if (K == 0 || N == 0) return SWG_OK;
  if (!dw_g || !dw_fc || (M > 0 && (!x || !dg || !dfc))) return SWG_ERR_NULLPTR;
  const void* all[] = {x, dg, dfc, dw_g, dw_fc};
  for (const void* p : all)
    if (!aligned16(p)) return SWG_ERR_UNSUPPORTED;
  const Range outs[] = {rng(dw_g, K * N * 2), rng(dw_fc, K * N * 2)};
  const Range ins[] = {rng(x, M * K * 2), rng(dg, M * N * 2), rng(dfc, M * N * 2)};
  if (any_overlap(outs, 2, ins, 3)) return SWG_ERR_PARAM_INVALID;
  st = check_device();
  if (st != SWG_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {
    st = zero_bf16(dw_g, K * N, s);
    return st != SWG_OK ? st : zero_bf16(dw_fc, K * N, s);
  }
  const WPlan plan = swg::w_plan(M, K, N, swg::device_sm_count());
  if (plan.ws_bytes > 0) {
    if (workspace == nullptr || workspace_bytes < plan.ws_bytes) return SWG_ERR_WORKSPACE;
    if (!aligned16(workspace)) return SWG_ERR_UNSUPPORTED;
    const Range w = rng(workspace, static_cast<int64_t>(plan.ws_bytes));
    if (any_overlap(&w, 1, outs, 2) || any_overlap(&w, 1, ins, 3)) return SWG_ERR_PARAM_INVALID;
  }
  return cuda_status(swg::launch_w_gemm(static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(dg),
                                        static_cast<const uint16_t*>(dfc), static_cast<uint16_t*>(dw_g),
                                        static_cast<uint16_t*>(dw_fc), M, K, N, workspace, plan, s));
}

// ---------------------------------------------------------------- x stage
swg_status swiglu_bwd_x(const void* dg, const void* dfc, const void* w_g, const void* w_fc, void* dx, int64_t M,
                        int64_t K, int64_t N, swg_stream_t stream) {
  swg_status st = check_shape(M, K, N);
  if (st != SWG_OK) return st;
  if (M == 0 || K == 0) return SWG_OK;
  if (!dg || !dfc || !w_g || !w_fc || !dx) return SWG_ERR_NULLPTR;
  const void* all[] = {dg, dfc, w_g, w_fc, dx};
  for (const void* p : all)
    if (!aligned16(p)) return SWG_ERR_UNSUPPORTED;
  const Range outs[] = {rng(dx, M * K * 2)};
  const Range ins[] = {rng(dg, M * N * 2), rng(dfc, M * N * 2), rng(w_g, K * N * 2), rng(w_fc, K * N * 2)};
  if (any_overlap(outs, 1, ins, 4)) return SWG_ERR_PARAM_INVALID;
  st = check_device();
  if (st != SWG_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (N == 0) return cuda_status(cudaMemsetAsync(dx, 0, static_cast<size_t>(M * K * 2), s));
  return cuda_status(swg::launch_x_gemm(static_cast<const uint16_t*>(dg), static_cast<const uint16_t*>(dfc),
                                        static_cast<const uint16_t*>(w_g), static_cast<const uint16_t*>(w_fc),
                                        static_cast<uint16_t*>(dx), M, K, N, s));
}

// ---------------------------------------------------------------- forward
swg_status swiglu_fwd(const void* x, const void* w_g, const void* w_fc, const void* b_g, const void* b_fc, void* g,
                      void* fc, void* y, int64_t M, int64_t K, int64_t N, swg_stream_t stream) {
  swg_status st = check_shape(M, K, N);
  if (st != SWG_OK) return st;
  if (K == 0) return SWG_ERR_UNSUPPORTED;  // the products need a reduction of positive length
  if (M == 0 || N == 0) return SWG_OK;
  if (!x || !w_g || !w_fc || !g || !fc || !y) return SWG_ERR_NULLPTR;
  const void* all[] = {x, w_g, w_fc, b_g, b_fc, g, fc, y};  // null biases count as aligned
  for (const void* p : all)
    if (!aligned16(p)) return SWG_ERR_UNSUPPORTED;
  const int64_t mn = M * N * 2, kn = K * N * 2;
  const Range outs[] = {rng(g, mn), rng(fc, mn), rng(y, mn)};
  const Range ins[] = {rng(x, M * K * 2), rng(w_g, kn), rng(w_fc, kn), rng(b_g, b_g ? N * 2 : 0),
                       rng(b_fc, b_fc ? N * 2 : 0)};
  if (any_overlap(outs, 3, ins, 5)) return SWG_ERR_PARAM_INVALID;
  st = check_device();
  if (st != SWG_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return cuda_status(swg::launch_fwd_gemm(
      static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(w_g), static_cast<const uint16_t*>(w_fc),
      static_cast<const uint16_t*>(b_g), static_cast<const uint16_t*>(b_fc), static_cast<uint16_t*>(g),
      static_cast<uint16_t*>(fc), static_cast<uint16_t*>(y), M, K, N, s));
}

// ---------------------------------------------------------------- fused stages
swg_status swiglu_bwd_x_fused(const void* dy, const void* g, const void* fc, const void* w_g, const void* w_fc,
                              void* dx, void* dg, void* dfc, int64_t M, int64_t K, int64_t N, swg_stream_t stream) {
  swg_status st = check_shape(M, K, N);
  if (st != SWG_OK) return st;
  if (M == 0 || K == 0) return SWG_OK;
  if (!dy || !g || !fc || !w_g || !w_fc || !dx) return SWG_ERR_NULLPTR;
  if ((dg == nullptr) != (dfc == nullptr)) return SWG_ERR_NULLPTR;
  const void* all[] = {dy, g, fc, w_g, w_fc, dx, dg, dfc};
  for (const void* p : all)
    if (!aligned16(p)) return SWG_ERR_UNSUPPORTED;
  const int64_t mn = M * N * 2, kn = K * N * 2;
  const Range outs[] = {rng(dx, M * K * 2), rng(dg, dg ? mn : 0), rng(dfc, dfc ? mn : 0)};
  const Range ins[] = {rng(dy, mn), rng(g, mn), rng(fc, mn), rng(w_g, kn), rng(w_fc, kn)};
  if (any_overlap(outs, 3, ins, 5)) return SWG_ERR_PARAM_INVALID;
  st = check_device();
  if (st != SWG_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (N == 0) return cuda_status(cudaMemsetAsync(dx, 0, static_cast<size_t>(M * K * 2), s));
  return cuda_status(swg::launch_fused_x(
      static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(g), static_cast<const uint16_t*>(fc),
      static_cast<const uint16_t*>(w_g), static_cast<const uint16_t*>(w_fc), static_cast<uint16_t*>(dx),
      static_cast<uint16_t*>(dg), static_cast<uint16_t*>(dfc), M, K, N, s));
}

size_t swiglu_bwd_w_fused_workspace_size(int64_t M, int64_t K, int64_t N) {
  if (M <= 0 || K <= 0 || N <= 0) return 0;
  return swg::fw_plan(M, K, N, swg::device_sm_count()).ws_bytes;
}

swg_status swiglu_bwd_w_fused(const void* x, const void* dy, const void* g, const void* fc, void* dw_g,
                              void* dw_fc, void* db_g, void* db_fc, int64_t M, int64_t K, int64_t N, void* workspace,
                              size_t workspace_bytes, swg_stream_t stream) {
  swg_status st = check_shape(M, K, N);
  if (st != SWG_OK) return st;
  if (K == 0 || N == 0) return SWG_OK;
  if (!dw_g || !dw_fc || !db_g || !db_fc || (M > 0 && (!x || !dy || !g || !fc))) return SWG_ERR_NULLPTR;
  const void* all[] = {x, dy, g, fc, dw_g, dw_fc, db_g, db_fc};
  for (const void* p : all)
    if (!aligned16(p)) return SWG_ERR_UNSUPPORTED;
  const int64_t mn = M * N * 2, kn = K * N * 2;
  const Range outs[] = {rng(dw_g, kn), rng(dw_fc, kn), rng(db_g, N * 2), rng(db_fc, N * 2)};
  const Range ins[] = {rng(x, M * K * 2), rng(dy, mn), rng(g, mn), rng(fc, mn)};
  if (any_overlap(outs, 4, ins, 4)) return SWG_ERR_PARAM_INVALID;
  st = check_device();
  if (st != SWG_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {
    st = zero_bf16(dw_g, K * N, s);
    if (st == SWG_OK) st = zero_bf16(dw_fc, K * N, s);
    if (st == SWG_OK) st = zero_bf16(db_g, N, s);
    return st != SWG_OK ? st : zero_bf16(db_fc, N, s);
  }
  const swg::FwPlan plan = swg::fw_plan(M, K, N, swg::device_sm_count());
  if (workspace == nullptr || workspace_bytes < plan.ws_bytes) return SWG_ERR_WORKSPACE;
  if (!aligned16(workspace)) return SWG_ERR_UNSUPPORTED;
  const Range w = rng(workspace, static_cast<int64_t>(plan.ws_bytes));
  if (any_overlap(&w, 1, outs, 4) || any_overlap(&w, 1, ins, 4)) return SWG_ERR_PARAM_INVALID;
  return cuda_status(swg::launch_fused_w(
      static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(g),
      static_cast<const uint16_t*>(fc), static_cast<uint16_t*>(dw_g), static_cast<uint16_t*>(dw_fc),
      static_cast<uint16_t*>(db_g), static_cast<uint16_t*>(db_fc), M, K, N, workspace, plan, s));
}

// ---------------------------------------------------------------- whole backward from host buffers
// The fused backward with every tensor in host memory. M is cut into chunks
// (equal ones, then a short last one); while chunk c is computed (dx, and the fused w
// stage's fp32 split partials into chunk c's own slots), chunk c + 1's rows are
// copied in on one internal stream and chunk c - 1's dx is copied out on
// another, each chunk's device buffers alternating between two sets. One
// fixed-order reduction over every chunk's partials gives dw and db with one
// rounding, as in the single-call backward. Workspace layout (256-byte aligned
// regions): W_g, W_fc | two input sets (x, dy, g, fc rows of a chunk) | two dx
// sets | dw_g, dw_fc, db_g, db_fc | dw partials [S total][2][K][N] fp32 |
// db partials [S total][2N] fp32 (a single chunk: the fused w stage's own
// workspace instead of the partial blocks).
namespace {

constexpr int64_t kHostChunkRows = 32768;
constexpr int64_t kMinLastRows = 16384;

struct HostPlan {
  int64_t chunks, rows;  // chunk count, rows per chunk (multiple of 64; the last may be shorter)
  int64_t splits_total;  // sum of the chunks' M-splits (chunks > 1)
  size_t off_w, off_in[2], off_dx[2], off_out, off_dwp, off_dbp, total;
};

HostPlan host_plan(int64_t M, int64_t K, int64_t N, int sms) {
  HostPlan p{};
  // floor(M / kHostChunkRows) chunks (at most 256): all but the last of one 64-row multiple, the
  // last as short as allowed (kMinLastRows to kMinLastRows + 64 (chunks - 1) rows), so that little
  // compute and dx copy-out is left after the last rows have come in. Every chunk keeps at least 16K
  // rows, so each one splits over M (its partials path needs two splits).
  p.chunks = M >= 2 * kHostChunkRows ? std::min<int64_t>(M / kHostChunkRows, 256) : (M > 0 ? 1 : 0);
  p.rows = p.chunks > 1 ? (M - kMinLastRows) / (p.chunks - 1) / 64 * 64 : (M + 63) / 64 * 64;
  size_t off = 0;
  p.off_w = off;
  off += align256(static_cast<size_t>(2 * K * N) * 2);
  const size_t in_bytes = static_cast<size_t>(p.rows) * static_cast<size_t>(K + 3 * N) * 2;
  const size_t dx_bytes = static_cast<size_t>(p.rows) * static_cast<size_t>(K) * 2;
  for (int b = 0; b < 2; ++b) {
    p.off_in[b] = off;
    off += align256(in_bytes);
  }
  for (int b = 0; b < 2; ++b) {
    p.off_dx[b] = off;
    off += align256(dx_bytes);
  }
  p.off_out = off;
  off += align256(static_cast<size_t>(2 * K * N + 2 * N) * 2);
  if (p.chunks > 1) {
    for (int64_t c = 0; c < p.chunks; ++c) {
      const int64_t r = std::min(p.rows, M - c * p.rows);
      p.splits_total += swg::fw_plan(r, K, N, sms).splits;
    }
    p.off_dwp = off;
    off += align256(static_cast<size_t>(p.splits_total) * 2 * K * N * 4);
    p.off_dbp = off;
    off += align256(static_cast<size_t>(p.splits_total) * 2 * N * 4);
  } else {
    p.off_dwp = off;
    off += align256(p.chunks == 1 ? swg::fw_plan(M, K, N, sms).ws_bytes : 0);
    p.off_dbp = p.off_dwp;
  }
  p.total = off;
  return p;
}

// the internal copy streams and the events that order them against the caller's stream (per device,
// created once; the enqueue of one call holds the lock, so calls from several host threads take turns)
struct HostStreams {
  cudaStream_t h2d = nullptr, d2h = nullptr;
  cudaEvent_t start = nullptr, w_in = nullptr, reduced = nullptr, end = nullptr;
  cudaEvent_t loaded[2] = {}, computed[2] = {}, dx_out[2] = {};
};
std::mutex g_host_mu;
HostStreams g_host[64];

cudaError_t host_streams(int dev, HostStreams** out) {
  HostStreams& h = g_host[dev];
  if (h.h2d == nullptr) {
    cudaError_t e = cudaStreamCreateWithFlags(&h.h2d, cudaStreamNonBlocking);
    if (e == cudaSuccess) e = cudaStreamCreateWithFlags(&h.d2h, cudaStreamNonBlocking);
    cudaEvent_t* evs[] = {&h.start, &h.w_in, &h.reduced, &h.end, &h.loaded[0], &h.loaded[1],
                          &h.computed[0], &h.computed[1], &h.dx_out[0], &h.dx_out[1]};
    for (cudaEvent_t* ev : evs)
      if (e == cudaSuccess) e = cudaEventCreateWithFlags(ev, cudaEventDisableTiming);
    if (e != cudaSuccess) return e;
  }
  *out = &h;
  return cudaSuccess;
}

}  // namespace

size_t swiglu_bwd_host_workspace_size(int64_t M, int64_t K, int64_t N) {
  if (M < 0 || K <= 0 || N <= 0) return 0;
  return host_plan(M, K, N, swg::device_sm_count()).total;
}

swg_status swiglu_bwd_host(const void* x, const void* w_g, const void* w_fc, const void* dy, const void* g,
                           const void* fc, void* dx, void* dw_g, void* dw_fc, void* db_g, void* db_fc, int64_t M,
                           int64_t K, int64_t N, void* workspace, size_t workspace_bytes, swg_stream_t stream) {
  swg_status st = check_shape(M, K, N);
  if (st != SWG_OK) return st;
  if (K == 0 || N == 0) return SWG_OK;
  if (!w_g || !w_fc || !dw_g || !dw_fc || !db_g || !db_fc) return SWG_ERR_NULLPTR;
  if (M > 0 && (!x || !dy || !g || !fc || !dx)) return SWG_ERR_NULLPTR;
  const int64_t kn = K * N * 2, mn = M * N * 2;
  const Range outs[] = {rng(dx, M * K * 2), rng(dw_g, kn), rng(dw_fc, kn), rng(db_g, N * 2), rng(db_fc, N * 2)};
  const Range ins[] = {rng(x, M * K * 2), rng(w_g, kn), rng(w_fc, kn), rng(dy, mn), rng(g, mn), rng(fc, mn)};
  if (any_overlap(outs, 5, ins, 6)) return SWG_ERR_PARAM_INVALID;
  st = check_device();
  if (st != SWG_OK) return st;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SWG_ERR_CUDA;
  const int sms = swg::device_sm_count();
  const HostPlan hp = host_plan(M, K, N, sms);
  if (workspace == nullptr || workspace_bytes < hp.total) return SWG_ERR_WORKSPACE;
  if (!aligned16(workspace)) return SWG_ERR_UNSUPPORTED;

  std::lock_guard<std::mutex> lk(g_host_mu);
  HostStreams* hs = nullptr;
  if (host_streams(dev, &hs) != cudaSuccess) return SWG_ERR_CUDA;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  auto dev16 = [&](size_t off) { return reinterpret_cast<uint16_t*>(ws + off); };
  uint16_t* wg_d = dev16(hp.off_w);
  uint16_t* wfc_d = wg_d + K * N;
  uint16_t* dwg_d = dev16(hp.off_out);
  uint16_t* dwfc_d = dwg_d + K * N;
  uint16_t* dbg_d = dwfc_d + K * N;
  uint16_t* dbfc_d = dbg_d + N;
  const auto* xh = static_cast<const uint8_t*>(x);
  const auto* dyh = static_cast<const uint8_t*>(dy);
  const auto* gh = static_cast<const uint8_t*>(g);
  const auto* fch = static_cast<const uint8_t*>(fc);
  auto* dxh = static_cast<uint8_t*>(dx);
  const cudaMemcpyKind h2d = cudaMemcpyHostToDevice, d2h = cudaMemcpyDeviceToHost;
  cudaError_t e = cudaSuccess;
  auto ok = [&](cudaError_t r) {
    if (e == cudaSuccess) e = r;
    return e == cudaSuccess;
  };

  ok(cudaEventRecord(hs->start, cs));
  ok(cudaStreamWaitEvent(hs->h2d, hs->start, 0));
  ok(cudaStreamWaitEvent(hs->d2h, hs->start, 0));
  ok(cudaMemcpyAsync(wg_d, w_g, kn, h2d, hs->h2d));
  ok(cudaMemcpyAsync(wfc_d, w_fc, kn, h2d, hs->h2d));
  ok(cudaEventRecord(hs->w_in, hs->h2d));
  ok(cudaStreamWaitEvent(cs, hs->w_in, 0));
  if (M == 0) {
    ok(cudaMemsetAsync(dwg_d, 0, static_cast<size_t>(2 * K * N + 2 * N) * 2, cs));
  }
  int64_t split_off = 0;
  for (int64_t c = 0; c < hp.chunks && e == cudaSuccess; ++c) {
    const int b = static_cast<int>(c & 1);
    const int64_t r0 = c * hp.rows, rows = std::min(hp.rows, M - r0);
    uint16_t* xin = dev16(hp.off_in[b]);
    uint16_t* dyin = xin + hp.rows * K;
    uint16_t* gin = dyin + hp.rows * N;
    uint16_t* fcin = gin + hp.rows * N;
    uint16_t* dxo = dev16(hp.off_dx[b]);
    // rows of chunk c in; buffer set b was last read by chunk c - 2's kernels
    if (c >= 2) ok(cudaStreamWaitEvent(hs->h2d, hs->computed[b], 0));
    ok(cudaMemcpyAsync(xin, xh + r0 * K * 2, static_cast<size_t>(rows * K * 2), h2d, hs->h2d));
    ok(cudaMemcpyAsync(dyin, dyh + r0 * N * 2, static_cast<size_t>(rows * N * 2), h2d, hs->h2d));
    ok(cudaMemcpyAsync(gin, gh + r0 * N * 2, static_cast<size_t>(rows * N * 2), h2d, hs->h2d));
    ok(cudaMemcpyAsync(fcin, fch + r0 * N * 2, static_cast<size_t>(rows * N * 2), h2d, hs->h2d));
    ok(cudaEventRecord(hs->loaded[b], hs->h2d));
    // compute; dx set b was last copied out for chunk c - 2
    ok(cudaStreamWaitEvent(cs, hs->loaded[b], 0));
    if (c >= 2) ok(cudaStreamWaitEvent(cs, hs->dx_out[b], 0));
    ok(swg::launch_fused_x(dyin, gin, fcin, wg_d, wfc_d, dxo, nullptr, nullptr, rows, K, N, cs));
    if (hp.chunks == 1) {
      const swg::FwPlan fp = swg::fw_plan(rows, K, N, sms);
      ok(swg::launch_fused_w(xin, dyin, gin, fcin, dwg_d, dwfc_d, dbg_d, dbfc_d, rows, K, N, ws + hp.off_dwp, fp,
                             cs));
    } else {
      const swg::FwPlan fp = swg::fw_plan(rows, K, N, sms);
      float* dwp = reinterpret_cast<float*>(ws + hp.off_dwp) + split_off * 2 * K * N;
      float* dbp = reinterpret_cast<float*>(ws + hp.off_dbp) + split_off * 2 * N;
      ok(swg::launch_fused_w_partials(xin, dyin, gin, fcin, rows, K, N, dwp, dbp, fp, cs));
      split_off += fp.splits;
    }
    ok(cudaEventRecord(hs->computed[b], cs));
    // dx of chunk c out
    ok(cudaStreamWaitEvent(hs->d2h, hs->computed[b], 0));
    ok(cudaMemcpyAsync(dxh + r0 * K * 2, dxo, static_cast<size_t>(rows * K * 2), d2h, hs->d2h));
    ok(cudaEventRecord(hs->dx_out[b], hs->d2h));
  }
  if (hp.chunks > 1) {
    ok(swg::launch_w_split_reduce(reinterpret_cast<const float*>(ws + hp.off_dwp), hp.splits_total, K, N, dwg_d,
                                  dwfc_d, cs));
    ok(swg::launch_db_reduce(reinterpret_cast<const float*>(ws + hp.off_dbp), hp.splits_total, N, dbg_d, dbfc_d,
                             cs));
  }
  ok(cudaEventRecord(hs->reduced, cs));
  ok(cudaStreamWaitEvent(hs->d2h, hs->reduced, 0));
  ok(cudaMemcpyAsync(dw_g, dwg_d, kn, d2h, hs->d2h));
  ok(cudaMemcpyAsync(dw_fc, dwfc_d, kn, d2h, hs->d2h));
  ok(cudaMemcpyAsync(db_g, dbg_d, N * 2, d2h, hs->d2h));
  ok(cudaMemcpyAsync(db_fc, dbfc_d, N * 2, d2h, hs->d2h));
  ok(cudaEventRecord(hs->end, hs->d2h));
  ok(cudaStreamWaitEvent(cs, hs->end, 0));
  return cuda_status(e);
}

// ---------------------------------------------------------------- whole backward
// Unfused workspace layout: [dg scratch 2MN | dfc scratch 2MN] (only when the
// caller passes NULL dg/dfc) | b-stage partials | w-stage partials; each
// region starts on a 256-byte boundary.
// SWG_AUTO: the chain measured faster for the shape on GB300. The fused chain
// forms dg, dfc once per 512 columns of K in each of its two kernels, the
// unfused one once in the b stage but writes and re-reads them through HBM.
// Measured (whole backward, N = 1024 unless stated): K = 512, M = 220000:
// fused 0.80 ms, unfused 1.07 ms; K = 512, M = 65537: 0.285 vs 0.346 ms;
// K = 512, M <= 4097: fused slower (fixed costs of its two persistent
// launches); K = 4096, N = 14336, M = 16384: fused 6.85 ms, unfused 5.48 ms.
namespace {

bool auto_fused(int64_t M, int64_t K) { return K <= 512 && M >= 32768; }

unsigned resolve_auto(int64_t M, int64_t K, unsigned flags) {
  if (!(flags & SWG_AUTO)) return flags;
  flags &= ~(SWG_AUTO | SWG_FUSED);
  return auto_fused(M, K) ? (flags | SWG_FUSED) : flags;
}

// The fused chain's x-stage work split: when the w stage occupies fewer CTAs than the GPU has
// SMs, the x stage's last side_tiles tiles run on side_ctas CTAs beside the w stage and the
// other main_tiles tiles in one persistent wave after it. The side share is what makes the
// main part one wave round shorter (main_tiles = (rounds - 1) * SMs), and it is taken only when
// its own rounds fit well inside the w stage. By operand volume a w-stage CTA does the work of
// kb_per / (2 * ceil(N / 64)) x-stage tiles (a 64-row stage of one band against a 128-row tile
// over all bands); in time it takes about three quarters of that (measured at K = 512,
// N = 1024: 382 stages against 8.8 tiles). The side rounds may use 0.6 of the volume figure,
// about 80% of the w stage's time.
struct FxSplit {
  int64_t main_tiles = 0, side_tiles = 0;
  int side_ctas = 0;
};
FxSplit fx_split(int64_t M, int64_t K, int64_t N, const swg::FwPlan& plan, int sms) {
  FxSplit sp;
  const int64_t tiles = swg::fused_x_tiles(M, K);
  sp.main_tiles = tiles;
  const int64_t idle = sms - swg::fused_w_ctas(K, N, plan);
  const int64_t rounds = (tiles + sms - 1) / sms;
  if (idle <= 0 || rounds < 2) return sp;
  const int64_t main = (rounds - 1) * sms, side = tiles - main;
  const int64_t side_rounds = (side + idle - 1) / idle;
  const int64_t nst = (N + 63) / 64;
  if (side_rounds * 2 * nst * 5 > plan.kb_per * 3) return sp;
  sp.main_tiles = main;
  sp.side_tiles = side;
  sp.side_ctas = static_cast<int>(idle);
  return sp;
}

// the side stream of the fused chain and its fork / join events (per device, created once;
// the enqueue of one call holds the lock)
struct SideStream {
  cudaStream_t side = nullptr;
  cudaEvent_t fork = nullptr, join = nullptr, fw_done = nullptr;
};
std::mutex g_side_mu;
SideStream g_side[64];

cudaError_t side_stream(int dev, SideStream** out) {
  SideStream& h = g_side[dev];
  if (h.side == nullptr) {
    cudaError_t e = cudaStreamCreateWithFlags(&h.side, cudaStreamNonBlocking);
    if (e == cudaSuccess) e = cudaEventCreateWithFlags(&h.fork, cudaEventDisableTiming);
    if (e == cudaSuccess) e = cudaEventCreateWithFlags(&h.join, cudaEventDisableTiming);
    if (e == cudaSuccess) e = cudaEventCreateWithFlags(&h.fw_done, cudaEventDisableTiming);
    if (e != cudaSuccess) return e;
  }
  *out = &h;
  return cudaSuccess;
}

}  // namespace

size_t swiglu_bwd_workspace_size(int64_t M, int64_t K, int64_t N, unsigned flags) {
  if (M <= 0 || K <= 0 || N <= 0) return 0;
  flags = resolve_auto(M, K, flags);
  const bool fused = (flags & SWG_FUSED) != 0;
  if (fused) return swg::fw_plan(M, K, N, swg::device_sm_count()).ws_bytes;
  size_t total = 0;
  if (!(flags & SWG_WS_DG_GIVEN)) total += 2 * align256(static_cast<size_t>(M) * N * 2);
  total += align256(swg::b_workspace_bytes(M, N));
  total += align256(swg::w_plan(M, K, N, swg::device_sm_count()).ws_bytes);
  return total;
}

int swiglu_bwd_kernel_count(int64_t M, int64_t K, int64_t N, unsigned flags) {
  if ((flags & ~(SWG_FUSED | SWG_ACCUMULATE | SWG_WS_DG_GIVEN | SWG_AUTO)) != 0) return 0;
  if (check_shape(M, K, N) != SWG_OK || M <= 0 || K == 0 || N == 0) return 0;
  flags = resolve_auto(M, K, flags);
  const int sms = swg::device_sm_count();
  if (flags & SWG_FUSED) {
    const swg::FwPlan fplan = swg::fw_plan(M, K, N, sms);
    const FxSplit sp = fx_split(M, K, N, fplan, sms);
    // x stage (one or two launches), w stage, its dw and db reductions (one launch)
    return (sp.side_tiles > 0 ? 2 : 1) + 1 + 1;
  }
  // b stage and its db reduce, w GEMM and its split reduce, x GEMM
  return 2 + 1 + (swg::w_plan(M, K, N, sms).splits > 1 ? 1 : 0) + 1;
}

swg_status swiglu_bwd(const void* x, const void* w_g, const void* w_fc, const void* dy, const void* g,
                      const void* fc, void* dg, void* dfc, void* dx, void* dw_g, void* dw_fc, void* db_g,
                      void* db_fc, int64_t M, int64_t K, int64_t N, unsigned flags, void* workspace,
                      size_t workspace_bytes, swg_stream_t stream) {
  if ((flags & ~(SWG_FUSED | SWG_ACCUMULATE | SWG_WS_DG_GIVEN | SWG_AUTO)) != 0) return SWG_ERR_PARAM_INVALID;
  flags = resolve_auto(M, K, flags);
  const bool acc = (flags & SWG_ACCUMULATE) != 0;
  swg_status st = check_shape(M, K, N);
  if (st != SWG_OK) return st;
  if (K == 0 || N == 0) return SWG_OK;
  // tensors with an M dimension may be NULL when M == 0 (empty)
  if (!w_g || !w_fc || !dw_g || !dw_fc || !db_g || !db_fc) return SWG_ERR_NULLPTR;
  if (M > 0 && (!x || !dy || !g || !fc || !dx)) return SWG_ERR_NULLPTR;
  if (M > 0 && (dg == nullptr) != (dfc == nullptr)) return SWG_ERR_NULLPTR;
  if (M == 0) dg = dfc = nullptr;
  const void* all[] = {x, w_g, w_fc, dy, g, fc, dx, dw_g, dw_fc, db_g, db_fc};
  for (const void* p : all)
    if (!aligned16(p)) return SWG_ERR_UNSUPPORTED;
  if (dg != nullptr && (!aligned16(dg) || !aligned16(dfc))) return SWG_ERR_UNSUPPORTED;
  const int64_t mn = M * N * 2, kn = K * N * 2;
  const Range outs[] = {rng(dx, M * K * 2), rng(dw_g, kn), rng(dw_fc, kn), rng(db_g, N * 2), rng(db_fc, N * 2),
                        rng(dg, dg ? mn : 0), rng(dfc, dfc ? mn : 0)};
  const Range ins[] = {rng(x, M * K * 2), rng(w_g, kn), rng(w_fc, kn), rng(dy, mn), rng(g, mn), rng(fc, mn)};
  if (any_overlap(outs, 7, ins, 6)) return SWG_ERR_PARAM_INVALID;
  if (M == 0 && acc) return SWG_OK;  // a sum over no rows adds nothing: no work at all
  st = check_device();
  if (st != SWG_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {
    st = zero_bf16(dw_g, K * N, s);
    if (st == SWG_OK) st = zero_bf16(dw_fc, K * N, s);
    if (st == SWG_OK) st = zero_bf16(db_g, N, s);
    if (st == SWG_OK) st = zero_bf16(db_fc, N, s);
    return st;
  }
  const unsigned wsflags = flags | (dg != nullptr ? SWG_WS_DG_GIVEN : 0u);
  const size_t need = swiglu_bwd_workspace_size(M, K, N, wsflags);
  if (workspace == nullptr || workspace_bytes < need) return SWG_ERR_WORKSPACE;
  if (!aligned16(workspace)) return SWG_ERR_UNSUPPORTED;
  const Range w = rng(workspace, static_cast<int64_t>(need));
  if (any_overlap(&w, 1, outs, 7) || any_overlap(&w, 1, ins, 6)) return SWG_ERR_PARAM_INVALID;

  uint8_t* wp = static_cast<uint8_t*>(workspace);
  if (flags & SWG_FUSED) {
    const int sms = swg::device_sm_count();
    const swg::FwPlan fplan = swg::fw_plan(M, K, N, sms);
    const FxSplit sp = fx_split(M, K, N, fplan, sms);
    auto fx = [&](cudaStream_t cs, int64_t t0, int64_t t1, int ctas) {
      return swg::launch_fused_x(static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(g),
                                 static_cast<const uint16_t*>(fc), static_cast<const uint16_t*>(w_g),
                                 static_cast<const uint16_t*>(w_fc), static_cast<uint16_t*>(dx),
                                 static_cast<uint16_t*>(dg), static_cast<uint16_t*>(dfc), M, K, N, cs, t0, t1, ctas);
    };
    auto fw = [&]() {
      return swg::launch_fused_w(static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(dy),
                                 static_cast<const uint16_t*>(g), static_cast<const uint16_t*>(fc),
                                 static_cast<uint16_t*>(dw_g), static_cast<uint16_t*>(dw_fc),
                                 static_cast<uint16_t*>(db_g), static_cast<uint16_t*>(db_fc), M, K, N, wp, fplan,
                                 s, acc);
    };
    if (sp.side_tiles == 0) {
      cudaError_t e = fx(s, 0, -1, 0);
      if (e == cudaSuccess) e = fw();
      return cuda_status(e);
    }
    // the w stage leaves SMs free: the last x-stage tiles run there at the same time, on a
    // side stream ordered after everything before this call, and the caller's stream waits
    // for them at the end; the other x-stage tiles follow the w stage in one persistent wave
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SWG_ERR_CUDA;
    std::lock_guard<std::mutex> lk(g_side_mu);
    SideStream* ss = nullptr;
    if (side_stream(dev, &ss) != cudaSuccess) return SWG_ERR_CUDA;
    cudaError_t e = cudaEventRecord(ss->fork, s);
    if (e == cudaSuccess) e = cudaStreamWaitEvent(ss->side, ss->fork, 0);
    if (e == cudaSuccess)
      e = swg::launch_fused_w_kernel(static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(dy),
                                     static_cast<const uint16_t*>(g), static_cast<const uint16_t*>(fc),
                                     static_cast<uint16_t*>(dw_g), static_cast<uint16_t*>(dw_fc), M, K, N, wp, fplan,
                                     s, acc);
    if (e == cudaSuccess) e = cudaEventRecord(ss->fw_done, s);
    if (e == cudaSuccess) e = fx(ss->side, sp.main_tiles, sp.main_tiles + sp.side_tiles, sp.side_ctas);
    // the w stage's reduction, too, goes on the side stream, in blocks small enough to run beside the
    // x stage's persistent wave, so that it leaves the critical path
    if (e == cudaSuccess) e = cudaStreamWaitEvent(ss->side, ss->fw_done, 0);
    if (e == cudaSuccess)
      e = swg::launch_fused_w_reduce(wp, fplan, K, N, static_cast<uint16_t*>(dw_g), static_cast<uint16_t*>(dw_fc),
                                     static_cast<uint16_t*>(db_g), static_cast<uint16_t*>(db_fc), ss->side, acc,
                                     sms);
    if (e == cudaSuccess) e = cudaEventRecord(ss->join, ss->side);
    if (e == cudaSuccess) e = fx(s, 0, sp.main_tiles, 0);
    if (e == cudaSuccess) e = cudaStreamWaitEvent(s, ss->join, 0);
    return cuda_status(e);
  }
  uint16_t* dgp = static_cast<uint16_t*>(dg);
  uint16_t* dfcp = static_cast<uint16_t*>(dfc);
  if (dgp == nullptr) {
    dgp = reinterpret_cast<uint16_t*>(wp);
    wp += align256(static_cast<size_t>(mn));
    dfcp = reinterpret_cast<uint16_t*>(wp);
    wp += align256(static_cast<size_t>(mn));
  }
  void* bws = wp;
  wp += align256(swg::b_workspace_bytes(M, N));
  void* wws = wp;
  const WPlan plan = swg::w_plan(M, K, N, swg::device_sm_count());

  cudaError_t e = swg::launch_b_stage(static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(g),
                                      static_cast<const uint16_t*>(fc), dgp, dfcp, static_cast<uint16_t*>(db_g),
                                      static_cast<uint16_t*>(db_fc), M, N, bws, s, acc);
  if (e != cudaSuccess) return SWG_ERR_CUDA;
  e = swg::launch_w_gemm(static_cast<const uint16_t*>(x), dgp, dfcp, static_cast<uint16_t*>(dw_g),
                         static_cast<uint16_t*>(dw_fc), M, K, N, wws, plan, s, acc);
  if (e != cudaSuccess) return SWG_ERR_CUDA;
  e = swg::launch_x_gemm(dgp, dfcp, static_cast<const uint16_t*>(w_g), static_cast<const uint16_t*>(w_fc),
                         static_cast<uint16_t*>(dx), M, K, N, s);
  return cuda_status(e);
}

// ---------------------------------------------------------------- row-wise operators
namespace {

inline bool known_dtype(int d) { return d == SWG_F32 || d == SWG_F16 || d == SWG_BF16; }
inline int64_t dtype_bytes(int d) { return d == SWG_F32 ? 4 : 2; }
inline bool aligned_to(const void* p, int64_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(bytes - 1)) == 0;
}
constexpr int64_t kMaxLd = int64_t(1) << 40;
// offsets in bytes of rows x n elements stay far inside 64 bits
inline bool too_large(int64_t rows, int64_t n) { return n > 0 && rows > (int64_t(1) << 58) / n; }

// rows of n elements ld apart: an input may share one row (ld 0), an output's rows are apart
inline bool ld_ok(int64_t ld, int64_t rows, int64_t n, bool output) {
  return rows <= 1 || ld >= n || (ld == 0 && !output);
}
// the bytes that such a tensor spans
inline Range rows_rng(const void* p, int64_t rows, int64_t n, int64_t ld, int64_t es) {
  return rng(p, p == nullptr || rows <= 0 || n <= 0 ? 0 : ((rows > 1 ? (rows - 1) * ld : 0) + n) * es);
}

// the checks that token_logprobs_* and distill_* share
swg_status check_vocab(const void* logits, int64_t T, int64_t V, int64_t ld, float temperature, int dtype, int itype) {
  if (T < 0 || V < 1 || !known_dtype(dtype) || (itype != SWG_I32 && itype != SWG_I64)) return SWG_ERR_PARAM_INVALID;
  const float inv = 1.0f / temperature;
  if (!(temperature > 0.0f) || !(inv > 0.0f) || inv > 3e38f) return SWG_ERR_PARAM_INVALID;
  if (!ld_ok(ld, T, V, false)) return SWG_ERR_PARAM_INVALID;
  if (T >= kMaxDim || V >= kMaxDim || too_large(T, V) || (T > 1 && (ld > kMaxLd || too_large(T, ld))))
    return SWG_ERR_UNSUPPORTED;
  if (!aligned_to(logits, dtype_bytes(dtype))) return SWG_ERR_UNSUPPORTED;
  return SWG_OK;
}
// dlogits against the logits (the same tensor, or apart from it) and the other inputs
swg_status check_dlogits(const void* dlogits, int64_t ldo, const void* logits, int64_t ld, int64_t T, int64_t V,
                         int dtype, const Range* ins, int nin) {
  const int64_t es = dtype_bytes(dtype);
  if (!ld_ok(ldo, T, V, true)) return SWG_ERR_PARAM_INVALID;
  if ((T > 1 && (ldo > kMaxLd || too_large(T, ldo))) || !aligned_to(dlogits, es)) return SWG_ERR_UNSUPPORTED;
  const Range o = rows_rng(dlogits, T, V, ldo, es);
  const bool same = dlogits == logits && (T <= 1 || ldo == ld);
  if (!same && overlap(o, rows_rng(logits, T, V, ld, es))) return SWG_ERR_PARAM_INVALID;
  return any_overlap(&o, 1, ins, nin) ? SWG_ERR_PARAM_INVALID : SWG_OK;
}

}  // namespace

swg_status layer_norm_fwd(const void* x, const void* residual, const void* gamma, const void* beta, void* h, void* y,
                          float* stats, int64_t M, int64_t N, int64_t ldx, int64_t ldr, float eps, swg_dtype dtype,
                          swg_dtype wdtype, swg_stream_t stream) {
  if (!known_dtype(dtype) || (wdtype != dtype && wdtype != SWG_F32)) return SWG_ERR_PARAM_INVALID;
  if (M < 0 || N < 0 || !(eps >= 0.0f)) return SWG_ERR_PARAM_INVALID;
  if (!ld_ok(ldx, M, N, false) || (residual != nullptr && !ld_ok(ldr, M, N, false))) return SWG_ERR_PARAM_INVALID;
  if (M >= kMaxDim || N >= kMaxDim || too_large(M, N)) return SWG_ERR_UNSUPPORTED;
  for (const int64_t ld : {ldx, residual != nullptr ? ldr : 0})
    if (M > 1 && (ld > kMaxLd || too_large(M, ld))) return SWG_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return SWG_OK;
  if (x == nullptr || y == nullptr || stats == nullptr) return SWG_ERR_NULLPTR;
  if ((residual == nullptr) != (h == nullptr)) return SWG_ERR_PARAM_INVALID;
  const int64_t es = dtype_bytes(dtype), ws = dtype_bytes(wdtype);
  if (!aligned_to(x, es) || !aligned_to(residual, es) || !aligned_to(h, es) || !aligned_to(y, es) ||
      !aligned_to(gamma, ws) || !aligned_to(beta, ws) || !aligned_to(stats, 4))
    return SWG_ERR_UNSUPPORTED;
  const Range outs[] = {rng(y, M * N * es), rng(h, h ? M * N * es : 0), rng(stats, M * 8)};
  const Range ins[] = {rows_rng(x, M, N, ldx, es), rows_rng(residual, M, N, ldr, es), rng(gamma, gamma ? N * ws : 0),
                       rng(beta, beta ? N * ws : 0)};
  if (any_overlap(outs, 3, ins, 4)) return SWG_ERR_PARAM_INVALID;
  const swg_status st = check_device();
  if (st != SWG_OK) return st;
  const swg::LnFwdArgs a{x, residual, gamma, beta, h, y, stats, M, N, M > 1 ? ldx : 0, M > 1 ? ldr : 0, eps,
                         static_cast<int>(wdtype)};
  return cuda_status(swg::launch_layer_norm_fwd(a, static_cast<int>(dtype), reinterpret_cast<cudaStream_t>(stream)));
}

size_t layer_norm_bwd_workspace_size(int64_t M, int64_t N) {
  if (M <= 0 || N <= 0 || M >= kMaxDim || N >= kMaxDim) return 0;
  return swg::ln_workspace_bytes(M, N);
}

swg_status layer_norm_bwd(const void* dy, const void* x, const float* stats, const void* gamma, const void* dh,
                          void* dx, void* dgamma, void* dbeta, int64_t M, int64_t N, int64_t lddy, int64_t ldx,
                          int64_t lddh, swg_dtype dtype, swg_dtype wdtype, void* workspace, size_t workspace_bytes,
                          swg_stream_t stream) {
  if (!known_dtype(dtype) || (wdtype != dtype && wdtype != SWG_F32)) return SWG_ERR_PARAM_INVALID;
  if (M < 0 || N < 0) return SWG_ERR_PARAM_INVALID;
  if (!ld_ok(lddy, M, N, false) || !ld_ok(ldx, M, N, false) || (dh != nullptr && !ld_ok(lddh, M, N, false)))
    return SWG_ERR_PARAM_INVALID;
  if (M >= kMaxDim || N >= kMaxDim || too_large(M, N)) return SWG_ERR_UNSUPPORTED;
  for (const int64_t ld : {lddy, ldx, dh != nullptr ? lddh : 0})
    if (M > 1 && (ld > kMaxLd || too_large(M, ld))) return SWG_ERR_UNSUPPORTED;
  if (N == 0) return SWG_OK;
  const int64_t es = dtype_bytes(dtype), ws = dtype_bytes(wdtype);
  if (!aligned_to(dy, es) || !aligned_to(x, es) || !aligned_to(dh, es) || !aligned_to(dx, es) ||
      !aligned_to(stats, 4) || !aligned_to(gamma, ws) || !aligned_to(dgamma, ws) || !aligned_to(dbeta, ws))
    return SWG_ERR_UNSUPPORTED;
  if (M > 0 && (dy == nullptr || x == nullptr || stats == nullptr || dx == nullptr)) return SWG_ERR_NULLPTR;
  const Range outs[] = {rng(dx, M * N * es), rng(dgamma, dgamma ? N * ws : 0), rng(dbeta, dbeta ? N * ws : 0)};
  const Range ins[] = {rows_rng(dy, M, N, lddy, es), rows_rng(x, M, N, ldx, es), rows_rng(dh, M, N, lddh, es),
                       rng(stats, M * 8), rng(gamma, gamma ? N * ws : 0)};
  if (any_overlap(outs, 3, ins, 5)) return SWG_ERR_PARAM_INVALID;
  const bool params = dgamma != nullptr || dbeta != nullptr;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {
    if (!params) return SWG_OK;
    const swg_status s = check_device();
    if (s != SWG_OK) return s;
    if (dgamma != nullptr && cudaMemsetAsync(dgamma, 0, static_cast<size_t>(N * ws), st) != cudaSuccess)
      return SWG_ERR_CUDA;
    if (dbeta != nullptr && cudaMemsetAsync(dbeta, 0, static_cast<size_t>(N * ws), st) != cudaSuccess)
      return SWG_ERR_CUDA;
    return SWG_OK;
  }
  if (params) {
    const size_t need = swg::ln_workspace_bytes(M, N);
    if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < need) return SWG_ERR_WORKSPACE;
    const Range w = rng(workspace, static_cast<int64_t>(need));
    if (any_overlap(&w, 1, outs, 3) || any_overlap(&w, 1, ins, 5)) return SWG_ERR_PARAM_INVALID;
  }
  const swg_status s = check_device();
  if (s != SWG_OK) return s;
  const swg::LnBwdArgs a{dy, x, stats, gamma, dh, dx, dgamma, dbeta, params ? static_cast<float*>(workspace) : nullptr,
                         M, N, M > 1 ? lddy : 0, M > 1 ? ldx : 0, M > 1 ? lddh : 0, static_cast<int>(wdtype)};
  return cuda_status(swg::launch_layer_norm_bwd(a, static_cast<int>(dtype), st));
}

swg_status token_logprobs_fwd(const void* logits, const void* targets, float* logp, float* entropy, float* stats,
                              float* top_logp, int64_t* top_idx, int64_t T, int64_t V, int64_t ld, int top_k,
                              float temperature, int64_t ignore_index, swg_dtype dtype, swg_itype itype,
                              swg_stream_t stream) {
  const swg_status st = check_vocab(logits, T, V, ld, temperature, dtype, itype);
  if (st != SWG_OK) return st;
  if (top_k < 0 || top_k > swg::kMaxTop || top_k > V) return SWG_ERR_PARAM_INVALID;
  if (T == 0) return SWG_OK;
  if (logits == nullptr || entropy == nullptr || stats == nullptr || (targets != nullptr && logp == nullptr) ||
      (top_k > 0 && (top_logp == nullptr || top_idx == nullptr)))
    return SWG_ERR_NULLPTR;
  const int64_t is = itype == SWG_I64 ? 8 : 4;
  if (!aligned_to(targets, is) || !aligned_to(logp, 4) || !aligned_to(entropy, 4) || !aligned_to(stats, 4) ||
      !aligned_to(top_logp, 4) || !aligned_to(top_idx, 8))
    return SWG_ERR_UNSUPPORTED;
  const Range outs[] = {rng(logp, targets ? T * 4 : 0), rng(entropy, T * 4), rng(stats, T * 8),
                        rng(top_logp, T * top_k * 4), rng(top_idx, T * top_k * 8)};
  const Range ins[] = {rows_rng(logits, T, V, ld, dtype_bytes(dtype)), rng(targets, targets ? T * is : 0)};
  if (any_overlap(outs, 5, ins, 2)) return SWG_ERR_PARAM_INVALID;
  const swg_status dv = check_device();
  if (dv != SWG_OK) return dv;
  const swg::TlpFwdArgs a{logits, targets, logp, entropy, stats, top_logp, top_idx, T, V, T > 1 ? ld : 0,
                          ignore_index, top_k, itype == SWG_I64, 1.0f / temperature};
  return cuda_status(
      swg::launch_token_logprobs_fwd(a, static_cast<int>(dtype), reinterpret_cast<cudaStream_t>(stream)));
}

swg_status token_logprobs_bwd(const float* dlogp, const void* logits, const void* targets, const float* stats,
                              const float* dentropy, const float* entropy, void* dlogits, int64_t T, int64_t V,
                              int64_t ld, int64_t ldo, float temperature, int64_t ignore_index, swg_dtype dtype,
                              swg_itype itype, swg_stream_t stream) {
  const swg_status st = check_vocab(logits, T, V, ld, temperature, dtype, itype);
  if (st != SWG_OK) return st;
  if (T == 0) return SWG_OK;
  if (logits == nullptr || stats == nullptr || dlogits == nullptr || (targets != nullptr && dlogp == nullptr) ||
      (dentropy != nullptr && entropy == nullptr))
    return SWG_ERR_NULLPTR;
  const int64_t is = itype == SWG_I64 ? 8 : 4;
  if (!aligned_to(targets, is) || !aligned_to(dlogp, 4) || !aligned_to(entropy, 4) || !aligned_to(stats, 4) ||
      !aligned_to(dentropy, 4))
    return SWG_ERR_UNSUPPORTED;
  const Range ins[] = {rng(targets, targets ? T * is : 0), rng(dlogp, dlogp ? T * 4 : 0), rng(stats, T * 8),
                       rng(entropy, dentropy ? T * 4 : 0), rng(dentropy, dentropy ? T * 4 : 0)};
  const swg_status al = check_dlogits(dlogits, ldo, logits, ld, T, V, dtype, ins, 5);
  if (al != SWG_OK) return al;
  const swg_status dv = check_device();
  if (dv != SWG_OK) return dv;
  const swg::TlpBwdArgs a{logits, targets, stats, dlogp, entropy, dentropy, dlogits, T, V, T > 1 ? ld : 0,
                          T > 1 ? ldo : 0, ignore_index, itype == SWG_I64, 1.0f / temperature};
  return cuda_status(
      swg::launch_token_logprobs_bwd(a, static_cast<int>(dtype), reinterpret_cast<cudaStream_t>(stream)));
}

namespace {

// the three distillation entry points: forward when loss is wanted, backward when dlogits is
swg_status distill(const void* logits, const void* ids, const void* teacher, const float* weight,
                   const float* stats_in, float* loss, float* stats, void* dlogits, int64_t T, int64_t V, int64_t ld,
                   int64_t ldo, int64_t K, float temperature, swg_dtype dtype, swg_dtype tdtype, swg_itype itype,
                   swg_stream_t stream, bool forward, bool backward) {
  const swg_status st = check_vocab(logits, T, V, ld, temperature, dtype, itype);
  if (st != SWG_OK) return st;
  if (K < 1 || !known_dtype(tdtype)) return SWG_ERR_PARAM_INVALID;
  if (K > swg::kKdMaxEntries) return SWG_ERR_UNSUPPORTED;
  if (T == 0) return SWG_OK;
  if (logits == nullptr || ids == nullptr || teacher == nullptr || (forward && (loss == nullptr || stats == nullptr)) ||
      (backward && (weight == nullptr || dlogits == nullptr)) || (!forward && stats_in == nullptr))
    return SWG_ERR_NULLPTR;
  const int64_t is = itype == SWG_I64 ? 8 : 4, es = dtype_bytes(dtype), ts = dtype_bytes(tdtype);
  if (!aligned_to(ids, is) || !aligned_to(teacher, ts) || !aligned_to(weight, 4) || !aligned_to(stats_in, 4) ||
      !aligned_to(loss, 4) || !aligned_to(stats, 4))
    return SWG_ERR_UNSUPPORTED;
  const Range ins[] = {rng(ids, T * K * is), rng(teacher, T * K * ts), rng(weight, backward ? T * 4 : 0),
                       rng(stats_in, forward ? 0 : T * 8), rng(loss, forward ? T * 4 : 0),
                       rng(stats, forward ? T * 8 : 0)};
  if (backward) {
    const swg_status al = check_dlogits(dlogits, ldo, logits, ld, T, V, dtype, ins, 6);
    if (al != SWG_OK) return al;
  }
  const Range in4[] = {ins[0], ins[1], ins[2], rows_rng(logits, T, V, ld, es)};
  if (forward && any_overlap(ins + 4, 2, in4, 4)) return SWG_ERR_PARAM_INVALID;
  const swg_status dv = check_device();
  if (dv != SWG_OK) return dv;
  const swg::KdArgs a{logits, ids, teacher, weight, stats_in, loss, stats, dlogits, T, V, T > 1 ? ld : 0,
                      T > 1 ? ldo : 0, static_cast<int>(K), static_cast<int>(tdtype), itype == SWG_I64,
                      1.0f / temperature};
  return cuda_status(swg::launch_distill(a, forward, backward, static_cast<int>(dtype),
                                         reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

swg_status distill_fwd(const void* logits, const void* ids, const void* teacher, float* loss, float* stats, int64_t T,
                       int64_t V, int64_t ld, int64_t K, float temperature, swg_dtype dtype, swg_dtype tdtype,
                       swg_itype itype, swg_stream_t stream) {
  return distill(logits, ids, teacher, nullptr, nullptr, loss, stats, nullptr, T, V, ld, 0, K, temperature, dtype,
                 tdtype, itype, stream, true, false);
}

swg_status distill_bwd(const float* weight, const void* logits, const void* ids, const void* teacher,
                       const float* stats, void* dlogits, int64_t T, int64_t V, int64_t ld, int64_t ldo, int64_t K,
                       float temperature, swg_dtype dtype, swg_dtype tdtype, swg_itype itype, swg_stream_t stream) {
  return distill(logits, ids, teacher, weight, stats, nullptr, nullptr, dlogits, T, V, ld, ldo, K, temperature, dtype,
                 tdtype, itype, stream, false, true);
}

swg_status distill_fwd_bwd(const void* logits, const void* ids, const void* teacher, const float* weight, float* loss,
                           float* stats, void* dlogits, int64_t T, int64_t V, int64_t ld, int64_t ldo, int64_t K,
                           float temperature, swg_dtype dtype, swg_dtype tdtype, swg_itype itype,
                           swg_stream_t stream) {
  return distill(logits, ids, teacher, weight, nullptr, loss, stats, dlogits, T, V, ld, ldo, K, temperature, dtype,
                 tdtype, itype, stream, true, true);
}

// ---------------------------------------------------------------- norms between blocks
namespace {

inline bool finite(float v) { return v - v == 0.0f; }

// sizes, types and flags that block_norm_fwd and block_norm_bwd share
swg_status check_block_norm(int64_t M, int64_t N, int64_t G, const void* gate, const void* gamma_post,
                            const void* gamma_pre, float alpha, unsigned flags, int dtype, int wdtype, int gdtype) {
  if (!known_dtype(dtype) || (wdtype != dtype && wdtype != SWG_F32) || (gdtype != dtype && gdtype != SWG_F32))
    return SWG_ERR_PARAM_INVALID;
  if (M < 0 || N < 0 || G < 0 || !finite(alpha)) return SWG_ERR_PARAM_INVALID;
  if (flags == 0 || (flags & ~(SWG_NORM_POST | SWG_NORM_PRE)) != 0) return SWG_ERR_PARAM_INVALID;
  if ((gamma_post != nullptr && !(flags & SWG_NORM_POST)) || (gamma_pre != nullptr && !(flags & SWG_NORM_PRE)))
    return SWG_ERR_PARAM_INVALID;
  if (M >= kMaxDim || N >= kMaxDim || too_large(M, N)) return SWG_ERR_UNSUPPORTED;
  if (G > 0 && M % G != 0) return SWG_ERR_PARAM_INVALID;
  if (gate != nullptr && G == 0 && M > 0) return SWG_ERR_PARAM_INVALID;
  const int64_t ws = dtype_bytes(wdtype);
  if (!aligned_to(gamma_post, ws) || !aligned_to(gamma_pre, ws) || !aligned_to(gate, dtype_bytes(gdtype)))
    return SWG_ERR_UNSUPPORTED;
  return SWG_OK;
}

}  // namespace

swg_status block_norm_fwd(const void* u, const void* residual, const void* gamma_post, const void* gamma_pre,
                          const void* gate, void* h, void* y, float* stats, int64_t M, int64_t N, int64_t G,
                          int64_t ldu, int64_t ldr, float alpha, float eps, unsigned flags, swg_dtype dtype,
                          swg_dtype wdtype, swg_dtype gdtype, swg_stream_t stream) {
  swg_status st = check_block_norm(M, N, G, gate, gamma_post, gamma_pre, alpha, flags, dtype, wdtype, gdtype);
  if (st != SWG_OK) return st;
  if (!(eps >= 0.0f)) return SWG_ERR_PARAM_INVALID;
  if (!ld_ok(ldu, M, N, false) || (residual != nullptr && !ld_ok(ldr, M, N, false))) return SWG_ERR_PARAM_INVALID;
  for (const int64_t ld : {ldu, residual != nullptr ? ldr : 0})
    if (M > 1 && (ld > kMaxLd || too_large(M, ld))) return SWG_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return SWG_OK;
  const bool post = (flags & SWG_NORM_POST) != 0, pre = (flags & SWG_NORM_PRE) != 0;
  if (u == nullptr || stats == nullptr || (pre && y == nullptr) || (G > 0 && gate == nullptr)) return SWG_ERR_NULLPTR;
  if ((!pre && y != nullptr) || (h != nullptr) != (post || residual != nullptr || gate != nullptr))
    return SWG_ERR_PARAM_INVALID;
  const int64_t es = dtype_bytes(dtype), ws = dtype_bytes(wdtype);
  if (!aligned_to(u, es) || !aligned_to(residual, es) || !aligned_to(h, es) || !aligned_to(y, es) ||
      !aligned_to(stats, 4))
    return SWG_ERR_UNSUPPORTED;
  const Range outs[] = {rng(y, y ? M * N * es : 0), rng(h, h ? M * N * es : 0), rng(stats, M * 8)};
  const Range ins[] = {rows_rng(u, M, N, ldu, es), rows_rng(residual, M, N, ldr, es),
                       rng(gamma_post, gamma_post ? N * ws : 0), rng(gamma_pre, gamma_pre ? N * ws : 0),
                       rng(gate, gate ? G * N * dtype_bytes(gdtype) : 0)};
  if (any_overlap(outs, 3, ins, 5)) return SWG_ERR_PARAM_INVALID;
  st = check_device();
  if (st != SWG_OK) return st;
  const swg::BnFwdArgs a{u, residual, gamma_post, gamma_pre, gate, h, y, stats, M, N, M > 1 ? ldu : 0,
                         M > 1 ? ldr : 0, gate != nullptr ? M / G : M, alpha, eps, static_cast<int>(wdtype),
                         static_cast<int>(gdtype), post, pre};
  return cuda_status(swg::launch_block_norm_fwd(a, static_cast<int>(dtype), reinterpret_cast<cudaStream_t>(stream)));
}

size_t block_norm_bwd_workspace_size(int64_t M, int64_t N, int64_t G) {
  if (M <= 0 || N <= 0 || G < 0 || M >= kMaxDim || N >= kMaxDim || (G > 0 && M % G != 0)) return 0;
  return swg::bn_workspace_bytes(M, N, G > 0 ? M / G : M);
}

swg_status block_norm_bwd(const void* dy, const void* dh, const void* u, const void* h, const float* stats,
                          const void* gamma_post, const void* gamma_pre, const void* gate, void* du, void* dresidual,
                          void* dgamma_post, void* dgamma_pre, void* dgate, int64_t M, int64_t N, int64_t G,
                          int64_t lddy, int64_t lddh, int64_t ldu, int64_t ldh, float alpha, unsigned flags,
                          swg_dtype dtype, swg_dtype wdtype, swg_dtype gdtype, void* workspace,
                          size_t workspace_bytes, swg_stream_t stream) {
  swg_status st = check_block_norm(M, N, G, gate, gamma_post, gamma_pre, alpha, flags, dtype, wdtype, gdtype);
  if (st != SWG_OK) return st;
  const bool post = (flags & SWG_NORM_POST) != 0, pre = (flags & SWG_NORM_PRE) != 0;
  if (!ld_ok(ldu, M, N, false) || (pre && (!ld_ok(lddy, M, N, false) || !ld_ok(ldh, M, N, false))) ||
      (dh != nullptr && !ld_ok(lddh, M, N, false)))
    return SWG_ERR_PARAM_INVALID;
  for (const int64_t ld : {ldu, pre ? lddy : 0, pre ? ldh : 0, dh != nullptr ? lddh : 0})
    if (M > 1 && (ld > kMaxLd || too_large(M, ld))) return SWG_ERR_UNSUPPORTED;
  if ((!pre && (dy != nullptr || h != nullptr || dgamma_pre != nullptr)) || (!post && dgamma_post != nullptr) ||
      (dgate != nullptr && G == 0 && M > 0))
    return SWG_ERR_PARAM_INVALID;
  if (N == 0) return SWG_OK;
  const int64_t es = dtype_bytes(dtype), ws = dtype_bytes(wdtype), gs = dtype_bytes(gdtype);
  if (!aligned_to(dy, es) || !aligned_to(dh, es) || !aligned_to(u, es) || !aligned_to(h, es) || !aligned_to(du, es) ||
      !aligned_to(dresidual, es) || !aligned_to(stats, 4) || !aligned_to(dgamma_post, ws) ||
      !aligned_to(dgamma_pre, ws) || !aligned_to(dgate, gs))
    return SWG_ERR_UNSUPPORTED;
  if (M > 0 && (u == nullptr || stats == nullptr || du == nullptr || (pre && (dy == nullptr || h == nullptr)) ||
                (!pre && dh == nullptr) || (G > 0 && gate == nullptr)))
    return SWG_ERR_NULLPTR;
  const Range outs[] = {rng(du, M * N * es), rng(dresidual, dresidual ? M * N * es : 0),
                        rng(dgamma_post, dgamma_post ? N * ws : 0), rng(dgamma_pre, dgamma_pre ? N * ws : 0),
                        rng(dgate, dgate ? G * N * gs : 0)};
  const Range ins[] = {rows_rng(dy, M, N, lddy, es), rows_rng(dh, M, N, lddh, es), rows_rng(u, M, N, ldu, es),
                       rows_rng(h, M, N, ldh, es), rng(stats, M * 8), rng(gamma_post, gamma_post ? N * ws : 0),
                       rng(gamma_pre, gamma_pre ? N * ws : 0), rng(gate, gate ? G * N * gs : 0)};
  if (any_overlap(outs, 5, ins, 8)) return SWG_ERR_PARAM_INVALID;
  const bool params = dgamma_post != nullptr || dgamma_pre != nullptr || dgate != nullptr;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {
    if (!params) return SWG_OK;
    st = check_device();
    if (st != SWG_OK) return st;
    const struct {
      void* p;
      int64_t bytes;
    } zero[] = {{dgamma_post, N * ws}, {dgamma_pre, N * ws}, {dgate, G * N * gs}};
    for (const auto& z : zero)
      if (z.p != nullptr && z.bytes > 0 && cudaMemsetAsync(z.p, 0, static_cast<size_t>(z.bytes), s) != cudaSuccess)
        return SWG_ERR_CUDA;
    return SWG_OK;
  }
  const int64_t per_gate = gate != nullptr ? M / G : M;
  if (params) {
    const size_t need = swg::bn_workspace_bytes(M, N, per_gate);
    if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < need) return SWG_ERR_WORKSPACE;
    const Range w = rng(workspace, static_cast<int64_t>(need));
    if (any_overlap(&w, 1, outs, 5) || any_overlap(&w, 1, ins, 8)) return SWG_ERR_PARAM_INVALID;
  }
  st = check_device();
  if (st != SWG_OK) return st;
  const swg::BnBwdArgs a{dy, dh, u, h, stats, gamma_post, gamma_pre, gate, du, dresidual, dgamma_post, dgamma_pre,
                         dgate, M, N, M > 1 ? lddy : 0, M > 1 ? lddh : 0, M > 1 ? ldu : 0, M > 1 ? ldh : 0, per_gate,
                         alpha, static_cast<int>(wdtype), static_cast<int>(gdtype), post, pre, nullptr, nullptr};
  return cuda_status(swg::launch_block_norm_bwd(a, params ? workspace : nullptr, static_cast<int>(dtype), s));
}

// ---------------------------------------------------------------- linear layer
namespace {

inline bool known_act(int act) {
  return act == SWG_ACT_SILU || act == SWG_ACT_GELU || act == SWG_ACT_HARDSWISH || act == SWG_ACT_NONE;
}
// rows of n elements that TMA reads: 16-byte multiples apart
inline swg_status tma_ld(int64_t ld, int64_t rows, int64_t n) {
  if (rows > 1 && ld < n) return SWG_ERR_PARAM_INVALID;
  return rows > 1 && (ld % 8 != 0 || ld > kMaxLd / 2 || too_large(rows, ld)) ? SWG_ERR_UNSUPPORTED : SWG_OK;
}
swg_status check_linear(int64_t M, int64_t K, int64_t N, int act, int dtype, int bdtype) {
  if ((dtype != SWG_F16 && dtype != SWG_BF16) || (bdtype != dtype && bdtype != SWG_F32) || !known_act(act))
    return SWG_ERR_PARAM_INVALID;
  const swg_status st = check_shape(M, K, N);
  if (st != SWG_OK) return st;
  // every tile's index fits 32 bits
  return too_large(M, std::max(K, N)) || too_large(K, N) || M > kMaxDim - 512 || K > kMaxDim - 512 || N > kMaxDim - 512
             ? SWG_ERR_UNSUPPORTED
             : SWG_OK;
}

}  // namespace

swg_status linear_fwd(const void* x, const void* w, const void* b, const void* residual, void* y, void* z, int64_t M,
                      int64_t K, int64_t N, int64_t ldx, int64_t ldr, swg_act act, swg_dtype dtype, swg_dtype bdtype,
                      swg_stream_t stream) {
  swg_status st = check_linear(M, K, N, act, dtype, bdtype);
  if (st == SWG_OK) st = tma_ld(ldx, M, K);
  if (st == SWG_OK && residual != nullptr) st = tma_ld(ldr, M, N);
  if (st != SWG_OK) return st;
  if (K == 0) return SWG_ERR_UNSUPPORTED;  // the product needs a reduction of positive length
  if (M == 0 || N == 0) return SWG_OK;
  if (!x || !w || !y) return SWG_ERR_NULLPTR;
  for (const void* p : {x, w, b, residual, static_cast<const void*>(y), static_cast<const void*>(z)})
    if (!aligned16(p)) return SWG_ERR_UNSUPPORTED;
  const int64_t mn = M * N * 2;
  const Range outs[] = {rng(y, mn), rng(z, z ? mn : 0)};
  const Range ins[] = {rows_rng(x, M, K, ldx, 2), rng(w, K * N * 2), rng(b, b ? N * dtype_bytes(bdtype) : 0)};
  const Range res = rows_rng(residual, M, N, ldr, 2);
  if (any_overlap(outs, 2, ins, 3) || overlap(outs[1], res)) return SWG_ERR_PARAM_INVALID;
  // the residual may be y itself
  if (overlap(outs[0], res) && !(residual == y && (M == 1 || ldr == N))) return SWG_ERR_PARAM_INVALID;
  st = check_device();
  if (st != SWG_OK) return st;
  const swg::LinearEpilogue e{b, residual, y, z, M > 1 ? ldr : N, static_cast<int>(act), dtype == SWG_F16,
                              bdtype == SWG_F32};
  return cuda_status(swg::launch_linear_fwd(x, w, e, M, K, N, M > 1 ? ldx : K, reinterpret_cast<cudaStream_t>(stream)));
}

size_t linear_bwd_workspace_size(int64_t M, int64_t K, int64_t N, swg_act act) {
  if (M <= 0 || K < 0 || N <= 0 || check_linear(M, K, N, act, SWG_BF16, SWG_BF16) != SWG_OK) return 0;
  return align256(swg::linear_dz_workspace_bytes(M, N)) +
         (K > 0 ? align256(swg::linear_dw_workspace_bytes(M, K, N)) : 0) +
         (act != SWG_ACT_NONE ? align256(static_cast<size_t>(M) * static_cast<size_t>(N) * 2) : 0);
}

swg_status linear_bwd(const void* dy, const void* x, const void* w, const void* z, void* dx, void* dw, void* db,
                      int64_t M, int64_t K, int64_t N, int64_t lddy, int64_t ldx, swg_act act, unsigned flags,
                      swg_dtype dtype, swg_dtype bdtype, void* workspace, size_t workspace_bytes,
                      swg_stream_t stream) {
  swg_status st = check_linear(M, K, N, act, dtype, bdtype);
  if (st == SWG_OK) st = tma_ld(lddy, M, N);
  if (st == SWG_OK && dw != nullptr) st = tma_ld(ldx, M, K);
  if (st != SWG_OK) return st;
  if ((flags & ~SWG_ACCUMULATE) != 0) return SWG_ERR_PARAM_INVALID;
  const bool acc = (flags & SWG_ACCUMULATE) != 0;
  const bool want_dx = dx != nullptr && K > 0 && M > 0, want_dw = dw != nullptr && K > 0 && N > 0,
             want_db = db != nullptr && N > 0;
  if (!want_dx && !want_dw && !want_db) return SWG_OK;
  const bool some = M > 0 && N > 0;  // dz has elements
  if (some && (!dy || (want_dw && !x) || (want_dx && !w) || (act != SWG_ACT_NONE && !z))) return SWG_ERR_NULLPTR;
  for (const void* p : {dy, x, w, z, static_cast<const void*>(dx), static_cast<const void*>(dw),
                        static_cast<const void*>(db)})
    if (!aligned16(p)) return SWG_ERR_UNSUPPORTED;
  const int64_t mn = M * N * 2, mk = M * K * 2, kn = K * N * 2;
  const Range outs[] = {rng(dx, dx ? mk : 0), rng(dw, dw ? kn : 0), rng(db, db ? N * dtype_bytes(bdtype) : 0)};
  const Range ins[] = {rows_rng(dy, M, N, lddy, 2), rows_rng(x, M, K, ldx, 2), rng(w, w ? kn : 0),
                       rng(z, z ? mn : 0)};
  if (any_overlap(outs, 3, ins, 4)) return SWG_ERR_PARAM_INVALID;
  const bool act_on = act != SWG_ACT_NONE;
  // the column sums' parts, those of dw, and dz
  const size_t sums = align256(swg::linear_dz_workspace_bytes(M, N));
  const size_t parts = some && K > 0 ? align256(swg::linear_dw_workspace_bytes(M, K, N)) : 0;
  if (some && (want_db || act_on || (want_dw && parts > 0))) {
    const size_t need = linear_bwd_workspace_size(M, K, N, act);
    if (workspace == nullptr || workspace_bytes < need) return SWG_ERR_WORKSPACE;
    if (!aligned16(workspace)) return SWG_ERR_UNSUPPORTED;
    const Range ws = rng(workspace, static_cast<int64_t>(need));
    if (any_overlap(&ws, 1, outs, 3) || any_overlap(&ws, 1, ins, 4)) return SWG_ERR_PARAM_INVALID;
  }
  st = check_device();
  if (st != SWG_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!some) {  // sums over nothing
    cudaError_t e = cudaSuccess;
    if (want_dx) e = cudaMemsetAsync(dx, 0, static_cast<size_t>(mk), s);
    if (e == cudaSuccess && want_dw && !acc) e = cudaMemsetAsync(dw, 0, static_cast<size_t>(kn), s);
    if (e == cudaSuccess && want_db && !acc)
      e = cudaMemsetAsync(db, 0, static_cast<size_t>(N * dtype_bytes(bdtype)), s);
    return cuda_status(e);
  }
  const bool f16 = dtype == SWG_F16;
  const void* dz = dy;
  int64_t lddz = M > 1 ? lddy : N;
  cudaError_t e = cudaSuccess;
  if (want_db || act_on) {
    void* to = act_on ? static_cast<char*>(workspace) + sums + parts : nullptr;
    e = swg::launch_linear_dz(dy, z, to, want_db ? db : nullptr, M, N, lddz, static_cast<int>(act), f16,
                              bdtype == SWG_F32, acc, static_cast<float*>(workspace), s);
    if (act_on) {
      dz = to;
      lddz = N;
    }
  }
  if (e == cudaSuccess && want_dw) {
    const swg::LinearEpilogue epi{nullptr, acc ? dw : nullptr, dw, nullptr, N, swg::kLinearNoAct, f16, false};
    e = swg::launch_linear_dw(x, dz, epi, M, K, N, M > 1 ? ldx : K, lddz,
                              reinterpret_cast<float*>(static_cast<char*>(workspace) + sums), s);
  }
  if (e == cudaSuccess && want_dx) {
    const swg::LinearEpilogue epi{nullptr, nullptr, dx, nullptr, K, swg::kLinearNoAct, f16, false};
    e = swg::launch_linear_dx(dz, w, epi, M, K, N, lddz, s);
  }
  return cuda_status(e);
}

}  // extern "C"
