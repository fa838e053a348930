// Layer norm over the last dimension, forward and backward.
//   h = x + r rounded to the I/O type (h = x without a residual r)
//   mu = sum h / N,  var = sum (h - mu)^2 / N,  rstd = 1 / sqrt(var + eps)
//   y = (h - mu) rstd gamma + beta
// Backward, with x_hat = (h - mu) rstd and g = dy gamma, from the saved (mu, rstd):
//   dx = rstd (g - mean(g) - x_hat mean(g x_hat)) (+ dh, the gradient that reaches h by another path)
//   dgamma = sum over rows of dy x_hat,  dbeta = sum over rows of dy
// All arithmetic is fp32; h, y and dx are rounded once.
#include "row_ops.cuh"
#include "swg_launch.h"

namespace swg {
namespace {

using namespace row;

constexpr int kThreads = 256;
constexpr int kColThreads = 128;    // columns per block of the weight-gradient kernel
constexpr int64_t kRowChunks = 64;  // row chunks of the weight-gradient kernel, at most

template <typename T>
__global__ void __launch_bounds__(kThreads) ln_fwd_kernel(const LnFwdArgs a) {
  __shared__ float buf[kThreads / 32];
  const float inv_n = 1.0f / static_cast<float>(a.N);
  for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    const T* res = a.residual != nullptr ? static_cast<const T*>(a.residual) + r * a.ldr : nullptr;
    T* h = a.h != nullptr ? static_cast<T*>(a.h) + r * a.N : nullptr;
    T* y = static_cast<T*>(a.y) + r * a.N;
    auto value = [&](int64_t j) {  // h_j, rounded as it is stored
      return res == nullptr ? to_f(x[j]) : to_f(from_f<T>(to_f(x[j]) + to_f(res[j])));
    };
    float s = 0.f;
    for (int64_t j = threadIdx.x; j < a.N; j += kThreads) s += value(j);
    const float mu = block_sum(s, buf) * inv_n;
    float q = 0.f;
    for (int64_t j = threadIdx.x; j < a.N; j += kThreads) {
      const float d = value(j) - mu;
      q = fmaf(d, d, q);
    }
    const float rstd = 1.0f / sqrtf(block_sum(q, buf) * inv_n + a.eps);
    for (int64_t j = threadIdx.x; j < a.N; j += kThreads) {
      const float v = value(j);
      const float g = a.gamma != nullptr ? load_any(a.gamma, j, a.wdtype) : 1.0f;
      const float b = a.beta != nullptr ? load_any(a.beta, j, a.wdtype) : 0.0f;
      y[j] = from_f<T>(fmaf((v - mu) * rstd, g, b));
      if (h != nullptr) h[j] = from_f<T>(v);
    }
    if (threadIdx.x == 0) {
      a.stats[2 * r] = mu;
      a.stats[2 * r + 1] = rstd;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) ln_dx_kernel(const LnBwdArgs a) {
  __shared__ float buf[kThreads / 32];
  const float inv_n = 1.0f / static_cast<float>(a.N);
  for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + r * a.lddy;
    const T* dh = a.dh != nullptr ? static_cast<const T*>(a.dh) + r * a.lddh : nullptr;
    T* dx = static_cast<T*>(a.dx) + r * a.N;
    const float mu = a.stats[2 * r], rstd = a.stats[2 * r + 1];
    float sa = 0.f, sb = 0.f;
    for (int64_t j = threadIdx.x; j < a.N; j += kThreads) {
      const float g = to_f(dy[j]) * (a.gamma != nullptr ? load_any(a.gamma, j, a.wdtype) : 1.0f);
      sa += g;
      sb = fmaf(g, (to_f(x[j]) - mu) * rstd, sb);
    }
    sa = block_sum(sa, buf) * inv_n;
    sb = block_sum(sb, buf) * inv_n;
    for (int64_t j = threadIdx.x; j < a.N; j += kThreads) {
      const float g = to_f(dy[j]) * (a.gamma != nullptr ? load_any(a.gamma, j, a.wdtype) : 1.0f);
      const float v = rstd * (g - sa - (to_f(x[j]) - mu) * rstd * sb);
      dx[j] = from_f<T>(dh != nullptr ? v + to_f(dh[j]) : v);
    }
  }
}

// one row chunk's column sums of dy x_hat and dy -> part [chunks][2][N]
template <typename T>
__global__ void __launch_bounds__(kColThreads) ln_param_kernel(const LnBwdArgs a, int64_t rows_per_chunk) {
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kColThreads + threadIdx.x;
  if (j >= a.N) return;
  const int64_t r0 = blockIdx.y * rows_per_chunk, r1 = min(a.M, r0 + rows_per_chunk);
  float sg = 0.f, sb = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const float d = to_f(static_cast<const T*>(a.dy)[r * a.lddy + j]);
    const float xh = (to_f(static_cast<const T*>(a.x)[r * a.ldx + j]) - a.stats[2 * r]) * a.stats[2 * r + 1];
    sg = fmaf(d, xh, sg);
    sb += d;
  }
  float* p = a.part + static_cast<int64_t>(blockIdx.y) * 2 * a.N;
  p[j] = sg;
  p[a.N + j] = sb;
}

__global__ void __launch_bounds__(kColThreads) ln_param_reduce_kernel(const float* part, int64_t chunks, int64_t N,
                                                                      void* dgamma, void* dbeta, int wdtype) {
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kColThreads + threadIdx.x;
  if (j >= N) return;
  float sg = 0.f, sb = 0.f;
  for (int64_t c = 0; c < chunks; ++c) {
    sg += part[c * 2 * N + j];
    sb += part[c * 2 * N + N + j];
  }
  if (dgamma != nullptr) store_any(dgamma, j, wdtype, sg);
  if (dbeta != nullptr) store_any(dbeta, j, wdtype, sb);
}

int64_t ln_chunks(int64_t M) { return M < kRowChunks ? M : kRowChunks; }
unsigned row_grid(int64_t M) { return static_cast<unsigned>(M < 65536 ? M : 65536); }

}  // namespace

size_t ln_workspace_bytes(int64_t M, int64_t N) {
  return static_cast<size_t>(ln_chunks(M)) * 2 * static_cast<size_t>(N) * sizeof(float);
}

cudaError_t launch_layer_norm_fwd(const LnFwdArgs& a, int dtype, cudaStream_t stream) {
  const unsigned grid = row_grid(a.M);
  if (dtype == 0) ln_fwd_kernel<float><<<grid, kThreads, 0, stream>>>(a);
  else if (dtype == 1) ln_fwd_kernel<__half><<<grid, kThreads, 0, stream>>>(a);
  else ln_fwd_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_layer_norm_bwd(const LnBwdArgs& a, int dtype, cudaStream_t stream) {
  const unsigned grid = row_grid(a.M);
  if (dtype == 0) ln_dx_kernel<float><<<grid, kThreads, 0, stream>>>(a);
  else if (dtype == 1) ln_dx_kernel<__half><<<grid, kThreads, 0, stream>>>(a);
  else ln_dx_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(a);
  if (a.dgamma != nullptr || a.dbeta != nullptr) {
    const int64_t chunks = ln_chunks(a.M), per = (a.M + chunks - 1) / chunks;
    const dim3 g(static_cast<unsigned>((a.N + kColThreads - 1) / kColThreads), static_cast<unsigned>(chunks));
    if (dtype == 0) ln_param_kernel<float><<<g, kColThreads, 0, stream>>>(a, per);
    else if (dtype == 1) ln_param_kernel<__half><<<g, kColThreads, 0, stream>>>(a, per);
    else ln_param_kernel<__nv_bfloat16><<<g, kColThreads, 0, stream>>>(a, per);
    ln_param_reduce_kernel<<<g.x, kColThreads, 0, stream>>>(a.part, chunks, a.N, a.dgamma, a.dbeta, a.wdtype);
  }
  return cudaGetLastError();
}

}  // namespace swg
