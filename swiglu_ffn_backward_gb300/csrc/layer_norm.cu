// Layer norm over the last dimension, forward and backward.
//   h = x + r rounded to the I/O type (h = x without a residual r)
//   mu = sum h / N,  var = sum (h - mu)^2 / N,  rstd = 1 / sqrt(var + eps)
//   y = (h - mu) rstd gamma + beta
// Backward, with x_hat = (h - mu) rstd and g = dy gamma, from the saved (mu, rstd):
//   dx = rstd (g - mean(g) - x_hat mean(g x_hat)) (+ dh, the gradient that reaches h by another path)
//   dgamma = sum over rows of dy x_hat,  dbeta = sum over rows of dy
// All arithmetic is fp32; h, y and dx are rounded once.
//
// Bound by HBM: two to four tensors of M N elements are read or written, with some ten operations an
// element. A group of 32 to 1024 threads holds a row in registers, so each element is read once: the
// variance is taken of centred values in a second pass over the registers. Vectors are the widest that
// the row length, strides and addresses allow (16 bytes, 4 bytes or one element). Rows too long for the
// registers of a block are read again (ln_fwd_long_kernel, ln_dx_long_kernel).
// The groups are persistent and load the next row under the work on this one.
// Backward: each thread has the same columns of every row, so the columns' sums of dgamma and dbeta stay
// in registers. The blocks' sums go to the workspace and are added by a second kernel in a fixed order.
#include <mutex>

#include "row_ops.cuh"
#include "swg_launch.h"

namespace swg {
namespace {

using namespace row;

// E elements in one load
template <int kBytes>
struct Raw;
template <>
struct Raw<16> {
  uint4 u;
};
template <>
struct Raw<8> {
  uint2 u;
};
template <>
struct Raw<4> {
  uint32_t u;
};
template <>
struct Raw<2> {
  uint16_t u;
};
template <int kBytes>
constexpr int kRegs = (kBytes + 3) / 4;  // registers of one
template <int kBytes>
__device__ __forceinline__ Raw<kBytes> ld_stream(const void* p);
template <>
__device__ __forceinline__ Raw<16> ld_stream<16>(const void* p) {
  Raw<16> r;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(r.u.x), "=r"(r.u.y), "=r"(r.u.z), "=r"(r.u.w)
      : "l"(p));
  return r;
}
template <>
__device__ __forceinline__ Raw<4> ld_stream<4>(const void* p) {
  return Raw<4>{__ldg(static_cast<const uint32_t*>(p))};
}
template <>
__device__ __forceinline__ Raw<2> ld_stream<2>(const void* p) {
  return Raw<2>{__ldg(static_cast<const uint16_t*>(p))};
}
// 16-bit elements are widened and narrowed two at a time, word by word
__device__ __forceinline__ float2 widen(uint32_t u, __half) {
  const __half2 h = *reinterpret_cast<const __half2*>(&u);
  return __half22float2(h);
}
__device__ __forceinline__ float2 widen(uint32_t u, __nv_bfloat16) { return bf16x2_to_f2(u); }
__device__ __forceinline__ uint32_t narrow(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t narrow(float a, float b, __nv_bfloat16) { return pack_bf16x2(a, b); }
template <typename T, int E>
__device__ __forceinline__ void to_floats(const Raw<E * sizeof(T)>& r, float (&f)[E]) {
  if constexpr (sizeof(T) == 2 && E >= 2) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const float2 v = widen(w[i], T());
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  } else {
    const T* t = reinterpret_cast<const T*>(&r);
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = to_f(t[e]);
  }
}
template <typename T, int E>
__device__ __forceinline__ Raw<E * sizeof(T)> from_floats(const float (&f)[E]) {
  Raw<E * sizeof(T)> r;
  if constexpr (sizeof(T) == 2 && E >= 2) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) w[i] = narrow(f[2 * i], f[2 * i + 1], T());
  } else {
    T* t = reinterpret_cast<T*>(&r);
#pragma unroll
    for (int e = 0; e < E; ++e) t[e] = from_f<T>(f[e]);
  }
  return r;
}
// The arithmetic is on pairs with the packed fp32x2 operations (half the instructions; a single element is
// a pair with an idle half): E elements are (E + 1) / 2 pairs.
template <int E>
constexpr int kPairs = (E + 1) / 2;
template <typename T, int E>
__device__ __forceinline__ void to_pairs(const Raw<E * sizeof(T)>& r, float2 (&p)[kPairs<E>]) {
  float f[E];
  to_floats<T, E>(r, f);
#pragma unroll
  for (int i = 0; i < kPairs<E>; ++i) p[i] = make_float2(f[2 * i], E > 1 ? f[(2 * i + 1) % E] : 0.0f);
}
template <typename T, int E>
__device__ __forceinline__ Raw<E * sizeof(T)> from_pairs(const float2 (&p)[kPairs<E>]) {
  float f[E];
#pragma unroll
  for (int e = 0; e < E; ++e) f[e] = e % 2 == 0 ? p[e / 2].x : p[e / 2].y;
  return from_floats<T, E>(f);
}
__device__ __forceinline__ float2 pair(float v) { return make_float2(v, v); }

template <int kBytes>
__device__ __forceinline__ void st_stream(void* p, const Raw<kBytes>& r) {
  *static_cast<Raw<kBytes>*>(p) = r;
}
// E weights of either type (cached: every row uses them)
template <typename T, int E>
__device__ __forceinline__ void load_weights(const void* p, int64_t j, bool f32, float2 (&f)[kPairs<E>]) {
  if (sizeof(T) == 4 || f32) {
    const float* w = static_cast<const float*>(p) + j;
    if constexpr (E % 4 == 0) {
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(w + e));
        f[e / 2] = make_float2(v.x, v.y);
        f[e / 2 + 1] = make_float2(v.z, v.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPairs<E>; ++i) f[i] = make_float2(__ldg(w + 2 * i), E > 1 ? __ldg(w + 2 * i + 1) : 0.0f);
    }
  } else {
    const T* w = static_cast<const T*>(p) + j;
    if constexpr (E * sizeof(T) == 16) {
      const Raw<16> r{__ldg(reinterpret_cast<const uint4*>(w))};
      to_pairs<T, E>(r, f);
    } else {
#pragma unroll
      for (int i = 0; i < kPairs<E>; ++i) f[i] = make_float2(to_f(w[2 * i]), E > 1 ? to_f(w[2 * i + 1]) : 0.0f);
    }
  }
}

// Sums over a group of G threads (a power of two from 32 on) in a block; every thread gets them, added in a
// fixed order. Groups above a warp use two alternating buffers, so that one barrier a sum is enough.
template <int kSums>
struct GroupSum {
  float* buf;  // of the group: 2 x kSums x warps
  int warps, warp, id, turn = 0;
  __device__ __forceinline__ GroupSum(float* smem, int G) {
    warps = G >> 5;
    warp = (threadIdx.x >> 5) & (warps - 1);
    id = 1 + static_cast<int>(threadIdx.x) / G;  // barrier of the group; groups above a warp: at most 8
    buf = smem + (threadIdx.x / G) * (2 * kSums * warps);
  }
  __device__ __forceinline__ void operator()(float (&v)[kSums]) {
#pragma unroll
    for (int i = 0; i < kSums; ++i) v[i] = warp_sum(v[i]);
    if (warps == 1) return;
    float* b = buf + turn * kSums * warps;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < kSums; ++i) b[i * warps + warp] = v[i];
    }
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(warps * 32) : "memory");
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
      const int lane = threadIdx.x & 31;
      v[i] = warp_sum(lane < warps ? b[i * warps + lane] : 0.0f);
    }
  }
};
constexpr int kBlock = 256;       // threads of a block, unless a row takes more
constexpr int kMaxGroup = 1024;
constexpr int kMaxBwdGroup = 512;  // the column sums take registers

// ---- forward
template <typename T, int E, int R, int kMost>  // kMost: the block's threads, at most
__global__ void __launch_bounds__(kMost) ln_fwd_kernel(const LnFwdArgs a, int G) {
  __shared__ float smem[2 * 32];
  constexpr int kBytes = E * sizeof(T);
  // the next row is loaded under the work on this one where the registers have room for it
  constexpr bool kAhead = R * kRegs<kBytes> <= 8;
  const int groups = blockDim.x / G;
  const int t = threadIdx.x & (G - 1);
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const int n = static_cast<int>(a.N / E);
  const bool add = a.residual != nullptr, f32 = a.wdtype == 0;
  const float inv_n = 1.0f / static_cast<float>(a.N);
  struct Row {
    Raw<kBytes> x[R], res[R];
  };
  auto load = [&](Row& w, int64_t r) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (t + i * G >= n) continue;
      const int64_t j = static_cast<int64_t>(t + i * G) * E;
      w.x[i] = ld_stream<kBytes>(x + j);
      if (add) w.res[i] = ld_stream<kBytes>(static_cast<const T*>(a.residual) + r * a.ldr + j);
    }
  };
  GroupSum<1> sum(smem, G);
  Row next;
  int64_t r = static_cast<int64_t>(blockIdx.x) * groups + threadIdx.x / G;
  if (kAhead && r < a.M) load(next, r);
  for (; r < a.M; r += step) {
    if (!kAhead) load(next, r);
    Row w = next;
    if (kAhead && r + step < a.M) load(next, r + step);
    constexpr int P = kPairs<E>;
    float2 f[R][P], s2 = pair(0.f);
    float s[1];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (t + i * G >= n) continue;
      if (add) {
        float2 g[P];
        to_pairs<T, E>(w.x[i], f[i]);
        to_pairs<T, E>(w.res[i], g);
#pragma unroll
        for (int e = 0; e < P; ++e) f[i][e] = __fadd2_rn(f[i][e], g[e]);
        w.x[i] = from_pairs<T, E>(f[i]);  // h as it is stored
        st_stream(static_cast<T*>(a.h) + r * a.N + static_cast<int64_t>(t + i * G) * E, w.x[i]);
      }
      to_pairs<T, E>(w.x[i], f[i]);
#pragma unroll
      for (int e = 0; e < P; ++e) s2 = __fadd2_rn(s2, f[i][e]);
    }
    s[0] = s2.x + s2.y;
    sum(s);
    const float mu = s[0] * inv_n;
    s2 = pair(0.f);
    const float2 nmu = pair(-mu);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (t + i * G >= n) continue;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        f[i][e] = __fadd2_rn(f[i][e], nmu);
        s2 = __ffma2_rn(f[i][e], f[i][e], s2);
      }
    }
    s[0] = E > 1 ? s2.x + s2.y : s2.x;
    sum(s);
    const float rstd = rsqrtf(fmaf(s[0], inv_n, a.eps));
    const float2 scale = pair(rstd);
    T* y = static_cast<T*>(a.y) + r * a.N;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (t + i * G >= n) continue;
      const int64_t j = static_cast<int64_t>(t + i * G) * E;
      float2 g[P], b[P];
#pragma unroll
      for (int e = 0; e < P; ++e) g[e] = pair(1.0f), b[e] = pair(0.0f);
      if (a.gamma != nullptr) load_weights<T, E>(a.gamma, j, f32, g);
      if (a.beta != nullptr) load_weights<T, E>(a.beta, j, f32, b);
#pragma unroll
      for (int e = 0; e < P; ++e) f[i][e] = __ffma2_rn(__fmul2_rn(f[i][e], scale), g[e], b[e]);
      st_stream(y + j, from_pairs<T, E>(f[i]));
    }
    if (t == 0) {
      a.stats[2 * r] = mu;
      a.stats[2 * r + 1] = rstd;
    }
  }
}

// rows of any length, element by element, read three times (from L2 where a row fits)
template <typename T>
__global__ void __launch_bounds__(kMaxGroup) ln_fwd_long_kernel(const LnFwdArgs a) {
  __shared__ float buf[32];
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
    for (int64_t j = threadIdx.x; j < a.N; j += blockDim.x) s += value(j);
    const float mu = block_sum(s, buf) * inv_n;
    float q = 0.f;
    for (int64_t j = threadIdx.x; j < a.N; j += blockDim.x) {
      const float d = value(j) - mu;
      q = fmaf(d, d, q);
    }
    const float rstd = rsqrtf(fmaf(block_sum(q, buf), inv_n, a.eps));
    for (int64_t j = threadIdx.x; j < a.N; j += blockDim.x) {
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

// ---- backward
// dx, and with a.part the block's column sums: part[block][0][j] of dy x_hat, part[block][1][j] of dy
template <typename T, int E, int R>
__global__ void __launch_bounds__(kMaxBwdGroup) ln_bwd_kernel(const LnBwdArgs a, int G) {
  extern __shared__ float dyn[];  // with several groups a block: 2 N column sums
  __shared__ float smem[2 * 2 * 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kBytes = E * sizeof(T);
  const int groups = blockDim.x / G, group = threadIdx.x / G;
  const int t = threadIdx.x & (G - 1);
  const int n = static_cast<int>(a.N / E);
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const float inv_n = 1.0f / static_cast<float>(a.N);
  const bool add = a.dh != nullptr;
  constexpr int P = kPairs<E>;
  float2 gam[R][P], sg[R][P], sb[R][P];
#pragma unroll
  for (int i = 0; i < R; ++i) {
#pragma unroll
    for (int e = 0; e < P; ++e) {
      gam[i][e] = pair(1.0f);
      sg[i][e] = sb[i][e] = pair(0.0f);
    }
    if (a.gamma != nullptr && t + i * G < n)
      load_weights<T, E>(a.gamma, static_cast<int64_t>(t + i * G) * E, a.wdtype == 0, gam[i]);
  }
  struct Row {
    Raw<kBytes> x[R], dy[R], dh[R];
    float mu, rstd;
  };
  auto load = [&](Row& w, int64_t r) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + r * a.lddy;
    w.mu = a.stats[2 * r];
    w.rstd = a.stats[2 * r + 1];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (t + i * G >= n) continue;
      const int64_t j = static_cast<int64_t>(t + i * G) * E;
      w.x[i] = ld_stream<kBytes>(x + j);
      w.dy[i] = ld_stream<kBytes>(dy + j);
      if (add) w.dh[i] = ld_stream<kBytes>(static_cast<const T*>(a.dh) + r * a.lddh + j);
    }
  };
  GroupSum<2> sum(smem, G);
  // two rows of 16 registers a tensor would not fit
  constexpr bool kAhead = R * kRegs<kBytes> <= 8;
  Row next;
  int64_t r = static_cast<int64_t>(blockIdx.x) * groups + group;
  if (kAhead && r < a.M) load(next, r);
  for (; r < a.M; r += step) {
    if (!kAhead) load(next, r);
    const Row w = next;
    if (kAhead && r + step < a.M) load(next, r + step);
    const float2 nmu = pair(-w.mu), rstd = pair(w.rstd);
    float2 s0 = pair(0.f), s1 = s0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (t + i * G >= n) continue;
      float2 x[P], dy[P];
      to_pairs<T, E>(w.x[i], x);
      to_pairs<T, E>(w.dy[i], dy);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float2 xh = __fmul2_rn(__fadd2_rn(x[e], nmu), rstd), g = __fmul2_rn(dy[e], gam[i][e]);
        sg[i][e] = __ffma2_rn(dy[e], xh, sg[i][e]);
        sb[i][e] = __fadd2_rn(sb[i][e], dy[e]);
        s0 = __fadd2_rn(s0, g);
        s1 = __ffma2_rn(g, xh, s1);
      }
    }
    float s[2] = {s0.x + s0.y, s1.x + s1.y};  // the idle half of a single element has dy = 0
    sum(s);
    // dx = rstd (g - mean(g) - x_hat mean(g x_hat))
    const float2 c0 = pair(-s[0] * inv_n * w.rstd), c1 = pair(-s[1] * inv_n * w.rstd);
    T* dx = static_cast<T*>(a.dx) + r * a.N;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (t + i * G >= n) continue;
      float2 x[P], dy[P];
      to_pairs<T, E>(w.x[i], x);
      to_pairs<T, E>(w.dy[i], dy);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float2 xh = __fmul2_rn(__fadd2_rn(x[e], nmu), rstd);
        x[e] = __ffma2_rn(__fmul2_rn(dy[e], gam[i][e]), rstd, __ffma2_rn(xh, c1, c0));
      }
      if (add) {
        to_pairs<T, E>(w.dh[i], dy);
#pragma unroll
        for (int e = 0; e < P; ++e) x[e] = __fadd2_rn(x[e], dy[e]);
      }
      st_stream(dx + static_cast<int64_t>(t + i * G) * E, from_pairs<T, E>(x));
    }
  }
  if (a.part == nullptr) return;
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.N;
  float* to = groups > 1 ? dyn : part;
  for (int k = 0; k < groups; ++k) {  // one group after the other: a fixed order
    if (k == group) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (t + i * G >= n) continue;
        const int64_t j = static_cast<int64_t>(t + i * G) * E;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float vg = e % 2 == 0 ? sg[i][e / 2].x : sg[i][e / 2].y;
          const float vb = e % 2 == 0 ? sb[i][e / 2].x : sb[i][e / 2].y;
          to[j + e] = k == 0 ? vg : to[j + e] + vg;
          to[a.N + j + e] = k == 0 ? vb : to[a.N + j + e] + vb;
        }
      }
    }
    if (groups > 1) __syncthreads();
  }
  if (groups > 1)
    for (int64_t j = threadIdx.x; j < 2 * a.N; j += blockDim.x) part[j] = dyn[j];
}

// rows of any length, element by element
template <typename T>
__global__ void __launch_bounds__(kMaxGroup) ln_dx_long_kernel(const LnBwdArgs a) {
  __shared__ float buf[32];
  const float inv_n = 1.0f / static_cast<float>(a.N);
  for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + r * a.lddy;
    const T* dh = a.dh != nullptr ? static_cast<const T*>(a.dh) + r * a.lddh : nullptr;
    T* dx = static_cast<T*>(a.dx) + r * a.N;
    const float mu = a.stats[2 * r], rstd = a.stats[2 * r + 1];
    float sa = 0.f, sb = 0.f;
    for (int64_t j = threadIdx.x; j < a.N; j += blockDim.x) {
      const float g = to_f(dy[j]) * (a.gamma != nullptr ? load_any(a.gamma, j, a.wdtype) : 1.0f);
      sa += g;
      sb = fmaf(g, (to_f(x[j]) - mu) * rstd, sb);
    }
    const float c0 = -block_sum(sa, buf) * inv_n * rstd, c1 = -block_sum(sb, buf) * inv_n * rstd;
    for (int64_t j = threadIdx.x; j < a.N; j += blockDim.x) {
      const float g = to_f(dy[j]) * (a.gamma != nullptr ? load_any(a.gamma, j, a.wdtype) : 1.0f);
      const float v = fmaf(g, rstd, fmaf((to_f(x[j]) - mu) * rstd, c1, c0));
      dx[j] = from_f<T>(dh != nullptr ? v + to_f(dh[j]) : v);
    }
  }
}
// one row chunk's column sums, for rows of any length
constexpr int kColThreads = 128;
template <typename T>
__global__ void __launch_bounds__(kColThreads) ln_param_long_kernel(const LnBwdArgs a, int64_t rows_per_chunk) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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

// dgamma, dbeta from part [rows][2 N]: 32 columns a block, eight threads a column take the rows in turn and
// are added in order. A programmatic dependent of the kernel before it: its writes are visible after
// griddepcontrol.wait.
constexpr int kReduceCols = 32, kReduceSlices = 16;
__global__ void __launch_bounds__(kReduceCols* kReduceSlices) ln_reduce_kernel(const float* part, int rows, int64_t N,
                                                                               void* dgamma, void* dbeta, int wdtype) {
  __shared__ float sums[kReduceSlices][kReduceCols];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = threadIdx.x % kReduceCols, k = threadIdx.x / kReduceCols;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kReduceCols + c;
  float s = 0.f;
  if (j < 2 * N) {
    const float* p = part + j;
    int i = k;
    for (; i + 3 * kReduceSlices < rows; i += 4 * kReduceSlices) {
      const float v0 = p[static_cast<int64_t>(i) * 2 * N], v1 = p[static_cast<int64_t>(i + kReduceSlices) * 2 * N];
      const float v2 = p[static_cast<int64_t>(i + 2 * kReduceSlices) * 2 * N];
      const float v3 = p[static_cast<int64_t>(i + 3 * kReduceSlices) * 2 * N];
      s += (v0 + v1) + (v2 + v3);
    }
    for (; i < rows; i += kReduceSlices) s += p[static_cast<int64_t>(i) * 2 * N];
  }
  sums[k][c] = s;
  __syncthreads();
  if (k != 0 || j >= 2 * N) return;
#pragma unroll
  for (int i = 1; i < kReduceSlices; ++i) s += sums[i][c];
  if (j < N) {
    if (dgamma != nullptr) store_any(dgamma, j, wdtype, s);
  } else if (dbeta != nullptr) {
    store_any(dbeta, j - N, wdtype, s);
  }
}

// ---- host
// elements of a load: the widest of 16 bytes, 4 bytes and one element that divides the row and that all
// addresses and row strides are multiples of
int vector_elems(int64_t N, int es, std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> lds,
                 std::initializer_list<const void*> weights) {
  for (int bytes : {16, 4}) {
    const int e = bytes / es;
    if (e < 1 || N % e != 0) continue;
    bool ok = true;
    for (const void* p : ptrs) ok = ok && reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0;
    for (int64_t ld : lds) ok = ok && ld % e == 0;
    // weights are loaded 16 bytes at a time with full vectors, else one by one
    if (bytes == 16)
      for (const void* p : weights) ok = ok && reinterpret_cast<uintptr_t>(p) % 16 == 0;
    if (ok) return e;
  }
  return 1;
}
// threads a row for R vectors each
int group_threads(int64_t n, int R) {
  int g = 32;
  while (static_cast<int64_t>(g) * R < n && g < kMaxGroup) g *= 2;
  return g;
}

// blocks of a persistent kernel that fit on the device at once (asked once for each device and block size)
struct FitCache {
  int device = -1, threads = 0, fit = 0;
  size_t bytes = 0;
};
template <typename Kernel>
cudaError_t blocks_that_fit(Kernel kernel, FitCache& cache, int block, size_t smem, int64_t& blocks) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (cache.device != dev || cache.threads != block || cache.bytes != smem) {
    int per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, block, smem);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorLaunchOutOfResources;
    cache = FitCache{dev, block, per_sm * device_sm_count(), smem};
  }
  blocks = cache.fit;
  return cudaSuccess;
}
template <typename T, int E, int R, int kMost>
cudaError_t fwd_one(const LnFwdArgs& a, int G, cudaStream_t stream) {
  const int block = G > kBlock ? G : kBlock, groups = block / G;
  int64_t blocks;
  {
    static std::mutex mu;
    static FitCache cache;
    std::lock_guard<std::mutex> lk(mu);
    const cudaError_t e = blocks_that_fit(ln_fwd_kernel<T, E, R, kMost>, cache, block, 0, blocks);
    if (e != cudaSuccess) return e;
  }
  const int64_t most = (a.M + groups - 1) / groups;
  if (blocks > most) blocks = most;
  ln_fwd_kernel<T, E, R, kMost><<<static_cast<unsigned>(blocks), block, 0, stream>>>(a, G);
  return cudaGetLastError();
}
// vectors a thread: as few as let a block of 512 hold the row, two for wide vectors from a warp on
template <typename T, int E, int R0>
cudaError_t fwd_any(const LnFwdArgs& a, cudaStream_t stream) {
  const int64_t n = a.N / E;
  if (n <= 32 * R0) return fwd_one<T, E, R0, 512>(a, 32, stream);
  if (n <= 512 * 2 * R0) return fwd_one<T, E, 2 * R0, 512>(a, group_threads(n, 2 * R0), stream);
  if (n <= kMaxGroup * 4 * R0) return fwd_one<T, E, 4 * R0, kMaxGroup>(a, group_threads(n, 4 * R0), stream);
  const unsigned grid = static_cast<unsigned>(a.M < 65536 ? a.M : 65536);
  ln_fwd_long_kernel<T><<<grid, kMaxGroup, 0, stream>>>(a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t fwd_type(const LnFwdArgs& a, cudaStream_t stream) {
  constexpr int es = sizeof(T);
  const int e = vector_elems(a.N, es, {a.x, a.residual, a.h, a.y}, {a.ldx, a.ldr}, {a.gamma, a.beta});
  if (e == 16 / es) return fwd_any<T, 16 / es, 1>(a, stream);
  if constexpr (es == 2)
    if (e == 2) return fwd_any<T, 2, 2>(a, stream);
  return fwd_any<T, 1, 4>(a, stream);
}

int reduce_grid(int64_t N) { return static_cast<int>((2 * N + kReduceCols - 1) / kReduceCols); }
cudaError_t launch_reduce(const LnBwdArgs& a, int64_t rows, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(reduce_grid(a.N)));
  cfg.blockDim = dim3(kReduceCols * kReduceSlices);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ln_reduce_kernel, static_cast<const float*>(a.part), static_cast<int>(rows), a.N,
                            a.dgamma, a.dbeta, a.wdtype);
}

constexpr int64_t kMaxBlocks = 4 * 256;  // rows of column sums in the workspace, at most
constexpr int64_t kLongChunks = 64;      // of them for rows too long for registers

template <typename T, int E, int R>
cudaError_t bwd_one(const LnBwdArgs& a, int G, cudaStream_t stream) {
  const int block = G > kBlock ? G : kBlock, groups = block / G;
  const size_t smem = groups > 1 && a.part != nullptr ? static_cast<size_t>(2 * a.N) * sizeof(float) : 0;
  int64_t blocks;
  {
    static std::mutex mu;
    static FitCache cache;
    std::lock_guard<std::mutex> lk(mu);
    const cudaError_t e = blocks_that_fit(ln_bwd_kernel<T, E, R>, cache, block, smem, blocks);
    if (e != cudaSuccess) return e;
  }
  const int64_t most = (a.M + groups - 1) / groups;
  if (blocks > most) blocks = most;
  if (blocks > kMaxBlocks) blocks = kMaxBlocks;
  ln_bwd_kernel<T, E, R><<<static_cast<unsigned>(blocks), block, smem, stream>>>(a, G);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.part == nullptr) return e;
  return launch_reduce(a, blocks, stream);
}
template <typename T>
cudaError_t bwd_long(const LnBwdArgs& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(a.M < 65536 ? a.M : 65536);
  ln_dx_long_kernel<T><<<grid, kMaxGroup, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.part == nullptr) return e;
  const int64_t chunks = a.M < kLongChunks ? a.M : kLongChunks, per = (a.M + chunks - 1) / chunks;
  const dim3 g(static_cast<unsigned>((a.N + kColThreads - 1) / kColThreads), static_cast<unsigned>(chunks));
  ln_param_long_kernel<T><<<g, kColThreads, 0, stream>>>(a, per);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_reduce(a, chunks, stream);
}
template <typename T, int E, int R0>
cudaError_t bwd_any(const LnBwdArgs& a, cudaStream_t stream) {
  const int64_t n = a.N / E;
  if (n <= 32 * R0) return bwd_one<T, E, R0>(a, 32, stream);
  if (n <= kMaxBwdGroup * 2 * R0) return bwd_one<T, E, 2 * R0>(a, group_threads(n, 2 * R0), stream);
  return bwd_long<T>(a, stream);
}
template <typename T>
cudaError_t bwd_type(const LnBwdArgs& a, cudaStream_t stream) {
  constexpr int es = sizeof(T);
  const int e = vector_elems(a.N, es, {a.dy, a.x, a.dh, a.dx}, {a.lddy, a.ldx, a.lddh}, {a.gamma});
  if (e == 16 / es) return bwd_any<T, 16 / es, es == 2 ? 1 : 2>(a, stream);
  if constexpr (es == 2)
    if (e == 2) return bwd_any<T, 2, 4>(a, stream);
  return bwd_any<T, 1, 4>(a, stream);
}

}  // namespace

size_t ln_workspace_bytes(int64_t M, int64_t N) {
  const int64_t rows = M < kMaxBlocks ? M : kMaxBlocks;
  return static_cast<size_t>(rows) * 2 * static_cast<size_t>(N) * sizeof(float);
}

cudaError_t launch_layer_norm_fwd(const LnFwdArgs& a, int dtype, cudaStream_t stream) {
  return dtype == 0   ? fwd_type<float>(a, stream)
         : dtype == 1 ? fwd_type<__half>(a, stream)
                      : fwd_type<__nv_bfloat16>(a, stream);
}

cudaError_t launch_layer_norm_bwd(const LnBwdArgs& a, int dtype, cudaStream_t stream) {
  return dtype == 0   ? bwd_type<float>(a, stream)
         : dtype == 1 ? bwd_type<__half>(a, stream)
                      : bwd_type<__nv_bfloat16>(a, stream);
}

}  // namespace swg
