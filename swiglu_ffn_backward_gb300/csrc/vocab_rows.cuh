// Rows of logits as the kernels of token_logprobs.cu and distill.cu take them.
//
// A row is cut into 16-byte vectors at 16-byte aligned addresses, whatever the address of its first
// element: vector g holds the elements [g E - shift, g E - shift + E), shift being the number of
// elements between the aligned address at or below the row's start and that start. Only a row's first
// and last vector can be partial; they are read and written element by element, inside the row. S blocks
// (or groups of threads) take a run of a row's vectors each, their share.
#pragma once

#include "row_ops.cuh"

namespace swg {
namespace row {

constexpr int kRowThreads = 256;
constexpr int kVecs = 8;                          // 16-byte vectors a thread holds: 32 registers
constexpr int kMaxCluster = 8;                    // portable cluster size

template <typename T>
struct Traits;
template <>
struct Traits<float> {
  static constexpr int E = 4;
  static constexpr uint32_t kNegInf = 0xff800000u;
};
template <>
struct Traits<__half> {
  static constexpr int E = 8;
  static constexpr uint32_t kNegInf = 0xfc00fc00u;
};
template <>
struct Traits<__nv_bfloat16> {
  static constexpr int E = 8;
  static constexpr uint32_t kNegInf = 0xff80ff80u;
};

struct Vec {
  uint32_t w[4];
};

template <bool kReadOnly>
__device__ __forceinline__ Vec ld_vec(const void* p) {
  Vec v;
  if (kReadOnly)
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
        : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3])
        : "l"(p));
  else
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3])
                 : "l"(p)
                 : "memory");
  return v;
}
__device__ __forceinline__ void st_vec(void* p, const Vec& v) {
  asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.w[0]), "r"(v.w[1]),
               "r"(v.w[2]), "r"(v.w[3])
               : "memory");
}

// elements 2 i and 2 i + 1 of a vector
template <typename T>
__device__ __forceinline__ float2 vec_pair(const Vec& v, int i);
template <>
__device__ __forceinline__ float2 vec_pair<float>(const Vec& v, int i) {
  return make_float2(__uint_as_float(v.w[2 * i]), __uint_as_float(v.w[2 * i + 1]));
}
template <>
__device__ __forceinline__ float2 vec_pair<__half>(const Vec& v, int i) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v.w[i]));
}
template <>
__device__ __forceinline__ float2 vec_pair<__nv_bfloat16>(const Vec& v, int i) {
  return bf16x2_to_f2(v.w[i]);
}
template <typename T>
__device__ __forceinline__ void set_pair(Vec& v, int i, float2 x);
template <>
__device__ __forceinline__ void set_pair<float>(Vec& v, int i, float2 x) {
  v.w[2 * i] = __float_as_uint(x.x);
  v.w[2 * i + 1] = __float_as_uint(x.y);
}
template <>
__device__ __forceinline__ void set_pair<__half>(Vec& v, int i, float2 x) {
  const __half2 h = __floats2half2_rn(x.x, x.y);
  v.w[i] = *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ void set_pair<__nv_bfloat16>(Vec& v, int i, float2 x) {
  v.w[i] = pack_bf16x2(x.x, x.y);
}
// the largest element, NaNs passed over
template <typename T>
__device__ __forceinline__ float vec_max(const Vec& v);
template <>
__device__ __forceinline__ float vec_max<float>(const Vec& v) {
  return fmaxf(fmaxf(__uint_as_float(v.w[0]), __uint_as_float(v.w[1])),
               fmaxf(__uint_as_float(v.w[2]), __uint_as_float(v.w[3])));
}
template <>
__device__ __forceinline__ float vec_max<__half>(const Vec& v) {
  const __half2* h = reinterpret_cast<const __half2*>(v.w);
  const float2 m = __half22float2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
  return fmaxf(m.x, m.y);
}
template <>
__device__ __forceinline__ float vec_max<__nv_bfloat16>(const Vec& v) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(v.w);
  const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
  return fmaxf(__low2float(m), __high2float(m));
}

// the largest element of four vectors
template <typename T>
__device__ __forceinline__ float vec_max4(const Vec (&v)[4]);
template <>
__device__ __forceinline__ float vec_max4<float>(const Vec (&v)[4]) {
  return fmaxf(fmaxf(vec_max<float>(v[0]), vec_max<float>(v[1])), fmaxf(vec_max<float>(v[2]), vec_max<float>(v[3])));
}
template <typename T, typename T2>
__device__ __forceinline__ Vec larger_halves(const Vec& a, const Vec& b) {
  Vec r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const T2 m = __hmax2(*reinterpret_cast<const T2*>(&a.w[i]), *reinterpret_cast<const T2*>(&b.w[i]));
    r.w[i] = *reinterpret_cast<const uint32_t*>(&m);
  }
  return r;
}
template <>
__device__ __forceinline__ float vec_max4<__half>(const Vec (&v)[4]) {
  return vec_max<__half>(larger_halves<__half, __half2>(larger_halves<__half, __half2>(v[0], v[1]),
                                                        larger_halves<__half, __half2>(v[2], v[3])));
}
template <>
__device__ __forceinline__ float vec_max4<__nv_bfloat16>(const Vec (&v)[4]) {
  const Vec lo = larger_halves<__nv_bfloat16, __nv_bfloat162>(v[0], v[1]);
  const Vec hi = larger_halves<__nv_bfloat16, __nv_bfloat162>(v[2], v[3]);
  return vec_max<__nv_bfloat16>(larger_halves<__nv_bfloat16, __nv_bfloat162>(lo, hi));
}

// bit i: element i is at or above `least` (which is not NaN; a NaN element is not)
template <typename T>
__device__ __forceinline__ uint32_t at_or_above(const Vec& v, T least);
template <>
__device__ __forceinline__ uint32_t at_or_above<float>(const Vec& v, float least) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m |= (__uint_as_float(v.w[i]) >= least ? 1u : 0u) << i;
  return m;
}
__device__ __forceinline__ uint32_t half_bits(uint32_t mask, int i) {  // of elements 2 i and 2 i + 1
  return (mask & (1u << (2 * i))) | ((mask >> 16) & (2u << (2 * i)));
}
template <>
__device__ __forceinline__ uint32_t at_or_above<__half>(const Vec& v, __half least) {
  const __half2 l = __half2half2(least);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m |= half_bits(__hge2_mask(*reinterpret_cast<const __half2*>(&v.w[i]), l), i);
  return m;
}
template <>
__device__ __forceinline__ uint32_t at_or_above<__nv_bfloat16>(const Vec& v, __nv_bfloat16 least) {
  const __nv_bfloat162 l = __bfloat162bfloat162(least);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m |= half_bits(__hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(&v.w[i]), l), i);
  return m;
}
// the type's lowest finite value
template <typename T>
__device__ __forceinline__ T lowest();
template <>
__device__ __forceinline__ float lowest<float>() { return -3.4028234663852886e38f; }
template <>
__device__ __forceinline__ __half lowest<__half>() { return __ushort_as_half(0xfbff); }
template <>
__device__ __forceinline__ __nv_bfloat16 lowest<__nv_bfloat16>() { return __ushort_as_bfloat16(0xff7f); }

template <typename T>
__device__ __forceinline__ int row_shift(const T* row) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
}

// the vector whose first element is element e0 of the row; -inf outside the row
template <typename T, bool kReadOnly>
__device__ __forceinline__ Vec load_row_vec(const T* row, int64_t e0, int64_t V) {
  constexpr int E = Traits<T>::E;
  if (e0 >= 0 && e0 + E <= V) return ld_vec<kReadOnly>(row + e0);
  Vec v;
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const int64_t e = e0 + 2 * i;
    set_pair<T>(v, i, make_float2(e >= 0 && e < V ? to_f(row[e]) : neg_inf(),
                                  e + 1 >= 0 && e + 1 < V ? to_f(row[e + 1]) : neg_inf()));
  }
  return v;
}
// the same vector of a row of outputs; `aligned`: out + e0 is 16-byte aligned
template <typename T>
__device__ __forceinline__ void store_row_vec(T* out, int64_t e0, int64_t V, bool aligned, const Vec& v) {
  constexpr int E = Traits<T>::E;
  if (aligned && e0 >= 0 && e0 + E <= V) {
    st_vec(out + e0, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const int64_t e = e0 + 2 * i;
    const float2 x = vec_pair<T>(v, i);
    if (e >= 0 && e < V) out[e] = from_f<T>(x.x);
    if (e + 1 >= 0 && e + 1 < V) out[e + 1] = from_f<T>(x.y);
  }
}

// A block's share of a row: `per` of its vectors (fewer than 2^30: a row has fewer than 2^31 elements).
struct Share {
  int begin, end;
  int shift;
};
template <typename T>
__device__ __forceinline__ Share share_of(const T* row, int64_t V, int per, int rank) {
  Share s;
  s.shift = row_shift(row);
  const int64_t n = (s.shift + V + Traits<T>::E - 1) / Traits<T>::E;
  s.begin = static_cast<int>(min(n, static_cast<int64_t>(rank) * per));
  s.end = static_cast<int>(min(n, static_cast<int64_t>(s.begin) + per));
  return s;
}
// the row's element at the start of vector g
template <typename T>
__device__ __forceinline__ int64_t first_element(const Share& s, int g) {
  return static_cast<int64_t>(g) * Traits<T>::E - s.shift;
}
// vectors c + i G + t of the share, t the thread's number in its group of G -> v[i]; -inf past its end
template <typename T, bool kReadOnly>
__device__ __forceinline__ void load_chunk(Vec (&v)[kVecs], const T* row, int64_t V, const Share& s, int c, int t,
                                           int G) {
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int g = c + i * G + t;
    if (g < s.end) {
      v[i] = load_row_vec<T, kReadOnly>(row, first_element<T>(s, g), V);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i].w[j] = Traits<T>::kNegInf;
    }
  }
}

__device__ __forceinline__ float finite_or_0(float m) { return m == neg_inf() ? 0.0f : m; }
// x = (z - max) log2(e) / tau, not below kLeast, where 2^x is 0 already: a -inf would give 0 * inf in
// sums of 2^x x. A NaN stays one.
constexpr float kLeast = -200.0f;
__device__ __forceinline__ float at_least(float x) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(kLeast));
  return r;
}

// Exponents under a reference logit m (a maximum, or one not far below it): x = fma(z, c, -ref) with
// c = log2(e) / tau and ref = m c rounded once, one rounding for an element. Sums of 2^x belong to ref, not
// to m c: parts are joined by the difference of their refs, and only the reported sum is moved to the
// maximum itself. From |m c| = 2^30 on (a row of the type's
// lowest value, for one) that rounding would be too large; there the next smaller logit's x is
// below -32, so 2^x is 1 at the maximum and 0 elsewhere to all digits kept: c is then a power of two that
// puts |m c| in [2^40, 2^41), exactly.
constexpr float kLargeRef = 1073741824.0f;
// c of an inverse temperature, finite: a difference of 0 stays one at the smallest temperatures (below 4.3e-39)
__device__ __forceinline__ float exponent_scale(float inv_temp) {
  return fminf(inv_temp * kLog2e, 3.4028234663852886e38f);
}
struct Scale {
  float c, ref;
};
__device__ __forceinline__ Scale scale_of(float m, float c) {
  const float me = m == neg_inf() ? 0.0f : m;
  Scale s{c, me * c};
  if (!(fabsf(s.ref) < kLargeRef)) {
    const int e = 294 - static_cast<int>((__float_as_uint(me) >> 23) & 0xffu);
    s.c = __uint_as_float(static_cast<uint32_t>(min(max(e, 1), 254)) << 23);
    s.ref = me * s.c;
  }
  return s;
}
// the exponent by which a sum under the reference logit `part` is moved to `joint` (s, k: their scales); a
// part with no logit above -inf has a sum of 0 (or NaN)
__device__ __forceinline__ float ref_shift(float part, const Scale& s, float joint, const Scale& k, float c) {
  if (part == neg_inf()) return 0.0f;
  const bool plain = fabsf(s.ref) < kLargeRef && fabsf(k.ref) < kLargeRef;
  return at_least(plain ? s.ref - k.ref : part == joint ? 0.0f : (part - joint) * c);
}
// the sum of exp((z - m) / tau) from the sum of 2^x, and back
__device__ __forceinline__ float sum_at_max(float s, float m, const Scale& k) {
  return m == neg_inf() ? s : s * ex2_approx(-fmaf(m, k.c, -k.ref));
}
__device__ __forceinline__ float sum_at_ref(float s, float m, const Scale& k) {
  return m == neg_inf() ? s : s * ex2_approx(fmaf(m, k.c, -k.ref));
}

// ---- clusters: a block of the cluster writes to, and only to, blocks that have started (the barrier's
// first phase) and that wait for the second one before they read
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}

}  // namespace row

// 16-byte vectors of a row of V elements: one more where rows may start inside a vector
inline int64_t row_vectors(const void* rows, int64_t V, int64_t ld, int elem_bytes) {
  const bool whole = reinterpret_cast<uintptr_t>(rows) % 16 == 0 && (ld * elem_bytes) % 16 == 0;
  return (V * elem_bytes + 15) / 16 + (whole ? 0 : 1);
}
// Blocks a row is given: shares of at most `share` vectors where the portable cluster size allows it,
// and more blocks when there are so few rows that SMs would stay idle (but no shares below kMinShare).
constexpr int64_t kMinShare = 256;
struct Split {
  int S;    // blocks a row
  int per;  // vectors a block takes
};
inline Split split_row(int64_t T, int64_t vectors, int64_t share, int num_sms) {
  const int64_t useful = (vectors + kMinShare - 1) / kMinShare, spread = num_sms / T;
  int64_t s = (vectors + share - 1) / share;
  if (s < spread && s < useful) s = spread < useful ? spread : useful;
  if (s > row::kMaxCluster) s = row::kMaxCluster;
  return Split{static_cast<int>(s), static_cast<int>((vectors + s - 1) / s)};
}

// The kernels that need no exchange (gradients from saved statistics): a group of G threads, 32 to 256,
// takes a share of up to kVecs vectors a thread of one row; a block of 256 threads has 256 / G such groups.
struct Groups {
  int S;    // groups a row
  int per;  // vectors a group takes
  int G;
};
inline Groups row_groups(int64_t T, int64_t vectors, int num_sms) {
  int G = 32;
  while (G < row::kRowThreads && G * row::kVecs < vectors) G *= 2;
  const int64_t chunk = static_cast<int64_t>(G) * row::kVecs;
  const int64_t useful = (vectors + G - 1) / G, spread = 4 * num_sms / T;  // at least a vector a thread
  int64_t s = (vectors + chunk - 1) / chunk;
  if (s < spread && s < useful) s = spread < useful ? spread : useful;
  return Groups{static_cast<int>(s), static_cast<int>((vectors + s - 1) / s), G};
}
// Launches of at most 2^22 blocks or so at a time, whatever the number of rows.
template <typename Args, typename K32, typename K16, typename KB>
cudaError_t launch_groups(const Args& a, int dtype, const Groups& p, cudaStream_t stream, K32 k32, K16 k16, KB kb) {
  const int per_block = row::kRowThreads / p.G;
  const int64_t most = (int64_t(1) << 22) * per_block;  // groups a launch
  const int64_t total = a.T * p.S;
  for (int64_t g0 = 0; g0 < total; g0 += most) {
    const int64_t n = total - g0 < most ? total - g0 : most;
    const unsigned blocks = static_cast<unsigned>((n + per_block - 1) / per_block);
    if (dtype == 0) k32<<<blocks, row::kRowThreads, 0, stream>>>(a, g0, p);
    else if (dtype == 1) k16<<<blocks, row::kRowThreads, 0, stream>>>(a, g0, p);
    else kb<<<blocks, row::kRowThreads, 0, stream>>>(a, g0, p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace swg
