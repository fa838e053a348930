// Rows of a matrix as 16-byte vectors in the registers of a group of threads: loads and stores of whole and
// ragged vectors, sums over a group and over the groups of a cluster. Shared by layer norm and by the norms
// between blocks.
#pragma once

#include <algorithm>
#include <initializer_list>
#include <mutex>
#include <numeric>
#include <type_traits>

#include "swg_launch.h"
#include "vocab_stream.cuh"

namespace swg {
namespace row {

struct Raw {  // 16 bytes
  uint32_t w[4];
};
template <typename T>
constexpr int kElems = 16 / static_cast<int>(sizeof(T));

__device__ __forceinline__ Raw ld_stream(const void* p) {
  Raw r;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
      : "l"(p));
  return r;
}
__device__ __forceinline__ Raw ld_cached(const void* p) {
  const uint4 u = __ldg(static_cast<const uint4*>(p));
  return Raw{{u.x, u.y, u.z, u.w}};
}
__device__ __forceinline__ void st_raw(void* p, const Raw& r) {
  *static_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
}

// 16-bit elements are widened and narrowed two at a time, and the arithmetic is on pairs with the packed
// fp32x2 operations (half the instructions)
__device__ __forceinline__ float2 widen(uint32_t u, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
__device__ __forceinline__ float2 widen(uint32_t u, __nv_bfloat16) { return bf16x2_to_f2(u); }
__device__ __forceinline__ uint32_t narrow(float2 v, __half) {
  const __half2 h = __floats2half2_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t narrow(float2 v, __nv_bfloat16) { return pack_bf16x2(v.x, v.y); }
template <typename T>
constexpr int kPairs = kElems<T> / 2;
template <typename T>
__device__ __forceinline__ float2 get_pair(const Raw& r, int i) {
  if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
  else return widen(r.w[i], T());
}
template <typename T>
__device__ __forceinline__ void set_pair(Raw& r, int i, float2 v) {
  if constexpr (sizeof(T) == 4) {
    r.w[2 * i] = __float_as_uint(v.x);
    r.w[2 * i + 1] = __float_as_uint(v.y);
  } else {
    r.w[i] = narrow(v, T());
  }
}
__device__ __forceinline__ float2 pair(float v) { return make_float2(v, v); }

// The 16 bytes that begin `shift` elements into the 32 bytes a, b.
template <typename T>
__device__ __forceinline__ Raw join(const Raw& a, const Raw& b, int shift) {
  const int words = shift * static_cast<int>(sizeof(T)) / 4;
  uint32_t w[7] = {a.w[0], a.w[1], a.w[2], a.w[3], b.w[0], b.w[1], b.w[2]};
  const uint32_t last = b.w[3];
  uint32_t v[6];
#pragma unroll
  for (int i = 0; i < 5; ++i) v[i] = words & 2 ? w[i + 2] : w[i];
  v[5] = words & 2 ? last : w[5];
  uint32_t u[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) u[i] = words & 1 ? v[i + 1] : v[i];
  Raw r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r.w[i] = sizeof(T) == 2 && (shift & 1) ? __funnelshift_r(u[i], u[i + 1], 16) : u[i];
  return r;
}
template <typename T>
__device__ __forceinline__ int shift_of(const T* p) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}
// The rows of a tensor.
template <typename T>
struct Rows {
  const T *first, *end;
  int64_t ld;
  __device__ __forceinline__ Rows(const void* p, int64_t ld_, int64_t M, int64_t N)
      : first(static_cast<const T*>(p)), end(first + (M - 1) * ld_ + N), ld(ld_) {}
};
// The columns from j on of row r of N, of which the row may have some only (kRagged: j below 0 or j + E above
// N); anything for the others. Nothing here waits for a load that is one aligned vector.
template <typename T, bool kRagged>
__device__ __forceinline__ Raw load_columns(const Rows<T>& rows, int64_t r, int j, int N) {
  const T *row = rows.first + r * rows.ld, *p = row + j;
  if constexpr (!kRagged) return ld_stream(p);
  constexpr int E = kElems<T>;
  const int shift = shift_of(p);
  if (shift == 0) {
    if (j >= 0 && j + E <= N) return ld_stream(p);
    if (p >= rows.first && p + E <= rows.end) return ld_stream(p);
  } else if (j >= shift && j - shift + 2 * E <= N) {
    return join<T>(ld_cached(p - shift), ld_cached(p - shift + E), shift);
  }
  Raw v;
#pragma unroll
  for (int i = 0; i < kPairs<T>; ++i) {
    const int k = j + 2 * i;
    const float lo = k >= 0 && k < N ? to_f(row[k]) : 0.0f, hi = k >= -1 && k + 1 < N ? to_f(row[k + 1]) : 0.0f;
    set_pair<T>(v, i, make_float2(lo, hi));
  }
  return v;
}
// zeros for the columns that the row does not have
template <typename T>
__device__ __forceinline__ void clear_others(Raw& v, int j, int N) {
  if (j >= 0 && j + kElems<T> <= N) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      if (j + i < 0 || j + i >= N) v.w[i] = 0;
    } else {
      const int k = j + 2 * i;
      v.w[i] &= (k >= 0 && k < N ? 0xffffu : 0u) | (k >= -1 && k + 1 < N ? 0xffff0000u : 0u);
    }
  }
}
template <typename T, bool kRagged>
__device__ __forceinline__ void store_columns(T* row, int j, int N, const Raw& r) {
  T* p = row + j;
  constexpr int E = kElems<T>;
  if (!kRagged || (shift_of(p) == 0 && j >= 0 && j + E <= N)) {
    st_raw(p, r);
    return;
  }
#pragma unroll
  for (int i = 0; i < kPairs<T>; ++i) {
    const float2 v = get_pair<T>(r, i);
    const int k = j + 2 * i;
    if (k >= 0 && k < N) row[k] = from_f<T>(v.x);
    if (k >= -1 && k + 1 < N) row[k + 1] = from_f<T>(v.y);
  }
}
// weights of either type (cached: every row uses them), 1 or 0 where there are none
template <typename T, typename W, bool kRagged>
__device__ __forceinline__ void weights_of(const W* w, int j, int N, float2 (&f)[kPairs<T>]) {
  constexpr int E = kElems<T>, V = 16 / static_cast<int>(sizeof(W)), L = E / V;
  const W* p = w + j;
  const int shift = kRagged ? shift_of(p) : 0;
  if (kRagged && (j < shift || j - shift + E + (shift > 0 ? V : 0) > N)) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float v = j + e >= 0 && j + e < N ? to_f(p[e]) : 0.0f;
      if (e % 2 == 0) f[e / 2].x = v;
      else f[e / 2].y = v;
    }
    return;
  }
  Raw r[L + 1];
#pragma unroll
  for (int i = 0; i < L; ++i) r[i] = ld_cached(p - shift + i * V);
  if (kRagged && shift > 0) {
    r[L] = ld_cached(p - shift + E);
#pragma unroll
    for (int i = 0; i < L; ++i) r[i] = join<W>(r[i], r[i + 1], shift);
  }
#pragma unroll
  for (int i = 0; i < kPairs<T>; ++i) f[i] = get_pair<W>(r[2 * i / V], i % (V / 2));
}
template <typename T, bool kRagged>
__device__ __forceinline__ void load_weights(const void* w, int j, int N, bool f32, float none,
                                             float2 (&f)[kPairs<T>]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < kPairs<T>; ++i) f[i] = pair(none);
  } else if (sizeof(T) == 4 || f32) {
    weights_of<T, float, kRagged>(static_cast<const float*>(w), j, N, f);
  } else {
    weights_of<T, T, kRagged>(static_cast<const T*>(w), j, N, f);
  }
}

// Sums over a group of G threads of a block (a power of two up to 32, or whole warps); every thread gets them,
// added in a fixed order. Groups above a warp use two alternating buffers, so that one barrier a sum is enough.
template <int kSums, bool kNarrow>  // kNarrow: G below 32 as well
struct GroupSum {
  float* buf;  // of the group: 2 x kSums x warps
  int warps, warp, id, width, turn = 0;
  __device__ __forceinline__ GroupSum(float* smem, int G) {
    warps = G > 32 ? G >> 5 : 1;
    width = G < 32 ? G : 32;
    warp = (threadIdx.x >> 5) % warps;
    id = 1 + static_cast<int>(threadIdx.x) / G;  // barrier of the group; groups above a warp: at most 8
    buf = smem + (threadIdx.x / G) * (2 * kSums * warps);
  }
  __device__ __forceinline__ void operator()(float (&v)[kSums]) {
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
      if (!kNarrow || width == 32) v[i] = warp_sum(v[i]);
      else
        for (int o = width >> 1; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
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
// Sums over the S blocks of a cluster, each of which comes with its own; every thread gets them, added in
// the blocks' order. Two slots alternate: a block sends into one again only after all have sent into the
// other, and so have read this one.
struct ClusterSlots {
  uint64_t come[2];
  float2 sums[2][kMaxCluster];
};
template <int kSums>
struct ClusterSum {
  ClusterSlots& slots;
  int S, rank, turn = 0;
  uint32_t parity = 0;
  Patience wait;
  __device__ __forceinline__ ClusterSum(ClusterSlots& s, int S_, const Stall& stall)
      : slots(s), S(S_), rank(cluster_ctarank()), wait(stall.limit, S_) {
    if (threadIdx.x == 0) {
      mbar_init(&slots.come[0], 1);
      mbar_init(&slots.come[1], 1);
      fence_mbar_init();
    }
    __syncthreads();
    cluster_arrive();
    cluster_wait();
  }
  __device__ __forceinline__ void operator()(float (&v)[kSums]) {
    uint64_t* come = &slots.come[turn];
    if (threadIdx.x == 0 && !wait.lost()) mbar_arrive_expect_tx(come, static_cast<uint32_t>(S) * sizeof(float2));
    if (static_cast<int>(threadIdx.x) < wait.open)
      send_f2(&slots.sums[turn][rank], come, threadIdx.x, v[0], v[kSums - 1]);
    __syncwarp();
    wait.cluster(come, parity);
    float2 t = make_float2(0.f, 0.f);
    for (int i = 0; i < S; ++i) {
      t.x += slots.sums[turn][i].x;
      t.y += slots.sums[turn][i].y;
    }
    v[0] = t.x;
    if (kSums > 1) v[kSums - 1] = t.y;
    turn ^= 1;
    parity ^= turn == 0 ? 1u : 0u;
  }
  __device__ __forceinline__ void end(uint32_t* status) {  // no block leaves while another may still write to it
    if (wait.lost() && status != nullptr) atomicOr(status, kStatusTimeout);
    cluster_arrive();
    cluster_wait();
    wait.leave();
  }
  __device__ __forceinline__ void silence() {  // for tests: the last block sends nothing any more
    if (rank == S - 1) wait.open = 0;
  }
};
// groups that are blocks of their own have nothing to join
template <int kSums>
struct NoSum {
  __device__ __forceinline__ NoSum(ClusterSlots&, int, const Stall&) {}
  __device__ __forceinline__ void operator()(float (&)[kSums]) {}
  __device__ __forceinline__ void silence() {}
  __device__ __forceinline__ void end(uint32_t*) {}
};
template <bool kShared, int kSums>
using SharedSum = std::conditional_t<kShared, ClusterSum<kSums>, NoSum<kSums>>;

// A thread's sums over its elements of a row of any length: add(part, j) for every one of them. 64 are added in
// sequence, and these parts with what each addition lost (Kahan's summation): like terms are rounded the same
// way, 4000003 equal fp32 elements gave a mean off by 3e-5 in one sequence.
template <int kSums, typename Add>
__device__ __forceinline__ void long_sums(int64_t N, float (&sums)[kSums], Add add) {
  float lost[kSums];
#pragma unroll
  for (int i = 0; i < kSums; ++i) sums[i] = lost[i] = 0.0f;
  for (int64_t from = threadIdx.x; from < N; from += 64 * blockDim.x) {
    float part[kSums];
#pragma unroll
    for (int i = 0; i < kSums; ++i) part[i] = 0.0f;
    const int64_t end = min(N, from + 64 * static_cast<int64_t>(blockDim.x));
    for (int64_t j = from; j < end; j += blockDim.x) add(part, j);
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
      const float v = part[i] - lost[i], t = sums[i] + v;
      const float l = (t - sums[i]) - v;
      lost[i] = l == l ? l : 0.0f;  // an infinite sum stays one
      sums[i] = t;
    }
  }
}

}  // namespace row

// whether all rows are whole 16-byte vectors (and the weights can be loaded 16 bytes at a time)
inline bool whole_vectors(int64_t N, int es, std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> lds,
                   std::initializer_list<const void*> weights) {
  bool ok = N * es % 16 == 0;
  for (const void* p : ptrs) ok = ok && reinterpret_cast<uintptr_t>(p) % 16 == 0;
  for (const void* p : weights) ok = ok && reinterpret_cast<uintptr_t>(p) % 16 == 0;
  for (int64_t ld : lds) ok = ok && ld * es % 16 == 0;
  return ok;
}
// threads a row for R vectors each: 8 or 16, or whole warps
inline int group_threads(int64_t n, int R) {
  const int64_t g = (n + R - 1) / R;
  return g <= 8 ? 8 : g <= 16 ? 16 : static_cast<int>((g + 31) / 32) * 32;
}

// a ragged group's rows are a multiple of 16 bytes apart: of so many rows
template <typename T>
int rows_apart(int64_t N) {
  return row::kElems<T> / static_cast<int>(std::gcd(N, static_cast<int64_t>(row::kElems<T>)));
}
// shared memory that a kernel has beside its static one without asking (48 KB with that)
constexpr size_t kPlainSmem = 40 * 1024;
// Lets a kernel take all shared memory that a block can have beside its static one. Always as much, whatever this call's
// plan takes: the limit is the kernel's, so a smaller one would fail the launch of another host thread's larger plan.
template <typename Kernel>
cudaError_t allow_all_smem(Kernel kernel, int dev) {
  cudaFuncAttributes of;
  int most = 0;
  cudaError_t e = cudaFuncGetAttributes(&of, kernel);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              most - static_cast<int>(of.sharedSizeBytes));
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
    if (smem > kPlainSmem) {
      e = allow_all_smem(kernel, dev);
      if (e != cudaSuccess) return e;
    }
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, block, smem);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorLaunchOutOfResources;
    cache = FitCache{dev, block, per_sm * device_sm_count(), smem};
  }
  blocks = cache.fit;
  return cudaSuccess;
}
}  // namespace swg
