// Distillation from a teacher's top logits: forward, backward, and both in one call.
//   teacher: entries (i_k, t_k), k < K, of a row; ids outside [0, V) are absent entries
//   q_k = softmax over the entries of t_k / tau
//   student: d_j = (z_j - max z) / tau, s = sum exp(d_j), ln p_j = d_j - ln s
//   loss = sum_k q_k (ln q_k - ln p_{i_k}),  dz_j = (w / tau) (Q p_j - q_j)
// with q_j the sum of the entries with i_k = j and Q = 1, or 0 for a row without entries (loss 0, no
// gradient). A weight w of 0 gives a zero gradient whatever the row holds.
//
// Bound by HBM: V elements a row are read, and written where there is a gradient. For loss and gradient
// at once a cluster of S blocks holds the row in registers (32 KB a block): each block's (max, sum) go to
// every block of the cluster through distributed shared memory, and the gradient is formed from the
// registers, so the logits are read once (a row longer than the cluster's registers is read again). One
// warp takes the teacher's entries while the row is on its way. The gradient's sparse part, at most K
// elements a row, is written over the dense part by the block that wrote it.
#include "swg_launch.h"
#include "vocab_rows.cuh"

namespace swg {
namespace {

using namespace row;

struct KdSmem {
  float lanes[kRowWarps];
  float sums[kRowWarps];
  float2 part[kMaxCluster];  // the blocks' max and sum
  float sq;                  // sum exp((t - max t) / tau), 0 for a row without entries
  int id[kKdMaxEntries];     // -1: absent
  float q[kKdMaxEntries];    // probabilities
  float td[kKdMaxEntries];   // teacher logits less their maximum
  float z[kKdMaxEntries];    // the student's logits at the entries (those that the block needs)
};

// One warp: the row's teacher entries -> shared memory. The student's logits are gathered for the ids in
// [e0, e1): a gradient in their place may overwrite them later.
template <typename T>
__device__ __forceinline__ void load_teacher(const KdArgs& a, int64_t r, const T* z, int64_t e0, int64_t e1,
                                             KdSmem& sm) {
  const int lane = threadIdx.x & 31;
  float m = neg_inf();
  for (int k = lane; k < a.K; k += 32) {
    const int64_t id = load_index(a.ids, r * a.K + k, a.wide);
    const bool there = id >= 0 && id < a.V;
    const float t = there ? load_any(a.teacher, r * a.K + k, a.tdtype) : neg_inf();
    sm.id[k] = there ? static_cast<int>(id) : -1;
    sm.td[k] = t;
    sm.z[k] = id >= e0 && id < e1 ? to_f(z[id]) : 0.0f;
    m = fmaxf(m, t);
  }
  const float me = finite_or_0(warp_max(m));
  float s = 0.f;
  for (int k = lane; k < a.K; k += 32) {
    const float d = sm.td[k] - me;
    const float e = ex2_approx(d * a.inv_temp * kLog2e);
    sm.td[k] = d;
    sm.q[k] = e;
    s += e;
  }
  s = warp_sum(s);
  const float inv = s == 0.0f ? 0.0f : 1.0f / s;
  for (int k = lane; k < a.K; k += 32) sm.q[k] *= inv;
  if (lane == 0) sm.sq = s;
}

struct Gradient {
  float me, c2;  // 2^((z - me) c2) is the unscaled probability
  float dense;   // w Q / (tau s)
  float sparse;  // w / tau
};
__device__ __forceinline__ Gradient make_gradient(const KdArgs& a, float m, float s, float w, float sq) {
  const float wt = w * a.inv_temp;
  return Gradient{finite_or_0(m), a.inv_temp * kLog2e, s == 0.0f || sq == 0.0f ? 0.0f : wt / s, wt};
}

// the dense part of the chunk at c
template <typename T>
__device__ __forceinline__ void store_dense(Vec (&v)[kVecs], const Gradient& g, T* out, int64_t V, bool aligned,
                                            const Share& sh, int64_t c) {
  constexpr int E = Traits<T>::E;
  const float2 nm2 = make_float2(-g.me, -g.me), cc2 = make_float2(g.c2, g.c2), k2 = make_float2(g.dense, g.dense);
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int64_t at = c + i * kRowThreads + threadIdx.x;
    if (at >= sh.end) break;
#pragma unroll
    for (int p = 0; p < E / 2; ++p) {
      const float2 x = __fmul2_rn(__fadd2_rn(vec_pair<T>(v[i], p), nm2), cc2);
      set_pair<T>(v[i], p, __fmul2_rn(make_float2(ex2_approx(x.x), ex2_approx(x.y)), k2));
    }
    store_row_vec(out, at * E - sh.shift, V, aligned, v[i]);
  }
}
// a gradient of zeros
template <typename T>
__device__ __forceinline__ void store_zeros(T* out, int64_t V, bool aligned, const Share& sh) {
  const Vec zero = {{0u, 0u, 0u, 0u}};
  for (int64_t at = sh.begin + threadIdx.x; at < sh.end; at += kRowThreads)
    store_row_vec(out, at * Traits<T>::E - sh.shift, V, aligned, zero);
}
// the elements at the entries in [e0, e1); an id that comes twice is written by its first entry
template <typename T>
__device__ __forceinline__ void store_sparse(const KdArgs& a, const Gradient& g, const KdSmem& sm, T* out, int64_t e0,
                                             int64_t e1) {
  for (int k = threadIdx.x; k < a.K; k += kRowThreads) {
    const int id = sm.id[k];
    if (id < 0 || id < e0 || id >= e1) continue;
    float q = 0.f;
    bool first = true;
    for (int n = 0; n < a.K; ++n) {
      if (sm.id[n] != id) continue;
      first = first && n >= k;
      q += sm.q[n];
    }
    if (first)
      out[id] = from_f<T>(fmaf(g.dense, ex2_approx((sm.z[k] - g.me) * g.c2), -g.sparse * q));
  }
}

// loss and statistics; with kGrad the gradient as well
template <typename T, bool kGrad>
__global__ void __launch_bounds__(kRowThreads) kd_fwd_kernel(const KdArgs a, int64_t row0, int S) {
  constexpr int E = Traits<T>::E;
  __shared__ KdSmem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  if (S > 1) cluster_arrive();
  const int64_t r = row0 + blockIdx.x / S;
  const T* z = static_cast<const T*>(a.logits) + r * a.ld;
  const Share sh = share_of(z, a.V, S, rank);
  const int64_t e0 = sh.begin * E - sh.shift, e1 = sh.end * E - sh.shift;  // the elements of the share
  const float c2 = a.inv_temp * kLog2e;

  float m = neg_inf(), s = 0.f;  // of the block, the same in every thread
  Vec v[kVecs];
  for (int64_t c = sh.begin; c < sh.end || c == sh.begin; c += kChunk) {
    load_chunk<T, !kGrad>(v, z, a.V, sh, c);
    // the first block forms the loss: it needs the logits at all entries
    if (c == sh.begin && warp == kRowWarps - 1) load_teacher(a, r, z, rank == 0 ? 0 : e0, rank == 0 ? a.V : e1, sm);
    float tm = neg_inf();
#pragma unroll
    for (int i = 0; i < kVecs; ++i) tm = fmaxf(tm, vec_max<T>(v[i]));
    tm = warp_max(tm);
    if (lane == 0) sm.lanes[warp] = tm;
    __syncthreads();
    float mn = m;
#pragma unroll
    for (int i = 0; i < kRowWarps; ++i) mn = fmaxf(mn, sm.lanes[i]);
    const float me = finite_or_0(mn);
    const float2 nm2 = make_float2(-me, -me), cc2 = make_float2(c2, c2);
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
#pragma unroll
      for (int p = 0; p < E / 2; ++p) {
        const float2 x = __fmul2_rn(__fadd2_rn(vec_pair<T>(v[i], p), nm2), cc2);
        s2 = __fadd2_rn(s2, make_float2(ex2_approx(x.x), ex2_approx(x.y)));
      }
    }
    const float ws = warp_sum(s2.x + s2.y);
    if (lane == 0) sm.sums[warp] = ws;
    __syncthreads();
    s *= ex2_approx(part_shift(m, mn, c2));
    float cs = 0.f;
#pragma unroll
    for (int i = 0; i < kRowWarps; ++i) cs += sm.sums[i];
    s += cs;
    m = mn;
  }
  if (S > 1) {
    cluster_wait();  // every block has started
    if (tid < S) {
      const uint32_t to = peer_addr(&sm.part[rank], static_cast<uint32_t>(tid));
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(m), "f"(s) : "memory");
    }
    cluster_arrive();
    cluster_wait();
    m = neg_inf();
    for (int i = 0; i < S; ++i) m = fmaxf(m, sm.part[i].x);
    s = 0.f;
    for (int i = 0; i < S; ++i) s = fmaf(ex2_approx(part_shift(sm.part[i].x, m, c2)), sm.part[i].y, s);
  }
  const float sq = sm.sq;
  if (rank == 0 && warp == kRowWarps - 1) {
    // sum q (ln q - ln p) = sum (q / tau) (td - (z - max z)) - ln sq + ln s: a mask of the type's lowest
    // value leaves the range of fp32 only where the loss does
    const float me = finite_or_0(m);
    float l = 0.f;
    for (int k = lane; k < a.K; k += 32) {
      const float q = sm.q[k];
      if (q == 0.0f || sm.id[k] < 0) continue;
      l = fmaf(q * a.inv_temp, sm.td[k] - (sm.z[k] - me), l);
    }
    l = warp_sum(l);
    if (lane == 0) {
      a.stats[2 * r] = m;
      a.stats[2 * r + 1] = s;
      a.loss[r] = sq == 0.0f ? 0.0f : l + ((s == 0.0f ? 0.0f : logf(s)) - logf(sq));
    }
  }
  if (kGrad) {
    T* out = static_cast<T*>(a.dlogits) + r * a.ldo;
    const bool aligned = row_shift(out) == sh.shift;
    const float w = a.weight[r];
    if (w == 0.0f) {
      store_zeros(out, a.V, aligned, sh);
      return;
    }
    const Gradient g = make_gradient(a, m, s, w, sq);
    const bool held = sh.end - sh.begin <= kChunk;  // the registers hold the whole share
    for (int64_t c = sh.begin; c < sh.end; c += kChunk) {
      if (!held) load_chunk<T, false>(v, z, a.V, sh, c);
      store_dense(v, g, out, a.V, aligned, sh, c);
    }
    __syncthreads();  // the sparse part goes over the dense one
    store_sparse(a, g, sm, out, e0, e1);
  }
}

// the gradient from saved statistics
template <typename T>
__global__ void __launch_bounds__(kRowThreads) kd_bwd_kernel(const KdArgs a, int64_t row0, int S) {
  constexpr int E = Traits<T>::E;
  __shared__ KdSmem sm;
  const int64_t r = row0 + blockIdx.x / S;
  const T* z = static_cast<const T*>(a.logits) + r * a.ld;
  T* out = static_cast<T*>(a.dlogits) + r * a.ldo;
  const Share sh = share_of(z, a.V, S, static_cast<int>(blockIdx.x % S));
  const bool aligned = row_shift(out) == sh.shift;
  const float w = a.weight[r];
  if (w == 0.0f) {
    store_zeros(out, a.V, aligned, sh);
    return;
  }
  const int64_t e0 = sh.begin * E - sh.shift, e1 = sh.end * E - sh.shift;
  Vec v[kVecs];
  load_chunk<T, false>(v, z, a.V, sh, sh.begin);
  if (threadIdx.x >= kRowThreads - 32) load_teacher(a, r, z, e0, e1, sm);
  __syncthreads();
  const Gradient g = make_gradient(a, a.stats_in[2 * r], a.stats_in[2 * r + 1], w, sm.sq);
  for (int64_t c = sh.begin; c < sh.end; c += kChunk) {
    if (c > sh.begin) load_chunk<T, false>(v, z, a.V, sh, c);
    store_dense(v, g, out, a.V, aligned, sh, c);
  }
  __syncthreads();  // the sparse part goes over the dense one
  store_sparse(a, g, sm, out, e0, e1);
}

}  // namespace

cudaError_t launch_distill(const KdArgs& a, bool forward, bool backward, int dtype, cudaStream_t stream) {
  const int S = row_blocks(a.T, row_vectors(a.logits, a.V, a.ld, dtype == 0 ? 4 : 2), device_sm_count());
  if (!forward)
    return launch_all_rows(a, dtype, S, false, stream, kd_bwd_kernel<float>, kd_bwd_kernel<__half>,
                           kd_bwd_kernel<__nv_bfloat16>);
  if (!backward)
    return launch_all_rows(a, dtype, S, S > 1, stream, kd_fwd_kernel<float, false>, kd_fwd_kernel<__half, false>,
                           kd_fwd_kernel<__nv_bfloat16, false>);
  return launch_all_rows(a, dtype, S, S > 1, stream, kd_fwd_kernel<float, true>, kd_fwd_kernel<__half, true>,
                         kd_fwd_kernel<__nv_bfloat16, true>);
}

}  // namespace swg
