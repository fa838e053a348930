// Distillation from a teacher's top logits: forward, backward, and both in one call.
//   teacher: entries (i_k, t_k), k < K, of a row; ids outside [0, V) are absent entries
//   q_k = softmax over the entries of t_k / tau
//   student: d_j = (z_j - max z) / tau, s = sum exp(d_j), ln p_j = d_j - ln s
//   loss = sum_k q_k (ln q_k - ln p_{i_k}),  dz_j = (w / tau) (Q p_j - q_j)
// with q_j the sum of the entries with i_k = j and Q = 1, or 0 for a row without entries (loss 0, no
// gradient). A weight w of 0 gives a zero gradient whatever the row holds.
#include "row_ops.cuh"
#include "swg_launch.h"

namespace swg {
namespace {

using namespace row;

constexpr int kThreads = 256;

struct TeacherSmem {
  int id[kKdMaxEntries];     // -1: absent
  float q[kKdMaxEntries];    // probabilities
  float td[kKdMaxEntries];   // teacher logits less their maximum
  float buf[kThreads / 32];
};

// the row's teacher entries -> shared memory; returns sum exp(td / tau), 0 for a row without entries
__device__ __forceinline__ float load_teacher(const KdArgs& a, int64_t r, TeacherSmem& sm) {
  float m = neg_inf();
  for (int k = threadIdx.x; k < a.K; k += kThreads) {
    const int64_t id = load_index(a.ids, r * a.K + k, a.wide);
    const bool there = id >= 0 && id < a.V;
    const float t = there ? load_any(a.teacher, r * a.K + k, a.tdtype) : neg_inf();
    sm.id[k] = there ? static_cast<int>(id) : -1;
    sm.td[k] = t;
    m = fmaxf(m, t);
  }
  m = block_max(m, sm.buf);
  const float me = m == neg_inf() ? 0.0f : m;
  float s = 0.f;
  for (int k = threadIdx.x; k < a.K; k += kThreads) {
    const float d = sm.td[k] - me;
    const float e = ex2_approx(d * a.inv_temp * kLog2e);
    sm.td[k] = d;
    sm.q[k] = e;
    s += e;
  }
  s = block_sum(s, sm.buf);
  const float inv = s == 0.0f ? 0.0f : 1.0f / s;
  for (int k = threadIdx.x; k < a.K; k += kThreads) sm.q[k] *= inv;
  __syncthreads();
  return s;
}

// mode: 1 loss and statistics, 2 gradient from saved statistics, 3 both
template <typename T, int kMode>
__global__ void __launch_bounds__(kThreads) kd_kernel(const KdArgs a) {
  __shared__ TeacherSmem sm;
  const int64_t r = blockIdx.x;
  const T* z = static_cast<const T*>(a.logits) + r * a.ld;
  const float sq = load_teacher(a, r, sm);
  const float Q = sq == 0.0f ? 0.0f : 1.0f;
  float m, s;
  if (kMode & 1) {
    m = neg_inf();
    for (int64_t j = threadIdx.x; j < a.V; j += kThreads) m = fmaxf(m, to_f(z[j]));
    m = block_max(m, sm.buf);
    const float me = m == neg_inf() ? 0.0f : m;
    s = 0.f;
    for (int64_t j = threadIdx.x; j < a.V; j += kThreads) s += ex2_approx((to_f(z[j]) - me) * a.inv_temp * kLog2e);
    s = block_sum(s, sm.buf);
  } else {
    m = a.stats_in[2 * r];
    s = a.stats_in[2 * r + 1];
  }
  const float me = m == neg_inf() ? 0.0f : m;
  if (kMode & 1) {
    // sum q (ln q - ln p) = sum (q / tau) (td - (z - max z)) - ln sq + ln s: a mask of the type's lowest
    // value leaves the range of fp32 only where the loss does
    float l = 0.f;
    for (int k = threadIdx.x; k < a.K; k += kThreads) {
      const float q = sm.q[k];
      if (q == 0.0f || sm.id[k] < 0) continue;
      l = fmaf(q * a.inv_temp, sm.td[k] - (to_f(z[sm.id[k]]) - me), l);
    }
    l = block_sum(l, sm.buf);
    if (threadIdx.x == 0) {
      a.stats[2 * r] = m;
      a.stats[2 * r + 1] = s;
      a.loss[r] = sq == 0.0f ? 0.0f : l + ((s == 0.0f ? 0.0f : logf(s)) - logf(sq));
    }
  }
  if (kMode & 2) {
    T* out = static_cast<T*>(a.dlogits) + r * a.ldo;
    const float w = a.weight[r] * a.inv_temp;
    const float inv_s = s == 0.0f ? 0.0f : 1.0f / s;
    // logits at the entries, before an output in their place overwrites them
    float zk[(kKdMaxEntries + kThreads - 1) / kThreads];
#pragma unroll
    for (int i = 0; i < (kKdMaxEntries + kThreads - 1) / kThreads; ++i) {
      const int k = threadIdx.x + i * kThreads;
      zk[i] = k < a.K && sm.id[k] >= 0 ? to_f(z[sm.id[k]]) : 0.0f;
    }
    __syncthreads();
    for (int64_t j = threadIdx.x; j < a.V; j += kThreads) {
      const float p = ex2_approx((to_f(z[j]) - me) * a.inv_temp * kLog2e) * inv_s;
      out[j] = from_f<T>(w == 0.0f ? 0.0f : w * (Q * p));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < (kKdMaxEntries + kThreads - 1) / kThreads; ++i) {
      const int k = threadIdx.x + i * kThreads;
      if (k >= a.K || sm.id[k] < 0) continue;
      float q = 0.f;
      for (int n = 0; n < a.K; ++n) q += sm.id[n] == sm.id[k] ? sm.q[n] : 0.0f;
      const float p = ex2_approx((zk[i] - me) * a.inv_temp * kLog2e) * inv_s;
      out[sm.id[k]] = from_f<T>(w == 0.0f ? 0.0f : w * (Q * p - q));
    }
  }
}

template <int kMode>
cudaError_t launch_mode(const KdArgs& a, int dtype, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(a.T);
  if (dtype == 0) kd_kernel<float, kMode><<<grid, kThreads, 0, stream>>>(a);
  else if (dtype == 1) kd_kernel<__half, kMode><<<grid, kThreads, 0, stream>>>(a);
  else kd_kernel<__nv_bfloat16, kMode><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_distill(const KdArgs& a, bool forward, bool backward, int dtype, cudaStream_t stream) {
  return forward ? (backward ? launch_mode<3>(a, dtype, stream) : launch_mode<1>(a, dtype, stream))
                 : launch_mode<2>(a, dtype, stream);
}

}  // namespace swg
