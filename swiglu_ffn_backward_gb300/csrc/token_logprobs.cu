// Log probabilities of given tokens over rows of logits, with the entropy and the k best alternatives,
// and their gradient.
//   d_j = (z_j - max z) / tau,  s = sum exp(d_j),  ln p_j = d_j - ln s
//   logp = ln p_t,  entropy H = ln s - (1/s) sum exp(d_j) d_j
//   dz_j = (1/tau) (dlogp ([j = t] - p_j) - dH p_j (ln p_j + H))
// Logits of -inf have probability 0; a row with no other logit has s = 0, H = 0, logp = -inf, no
// gradient. A NaN or +inf logit makes its row's results NaN.
#include "row_ops.cuh"
#include "swg_launch.h"

namespace swg {
namespace {

using namespace row;

constexpr int kThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kThreads) tlp_fwd_kernel(const TlpFwdArgs a) {
  __shared__ float buf[kThreads / 32];
  __shared__ uint64_t kbuf[kThreads / 32];
  const int64_t r = blockIdx.x;
  const T* z = static_cast<const T*>(a.logits) + r * a.ld;
  float m = neg_inf();
  for (int64_t j = threadIdx.x; j < a.V; j += kThreads) m = fmaxf(m, to_f(z[j]));
  m = block_max(m, buf);
  const float me = m == neg_inf() ? 0.0f : m;
  float s = 0.f, e1 = 0.f;
  for (int64_t j = threadIdx.x; j < a.V; j += kThreads) {
    const float d = (to_f(z[j]) - me) * a.inv_temp;
    const float e = ex2_approx(d * kLog2e);
    s += e;
    e1 += e == 0.0f ? 0.0f : e * d;
  }
  s = block_sum(s, buf);
  e1 = block_sum(e1, buf);
  const float log_s = logf(s);
  auto logp_of = [&](float v) { return v == neg_inf() && s == s ? neg_inf() : (v - me) * a.inv_temp - log_s; };
  if (threadIdx.x == 0) {
    a.stats[2 * r] = m;
    a.stats[2 * r + 1] = s;
    a.entropy[r] = s == 0.0f ? 0.0f : log_s - e1 / s;
    if (a.targets != nullptr) {
      const int64_t t = load_index(a.targets, r, a.wide);
      a.logp[r] = t == a.ignore ? 0.0f
                  : (t >= 0 && t < a.V) ? logp_of(to_f(z[t])) : __int_as_float(0x7fc00000);
    }
  }
  uint64_t below = ~0ull;
  for (int k = 0; k < a.top; ++k) {
    uint64_t best = 0;
    for (int64_t j = threadIdx.x; j < a.V; j += kThreads) {
      const uint64_t key = rank_key(to_f(z[j]), static_cast<uint32_t>(j));
      if (key < below && key > best) best = key;
    }
    below = block_reduce(warp_max(best), kbuf, [](uint64_t p, uint64_t q) { return p > q ? p : q; });
    if (threadIdx.x == 0) {
      a.top_idx[r * a.top + k] = rank_index(below);
      a.top_logp[r * a.top + k] = logp_of(rank_logit(below));
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) tlp_bwd_kernel(const TlpBwdArgs a) {
  const int64_t r = blockIdx.x;
  const T* z = static_cast<const T*>(a.logits) + r * a.ld;
  T* out = static_cast<T*>(a.dlogits) + r * a.ldo;
  const float m = a.stats[2 * r], s = a.stats[2 * r + 1];
  const float me = m == neg_inf() ? 0.0f : m;
  const float inv_s = s == 0.0f ? 0.0f : 1.0f / s, log_s = s == 0.0f ? 0.0f : logf(s);
  const int64_t t = a.targets != nullptr ? load_index(a.targets, r, a.wide) : a.ignore;
  const bool valid = t >= 0 && t < a.V;
  const float dl = t == a.ignore ? 0.0f : valid ? a.dlogp[r] : __int_as_float(0x7fc00000);
  const float dh = a.dentropy != nullptr ? a.dentropy[r] : 0.0f;
  const float H = a.dentropy != nullptr ? a.entropy[r] : 0.0f;
  for (int64_t j = threadIdx.x; j < a.V; j += kThreads) {
    const float d = (to_f(z[j]) - me) * a.inv_temp;
    const float p = ex2_approx(d * kLog2e) * inv_s;
    float g = -p * (dl + (p == 0.0f ? 0.0f : dh * (d - log_s + H)));
    if (j == t && s != 0.0f) g += dl;
    out[j] = from_f<T>(g * a.inv_temp);
  }
}

}  // namespace

cudaError_t launch_token_logprobs_fwd(const TlpFwdArgs& a, int dtype, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(a.T);
  if (dtype == 0) tlp_fwd_kernel<float><<<grid, kThreads, 0, stream>>>(a);
  else if (dtype == 1) tlp_fwd_kernel<__half><<<grid, kThreads, 0, stream>>>(a);
  else tlp_fwd_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_token_logprobs_bwd(const TlpBwdArgs& a, int dtype, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(a.T);
  if (dtype == 0) tlp_bwd_kernel<float><<<grid, kThreads, 0, stream>>>(a);
  else if (dtype == 1) tlp_bwd_kernel<__half><<<grid, kThreads, 0, stream>>>(a);
  else tlp_bwd_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace swg
