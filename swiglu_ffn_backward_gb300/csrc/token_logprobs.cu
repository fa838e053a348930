// Log probabilities of given tokens over rows of logits, with the entropy and the k best alternatives,
// and their gradient.
//   d_j = (z_j - max z) / tau,  s = sum exp(d_j),  ln p_j = d_j - ln s
//   logp = ln p_t,  entropy H = ln s - (1/s) sum exp(d_j) d_j
//   dz_j = (1/tau) (dlogp ([j = t] - p_j) - dH p_j (ln p_j + H))
// Logits of -inf have probability 0; a row with no other logit has s = 0, H = 0, logp = -inf, no
// gradient. A NaN or +inf logit makes its row's results NaN.
//
// Forward: bound by HBM (V elements read a row). A cluster of S blocks takes a row, each block its share in
// registers (32 KB), so the row is read once: the block's maximum, then the two sums under it in one
// pass over the registers. The alternatives come from the same registers: the block's 32 lane columns
// have 32 maxima, the k-th largest of which is a bound that at least k logits reach, so the few logits
// at or above it (about k + k^2 / 64 of them) are collected and ranked against one another. The
// blocks send (max, sums, best keys) to the first one, which joins them in the blocks' order.
#include "swg_launch.h"
#include "vocab_rows.cuh"

namespace swg {
namespace {

using namespace row;

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kCand = 1024;  // candidates collected, at most (else the slower exact search)

struct TlpSmem {
  float lanes[kRowWarps][32];
  float2 sums[kRowWarps];
  uint64_t rounds[2][kRowWarps];
  uint64_t cand[kCand + kMaxTop];
  uint64_t best[kMaxTop];
  float4 part[kMaxCluster];  // of the first block: the blocks' max, sum 2^x, sum 2^x x, number of keys
  uint64_t part_best[kMaxCluster][kMaxTop];
  int ncand;
};

// The rare cases of the selection read the chunk at c again (from L2) instead of holding it in registers
// beside the sums.
//
// One warp: the first `need` logits equal to `bound` in index order -> cand; returns how many there are
// (at most need).
template <typename T>
__device__ __noinline__ int collect_equal(const T* z, int64_t V, const Share& sh, int c, float bound, int need,
                                          uint64_t* cand) {
  constexpr int E = Traits<T>::E;
  const int lane = threadIdx.x & 31;
  const int end = min(sh.end, c + kChunk);
  int found = 0;
  for (int g0 = c; g0 < end && found < need; g0 += 32) {
    const int64_t e0 = first_element<T>(sh, g0 + lane);
    uint32_t hits = 0;
    if (g0 + lane < end) {
      const Vec v = load_row_vec<T, true>(z, e0, V);
#pragma unroll
      for (int p = 0; p < E / 2; ++p) {
        const float2 x = vec_pair<T>(v, p);
        hits |= (x.x == bound ? 1u : 0u) << (2 * p) | (x.y == bound ? 2u : 0u) << (2 * p);
      }
    }
    int upto = __popc(hits);  // of the lanes up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += t;
    }
    for (int at = found + upto - __popc(hits); hits != 0 && at < need; ++at, hits &= hits - 1)
      cand[at] = rank_key(bound, static_cast<uint32_t>(e0) + __ffs(hits) - 1);
    found += __shfl_sync(0xffffffffu, upto, 31);
  }
  return found < need ? found : need;
}
// the thread's best key below `below` among its logits above -inf, 0 if there is none
template <typename T>
__device__ __noinline__ uint64_t best_below(const T* z, int64_t V, const Share& sh, int c, uint64_t below) {
  constexpr int E = Traits<T>::E;
  const int end = min(sh.end, c + kChunk);
  uint64_t best = 0;
  for (int g = c + static_cast<int>(threadIdx.x); g < end; g += kRowThreads) {
    const int64_t e0 = first_element<T>(sh, g);
    const Vec v = load_row_vec<T, true>(z, e0, V);
#pragma unroll
    for (int p = 0; p < E / 2; ++p) {
      const float2 x = vec_pair<T>(v, p);
      const uint32_t at = static_cast<uint32_t>(e0 + 2 * p);
      const uint64_t k0 = rank_key(x.x, at), k1 = rank_key(x.y, at + 1);
      if (x.x > neg_inf() && k0 < below && k0 > best) best = k0;
      if (x.y > neg_inf() && k1 < below && k1 > best) best = k1;
    }
  }
  return best;
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads, 3) tlp_fwd_kernel(const TlpFwdArgs a, int64_t row0, Split split) {
  constexpr int E = Traits<T>::E;
  __shared__ TlpSmem sm;
  const int S = split.S;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  if (S > 1) cluster_arrive();
  const int64_t r = row0 + blockIdx.x / S;
  const T* z = static_cast<const T*>(a.logits) + r * a.ld;
  const Share sh = share_of(z, a.V, split.per, rank);
  const float c2 = a.inv_temp * kLog2e;

  // What the block has seen, the same in every thread: max, sum 2^x and sum 2^x x with
  // x = (z - max) log2(e) / tau, number of best keys.
  float m = neg_inf(), s = 0.f, w = 0.f;
  int nbest = 0;
  for (int c = sh.begin; c < sh.end; c += kChunk) {
    Vec v[kVecs];
    load_chunk<T, true>(v, z, a.V, sh, c);
    float tm = neg_inf();
#pragma unroll
    for (int i = 0; i < kVecs; ++i) tm = fmaxf(tm, vec_max<T>(v[i]));
    sm.lanes[warp][lane] = tm;
    if (tid == 0) sm.ncand = 0;
    __syncthreads();
    float lm = sm.lanes[0][lane];
#pragma unroll
    for (int i = 1; i < kRowWarps; ++i) lm = fmaxf(lm, sm.lanes[i][lane]);
    const float mn = fmaxf(m, warp_max(lm));
    const Scale kn = scale_of(mn, c2);

    float2 s2 = make_float2(0.f, 0.f), w2 = s2;
    const float2 nref = make_float2(-kn.ref, -kn.ref), kc = make_float2(kn.c, kn.c);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
#pragma unroll
      for (int p = 0; p < E / 2; ++p) {
        float2 x = __ffma2_rn(vec_pair<T>(v[i], p), kc, nref);
        x = make_float2(at_least(x.x), at_least(x.y));
        const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
        s2 = __fadd2_rn(s2, e);
        w2 = __ffma2_rn(e, x, w2);
      }
    }
    const float ws = warp_sum(s2.x + s2.y), ww = warp_sum(w2.x + w2.y);
    if (lane == 0) sm.sums[warp] = make_float2(ws, ww);

    float bound = neg_inf(), kept = neg_inf();
    // the thread's logits at or above the bound (strict: above it) and above `kept` -> the candidates
    auto collect = [&](bool strict) {
      auto good = [&](float x) { return (strict ? x > bound : x >= bound) && x > kept; };
      if (!good(tm)) return;
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        if (!good(vec_max<T>(v[i]))) continue;
        const uint32_t e0 = static_cast<uint32_t>(first_element<T>(sh, c + i * kRowThreads + tid));
#pragma unroll
        for (int p = 0; p < E / 2; ++p) {
          const float2 x = vec_pair<T>(v[i], p);
          if (good(x.x)) {
            const int n = atomicAdd(&sm.ncand, 1);
            if (n < kCand) sm.cand[n] = rank_key(x.x, e0 + 2 * p);
          }
          if (good(x.y)) {
            const int n = atomicAdd(&sm.ncand, 1);
            if (n < kCand) sm.cand[n] = rank_key(x.y, e0 + 2 * p + 1);
          }
        }
      }
    };
    if (a.top > 0) {
      // the top-th largest of the lane columns' maxima
      int above = 0;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float o = __shfl_sync(0xffffffffu, lm, j);
        above += (o > lm || (o == lm && j < lane)) ? 1 : 0;
      }
      const uint32_t at = __ballot_sync(0xffffffffu, above == a.top - 1);
      bound = __shfl_sync(0xffffffffu, lm, __ffs(at) - 1);
      // later logits that only equal the worst one kept come after it
      kept = nbest == a.top ? rank_logit(sm.best[a.top - 1]) : neg_inf();
      collect(false);
    }
    __syncthreads();

    // join the sums with the earlier chunks'
    const float x0 = ref_shift(m, scale_of(m, c2), mn, kn, c2), f = ex2_approx(x0);
    w = f * fmaf(s, x0, w);
    s *= f;
    float cs = 0.f, cw = 0.f;
#pragma unroll
    for (int i = 0; i < kRowWarps; ++i) {
      const float2 t = sm.sums[i];
      cs += t.x;
      cw += t.y;
    }
    s += cs;
    w += cw;
    m = mn;

    if (a.top > 0) {
      int n = sm.ncand;
      if (n > kCand) {
        // a plateau at the bound: the logits above it, then the first ones equal to it
        __syncthreads();
        if (tid == 0) sm.ncand = 0;
        __syncthreads();
        collect(true);
        __syncthreads();
        n = sm.ncand;
        if (n < a.top) {
          __syncthreads();
          if (warp == 0 && bound > kept) {
            const int more = collect_equal(z, a.V, sh, c, bound, a.top - n, sm.cand + n);
            if (lane == 0) sm.ncand = n + more;
          }
          __syncthreads();
          n = sm.ncand;
        }
      }
      if (n > kCand) {
        // the best logits in few lane columns: one round for each of the best, in which only the thread
        // that had it looks through its logits again
        uint64_t mine = best_below(z, a.V, sh, c, ~0ull);
        for (n = 0; n < a.top; ++n) {
          const uint64_t wm = warp_max(mine);
          if (lane == 0) sm.rounds[n & 1][warp] = wm;
          __syncthreads();
          uint64_t b = 0;
#pragma unroll
          for (int i = 0; i < kRowWarps; ++i) b = sm.rounds[n & 1][i] > b ? sm.rounds[n & 1][i] : b;
          if (b == 0) break;
          if (mine == b) {
            sm.cand[n] = b;
            mine = best_below(z, a.V, sh, c, b);
          }
        }
        __syncthreads();
      }
      if (nbest > 0) {
        if (tid < nbest) sm.cand[n + tid] = sm.best[tid];
        n += nbest;
        __syncthreads();
      }
      for (int t = tid; t < n; t += kRowThreads) {
        const uint64_t key = sm.cand[t];
        int place = 0;
        for (int j = 0; j < n; ++j) place += sm.cand[j] > key ? 1 : 0;
        if (place < a.top) sm.best[place] = key;
      }
      nbest = n < a.top ? n : a.top;
    }
    __syncthreads();
  }

  uint64_t* best = sm.best;
  if (S > 1) {
    cluster_wait();  // every block has started
    if (tid == 0) st_peer_f4(&sm.part[rank], 0, make_float4(m, s, w, __int_as_float(nbest)));
    if (tid < nbest) st_peer_u64(&sm.part_best[rank][tid], 0, sm.best[tid]);
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    m = neg_inf();
    for (int i = 0; i < S; ++i) m = fmaxf(m, sm.part[i].x);
    const Scale k = scale_of(m, c2);
    s = w = 0.f;
    nbest = 0;
    for (int i = 0; i < S; ++i) {
      const float4 p = sm.part[i];
      const float x0 = ref_shift(p.x, scale_of(p.x, c2), m, k, c2), f = ex2_approx(x0);
      s = fmaf(f, p.y, s);
      w = fmaf(f, fmaf(p.y, x0, p.z), w);
      nbest += __float_as_int(p.w);
    }
    if (a.top > 0) {
      best = sm.cand;
      const int mine = tid / kMaxTop, at = tid % kMaxTop;  // kMaxCluster * kMaxTop = kRowThreads
      if (mine < S && at < __float_as_int(sm.part[mine].w)) {
        const uint64_t key = sm.part_best[mine][at];
        int place = 0;
        for (int i = 0; i < S; ++i) {
          const int n = __float_as_int(sm.part[i].w);
          for (int j = 0; j < n; ++j) place += sm.part_best[i][j] > key ? 1 : 0;
        }
        if (place < a.top) best[place] = key;
      }
      nbest = nbest < a.top ? nbest : a.top;
    }
    __syncthreads();
  }

  // H = ln s - (1/s) sum 2^x x ln 2, with s and x of one reference; then s at the maximum
  const float ent = s == 0.0f ? 0.0f : logf(s) - w * kLn2 / s;
  s = sum_at_max(s, m, scale_of(m, c2));
  const float me = finite_or_0(m), log_s = logf(s);
  auto logp_of = [&](float x) { return x == neg_inf() && s == s ? neg_inf() : (x - me) * a.inv_temp - log_s; };
  if (tid == 0) {
    a.stats[2 * r] = m;
    a.stats[2 * r + 1] = s;
    a.entropy[r] = ent;
    if (a.targets != nullptr) {
      const int64_t t = load_index(a.targets, r, a.wide);
      a.logp[r] = t == a.ignore ? 0.0f
                  : (t >= 0 && t < a.V) ? logp_of(to_f(z[t])) : __int_as_float(0x7fc00000);
    }
    // fewer logits above -inf than wanted: all of them are in the list, the lowest other indices follow
    for (uint32_t j = 0; nbest < a.top; ++j) {
      bool there = false;
      for (int i = 0; i < nbest; ++i) there = there || rank_index(best[i]) == j;
      if (!there) best[nbest++] = rank_key(neg_inf(), j);
    }
  }
  if (warp == 0) {
    __syncwarp();
    if (lane < a.top) {
      a.top_idx[r * a.top + lane] = rank_index(best[lane]);
      a.top_logp[r * a.top + lane] = logp_of(rank_logit(best[lane]));
    }
  }
}
static_assert(kMaxCluster * kMaxTop == kRowThreads, "one thread for each key of a cluster");
static_assert(kMaxTop == 32, "one lane for each alternative");

// Backward: bound by HBM (V elements read and written a row); no block needs another's results.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) tlp_bwd_kernel(const TlpBwdArgs a, int64_t row0, Split split) {
  constexpr int E = Traits<T>::E;
  const int64_t r = row0 + blockIdx.x / split.S;
  const T* z = static_cast<const T*>(a.logits) + r * a.ld;
  T* out = static_cast<T*>(a.dlogits) + r * a.ldo;
  const Share sh = share_of(z, a.V, split.per, static_cast<int>(blockIdx.x % split.S));
  const bool aligned = row_shift(out) == sh.shift;
  const float m = a.stats[2 * r];
  const Scale k = scale_of(m, a.inv_temp * kLog2e);
  const float s = sum_at_ref(a.stats[2 * r + 1], m, k);
  const int64_t t = a.targets != nullptr ? load_index(a.targets, r, a.wide) : a.ignore;
  const bool valid = t >= 0 && t < a.V;
  const float dl = t == a.ignore ? 0.0f : valid ? a.dlogp[r] : __int_as_float(0x7fc00000);
  const bool ent = a.dentropy != nullptr;
  const float dh = ent ? a.dentropy[r] : 0.0f;
  // dz = -(p / tau) (dl + dh (ln p + H)) = 2^x (k0 + k1 x), x as in scale_of, and dl / tau
  // more at the target
  const float inv_s = s == 0.0f ? 0.0f : 1.0f / s;
  const float scale = -inv_s * a.inv_temp;
  const float k0 = scale * (dl + (ent && s != 0.0f ? dh * (a.entropy[r] - logf(s)) : 0.0f));
  const float k1 = scale * dh * kLn2;
  const int64_t tt = t != a.ignore && valid && s != 0.0f ? t : -1;
  const float2 nref = make_float2(-k.ref, -k.ref), kc = make_float2(k.c, k.c), k02 = make_float2(k0, k0);
  const float2 k12 = make_float2(k1, k1);
  for (int c = sh.begin; c < sh.end; c += kChunk) {
    Vec v[kVecs];
    load_chunk<T, false>(v, z, a.V, sh, c);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int g = c + i * kRowThreads + static_cast<int>(threadIdx.x);
      if (g >= sh.end) break;
      const int64_t e0 = first_element<T>(sh, g);
#pragma unroll
      for (int p = 0; p < E / 2; ++p) {
        float2 x = __ffma2_rn(vec_pair<T>(v[i], p), kc, nref);
        x = make_float2(at_least(x.x), at_least(x.y));
        const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
        set_pair<T>(v[i], p, __fmul2_rn(e, __ffma2_rn(k12, x, k02)));
      }
      if (tt >= e0 && tt < e0 + E) {  // the target: formed anew, rounded once
        const float x0 = at_least(fmaf(to_f(z[tt]), k.c, -k.ref));
        const float x = fmaf(dl, a.inv_temp, ex2_approx(x0) * fmaf(k1, x0, k0));
        const int at = static_cast<int>(tt - e0);
#pragma unroll
        for (int p = 0; p < E / 2; ++p) {
          float2 y = vec_pair<T>(v[i], p);
          if (at == 2 * p) y.x = x;
          if (at == 2 * p + 1) y.y = x;
          set_pair<T>(v[i], p, y);
        }
      }
      store_row_vec(out, e0, a.V, aligned, v[i]);
    }
  }
}

}  // namespace

cudaError_t launch_token_logprobs_fwd(const TlpFwdArgs& a, int dtype, cudaStream_t stream) {
  const Split p = split_row(a.T, row_vectors(a.logits, a.V, a.ld, dtype == 0 ? 4 : 2), kChunk, device_sm_count());
  return launch_all_rows(a, dtype, p, p.S > 1, stream, tlp_fwd_kernel<float>, tlp_fwd_kernel<__half>,
                         tlp_fwd_kernel<__nv_bfloat16>);
}

cudaError_t launch_token_logprobs_bwd(const TlpBwdArgs& a, int dtype, cudaStream_t stream) {
  const Split p = split_row(a.T, row_vectors(a.logits, a.V, a.ld, dtype == 0 ? 4 : 2), kChunk, device_sm_count());
  return launch_all_rows(a, dtype, p, false, stream, tlp_bwd_kernel<float>, tlp_bwd_kernel<__half>,
                         tlp_bwd_kernel<__nv_bfloat16>);
}

}  // namespace swg
