// Log probabilities of given tokens over rows of logits, with the entropy and the k best alternatives,
// and their gradient.
//   d_j = (z_j - max z) / tau,  s = sum exp(d_j),  ln p_j = d_j - ln s
//   logp = ln p_t,  entropy H = ln s - (1/s) sum exp(d_j) d_j
//   dz_j = (1/tau) (dlogp ([j = t] - p_j) - dH p_j (ln p_j + H))
// Logits of -inf have probability 0; a row with no other logit has s = 0, H = 0, logp = -inf, no
// gradient. A NaN or +inf logit makes its row's results NaN.
//
// Forward: bound by HBM (V elements read a row). A persistent kernel streams rows through shared memory
// (vocab_stream.cuh); S blocks of a cluster share a row only when there are too few rows for the SMs.
// The 16 computing warps keep (max, sum 2^x, sum 2^x x) and each thread its best logit and the run of four
// vectors that has it. Four more warps finish rows in turn, under the work on the next ones: they join
// the sums, and select the alternatives from the threads' bests. The 32 lane columns' bests have a k-th
// largest, which at least k logits reach; the few threads with a best at or above it (about k + k^2 / 64)
// are looked through again (their runs come from L2), and the logits found are ranked against one another.
#include <mutex>

#include "swg_launch.h"
#include "vocab_stream.cuh"

namespace swg {
namespace {

using namespace row;

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kStages = 5;      // of the ring
constexpr int kRingBytes = kStages * kStageBytes;
constexpr int kSelectors = 4;   // warps that finish rows
constexpr int kFwdThreads = kStreamThreads + 32 * (1 + kSelectors);
constexpr int kCand = 512;      // candidates held; more are cut to the best before the search goes on

struct TlpSync {
  Ring<kStages> ring;
  uint64_t told[kSelectors];   // the computing warps have written a row's results
  uint64_t taken[kSelectors];  // the selector has read them
  uint64_t sent;               // first block: the other blocks' results have come
};
// one selector's, behind the ring in dynamic shared memory
struct Finish {
  uint64_t keys[kStreamThreads];         // a thread's best logit and its run, 0 for none
  uint64_t cand[kCand];
  uint64_t best[kMaxCluster][kMaxTop];   // by block; sorted, the better first
  float4 block[kMaxCluster];             // the blocks' sums (WarpSums::result)
  float4 part[kStreamWarps];             // the computing warps'
  uint16_t who[kStreamThreads];          // threads to look through again
  int count;
};
constexpr size_t kFwdSmem = kRingBytes + kSelectors * sizeof(Finish);

// One warp: the `top` best of cand[0 .. n) -> best, in order; returns how many there are.
__device__ __forceinline__ int rank_candidates(const uint64_t* cand, int n, int top, uint64_t* best) {
  __syncwarp();
  for (int t = threadIdx.x & 31; t < n; t += 32) {
    const uint64_t key = cand[t];
    int place = 0;
    for (int j = 0; j < n; ++j) place += cand[j] > key ? 1 : 0;
    if (place < top) best[place] = key;
  }
  __syncwarp();
  return n < top ? n : top;
}

// Two descending lists of 32 keys, one key a lane -> the 32 best of both, descending: the larger of one
// list and the other one reversed are those, in bitonic order.
__device__ __forceinline__ uint64_t merge_lists(uint64_t a, uint64_t b) {
  const int lane = threadIdx.x & 31;
  const uint64_t r = __shfl_sync(0xffffffffu, b, 31 - lane);
  a = r > a ? r : a;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t p = __shfl_xor_sync(0xffffffffu, a, o);
    a = ((lane & o) == 0) == (p > a) ? p : a;
  }
  return a;
}

// One warp: the `top` best logits above -inf of a share, from the threads' bests -> best. done(): the
// threads' bests have been read; load(g): the row's vector g.
template <typename T, typename Done, typename Load>
__device__ __forceinline__ int select_best(const Share& sh, int top, Finish& f, uint64_t* best, Done done, Load load) {
  constexpr int E = Traits<T>::E;
  const int lane = threadIdx.x & 31;
  uint64_t column = 0;
#pragma unroll
  for (int i = 0; i < kStreamWarps; ++i) {
    const uint64_t k = f.keys[i * 32 + lane];
    column = k > column ? k : column;
  }
  f.cand[lane] = column;
  __syncwarp();
  int above = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const uint64_t o = f.cand[j];
    above += o > column || (o == column && j < lane) ? 1 : 0;
  }
  const uint64_t bound = __shfl_sync(0xffffffffu, column, __ffs(__ballot_sync(0xffffffffu, above == top - 1)) - 1);
  int threads = 0;
#pragma unroll
  for (int i = 0; i < kStreamWarps; ++i) {
    const uint64_t k = f.keys[i * 32 + lane];
    const bool good = k != 0 && k >= bound;
    const uint32_t all = __ballot_sync(0xffffffffu, good);
    if (good) f.who[threads + __popc(all & ((1u << lane) - 1u))] = static_cast<uint16_t>(i * 32 + lane);
    threads += __popc(all);
  }
  if (lane == 0) f.count = 0;
  __syncwarp();
  done();
  // a logit reaches the bound if it is larger, or equal and in the same run or before it
  float least = bound != 0 ? rank_logit(bound) : neg_inf();
  uint64_t least_key =
      bound != 0 ? rank_key(least, static_cast<uint32_t>(first_element<T>(sh, sh.begin + 4 * static_cast<int>(rank_index(bound)) + 4) - 1)) : 0;
  const int stages = (sh.end - sh.begin + kStageVecs - 1) / kStageVecs, items = threads * stages;
  for (int i0 = 0; i0 < items; i0 += 32) {  // a run for each lane
    Vec v[4];
    const int i = i0 + lane, q = i / stages;
    const int g = i < items ? sh.begin + (i - q * stages) * kStageVecs + 4 * f.who[q] : sh.end;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (g + u < sh.end) {
        v[u] = load(g + u);
      } else {
#pragma unroll
        for (int w = 0; w < 4; ++w) v[u].w[w] = Traits<T>::kNegInf;
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      int n = f.count;
      if (n > kCand - 32 * E) {
        // the list could overflow: only the best stay, and the worst of them is the new bound
        n = rank_candidates(f.cand, n, top, best);
        for (int t = lane; t < n; t += 32) f.cand[t] = best[t];
        if (n == top) {
          least_key = best[top - 1];
          least = rank_logit(least_key);
        }
        if (lane == 0) f.count = n;
        __syncwarp();
      }
      const float vm = vec_max<T>(v[u]);
      if (vm >= least && vm > neg_inf()) {
        const uint32_t e0 = static_cast<uint32_t>(first_element<T>(sh, g + u));
#pragma unroll
        for (int p = 0; p < E / 2; ++p) {
          const float2 x = vec_pair<T>(v[u], p);
          const uint64_t k0 = rank_key(x.x, e0 + 2 * p), k1 = rank_key(x.y, e0 + 2 * p + 1);
          if (x.x > neg_inf() && k0 >= least_key) f.cand[atomicAdd(&f.count, 1)] = k0;
          if (x.y > neg_inf() && k1 >= least_key) f.cand[atomicAdd(&f.count, 1)] = k1;
        }
      }
      __syncwarp();
    }
  }
  return rank_candidates(f.cand, f.count, top, best);
}
static_assert(kCand - 32 * 8 >= kMaxTop, "room for the best and one vector of every lane");

template <typename T>
__global__ void __launch_bounds__(kFwdThreads, 1) tlp_fwd_kernel(const TlpFwdArgs a, Split split, uint32_t* status) {
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ TlpSync sm;
  Finish* finish = reinterpret_cast<Finish*>(dyn + kRingBytes);
  const int S = split.S;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_ctarank());
  const int64_t first = blockIdx.x / S, step = gridDim.x / S;
  const float c2 = a.inv_temp * kLog2e;
  if (tid == 0) {
    ring_init(sm.ring);
    for (int i = 0; i < kSelectors; ++i) {
      mbar_init(&sm.told[i], kStreamWarps);
      mbar_init(&sm.taken[i], 1);
    }
    mbar_init(&sm.sent, 1);
    fence_mbar_init();
    // a cluster of several blocks has one row: the first block hears from the others once
    mbar_arrive_expect_tx(&sm.sent, static_cast<uint32_t>(S - 1) * (sizeof(float4) + kMaxTop * sizeof(uint64_t)));
  }
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  Patience wait;

  if (warp == kStreamWarps) {
    produce_rows<T>(a.logits, a.ld, a.V, first, a.T, step, split.per, rank, dyn, sm.ring, wait);
  } else if (warp > kStreamWarps) {
    const int me = warp - kStreamWarps - 1;
    Finish& f = finish[me];
    uint32_t parity = 0;
    for (int64_t r = first + me * step; r < a.T; r += kSelectors * step, parity ^= 1u) {
      const T* z = static_cast<const T*>(a.logits) + r * a.ld;
      const Share sh = share_of(z, a.V, split.per, rank);
      int64_t t = a.ignore;
      float zt = 0.0f;
      bool given = false;
      if (rank == 0 && a.targets != nullptr) {
        t = load_index(a.targets, r, a.wide);
        given = t >= 0 && t < a.V;
        if (given) zt = to_f(z[t]);
      }
      wait(&sm.told[me], parity);
      const float4 none = make_float4(neg_inf(), 0.f, 0.f, neg_inf());
      Scale k;
      float4 p = join_sums(lane < kStreamWarps ? f.part[lane] : none, c2, k);
      int n = 0;
      auto taken = [&]() {
        if (lane == 0) mbar_arrive(&sm.taken[me]);
      };
      __syncwarp();
      if (a.top > 0) {
        // a row of its own is still in the ring; else it has left it for L2
        const bool held = S > 1 && sh.end - sh.begin <= kStages * kStageVecs;
        n = select_best<T>(sh, a.top, f, f.best[rank], taken, [&](int g) {
          if (!held) return load_row_vec<T, true>(z, first_element<T>(sh, g), a.V);
          const uint4 u = reinterpret_cast<const uint4*>(dyn)[g - sh.begin];
          return Vec{{u.x, u.y, u.z, u.w}};
        });
      } else {
        taken();
      }
      uint64_t mine = lane < n ? f.best[rank][lane] : 0;  // lane i: the i-th best
      if (rank != 0) {
        if (lane == 0) send_f4(&f.block[rank], &sm.sent, 0, p);
        send_u64(&f.best[rank][lane], &sm.sent, 0, mine);
        continue;
      }
      if (S > 1) {
        if (lane == 0) f.block[0] = p;
        f.best[0][lane] = mine;
        __syncwarp();
        wait.cluster(&sm.sent, 0);
        p = join_sums(lane < S ? f.block[lane] : none, c2, k);
        if (a.top > 0) {
          uint64_t list[kMaxCluster];
#pragma unroll
          for (int i = 0; i < kMaxCluster; ++i) list[i] = i < S ? f.best[i][lane] : 0;
#pragma unroll
          for (int half = kMaxCluster / 2; half > 0; half /= 2) {
#pragma unroll
            for (int i = 0; i < half; ++i) list[i] = merge_lists(list[i], list[i + half]);
          }
          mine = list[0];
          n = min(a.top, __popc(__ballot_sync(0xffffffffu, mine != 0)));
        }
      }
      const float m = p.w;
      // H = ln s - (1/s) sum 2^x x ln 2, with s and x of one reference; then s at the maximum
      const float ent = p.y == 0.0f ? 0.0f : logf(p.y) - p.z * kLn2 / p.y;
      const float s = sum_at_max(p.y, m, k), log_s = logf(s), top = finite_or_0(m);
      auto logp_of = [&](float x) { return x == neg_inf() && s == s ? neg_inf() : (x - top) * a.inv_temp - log_s; };
      if (lane == 0) {
        a.stats[2 * r] = m;
        a.stats[2 * r + 1] = s;
        a.entropy[r] = ent;
        if (a.targets != nullptr)
          a.logp[r] = t == a.ignore ? 0.0f : given ? logp_of(zt) : __int_as_float(0x7fc00000);
      }
      // fewer logits above -inf than wanted: all of them are there, the lowest other indices follow
      for (uint32_t j = 0; n < a.top; ++j) {
        if (__any_sync(0xffffffffu, lane < n && rank_index(mine) == j)) continue;
        if (lane == n) mine = rank_key(neg_inf(), j);
        ++n;
      }
      if (lane < a.top) {
        a.top_idx[r * a.top + lane] = rank_index(mine);
        a.top_logp[r * a.top + lane] = logp_of(rank_logit(mine));
      }
      __syncwarp();
    }
  } else {
    Place<kStages> in;
    int sel = 0;            // the selector of the row
    uint32_t parity = 1;    // of its `taken`
    for (int64_t r = first; r < a.T; r += step) {
      const Share sh = share_of(static_cast<const T*>(a.logits) + r * a.ld, a.V, split.per, rank);
      WarpSums<T, true> sums(c2);
      float most = neg_inf();  // the thread's maximum and the first run that has it
      int run = 0;
      for (int at = sh.begin; at < sh.end; at += kStageVecs) {
        Vec v[4];
        const int cnt = min(sh.end - at, kStageVecs);
        wait(&sm.ring.full[in.stage], in.parity);
        read_stage_runs<T>(v, dyn + in.stage * kStageBytes, cnt);
        const float x = sums.add(v, c2, cnt < kStageVecs);
        if (x > most) {
          most = x;
          run = (at - sh.begin) / 4 + tid;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.ring.empty[in.stage]);
        in.next();
      }
      const float4 p = sums.result();
      Finish& f = finish[sel];
      wait(&sm.taken[sel], parity);
      if (lane == 0) f.part[warp] = p;
      if (a.top > 0) f.keys[tid] = most > neg_inf() ? rank_key(most, static_cast<uint32_t>(run)) : 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.told[sel]);
      if (++sel == kSelectors) {
        sel = 0;
        parity ^= 1u;
      }
    }
  }
  __syncwarp();
  if (wait.lost && status != nullptr) atomicOr(status, kStatusTimeout);
  cluster_arrive();  // no block leaves while another may still write to it
  cluster_wait();
}
static_assert(kMaxTop == 32, "one lane for each alternative");

template <typename T>
cudaError_t launch_fwd(const TlpFwdArgs& a, Split split, cudaStream_t stream) {
  static std::mutex mu;  // guards the occupancy cache
  static StreamCache cache;
  std::lock_guard<std::mutex> lk(mu);
  // a cluster of several blocks takes one row
  return launch_stream(tlp_fwd_kernel<T>, cache, kFwdThreads, kFwdSmem, a.T, split.S, split.S > 1, stream, a, split,
                       status_word_ptr());
}

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
  const int64_t vectors = row_vectors(a.logits, a.V, a.ld, dtype == 0 ? 4 : 2);
  const Split p = split_row(a.T, vectors, vectors, device_sm_count());
  return dtype == 0   ? launch_fwd<float>(a, p, stream)
         : dtype == 1 ? launch_fwd<__half>(a, p, stream)
                      : launch_fwd<__nv_bfloat16>(a, p, stream);
}

cudaError_t launch_token_logprobs_bwd(const TlpBwdArgs& a, int dtype, cudaStream_t stream) {
  const Split p = split_row(a.T, row_vectors(a.logits, a.V, a.ld, dtype == 0 ? 4 : 2), kChunk, device_sm_count());
  return launch_all_rows(a, dtype, p, false, stream, tlp_bwd_kernel<float>, tlp_bwd_kernel<__half>,
                         tlp_bwd_kernel<__nv_bfloat16>);
}

}  // namespace swg
