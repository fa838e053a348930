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
// The computing warps (16, or four) keep (max, sum 2^x, sum 2^x x) and each thread its best logit and the run of four
// vectors that has it. A few more warps finish rows in turn, under the work on the next ones: they join
// the sums, and select the alternatives from the threads' bests. The 32 lane columns' bests have a k-th
// largest, which at least k logits reach; the few threads with a best at or above it (about k + k^2 / 64)
// are looked through again (their runs come from L2), and the logits found are ranked against one another.
// log2 e / tau is rounded to fp32 once, so that all exponents of a row are off by the same 2^-24 or so of their
// size, and ex2.approx is the exponential: both within the fp32 error that the tests allow.
// Measured with the 20 best: bf16 4096 x 131072 172 us, 93% of the copy bandwidth; 16384 x 32768 225 us, 72% (the
// computing warps' work on a row and the turn between rows: the schedulers issue in 60% of the cycles); fp32 8192
// x 32768 177 us, 91%; one row of 131072 fp32 12.5 us, shared by eight blocks.
#include <mutex>

#include "swg_launch.h"
#include "vocab_stream.cuh"

namespace swg {
namespace {

using namespace row;

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kCand = 512;      // candidates held; more are cut to the best before the search goes on
constexpr int kListed = 288;    // groups of runs listed before they are looked through

// blocks of 16 computing warps take long rows and share a row, those of four take many short ones
template <int W>
struct Plan {
  static constexpr int kStages = W == 16 ? 5 : 4;              // of the ring
  static constexpr int kSelectors = 3;                         // warps that finish rows
  static constexpr int kTableBytes = W == 16 ? 8192 : 4096;
  static constexpr int kBlocks = W == 16 ? kMaxCluster : 1;    // of a row, at most
  static constexpr int kThreads = 32 * (W + 1 + kSelectors);
};

template <int W>
struct TlpSync {
  Ring<W, Plan<W>::kStages> ring;
  uint64_t told[Plan<W>::kSelectors];   // the computing warps have written a row's results
  uint64_t taken[Plan<W>::kSelectors];  // the selector has read them
  uint64_t sent;                  // first block: the other blocks' results have come
};
// one selector's, behind the ring in dynamic shared memory
template <int W>
struct Finish {
  // the largest logit of every group of a thread's runs (as they are in the row, -inf for none): group j
  // of thread t at j * threads + t
  unsigned char table[Plan<W>::kTableBytes];
  uint64_t keys[Shape<W>::kThreads];     // a thread's best logit and its group, 0 for none
  alignas(16) uint64_t cand[kCand];
  uint4 runs[4][32];                     // the runs looked at: vector u of lane l at [u][l]
  uint64_t best[Plan<W>::kBlocks][kMaxTop];  // by block; sorted, the better first
  float4 block[Plan<W>::kBlocks];        // the blocks' sums (WarpSums::result)
  float4 part[W];                        // the computing warps'
  uint16_t list[kListed];                // groups to look through
};
template <int W>
constexpr size_t kFwdSmem = Plan<W>::kStages * Shape<W>::kStageBytes + Plan<W>::kSelectors * sizeof(Finish<W>);

// One warp: the `top` best of cand[0 .. n) -> best, in order; returns how many there are.
__device__ __forceinline__ int rank_candidates(const uint64_t* cand, int n, int top, uint64_t* best) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  for (int t0 = 0; t0 < n; t0 += 64) {  // two keys a lane against all
    const uint64_t a = t0 + lane < n ? cand[t0 + lane] : 0, b = t0 + 32 + lane < n ? cand[t0 + 32 + lane] : 0;
    int pa = 0, pb = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const uint64_t o = cand[j];
      pa += o > a ? 1 : 0;
      pb += o > b ? 1 : 0;
    }
    if (a != 0 && pa < top) best[pa] = a;
    if (b != 0 && pb < top) best[pb] = b;
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

// stages of one thread's group: one, or as many as let the table hold the share
template <typename T, int W>
__device__ __forceinline__ int group_stages(const Share& sh) {
  const int stages = (sh.end - sh.begin + Shape<W>::kStageVecs - 1) / Shape<W>::kStageVecs;
  constexpr int kGroups = Plan<W>::kTableBytes / static_cast<int>(sizeof(T)) / Shape<W>::kThreads;  // a thread
  return stages <= kGroups ? 1 : (stages + kGroups - 1) / kGroups;
}

// One warp: the `top` best logits above -inf of a share, from the threads' bests and the table -> best.
// done(): both have been read; load(g): the row's vector g.
template <typename T, int W, typename Done, typename Load>
__device__ __forceinline__ int select_best(const Share& sh, int top, Finish<W>& f, uint64_t* best, Done done,
                                           Load load) {
  constexpr int E = Traits<T>::E, kThreads = Shape<W>::kThreads, kStageVecs = Shape<W>::kStageVecs;
  const int lane = threadIdx.x & 31;
  // the lane columns' bests; an empty one counts as a key of its own below all others
  uint64_t column = 31 - lane;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const uint64_t k = f.keys[i * 32 + lane];
    column = k > column ? k : column;
  }
  f.cand[lane] = column;
  __syncwarp();
  int above = 0;
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(f.cand + j);
    above += (o.x > column ? 1 : 0) + (o.y > column ? 1 : 0);
  }
  uint64_t bound = __shfl_sync(0xffffffffu, column, __ffs(__ballot_sync(0xffffffffu, above == top - 1)) - 1);
  if (bound < 32) bound = 0;
  __syncwarp();
  // A group reaches the bound with a larger logit, or with an equal one if it is the bound's group or one
  // before it in the row: groups of one run follow each other, those of several stages only by stages. A
  // logit reaches it likewise, up to the end of those groups.
  T least = lowest<T>();
  int last = 0x7fffffff;  // group
  uint64_t least_key = 0;
  const int depth = group_stages<T, W>(sh);  // stages a group
  if (bound != 0) {
    least = from_f<T>(rank_logit(bound));
    last = static_cast<int>(rank_index(bound));
    if (depth > 1) last |= kThreads - 1;
    const int64_t stage = static_cast<int64_t>(last / kThreads + 1) * depth - 1;
    const int64_t end = stage * kStageVecs + 4 * (last % kThreads) + 4;  // of the share's vectors
    const int64_t behind = first_element<T>(sh, sh.begin) + end * E - 1;
    least_key = rank_key(rank_logit(bound), static_cast<uint32_t>(min(behind, static_cast<int64_t>(0xfffffffe))));
  }

  // the runs of the groups listed, one run a lane at a time
  int have = 0;  // candidates
  auto look_through = [&](int groups) {
    const int items = groups * depth;
    for (int i0 = 0; i0 < items; i0 += 32) {
      const int i = i0 + lane;
      int g = sh.end;
      if (i < items) {
        const int q = i / depth, group = f.list[q];
        g = sh.begin + ((group / kThreads) * depth + (i - q * depth)) * kStageVecs + 4 * (group % kThreads);
      }
      Vec v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (g + u < sh.end) v[u] = load(g + u);
      uint32_t hits = 0;  // bit by bit, the lane's logits that reach the bound
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (g + u >= sh.end) continue;
        f.runs[u][lane] = make_uint4(v[u].w[0], v[u].w[1], v[u].w[2], v[u].w[3]);
        hits |= at_or_above<T>(v[u], least) << (u * E);
      }
      const int64_t e0 = first_element<T>(sh, g);
      while (__any_sync(0xffffffffu, hits != 0)) {  // one logit a lane at a time
        uint64_t key = 0;
        if (hits != 0) {
          const int at = __ffs(hits) - 1;
          hits &= hits - 1;
          const T x = reinterpret_cast<const T*>(&f.runs[at / E][lane])[at % E];
          key = rank_key(to_f(x), static_cast<uint32_t>(e0 + at));
        }
        if (have > kCand - 32) {
          // only the best candidates stay, and the worst of them is the new bound
          have = rank_candidates(f.cand, have, top, best);
          for (int t = lane; t < have; t += 32) f.cand[t] = best[t];
          if (have == top) {
            least_key = best[top - 1];
            least = from_f<T>(rank_logit(least_key));
            last = 0x7fffffff;
          }
          __syncwarp();
        }
        const bool good = key > least_key || (key != 0 && key == least_key);
        const uint32_t all = __ballot_sync(0xffffffffu, good);
        if (good) f.cand[have + __popc(all & ((1u << lane) - 1u))] = key;
        have += __popc(all);
      }
      __syncwarp();
    }
  };

  const int groups = ((sh.end - sh.begin + kStageVecs - 1) / kStageVecs + depth - 1) / depth * kThreads;
  int listed = 0;
  if (groups == 0) done();
  for (int i0 = 0; i0 < groups; i0 += 32 * E) {  // E groups a lane
    const int i = i0 + lane * E;
    uint32_t hits = 0;
    if (i < groups) {
      const uint4 u = reinterpret_cast<const uint4*>(f.table)[i / E];
      const Vec v = Vec{{u.x, u.y, u.z, u.w}};
      hits = at_or_above<T>(v, least);
      if (i + E - 1 > last && hits != 0) {  // behind the bound's group only larger ones count
#pragma unroll
        for (int p = 0; p < E / 2; ++p) {
          const float2 x = vec_pair<T>(v, p);
          if (i + 2 * p > last && x.x == to_f(least)) hits &= ~(1u << (2 * p));
          if (i + 2 * p + 1 > last && x.y == to_f(least)) hits &= ~(2u << (2 * p));
        }
      }
    }
    while (__any_sync(0xffffffffu, hits != 0)) {
      const bool some = hits != 0;
      const uint32_t all = __ballot_sync(0xffffffffu, some);
      if (some) f.list[listed + __popc(all & ((1u << lane) - 1u))] = static_cast<uint16_t>(i + __ffs(hits) - 1);
      hits &= hits - 1;
      listed += __popc(all);
    }
    __syncwarp();
    if (i0 + 32 * E >= groups) done();
    if (listed > kListed - 32 * E || i0 + 32 * E >= groups) {
      look_through(listed);
      listed = 0;
    }
  }
  return rank_candidates(f.cand, have, top, best);
}
static_assert(kListed >= 32 * 8, "the list takes what one step adds");
static_assert(Plan<16>::kTableBytes / 2 <= 65536, "16-bit groups");

template <typename T, int W, bool kLong>  // kLong: as in WarpSums
__global__ void __launch_bounds__(Plan<W>::kThreads, W == 16 ? 1 : 3)
    tlp_fwd_kernel(const TlpFwdArgs a, Split split, Stall stall, uint32_t* status) {
  constexpr int kStageVecs = Shape<W>::kStageVecs, kStageBytes = Shape<W>::kStageBytes, kThreads = Shape<W>::kThreads;
  constexpr int kStages = Plan<W>::kStages, kSelectors = Plan<W>::kSelectors;
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ TlpSync<W> sm;
  Finish<W>* finish = reinterpret_cast<Finish<W>*>(dyn + kStages * kStageBytes);
  const int S = split.S;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_ctarank());
  const int64_t first = blockIdx.x / S, step = gridDim.x / S;
  const float c2 = a.inv_temp * kLog2e;
  if (tid == 0) {
    ring_init(sm.ring);
    for (int i = 0; i < kSelectors; ++i) {
      mbar_init(&sm.told[i], W);
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
  Patience wait(stall.limit);

  if (warp == W) {
    produce_rows<T, W>(a.logits, a.ld, a.V, first, a.T, step, split.per, rank, dyn, kStages, sm.ring, wait,
                       rank == S - 1 ? stall.at : -1);
  } else if (warp > W) {
    const int me = warp - W - 1;
    Finish<W>& f = finish[me];
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
      float4 p = join_sums(lane < W ? f.part[lane] : none, c2, k);
      int n = 0;
      auto taken = [&]() {
        if (lane == 0) mbar_arrive(&sm.taken[me]);
      };
      __syncwarp();
      if (a.top > 0) {
        // a row of its own is still in the ring; else it has left it for L2
        const bool held = S > 1 && sh.end - sh.begin <= kStages * kStageVecs;
        n = select_best<T, W>(sh, a.top, f, f.best[rank], taken, [&](int g) {
          if (!held) return load_row_vec<T, true>(z, first_element<T>(sh, g), a.V);
          const uint4 u = reinterpret_cast<const uint4*>(dyn)[g - sh.begin];
          return Vec{{u.x, u.y, u.z, u.w}};
        });
      } else {
        taken();
      }
      uint64_t mine = lane < n ? f.best[rank][lane] : 0;  // lane i: the i-th best
      if (Plan<W>::kBlocks > 1 && rank != 0) {  // once, whatever was lost: the first block has one row to hear of
        if (lane == 0) send_f4(&f.block[rank], &sm.sent, 0, p);
        send_u64(&f.best[rank][lane], &sm.sent, 0, mine);
        continue;
      }
      if constexpr (Plan<W>::kBlocks > 1) if (S > 1) {
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
    Place in;
    int sel = 0;            // the selector of the row
    uint32_t parity = 1;    // of its `taken`
    for (int64_t r = first; r < a.T; r += step) {
      const Share sh = share_of(static_cast<const T*>(a.logits) + r * a.ld, a.V, split.per, rank);
      Finish<W>& f = finish[sel];
      wait(&sm.taken[sel], parity);  // the selector has read the row before in its place
      T* table = reinterpret_cast<T*>(f.table);
      WarpSums<T, true, kLong> sums(c2);
      const int depth = group_stages<T, W>(sh);
      float most = neg_inf(), group_most = neg_inf();  // the thread's maximum, and that of its open group
      int best = 0, group = tid, left = depth;         // the first group that has it; the open group
      for (int at = sh.begin; at < sh.end; at += kStageVecs) {
        const int cnt = min(sh.end - at, kStageVecs);
        wait(&sm.ring.full[in.stage], in.parity);
        if (warp * kWarpVecs < cnt) {
          Vec v[4];
          read_stage_runs<T, W>(v, dyn + in.stage * kStageBytes, cnt);
          group_most = fmaxf(group_most, sums.add(v, c2, cnt < kStageVecs));
        }
        if (--left == 0 || at + kStageVecs >= sh.end) {
          if (a.top > 0) table[group] = from_f<T>(group_most);
          if (group_most > most) {
            most = group_most;
            best = group;
          }
          group += kThreads;
          left = depth;
          group_most = neg_inf();
        }
        __syncwarp();
        if (lane < wait.open) mbar_arrive(&sm.ring.empty[in.stage]);
        in.next(kStages);
      }
      const float4 p = sums.result();
      if (lane == 0) f.part[warp] = p;
      if (a.top > 0) f.keys[tid] = most > neg_inf() ? rank_key(most, static_cast<uint32_t>(best)) : 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.told[sel]);
      if (++sel == kSelectors) {
        sel = 0;
        parity ^= 1u;
      }
    }
  }
  __syncwarp();
  if (wait.lost() && status != nullptr) atomicOr(status, kStatusTimeout);
  cluster_arrive();  // no block leaves while another may still write to it
  cluster_wait();
  wait.leave();
}
static_assert(kMaxTop == 32, "one lane for each alternative");

template <typename T, int W, bool kLong>
cudaError_t launch_fwd(const TlpFwdArgs& a, Split split, cudaStream_t stream) {
  static std::mutex mu;  // guards the occupancy cache
  static StreamCache cache;
  std::lock_guard<std::mutex> lk(mu);
  // a cluster of several blocks takes one row
  return launch_stream(tlp_fwd_kernel<T, W, kLong>, cache, Plan<W>::kThreads, kFwdSmem<W>, a.T, split.S,
                       split.S > 1, stream, a, split, take_stall(kInjectTokenLogprobs), status_word_ptr());
}
template <int W, bool kLong>
cudaError_t launch_fwd_any(const TlpFwdArgs& a, int dtype, Split split, cudaStream_t stream) {
  return dtype == 0   ? launch_fwd<float, W, kLong>(a, split, stream)
         : dtype == 1 ? launch_fwd<__half, W, kLong>(a, split, stream)
                      : launch_fwd<__nv_bfloat16, W, kLong>(a, split, stream);
}

// Backward: bound by HBM (V elements read and written a row); no block needs another's results, so groups of
// 32 to 256 threads take shares of rows in registers, read once and written once. Measured with the entropy's
// gradient: 4096 x 65536 bf16 158 us, 102% of the copy bandwidth, 4096 x 50001 136 us, 90%.
template <typename T>
__global__ void __launch_bounds__(kRowThreads, 4) tlp_bwd_kernel(const TlpBwdArgs a, int64_t group0, Groups p) {
  constexpr int E = Traits<T>::E;
  const int64_t group = group0 + static_cast<int64_t>(blockIdx.x) * (kRowThreads / p.G) + threadIdx.x / p.G;
  const int tid = threadIdx.x & (p.G - 1);
  const int64_t r = group / p.S;
  if (r >= a.T) return;
  const T* z = static_cast<const T*>(a.logits) + r * a.ld;
  T* out = static_cast<T*>(a.dlogits) + r * a.ldo;
  const Share sh = share_of(z, a.V, p.per, static_cast<int>(group - r * p.S));
  const bool aligned = row_shift(out) == sh.shift;
  // fp32 logits are loaded ahead of the row's constants (1024 x 131072: 163 us instead of 193); with two
  // elements a register that costs registers and time (bf16 2048 x 131072: 163 us instead of 156)
  constexpr bool kFirst = sizeof(T) == 4;
  Vec v[kVecs];
  if (kFirst) load_chunk<T, false>(v, z, a.V, sh, sh.begin, tid, p.G);
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
  for (int c = sh.begin; c < sh.end; c += kVecs * p.G) {
    if (!kFirst || c > sh.begin) load_chunk<T, false>(v, z, a.V, sh, c, tid, p.G);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int g = c + i * p.G + tid;
      if (g >= sh.end) break;
      const int64_t e0 = first_element<T>(sh, g);
#pragma unroll
      for (int n = 0; n < E / 2; ++n) {
        float2 x = __ffma2_rn(vec_pair<T>(v[i], n), kc, nref);
        x = make_float2(at_least(x.x), at_least(x.y));
        const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
        set_pair<T>(v[i], n, __fmul2_rn(e, __ffma2_rn(k12, x, k02)));
      }
      if (tt >= e0 && tt < e0 + E) {  // the target: formed anew, rounded once
        const float x0 = at_least(fmaf(to_f(z[tt]), k.c, -k.ref));
        const float x = fmaf(dl, a.inv_temp, ex2_approx(x0) * fmaf(k1, x0, k0));
        const int at = static_cast<int>(tt - e0);
#pragma unroll
        for (int n = 0; n < E / 2; ++n) {
          float2 y = vec_pair<T>(v[i], n);
          if (at == 2 * n) y.x = x;
          if (at == 2 * n + 1) y.y = x;
          set_pair<T>(v[i], n, y);
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
  // Blocks of four computing warps, three an SM, take short rows, and rows up to 100 KB when each of those
  // blocks has two; blocks of 16 take the others. 1 GB of logits, the 20 best, four warps against 16: bf16 32768
  // columns 225 us against 255, 51200 (6400 vectors) 222 against 229, 60000 215 against 210, 131072 201 against 172;
  // fp32 8192 columns 209 against 379, 25600 (6400 vectors) 177 against 205, 32768 174 against 177, 50257 187
  // against 169.
  const int64_t sms = device_sm_count();
  const bool small = p.S == 1 && (vectors <= 1024 || (vectors <= 6400 && a.T >= 6 * sms));
  static_assert(6400 <= kFewStages * Shape<4>::kStageVecs, "rows of four warps are not long");
  if (small) return launch_fwd_any<4, false>(a, dtype, p, stream);
  return p.per > kFewStages * Shape<16>::kStageVecs ? launch_fwd_any<16, true>(a, dtype, p, stream)
                                                    : launch_fwd_any<16, false>(a, dtype, p, stream);
}

cudaError_t launch_token_logprobs_bwd(const TlpBwdArgs& a, int dtype, cudaStream_t stream) {
  const int64_t vectors = row_vectors(a.logits, a.V, a.ld, dtype == 0 ? 4 : 2);
  return launch_groups(a, dtype, row_groups(a.T, vectors, device_sm_count()), stream, tlp_bwd_kernel<float>,
                       tlp_bwd_kernel<__half>, tlp_bwd_kernel<__nv_bfloat16>);
}

}  // namespace swg
