// Distillation from a teacher's top logits: forward, backward, and both in one call.
//   teacher: entries (i_k, t_k), k < K, of a row; ids outside [0, V) are absent entries
//   q_k = softmax over the entries of t_k / tau
//   student: d_j = (z_j - max z) / tau, s = sum exp(d_j), ln p_j = d_j - ln s
//   loss = sum_k q_k (ln q_k - ln p_{i_k}),  dz_j = (w / tau) (Q p_j - q_j)
// with q_j the sum of the entries with i_k = j and Q = 1, or 0 for a row without entries (loss 0, no
// gradient). A weight w of 0 gives a zero gradient whatever the row holds.
//
// Bound by HBM: V elements a row are read, and written where there is a gradient.
// Loss, and loss with gradient: a persistent kernel streams rows through shared memory (vocab_stream.cuh).
// With a gradient a row's shares stay in the rings of a cluster of S blocks until it is written, so the
// logits are read once. The warps' (max, sum) go to every block of the cluster, where one warp joins them;
// the gradient of a row is formed after the sums of the next one, so the exchange is off the path. Two
// more warps take the teacher's entries of every other row each, a row ahead, and write the gradient's
// sparse part, at most K elements a row, over the dense one.
// The gradient alone needs no exchange: blocks take shares of rows in registers.
// Measured, bf16 with 64 entries: loss and gradient 4096 x 131072 323 us, 99% of the copy bandwidth, 16384 x 32768
// 328 us, 98%, 10682 x 50257 451 us, 71% (half-full stages), 65536 x 8192 444 us, 74% (the teachers' work on a
// row's entries); loss alone 4096 x 131072 161 us, gradient alone 314 us: the copy's rate.
#include <mutex>

#include "swg_launch.h"
#include "vocab_stream.cuh"

namespace swg {
namespace {

using namespace row;

struct Gradient {
  Scale k;       // 2^fma(z, k.c, -k.ref) / s is the probability
  float dense;   // w Q / (tau s)
  float sparse;  // w / (tau sq)
};
__device__ __forceinline__ Gradient make_gradient(const KdArgs& a, const Scale& k, float s, float w, float sq) {
  const float wt = w * a.inv_temp;
  return Gradient{k, s == 0.0f || sq == 0.0f ? 0.0f : wt / s, sq == 0.0f ? 0.0f : wt / sq};
}
// two elements of the dense part
__device__ __forceinline__ float2 dense_pair(const Gradient& g, float2 z) {
  const float2 x = __ffma2_rn(z, make_float2(g.k.c, g.k.c), make_float2(-g.k.ref, -g.k.ref));
  return __fmul2_rn(make_float2(ex2_approx(x.x), ex2_approx(x.y)), make_float2(g.dense, g.dense));
}

// ---- loss, and loss with gradient

constexpr int kExtraWarps = 4;  // producer, two teachers, joiner
constexpr int kStages = 6;      // of the ring, at most (fewer beside many entries)
constexpr int kSlots = 4;       // of exchange and entries: a slot is written again four rows later
constexpr int kShareStages = 2; // stages a row's share may hold: two rows' shares, and two stages ahead

template <int W>
struct KdStream {
  Ring<W, kStages> ring;
  uint64_t joined[kSlots];  // the row's maxima and sums have come from all blocks
  uint64_t ready[kSlots];   // the row's entries are in shared memory
  uint64_t spare[kSlots];   // the joiner is done with them
  uint64_t dense[kSlots];   // the dense part of the row's gradient is written
  uint64_t solved[kSlots];  // the row's gradient constants are in shared memory
  float4 part[kSlots][kMaxCluster][W];  // every warp's sums (WarpSums::result)
  float2 note[kSlots];      // from the first block: its entries' logits have been read
  Gradient grad[kSlots];
  float weight[kSlots];
  float sq[kSlots];         // sum exp((t - max t) / tau), 0 for a row without entries
};
// the entries of kSlots rows follow the ring in dynamic shared memory, K of each array, and behind them
// the teachers' tables of ids
struct EntryArrays {
  int* id;    // -1: absent
  float* td;  // teacher logits less their maximum; exp(td / tau) / sq are the probabilities
  float* z;   // the student's logits (first block: all, else those in the block's share)
};
__device__ __forceinline__ EntryArrays entry_arrays(unsigned char* at, int K, int b) {
  int* p = reinterpret_cast<int*>(at) + b * 3 * K;
  return EntryArrays{p, reinterpret_cast<float*>(p + K), reinterpret_cast<float*>(p + 2 * K)};
}
// slots of the table of ids: a power of two, eight times the entries, or twice where they are many (an entry's
// search takes a few hundred cycles a step, and the longest one of a warp counts)
__host__ __device__ __forceinline__ int table_slots(int K) {
  int n = 64;
  while (n < (K <= 128 ? 8 : 2) * K) n *= 2;
  return n;
}
// the table behind one row's entries, in words from them (16-byte aligned)
__host__ __device__ constexpr int table_at(int K) { return (3 * K + 3) / 4 * 4; }
__host__ __device__ constexpr size_t entry_bytes(int K) { return static_cast<size_t>(kSlots) * 3 * 4 * K; }

// A teacher warp takes the entries of row after row. The first kAhead of a row are loaded two rows ahead,
// and the student's logits at them a row ahead; they are kept as loaded, so that a load does not wait for the
// one before it.
constexpr int kAhead = 128;
struct EntryLoads {
  int64_t id[kAhead / 32];
  uint32_t t[kAhead / 32];
};
// the entries k0 .. k0 + kAhead - 1 of row r
__device__ __forceinline__ void load_some(const KdArgs& a, int64_t r, int k0, EntryLoads& n) {
  const int64_t at = r * a.K;
  const int k = k0 + static_cast<int>(threadIdx.x & 31);
  if (a.wide) {
#pragma unroll
    for (int i = 0; i < kAhead / 32; ++i)
      if (k + 32 * i < a.K) n.id[i] = static_cast<const int64_t*>(a.ids)[at + k + 32 * i];
  } else {
#pragma unroll
    for (int i = 0; i < kAhead / 32; ++i)
      if (k + 32 * i < a.K) n.id[i] = static_cast<const uint32_t*>(a.ids)[at + k + 32 * i];
  }
  if (a.tdtype == 0) {
#pragma unroll
    for (int i = 0; i < kAhead / 32; ++i)
      if (k + 32 * i < a.K) n.t[i] = static_cast<const uint32_t*>(a.teacher)[at + k + 32 * i];
  } else {
#pragma unroll
    for (int i = 0; i < kAhead / 32; ++i)
      if (k + 32 * i < a.K) n.t[i] = static_cast<const uint16_t*>(a.teacher)[at + k + 32 * i];
  }
}
// ids (-1 for absent entries), the teacher's logits, and the student's at the ids in [e0, e1), as loaded
template <typename T>
struct EntryValues {
  int id[kAhead / 32];
  uint32_t t[kAhead / 32];
  T z[kAhead / 32];
};
template <typename T>
__device__ __forceinline__ void gather_some(const KdArgs& a, int64_t r, int k0, const EntryLoads& n, int64_t e0,
                                            int64_t e1, EntryValues<T>& v) {
  const T* z = static_cast<const T*>(a.logits) + r * a.ld;
  const int k = k0 + static_cast<int>(threadIdx.x & 31);
#pragma unroll
  for (int i = 0; i < kAhead / 32; ++i) {
    const int64_t id = k + 32 * i >= a.K ? -1 : a.wide ? n.id[i] : static_cast<int32_t>(n.id[i]);
    v.id[i] = id >= 0 && id < a.V ? static_cast<int>(id) : -1;
    v.t[i] = n.t[i];
    v.z[i] = from_f<T>(0.0f);
    if (v.id[i] >= e0 && v.id[i] < e1 && v.id[i] >= 0) v.z[i] = z[v.id[i]];
  }
}
__device__ __forceinline__ float teacher_logit(const KdArgs& a, uint32_t u) {
  return a.tdtype == 0   ? __uint_as_float(u)
         : a.tdtype == 1 ? __half2float(__ushort_as_half(static_cast<uint16_t>(u)))
                         : __uint_as_float(u << 16);
}
// row r's entries, the first of them in v, -> shared memory; returns sum exp((t - max t) / tau)
template <typename T>
__device__ __forceinline__ float take_entries(const KdArgs& a, int64_t r, EntryValues<T>& v, const EntryArrays& n,
                                              int64_t e0, int64_t e1) {
  const int lane = threadIdx.x & 31;
  const float c2 = exponent_scale(a.inv_temp);
  float m = neg_inf();
  for (int k0 = 0;;) {
#pragma unroll
    for (int i = 0; i < kAhead / 32; ++i) {
      const int k = k0 + i * 32 + lane;
      if (k >= a.K) break;
      const float t = v.id[i] < 0 ? neg_inf() : teacher_logit(a, v.t[i]);
      m = fmaxf(m, t);
      n.id[k] = v.id[i];
      n.td[k] = t;
      n.z[k] = to_f(v.z[i]);
    }
    k0 += kAhead;
    if (k0 >= a.K) break;
    EntryLoads more;
    load_some(a, r, k0, more);
    gather_some(a, r, k0, more, e0, e1, v);
  }
  const float me = finite_or_0(warp_max(m));
  float s = 0.f;
  for (int k = lane; k < a.K; k += 32) {  // the lane's own entries
    const float d = n.td[k] - me;
    n.td[k] = d;
    s += ex2_approx(d * c2);
  }
  return warp_sum(s);
}
// Of the lane's entries (bit i: entry 32 i + lane) one for each id in [e0, e1); shared: those whose id comes
// again in the row. Which entry of an id it is may differ from run to run, what comes of it does not.
// (Finding the lanes of one id with a warp match first, 32 ids at a time, took 6 us more a row of 64 entries.)
__device__ __forceinline__ uint32_t first_entries(const KdArgs& a, const EntryArrays& n, int* table, int slots,
                                                  int64_t e0, int64_t e1, uint32_t& shared) {
  constexpr int kAgain = static_cast<int>(0x80000000u);  // an id that has come again; ids are below 2^31 - 1
  const int lane = threadIdx.x & 31;
  for (int i = lane; i < slots / 4; i += 32) reinterpret_cast<int4*>(table)[i] = make_int4(-1, -1, -1, -1);
  __syncwarp();
  auto place = [&](int id) { return static_cast<int>((static_cast<uint32_t>(id) * 2654435761u) >> 16) & (slots - 1); };
  uint32_t mine = 0;
  bool again = false;
  for (int k0 = 0; k0 < a.K; k0 += 32) {
    const int id = k0 + lane < a.K ? n.id[k0 + lane] : -1;
    if (id < 0 || id < e0 || id >= e1) continue;
    for (int at = place(id), step = 0; step < slots; at = (at + 1) & (slots - 1), ++step) {
      const int old = atomicCAS(&table[at], -1, id);
      if (old == -1) {
        mine |= 1u << (k0 / 32);
        break;
      }
      if ((old & ~kAgain) == id) {
        atomicOr(&table[at], kAgain);
        again = true;
        break;
      }
    }
  }
  shared = 0;
  if (!__any_sync(0xffffffffu, again)) return mine;
  __syncwarp();
  for (uint32_t todo = mine; todo != 0; todo &= todo - 1) {
    const int i = __ffs(todo) - 1, id = n.id[32 * i + lane];
    int at = place(id);
    for (int step = 0; step < slots && (table[at] & ~kAgain) != id; ++step) at = (at + 1) & (slots - 1);
    if ((table[at] & kAgain) != 0) shared |= 1u << i;
  }
  __syncwarp();
  return mine;
}
static_assert(kKdMaxEntries <= 32 * 32, "a bit for each of a lane's entries");
// One warp: the elements at the entries in `mine`; the probabilities of an id in `shared` are added lane by
// lane.
template <typename T>
__device__ __forceinline__ void store_sparse(const KdArgs& a, const Gradient& g, const EntryArrays& n, uint32_t mine,
                                             uint32_t shared, T* out) {
  const int lane = threadIdx.x & 31;
  const float c2 = exponent_scale(a.inv_temp);
  for (int k0 = 0; k0 < a.K; k0 += 32) {
    const bool own = mine >> (k0 / 32) & 1u;
    const int id = own ? n.id[k0 + lane] : -1;
    float q = own ? ex2_approx(n.td[k0 + lane] * c2) : 0.0f;
    for (uint32_t todo = __ballot_sync(0xffffffffu, shared >> (k0 / 32) & 1u); todo != 0; todo &= todo - 1) {
      const int from = __ffs(todo) - 1, its = __shfl_sync(0xffffffffu, id, from);
      float t = 0.f;
      for (int j = lane; j < a.K; j += 32)
        if (n.id[j] == its) t += ex2_approx(n.td[j] * c2);
      t = warp_sum(t);
      if (lane == from) q = t;
    }
    if (own)
      out[id] = from_f<T>(fmaf(g.dense, ex2_approx(fmaf(n.z[k0 + lane], g.k.c, -g.k.ref)), -g.sparse * q));
  }
}

template <typename T, bool kGrad, int W, bool kLong>  // kLong: as in WarpSums (with a gradient a share is short)
__global__ void __launch_bounds__(32 * (W + kExtraWarps), W == 16 ? 1 : 3)
    kd_fwd_kernel(const KdArgs a, Split split, int stages, int slots, Stall stall, uint32_t* status) {
  constexpr int E = Traits<T>::E;
  constexpr int kStreamThreads = Shape<W>::kThreads, kStageVecs = Shape<W>::kStageVecs;
  constexpr int kStageBytes = Shape<W>::kStageBytes;
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ KdStream<W> sm;
  const int S = split.S;
  auto entries = [&](int slot) { return entry_arrays(dyn + stages * kStageBytes, a.K, slot); };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_ctarank());
  const int64_t first = blockIdx.x / S, step = gridDim.x / S;
  const uint32_t bytes = static_cast<uint32_t>(S * W * sizeof(float4) + sizeof(float2));
  if (tid == 0) {
    ring_init(sm.ring);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sm.joined[i], 1);
      mbar_init(&sm.ready[i], 1);
      mbar_init(&sm.spare[i], 1);
      mbar_init(&sm.dense[i], W);
      mbar_init(&sm.solved[i], 1);
    }
    fence_mbar_init();
    for (int i = 0; i < kSlots; ++i) mbar_arrive_expect_tx(&sm.joined[i], bytes);
  }
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  Patience wait(stall.limit, S);
  const float c2 = exponent_scale(a.inv_temp);

  if (warp == W) {
    produce_rows<T, W>(a.logits, a.ld, a.V, first, a.T, step, split.per, rank, dyn, stages, sm.ring, wait,
                       rank == S - 1 ? stall.at : -1);
  } else if (warp == W + 1 || warp == W + 2) {
    // the teachers take the entries of every other row each; the sparse part of a row comes after the
    // entries of the teacher's next one, so nothing waits for it
    const int odd = warp - W - 1;
    int* table = reinterpret_cast<int*>(dyn + stages * kStageBytes + entry_bytes(a.K)) + odd * slots;
    const int64_t begin = first + odd * step;
    EntryLoads loads;
    EntryValues<T> next;
    auto share = [&](int64_t r) {
      return share_of(static_cast<const T*>(a.logits) + r * a.ld, a.V, split.per, rank);
    };
    // the student's logits at row r's entries: the first block forms the loss and needs them all
    auto gather = [&](int64_t r) {
      const Share sh = share(r);
      gather_some(a, r, 0, loads, rank == 0 ? 0 : first_element<T>(sh, sh.begin),
                  rank == 0 ? a.V : first_element<T>(sh, sh.end), next);
    };
    // the elements at the entries of row r, the it-th, over the dense part
    auto sparse = [&](int64_t r, int64_t it, uint32_t mine, uint32_t shared) {
      const int slot = static_cast<int>(it & (kSlots - 1));
      wait(&sm.dense[slot], static_cast<uint32_t>((it / kSlots) & 1));
      if (sm.weight[slot] == 0.0f) return;
      const EntryArrays n = entries(slot);
      const Gradient g = sm.grad[slot];
      store_sparse<T>(a, g, n, mine, shared, static_cast<T*>(a.dlogits) + r * a.ldo);
      __syncwarp();
    };
    if (begin < a.T) {
      load_some(a, begin, 0, loads);
      gather(begin);
      if (begin + 2 * step < a.T) load_some(a, begin + 2 * step, 0, loads);
    }
    int64_t it = odd;
    uint32_t mine = 0, shared = 0;
    for (int64_t r = begin; r < a.T; r += 2 * step, it += 2) {
      const int slot = static_cast<int>(it & (kSlots - 1));
      const EntryArrays n = entries(slot);
      const float w = kGrad ? a.weight[r] : 0.0f;
      EntryValues<T> now = next;
      if (r + 2 * step < a.T) {
        gather(r + 2 * step);
        if (r + 4 * step < a.T) load_some(a, r + 4 * step, 0, loads);
      }
      const Share sh = share(r);
      const int64_t e0 = first_element<T>(sh, sh.begin), e1 = first_element<T>(sh, sh.end);
      wait(&sm.spare[slot], static_cast<uint32_t>((it / kSlots) & 1) ^ 1u);
      const float sq = take_entries<T>(a, r, now, n, rank == 0 ? 0 : e0, rank == 0 ? a.V : e1);
      if (lane == 0) {
        sm.sq[slot] = sq;
        sm.weight[slot] = w;
      }
      __syncwarp();
      if (lane == 0 && !wait.lost()) mbar_arrive(&sm.ready[slot]);
      // A gradient over the logits may be written once the first block has read them here. Row it - 2 has
      // been joined here, so every block has been through row it - 4 and its barrier of this slot is set
      // for this row.
      if (rank == 0 && it >= 2)
        wait(&sm.spare[(it - 2) & (kSlots - 1)], static_cast<uint32_t>(((it - 2) / kSlots) & 1));
      if (rank == 0 && lane < wait.open)
        send_f2(&sm.note[slot], &sm.joined[slot], static_cast<uint32_t>(lane), 0.f, 0.f);
      __syncwarp();
      if (kGrad) {
        if (r != begin) sparse(r - 2 * step, it - 2, mine, shared);
        mine = first_entries(a, n, table, slots, e0, e1, shared);
      }
    }
    if (kGrad && begin < a.T) sparse(first + (it - 2) * step, it - 2, mine, shared);
  } else if (warp == W + 3) {
    // joins the row's maxima and sums, and forms the constants of its gradient and (first block) its loss
    int64_t it = 0;
    for (int64_t r = first; r < a.T; r += step, ++it) {
      const int slot = static_cast<int>(it & (kSlots - 1));
      const uint32_t parity = static_cast<uint32_t>((it / kSlots) & 1);
      wait.cluster(&sm.joined[slot], parity);
      if (lane == 0 && !wait.lost()) mbar_arrive_expect_tx(&sm.joined[slot], bytes);
      // lane by lane (up to four parts each), then the lanes
      const float4* part = &sm.part[slot][0][0];
      float m = neg_inf(), s = 0.f, top = neg_inf();
      for (int i = lane; i < S * W; i += 32) m = fmaxf(m, part[i].x);
      m = warp_max(m);
      const Scale k = scale_of(m, c2);
      for (int i = lane; i < S * W; i += 32) {
        const float4 p = part[i];
        s = fmaf(ex2_approx(ref_shift(p.x, scale_of(p.x, c2), m, k, c2)), p.y, s);
        top = fmaxf(top, p.w);
      }
      s = warp_sum(s);
      top = warp_max(top);
      wait(&sm.ready[slot], parity);
      const float sq = sm.sq[slot];
      if (lane == 0) {
        if (kGrad) sm.grad[slot] = make_gradient(a, k, s, sm.weight[slot], sq);
        if (!wait.lost()) mbar_arrive(&sm.solved[slot]);
      }
      if (rank == 0) {
        // sum q (ln q - ln p) = sum (q / tau) (td - (z - max z)) - ln sq + ln s: a mask of the type's
        // lowest value leaves the range of fp32 only where the loss does
        const EntryArrays n = entries(slot);
        const float me = finite_or_0(top), f = a.inv_temp / sq;
        float l = 0.f;
        for (int i = lane; i < a.K; i += 32) {
          const float e = ex2_approx(n.td[i] * c2);
          if (n.id[i] != -1 && e != 0.0f) l = fmaf(e * f, n.td[i] - (n.z[i] - me), l);
        }
        l = warp_sum(l);
        if (lane == 0) {
          s = sum_at_max(s, top, k);
          a.stats[2 * r] = top;
          a.stats[2 * r + 1] = s;
          a.loss[r] = sq == 0.0f ? 0.0f : l + ((s == 0.0f ? 0.0f : logf(s)) - logf(sq));
        }
      }
      __syncwarp();
      if (lane == 0 && !wait.lost()) mbar_arrive(&sm.spare[slot]);
    }
  } else {
    Place in, held;  // the next stage to read, and (with a gradient) the next one of the row before
    // max and sum of the warp's part of row r, sent to every block
    auto sums = [&](int64_t r, int slot) {
      const Share sh = share_of(static_cast<const T*>(a.logits) + r * a.ld, a.V, split.per, rank);
      WarpSums<T, false, kLong> sum(c2);
      for (int at = sh.begin; at < sh.end; at += kStageVecs) {
        const int cnt = min(sh.end - at, kStageVecs);
        wait(&sm.ring.full[in.stage], in.parity);
        // (with a gradient this costs more than it saves: 345 us instead of 325 for 4096 x 131072 bf16)
        if (kGrad || warp * kWarpVecs < cnt) {
          Vec v[4];
          if (kGrad || cnt == kStageVecs) read_stage<T, W>(v, dyn + in.stage * kStageBytes, cnt);
          else read_stage_runs<T, W>(v, dyn + in.stage * kStageBytes, cnt);  // the last warps have nothing to add
          sum.add(v, c2, false);
        }
        if (!kGrad) {
          __syncwarp();
          if (lane == 0 && !wait.lost()) mbar_arrive(&sm.ring.empty[in.stage]);
        }
        in.next(stages);
      }
      const float4 p = sum.result();
      if (lane < wait.open) send_f4(&sm.part[slot][rank][warp], &sm.joined[slot], static_cast<uint32_t>(lane), p);
      __syncwarp();
    };
    // The gradient of row r, the it-th of the block. Without a gradient only the wait is left: a warp is
    // at most a row ahead of the joiner, so the exchange slots are read before they are written again.
    auto finish = [&](int64_t r, int64_t it) {
      const int slot = static_cast<int>(it & (kSlots - 1));
      wait(&sm.solved[slot], static_cast<uint32_t>((it / kSlots) & 1));
      if (!kGrad) return;
      const T* z = static_cast<const T*>(a.logits) + r * a.ld;
      T* out = static_cast<T*>(a.dlogits) + r * a.ldo;
      const Share sh = share_of(z, a.V, split.per, rank);
      const bool aligned = row_shift(out) == sh.shift;
      const Gradient g = sm.grad[slot];
      const bool some = sm.weight[slot] != 0.0f;
      for (int c = sh.begin; c < sh.end; c += kStageVecs) {
        Vec v[4];
        const int cnt = min(sh.end - c, kStageVecs);
        read_stage<T, W>(v, dyn + held.stage * kStageBytes, cnt);
        __syncwarp();
        if (lane == 0 && !wait.lost()) mbar_arrive(&sm.ring.empty[held.stage]);
        held.next(stages);
        const int64_t e0 = first_element<T>(sh, c), e1 = first_element<T>(sh, c + cnt);
        T* to = out + e0 + tid * E;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (some) {
#pragma unroll
            for (int p = 0; p < E / 2; ++p) set_pair<T>(v[i], p, dense_pair(g, vec_pair<T>(v[i], p)));
          } else {
            v[i] = Vec{{0u, 0u, 0u, 0u}};
          }
        }
        // the stage's first and last vector may be partial
        const int whole0 = e0 < 0 ? 1 : 0, whole1 = e1 > a.V ? cnt - 1 : cnt;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = i * kStreamThreads + tid;
          if (aligned && at >= whole0 && at < whole1) st_vec(to + i * kStreamThreads * E, v[i]);
          else if (at < cnt) store_row_vec(out, e0 + at * E, a.V, aligned, v[i]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.dense[slot]);
    };
    int64_t it = 0;
    for (int64_t r = first; r < a.T; r += step, ++it) {
      sums(r, static_cast<int>(it & (kSlots - 1)));
      if (it > 0) finish(r - step, it - 1);
    }
    if (it > 0) finish(first + (it - 1) * step, it - 1);
  }
  __syncwarp();
  if (wait.lost() && status != nullptr) atomicOr(status, kStatusTimeout);
  cluster_arrive();  // no block leaves while another may still write to it
  cluster_wait();
  wait.leave();
}

template <typename T, bool kGrad, int W, bool kLong>
cudaError_t launch_fwd(const KdArgs& a, Split split, cudaStream_t stream) {
  static std::mutex mu;  // guards the occupancy cache
  static StreamCache cache;
  // two rows' shares need four stages; what the entries leave is for the rows ahead
  const int stages = a.K <= 256 ? kStages : a.K <= 512 ? kStages - 1 : kStages - 2, slots = table_slots(a.K);
  const size_t smem = stages * Shape<W>::kStageBytes + entry_bytes(a.K) + static_cast<size_t>(2) * slots * sizeof(int);
  std::lock_guard<std::mutex> lk(mu);
  return launch_stream(kd_fwd_kernel<T, kGrad, W, kLong>, cache, 32 * (W + kExtraWarps), smem, a.T, split.S, false,
                       stream, a, split, stages, slots, take_stall(kInjectDistill), status_word_ptr());
}
template <bool kGrad, int W, bool kLong>
cudaError_t launch_fwd_any(const KdArgs& a, int dtype, Split split, cudaStream_t stream) {
  return dtype == 0   ? launch_fwd<float, kGrad, W, kLong>(a, split, stream)
         : dtype == 1 ? launch_fwd<__half, kGrad, W, kLong>(a, split, stream)
                      : launch_fwd<__nv_bfloat16, kGrad, W, kLong>(a, split, stream);
}

// ---- gradient alone

// the block's barrier, from whichever place a warp comes to it
__device__ __forceinline__ void block_sync() { asm volatile("barrier.sync 0;" ::: "memory"); }

// The gradient from saved statistics: a block of G threads (64 to 256) takes a share of a row, up to 128 bytes a
// thread in registers at a time. A warp more takes the teacher's entries while it arrives, looks for ids that come
// again while the others form the dense part, and writes the sparse part over it. (With the first of the G threads'
// warps doing that too, 4096 x 32768 bf16 with 64 entries took 101 us instead of 85.)
template <typename T>
__global__ void __launch_bounds__(kRowThreads + 32, 4)
    kd_bwd_kernel(const KdArgs a, int64_t share0, Groups p, int slots) {
  constexpr int E = Traits<T>::E;
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ float sq_all;
  const int tid = threadIdx.x;
  const int64_t at = share0 + blockIdx.x, r = at / p.S;
  const T* z = static_cast<const T*>(a.logits) + r * a.ld;
  T* out = static_cast<T*>(a.dlogits) + r * a.ldo;
  const Share sh = share_of(z, a.V, p.per, static_cast<int>(at - r * p.S));
  const bool aligned = row_shift(out) == sh.shift;
  const float w = a.weight[r], c2 = exponent_scale(a.inv_temp);
  if (w == 0.0f) {
    const Vec zero = {{0u, 0u, 0u, 0u}};
    for (int g = sh.begin + tid; g < sh.end && tid < p.G; g += p.G)
      store_row_vec(out, first_element<T>(sh, g), a.V, aligned, zero);
    return;
  }
  const float m = a.stats_in[2 * r], s = a.stats_in[2 * r + 1];
  auto gradient = [&](float sq) {
    const Scale k = scale_of(m, c2);
    return make_gradient(a, k, sum_at_ref(s, m, k), w, sq);
  };
  if (tid >= p.G) {
    const int64_t e0 = first_element<T>(sh, sh.begin), e1 = first_element<T>(sh, sh.end);
    const EntryArrays n = entry_arrays(dyn, a.K, 0);
    EntryLoads loads;
    load_some(a, r, 0, loads);
    EntryValues<T> values;
    gather_some(a, r, 0, loads, e0, e1, values);
    const float sq = take_entries<T>(a, r, values, n, e0, e1);
    if (tid == p.G) sq_all = sq;
    block_sync();
    uint32_t shared;
    const uint32_t mine = first_entries(a, n, reinterpret_cast<int*>(dyn) + table_at(a.K), slots, e0, e1, shared);
    block_sync();
    store_sparse<T>(a, gradient(sq), n, mine, shared, out);
    return;
  }
  Vec v[kVecs];
  load_chunk<T, false>(v, z, a.V, sh, sh.begin, tid, p.G);
  block_sync();
  const Gradient g = gradient(sq_all);
  for (int c = sh.begin; c < sh.end; c += kVecs * p.G) {
    if (c > sh.begin) load_chunk<T, false>(v, z, a.V, sh, c, tid, p.G);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int at = c + i * p.G + tid;
      if (at >= sh.end) break;
#pragma unroll
      for (int q = 0; q < E / 2; ++q) set_pair<T>(v[i], q, dense_pair(g, vec_pair<T>(v[i], q)));
      store_row_vec(out, first_element<T>(sh, at), a.V, aligned, v[i]);
    }
  }
  block_sync();
}

cudaError_t launch_bwd(const KdArgs& a, int dtype, int64_t vectors, int sms, cudaStream_t stream) {
  Groups p = row_groups(a.T, vectors, sms);
  if (p.G < 64) p.G = 64;
  const int slots = table_slots(a.K);
  const size_t smem = static_cast<size_t>(table_at(a.K) + slots) * sizeof(int);  // 20 KB at most
  const int64_t total = a.T * p.S, most = int64_t(1) << 30;
  for (int64_t s0 = 0; s0 < total; s0 += most) {
    const unsigned blocks = static_cast<unsigned>(total - s0 < most ? total - s0 : most);
    if (dtype == 0) kd_bwd_kernel<float><<<blocks, p.G + 32, smem, stream>>>(a, s0, p, slots);
    else if (dtype == 1) kd_bwd_kernel<__half><<<blocks, p.G + 32, smem, stream>>>(a, s0, p, slots);
    else kd_bwd_kernel<__nv_bfloat16><<<blocks, p.G + 32, smem, stream>>>(a, s0, p, slots);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_distill(const KdArgs& a, bool forward, bool backward, int dtype, cudaStream_t stream) {
  const int sms = device_sm_count();
  const int64_t vectors = row_vectors(a.logits, a.V, a.ld, dtype == 0 ? 4 : 2);
  // Blocks of four computing warps, three an SM, take rows of up to 32 KB, one or two blocks a row, blocks of 16
  // longer ones: bf16 logits with 64 entries, loss and gradient, 8192 columns 126 us against 291 us with 16
  // warps (16384 rows), 16384 columns 122 against 157 us (8192 rows), 32768 columns (4096 rows, four blocks
  // a row) 121 us against 98. Without a gradient four warps are as fast for long rows too, once each of those
  // blocks has two rows; rows of more stages than add up in one sequence are left to 16.
  constexpr int64_t big = kShareStages * Shape<16>::kStageVecs, small = kShareStages * Shape<4>::kStageVecs;
  // the row's shares have to stay in the rings for the gradient: a longer row is read twice
  if (forward && backward && vectors <= 2 * small)
    return launch_fwd_any<true, 4, false>(a, dtype, split_row(a.T, vectors, small, sms), stream);
  if (forward && backward && vectors <= kMaxCluster * big)
    return launch_fwd_any<true, 16, false>(a, dtype, split_row(a.T, vectors, big, sms), stream);
  if (forward) {
    const Split all = split_row(a.T, vectors, vectors, sms);
    const bool four = vectors <= small || (a.T >= 6 * sms && vectors <= kFewStages * Shape<4>::kStageVecs);
    const cudaError_t e = four ? launch_fwd_any<false, 4, false>(a, dtype, all, stream)
                          : all.per > kFewStages * Shape<16>::kStageVecs
                              ? launch_fwd_any<false, 16, true>(a, dtype, all, stream)
                              : launch_fwd_any<false, 16, false>(a, dtype, all, stream);
    if (e != cudaSuccess || !backward) return e;
  }
  KdArgs b = a;
  if (forward) b.stats_in = a.stats;
  return launch_bwd(b, dtype, vectors, sms, stream);
}

}  // namespace swg
