// Backward of the norms between blocks (block_norm_fwd.cu has the formulas).
#include "block_norm.cuh"
#include "row_chunks.h"

namespace swg {
namespace {

using namespace bn;

// ---- backward: a row in the registers of a group of threads, one vector of each tensor a thread
// A group takes chunks of rows, chunk after chunk, and writes the chunk's two column sums. kShared: as in the forward.
// For few rows and rows that a cluster shares (257 x 1001 fp32 10 us with the sums); 16384 x 4096 bf16, 8 gates, 265 us
// against the ring's 144.
struct Sums4 {
  uint64_t come[2];
  float4 sums[2][kMaxCluster];
};
// three sums over the S blocks of a cluster, as ClusterSum's
struct ClusterSum3 {
  Sums4& slots;
  int S, rank, turn = 0;
  uint32_t parity = 0;
  Patience wait;
  __device__ __forceinline__ ClusterSum3(Sums4& s, int S_, const Stall& stall)
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
  __device__ __forceinline__ void operator()(float (&v)[3]) {
    uint64_t* come = &slots.come[turn];
    if (threadIdx.x == 0 && !wait.lost()) mbar_arrive_expect_tx(come, static_cast<uint32_t>(S) * sizeof(float4));
    if (static_cast<int>(threadIdx.x) < wait.open)
      send_f4(&slots.sums[turn][rank], come, threadIdx.x, make_float4(v[0], v[1], v[2], 0.0f));
    __syncwarp();
    wait.cluster(come, parity);
    v[0] = v[1] = v[2] = 0.0f;
    for (int i = 0; i < S; ++i) {
      const float4 o = slots.sums[turn][i];
      v[0] += o.x;
      v[1] += o.y;
      v[2] += o.z;
    }
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
struct NoSum3 {
  __device__ __forceinline__ NoSum3(Sums4&, int, const Stall&) {}
  __device__ __forceinline__ void operator()(float (&)[3]) {}
  __device__ __forceinline__ void silence() {}
  __device__ __forceinline__ void end(uint32_t*) {}
};

template <typename T, bool kRagged, bool kNarrow, bool kShared>
__global__ void __launch_bounds__(kMaxGroup)
    bn_bwd_kernel(const BnBwdArgs a, const BnChunks k, int G, int S, Stall stall, uint32_t* status) {
  __shared__ float smem[2 * 3 * 32];
  __shared__ Sums4 slots;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int E = kElems<T>, P = kPairs<T>;
  const int groups = kShared ? 1 : blockDim.x / G;
  const int t = kShared ? threadIdx.x + cluster_ctarank() * G : threadIdx.x % G;  // the vector
  const int64_t units = static_cast<int64_t>(kShared ? gridDim.x / S : gridDim.x) * groups;
  const int N = static_cast<int>(a.N);
  const float inv_n = 1.0f / static_cast<float>(a.N);
  const bool f32 = a.wdtype == 0, gated = a.gate != nullptr, gate32 = a.gdtype == 0, add = a.dh != nullptr;
  const bool row_gates = a.rows_per_gate == 1 && gated, dgate_rows = a.dgate != nullptr && a.rows_per_gate == 1;
  const uint32_t per_gate = static_cast<uint32_t>(a.rows_per_gate);
  const Rows<T> xu(a.u, a.ldu, a.M, a.N), xh(a.h, a.ldh, a.M, a.N), xy(a.dy, a.lddy, a.M, a.N), xd(a.dh, a.lddh, a.M, a.N);
  GroupSum<3, kNarrow> sum(smem, G);
  std::conditional_t<kShared, ClusterSum3, NoSum3> share(slots, S, stall);
  struct Row {
    Raw u, h, dy, dh;
    float ru, rh;
  };
  const int late = kNarrow ? (threadIdx.x & 31) / G : 0;  // the groups of a warp go through their loops together
  for (int64_t c = kShared ? blockIdx.x / S : static_cast<int64_t>(blockIdx.x) * groups + threadIdx.x / G;
       c < k.chunks + late; c += units) {
    const bool mine = !kNarrow || c < k.chunks;
    // the chunk's rows: count of them, `apart` rows from one to the next
    const ChunkRows<int64_t> rows = chunk_rows<true>(k, c);
    int count = mine && rows.first < rows.end ? static_cast<int>((rows.end - rows.first + k.apart - 1) / k.apart) : 0;
    const int64_t r0 = rows.first;
    const int shift = kRagged ? shift_of(static_cast<const T*>(a.du) + r0 * a.N) : 0;
    const int j = t * E - shift;
    const bool in_row = mine && j < N;
    const int own = count;
    if (kNarrow) count = __reduce_max_sync(0xffffffffu, count);
    float2 pre[P], post[P], ss[P], sp[P];
#pragma unroll
    for (int e = 0; e < P; ++e) ss[e] = sp[e] = pair(0.0f);
    if (in_row) {
      load_weights<T, kRagged>(a.gamma_pre, j, N, f32, 1.0f, pre);
      load_weights<T, kRagged>(a.gamma_post, j, N, f32, 1.0f, post);
    }
    auto load = [&](Row& w, int64_t r) {
      w.ru = a.post ? a.stats[2 * r] : 1.0f;
      w.rh = a.pre ? a.stats[2 * r + 1] : 0.0f;
      w.u = load_columns<T, kRagged>(xu, r, j, N);
      if (a.pre) {
        w.h = load_columns<T, kRagged>(xh, r, j, N);
        w.dy = load_columns<T, kRagged>(xy, r, j, N);
      }
      if (add) w.dh = load_columns<T, kRagged>(xd, r, j, N);
    };
    Row next = {};
    if (in_row && own > 0) load(next, r0);
    for (int i = 0; i < count; ++i) {
      const int64_t r = r0 + i * k.apart;
      if (kShared && static_cast<uint64_t>(r) >= static_cast<uint64_t>(stall.at)) share.silence();
      const bool on = in_row && i < own;
      Row w = next;
      if (on && i + 1 < own) load(next, r + k.apart);
      float2 q[P];
      if (on && gated) {
        const char* g = static_cast<const char*>(a.gate) +
                        static_cast<int64_t>(static_cast<uint32_t>(r) / per_gate) * a.N * (gate32 ? 4 : 2);
        load_weights<T, kRagged>(g, j, N, gate32, 1.0f, q);
      } else {
#pragma unroll
        for (int e = 0; e < P; ++e) q[e] = pair(1.0f);
      }
      if (kRagged) {
        clear_others<T>(w.u, j, N);
        clear_others<T>(w.h, j, N);
        clear_others<T>(w.dy, j, N);
        clear_others<T>(w.dh, j, N);
      }
      const float2 ru = pair(w.ru), rh = pair(w.rh);
      float2 s0 = pair(0.0f), s1 = s0, s2 = s0;
      if (on) {
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float2 uh = __fmul2_rn(get_pair<T>(w.u, e), ru), hh = __fmul2_rn(get_pair<T>(w.h, e), rh);
          const float2 dy = get_pair<T>(w.dy, e), g = __fmul2_rn(dy, pre[e]);
          const float2 qu = __fmul2_rn(__fmul2_rn(q[e], post[e]), uh);
          sp[e] = __ffma2_rn(dy, hh, sp[e]);
          s0 = __ffma2_rn(g, hh, s0);
          s1 = __ffma2_rn(qu, __ffma2_rn(rh, g, get_pair<T>(w.dh, e)), s1);
          s2 = __ffma2_rn(qu, hh, s2);
        }
      }
      float s[3] = {s0.x + s0.y, s1.x + s1.y, s2.x + s2.y};
      sum(s);
      share(s);
      const float m1 = s[0] * inv_n * w.rh;  // rstd(h) mean(a h^)
      const float2 c1 = pair(-m1), c2 = pair(a.post ? -fmaf(-m1, s[2], s[1]) * inv_n : 0.0f);
      if (!on) continue;
      Raw du, dres, dg;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float2 uh = __fmul2_rn(get_pair<T>(w.u, e), ru), hh = __fmul2_rn(get_pair<T>(w.h, e), rh);
        const float2 g = __fmul2_rn(get_pair<T>(w.dy, e), pre[e]);
        const float2 d = __ffma2_rn(rh, g, __ffma2_rn(c1, hh, get_pair<T>(w.dh, e)));
        const float2 du_hat = __fmul2_rn(d, uh);
        ss[e] = row_gates ? __ffma2_rn(du_hat, q[e], ss[e]) : __fadd2_rn(du_hat, ss[e]);
        if (dgate_rows && !gate32) set_pair<T>(dg, e, __fmul2_rn(du_hat, post[e]));
        set_pair<T>(dres, e, __fmul2_rn(pair(a.alpha), d));
        const float2 v = __ffma2_rn(uh, c2, __fmul2_rn(__fmul2_rn(q[e], post[e]), d));
        set_pair<T>(du, e, a.post ? __fmul2_rn(ru, v) : v);
        if (dgate_rows && gate32) {
          const float2 v = __fmul2_rn(du_hat, post[e]);
          float* to = static_cast<float*>(a.dgate) + r * a.N;
          const int at = j + 2 * e;
          if (at >= 0 && at < N) to[at] = v.x;
          if (at >= -1 && at + 1 < N) to[at + 1] = v.y;
        }
      }
      store_columns<T, kRagged>(static_cast<T*>(a.du) + r * a.N, j, N, du);
      if (a.dres != nullptr) store_columns<T, kRagged>(static_cast<T*>(a.dres) + r * a.N, j, N, dres);
      if (dgate_rows && !gate32) store_columns<T, kRagged>(static_cast<T*>(a.dgate) + r * a.N, j, N, dg);
    }
    if (a.part == nullptr || !in_row) continue;
    float* to = a.part + c * 2 * a.N + j;
#pragma unroll
    for (int e = 0; e < P; ++e) {
      if constexpr (!kRagged) {
        *reinterpret_cast<float2*>(to + 2 * e) = ss[e];
        *reinterpret_cast<float2*>(to + N + 2 * e) = sp[e];
      } else {
        const int at = j + 2 * e;
        if (at >= 0 && at < N) {
          to[2 * e] = ss[e].x;
          to[N + 2 * e] = sp[e].x;
        }
        if (at >= -1 && at + 1 < N) {
          to[2 * e + 1] = ss[e].y;
          to[N + 2 * e + 1] = sp[e].y;
        }
      }
    }
  }
  share.end(status);
}

// Backward over a ring, R vectors of a row a thread. HBM-bound: 16384 x 4096 bf16, 8 gates, 144 us with the sums (83% of
// the copy rate), 220000 x 512 248 us (80%), 8192 x 4096 fp32 140 us (85%). Forms of 16 bits that spill at 128 registers are
// slower: a gate for each row 222 us (71%; 104 bytes of stores a thread), ragged rows 231 us for 16384 x 4001 (50%; 72 bytes, with
// a gate for each row 144; in fp32, without spills, 8192 x 4001 173 to 185 us, 63 to 67%). The gate row is the chunk's own (kRowGate: one more
// tensor in the ring), so that its columns and gamma_post's are one factor in registers.
constexpr int kBwdBlock = 256, kBwdBlocks = 2;  // threads of a block, at most, and such blocks an SM
template <typename T, int R, bool kShared, bool kRowGate, bool kFull, bool kRagged>
__global__ void __launch_bounds__(kBwdBlock, kBwdBlocks)
    bn_bwd_ring_kernel(const BnBwdArgs a, const BnChunks k, const RingPlan plan, int G, int S, Stall stall,
                       uint32_t* status) {
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ uint64_t bars[8 * kMaxStages];
  __shared__ float smem[8 * 64];
  __shared__ Sums4 slots;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int E = kElems<T>, P = kPairs<T>, kTensors = kRowGate ? 5 : 4;
  const int groups = kShared ? 1 : blockDim.x / G, group = kShared ? 0 : threadIdx.x / G;
  const int rank = kShared ? static_cast<int>(cluster_ctarank()) : 0, in = kShared ? threadIdx.x : threadIdx.x % G;
  const uint32_t units = (kShared ? gridDim.x / S : gridDim.x) * groups;
  const uint32_t unit = kShared ? blockIdx.x / S : blockIdx.x * groups + group;
  const int N = static_cast<int>(a.N), n0 = rank * R * G;
  const bool first = in == 0;
  const float inv_n = 1.0f / static_cast<float>(a.N);
  const bool post_norm = kFull || a.post, pre_norm = kFull || a.pre, add = kFull || a.dh != nullptr;
  const bool f32 = a.wdtype == 0, gate32 = a.gdtype == 0, dgate_rows = kRowGate && a.dgate != nullptr;
  RowRing<kTensors, kRagged> ring(dyn, bars, plan, group, stall);
  if (first) {
    ring.init();
    fence_mbar_init();
  }
  __syncthreads();
  WarpRows sums(smem, G);
  std::conditional_t<kShared, ClusterSum3, NoSum3> share(slots, S, stall);
  const int64_t stop_at = kShared ? -1 : stall.at;
  // the rows of the group's chunks in turn: of chunk c r, r + apart, ... below end
  const uint32_t chunks = static_cast<uint32_t>(k.chunks);
  const uint32_t apart = kRagged ? static_cast<uint32_t>(k.apart) : 1u;
  struct Walk {  // 32 bits hold them
    uint32_t c, r, end;
    int shift, n, mine;  // elements from the 16-byte boundary before a row, its vectors, and this block's
  };
  auto enter = [&](Walk& w) {
    const ChunkRows<uint32_t> rows = chunk_rows<kRagged>(k, w.c);
    w.r = rows.first;
    w.end = rows.end;
    if constexpr (kRagged) {
      w.shift = shift_of(static_cast<const T*>(a.du) + static_cast<int64_t>(w.r) * a.N);
      w.n = (N + w.shift + E - 1) / E;
      w.mine = min(R * G, w.n - n0);
    }
  };
  const int whole = min(R * G, N / E - n0);  // the block's vectors of a whole row
  auto mine_of = [&](const Walk& w) { return kRagged ? w.mine : whole; };
  auto shift_in = [&](const Walk& w) { return kRagged ? w.shift : 0; };
  // a walk behind its chunk's last row goes on to the next chunk that has rows (a phase of ragged rows may have none)
  auto settle = [&](Walk& w) {
    while (w.c < chunks && w.r >= w.end) {
      w.c += units;
      if (w.c < chunks) enter(w);
    }
  };
  Walk ahead{unit, 0, 0, 0, 0, 0};
  if (ahead.c < chunks) {
    enter(ahead);
    if (kRagged) settle(ahead);
  }
  auto issue = [&]() {
    if (ahead.c >= chunks) return;
    const int64_t r = ahead.r;
    const void* from[kTensors];
    uint32_t bytes[kTensors];
    const Span span = kRagged ? span_of(r, a.M, ahead.n, n0, ahead.mine, ahead.shift, ahead.n * E - ahead.shift - N)
                              : Span{0, whole};
    const int j0 = (n0 + span.first) * E - shift_in(ahead);  // the first column that is copied
    from[0] = static_cast<const T*>(a.u) + r * a.ldu + j0;
    from[1] = pre_norm ? static_cast<const T*>(a.h) + r * a.ldh + j0 : nullptr;
    from[2] = pre_norm ? static_cast<const T*>(a.dy) + r * a.lddy + j0 : nullptr;
    from[3] = add ? static_cast<const T*>(a.dh) + r * a.lddh + j0 : nullptr;
#pragma unroll
    for (int i = 0; i < 4; ++i) bytes[i] = static_cast<uint32_t>(span.count) * 16u;
    if constexpr (kRowGate) {
      const int64_t es = gate32 ? 4 : sizeof(T);
      from[4] = static_cast<const char*>(a.gate) + (r * a.N + j0) * es;
      bytes[4] = static_cast<uint32_t>(span.count) * static_cast<uint32_t>(E * es);
    }
    ring.issue(from, bytes, R * G * 16, stop_at, span.first * 16);
    ahead.r += apart;
    settle(ahead);
  };
  if (first)
    for (int i = 0; i < ring.stages; ++i) issue();
  Walk w{unit, 0, 0, 0, 0, 0};
  if (w.c < chunks) enter(w);
  auto column = [&](int i) { return (n0 + in + i * G) * E - shift_in(w); };
  float2 pre[R][P], post[R][P];  // gamma_pre; gamma_post, without kRowGate times the gate
  if (!kRagged) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (in + i * G < mine_of(w)) load_weights<T, false>(a.gamma_pre, column(i), N, f32, 1.0f, pre[i]);
  }
  bool refill = false;
  struct Vectors {  // a thread's vector of each tensor, from the stage
    Raw u, h, dy, dh;
  };
  const Rows<T> rows_u(a.u, a.ldu, a.M, a.N), rows_h(a.h, a.ldh, a.M, a.N), rows_y(a.dy, a.lddy, a.M, a.N);
  const Rows<T> rows_d(a.dh, a.lddh, a.M, a.N), rows_g(a.gate, a.N, a.M, a.N);
  auto place_of = [&](unsigned char* stage, int tensor, int i) { return stage + (tensor * R * G + in + i * G) * 16; };
  auto vectors = [&](unsigned char* stage, int i) {
    Vectors v = {};
    v.u = ld_stage(place_of(stage, 0, i));
    if (pre_norm) {
      v.h = ld_stage(place_of(stage, 1, i));
      v.dy = ld_stage(place_of(stage, 2, i));
    }
    if (add) v.dh = ld_stage(place_of(stage, 3, i));
    return v;
  };
  for (; w.c < chunks; w.c += units) {
    enter(w);
    bool edge[R];  // vectors that reach beyond the row
#pragma unroll
    for (int i = 0; i < R; ++i) edge[i] = kRagged && in + i * G < mine_of(w) && (column(i) < 0 || column(i) + E > N);
    float2 ss[R][P], sp[R][P];
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int e = 0; e < P; ++e) ss[i][e] = sp[i][e] = pair(0.0f);
      if (in + i * G >= mine_of(w)) continue;
      if (kRagged) load_weights<T, kRagged>(a.gamma_pre, column(i), N, f32, 1.0f, pre[i]);
      load_weights<T, kRagged>(a.gamma_post, column(i), N, f32, 1.0f, post[i]);
      if (!kRowGate && a.gate != nullptr) {
        float2 g[P];
        // the chunk's segment: a chunk without rows has its first row elsewhere, or nowhere
        const int64_t row = w.c / static_cast<uint32_t>(k.per_segment);
        load_weights<T, kRagged>(static_cast<const char*>(a.gate) + row * a.N * (gate32 ? 4 : sizeof(T)), column(i), N,
                                 gate32, 1.0f, g);
#pragma unroll
        for (int e = 0; e < P; ++e) post[i][e] = __fmul2_rn(g[e], post[i][e]);
      }
    }
    auto rstds = [&](uint32_t r) {  // 4-byte aligned
      const float* p = a.stats + 2 * static_cast<int64_t>(r);
      return make_float2(p[0], p[1]);
    };
    float2 stats = make_float2(0.0f, 0.0f);
    if (!kRagged || w.r < w.end) stats = rstds(w.r);
    int64_t at = static_cast<int64_t>(w.r) * a.N;  // the row's
    for (uint32_t r = w.r; r < w.end; r += apart, at += static_cast<int64_t>(apart) * a.N) {
      if (kShared && static_cast<uint64_t>(r) >= static_cast<uint64_t>(stall.at)) share.silence();
      const float fu = post_norm ? stats.x : 1.0f, fh = pre_norm ? stats.y : 0.0f;
      if (r + apart < w.end) stats = rstds(r + apart);
      unsigned char* stage = ring.next();
      if constexpr (kRagged) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          if (!edge[i]) continue;
          const int j = column(i);
          mend_edge(place_of(stage, 0, i), rows_u, r, a.M, j, N);
          if (pre_norm) {
            mend_edge(place_of(stage, 1, i), rows_h, r, a.M, j, N);
            mend_edge(place_of(stage, 2, i), rows_y, r, a.M, j, N);
          }
          if (add) mend_edge(place_of(stage, 3, i), rows_d, r, a.M, j, N);
          if (kRowGate) mend_edge(place_of(stage, 4, i), rows_g, r, a.M, j, N);
        }
      }
      const float2 rh = pair(fh);
      // sums of dy gamma_pre h, of q u (dh + rstd(h) dy gamma_pre) and of q u h: the rows' factors come behind them
      float2 s0 = pair(0.0f), s1 = s0, s2 = s0;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (in + i * G >= mine_of(w)) continue;
        const Vectors v = vectors(stage, i);
        float2 q[P];
        if constexpr (kRowGate) stage_pairs<T>(stage + 4 * R * G * 16, in + i * G, !kRagged && gate32, q);
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float2 h = get_pair<T>(v.h, e), dy = get_pair<T>(v.dy, e), x = __fmul2_rn(dy, h);
          float2 qu = __fmul2_rn(post[i][e], get_pair<T>(v.u, e));
          if constexpr (kRowGate) qu = __fmul2_rn(q[e], qu);
          sp[i][e] = __ffma2_rn(x, rh, sp[i][e]);
          s0 = __ffma2_rn(x, pre[i][e], s0);
          s1 = __ffma2_rn(qu, __ffma2_rn(__fmul2_rn(rh, pre[i][e]), dy, get_pair<T>(v.dh, e)), s1);
          s2 = __ffma2_rn(qu, h, s2);
        }
      }
      float s[3] = {s0.x + s0.y, s1.x + s1.y, s2.x + s2.y};
      sums.three(s);
      if (first && refill) issue();  // the group has read the row before
      refill = true;
      share(s);
      const float m1 = s[0] * fh * inv_n * fh;  // rstd(h) mean(a h^)
      // d = dh + rstd(h) a - m1 h^;  du = rstd(u) q d - u c2
      const float2 c1 = pair(-m1 * fh), ru = pair(fu);
      const float2 c2 = pair(post_norm ? -fmaf(-m1 * fh, s[2], s[1]) * fu * inv_n : 0.0f);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (in + i * G >= mine_of(w)) continue;
        Vectors x = vectors(stage, i);
        float2 q[P];
        if constexpr (kRowGate) stage_pairs<T>(stage + 4 * R * G * 16, in + i * G, !kRagged && gate32, q);
        Raw dg;
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float2 d = __ffma2_rn(__fmul2_rn(rh, pre[i][e]), get_pair<T>(x.dy, e),
                                      __ffma2_rn(c1, get_pair<T>(x.h, e), get_pair<T>(x.dh, e)));
          const float2 uh = __fmul2_rn(get_pair<T>(x.u, e), ru);
          float2 qd = __fmul2_rn(post[i][e], d);
          if constexpr (kRowGate) {
            const float2 du_hat = __fmul2_rn(d, uh);
            ss[i][e] = __ffma2_rn(du_hat, q[e], ss[i][e]);
            qd = __fmul2_rn(q[e], qd);
            const float2 v = __fmul2_rn(du_hat, post[i][e]);
            if (!kRagged && sizeof(T) == 2 && gate32 && dgate_rows) *reinterpret_cast<float2*>(static_cast<float*>(a.dgate) + at + column(i) + 2 * e) = v;
            else set_pair<T>(dg, e, v);
          } else {
            ss[i][e] = __ffma2_rn(d, uh, ss[i][e]);
          }
          set_pair<T>(x.dh, e, __fmul2_rn(pair(a.alpha), d));
          const float2 v = __ffma2_rn(uh, c2, qd);
          set_pair<T>(x.u, e, post_norm ? __fmul2_rn(ru, v) : v);
        }
        store_vector<T, kRagged>(static_cast<T*>(a.du) + at, column(i), N, edge[i], x.u);
        if (kFull || a.dres != nullptr) store_vector<T, kRagged>(static_cast<T*>(a.dres) + at, column(i), N, edge[i], x.dh);
        if (dgate_rows && (sizeof(T) == 4 || !gate32))
          store_vector<T, kRagged>(static_cast<T*>(a.dgate) + at, column(i), N, edge[i], dg);
      }
    }
    if (a.part == nullptr) continue;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (in + i * G >= mine_of(w)) continue;
      float* to = a.part + static_cast<int64_t>(w.c) * 2 * a.N + column(i);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        if constexpr (!kRagged) {
          *reinterpret_cast<float2*>(to + 2 * e) = ss[i][e];
          *reinterpret_cast<float2*>(to + N + 2 * e) = sp[i][e];
        } else {
          const int j = column(i) + 2 * e;
          if (j >= 0 && j < N) {
            to[2 * e] = ss[i][e].x;
            to[N + 2 * e] = sp[i][e].x;
          }
          if (j >= -1 && j + 1 < N) {
            to[2 * e + 1] = ss[i][e].y;
            to[N + 2 * e + 1] = sp[i][e].y;
          }
        }
      }
    }
  }
  if (first) ring.end(status);
  else if (ring.wait.lost() && status != nullptr) atomicOr(status, kStatusTimeout);
  share.end(status);
}

// What belongs to element j of row r in the backward, for rows of any length. u^ is u where there is no norm after the block.
template <typename T>
struct Element {
  float uh, hh, a, dh, q, gate, post;
  __device__ __forceinline__ Element(const BnBwdArgs& p, int64_t r, int64_t j, float ru, float rh) {
    uh = to_f(static_cast<const T*>(p.u)[r * p.ldu + j]) * (p.post ? ru : 1.0f);
    hh = p.pre ? to_f(static_cast<const T*>(p.h)[r * p.ldh + j]) * rh : 0.0f;
    a = p.pre ? to_f(static_cast<const T*>(p.dy)[r * p.lddy + j]) : 0.0f;  // dy; times gamma_pre below
    dh = p.dh != nullptr ? to_f(static_cast<const T*>(p.dh)[r * p.lddh + j]) : 0.0f;
    post = p.post && p.gamma_post != nullptr ? load_any(p.gamma_post, j, p.wdtype) : 1.0f;
    gate = p.gate != nullptr ? load_any(p.gate, r / p.rows_per_gate * p.N + j, p.gdtype) : 1.0f;
    q = gate * post;
  }
};
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) bn_dx_long_kernel(const BnBwdArgs a) {
  __shared__ float buf[32];
  const float inv_n = 1.0f / static_cast<float>(a.N);
  const bool rows_gate = a.dgate != nullptr && a.rows_per_gate == 1;
  for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
    const float ru = a.post ? a.stats[2 * r] : 0.0f, rh = a.pre ? a.stats[2 * r + 1] : 0.0f;
    auto pre = [&](int64_t j) { return a.pre && a.gamma_pre != nullptr ? load_any(a.gamma_pre, j, a.wdtype) : 1.0f; };
    float s[3];
    long_sums(a.N, s, [&](float (&p)[3], int64_t j) {
      const Element<T> e(a, r, j, ru, rh);
      const float g = e.a * pre(j), qu = e.q * e.uh;
      p[0] = fmaf(g, e.hh, p[0]);
      p[1] = fmaf(qu, fmaf(rh, g, e.dh), p[1]);
      p[2] = fmaf(qu, e.hh, p[2]);
    });
    const float c1 = block_sum(s[0], buf) * inv_n * rh, s1 = block_sum(s[1], buf), s2 = block_sum(s[2], buf);
    const float c2 = a.post ? fmaf(-c1, s2, s1) * inv_n : 0.0f;
    for (int64_t j = threadIdx.x; j < a.N; j += blockDim.x) {
      const Element<T> e(a, r, j, ru, rh);
      const float d = fmaf(rh, e.a * pre(j), fmaf(-c1, e.hh, e.dh));
      if (a.dres != nullptr) static_cast<T*>(a.dres)[r * a.N + j] = from_f<T>(a.alpha * d);
      const float du = a.post ? ru * fmaf(-e.uh, c2, e.q * d) : e.q * d;
      static_cast<T*>(a.du)[r * a.N + j] = from_f<T>(du);
      if (rows_gate) store_any(a.dgate, r * a.N + j, a.gdtype, d * e.uh * e.post);
    }
    if (threadIdx.x == 0 && a.mean != nullptr) a.mean[r] = c1;
  }
}

// One chunk's column sums, for rows of any length: part[chunk][0][j] of D u^ (times the gate where it has a row for
// each row), part[chunk][1][j] of dy h^.
constexpr int kColThreads = 128;
template <typename T>
__global__ void __launch_bounds__(kColThreads) bn_param_long_kernel(const BnBwdArgs a, const BnChunks k, int64_t first) {
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kColThreads + threadIdx.x, chunk = first + blockIdx.y;
  if (j >= a.N) return;
  const ChunkRows<int64_t> rows = chunk_rows<false>(k, chunk);  // apart is 1
  const float pre = a.pre && a.gamma_pre != nullptr ? load_any(a.gamma_pre, j, a.wdtype) : 1.0f;
  float s = 0.0f, p = 0.0f;
  for (int64_t r = rows.first; r < rows.end; ++r) {
    const float ru = a.post ? a.stats[2 * r] : 0.0f, rh = a.pre ? a.stats[2 * r + 1] : 0.0f;
    const Element<T> e(a, r, j, ru, rh);
    const float d = fmaf(rh, e.a * pre, fmaf(-a.mean[r], e.hh, e.dh));
    s = fmaf(d * e.uh, a.rows_per_gate == 1 ? e.gate : 1.0f, s);
    p = fmaf(e.a, e.hh, p);
  }
  float* to = a.part + chunk * 2 * a.N;
  to[j] = s;
  to[a.N + j] = p;
}

// The parameters' gradients from the chunks' sums, 128 columns a block (four a lane), sixteen warps. The first
// `sum_blocks` blocks sum all chunks, for dgamma_post (each times its gate row) and dgamma_pre: a cluster of Q blocks
// takes 128 columns, its 16 Q warps the chunks in turn. In the others `slices` warps sum the chunks of a gate row. A
// lane adds 64 terms in sequence, then these parts, then the warps' and the blocks' sums: a fixed order. A programmatic dependent of the kernel before it, whose
// writes are visible after griddepcontrol.wait. Its time is that of a few loads in turn: 304 chunks of 4096 columns,
// eight gate rows 6 us; by blocks of 1024 threads for 32 columns and each gate row it took 36.
constexpr int kReduceCols = 128, kReduceWarps = 16;
__global__ void __launch_bounds__(32 * kReduceWarps)
    bn_reduce_kernel(const BnBwdArgs a, const BnChunks k, int Q, int64_t sum_blocks, int slices, int64_t first_gate) {
  __shared__ float acc[kReduceWarps][kReduceCols];
  __shared__ float all[kReduceCols];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the warp's sums of the chunks begin, begin + step, ... before end, at columns j0 + lane + 32 e below most; eight
  // chunks' loads at once (anything behind the last column)
  auto sum = [&](int64_t begin, int64_t end, int64_t step, int64_t j0, int64_t most, bool weigh) {
    constexpr int kDeep = 8;
    const float* part[4];
    int64_t col[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      col[e] = min(j0 + lane + 32 * e, most - 1);
      part[e] = a.part + col[e];
    }
    const uint32_t per_segment = static_cast<uint32_t>(k.per_segment);
    // the chunk's gate at the lane's columns (1 for those of dgamma_pre): bits, and as values
    auto gate_bits = [&](int64_t n, int e) -> uint32_t {
      const int64_t at = static_cast<uint32_t>(n) / per_segment * a.N + min(col[e], a.N - 1);
      return a.gdtype == 0 ? static_cast<const uint32_t*>(a.gate)[at] : static_cast<const uint16_t*>(a.gate)[at];
    };
    auto gate_of = [&](uint32_t bits, int e) {
      if (col[e] >= a.N) return 1.0f;
      const unsigned short h = static_cast<unsigned short>(bits);
      return a.gdtype == 0   ? __uint_as_float(bits)
             : a.gdtype == 1 ? __half2float(__ushort_as_half(h))
                             : __uint_as_float(bits << 16);
    };
    float t[4] = {}, s[4] = {};
    int64_t n = begin;
    for (int count = 1; n + (kDeep - 1) * step < end; n += kDeep * step, ++count) {
      float v[kDeep][4];
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[u][e] = part[e][(n + u * step) * 2 * a.N];
      }
      if (weigh) {
        uint32_t g[kDeep][4];
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
#pragma unroll
          for (int e = 0; e < 4; ++e) g[u][e] = gate_bits(n + u * step, e);
        }
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[u][e] *= gate_of(g[u][e], e);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s[e] += ((v[0][e] + v[1][e]) + (v[2][e] + v[3][e])) + ((v[4][e] + v[5][e]) + (v[6][e] + v[7][e]));
      if (count % 8 == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          t[e] += s[e];
          s[e] = 0.0f;
        }
      }
    }
    float v[kDeep][4];
    uint32_t g[kDeep][4] = {};
#pragma unroll
    for (int u = 0; u < kDeep - 1; ++u) {
      if (n + u * step >= end) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[u][e] = part[e][(n + u * step) * 2 * a.N];
        if (weigh) g[u][e] = gate_bits(n + u * step, e);
      }
    }
#pragma unroll
    for (int u = 0; u < kDeep - 1; ++u) {
      if (n + u * step >= end) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += weigh ? v[u][e] * gate_of(g[u][e], e) : v[u][e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[warp][lane + 32 * e] = t[e] + s[e];
    __syncthreads();
  };
  if (blockIdx.x < sum_blocks) {
    const int rank = static_cast<int>(blockIdx.x % Q);
    const int64_t j0 = static_cast<int64_t>(blockIdx.x / Q) * kReduceCols;
    sum(rank * kReduceWarps + warp, k.chunks, static_cast<int64_t>(Q) * kReduceWarps, j0, 2 * a.N,
        a.gate != nullptr && a.rows_per_gate > 1 && j0 < a.N);
    float t = 0.0f;
    if (threadIdx.x < kReduceCols) {
#pragma unroll
      for (int w = 0; w < kReduceWarps; ++w) t += acc[w][threadIdx.x];
      all[threadIdx.x] = t;
    }
    if (Q > 1) {
      cluster_sync();
      if (rank == 0 && threadIdx.x < kReduceCols)
        for (int i = 1; i < Q; ++i) t += ld_cluster_f32(&all[threadIdx.x], i);
      cluster_sync();  // no block leaves before its sums have been read
    }
    const int64_t j = j0 + threadIdx.x;
    if (rank != 0 || threadIdx.x >= kReduceCols || j >= 2 * a.N) return;
    if (j < a.N) {
      if (a.dgamma_post != nullptr) store_any(a.dgamma_post, j, a.wdtype, t);
    } else if (a.dgamma_pre != nullptr) {
      store_any(a.dgamma_pre, j - a.N, a.wdtype, t);
    }
    return;
  }
  const int64_t id = blockIdx.x - sum_blocks, blocks = (a.N + kReduceCols - 1) / kReduceCols;
  const int rows = kReduceWarps / slices;  // gate rows of a block
  const int64_t g0 = first_gate + id / blocks * rows, gates = a.M / a.rows_per_gate, j0 = id % blocks * kReduceCols;
  const int64_t g = g0 + warp / slices, begin = g * k.per_segment;
  sum(begin + warp % slices, g < gates ? begin + k.per_segment : begin, slices, j0, a.N, false);
  for (int i = threadIdx.x; i < rows * kReduceCols; i += blockDim.x) {
    const int row = i / kReduceCols, c = i % kReduceCols;
    const int64_t j = j0 + c;
    if (g0 + row >= gates || j >= a.N) continue;
    float t = 0.0f;
    for (int w = 0; w < slices; ++w) t += acc[row * slices + w][c];
    const float post = a.post && a.gamma_post != nullptr ? load_any(a.gamma_post, j, a.wdtype) : 1.0f;
    store_any(a.dgate, (g0 + row) * a.N + j, a.gdtype, t * post);
  }
}

// ---- host
// The groups of threads that take chunks: those of one block of 512 threads (or a cluster of blocks) on each of 152
// SMs, for rows of n vectors. A plan that does not depend on the device, so that the workspace's size does not.
int64_t units_of(int64_t n) {
  constexpr int64_t kSms = 152;
  if (n <= kMaxGroup) return kSms * (kMaxGroup / group_threads(n, 1));
  return std::max<int64_t>(1, kSms / ((n + kMaxGroup - 1) / kMaxGroup));
}
constexpr int64_t kLongUnits = 304;  // for rows of any length
// the same for whole rows in rings: groups of two vectors a thread, 512 threads an SM
int64_t ring_units(int64_t n) {
  constexpr int64_t kSms = 152;
  if (n <= 2 * kBwdBlock) return kSms * (kBwdBlocks * kBwdBlock / group_threads(n, 2));
  const Shared s = share_row(n, 2);
  return std::max<int64_t>(1, kSms * (kBwdBlocks * kBwdBlock / s.G) / s.S);
}

cudaError_t launch_reduce(const BnBwdArgs& a, const BnChunks& k, cudaStream_t stream) {
  const bool sums = a.dgamma_post != nullptr || a.dgamma_pre != nullptr;
  const int64_t gates = a.dgate != nullptr && a.rows_per_gate > 1 ? a.M / a.rows_per_gate : 0;
  int Q = 1;  // eight chunks a warp or more
  while (Q < kMaxCluster && k.chunks >= 2 * Q * kReduceWarps * 8) Q *= 2;
  int slices = 1;
  while (slices < kReduceWarps && k.per_segment >= 2 * slices * 4) slices *= 2;
  const int64_t rows = kReduceWarps / slices, columns = (a.N + kReduceCols - 1) / kReduceCols;
  const int64_t sum_blocks = sums ? (2 * a.N + kReduceCols - 1) / kReduceCols * Q : 0;
  const int64_t most = std::max<int64_t>(1, (int64_t(1) << 30) / columns);  // groups of gate rows of a launch
  int64_t from = 0;
  const int64_t all = (gates + rows - 1) / rows;
  do {
    const int64_t n = std::min(most, all - from);
    const bool first = from == 0;
    const int64_t lead = first ? sum_blocks : 0, blocks = (lead + n * columns + Q - 1) / Q * Q;
    if (blocks == 0) break;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(32 * kReduceWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(Q);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = first ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, bn_reduce_kernel, a, k, Q, lead, slices, from * rows);
    if (e != cudaSuccess) return e;
    from += n;
  } while (from < all);
  return cudaSuccess;
}

template <typename T>
cudaError_t bwd_long(const BnBwdArgs& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.M, 65536));
  bn_dx_long_kernel<T><<<grid, kMaxThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.part == nullptr) return e;
  const BnChunks k = chunks_of(a.M, a.rows_per_gate, kLongUnits, 1);
  for (int64_t c = 0; c < k.chunks; c += 65535) {
    const dim3 g(static_cast<unsigned>((a.N + kColThreads - 1) / kColThreads),
                 static_cast<unsigned>(std::min<int64_t>(65535, k.chunks - c)));
    bn_param_long_kernel<T><<<g, kColThreads, 0, stream>>>(a, k, c);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return launch_reduce(a, k, stream);
}

template <typename T, bool kRagged, bool kNarrow>
cudaError_t bwd_groups(const BnBwdArgs& a, int64_t n, cudaStream_t stream) {
  const int G = group_threads(n, 1);
  const BnChunks k = chunks_of(a.M, a.rows_per_gate, units_of(n), kRagged ? rows_apart<T>(a.N) : 1);
  // one block an SM, or smaller ones for few rows
  int groups = kMaxGroup / G;
  while (groups > 1 && groups * G > 32 && (k.chunks + groups - 1) / groups < device_sm_count()) groups = (groups + 1) / 2;
  const int block = groups * G;
  int64_t blocks;
  {
    static std::mutex mu;
    static FitCache cache;
    std::lock_guard<std::mutex> lk(mu);
    const cudaError_t e = blocks_that_fit(bn_bwd_kernel<T, kRagged, kNarrow, false>, cache, block, 0, blocks);
    if (e != cudaSuccess) return e;
  }
  blocks = std::min(blocks, (k.chunks + groups - 1) / groups);
  bn_bwd_kernel<T, kRagged, kNarrow, false>
      <<<static_cast<unsigned>(blocks), block, 0, stream>>>(a, k, G, 1, Stall(), nullptr);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess || a.part == nullptr ? e : launch_reduce(a, k, stream);
}
template <typename T, bool kRagged>
cudaError_t bwd_shared(const BnBwdArgs& a, int64_t n, cudaStream_t stream) {
  const auto kernel = bn_bwd_kernel<T, kRagged, false, true>;
  const int S = static_cast<int>((n + kMaxGroup - 1) / kMaxGroup);
  const int G = static_cast<int>((n + 32 * S - 1) / (32 * S)) * 32;
  const BnChunks k = chunks_of(a.M, a.rows_per_gate, units_of(n), kRagged ? rows_apart<T>(a.N) : 1);
  {
    static std::mutex mu;
    static StreamCache cache;
    std::lock_guard<std::mutex> lk(mu);
    cudaError_t e = clusters_that_fit(kernel, cache, G, 0, S);
    if (e != cudaSuccess) return e;
    if (cache.clusters < 1) return bwd_long<T>(a, stream);
    ClusterLaunch l(G, 0, S, std::min<int64_t>(cache.clusters, k.chunks), stream);
    e = cudaLaunchKernelEx(&l.cfg, kernel, a, k, G, S, take_stall(kInjectBlockNormBwd), status_word_ptr());
    if (e != cudaSuccess) return e;
  }
  return a.part == nullptr ? cudaSuccess : launch_reduce(a, k, stream);
}
template <typename T, bool kRowGate, bool kFull, bool kRagged>
cudaError_t bwd_ring_one(const BnBwdArgs& a, const BnChunks& k, int64_t n, cudaStream_t stream) {
  const auto kernel = bn_bwd_ring_kernel<T, 2, false, kRowGate, kFull, kRagged>;
  const int G = group_threads(n, 2), groups = kBwdBlock / G, block = groups * G;
  const RingPlan p = ring_plan((4 + (kRowGate ? gate_slots<T>(a.gdtype) : 0)) * 2 * G * 16,
                               std::max(kBwdBlocks, kBwdBlocks * kBwdBlock / block), groups);
  const size_t smem = static_cast<size_t>(groups) * p.group_bytes;
  int64_t blocks;
  {
    static std::mutex mu;
    static FitCache cache;
    std::lock_guard<std::mutex> lk(mu);
    const cudaError_t e = blocks_that_fit(kernel, cache, block, smem, blocks);
    if (e != cudaSuccess) return e;
  }
  blocks = std::min(blocks, (k.chunks + groups - 1) / groups);
  kernel<<<static_cast<unsigned>(blocks), block, smem, stream>>>(a, k, p, G, 1, take_stall(kInjectBlockNormBwd),
                                                                status_word_ptr());
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess || a.part == nullptr ? e : launch_reduce(a, k, stream);
}
template <typename T, bool kRowGate, bool kFull, bool kRagged>
cudaError_t bwd_ring_shared(const BnBwdArgs& a, const BnChunks& k, int64_t n, cudaStream_t stream) {
  const auto kernel = bn_bwd_ring_kernel<T, 2, true, kRowGate, kFull, kRagged>;
  const Shared s = share_row(n, 2);
  const RingPlan p = ring_plan((4 + (kRowGate ? gate_slots<T>(a.gdtype) : 0)) * 2 * s.G * 16,
                               std::max(kBwdBlocks, kBwdBlocks * kBwdBlock / s.G), 1);
  {
    static std::mutex mu;
    static StreamCache cache;
    std::lock_guard<std::mutex> lk(mu);
    cudaError_t e = clusters_that_fit(kernel, cache, s.G, p.group_bytes, s.S);
    if (e != cudaSuccess) return e;
    if (cache.clusters < 1) return bwd_long<T>(a, stream);
    ClusterLaunch l(s.G, p.group_bytes, s.S, std::min<int64_t>(cache.clusters, k.chunks), stream);
    e = cudaLaunchKernelEx(&l.cfg, kernel, a, k, p, s.G, s.S, take_stall(kInjectBlockNormBwd), status_word_ptr());
    if (e != cudaSuccess) return e;
  }
  return a.part == nullptr ? cudaSuccess : launch_reduce(a, k, stream);
}
template <typename T, bool kRowGate, bool kFull, bool kRagged>
cudaError_t bwd_ring(const BnBwdArgs& a, const BnChunks& k, int64_t n, cudaStream_t stream) {
  return n <= 2 * kBwdBlock ? bwd_ring_one<T, kRowGate, kFull, kRagged>(a, k, n, stream)
                            : bwd_ring_shared<T, kRowGate, kFull, kRagged>(a, k, n, stream);
}
template <typename T, bool kRagged>
cudaError_t bwd_any(const BnBwdArgs& a, cudaStream_t stream) {
  const int64_t n = (a.N + (kRagged ? 2 * kElems<T> - 2 : 0)) / kElems<T>;
  const bool row_gate = a.gate != nullptr && a.rows_per_gate == 1;
  const bool ring = !kRagged || (same_offsets(a.M, a.N, sizeof(T), a.du,
                                              {a.u, a.h, a.dy, a.dh, a.dres, row_gate ? a.gate : nullptr,
                                               row_gate ? a.dgate : nullptr},
                                              {a.ldu, a.pre ? a.ldh : a.N, a.pre ? a.lddy : a.N,
                                               a.dh != nullptr ? a.lddh : a.N}) &&
                                 (!row_gate || sizeof(T) == 4 || a.gdtype != 0));
  const int64_t units = ring_units(n);
  if (ring && n > 32 && n <= 2 * kMaxCluster * kBwdBlock && a.M >= kRingRows * units) {
    const BnChunks k = chunks_of(a.M, a.rows_per_gate, units, kRagged ? rows_apart<T>(a.N) : 1);
    const bool full = a.post && a.pre && a.dh != nullptr && a.dres != nullptr;
    if (row_gate)
      return full ? bwd_ring<T, true, true, kRagged>(a, k, n, stream) : bwd_ring<T, true, false, kRagged>(a, k, n, stream);
    return full ? bwd_ring<T, false, true, kRagged>(a, k, n, stream) : bwd_ring<T, false, false, kRagged>(a, k, n, stream);
  }
  if (n <= 16) return bwd_groups<T, kRagged, true>(a, n, stream);
  if (n <= kMaxGroup) return bwd_groups<T, kRagged, false>(a, n, stream);
  if (n <= kMaxCluster * kMaxGroup) return bwd_shared<T, kRagged>(a, n, stream);
  return bwd_long<T>(a, stream);
}
template <typename T>
cudaError_t bwd_type(const BnBwdArgs& a, cudaStream_t stream) {
  // dgate with a row for each row goes out as vectors, whatever its type (a shared one element by element)
  const bool whole = whole_vectors(a.N, sizeof(T),
                                   {a.dy, a.dh, a.u, a.h, a.du, a.dres, a.rows_per_gate == 1 ? a.dgate : nullptr},
                                   {a.lddy, a.lddh, a.ldu, a.ldh}, {a.gamma_post, a.gamma_pre, a.gate});
  return whole ? bwd_any<T, false>(a, stream) : bwd_any<T, true>(a, stream);
}

// of all paths that a call may take, whatever its type and alignment
int64_t most_chunks(int64_t M, int64_t N, int64_t rows_per_gate) {
  int64_t most = chunks_of(M, rows_per_gate, kLongUnits, 1).chunks;
  for (const int64_t e : {4, 8}) {       // elements of a vector
    for (const int64_t ragged : {0, 1}) {
      const int64_t n = (N + (ragged ? 2 * e - 2 : e - 1)) / e, apart = ragged ? e / std::gcd(N, e) : 1;
      most = std::max(most, chunks_of(M, rows_per_gate, units_of(n), apart).chunks);
      most = std::max(most, chunks_of(M, rows_per_gate, ring_units(n), apart).chunks);
    }
  }
  return most;
}

// the rows' means, whose place is a multiple of 16 bytes
int64_t mean_floats(int64_t M) { return (M + 3) / 4 * 4; }

}  // namespace

size_t bn_workspace_bytes(int64_t M, int64_t N, int64_t rows_per_gate) {
  return (static_cast<size_t>(most_chunks(M, N, rows_per_gate)) * 2 * N + mean_floats(M)) * sizeof(float);
}

cudaError_t launch_block_norm_bwd(const BnBwdArgs& given, void* workspace, int dtype, cudaStream_t stream) {
  BnBwdArgs a = given;
  if (workspace != nullptr) {  // the rows' means, then the chunks' sums
    a.mean = static_cast<float*>(workspace);
    a.part = a.mean + mean_floats(a.M);
  }
  return dtype == 0   ? bwd_type<float>(a, stream)
         : dtype == 1 ? bwd_type<__half>(a, stream)
                      : bwd_type<__nv_bfloat16>(a, stream);
}

}  // namespace swg
