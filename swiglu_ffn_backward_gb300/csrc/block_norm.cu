// The junction of two blocks of a transformer: the norm after a block, its gate, the scaled residual, and the norm
// before the next block (root mean square norms, over the last dimension), forward and backward.
//   rstd(t) = 1 / sqrt(sum t^2 / N + eps)
//   v = u rstd(u) gamma_post  (v = u without the norm after the block)
//   h = alpha r + gate v, rounded to the I/O type;  y = h rstd(h) gamma_pre
// A row of the gate serves M / G rows, one after the other. Backward, with u^ = u rstd(u), h^ = h rstd(h),
// a = dy gamma_pre and q = gate gamma_post, from dy and dh, the gradient that reaches h past the second norm:
//   D  = dh + rstd(h) (a - h^ mean(a h^)),  dr = alpha D
//   du = rstd(u) (q D - u^ mean(q D u^))
//   dgamma_pre = sum dy h^;  with S = sum D u^ over the rows of a gate row: dgate = gamma_post S, and
//   dgamma_post = the sum of gate S over the gate's rows
// so that two column sums give all three parameter gradients. The second mean needs no second round over the row:
//   sum q D u^ = sum q u^ (dh + rstd(h) a) - rstd(h) mean(a h^) sum q h^ u^
// All arithmetic is fp32; h, y, dr, du and the parameters' gradients are rounded once.
#include <algorithm>

#include "row_vectors.cuh"

namespace swg {
namespace {

using namespace row;

constexpr int kMaxThreads = 1024;

// ---- forward: a row in the registers of a group of threads, R vectors each
// kShared: the S blocks of a cluster, of one group each, share a row.
constexpr int kBlock = 256;      // threads of a block, unless a row takes more
constexpr int kMaxGroup = 512;   // threads of a group, and of a block
template <bool kRagged>
constexpr int kFwdRegs = kRagged ? 128 : 80;
template <typename T, int R, bool kRagged, bool kShared>
__global__ void __maxnreg__(kFwdRegs<kRagged>)
    bn_fwd_kernel(const BnFwdArgs a, int G, int S, Stall stall, uint32_t* status) {
  __shared__ float smem[2 * 32];
  __shared__ ClusterSlots slots;
  constexpr int E = kElems<T>, P = kPairs<T>;
  constexpr bool kNarrow = R == 1;  // groups of less than a warp
  const int groups = kShared ? 1 : blockDim.x / G;
  const int t = kShared ? threadIdx.x + cluster_ctarank() * R * G : threadIdx.x % G;  // vectors t, t + G, ...
  const int64_t step = static_cast<int64_t>(kShared ? gridDim.x / S : gridDim.x) * groups;
  const int N = static_cast<int>(a.N);
  int64_t r = kShared ? blockIdx.x / S : static_cast<int64_t>(blockIdx.x) * groups + threadIdx.x / G;
  const int shift = kRagged ? shift_of(static_cast<const T*>(a.pre ? a.y : a.h) + r * a.N) : 0;
  int n = (N + shift + E - 1) / E;  // vectors of the row
  const bool add = a.residual != nullptr, f32 = a.wdtype == 0, gated = a.gate != nullptr, join = a.h != nullptr;
  const float inv_n = 1.0f / static_cast<float>(a.N);
  const float2 alpha = pair(a.alpha);
  const uint32_t per_gate = static_cast<uint32_t>(a.rows_per_gate);
  auto column = [&](int i) { return (t + i * G) * E - shift; };
  struct Row {
    Raw u[R], res[R];
  };
  const Rows<T> u(a.u, a.ldu, a.M, a.N), res(a.residual, a.ldr, a.M, a.N);
  auto load = [&](Row& w, int64_t r) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (t + i * G >= n) continue;
      w.u[i] = load_columns<T, kRagged>(u, r, column(i), N);
      if (add) w.res[i] = load_columns<T, kRagged>(res, r, column(i), N);
    }
  };
  GroupSum<1, kNarrow> sum(smem, G);
  SharedSum<kShared, 1> share(slots, S, stall);
  auto rstd_of = [&](float2 s2) {
    float s[1] = {s2.x + s2.y};
    sum(s);
    share(s);
    return rsqrtf(fmaf(s[0], inv_n, a.eps));
  };
  Row next;
  const int64_t M = a.M + (kNarrow ? (threadIdx.x & 31) / G : 0);  // the rows of a warp's groups end together
  if (r < a.M) load(next, r);
  for (; r < M; r += step) {
    if (kNarrow && r >= a.M) n = 0;
    if (kShared && static_cast<uint64_t>(r) >= static_cast<uint64_t>(stall.at)) share.silence();
    Row w = next;
    if (r + step < a.M) load(next, r + step);
    if constexpr (kRagged) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        clear_others<T>(w.u[i], column(i), N);
        if (add) clear_others<T>(w.res[i], column(i), N);
      }
    }
    // the gate's columns and those of its norm: under way while the row's sum is taken
    float2 q[R][P];
    const char* gate = static_cast<const char*>(a.gate) +
                       (gated ? static_cast<int64_t>(static_cast<uint32_t>(r) / per_gate) * a.N * (a.gdtype == 0 ? 4 : 2) : 0);
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (gated && t + i * G < n) load_weights<T, kRagged>(gate, column(i), N, a.gdtype == 0, 1.0f, q[i]);
    float ru = 0.0f, rh = 0.0f;
    if (a.post) {
      float2 s2 = pair(0.0f);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (t + i * G >= n) continue;
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float2 v = get_pair<T>(w.u[i], e);
          s2 = __ffma2_rn(v, v, s2);
        }
      }
      ru = rstd_of(s2);
    }
    float2 s2 = pair(0.0f);
    if (join) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (t + i * G >= n) continue;
        float2 post[P];
        if (a.post) load_weights<T, kRagged>(a.gamma_post, column(i), N, f32, 1.0f, post);
#pragma unroll
        for (int e = 0; e < P; ++e) {
          float2 v = get_pair<T>(w.u[i], e);
          if (a.post) v = __fmul2_rn(v, __fmul2_rn(pair(ru), post[e]));
          if (gated) v = __fmul2_rn(v, q[i][e]);
          if (add) v = __ffma2_rn(alpha, get_pair<T>(w.res[i], e), v);
          set_pair<T>(w.u[i], e, v);  // h as it is stored
          v = get_pair<T>(w.u[i], e);
          s2 = __ffma2_rn(v, v, s2);
        }
        store_columns<T, kRagged>(static_cast<T*>(a.h) + r * a.N, column(i), N, w.u[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (t + i * G >= n) continue;
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float2 v = get_pair<T>(w.u[i], e);
          s2 = __ffma2_rn(v, v, s2);
        }
      }
    }
    if (a.pre) {
      rh = rstd_of(s2);
      T* y = static_cast<T*>(a.y) + r * a.N;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (t + i * G >= n) continue;
        float2 pre[P];
        load_weights<T, kRagged>(a.gamma_pre, column(i), N, f32, 1.0f, pre);
#pragma unroll
        for (int e = 0; e < P; ++e)
          set_pair<T>(w.u[i], e, __fmul2_rn(get_pair<T>(w.u[i], e), __fmul2_rn(pair(rh), pre[e])));
        store_columns<T, kRagged>(y, column(i), N, w.u[i]);
      }
    }
    if (t == 0 && (!kNarrow || n > 0)) {
      a.stats[2 * r] = ru;
      a.stats[2 * r + 1] = rh;
    }
  }
  share.end(status);
}

// ---- rows of any length, element by element, read three times (from L2 where a row fits)
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) bn_fwd_long_kernel(const BnFwdArgs a) {
  __shared__ float buf[32];
  const float inv_n = 1.0f / static_cast<float>(a.N);
  for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
    const T* u = static_cast<const T*>(a.u) + r * a.ldu;
    const T* res = a.residual != nullptr ? static_cast<const T*>(a.residual) + r * a.ldr : nullptr;
    const int64_t gate = r / a.rows_per_gate * a.N;
    T* h = a.h != nullptr ? static_cast<T*>(a.h) + r * a.N : nullptr;
    float s[1], ru = 0.0f, rh = 0.0f;
    if (a.post) {
      long_sums(a.N, s, [&](float (&p)[1], int64_t j) {
        const float v = to_f(u[j]);
        p[0] = fmaf(v, v, p[0]);
      });
      ru = rsqrtf(fmaf(block_sum(s[0], buf), inv_n, a.eps));
    }
    auto value = [&](int64_t j) {  // h_j, rounded as it is stored
      if (a.h == nullptr) return to_f(u[j]);
      float v = to_f(u[j]);
      if (a.post) v *= ru * (a.gamma_post != nullptr ? load_any(a.gamma_post, j, a.wdtype) : 1.0f);
      if (a.gate != nullptr) v *= load_any(a.gate, gate + j, a.gdtype);
      if (res != nullptr) v = fmaf(a.alpha, to_f(res[j]), v);
      return to_f(from_f<T>(v));
    };
    if (a.pre) {
      long_sums(a.N, s, [&](float (&p)[1], int64_t j) {
        const float v = value(j);
        p[0] = fmaf(v, v, p[0]);
      });
      rh = rsqrtf(fmaf(block_sum(s[0], buf), inv_n, a.eps));
    }
    for (int64_t j = threadIdx.x; j < a.N; j += blockDim.x) {
      const float v = value(j);
      if (h != nullptr) h[j] = from_f<T>(v);
      if (a.pre)
        static_cast<T*>(a.y)[r * a.N + j] =
            from_f<T>(v * (rh * (a.gamma_pre != nullptr ? load_any(a.gamma_pre, j, a.wdtype) : 1.0f)));
    }
    if (threadIdx.x == 0) {
      a.stats[2 * r] = ru;
      a.stats[2 * r + 1] = rh;
    }
  }
}

// ---- backward: a row in the registers of a group of threads, one vector of each tensor a thread
// A group takes chunks of rows, chunk after chunk, and writes the chunk's two column sums. kShared: as in the forward.
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
    const int64_t seg = c / k.per_segment, in = c - seg * k.per_segment, block = in / k.apart;
    const int64_t first = in - block * k.apart + k.apart * block * k.rows;  // within the segment
    const int64_t left = (k.segment - first + k.apart - 1) / k.apart;
    int count = mine ? static_cast<int>(max(static_cast<int64_t>(0), min(left, k.rows))) : 0;
    const int64_t r0 = seg * k.segment + first;
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
  const int64_t seg = chunk / k.per_segment, r0 = seg * k.segment + chunk % k.per_segment * k.rows;  // apart is 1
  const int64_t r1 = min((seg + 1) * k.segment, r0 + k.rows);
  const float pre = a.pre && a.gamma_pre != nullptr ? load_any(a.gamma_pre, j, a.wdtype) : 1.0f;
  float s = 0.0f, p = 0.0f;
  for (int64_t r = r0; r < r1; ++r) {
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

// The parameters' gradients from the chunks' sums: 32 columns a block, 32 threads a column take the chunks in turn and
// are added in order. Blocks of the first row sum all chunks, for dgamma_post (each times its gate row) and
// dgamma_pre; those of row 1 + g the chunks of gate row g. At most 64 terms are added in fp32, these parts in fp64. A
// programmatic dependent of the kernel before it, whose writes are visible after griddepcontrol.wait.
constexpr int kReduceCols = 32, kReduceSlices = 32;
__global__ void __launch_bounds__(kReduceCols* kReduceSlices)
    bn_reduce_kernel(const BnBwdArgs a, const BnChunks k, int64_t first_gate, bool sums) {
  __shared__ double acc[kReduceSlices][kReduceCols];
  const int c = threadIdx.x % kReduceCols, slice = threadIdx.x / kReduceCols;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kReduceCols + c;
  const bool whole = sums && blockIdx.y == 0;  // over all chunks
  const int64_t g = first_gate + blockIdx.y - (sums ? 1 : 0);
  const int64_t begin = whole ? 0 : g * k.per_segment, end = whole ? k.chunks : begin + k.per_segment;
  const bool weigh = whole && a.gate != nullptr && a.rows_per_gate > 1 && j < a.N;
  const int64_t most = whole ? 2 * a.N : a.N;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  double t = 0.0;
  if (j < most) {
    const float* part = a.part + j;
    auto term = [&](int64_t n) {
      const float v = part[n * 2 * a.N];
      return weigh ? v * load_any(a.gate, n / k.per_segment * a.N + j, a.gdtype) : v;
    };
    for (int64_t i = begin + slice; i < end; i += 64 * kReduceSlices) {
      const int64_t stop = min(end, i + 64 * kReduceSlices);
      float s = 0.0f;
      int64_t n = i;
      for (; n + 7 * kReduceSlices < stop; n += 8 * kReduceSlices) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = term(n + e * kReduceSlices);
        s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
      }
      for (; n < stop; n += kReduceSlices) s += term(n);
      t += static_cast<double>(s);
    }
  }
  acc[slice][c] = t;
  __syncthreads();
  if (slice != 0 || j >= most) return;
  for (int i = 1; i < kReduceSlices; ++i) t += acc[i][c];
  const float v = static_cast<float>(t);
  if (!whole) {
    const float post = a.post && a.gamma_post != nullptr ? load_any(a.gamma_post, j, a.wdtype) : 1.0f;
    store_any(a.dgate, g * a.N + j, a.gdtype, v * post);
  } else if (j < a.N) {
    if (a.dgamma_post != nullptr) store_any(a.dgamma_post, j, a.wdtype, v);
  } else if (a.dgamma_pre != nullptr) {
    store_any(a.dgamma_pre, j - a.N, a.wdtype, v);
  }
}

// ---- host
// Chunks of rows whose column sums are taken together: of one gate row where the gate has fewer rows than M, of at most
// 128 rows (like terms are rounded the same way, and a longer chain drifts), and such that `units` groups that take
// them in turn have nearly equal work: rows, and for each chunk the writing of its sums, about one row's.
constexpr int64_t kMostRows = 128;
BnChunks chunks_of(int64_t M, int64_t rows_per_gate, int64_t units, int64_t apart) {
  BnChunks k;
  k.segment = rows_per_gate > 1 ? rows_per_gate : M;
  k.apart = apart;
  const int64_t segments = M / k.segment, rows = (k.segment + apart - 1) / apart;  // of a phase, at most
  int64_t best = INT64_MAX;
  const int64_t least = (rows + kMostRows - 1) / kMostRows;
  const int64_t most = std::min(rows, std::max(least, (2 * units + segments * apart - 1) / (segments * apart)));
  const int64_t step = std::max<int64_t>(1, (most - least) / 64);
  for (int64_t n = least; n <= most; n += step) {
    const int64_t per = (rows + n - 1) / n, chunks = segments * apart * ((rows + per - 1) / per);
    const int64_t cost = (chunks + units - 1) / units * (per + 1);
    if (cost < best) {
      best = cost;
      k.rows = per;
      k.per_segment = apart * ((rows + per - 1) / per);
      k.chunks = chunks;
    }
  }
  return k;
}
// The groups of threads that take chunks: those of one block of 512 threads (or a cluster of blocks) on each of 152
// SMs, for rows of n vectors. A plan that does not depend on the device, so that the workspace's size does not.
int64_t units_of(int64_t n) {
  constexpr int64_t kSms = 152;
  if (n <= kMaxGroup) return kSms * (kMaxGroup / group_threads(n, 1));
  return std::max<int64_t>(1, kSms / ((n + kMaxGroup - 1) / kMaxGroup));
}
constexpr int64_t kLongUnits = 304;  // for rows of any length

cudaError_t launch_reduce(const BnBwdArgs& a, const BnChunks& k, cudaStream_t stream) {
  const bool sums = a.dgamma_post != nullptr || a.dgamma_pre != nullptr;
  const int64_t gates = a.dgate != nullptr && a.rows_per_gate > 1 ? a.M / a.rows_per_gate : 0;
  const int64_t all = gates + (sums ? 1 : 0);
  const unsigned gx = static_cast<unsigned>(((sums ? 2 : 1) * a.N + kReduceCols - 1) / kReduceCols);
  for (int64_t y = 0; y < all; y += 65535) {
    const bool first = sums && y == 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(gx, static_cast<unsigned>(std::min<int64_t>(65535, all - y)));
    cfg.blockDim = dim3(kReduceCols * kReduceSlices);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = y == 0 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, bn_reduce_kernel, a, k, first ? int64_t(0) : y - (sums ? 1 : 0), first);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Rows shared by a cluster: S blocks of G threads, R vectors each
struct Shared {
  int S, G;
};
Shared share_row(int64_t n, int R) {
  const int64_t threads = (n + R - 1) / R;
  const int S = static_cast<int>(threads <= kMaxCluster * kBlock ? (threads + kBlock - 1) / kBlock : kMaxCluster);
  return Shared{S, static_cast<int>((threads + 32 * S - 1) / (32 * S)) * 32};
}

template <typename T>
cudaError_t fwd_long(const BnFwdArgs& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.M, 65536));
  bn_fwd_long_kernel<T><<<grid, kMaxThreads, 0, stream>>>(a);
  return cudaGetLastError();
}
template <typename T, int R, bool kRagged>
cudaError_t fwd_one(const BnFwdArgs& a, int64_t n, cudaStream_t stream) {
  const int G = group_threads(n, R), groups = G < kBlock ? kBlock / G : 1, block = groups * G;
  int64_t blocks;
  {
    static std::mutex mu;
    static FitCache cache;
    std::lock_guard<std::mutex> lk(mu);
    const cudaError_t e = blocks_that_fit(bn_fwd_kernel<T, R, kRagged, false>, cache, block, 0, blocks);
    if (e != cudaSuccess) return e;
  }
  blocks = persistent_blocks(blocks, (a.M + groups - 1) / groups, kRagged ? rows_apart<T>(a.N) : 1);
  if (blocks == 0) return fwd_long<T>(a, stream);
  bn_fwd_kernel<T, R, kRagged, false><<<static_cast<unsigned>(blocks), block, 0, stream>>>(a, G, 1, Stall(), nullptr);
  return cudaGetLastError();
}
template <typename T, bool kRagged>
cudaError_t fwd_shared(const BnFwdArgs& a, int64_t n, cudaStream_t stream) {
  static std::mutex mu;
  static StreamCache cache;
  std::lock_guard<std::mutex> lk(mu);
  const Shared p = share_row(n, 2);
  const auto kernel = bn_fwd_kernel<T, 2, kRagged, true>;
  const cudaError_t e = clusters_that_fit(kernel, cache, p.G, 0, p.S);
  if (e != cudaSuccess) return e;
  const int64_t clusters = persistent_blocks(cache.clusters, a.M, kRagged ? rows_apart<T>(a.N) : 1);
  if (clusters == 0) return fwd_long<T>(a, stream);
  ClusterLaunch l(p.G, 0, p.S, clusters, stream);
  return cudaLaunchKernelEx(&l.cfg, kernel, a, p.G, p.S, take_stall(kInjectBlockNormFwd), status_word_ptr());
}
template <typename T, bool kRagged>
cudaError_t fwd_any(const BnFwdArgs& a, cudaStream_t stream) {
  const int64_t n = (a.N + (kRagged ? 2 * kElems<T> - 2 : 0)) / kElems<T>;
  if (n <= 32) return fwd_one<T, 1, kRagged>(a, n, stream);
  if (n <= 2 * kMaxGroup) return fwd_one<T, 2, kRagged>(a, n, stream);
  if (n <= 2 * kMaxCluster * kMaxGroup) return fwd_shared<T, kRagged>(a, n, stream);
  return fwd_long<T>(a, stream);
}
template <typename T>
cudaError_t fwd_type(const BnFwdArgs& a, cudaStream_t stream) {
  const bool whole = whole_vectors(a.N, sizeof(T), {a.u, a.residual, a.h, a.y}, {a.ldu, a.ldr},
                                   {a.gamma_post, a.gamma_pre, a.gate});
  return whole ? fwd_any<T, false>(a, stream) : fwd_any<T, true>(a, stream);
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
template <typename T, bool kRagged>
cudaError_t bwd_any(const BnBwdArgs& a, cudaStream_t stream) {
  const int64_t n = (a.N + (kRagged ? 2 * kElems<T> - 2 : 0)) / kElems<T>;
  if (n <= 16) return bwd_groups<T, kRagged, true>(a, n, stream);
  if (n <= kMaxGroup) return bwd_groups<T, kRagged, false>(a, n, stream);
  if (n <= kMaxCluster * kMaxGroup) return bwd_shared<T, kRagged>(a, n, stream);
  return bwd_long<T>(a, stream);
}
template <typename T>
cudaError_t bwd_type(const BnBwdArgs& a, cudaStream_t stream) {
  const bool whole = whole_vectors(a.N, sizeof(T), {a.dy, a.dh, a.u, a.h, a.du, a.dres, a.gdtype != 0 ? a.dgate : nullptr},
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
    }
  }
  return most;
}

}  // namespace

size_t bn_workspace_bytes(int64_t M, int64_t N, int64_t rows_per_gate) {
  return (static_cast<size_t>(most_chunks(M, N, rows_per_gate)) * 2 * N + M) * sizeof(float);
}

cudaError_t launch_block_norm_fwd(const BnFwdArgs& a, int dtype, cudaStream_t stream) {
  return dtype == 0   ? fwd_type<float>(a, stream)
         : dtype == 1 ? fwd_type<__half>(a, stream)
                      : fwd_type<__nv_bfloat16>(a, stream);
}

cudaError_t launch_block_norm_bwd(const BnBwdArgs& given, void* workspace, int dtype, cudaStream_t stream) {
  BnBwdArgs a = given;
  if (workspace != nullptr) {  // the rows' means, then the chunks' sums
    a.part = static_cast<float*>(workspace);
    a.mean = a.part + most_chunks(a.M, a.N, a.rows_per_gate) * 2 * a.N;
  }
  return dtype == 0   ? bwd_type<float>(a, stream)
         : dtype == 1 ? bwd_type<__half>(a, stream)
                      : bwd_type<__nv_bfloat16>(a, stream);
}

}  // namespace swg
