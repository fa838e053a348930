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
#include "block_norm.cuh"

namespace swg {
namespace {

using namespace bn;

// ---- forward: a row in the registers of a group of threads, R vectors each: for few rows and for rows that a cluster
// shares (1 x 4096 bf16 4.1 us). With many rows the reads pause for each row's reductions: 16384 x 4096 bf16, 8 gates,
// 111.6 us against the ring's 97.6 to 100.
// kShared: the S blocks of a cluster, of one group each, share a row.
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
    return inverse_root(fmaf(s[0], inv_n, a.eps));
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
      ru = inverse_root(fmaf(block_sum(s[0], buf), inv_n, a.eps));
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
      rh = inverse_root(fmaf(block_sum(s[0], buf), inv_n, a.eps));
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

// Forward, HBM-bound: 16384 x 4096 bf16, 8 gates, 97.6 to 100 us (79 to 81% of the copy rate), with a gate for each row 105
// (94%; the gate in fp32 137, 87%), 8192 x 4096 fp32 97 (82%); ragged, 16384 x 4001 bf16 131 (59%), 8192 x 4001 fp32 164 (47%). A
// group takes rows one after the other, so that it keeps its gate row's columns in registers until the next
// gate row begins; kRowGate: a gate for each row is one more tensor in the ring.
constexpr int kFwdBlocks = 3;  // blocks of 256 threads an SM, with 80 registers a thread
// Such blocks an SM over a ring: in 16 bits two with 128 registers a thread (16384 x 4096 bf16, 8 gates, 95 us, three with
// 80 spill: 109), in fp32 three (8192 x 4096 90 us, two 116; whole rows only were measured: ragged fp32 ones spill with 80
// registers, 220 bytes of stores a thread at most).
template <typename T>
constexpr int kFwdRingBlocks = sizeof(T) == 4 ? 3 : 2;
template <typename T, int R, bool kShared, bool kRowGate, bool kFull, bool kRagged>
__global__ void __maxnreg__(sizeof(T) == 4 ? 80 : 128)
    bn_fwd_ring_kernel(const BnFwdArgs a, const RingPlan plan, int G, int S, int apart, Stall stall, uint32_t* status) {
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ uint64_t bars[8 * kMaxStages];
  __shared__ float smem[8 * 64];
  __shared__ ClusterSlots slots;
  constexpr int E = kElems<T>, P = kPairs<T>, kTensors = kRowGate ? 3 : 2;
  const int groups = kShared ? 1 : blockDim.x / G, group = kShared ? 0 : threadIdx.x / G;
  const int rank = kShared ? static_cast<int>(cluster_ctarank()) : 0, in = kShared ? threadIdx.x : threadIdx.x % G;
  const int64_t units = static_cast<int64_t>(kShared ? gridDim.x / S : gridDim.x) * groups;
  const int64_t unit = kShared ? blockIdx.x / S : static_cast<int64_t>(blockIdx.x) * groups + group;
  // The group's rows: begin, begin + step, ... below end; of ragged rows every `apart`-th, that lie on one offset
  // within 16 bytes, so that the columns of its vectors are the same in all of them.
  const int64_t step = kRagged ? apart : 1, phase = unit % step, of = (a.M - phase + step - 1) / step;
  const int64_t place = unit / step, places = units / step;
  const int64_t begin = phase + of * place / places * step, end = min(a.M, phase + of * (place + 1) / places * step);
  const int N = static_cast<int>(a.N);
  const int shift = kRagged ? shift_of(static_cast<const T*>(kFull || a.pre ? a.y : a.h) + begin * a.N) : 0;
  const int n = (N + shift + E - 1) / E, n0 = rank * R * G;  // vectors of a row, and the first of this block's
  const int mine = min(R * G, n - n0), over = n * E - shift - N;
  auto column = [&](int i) { return (n0 + in + i * G) * E - shift; };
  const bool add = kFull || a.residual != nullptr, post_norm = kFull || a.post, pre_norm = kFull || a.pre;
  const bool f32 = a.wdtype == 0, gated = a.gate != nullptr, gate32 = a.gdtype == 0;
  const float inv_n = 1.0f / static_cast<float>(a.N);
  const float2 alpha = pair(a.alpha);
  const uint32_t per_gate = static_cast<uint32_t>(a.rows_per_gate);
  RowRing<kTensors, kRagged> ring(dyn, bars, plan, group, stall);
  const bool first = in == 0;
  if (first) {
    ring.init();
    fence_mbar_init();
  }
  __syncthreads();
  WarpRows sums(smem, G);
  SharedSum<kShared, 1> share(slots, S, stall);
  const int64_t stop_at = kShared ? -1 : stall.at;
  auto issue = [&](int64_t r) {
    const void* from[kTensors];
    uint32_t bytes[kTensors];
    const Span span = kRagged ? span_of(r, a.M, n, n0, mine, shift, over) : Span{0, mine};
    const int j0 = (n0 + span.first) * E - shift;  // the first column that is copied
    from[0] = static_cast<const T*>(a.u) + r * a.ldu + j0;
    from[1] = add ? static_cast<const T*>(a.residual) + r * a.ldr + j0 : nullptr;
    bytes[0] = bytes[1] = static_cast<uint32_t>(span.count) * 16u;
    if constexpr (kRowGate) {
      const int64_t es = gate32 ? 4 : sizeof(T);
      from[2] = static_cast<const char*>(a.gate) + (r * a.N + j0) * es;
      bytes[2] = static_cast<uint32_t>(span.count) * static_cast<uint32_t>(E * es);
    }
    ring.issue(from, bytes, R * G * 16, stop_at, span.first * 16);
  };
  if (first)
    for (int64_t r = begin, i = 0; r < end && i < ring.stages; r += step, ++i) issue(r);
  float2 pre[R][P], q[R][P];  // gamma_pre; gamma_post, or (without kRowGate) that times the gate
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (in + i * G < mine) {
      load_weights<T, kRagged>(a.gamma_pre, column(i), N, f32, 1.0f, pre[i]);
      if (kRowGate || !gated) load_weights<T, kRagged>(a.gamma_post, column(i), N, f32, 1.0f, q[i]);
    }
  int64_t gate_end = gated && !kRowGate ? begin : INT64_MAX;  // the row from which on another gate row holds
  int64_t ahead = begin + ring.stages * step;  // the row to copy next
  bool refill = false;
  auto rstd_of = [&](float2 s2) {
    float s[1] = {sums.one(s2.x + s2.y)};
    if (refill && ahead < end) {
      issue(ahead);
      ahead += step;
    }
    refill = false;
    share(s);
    return inverse_root(fmaf(s[0], inv_n, a.eps));
  };
  T *h = static_cast<T*>(a.h) + begin * a.N, *y = static_cast<T*>(a.y) + begin * a.N;  // of the row
  const Rows<T> rows_u(a.u, a.ldu, a.M, a.N), rows_r(a.residual, a.ldr, a.M, a.N), rows_g(a.gate, a.N, a.M, a.N);
  bool edge[R];  // vectors that reach beyond the row
#pragma unroll
  for (int i = 0; i < R; ++i) edge[i] = kRagged && in + i * G < mine && (column(i) < 0 || column(i) + E > N);
  auto place_of = [&](unsigned char* stage, int tensor, int i) { return stage + (tensor * R * G + in + i * G) * 16; };
  for (int64_t r = begin; r < end; r += step, h += step * a.N, y += step * a.N) {
    if (kShared && static_cast<uint64_t>(r) >= static_cast<uint64_t>(stall.at)) share.silence();
    unsigned char* stage = ring.next();
    if constexpr (kRagged) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (!edge[i]) continue;
        const int j = column(i);
        mend_edge(place_of(stage, 0, i), rows_u, r, a.M, j, N);
        if (add) mend_edge(place_of(stage, 1, i), rows_r, r, a.M, j, N);
        if (kRowGate) mend_edge(place_of(stage, 2, i), rows_g, r, a.M, j, N);
      }
    }
    refill = first && r > begin;  // behind the row's first sum the group has read the row before
    if (!kRowGate && r >= gate_end) {
      const int64_t g = static_cast<uint32_t>(r) / per_gate;
      gate_end = (g + 1) * per_gate;
      const char* gate = static_cast<const char*>(a.gate) + g * a.N * (gate32 ? 4 : sizeof(T));
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (in + i * G >= mine) continue;
        float2 post[P];
        load_weights<T, kRagged>(gate, column(i), N, gate32, 1.0f, q[i]);
        load_weights<T, kRagged>(a.gamma_post, column(i), N, f32, 1.0f, post);
#pragma unroll
        for (int e = 0; e < P; ++e) q[i][e] = __fmul2_rn(q[i][e], post[e]);
      }
    }
    Raw w[R];
    float2 s2 = pair(0.0f);
    float ru = 1.0f, rh = 0.0f;
    if (post_norm) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (in + i * G >= mine) continue;
        const Raw u = ld_stage(place_of(stage, 0, i));
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float2 v = get_pair<T>(u, e);
          s2 = __ffma2_rn(v, v, s2);
        }
      }
      ru = rstd_of(s2);
      s2 = pair(0.0f);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (in + i * G >= mine) continue;
      w[i] = ld_stage(place_of(stage, 0, i));
      Raw res = {};
      if (add) res = ld_stage(place_of(stage, 1, i));
      float2 gate[P];
      if constexpr (kRowGate) stage_pairs<T>(stage + 2 * R * G * 16, in + i * G, !kRagged && gate32, gate);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        float2 v = get_pair<T>(w[i], e);
        if (post_norm || gated) {
          v = __fmul2_rn(v, __fmul2_rn(pair(ru), q[i][e]));
          if constexpr (kRowGate) v = __fmul2_rn(v, gate[e]);
        }
        if (add) v = __ffma2_rn(alpha, get_pair<T>(res, e), v);
        set_pair<T>(w[i], e, v);  // h as it is stored
        v = get_pair<T>(w[i], e);
        s2 = __ffma2_rn(v, v, s2);
      }
      if (kFull || a.h != nullptr) store_vector<T, kRagged>(h, column(i), N, edge[i], w[i]);
    }
    if (pre_norm) {
      rh = rstd_of(s2);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (in + i * G >= mine) continue;
#pragma unroll
        for (int e = 0; e < P; ++e)
          set_pair<T>(w[i], e, __fmul2_rn(get_pair<T>(w[i], e), __fmul2_rn(pair(rh), pre[i][e])));
        store_vector<T, kRagged>(y, column(i), N, edge[i], w[i]);
      }
    }
    if (in + n0 == 0) {
      a.stats[2 * r] = post_norm ? ru : 0.0f;
      a.stats[2 * r + 1] = rh;
    }
  }
  if (first) ring.end(status);
  else if (ring.wait.lost() && status != nullptr) atomicOr(status, kStatusTimeout);
  share.end(status);
}

// ---- host
template <typename T>
cudaError_t fwd_long(const BnFwdArgs& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.M, 65536));
  bn_fwd_long_kernel<T><<<grid, kMaxThreads, 0, stream>>>(a);
  return cudaGetLastError();
}
template <typename T, bool kRowGate, bool kFull, bool kRagged>
cudaError_t fwd_ring_one(const BnFwdArgs& a, int64_t n, cudaStream_t stream) {
  const auto kernel = bn_fwd_ring_kernel<T, 2, false, kRowGate, kFull, kRagged>;
  const int G = group_threads(n, 2), groups = G < kBlock ? kBlock / G : 1, block = groups * G;
  const RingPlan p = ring_plan((2 + (kRowGate ? gate_slots<T>(a.gdtype) : 0)) * 2 * G * 16,
                               std::max(1, kFwdRingBlocks<T> * kBlock / block), groups);
  const size_t smem = static_cast<size_t>(groups) * p.group_bytes;
  int64_t blocks;
  {
    static std::mutex mu;
    static FitCache cache;
    std::lock_guard<std::mutex> lk(mu);
    const cudaError_t e = blocks_that_fit(kernel, cache, block, smem, blocks);
    if (e != cudaSuccess) return e;
  }
  const int apart = kRagged ? rows_apart<T>(a.N) : 1;
  blocks = persistent_blocks(blocks, (a.M + groups - 1) / groups / apart * apart, apart);
  if (blocks < 1) return fwd_long<T>(a, stream);
  kernel<<<static_cast<unsigned>(blocks), block, smem, stream>>>(a, p, G, 1, apart, take_stall(kInjectBlockNormFwd),
                                                                status_word_ptr());
  return cudaGetLastError();
}
template <typename T, bool kRowGate, bool kFull, bool kRagged>
cudaError_t fwd_ring_shared(const BnFwdArgs& a, int64_t n, cudaStream_t stream) {
  const auto kernel = bn_fwd_ring_kernel<T, 2, true, kRowGate, kFull, kRagged>;
  const Shared s = share_row(n, 2);
  const RingPlan p = ring_plan((2 + (kRowGate ? gate_slots<T>(a.gdtype) : 0)) * 2 * s.G * 16,
                               std::max(1, kFwdRingBlocks<T> * kBlock / s.G), 1);
  static std::mutex mu;
  static StreamCache cache;
  std::lock_guard<std::mutex> lk(mu);
  const cudaError_t e = clusters_that_fit(kernel, cache, s.G, p.group_bytes, s.S);
  if (e != cudaSuccess) return e;
  const int apart = kRagged ? rows_apart<T>(a.N) : 1;
  const int64_t clusters = persistent_blocks(cache.clusters, a.M / apart * apart, apart);
  if (clusters < 1) return fwd_long<T>(a, stream);
  ClusterLaunch l(s.G, p.group_bytes, s.S, clusters, stream);
  return cudaLaunchKernelEx(&l.cfg, kernel, a, p, s.G, s.S, apart, take_stall(kInjectBlockNormFwd), status_word_ptr());
}

template <typename T, bool kRowGate, bool kFull, bool kRagged>
cudaError_t fwd_ring(const BnFwdArgs& a, int64_t n, cudaStream_t stream) {
  return n <= 2 * kBlock ? fwd_ring_one<T, kRowGate, kFull, kRagged>(a, n, stream)
                         : fwd_ring_shared<T, kRowGate, kFull, kRagged>(a, n, stream);
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
  const bool row_gate = a.gate != nullptr && a.rows_per_gate == 1;
  const bool ring = !kRagged || (same_offsets(a.M, a.N, sizeof(T), a.pre ? a.y : a.h,
                                              {a.u, a.residual, a.pre ? a.h : nullptr, row_gate ? a.gate : nullptr},
                                              {a.ldu, a.residual != nullptr ? a.ldr : a.N}) &&
                                 (!row_gate || sizeof(T) == 4 || a.gdtype != 0));
  if (ring && n <= 2 * kMaxCluster * kBlock && a.M * ((n + 1) / 2) >= kRingRows * kFwdBlocks * kBlock * device_sm_count()) {
    const bool full = a.post && a.pre && a.residual != nullptr;
    if (row_gate)
      return full ? fwd_ring<T, true, true, kRagged>(a, n, stream) : fwd_ring<T, true, false, kRagged>(a, n, stream);
    return full ? fwd_ring<T, false, true, kRagged>(a, n, stream) : fwd_ring<T, false, false, kRagged>(a, n, stream);
  }
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
}  // namespace

cudaError_t launch_block_norm_fwd(const BnFwdArgs& a, int dtype, cudaStream_t stream) {
  return dtype == 0   ? fwd_type<float>(a, stream)
         : dtype == 1 ? fwd_type<__half>(a, stream)
                      : fwd_type<__nv_bfloat16>(a, stream);
}

}  // namespace swg
