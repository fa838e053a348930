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

// ---- many whole rows: a group's next rows are on their way into shared memory
// A thread that holds a row's vectors has but one more row of them under way; four rows of all tensors in a ring of
// shared memory, one bulk copy a tensor and row, keep the memory busy over a row's reductions. The group's first thread
// issues the next copy into a row's stage behind the barrier of the next row's first sum, when the whole group has
// read it. The stage is read again for each pass over the row, so that the row takes no registers between them.
struct RingPlan {
  int stages;        // rows of the ring of a group
  int stage_bytes;   // of a row's tensors
  int group_bytes;   // of a group's ring
};
constexpr int kMaxStages = 8;
template <int kTensors>
struct Ring {
  uint64_t* full;
  unsigned char* buf;
  int stages, stage_bytes, at = 0;  // stage of the row that is read next
  uint32_t parity = 0;
  int64_t issued = 0;
  Patience wait;
  __device__ __forceinline__ Ring(unsigned char* smem, uint64_t* bars, const RingPlan& p, int group, const Stall& stall)
      : full(bars + group * kMaxStages), buf(smem + group * p.group_bytes), stages(p.stages), stage_bytes(p.stage_bytes),
        wait(stall.limit) {}
  __device__ __forceinline__ void init() {
    for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
  }
  // by the group's first thread: the next row's tensors, `bytes` of each from `from` (null: none) into the stage's
  // slots of `slot` bytes
  __device__ __forceinline__ void issue(const void* const (&from)[kTensors], const uint32_t (&bytes)[kTensors], int slot,
                                        int64_t stall_at) {
    if (wait.lost() || issued == stall_at) return;
    const int st = static_cast<int>(issued % stages);
    uint32_t all = 0;
#pragma unroll
    for (int i = 0; i < kTensors; ++i) all += from[i] != nullptr ? bytes[i] : 0u;
    mbar_arrive_expect_tx(&full[st], all);
#pragma unroll
    for (int i = 0; i < kTensors; ++i)
      if (from[i] != nullptr && bytes[i] > 0) bulk_g2s(buf + st * stage_bytes + i * slot, from[i], bytes[i], &full[st]);
    ++issued;
  }
  // the stage of the next row, landed
  __device__ __forceinline__ const unsigned char* next() {
    wait(&full[at], parity);
    const unsigned char* p = buf + at * stage_bytes;
    if (++at == stages) {
      at = 0;
      parity ^= 1u;
    }
    return p;
  }
  // copies that nothing waited for have to land before the block ends
  __device__ __forceinline__ void end(uint32_t* status) {
    if (!wait.lost()) return;
    if (status != nullptr) atomicOr(status, kStatusTimeout);
    for (int64_t i = issued > stages ? issued - stages : 0; i < issued; ++i)
      if (!mbar_wait(&full[i % stages], static_cast<uint32_t>(i / stages) & 1u)) break;
  }
};
__device__ __forceinline__ Raw ld_stage(const unsigned char* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  return Raw{{u.x, u.y, u.z, u.w}};
}
// eight or four columns of a gate in a stage, of the tensor's type or fp32
template <typename T>
__device__ __forceinline__ void stage_pairs(const unsigned char* p, int vector, bool f32, float2 (&f)[kPairs<T>]) {
  if (sizeof(T) == 2 && f32) {
    const Raw a = ld_stage(p + vector * 32), b = ld_stage(p + vector * 32 + 16);
    f[0] = get_pair<float>(a, 0);
    f[1] = get_pair<float>(a, 1);
    f[2 % kPairs<T>] = get_pair<float>(b, 0);
    f[3 % kPairs<T>] = get_pair<float>(b, 1);
    return;
  }
  const Raw a = ld_stage(p + vector * 16);
#pragma unroll
  for (int e = 0; e < kPairs<T>; ++e) f[e] = get_pair<T>(a, e);
}
// Sums over a group of whole warps, up to eight; every thread gets them, added in a fixed order. Two buffers alternate,
// so that one barrier a sum is enough.
struct WarpRows {
  float* buf;  // of the group: 2 x 32
  int warps, id, turn = 0;
  __device__ __forceinline__ WarpRows(float* smem, int G)
      : buf(smem + (threadIdx.x / G) * 64), warps(G >> 5), id(1 + static_cast<int>(threadIdx.x) / G) {}
  __device__ __forceinline__ float* next() {
    float* b = buf + turn;
    turn ^= 32;
    return b;
  }
  __device__ __forceinline__ void meet() const {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(warps * 32) : "memory");
  }
  __device__ __forceinline__ float one(float v) {
    v = warp_sum(v);
    if (warps == 1) {
      __syncwarp();
      return v;
    }
    float* b = next();
    const int lane = threadIdx.x & 31;
    if (lane == 0) b[threadIdx.x / 32 % warps] = v;
    meet();
    v = (lane & 7) < warps ? b[lane & 7] : 0.0f;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  // Three at once: lanes exchange halves of what they hold, so that it takes six shuffles in place of fifteen.
  __device__ __forceinline__ void three(float (&v)[3]) {
    const int lane = threadIdx.x & 31;
    const bool b4 = (lane & 16) != 0, b3 = (lane & 8) != 0;
    // lanes with bit 4: v[2] (and nothing), the others v[0] and v[1]
    float x = (b4 ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, b4 ? v[0] : v[2], 16);
    float y = (b4 ? 0.0f : v[1]) + __shfl_xor_sync(0xffffffffu, b4 ? v[1] : 0.0f, 16);
    x = (b3 ? y : x) + __shfl_xor_sync(0xffffffffu, b3 ? x : y, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    // lanes 0 .. 7: v[0], 8 .. 15: v[1], 16 .. 23: v[2]
    if (warps > 1) {
      float* b = next();
      if ((lane & 7) == 0) b[(threadIdx.x / 32 % warps) * 4 + (lane >> 3)] = x;
      meet();
      x = (lane & 7) < warps ? b[(lane & 7) * 4 + (lane >> 3)] : 0.0f;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    } else {
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] = __shfl_sync(0xffffffffu, x, 8 * i);
  }
};

// Forward: a group takes rows one after the other, so that it keeps its gate row's columns in registers until the next
// gate row begins; kRowGate: a gate for each row is one more tensor in the ring.
constexpr int kFwdBlocks = 3;  // blocks of 256 threads an SM, with 80 registers a thread
template <bool kRowGate>
constexpr int kFwdRingBlocks = 2;
template <typename T, int R, bool kShared, bool kRowGate, bool kFull>
__global__ void __maxnreg__(128)
    bn_fwd_ring_kernel(const BnFwdArgs a, const RingPlan plan, int G, int S, Stall stall, uint32_t* status) {
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ uint64_t bars[8 * kMaxStages];
  __shared__ float smem[8 * 64];
  __shared__ ClusterSlots slots;
  constexpr int E = kElems<T>, P = kPairs<T>, kTensors = kRowGate ? 3 : 2;
  const int groups = kShared ? 1 : blockDim.x / G, group = kShared ? 0 : threadIdx.x / G;
  const int rank = kShared ? static_cast<int>(cluster_ctarank()) : 0, in = kShared ? threadIdx.x : threadIdx.x % G;
  const int64_t units = static_cast<int64_t>(kShared ? gridDim.x / S : gridDim.x) * groups;
  const int64_t unit = kShared ? blockIdx.x / S : static_cast<int64_t>(blockIdx.x) * groups + group;
  const int64_t begin = a.M * unit / units, end = a.M * (unit + 1) / units;
  const int n = static_cast<int>(a.N) / E, n0 = rank * R * G;  // vectors of a row, and the first of this block's
  const int mine = min(R * G, n - n0);
  const bool add = kFull || a.residual != nullptr, post_norm = kFull || a.post, pre_norm = kFull || a.pre;
  const bool f32 = a.wdtype == 0, gated = a.gate != nullptr, gate32 = a.gdtype == 0;
  const float inv_n = 1.0f / static_cast<float>(a.N);
  const float2 alpha = pair(a.alpha);
  const uint32_t per_gate = static_cast<uint32_t>(a.rows_per_gate);
  Ring<kTensors> ring(dyn, bars, plan, group, stall);
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
    from[0] = static_cast<const T*>(a.u) + r * a.ldu + n0 * E;
    from[1] = add ? static_cast<const T*>(a.residual) + r * a.ldr + n0 * E : nullptr;
    bytes[0] = bytes[1] = static_cast<uint32_t>(mine) * 16u;
    if constexpr (kRowGate) {
      const int64_t es = gate32 ? 4 : sizeof(T);
      from[2] = static_cast<const char*>(a.gate) + (r * a.N + n0 * E) * es;
      bytes[2] = static_cast<uint32_t>(mine) * static_cast<uint32_t>(E * es);
    }
    ring.issue(from, bytes, R * G * 16, stop_at);
  };
  if (first)
    for (int64_t r = begin; r < min(end, begin + ring.stages); ++r) issue(r);
  float2 pre[R][P], q[R][P];  // gamma_pre; gamma_post, or (without kRowGate) that times the gate
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (in + i * G < mine) {
      load_weights<T, false>(a.gamma_pre, (n0 + in + i * G) * E, a.N, f32, 1.0f, pre[i]);
      if (kRowGate || !gated) load_weights<T, false>(a.gamma_post, (n0 + in + i * G) * E, a.N, f32, 1.0f, q[i]);
    }
  int64_t gate_end = gated && !kRowGate ? begin : INT64_MAX;  // the row from which on another gate row holds
  int64_t ahead = begin + ring.stages;  // the row to copy next
  bool refill = false;
  auto rstd_of = [&](float2 s2) {
    float s[1] = {sums.one(s2.x + s2.y)};
    if (refill && ahead < end) issue(ahead++);
    refill = false;
    share(s);
    return rsqrtf(fmaf(s[0], inv_n, a.eps));
  };
  T *h = static_cast<T*>(a.h) + begin * a.N + (n0 + in) * E, *y = static_cast<T*>(a.y) + begin * a.N + (n0 + in) * E;
  for (int64_t r = begin; r < end; ++r, h += a.N, y += a.N) {
    if (kShared && static_cast<uint64_t>(r) >= static_cast<uint64_t>(stall.at)) share.silence();
    const unsigned char* stage = ring.next();
    refill = first && r > begin;  // behind the row's first sum the group has read the row before
    if (!kRowGate && r >= gate_end) {
      const int64_t g = static_cast<uint32_t>(r) / per_gate;
      gate_end = (g + 1) * per_gate;
      const char* gate = static_cast<const char*>(a.gate) + g * a.N * (gate32 ? 4 : sizeof(T));
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (in + i * G >= mine) continue;
        float2 post[P];
        load_weights<T, false>(gate, (n0 + in + i * G) * E, a.N, gate32, 1.0f, q[i]);
        load_weights<T, false>(a.gamma_post, (n0 + in + i * G) * E, a.N, f32, 1.0f, post);
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
        const Raw u = ld_stage(stage + (in + i * G) * 16);
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
      w[i] = ld_stage(stage + (in + i * G) * 16);
      Raw res = {};
      if (add) res = ld_stage(stage + (R * G + in + i * G) * 16);
      float2 gate[P];
      if constexpr (kRowGate) stage_pairs<T>(stage + 2 * R * G * 16, in + i * G, gate32, gate);
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
      if (kFull || a.h != nullptr) st_raw(h + i * G * E, w[i]);
    }
    if (pre_norm) {
      rh = rstd_of(s2);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (in + i * G >= mine) continue;
#pragma unroll
        for (int e = 0; e < P; ++e)
          set_pair<T>(w[i], e, __fmul2_rn(get_pair<T>(w[i], e), __fmul2_rn(pair(rh), pre[i][e])));
        st_raw(y + i * G * E, w[i]);
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

// Backward over a ring, R vectors of a row a thread. The gate row is the chunk's own (kRowGate: one more tensor in the
// ring), so that its columns and gamma_post's are one factor in registers.
constexpr int kBwdBlock = 256, kBwdBlocks = 2;  // threads of a block, at most, and such blocks an SM
template <typename T, int R, bool kShared, bool kRowGate, bool kFull>
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
  const int n = static_cast<int>(a.N) / E, n0 = rank * R * G, mine = min(R * G, n - n0);
  const bool first = in == 0;
  const float inv_n = 1.0f / static_cast<float>(a.N);
  const bool post_norm = kFull || a.post, pre_norm = kFull || a.pre, add = kFull || a.dh != nullptr;
  const bool f32 = a.wdtype == 0, gate32 = a.gdtype == 0, dgate_rows = kRowGate && a.dgate != nullptr;
  auto column = [&](int i) { return (n0 + in + i * G) * E; };
  Ring<kTensors> ring(dyn, bars, plan, group, stall);
  if (first) {
    ring.init();
    fence_mbar_init();
  }
  __syncthreads();
  WarpRows sums(smem, G);
  std::conditional_t<kShared, ClusterSum3, NoSum3> share(slots, S, stall);
  const int64_t stop_at = kShared ? -1 : stall.at;
  // the rows of the group's chunks in turn: chunk c, rows r .. end - 1
  struct Walk {  // 32 bits hold them: at most as many chunks as rows
    uint32_t c, r, end;
  };
  const uint32_t chunks = static_cast<uint32_t>(k.chunks), per_segment = static_cast<uint32_t>(k.per_segment);
  const uint32_t segment = static_cast<uint32_t>(k.segment), chunk_rows = static_cast<uint32_t>(k.rows);
  auto enter = [&](Walk& w) {
    const uint32_t seg = w.c / per_segment;
    w.r = seg * segment + (w.c - seg * per_segment) * chunk_rows;
    w.end = min((seg + 1) * segment, w.r + chunk_rows);
  };
  Walk ahead{unit, 0, 0};
  if (ahead.c < chunks) enter(ahead);
  auto issue = [&]() {
    if (ahead.c >= chunks) return;
    const int64_t r = ahead.r;
    const void* from[kTensors];
    uint32_t bytes[kTensors];
    from[0] = static_cast<const T*>(a.u) + r * a.ldu + n0 * E;
    from[1] = pre_norm ? static_cast<const T*>(a.h) + r * a.ldh + n0 * E : nullptr;
    from[2] = pre_norm ? static_cast<const T*>(a.dy) + r * a.lddy + n0 * E : nullptr;
    from[3] = add ? static_cast<const T*>(a.dh) + r * a.lddh + n0 * E : nullptr;
#pragma unroll
    for (int i = 0; i < 4; ++i) bytes[i] = static_cast<uint32_t>(mine) * 16u;
    if constexpr (kRowGate) {
      const int64_t es = gate32 ? 4 : sizeof(T);
      from[4] = static_cast<const char*>(a.gate) + (r * a.N + n0 * E) * es;
      bytes[4] = static_cast<uint32_t>(mine) * static_cast<uint32_t>(E * es);
    }
    ring.issue(from, bytes, R * G * 16, stop_at);
    if (++ahead.r == ahead.end) {
      ahead.c += units;
      if (ahead.c < chunks) enter(ahead);
    }
  };
  if (first)
    for (int i = 0; i < ring.stages; ++i) issue();
  float2 pre[R][P], post[R][P];  // gamma_pre; gamma_post, without kRowGate times the gate
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (in + i * G < mine) load_weights<T, false>(a.gamma_pre, column(i), a.N, f32, 1.0f, pre[i]);
  bool refill = false;
  struct Vectors {  // a thread's vector of each tensor, from the stage
    Raw u, h, dy, dh;
  };
  auto vectors = [&](const unsigned char* stage, int i) {
    Vectors v = {};
    const unsigned char* p = stage + (in + i * G) * 16;
    v.u = ld_stage(p);
    if (pre_norm) {
      v.h = ld_stage(p + R * G * 16);
      v.dy = ld_stage(p + 2 * R * G * 16);
    }
    if (add) v.dh = ld_stage(p + 3 * R * G * 16);
    return v;
  };
  for (Walk w{unit, 0, 0}; w.c < chunks; w.c += units) {
    enter(w);
    float2 ss[R][P], sp[R][P];
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int e = 0; e < P; ++e) ss[i][e] = sp[i][e] = pair(0.0f);
      if (in + i * G >= mine) continue;
      load_weights<T, false>(a.gamma_post, column(i), a.N, f32, 1.0f, post[i]);
      if (!kRowGate && a.gate != nullptr) {
        float2 g[P];
        const int64_t row = static_cast<uint32_t>(w.r) / static_cast<uint32_t>(a.rows_per_gate);
        load_weights<T, false>(static_cast<const char*>(a.gate) + row * a.N * (gate32 ? 4 : sizeof(T)), column(i), a.N,
                               gate32, 1.0f, g);
#pragma unroll
        for (int e = 0; e < P; ++e) post[i][e] = __fmul2_rn(g[e], post[i][e]);
      }
    }
    auto rstds = [&](uint32_t r) {  // 4-byte aligned
      const float* p = a.stats + 2 * static_cast<int64_t>(r);
      return make_float2(p[0], p[1]);
    };
    float2 stats = rstds(w.r);
    int64_t at = static_cast<int64_t>(w.r) * a.N + column(0);
    for (uint32_t r = w.r; r < w.end; ++r) {
      if (kShared && static_cast<uint64_t>(r) >= static_cast<uint64_t>(stall.at)) share.silence();
      const float fu = post_norm ? stats.x : 1.0f, fh = pre_norm ? stats.y : 0.0f;
      if (r + 1 < w.end) stats = rstds(r + 1);
      const unsigned char* stage = ring.next();
      const float2 rh = pair(fh);
      // sums of dy gamma_pre h, of q u (dh + rstd(h) dy gamma_pre) and of q u h: the rows' factors come behind them
      float2 s0 = pair(0.0f), s1 = s0, s2 = s0;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (in + i * G >= mine) continue;
        const Vectors v = vectors(stage, i);
        float2 q[P];
        if constexpr (kRowGate) stage_pairs<T>(stage + 4 * R * G * 16, in + i * G, gate32, q);
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
        if (in + i * G >= mine) continue;
        Vectors x = vectors(stage, i);
        float2 q[P];
        if constexpr (kRowGate) stage_pairs<T>(stage + 4 * R * G * 16, in + i * G, gate32, q);
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
            if (gate32 && dgate_rows) *reinterpret_cast<float2*>(static_cast<float*>(a.dgate) + (at + i * G * E) + 2 * e) = v;
            else set_pair<T>(dg, e, v);
          } else {
            ss[i][e] = __ffma2_rn(d, uh, ss[i][e]);
          }
          set_pair<T>(x.dh, e, __fmul2_rn(pair(a.alpha), d));
          const float2 v = __ffma2_rn(uh, c2, qd);
          set_pair<T>(x.u, e, post_norm ? __fmul2_rn(ru, v) : v);
        }
        st_raw(static_cast<T*>(a.du) + at + i * G * E, x.u);
        if (kFull || a.dres != nullptr) st_raw(static_cast<T*>(a.dres) + at + i * G * E, x.dh);
        if (dgate_rows && !gate32) st_raw(static_cast<T*>(a.dgate) + at + i * G * E, dg);
      }
      at += a.N;
    }
    if (a.part == nullptr) continue;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (in + i * G >= mine) continue;
      float* to = a.part + static_cast<int64_t>(w.c) * 2 * a.N + column(i);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        *reinterpret_cast<float2*>(to + 2 * e) = ss[i][e];
        *reinterpret_cast<float2*>(to + a.N + 2 * e) = sp[i][e];
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
// Rows shared by a cluster: S blocks of G threads, R vectors each
struct Shared {
  int S, G;
};
Shared share_row(int64_t n, int R) {
  const int64_t threads = (n + R - 1) / R;
  const int S = static_cast<int>(threads <= kMaxCluster * kBlock ? (threads + kBlock - 1) / kBlock : kMaxCluster);
  return Shared{S, static_cast<int>((threads + 32 * S - 1) / (32 * S)) * 32};
}

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
cudaError_t fwd_long(const BnFwdArgs& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.M, 65536));
  bn_fwd_long_kernel<T><<<grid, kMaxThreads, 0, stream>>>(a);
  return cudaGetLastError();
}
// The ring of a group: as many rows of `row` bytes as fit beside one another in the memory of `blocks` blocks an SM,
// `groups` groups each.
constexpr int64_t kRingMemory = 220 * 1024;  // of an SM's 228 KB: what is static and 1 KB a block stay free
RingPlan ring_plan(int64_t row, int blocks, int groups) {
  const int64_t fit = kRingMemory / blocks / groups / row;
  RingPlan p;
  p.stages = static_cast<int>(std::min<int64_t>(kMaxStages, fit));
  p.stage_bytes = static_cast<int>(row);
  p.group_bytes = p.stages * p.stage_bytes;
  return p;
}
// Rows from which on a group's ring pays: below, the first rows' copies cost more than loads (1 to 2 us).
constexpr int64_t kRingRows = 4;

// bytes of a row of a gate for each row, in those of the row itself
template <typename T>
int64_t gate_slots(int gdtype) {
  return gdtype == 0 ? 4 / sizeof(T) : 1;
}
template <typename T, bool kRowGate, bool kFull>
cudaError_t fwd_ring_one(const BnFwdArgs& a, int64_t n, cudaStream_t stream) {
  const auto kernel = bn_fwd_ring_kernel<T, 2, false, kRowGate, kFull>;
  const int G = group_threads(n, 2), groups = G < kBlock ? kBlock / G : 1, block = groups * G;
  const RingPlan p = ring_plan((2 + (kRowGate ? gate_slots<T>(a.gdtype) : 0)) * 2 * G * 16,
                               std::max(1, kFwdRingBlocks<kRowGate> * kBlock / block), groups);
  const size_t smem = static_cast<size_t>(groups) * p.group_bytes;
  int64_t blocks;
  {
    static std::mutex mu;
    static FitCache cache;
    std::lock_guard<std::mutex> lk(mu);
    const cudaError_t e = blocks_that_fit(kernel, cache, block, smem, blocks);
    if (e != cudaSuccess) return e;
  }
  blocks = std::min(blocks, (a.M + groups - 1) / groups);
  kernel<<<static_cast<unsigned>(blocks), block, smem, stream>>>(a, p, G, 1, take_stall(kInjectBlockNormFwd),
                                                                status_word_ptr());
  return cudaGetLastError();
}
template <typename T, bool kRowGate, bool kFull>
cudaError_t fwd_ring_shared(const BnFwdArgs& a, int64_t n, cudaStream_t stream) {
  const auto kernel = bn_fwd_ring_kernel<T, 2, true, kRowGate, kFull>;
  const Shared s = share_row(n, 2);
  const RingPlan p = ring_plan((2 + (kRowGate ? gate_slots<T>(a.gdtype) : 0)) * 2 * s.G * 16,
                               std::max(1, kFwdRingBlocks<kRowGate> * kBlock / s.G), 1);
  static std::mutex mu;
  static StreamCache cache;
  std::lock_guard<std::mutex> lk(mu);
  const cudaError_t e = clusters_that_fit(kernel, cache, s.G, p.group_bytes, s.S);
  if (e != cudaSuccess) return e;
  if (cache.clusters < 1) return fwd_long<T>(a, stream);
  ClusterLaunch l(s.G, p.group_bytes, s.S, std::min<int64_t>(cache.clusters, a.M), stream);
  return cudaLaunchKernelEx(&l.cfg, kernel, a, p, s.G, s.S, take_stall(kInjectBlockNormFwd), status_word_ptr());
}

template <typename T, bool kRowGate, bool kFull>
cudaError_t fwd_ring(const BnFwdArgs& a, int64_t n, cudaStream_t stream) {
  return n <= 2 * kBlock ? fwd_ring_one<T, kRowGate, kFull>(a, n, stream)
                         : fwd_ring_shared<T, kRowGate, kFull>(a, n, stream);
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
  if (!kRagged && n <= 2 * kMaxCluster * kBlock) {
    if (a.M * ((n + 1) / 2) >= kRingRows * kFwdBlocks * kBlock * device_sm_count()) {
      const bool row_gate = a.gate != nullptr && a.rows_per_gate == 1, full = a.post && a.pre && a.residual != nullptr;
      if (row_gate) return full ? fwd_ring<T, true, true>(a, n, stream) : fwd_ring<T, true, false>(a, n, stream);
      return full ? fwd_ring<T, false, true>(a, n, stream) : fwd_ring<T, false, false>(a, n, stream);
    }
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
template <typename T, bool kRowGate, bool kFull>
cudaError_t bwd_ring_one(const BnBwdArgs& a, const BnChunks& k, int64_t n, cudaStream_t stream) {
  const auto kernel = bn_bwd_ring_kernel<T, 2, false, kRowGate, kFull>;
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
  return cudaGetLastError();
}
template <typename T, bool kRowGate, bool kFull>
cudaError_t bwd_ring_shared(const BnBwdArgs& a, const BnChunks& k, int64_t n, cudaStream_t stream) {
  const auto kernel = bn_bwd_ring_kernel<T, 2, true, kRowGate, kFull>;
  const Shared s = share_row(n, 2);
  const RingPlan p = ring_plan((4 + (kRowGate ? gate_slots<T>(a.gdtype) : 0)) * 2 * s.G * 16,
                               std::max(kBwdBlocks, kBwdBlocks * kBwdBlock / s.G), 1);
  static std::mutex mu;
  static StreamCache cache;
  std::lock_guard<std::mutex> lk(mu);
  const cudaError_t e = clusters_that_fit(kernel, cache, s.G, p.group_bytes, s.S);
  if (e != cudaSuccess) return e;
  if (cache.clusters < 1) return cudaErrorLaunchOutOfResources;
  ClusterLaunch l(s.G, p.group_bytes, s.S, std::min<int64_t>(cache.clusters, k.chunks), stream);
  return cudaLaunchKernelEx(&l.cfg, kernel, a, k, p, s.G, s.S, take_stall(kInjectBlockNormBwd), status_word_ptr());
}
template <typename T, bool kRowGate, bool kFull>
cudaError_t bwd_ring(const BnBwdArgs& a, const BnChunks& k, int64_t n, cudaStream_t stream) {
  const cudaError_t e = n <= 2 * kBwdBlock ? bwd_ring_one<T, kRowGate, kFull>(a, k, n, stream)
                                           : bwd_ring_shared<T, kRowGate, kFull>(a, k, n, stream);
  return e != cudaSuccess || a.part == nullptr ? e : launch_reduce(a, k, stream);
}
template <typename T, bool kRagged>
cudaError_t bwd_any(const BnBwdArgs& a, cudaStream_t stream) {
  const int64_t n = (a.N + (kRagged ? 2 * kElems<T> - 2 : 0)) / kElems<T>;
  if (!kRagged && n > 32 && n <= 2 * kMaxCluster * kBwdBlock) {
    const int64_t units = ring_units(n);
    if (a.M >= kRingRows * units) {
      const BnChunks k = chunks_of(a.M, a.rows_per_gate, units, 1);
      const bool row_gate = a.gate != nullptr && a.rows_per_gate == 1;
      const bool full = a.post && a.pre && a.dh != nullptr && a.dres != nullptr;
      if (row_gate) return full ? bwd_ring<T, true, true>(a, k, n, stream) : bwd_ring<T, true, false>(a, k, n, stream);
      return full ? bwd_ring<T, false, true>(a, k, n, stream) : bwd_ring<T, false, false>(a, k, n, stream);
    }
  }
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
      if (!ragged) most = std::max(most, chunks_of(M, rows_per_gate, ring_units(n), 1).chunks);
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
