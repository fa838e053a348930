// Layer norm over the last dimension, forward and backward.
//   h = x + r rounded to the I/O type (h = x without a residual r)
//   mu = sum h / N,  var = sum (h - mu)^2 / N,  rstd = 1 / sqrt(var + eps)
//   y = (h - mu) rstd gamma + beta
// Backward, with x_hat = (h - mu) rstd and g = dy gamma, from the saved (mu, rstd):
//   dx = rstd (g - mean(g) - x_hat mean(g x_hat)) (+ dh, the gradient that reaches h by another path)
//   dgamma = sum over rows of dy x_hat,  dbeta = sum over rows of dy
// All arithmetic is fp32; h, y and dx are rounded once.
//
// Bound by HBM: two to four tensors of M N elements are read or written, with some ten operations an
// element. A group of 8 to 512 threads holds a row in registers, one or two 16-byte vectors of fixed columns
// a thread, so each element is read once: the variance is taken of centred values in a second pass over the
// registers. The groups are persistent and load a row ahead. Rows of more than 1024 vectors are shared by a
// cluster of blocks, which send one another their sums (st.async, counted by an mbarrier). Only rows above
// 8192 vectors (ragged ones forward: 4096) are read again (ln_fwd_long_kernel, ln_dx_long_kernel).
// Ragged rows, that begin or end inside 16 bytes: a thread's columns are those of a 16-byte vector of the
// output, so that its stores are aligned. A group takes rows that lie a multiple of 16 bytes apart: it keeps
// its columns, and the weights and the column sums that belong to them, in registers. An input with the same
// offset is loaded as aligned vectors too, the row's first and last one with elements of the neighbours,
// that are cleared; with another offset it is put together from two. Element by element (groups of one
// column a lane) took 78 us for 4000 x 4001 bf16 forward and 164 us backward, this takes 33 and 53.
// Backward: the columns' sums of dgamma and dbeta stay in registers over all of a group's rows. The blocks'
// sums go to the workspace and are added by a second kernel in a fixed order.
// Measured, bf16: 16384 x 4096 with residual 87 us, 92% of the copy bandwidth; backward with dh 220000 x 512
// 146 us, 92%, 16384 x 4096 94 us, 85%, 65536 x 4096 344 us, 93%.
#include <algorithm>
#include <cmath>
#include <mutex>
#include <numeric>
#include <type_traits>

#include "row_vectors.cuh"

namespace swg {
namespace {

using namespace row;

constexpr int kBlock = 256;         // threads of a block, unless a row takes more
constexpr int kMaxGroup = 512;      // threads of a group, and of a block
constexpr int kMaxThreads = 1024;   // of the kernels for longest rows

// ---- forward
// kShared: the S blocks of a cluster, of one group each, share a row. 80 registers a thread keep three blocks
// of 256 threads on an SM (96: 97 us instead of 87 for 16384 x 4096 bf16 with residual; 64: 91 us).
template <bool kRagged>
constexpr int kFwdRegs = kRagged ? 128 : 80;
template <typename T, int R, bool kRagged, bool kShared>
__global__ void __maxnreg__(kFwdRegs<kRagged>)
    ln_fwd_kernel(const LnFwdArgs a, int G, int S, Stall stall, uint32_t* status) {
  __shared__ float smem[2 * 32];
  __shared__ ClusterSlots slots;
  constexpr int E = kElems<T>, P = kPairs<T>;
  constexpr bool kNarrow = R == 1;  // groups of less than a warp
  const int groups = kShared ? 1 : blockDim.x / G;
  const int t = kShared ? threadIdx.x + cluster_ctarank() * R * G : threadIdx.x % G;  // vectors t, t + G, ...
  const int64_t step = static_cast<int64_t>(kShared ? gridDim.x / S : gridDim.x) * groups;
  const int N = static_cast<int>(a.N);
  int64_t r = kShared ? blockIdx.x / S : static_cast<int64_t>(blockIdx.x) * groups + threadIdx.x / G;
  const int shift = kRagged ? shift_of(static_cast<const T*>(a.y) + r * a.N) : 0;
  int n = (N + shift + E - 1) / E;  // vectors of the row
  const bool add = a.residual != nullptr, f32 = a.wdtype == 0;
  const float inv_n = 1.0f / static_cast<float>(a.N);
  auto column = [&](int i) { return (t + i * G) * E - shift; };
  struct Row {
    Raw x[R], res[R];
  };
  const Rows<T> x(a.x, a.ldx, a.M, a.N), res(a.residual, a.ldr, a.M, a.N);
  auto load = [&](Row& w, int64_t r) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (t + i * G >= n) continue;
      w.x[i] = load_columns<T, kRagged>(x, r, column(i), N);
      if (add) w.res[i] = load_columns<T, kRagged>(res, r, column(i), N);
    }
  };
  constexpr bool kHeld = kRagged;  // the weights: those of ragged columns take several loads and a join
  float2 gam[kHeld ? R : 1][P], bet[kHeld ? R : 1][P];
  auto weights = [&](int i, int to) {
    load_weights<T, kRagged>(a.gamma, column(i), N, f32, 1.0f, gam[to]);
    load_weights<T, kRagged>(a.beta, column(i), N, f32, 0.0f, bet[to]);
  };
  if constexpr (kHeld) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (t + i * G < n) weights(i, i);
  }
  GroupSum<1, kNarrow> sum(smem, G);
  SharedSum<kShared, 1> join(slots, S, stall);
  Row next;
  const int64_t M = a.M + (kNarrow ? (threadIdx.x & 31) / G : 0);  // the rows of a warp's groups end together
  if (r < a.M) load(next, r);
  for (; r < M; r += step) {
    if (kNarrow && r >= a.M) n = 0;
    if (kShared && static_cast<uint64_t>(r) >= static_cast<uint64_t>(stall.at)) join.silence();
    Row w = next;
    if (r + step < a.M) load(next, r + step);
    if constexpr (kRagged) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        clear_others<T>(w.x[i], column(i), N);
        if (add) clear_others<T>(w.res[i], column(i), N);
      }
    }
    float2 s2 = pair(0.f), f[R][P];  // the row in fp32
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (t + i * G >= n) continue;
      if (add) {
#pragma unroll
        for (int e = 0; e < P; ++e)  // h as it is stored
          set_pair<T>(w.x[i], e, __fadd2_rn(get_pair<T>(w.x[i], e), get_pair<T>(w.res[i], e)));
        store_columns<T, kRagged>(static_cast<T*>(a.h) + r * a.N, column(i), N, w.x[i]);
      }
#pragma unroll
      for (int e = 0; e < P; ++e) {
        f[i][e] = get_pair<T>(w.x[i], e);
        s2 = __fadd2_rn(s2, f[i][e]);
      }
    }
    float s[1] = {s2.x + s2.y};
    sum(s);
    join(s);
    const float mu = s[0] * inv_n;
    const float2 nmu = pair(-mu);
    s2 = pair(0.f);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (t + i * G >= n) continue;
      if (kRagged && (column(i) < 0 || column(i) + E > N)) {
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const int j = column(i) + 2 * e;
          const float2 d = __fadd2_rn(f[i][e], nmu);
          s2 = __ffma2_rn(d, make_float2(j >= 0 && j < N ? d.x : 0.0f, j >= -1 && j + 1 < N ? d.y : 0.0f), s2);
        }
        continue;
      }
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float2 d = __fadd2_rn(f[i][e], nmu);
        s2 = __ffma2_rn(d, d, s2);
      }
    }
    s[0] = s2.x + s2.y;
    sum(s);
    join(s);
    const float rstd = rsqrtf(fmaf(s[0], inv_n, a.eps));
    const float2 scale = pair(rstd);
    T* y = static_cast<T*>(a.y) + r * a.N;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (t + i * G >= n) continue;
      constexpr int k = kHeld ? 1 : 0;
      if (!kHeld) weights(i, 0);
#pragma unroll
      for (int e = 0; e < P; ++e)
        set_pair<T>(w.x[i], e,
                    __ffma2_rn(__fmul2_rn(__fadd2_rn(f[i][e], nmu), scale), gam[k * i][e], bet[k * i][e]));
      store_columns<T, kRagged>(y, column(i), N, w.x[i]);
    }
    if (t == 0 && (!kNarrow || n > 0)) {
      a.stats[2 * r] = mu;
      a.stats[2 * r + 1] = rstd;
    }
  }
  join.end(status);
}

// rows of any length, element by element, read three times (from L2 where a row fits)
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) ln_fwd_long_kernel(const LnFwdArgs a) {
  __shared__ float buf[32];
  const float inv_n = 1.0f / static_cast<float>(a.N);
  for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    const T* res = a.residual != nullptr ? static_cast<const T*>(a.residual) + r * a.ldr : nullptr;
    T* h = a.h != nullptr ? static_cast<T*>(a.h) + r * a.N : nullptr;
    T* y = static_cast<T*>(a.y) + r * a.N;
    auto value = [&](int64_t j) {  // h_j, rounded as it is stored
      return res == nullptr ? to_f(x[j]) : to_f(from_f<T>(to_f(x[j]) + to_f(res[j])));
    };
    float s[1];
    long_sums(a.N, s, [&](float (&p)[1], int64_t j) { p[0] += value(j); });
    const float mu = block_sum(s[0], buf) * inv_n;
    long_sums(a.N, s, [&](float (&p)[1], int64_t j) {
      const float d = value(j) - mu;
      p[0] = fmaf(d, d, p[0]);
    });
    const float rstd = rsqrtf(fmaf(block_sum(s[0], buf), inv_n, a.eps));
    for (int64_t j = threadIdx.x; j < a.N; j += blockDim.x) {
      const float v = value(j);
      const float g = a.gamma != nullptr ? load_any(a.gamma, j, a.wdtype) : 1.0f;
      const float b = a.beta != nullptr ? load_any(a.beta, j, a.wdtype) : 0.0f;
      y[j] = from_f<T>(fmaf((v - mu) * rstd, g, b));
      if (h != nullptr) h[j] = from_f<T>(v);
    }
    if (threadIdx.x == 0) {
      a.stats[2 * r] = mu;
      a.stats[2 * r + 1] = rstd;
    }
  }
}

// ---- backward
// dx, and with a.part the block's column sums: part[block][0][j] of dy x_hat, part[block][1][j] of dy.
// kFold: a thread's column sums go to slots of its own in shared memory every `fold` rows. Terms that are much
// alike are rounded the same way, so that one accumulator over n rows may be off by n / 2 ulp: 264000 equal rows
// of 8192 (1737 a group) gave weight gradients off by 2.6e-5, with a fold every 128 rows 2.1e-6. It costs -3 to
// +1% (100000 x 8192 bf16 1044 us, 1057 without; ragged rows of a cluster +5%) where whole rows end a run before
// it and ragged ones go on; with either form for both the registers do not suffice (100000 x 2001 fp32 797 us
// instead of 559). Rows are counted in 32 bits for the same reason.
template <typename T, int R, bool kRagged, bool kShared, bool kFold>
__global__ void __launch_bounds__(kMaxGroup)
    ln_bwd_kernel(const LnBwdArgs a, int G, int S, int fold, Stall stall, uint32_t* status) {
  extern __shared__ __align__(16) float dyn[];  // the slots; then, with several groups a block, 2 N column sums
  __shared__ float smem[2 * 2 * 32];
  __shared__ ClusterSlots slots;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int E = kElems<T>, P = kPairs<T>;
  constexpr bool kNarrow = R == 1;  // groups of less than a warp
  const int groups = kShared ? 1 : blockDim.x / G, group = kShared ? 0 : threadIdx.x / G;
  const int t = kShared ? threadIdx.x + cluster_ctarank() * R * G : threadIdx.x % G;  // vectors t, t + G, ...
  using Index = std::conditional_t<kFold, uint32_t, int64_t>;  // of rows
  const Index unit = kShared ? blockIdx.x / S : blockIdx.x;
  const int N = static_cast<int>(a.N);
  Index r = unit * groups + group;
  const int shift = kRagged ? shift_of(static_cast<const T*>(a.dx) + static_cast<int64_t>(r) * a.N) : 0;
  const int vectors = (N + shift + E - 1) / E;
  int n = vectors;
  const Index step = static_cast<Index>(kShared ? gridDim.x / S : gridDim.x) * groups;
  const float inv_n = 1.0f / static_cast<float>(a.N);
  const bool add = a.dh != nullptr, f32 = a.wdtype == 0;
  auto column = [&](int i) { return (t + i * G) * E - shift; };
  float2 gam[R][P], sg[R][P], sb[R][P];
#pragma unroll
  for (int i = 0; i < R; ++i) {
#pragma unroll
    for (int e = 0; e < P; ++e) sg[i][e] = sb[i][e] = pair(0.0f);
    if (t + i * G < n) load_weights<T, kRagged>(a.gamma, column(i), N, f32, 1.0f, gam[i]);
  }
  struct Row {
    Raw x[R], dy[R], dh[R];
    float mu, rstd;
  };
  const Rows<T> x(a.x, a.ldx, a.M, a.N), dy(a.dy, a.lddy, a.M, a.N), dh(a.dh, a.lddh, a.M, a.N);
  auto load = [&](Row& w, int64_t r) {
    w.mu = a.stats[2 * r];
    w.rstd = a.stats[2 * r + 1];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (t + i * G >= n) continue;
      w.x[i] = load_columns<T, kRagged>(x, r, column(i), N);
      w.dy[i] = load_columns<T, kRagged>(dy, r, column(i), N);
      if (add) w.dh[i] = load_columns<T, kRagged>(dh, r, column(i), N);
    }
  };
  GroupSum<2, kNarrow> sum(smem, G);
  SharedSum<kShared, 2> join(slots, S, stall);
  auto slot = [&](int i, int e) -> float4& {  // of pair e of the thread's vector i
    return reinterpret_cast<float4*>(dyn)[(i * P + e) * blockDim.x + threadIdx.x];
  };
  if (kFold) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int e = 0; e < P; ++e) slot(i, e) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  const Index rows = a.M;
  const Index M = rows + (kNarrow ? (threadIdx.x & 31) / G : 0);  // the rows of a warp's groups end together
  auto to_slots = [&]() {
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float4 o = slot(i, e);
        slot(i, e) = make_float4(o.x + sg[i][e].x, o.y + sg[i][e].y, o.z + sb[i][e].x, o.w + sb[i][e].y);
        sg[i][e] = sb[i][e] = pair(0.0f);
      }
    }
  };
  constexpr bool kRuns = kFold && !kRagged;
  int left = fold;
#pragma unroll 1
  do {
    const Index stop = kRuns ? min(M, r + fold * step) : M;
    Row next;
    if (r < rows) load(next, r);
    for (; r < stop; r += step) {
      if (kNarrow && r >= rows) n = 0;
      if (kShared && static_cast<uint64_t>(r) >= static_cast<uint64_t>(stall.at)) join.silence();
      Row w = next;
      if ((!kRuns || r + step < stop) && ((kRuns && !kNarrow) || r + step < rows)) load(next, r + step);
      if constexpr (kRagged) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          clear_others<T>(w.x[i], column(i), N);
          clear_others<T>(w.dy[i], column(i), N);
        }
      }
      const float2 nmu = pair(-w.mu), rstd = pair(w.rstd);
      float2 s0 = pair(0.f), s1 = s0;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (t + i * G >= n) continue;
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float2 xh = __fmul2_rn(__fadd2_rn(get_pair<T>(w.x[i], e), nmu), rstd), d = get_pair<T>(w.dy[i], e);
          const float2 g = __fmul2_rn(d, gam[i][e]);
          sg[i][e] = __ffma2_rn(d, xh, sg[i][e]);
          sb[i][e] = __fadd2_rn(sb[i][e], d);
          s0 = __fadd2_rn(s0, g);
          s1 = __ffma2_rn(g, xh, s1);
        }
      }
      float s[2] = {s0.x + s0.y, s1.x + s1.y};  // columns behind the row have dy = 0
      sum(s);
      join(s);
      // dx = rstd (g - mean(g) - x_hat mean(g x_hat))
      const float2 c0 = pair(-s[0] * inv_n * w.rstd), c1 = pair(-s[1] * inv_n * w.rstd);
      T* dx = static_cast<T*>(a.dx) + static_cast<int64_t>(r) * a.N;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (t + i * G >= n) continue;
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float2 xh = __fmul2_rn(__fadd2_rn(get_pair<T>(w.x[i], e), nmu), rstd);
          float2 v = __ffma2_rn(__fmul2_rn(get_pair<T>(w.dy[i], e), gam[i][e]), rstd, __ffma2_rn(xh, c1, c0));
          if (add) v = __fadd2_rn(v, get_pair<T>(w.dh[i], e));
          set_pair<T>(w.x[i], e, v);
        }
        store_columns<T, kRagged>(dx, column(i), N, w.x[i]);
      }
      if (kFold && !kRuns && --left == 0) {
        to_slots();
        left = fold;
      }
    }
    if (kRuns) to_slots();
  } while (kRuns && r < M);
  if (kFold && !kRuns) to_slots();
  join.end(status);
  if (a.part == nullptr) return;
  if (kFold) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float4 o = slot(i, e);
        sg[i][e] = make_float2(o.x, o.y);
        sb[i][e] = make_float2(o.z, o.w);
      }
    }
    __syncthreads();  // the slots' place is written anew
  }
  // the block's sums, one group after the other: a fixed order. Groups of less than a warp with the same
  // columns are added first.
  const bool merge = !kRagged && kNarrow && G < 32;
  if (merge) {
    for (int o = 16; o >= G; o >>= 1) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int e = 0; e < P; ++e) {
          sg[i][e].x += __shfl_xor_sync(0xffffffffu, sg[i][e].x, o);
          sg[i][e].y += __shfl_xor_sync(0xffffffffu, sg[i][e].y, o);
          sb[i][e].x += __shfl_xor_sync(0xffffffffu, sb[i][e].x, o);
          sb[i][e].y += __shfl_xor_sync(0xffffffffu, sb[i][e].y, o);
        }
      }
    }
  }
  const int wide = merge ? 32 : G, parts = kShared ? 1 : blockDim.x / wide;
  float* part = a.part + static_cast<int64_t>(unit) * 2 * a.N;
  float* to = parts > 1 ? dyn : part;
  for (int k = 0; k < parts; ++k) {
    if (k == static_cast<int>(threadIdx.x) / wide && static_cast<int>(threadIdx.x) % wide < G) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (t + i * G >= vectors) continue;
        if constexpr (!kRagged) {  // 16 bytes at a time: 2N and the columns are multiples of 4
#pragma unroll
          for (int e = 0; e < P; e += 2) {
            float4* dg = reinterpret_cast<float4*>(to + column(i) + 2 * e);
            float4* db = reinterpret_cast<float4*>(to + N + column(i) + 2 * e);
            float4 vg = make_float4(sg[i][e].x, sg[i][e].y, sg[i][e + 1].x, sg[i][e + 1].y);
            float4 vb = make_float4(sb[i][e].x, sb[i][e].y, sb[i][e + 1].x, sb[i][e + 1].y);
            if (k > 0) {
              const float4 og = *dg, ob = *db;
              vg = make_float4(og.x + vg.x, og.y + vg.y, og.z + vg.z, og.w + vg.w);
              vb = make_float4(ob.x + vb.x, ob.y + vb.y, ob.z + vb.z, ob.w + vb.w);
            }
            *dg = vg;
            *db = vb;
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int j = column(i) + e;
            if (j < 0 || j >= N) continue;
            const float vg = e % 2 == 0 ? sg[i][e / 2].x : sg[i][e / 2].y;
            const float vb = e % 2 == 0 ? sb[i][e / 2].x : sb[i][e / 2].y;
            to[j] = k == 0 ? vg : to[j] + vg;
            to[N + j] = k == 0 ? vb : to[N + j] + vb;
          }
        }
      }
    }
    if (parts > 1) __syncthreads();
  }
  if (parts > 1)
    for (int j = threadIdx.x; j < 2 * N; j += blockDim.x) part[j] = dyn[j];
}

// rows of any length, element by element
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) ln_dx_long_kernel(const LnBwdArgs a) {
  __shared__ float buf[32];
  const float inv_n = 1.0f / static_cast<float>(a.N);
  for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + r * a.lddy;
    const T* dh = a.dh != nullptr ? static_cast<const T*>(a.dh) + r * a.lddh : nullptr;
    T* dx = static_cast<T*>(a.dx) + r * a.N;
    const float mu = a.stats[2 * r], rstd = a.stats[2 * r + 1];
    float s[2];
    long_sums(a.N, s, [&](float (&p)[2], int64_t j) {
      const float g = to_f(dy[j]) * (a.gamma != nullptr ? load_any(a.gamma, j, a.wdtype) : 1.0f);
      p[0] += g;
      p[1] = fmaf(g, (to_f(x[j]) - mu) * rstd, p[1]);
    });
    const float c0 = -block_sum(s[0], buf) * inv_n * rstd, c1 = -block_sum(s[1], buf) * inv_n * rstd;
    for (int64_t j = threadIdx.x; j < a.N; j += blockDim.x) {
      const float g = to_f(dy[j]) * (a.gamma != nullptr ? load_any(a.gamma, j, a.wdtype) : 1.0f);
      const float v = fmaf(g, rstd, fmaf((to_f(x[j]) - mu) * rstd, c1, c0));
      dx[j] = from_f<T>(dh != nullptr ? v + to_f(dh[j]) : v);
    }
  }
}
// one row chunk's column sums, for rows of any length
constexpr int kColThreads = 128;
template <typename T, bool kFold>  // kFold: as in ln_bwd_kernel
__global__ void __launch_bounds__(kColThreads) ln_param_long_kernel(const LnBwdArgs a, int64_t rows_per_chunk,
                                                                   int fold) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kColThreads + threadIdx.x;
  if (j >= a.N) return;
  const int64_t r0 = blockIdx.y * rows_per_chunk, r1 = min(a.M, r0 + rows_per_chunk);
  float sg = 0.f, sb = 0.f, all_g = 0.f, all_b = 0.f;
  int left = fold;
  for (int64_t r = r0; r < r1; ++r) {
    const float d = to_f(static_cast<const T*>(a.dy)[r * a.lddy + j]);
    const float xh = (to_f(static_cast<const T*>(a.x)[r * a.ldx + j]) - a.stats[2 * r]) * a.stats[2 * r + 1];
    sg = fmaf(d, xh, sg);
    sb += d;
    if (kFold && --left == 0) {
      all_g += sg;
      all_b += sb;
      sg = sb = 0.f;
      left = fold;
    }
  }
  if (kFold) {
    sg += all_g;
    sb += all_b;
  }
  float* p = a.part + static_cast<int64_t>(blockIdx.y) * 2 * a.N;
  p[j] = sg;
  p[a.N + j] = sb;
}

// dgamma, dbeta from part [rows][2 N]: 32 columns a block, sixteen threads a column take the rows in turn and
// are added in order. A programmatic dependent of the kernel before it: its writes are visible after
// griddepcontrol.wait. Bound by the latency of its few loads: 152 rows of 2 x 4096 sums, 5 MB, take 7 us by
// themselves and cold; 32 threads a column with eight loads at once 1 us less of that behind a long kernel,
// but 3 us more behind a short one.
constexpr int kReduceCols = 32, kReduceSlices = 16;
__global__ void __launch_bounds__(kReduceCols* kReduceSlices) ln_reduce_kernel(const float* part, int rows, int64_t N,
                                                                               void* dgamma, void* dbeta, int wdtype) {
  __shared__ float sums[kReduceSlices][kReduceCols];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = threadIdx.x % kReduceCols, k = threadIdx.x / kReduceCols;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kReduceCols + c;
  float s = 0.f;
  if (j < 2 * N) {
    const float* p = part + j;
    int i = k;
    for (; i + 3 * kReduceSlices < rows; i += 4 * kReduceSlices) {
      const float v0 = p[static_cast<int64_t>(i) * 2 * N], v1 = p[static_cast<int64_t>(i + kReduceSlices) * 2 * N];
      const float v2 = p[static_cast<int64_t>(i + 2 * kReduceSlices) * 2 * N];
      const float v3 = p[static_cast<int64_t>(i + 3 * kReduceSlices) * 2 * N];
      s += (v0 + v1) + (v2 + v3);
    }
    for (; i < rows; i += kReduceSlices) s += p[static_cast<int64_t>(i) * 2 * N];
  }
  sums[k][c] = s;
  __syncthreads();
  if (k != 0 || j >= 2 * N) return;
#pragma unroll
  for (int i = 1; i < kReduceSlices; ++i) s += sums[i][c];
  if (j < N) {
    if (dgamma != nullptr) store_any(dgamma, j, wdtype, s);
  } else if (dbeta != nullptr) {
    store_any(dbeta, j - N, wdtype, s);
  }
}

// ---- host
// Rows shared by a cluster: S blocks of G threads, two vectors each. Several small blocks an SM work on
// while one waits for its cluster.
struct Shared {
  int S, G;
};
Shared share_row(int64_t n) {
  const int64_t half = (n + 1) / 2;  // threads
  const int S = static_cast<int>(half <= kMaxCluster * kBlock ? (half + kBlock - 1) / kBlock : kMaxCluster);
  return Shared{S, static_cast<int>((half + 32 * S - 1) / (32 * S)) * 32};
}
constexpr int64_t kMostShared = 2 * kMaxCluster * kMaxGroup;  // vectors

template <typename T>
cudaError_t fwd_long(const LnFwdArgs& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(a.M < 65536 ? a.M : 65536);
  ln_fwd_long_kernel<T><<<grid, kMaxThreads, 0, stream>>>(a);
  return cudaGetLastError();
}
template <typename T, int R, bool kRagged>
cudaError_t fwd_one(const LnFwdArgs& a, int64_t n, cudaStream_t stream) {
  const int G = group_threads(n, R), groups = G < kBlock ? kBlock / G : 1, block = groups * G;
  int64_t blocks;
  {
    static std::mutex mu;
    static FitCache cache;
    std::lock_guard<std::mutex> lk(mu);
    const cudaError_t e = blocks_that_fit(ln_fwd_kernel<T, R, kRagged, false>, cache, block, 0, blocks);
    if (e != cudaSuccess) return e;
  }
  blocks = persistent_blocks(blocks, (a.M + groups - 1) / groups, kRagged ? rows_apart<T>(a.N) : 1);
  if (blocks == 0) return fwd_long<T>(a, stream);
  ln_fwd_kernel<T, R, kRagged, false><<<static_cast<unsigned>(blocks), block, 0, stream>>>(a, G, 1, Stall(), nullptr);
  return cudaGetLastError();
}
template <typename T, bool kRagged>
cudaError_t fwd_shared(const LnFwdArgs& a, int64_t n, cudaStream_t stream) {
  static std::mutex mu;
  static StreamCache cache;
  std::lock_guard<std::mutex> lk(mu);
  const Shared p = share_row(n);
  const auto kernel = ln_fwd_kernel<T, 2, kRagged, true>;
  const cudaError_t e = clusters_that_fit(kernel, cache, p.G, 0, p.S);
  if (e != cudaSuccess) return e;
  const int64_t clusters = persistent_blocks(cache.clusters, a.M, kRagged ? rows_apart<T>(a.N) : 1);
  if (clusters == 0) return fwd_long<T>(a, stream);
  ClusterLaunch l(p.G, 0, p.S, clusters, stream);
  return cudaLaunchKernelEx(&l.cfg, kernel, a, p.G, p.S, take_stall(kInjectLayerNormFwd), status_word_ptr());
}
// Vectors a thread: one for rows of up to a warp, else two. Rows of more than 1024 vectors are shared by a
// cluster: 3000 x 12288 bf16 with residual 70 us, 88 by a block with four vectors a thread, 181 read again; backward
// with dh 74 us against 117 and 240; 3000 x 16384 fp32 151 and 146 us, read again 254 and 320. A shared row below
// that costs more than it gives (8192 x 6144 bf16, backward with dh: 109 us instead of 83). Ragged rows of more than
// 256 threads a block have one block an SM: forward 3000 x 16383 fp32 with residual takes 514 us, read again 258.
// Backward they are shared up to the same length as whole ones: 3000 x 32761 bf16 287 us, read again 563, 3000 x
// 30001 fp32 501 against 585, though 3000 x 16383 fp32, the shortest with such blocks, 448 against 321.
template <typename T, bool kRagged>
cudaError_t fwd_any(const LnFwdArgs& a, cudaStream_t stream) {
  const int64_t n = (a.N + (kRagged ? 2 * kElems<T> - 2 : 0)) / kElems<T>;
  if (n <= 32) return fwd_one<T, 1, kRagged>(a, n, stream);
  if (n <= 2 * kMaxGroup) return fwd_one<T, 2, kRagged>(a, n, stream);
  if (n <= (kRagged ? kMostShared / 2 : kMostShared)) return fwd_shared<T, kRagged>(a, n, stream);
  return fwd_long<T>(a, stream);
}
template <typename T>
cudaError_t fwd_type(const LnFwdArgs& a, cudaStream_t stream) {
  const bool whole = whole_vectors(a.N, sizeof(T), {a.x, a.residual, a.h, a.y}, {a.ldx, a.ldr}, {a.gamma, a.beta});
  return whole ? fwd_any<T, false>(a, stream) : fwd_any<T, true>(a, stream);
}

int reduce_grid(int64_t N) { return static_cast<int>((2 * N + kReduceCols - 1) / kReduceCols); }
cudaError_t launch_reduce(const LnBwdArgs& a, int64_t rows, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(reduce_grid(a.N)));
  cfg.blockDim = dim3(kReduceCols * kReduceSlices);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ln_reduce_kernel, static_cast<const float*>(a.part), static_cast<int>(rows), a.N,
                            a.dgamma, a.dbeta, a.wdtype);
}

// Rows between two folds of a thread's column sums where (at least) so many groups share M rows: kFewRows or, if
// that is more, as many as there are folds; 0 for groups of at most kFewRows rows, that need none.
constexpr int kFewRows = 128;
int fold_rows(int64_t M, int64_t groups) {
  const int64_t rows = (M + groups - 1) / groups;
  if (rows <= kFewRows) return 0;
  return std::max(kFewRows, static_cast<int>(std::ceil(std::sqrt(static_cast<double>(rows)))));
}
// bytes of the slots of a block of `threads`
template <typename T, int R>
constexpr size_t fold_bytes(int threads) {
  return static_cast<size_t>(threads) * R * kPairs<T> * sizeof(float4);
}

// Rows of column sums in the workspace, at most, for rows of n vectors; no more for longer rows. Groups of up to a
// warp: several blocks an SM. To 1024 vectors: one block of 512 threads an SM, or for few rows up to twice as many
// smaller ones. Shared rows: clusters of S blocks, two blocks an SM. Longer ones: chunks.
constexpr int64_t kLongChunks = 64;
int64_t most_sums(int64_t n) {
  if (n <= 32) return 1024;
  if (n <= 2 * kMaxGroup) return 320;
  if (n <= kMostShared) return std::max(kLongChunks, static_cast<int64_t>((320 / share_row(n).S + 7) / 8 * 8));
  return kLongChunks;
}

template <typename T>
cudaError_t bwd_long(const LnBwdArgs& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(a.M < 65536 ? a.M : 65536);
  ln_dx_long_kernel<T><<<grid, kMaxThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.part == nullptr) return e;
  const int64_t chunks = a.M < kLongChunks ? a.M : kLongChunks, per = (a.M + chunks - 1) / chunks;
  const dim3 g(static_cast<unsigned>((a.N + kColThreads - 1) / kColThreads), static_cast<unsigned>(chunks));
  const int fold = fold_rows(per, 1);
  if (fold > 0) ln_param_long_kernel<T, true><<<g, kColThreads, 0, stream>>>(a, per, fold);
  else ln_param_long_kernel<T, false><<<g, kColThreads, 0, stream>>>(a, per, 0);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_reduce(a, chunks, stream);
}
template <typename T, int R, bool kRagged, bool kFold>
cudaError_t bwd_groups(const LnBwdArgs& a, int64_t n, int G, int groups, int fold, cudaStream_t stream) {
  const int block = groups * G;
  const size_t sums = groups > 1 && a.part != nullptr ? static_cast<size_t>(2 * a.N) * sizeof(float) : 0;
  const size_t smem = kFold ? std::max(sums, fold_bytes<T, R>(block)) : sums;
  int64_t blocks;
  {
    static std::mutex mu;
    static FitCache cache;
    std::lock_guard<std::mutex> lk(mu);
    const cudaError_t e = blocks_that_fit(ln_bwd_kernel<T, R, kRagged, false, kFold>, cache, block, smem, blocks);
    if (e != cudaSuccess) return e;
  }
  blocks = persistent_blocks(std::min(blocks, most_sums(n)), (a.M + groups - 1) / groups,
                             kRagged ? rows_apart<T>(a.N) : 1);
  if (blocks == 0) return bwd_long<T>(a, stream);
  ln_bwd_kernel<T, R, kRagged, false, kFold>
      <<<static_cast<unsigned>(blocks), block, smem, stream>>>(a, G, 1, fold, Stall(), nullptr);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.part == nullptr) return e;
  return launch_reduce(a, blocks, stream);
}
template <typename T, int R, bool kRagged>
cudaError_t bwd_one(const LnBwdArgs& a, int64_t n, cudaStream_t stream) {
  const int G = group_threads(n, R);
  // One block an SM, so that there are few rows of column sums to write and add, or smaller ones for few rows
  // (blocks of 256 threads and sums stored element by element: 2048 x 4096 bf16 with dh 30 us, now 22).
  int groups = kMaxGroup / G;
  while (groups > 1 && groups * G > 32 && (a.M + groups - 1) / groups < device_sm_count()) groups = (groups + 1) / 2;
  const int fold = a.part != nullptr ? fold_rows(a.M, static_cast<int64_t>(groups) * device_sm_count()) : 0;
  return fold > 0 ? bwd_groups<T, R, kRagged, true>(a, n, G, groups, fold, stream)
                  : bwd_groups<T, R, kRagged, false>(a, n, G, groups, 0, stream);
}
template <typename T, bool kRagged, bool kFold>
cudaError_t bwd_clusters(const LnBwdArgs& a, int64_t n, const Shared& p, int fold, cudaStream_t stream) {
  const auto kernel = ln_bwd_kernel<T, 2, kRagged, true, kFold>;
  const size_t smem = kFold ? fold_bytes<T, 2>(p.G) : 0;
  int64_t clusters;
  {
    static std::mutex mu;
    static StreamCache cache;
    std::lock_guard<std::mutex> lk(mu);
    cudaError_t e = clusters_that_fit(kernel, cache, p.G, smem, p.S);
    if (e != cudaSuccess) return e;
    const int64_t fit = std::min(static_cast<int64_t>(cache.clusters), most_sums(n));
    clusters = persistent_blocks(fit, a.M, kRagged ? rows_apart<T>(a.N) : 1);
    if (clusters > 0) {
      ClusterLaunch l(p.G, smem, p.S, clusters, stream);
      e = cudaLaunchKernelEx(&l.cfg, kernel, a, p.G, p.S, fold, take_stall(kInjectLayerNormBwd), status_word_ptr());
      if (e != cudaSuccess) return e;
    }
  }
  if (clusters == 0) return bwd_long<T>(a, stream);
  return a.part == nullptr ? cudaSuccess : launch_reduce(a, clusters, stream);
}
template <typename T, bool kRagged>
cudaError_t bwd_shared(const LnBwdArgs& a, int64_t n, cudaStream_t stream) {
  const Shared p = share_row(n);
  const int fold = a.part != nullptr ? fold_rows(a.M, std::max(1, device_sm_count() / p.S)) : 0;
  return fold > 0 ? bwd_clusters<T, kRagged, true>(a, n, p, fold, stream)
                  : bwd_clusters<T, kRagged, false>(a, n, p, 0, stream);
}
template <typename T, bool kRagged>
cudaError_t bwd_any(const LnBwdArgs& a, cudaStream_t stream) {
  const int64_t n = (a.N + (kRagged ? 2 * kElems<T> - 2 : 0)) / kElems<T>;
  if (n <= 32) return bwd_one<T, 1, kRagged>(a, n, stream);
  if (n <= 2 * kMaxGroup) return bwd_one<T, 2, kRagged>(a, n, stream);
  if (n <= kMostShared) return bwd_shared<T, kRagged>(a, n, stream);
  return bwd_long<T>(a, stream);
}
template <typename T>
cudaError_t bwd_type(const LnBwdArgs& a, cudaStream_t stream) {
  const bool whole = whole_vectors(a.N, sizeof(T), {a.dy, a.x, a.dh, a.dx}, {a.lddy, a.ldx, a.lddh}, {a.gamma});
  return whole ? bwd_any<T, false>(a, stream) : bwd_any<T, true>(a, stream);
}

}  // namespace

size_t ln_workspace_bytes(int64_t M, int64_t N) {
  // of the type with the fewest vectors, aligned: it has the most rows of sums
  const int64_t rows = std::min(M, most_sums((N + 7) / 8));
  return static_cast<size_t>(rows) * 2 * static_cast<size_t>(N) * sizeof(float);
}

cudaError_t launch_layer_norm_fwd(const LnFwdArgs& a, int dtype, cudaStream_t stream) {
  return dtype == 0   ? fwd_type<float>(a, stream)
         : dtype == 1 ? fwd_type<__half>(a, stream)
                      : fwd_type<__nv_bfloat16>(a, stream);
}

cudaError_t launch_layer_norm_bwd(const LnBwdArgs& a, int dtype, cudaStream_t stream) {
  return dtype == 0   ? bwd_type<float>(a, stream)
         : dtype == 1 ? bwd_type<__half>(a, stream)
                      : bwd_type<__nv_bfloat16>(a, stream);
}

}  // namespace swg
