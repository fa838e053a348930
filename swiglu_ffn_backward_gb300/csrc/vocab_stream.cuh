// Rows of logits streamed through shared memory by persistent blocks.
//
// A block has W computing warps and a producer warp that keeps a ring of stages (four vectors for each
// computing thread) full with bulk copies, across rows: the copies of the next rows run under the work on
// this one, so the reads do not pause for a reduction. Cluster c takes the rows c, c + #clusters, ...; its S
// blocks take a share of the row each (vocab_rows.cuh: aligned 16-byte vectors). A row's first and last
// vector, when they are partial, are put together by the producer warp, with -inf outside the row.
#pragma once

#include "row_grid.h"
#include "vocab_rows.cuh"

namespace swg {
namespace row {

constexpr int kWarpVecs = 4 * 32;  // vectors of a stage that a warp takes
template <int W>
struct Shape {
  static constexpr int kThreads = 32 * W;             // computing threads
  static constexpr int kStageVecs = 4 * kThreads;     // vectors a stage holds: four for each thread
  static constexpr int kStageBytes = 16 * kStageVecs;
};

// What a launch is told for tests of the waits that run out: the ring entry (or row) from which on the last block of
// each cluster falls silent (-1: none), and the cycles that a wait takes at most.
struct Stall {
  int64_t at = -1;
  uint32_t limit = kWaitLimitCycles;
};

// Waits are bounded. After one that ran out the thread's later waits only look once, so that the block still comes
// to its end (its results are then void and the status word says so). A barrier that counts bytes must not be set
// or fed out of turn by then, or its counts are overrun: such a thread arrives at no barrier that others send or
// copy behind, and sends nothing. Hence `open`, the lanes that may (the peers to send to, or one): 0 once a wait
// has run out. The clock is read in 32 bits, which hold the limit: with 64 the waiting warps took 2% of the log
// probabilities' time at 8192 to 50001 columns, and a flag beside the number of peers 3% of a distillation step.
struct Patience {
  uint32_t limit;
  int open;
  __device__ __forceinline__ explicit Patience(uint32_t limit_, int open_ = 1) : limit(limit_), open(open_) {}
  __device__ __forceinline__ bool lost() const { return open == 0; }
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
    const uint32_t at = smem_u32(bar);
    until([&]() { return mbar_try_wait(at, parity); });
  }
  // of a barrier that other blocks of the cluster complete: what they wrote is visible after it
  __device__ __forceinline__ void cluster(uint64_t* bar, uint32_t parity) {
    const uint32_t at = smem_u32(bar);
    until([&]() {
      uint32_t ok;
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(at), "r"(parity)
          : "memory");
      return ok != 0;
    });
  }
  // After a wait that ran out, at the end of the kernel behind the cluster's last barrier, when no block sends any
  // more: what was sent before is given half a millisecond to come (it takes some microseconds), so that no block
  // leaves while something is on its way into it. A block whose waits all ended has received everything.
  __device__ __forceinline__ void leave() const {
    if (!lost()) return;
    const uint32_t t0 = static_cast<uint32_t>(clock());
    while (static_cast<uint32_t>(clock()) - t0 < (1u << 20)) __nanosleep(1000);
  }

 private:
  template <typename Done>
  __device__ __forceinline__ void until(Done done) {
    if (done()) return;
    const uint32_t t0 = static_cast<uint32_t>(clock());
    while (!done())
      if (static_cast<uint32_t>(clock()) - t0 > (lost() ? 0u : limit)) {
        open = 0;
        return;
      }
  }
};
static_assert(kWaitLimitCycles < (1LL << 32) - (1LL << 27), "the clock's low half");

template <int W, int N>  // up to N stages
struct Ring {
  uint64_t full[N];   // a stage's copies have landed
  uint64_t empty[N];  // the computing warps have read it
};
template <int W, int N>
__device__ __forceinline__ void ring_init(Ring<W, N>& ring) {
  for (int i = 0; i < N; ++i) {
    mbar_init(&ring.full[i], 1);
    mbar_init(&ring.empty[i], W);
  }
}
// a position in the ring: stage and the parity of its use
struct Place {
  int stage = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) {
      stage = 0;
      parity ^= 1u;
    }
  }
};

// The producer warp: all rows of the block's cluster, row r's share at `rank` of S. It issues no more copies
// once a wait has run out (or from ring entry `stall` on), and ends when the copies it has issued have landed.
template <typename T, int W, int N>
__device__ __forceinline__ void produce_rows(const void* logits, int64_t ld, int64_t V, int64_t first, int64_t rows,
                                             int64_t step, int per, int rank, unsigned char* buf, int stages,
                                             Ring<W, N>& ring, Patience& wait, int64_t stall) {
  constexpr int E = Traits<T>::E, kStageVecs = Shape<W>::kStageVecs, kStageBytes = Shape<W>::kStageBytes;
  const int lane = threadIdx.x & 31;
  const T* base = static_cast<const T*>(logits);
  // a lane's element of the partial vectors of row r: lanes 0 .. E - 1 the first one's, 16 .. 16 + E - 1
  // the last one's; loaded a row ahead
  auto edge = [&](int64_t r) {
    T x = from_f<T>(neg_inf());
    if (r >= rows) return x;
    const T* z = base + r * ld;
    const Share sh = share_of(z, V, per, rank);
    const int at = lane & 15;
    if (at >= E || sh.begin == sh.end) return x;
    const int64_t e = first_element<T>(sh, lane < 16 ? sh.begin : sh.end - 1) + at;
    if (e >= 0 && e < V) x = z[e];
    return x;
  };
  Place p;
  T mine = edge(first);
  bool go = true;
  for (int64_t r = first; r < rows && go; r += step) {
    const T* z = base + r * ld;
    const Share sh = share_of(z, V, per, rank);
    const T ahead = edge(r + step);
    const int64_t e0 = first_element<T>(sh, sh.begin), e1 = first_element<T>(sh, sh.end);
    const int whole0 = sh.begin + (e0 < 0 ? 1 : 0), whole1 = max(whole0, sh.end - (e1 > V ? 1 : 0));
    for (int c = sh.begin; c < sh.end; c += kStageVecs) {
      const int end = min(sh.end, c + kStageVecs);
      unsigned char* to = buf + p.stage * kStageBytes;
      wait(&ring.empty[p.stage], p.parity ^ 1u);
      go = !__any_sync(0xffffffffu, wait.lost()) && stall-- != 0;
      if (!go) break;
      const int w0 = max(c, whole0), w1 = min(end, whole1);
      // a partial vector's elements, lane by lane
      const bool head = c == sh.begin && e0 < 0, tail = end == sh.end && e1 > V;
      if (lane < E && head) reinterpret_cast<T*>(to)[lane] = mine;
      if (lane >= 16 && lane < 16 + E && tail && !(head && end - c == 1))
        reinterpret_cast<T*>(to + (end - 1 - c) * 16)[lane - 16] = mine;
      __syncwarp();
      if (lane == 0) {
        fence_proxy_async_smem();
        const uint32_t bytes = w1 > w0 ? static_cast<uint32_t>(w1 - w0) * 16u : 0u;
        mbar_arrive_expect_tx(&ring.full[p.stage], bytes);
        if (bytes > 0) bulk_g2s(to + (w0 - c) * 16, z + first_element<T>(sh, w0), bytes, &ring.full[p.stage]);
      }
      __syncwarp();
      p.next(stages);
    }
    mine = ahead;
  }
  for (int i = 0; i < stages; ++i)  // the last use of every stage; one that has had none is done
    if (!mbar_wait(&ring.full[i], i < p.stage ? p.parity : p.parity ^ 1u)) wait.open = 0;
}

// a computing thread's four vectors of a stage that holds n; -inf past them
template <typename T, int W>
__device__ __forceinline__ void read_stage(Vec (&v)[4], const unsigned char* stage, int n) {
  constexpr int kThreads = Shape<W>::kThreads;
  const uint4* p = reinterpret_cast<const uint4*>(stage) + threadIdx.x;
  if (n == Shape<W>::kStageVecs) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 u = p[i * kThreads];
      v[i] = Vec{{u.x, u.y, u.z, u.w}};
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 u = make_uint4(Traits<T>::kNegInf, Traits<T>::kNegInf, Traits<T>::kNegInf, Traits<T>::kNegInf);
    if (i * kThreads + static_cast<int>(threadIdx.x) < n) u = p[i * kThreads];
    v[i] = Vec{{u.x, u.y, u.z, u.w}};
  }
}

// The same with four vectors that follow each other, 4 threadIdx.x .. 4 threadIdx.x + 3, in an order by
// thread in which the eight lanes of a shared-memory phase meet all banks.
template <typename T, int W>
__device__ __forceinline__ void read_stage_runs(Vec (&v)[4], const unsigned char* stage, int n) {
  const uint4* p = reinterpret_cast<const uint4*>(stage);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = 4 * static_cast<int>(threadIdx.x) + ((i + (static_cast<int>(threadIdx.x) >> 1)) & 3);
    uint4 u = make_uint4(Traits<T>::kNegInf, Traits<T>::kNegInf, Traits<T>::kNegInf, Traits<T>::kNegInf);
    if (n == Shape<W>::kStageVecs || at < n) u = p[at];
    v[i] = Vec{{u.x, u.y, u.z, u.w}};
  }
}

// A warp's sums over its part of a row, four vectors a thread at a time: sum 2^x, with kSecond sum 2^x x
// too, under a reference logit that is raised only when a logit passes it by 2^kRoom or more, so that the
// warp does not have to agree on its maximum every time. Terms that are much alike are rounded the same way, so
// that one accumulator over n of them may be off by n / 2 ulp: a stage's terms are added first (16 a thread),
// then the stages, and with kLong, for rows of more than kFewStages of them, each kFewStages are put by. With
// all of a thread's terms in one sequence, 1000 x 262144 bf16 of like logits had sums off by 1.1e-5 in blocks of
// four warps. The stages' own sums cost nothing, putting by costs up to 3%.
constexpr float kRoom = 10.0f;
constexpr int kFewStages = 64;
template <typename T, bool kSecond, bool kLong>
struct WarpSums {
  float m = neg_inf();    // reference logit
  float lim = neg_inf();  // a logit above it raises the reference
  float top = neg_inf();  // the thread's maximum
  bool masked = false;    // the row has shown a -inf: more are likely
  Scale k;
  float2 s2{0.f, 0.f}, w2{0.f, 0.f};  // of the last stages
  float2 s3{0.f, 0.f}, w3{0.f, 0.f};  // kLong: of those before
  int left = kFewStages;

  __device__ __forceinline__ explicit WarpSums(float c) : k{c, 0.0f} {}

  // adds a stage's terms; false, and nothing added, where the second sum is NaN
  template <bool kMasked>
  __device__ __forceinline__ bool add_terms(const Vec (&v)[4]) {
    const float2 c = make_float2(k.c, k.c), ref = make_float2(-k.ref, -k.ref);
    float2 s{0.f, 0.f}, w{0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int p = 0; p < Traits<T>::E / 2; ++p) {
        float2 x = __ffma2_rn(vec_pair<T>(v[i], p), c, ref);
        if (kMasked) x = make_float2(at_least(x.x), at_least(x.y));
        const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
        s = i + p == 0 ? e : __fadd2_rn(s, e);
        if (kSecond) w = i + p == 0 ? __fmul2_rn(e, x) : __ffma2_rn(e, x, w);
      }
    }
    if (kSecond && !kMasked && __any_sync(0xffffffffu, !(w.x + w.y == w.x + w.y))) return false;
    s2 = __fadd2_rn(s2, s);
    if (kSecond) w2 = __fadd2_rn(w2, w);
    if (kLong && --left == 0) {
      s3 = __fadd2_rn(s3, s2);
      if (kSecond) w3 = __fadd2_rn(w3, w2);
      s2 = w2 = make_float2(0.f, 0.f);
      left = kFewStages;
    }
    return true;
  }
  // returns the largest of the thread's logits; padded: some of them are -inf for being behind the row
  __device__ __forceinline__ float add(const Vec (&v)[4], float c, bool padded) {
    const float most = vec_max4<T>(v);
    if (__any_sync(0xffffffffu, most > lim)) {
      const float mn = warp_max(fmaxf(most, m));
      const Scale kn = scale_of(mn, c);
      const float x0 = ref_shift(m, k, mn, kn, c), f = ex2_approx(x0);
      if (kSecond) w2 = __fmul2_rn(__ffma2_rn(s2, make_float2(x0, x0), w2), make_float2(f, f));
      s2 = __fmul2_rn(s2, make_float2(f, f));
      if (kLong && kSecond) w3 = __fmul2_rn(__ffma2_rn(s3, make_float2(x0, x0), w3), make_float2(f, f));
      if (kLong) s3 = __fmul2_rn(s3, make_float2(f, f));
      m = mn;
      k = kn;
      lim = fabsf(k.ref) < kLargeRef ? m + kRoom / c : m;
    }
    top = fmaxf(top, most);
    // a -inf makes the second sum 0 * inf: only then the exponents are kept above it
    if (!kSecond || (!masked && !padded)) {
      if (add_terms<false>(v)) return most;
      masked = true;
    }
    add_terms<true>(v);
    return most;
  }
  // reference logit, sum 2^x, sum 2^x x, maximum
  __device__ __forceinline__ float4 result() const {
    const float2 s = kLong ? __fadd2_rn(s2, s3) : s2, w = kLong ? __fadd2_rn(w2, w3) : w2;
    return make_float4(m, warp_sum(s.x + s.y), kSecond ? warp_sum(w.x + w.y) : 0.f, warp_max(top));
  }
};
// such results, one in each lane (a reference of -inf and sums of 0 for none), joined in every lane
__device__ __forceinline__ float4 join_sums(const float4& p, float c, Scale& k) {
  const float m = warp_max(p.x);
  k = scale_of(m, c);
  const float x0 = ref_shift(p.x, scale_of(p.x, c), m, k, c), f = ex2_approx(x0);
  return make_float4(m, warp_sum(f * p.y), warp_sum(f * fmaf(p.y, x0, p.z)), warp_max(p.w));
}

// Sends into block `rank` of the cluster, their bytes counted by its barrier at the offset of `bar`.
__device__ __forceinline__ void send_f2(const float2* to, const uint64_t* bar, uint32_t rank, float x, float y) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
                   peer_addr(to, rank)),
               "f"(x), "f"(y), "r"(peer_addr(bar, rank))
               : "memory");
}

__device__ __forceinline__ void send_f4(const float4* to, const uint64_t* bar, uint32_t rank, float4 v) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                   peer_addr(to, rank)),
               "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(peer_addr(bar, rank))
               : "memory");
}
__device__ __forceinline__ void send_u64(const uint64_t* to, const uint64_t* bar, uint32_t rank, uint64_t v) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(peer_addr(to, rank)),
               "l"(v), "r"(peer_addr(bar, rank))
               : "memory");
}

}  // namespace row

// what the next launch of `kernel` is told (one launch)
inline row::Stall take_stall(int kernel) {
  const Injection i = take_injection(kernel);
  row::Stall s;
  s.at = i.stall_at;
  if (i.wait_limit < kWaitLimitCycles) s.limit = static_cast<uint32_t>(i.wait_limit);
  return s;
}

// How many clusters of a persistent kernel fit on the device at once: of a (cluster size, block, shared memory)
// asked once for each device.
struct StreamCache {
  int device = -1, S = 0, threads = 0, clusters = 0;
  size_t smem = 0;
};
struct ClusterLaunch {  // a launch of `clusters` clusters of S blocks
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  ClusterLaunch(int threads, size_t smem, int S, int64_t clusters, cudaStream_t stream) {
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * S));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(S);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  ClusterLaunch(const ClusterLaunch&) = delete;
};
template <typename Kernel>
cudaError_t clusters_that_fit(Kernel kernel, StreamCache& cache, int threads, size_t smem, int S) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (cache.device == dev && cache.S == S && cache.threads == threads && cache.smem == smem) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  ClusterLaunch one(threads, smem, S, 1, nullptr);
  int n = 0;
  e = cudaOccupancyMaxActiveClusters(&n, kernel, &one.cfg);
  if (e != cudaSuccess) return e;
  cache = StreamCache{dev, S, threads, n, smem};
  return cudaSuccess;
}
// A persistent launch for `rows` rows: as many clusters as fit, at most one a row (`all`: one for every row,
// however many fit).
template <typename Kernel, typename... Args>
cudaError_t launch_stream(Kernel kernel, StreamCache& cache, int threads, size_t smem, int64_t rows, int S,
                          bool all, cudaStream_t stream, const Args&... args) {
  const cudaError_t e = clusters_that_fit(kernel, cache, threads, smem, S);
  if (e != cudaSuccess) return e;
  if (cache.clusters < 1) return cudaErrorLaunchOutOfResources;
  ClusterLaunch l(threads, smem, S, all ? rows : persistent_blocks(cache.clusters, rows, 1), stream);
  return cudaLaunchKernelEx(&l.cfg, kernel, args...);
}

}  // namespace swg
