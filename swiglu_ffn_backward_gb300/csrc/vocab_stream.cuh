// Rows of logits streamed through shared memory by persistent blocks.
//
// A block has 16 computing warps and a producer warp that keeps a ring of six 32 KB stages full with
// bulk copies, across rows: the copies of the next rows run under the work on this one, so the reads
// never pause for a reduction. Cluster c takes the rows c, c + #clusters, ...; its S blocks take a share
// of the row each (vocab_rows.cuh: aligned 16-byte vectors). A row's first and last vector, when they
// are partial, are put together by the producer warp, with -inf outside the row.
#pragma once

#include "vocab_rows.cuh"

namespace swg {
namespace row {

constexpr int kStreamWarps = 16;
constexpr int kStreamThreads = kStreamWarps * 32;   // computing threads
constexpr int kStageVecs = 4 * kStreamThreads;      // vectors a stage holds: four for each thread
constexpr int kStageBytes = kStageVecs * 16;
constexpr int kStages = 6;
constexpr int kRingBytes = kStages * kStageBytes;

// Waits are bounded: after the first one that ran out, the later ones of the thread only look once, so
// that the block still comes to its end (its results are then void and the status word says so).
struct Patience {
  bool lost = false;
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
    if (!mbar_wait(bar, parity, lost ? 0 : kWaitLimitCycles)) lost = true;
  }
  // of a barrier that other blocks of the cluster complete: what they wrote is visible after it
  __device__ __forceinline__ void cluster(uint64_t* bar, uint32_t parity) {
    const uint32_t at = smem_u32(bar);
    auto done = [&]() {
      uint32_t ok;
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(at), "r"(parity)
          : "memory");
      return ok != 0;
    };
    if (done()) return;
    const long long t0 = clock64();
    while (!done())
      if (clock64() - t0 > (lost ? 0 : kWaitLimitCycles)) {
        lost = true;
        return;
      }
  }
};

struct Ring {
  uint64_t full[kStages];   // a stage's copies have landed
  uint64_t empty[kStages];  // the computing warps have read it
};
__device__ __forceinline__ void ring_init(Ring& ring) {
  for (int i = 0; i < kStages; ++i) {
    mbar_init(&ring.full[i], 1);
    mbar_init(&ring.empty[i], kStreamWarps);
  }
}
// a position in the ring: stage and the parity of its use
struct Place {
  int stage = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++stage == kStages) {
      stage = 0;
      parity ^= 1u;
    }
  }
};

// The producer warp: all rows of the block's cluster, row r's share at `rank` of S.
template <typename T>
__device__ __forceinline__ void produce_rows(const void* logits, int64_t ld, int64_t V, int64_t first, int64_t rows,
                                             int64_t step, int per, int rank, unsigned char* buf, Ring& ring,
                                             Patience& wait) {
  constexpr int E = Traits<T>::E;
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
  for (int64_t r = first; r < rows; r += step) {
    const T* z = base + r * ld;
    const Share sh = share_of(z, V, per, rank);
    const T ahead = edge(r + step);
    const int64_t e0 = first_element<T>(sh, sh.begin), e1 = first_element<T>(sh, sh.end);
    const int whole0 = sh.begin + (e0 < 0 ? 1 : 0), whole1 = max(whole0, sh.end - (e1 > V ? 1 : 0));
    for (int c = sh.begin; c < sh.end; c += kStageVecs) {
      const int end = min(sh.end, c + kStageVecs);
      unsigned char* to = buf + p.stage * kStageBytes;
      wait(&ring.empty[p.stage], p.parity ^ 1u);
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
      p.next();
    }
    mine = ahead;
  }
}

// a computing thread's four vectors of a stage that holds n; -inf past them
template <typename T>
__device__ __forceinline__ void read_stage(Vec (&v)[4], const unsigned char* stage, int n) {
  const uint4* p = reinterpret_cast<const uint4*>(stage) + threadIdx.x;
  if (n == kStageVecs) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 u = p[i * kStreamThreads];
      v[i] = Vec{{u.x, u.y, u.z, u.w}};
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 u = make_uint4(Traits<T>::kNegInf, Traits<T>::kNegInf, Traits<T>::kNegInf, Traits<T>::kNegInf);
    if (i * kStreamThreads + static_cast<int>(threadIdx.x) < n) u = p[i * kStreamThreads];
    v[i] = Vec{{u.x, u.y, u.z, u.w}};
  }
}

// 8 bytes into block `rank` of the cluster, counted by its barrier at the offset of `bar`
__device__ __forceinline__ void send_f2(const float2* to, const uint64_t* bar, uint32_t rank, float x, float y) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
                   peer_addr(to, rank)),
               "f"(x), "f"(y), "r"(peer_addr(bar, rank))
               : "memory");
}

}  // namespace row

// A persistent launch: as many clusters as fit on the device at once, at most one a row. The occupancy of
// a (kernel, cluster size, shared memory) is asked once for each device.
struct StreamCache {
  int device = -1, S = 0, clusters = 0;
  size_t smem = 0;
};
template <typename Kernel, typename... Args>
cudaError_t launch_stream(Kernel kernel, StreamCache& cache, int threads, size_t smem, int64_t rows, int S,
                          cudaStream_t stream, const Args&... args) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(S);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cache.device != dev || cache.S != S || cache.smem != smem) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(S));
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorLaunchOutOfResources;
    cache = StreamCache{dev, S, n, smem};
  }
  const int64_t clusters = rows < cache.clusters ? rows : cache.clusters;
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * S));
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace swg
