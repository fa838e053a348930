// The element-wise part of the linear layer's backward:
//   dz = dy f'(z), rounded to the element type;  db = sum over rows of dz (in fp32, before the rounding)
// HBM-bound: reads dy (and z), writes dz (without an activation dz is dy itself, and only the sums are taken).
// A block takes 256 columns of a run of rows: warp w the columns (w & 3) 64 .. + 63 and the row group w >> 2, a lane
// one 16-byte vector of them, so that eight rows are under way at once, with four or eight such steps in flight. No sum takes
// more than 128 rows in one accumulator (like terms are rounded the same way, and a longer chain drifts); a second
// kernel adds the blocks' partial rows in a fixed order. Measured: GELU, 65536 x 1024 bf16, 79 us (5.1 TB/s; the
// activation's gradient takes four special-function results a pair of elements), the sums alone of 220000 x 512 36 us
// (6.2 TB/s).
#include <algorithm>

#include "linear.cuh"

namespace swg {
namespace {

using namespace lin;

constexpr int kThreads = 256;
constexpr int kCols = 256;    // columns of a block
constexpr int kRowStep = 8;   // rows of one step
constexpr int kBlocks = 3;    // blocks an SM: 80 registers a thread (64 or 128 spill or leave too few loads under way)
constexpr int kMaxRows = 128 * kRowStep;  // rows of a block, at most

__device__ __forceinline__ uint4 ld_stream(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// where the column sums go: partial rows for a second kernel, or, from a cluster that has all rows, db itself
struct SumsTo {
  float* part;  // or null
  void* db;     // or null
  int dtype;
  bool accumulate;
};

template <int kActOf, bool kF16>
__global__ void __launch_bounds__(kThreads, kBlocks)
    linear_dz_kernel(const uint16_t* dy, const uint16_t* z, uint16_t* dz, const SumsTo to, int64_t M, int64_t N,
                     int64_t lddy, int64_t rows_per_block) {
  constexpr bool kAct = kActOf != kActNone;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = (warp & 3) * 64 + (lane & 7) * 8;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * kCols + c;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * rows_per_block, r1 = min(M, r0 + rows_per_block);
  float2 sum[4] = {};
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (col < N) {
    auto step = [&](const uint4& g, const uint4& v, int64_t row) {
      float2 d[4], t[4];
      widen8<kF16>(g, d);
      if (kAct) {
        widen8<kF16>(v, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = __fmul2_rn(d[e], activate_grad<kActOf>(t[e]));
        *reinterpret_cast<uint4*>(dz + row * N + col) = narrow8<kF16>(d);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] = __fadd2_rn(sum[e], d[e]);
    };
    int64_t row = r0 + (warp >> 2) * 4 + (lane >> 3);
    constexpr int kDeep = kAct ? 4 : 8;
    for (; row + (kDeep - 1) * kRowStep < r1; row += kDeep * kRowStep) {
      uint4 g[kDeep], v[kDeep];
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        g[u] = ld_stream(dy + (row + u * kRowStep) * lddy + col);
        if (kAct) v[u] = ld_stream(z + (row + u * kRowStep) * N + col);
      }
#pragma unroll
      for (int u = 0; u < kDeep; ++u) step(g[u], v[u], row + u * kRowStep);
    }
    for (; row < r1; row += kRowStep)
      step(ld_stream(dy + row * lddy + col), kAct ? ld_stream(z + row * N + col) : make_uint4(0u, 0u, 0u, 0u), row);
  }
  if (to.part == nullptr && to.db == nullptr) return;
  // the four row lanes of a warp, then the two row groups
  __shared__ float red[2][kCols];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
#pragma unroll
    for (int o = 8; o <= 16; o *= 2) {
      sum[e].x += __shfl_xor_sync(0xffffffffu, sum[e].x, o);
      sum[e].y += __shfl_xor_sync(0xffffffffu, sum[e].y, o);
    }
    if (lane < 8) {
      red[warp >> 2][c + 2 * e] = sum[e].x;
      red[warp >> 2][c + 2 * e + 1] = sum[e].y;
    }
  }
  __syncthreads();
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kCols + threadIdx.x;
  const float total = red[0][threadIdx.x] + red[1][threadIdx.x];
  if (to.db == nullptr) {
    if (j < N) to.part[static_cast<int64_t>(blockIdx.y) * N + j] = total;
    return;
  }
  red[0][threadIdx.x] = total;
  cluster_sync();
  const uint32_t blocks = gridDim.y;  // of the cluster: each adds up some of the columns, in the blocks' order
  if (static_cast<uint32_t>(threadIdx.x) % blocks == cluster_ctarank() && j < N) {
    const uint32_t* mine = reinterpret_cast<const uint32_t*>(&red[0][threadIdx.x]);
    float t = 0.0f;
    for (uint32_t i = 0; i < blocks; ++i) t += __uint_as_float(ld_cluster_u32(mine, i));
    if (to.accumulate) t += row::load_any(to.db, j, to.dtype);
    row::store_any(to.db, j, to.dtype, t);
  }
  __syncwarp();
  cluster_sync();  // no block leaves while another reads its sums
}

// db from part [rows][N]: 32 columns a block, sixteen warps take the rows in turn, eight loads under way, and are added in
// order; at most 64 terms in sequence, then these parts.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(32 * kSumWarps) linear_db_kernel(const float* part, int64_t rows, int64_t N, void* db,
                                                                   int dtype, bool accumulate) {
  __shared__ float acc[kSumWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float* p = part + min(j, N - 1);
  float t = 0.0f, s = 0.0f;
  int64_t i = warp;
  for (int n = 1; i + 7 * kSumWarps < rows; i += 8 * kSumWarps, ++n) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = p[(i + u * kSumWarps) * N];
    s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    if (n % 8 == 0) {
      t += s;
      s = 0.0f;
    }
  }
  float v[7];
#pragma unroll
  for (int u = 0; u < 7; ++u) v[u] = i + u * kSumWarps < rows ? p[(i + u * kSumWarps) * N] : 0.0f;
#pragma unroll
  for (int u = 0; u < 7; ++u) s += v[u];
  acc[warp][lane] = t + s;
  __syncthreads();
  if (warp != 0 || j >= N) return;
  t = acc[0][lane];
#pragma unroll
  for (int w = 1; w < kSumWarps; ++w) t += acc[w][lane];
  if (accumulate) t += row::load_any(db, j, dtype);
  row::store_any(db, j, dtype, t);
}

// rows of a block: about three blocks on each of 152 SMs (a plan that does not depend on the device, so that the
// workspace's size does not either)
int64_t rows_per_block(int64_t M, int64_t N) {
  const int64_t gx = (N + kCols - 1) / kCols, blocks = std::max<int64_t>(1, 152 * kBlocks / gx);
  const int64_t rows = ((M + blocks - 1) / blocks + kRowStep - 1) / kRowStep * kRowStep;
  return std::min<int64_t>(kMaxRows, std::max<int64_t>(rows, 4 * kRowStep));
}

// Up to this many rows a cluster of at most eight blocks takes all of them and writes db, without the second launch, for
// the host's sake: a call of linear_bwd for 257 x 512 x 1024 with GELU took 37.2, 37.4 and 32.8 us, and 36.8, 40.4 and
// 36.3 with it, in runs in turn; on the GPU the exchange in the cluster costs more than the launch (16.7 us a call in a
// graph, 15.4 with it).
constexpr int64_t kFewRows = 512, kFewBlocks = 8;

// a programmatic dependent launch: its blocks may come while the kernel before it ends, and wait for it
cudaLaunchConfig_t dependent_launch(const dim3& grid, int threads, cudaStream_t stream, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}
template <bool kF16>
cudaError_t launch_dz(const dim3& grid, const uint16_t* dy, const uint16_t* z, uint16_t* dz, const SumsTo& to, int64_t M,
                      int64_t N, int64_t lddy, int64_t per, int act, cudaStream_t stream) {
  const auto kernel = act == kLinearNoAct ? linear_dz_kernel<kActNone, kF16>
                      : act == 0          ? linear_dz_kernel<0, kF16>
                      : act == 1          ? linear_dz_kernel<1, kF16>
                                          : linear_dz_kernel<2, kF16>;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = dependent_launch(grid, kThreads, stream, attr);
  if (to.db != nullptr) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = grid.y;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kernel, dy, z, dz, to, M, N, lddy, per);
}

}  // namespace

size_t linear_dz_workspace_bytes(int64_t M, int64_t N) {
  const int64_t per = rows_per_block(M, N);
  return static_cast<size_t>((M + per - 1) / per) * static_cast<size_t>(N) * sizeof(float);
}

cudaError_t launch_linear_dz(const void* dy, const void* z, void* dz, void* db, int64_t M, int64_t N, int64_t lddy,
                             int act, bool f16, bool db_f32, bool accumulate, float* part, cudaStream_t stream) {
  const int dtype = db_f32 ? 0 : (f16 ? 1 : 2);
  const bool few = db != nullptr && M <= kFewRows;
  const int64_t per = few ? ((M + kFewBlocks - 1) / kFewBlocks + kRowStep - 1) / kRowStep * kRowStep : rows_per_block(M, N);
  // blocks beyond the grid's second dimension go in further launches
  const int64_t chunks = (M + per - 1) / per;
  const bool store = act != kLinearNoAct;
  for (int64_t c = 0; c < chunks; c += 65535) {
    const int64_t n = std::min<int64_t>(65535, chunks - c), r = c * per, rows = std::min(M - r, n * per);
    const dim3 grid(static_cast<unsigned>((N + kCols - 1) / kCols), static_cast<unsigned>(n));
    const uint16_t* g = static_cast<const uint16_t*>(dy) + r * lddy;
    const uint16_t* v = store ? static_cast<const uint16_t*>(z) + r * N : nullptr;
    uint16_t* to = store ? static_cast<uint16_t*>(dz) + r * N : nullptr;
    const SumsTo p{db != nullptr && !few ? part + c * N : nullptr, few ? db : nullptr, dtype, accumulate};
    const cudaError_t e = f16 ? launch_dz<true>(grid, g, v, to, p, rows, N, lddy, per, act, stream)
                              : launch_dz<false>(grid, g, v, to, p, rows, N, lddy, per, act, stream);
    if (e != cudaSuccess) return e;
  }
  if (db == nullptr || few) return cudaSuccess;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = dependent_launch(dim3(static_cast<unsigned>((N + 31) / 32)), 32 * kSumWarps, stream, attr);
  return cudaLaunchKernelEx(&cfg, linear_db_kernel, static_cast<const float*>(part), chunks, N, db,
                            dtype, accumulate);
}

}  // namespace swg
