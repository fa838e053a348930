// The linear layer's products with a large result, on CTA pairs: out[i][j] = sum_r A[i, r] B[j, r] with
//   forward  y[m][n]:  i = m, j = n, r = k   A = x (r innermost), B = w (r outermost)
//   dx[m][k]:          i = m, j = k, r = n   A = dz, B = w (r innermost in both)
//   dw[k][n]:          i = k, j = n, r = m   A = x, B = dz (r outermost in both)
// Bound by the tensor cores. One persistent pair (a cluster of two) for every two SMs walks over tiles of 256 x 256
// outputs, or 256 x 512 (see pair_plan_of), ten warps a CTA, here for 256 x 256:
//   warp 0 lane 0   copies, for every 64 of r, this CTA's 128 rows of A and its 128 of the 256 columns of B (16 KB each)
//                   into a ring of five stages with TMA, counted on the leader's barrier: each SM copies half of B
//   warp 1          tensor memory (512 columns in each CTA: two accumulators of 256); lane 0 of the leader issues
//                   tcgen05.mma.cta_group::2 (M = 256, N = 256, K = 16)
//   warps 2-9       drain the finished accumulator (each CTA its own 128 rows; two warps a quarter of the lanes, each on
//                   half of the columns) while the tensor cores fill the other one: bias, activation and residual in
//                   fp32, 64 columns at a time, through staging blocks of 32 rows x 128 bytes and TMA stores. The bias is
//                   loaded under the products and passed around through shared memory (by shuffles: 1130
//                   clocks for 64 columns instead of 550); a residual (or the old dw) comes by TMA loads two blocks ahead.
// Tiles in flight share operands: eight tile rows at a time, the row index fastest (Walk).
// Measured, bf16: 16384 x 14336 x 4096 with residual 1128 to 1157 us a call, which runs under the power cap (85 to 87% of the
// measured tensor rate, 97 to 100% of the sustained one; 1010 us before the clock slows), 220000 x 512 x 1024 with GELU and z
// 274 to 299 us, bound by the epilogue: of 11000 clocks a tile 7800 are the activation's. The wide form's epilogue spills 240
// bytes a thread and loads 300, for its residual's registers.
// A reduction too long for too few tiles, or for one accumulator (dw), is cut into parts: fp32 partial results, added by a
// second kernel in a fixed order.
//
// Every wait is bounded; a timeout sets the status word, stops issuing, drains the pair's copies, frees TMEM and returns.
#include <algorithm>

#include "linear.cuh"

namespace swg {
namespace {

using namespace lin;

constexpr int BM = 128;                // rows of a tile in each CTA
constexpr int BN = 256;                // columns of an instruction
constexpr int BK = 64;                 // reduction block
constexpr int kHalf = 128 * BK * 2;    // 16 KB: an operand's share of a stage in a CTA
constexpr int kBox = 64 * BK * 2;      // a box of 64 x 64 elements
constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int kOut = 4096;             // a staged block of 32 rows x 64 columns
constexpr int kRes = 2048;             // a residual block of 32 x 32
constexpr uint32_t kTmemCols = 512;

// kWide: tiles of 256 x 512 (see pair_plan_of)
template <bool kWide>
struct Form {
  static constexpr int kHalves = kWide ? 2 : 1;      // of 256 columns
  static constexpr int kStages = kWide ? 4 : 5;
  static constexpr int kBuffers = kWide ? 1 : 2;     // accumulators in TMEM
  static constexpr int kColumns = BN * kHalves;      // of a tile
  static constexpr int kStaged = kWide ? 4096 : 8192;
};
template <bool kWide>
struct __align__(1024) PairSmem {
  static constexpr int STAGES = Form<kWide>::kStages;
  uint8_t a[STAGES][kHalf];
  uint8_t b[STAGES][Form<kWide>::kHalves * kHalf];
  // a warp's blocks for TMA stores: two, or with a residual one and two residual blocks; of wide tiles one
  uint8_t stage[kEpiWarps][Form<kWide>::kStaged];
  float bias[kEpiWarps][32];          // of a warp's 32 columns
  uint64_t full[STAGES];              // leader: both CTAs' copies of the stage have landed
  uint64_t empty[STAGES];             // the MMAs reading the stage are done (committed to both CTAs)
  uint64_t tmem_full[2];              // the tile's MMAs into this accumulator are done (both CTAs)
  uint64_t tmem_empty[2];             // leader: both CTAs' epilogue warps have read it out
  uint64_t res_full[kEpiWarps][2];    // a residual block has landed
  uint32_t tmem_base;
  volatile uint32_t abort_flag;
  volatile uint32_t issued, consumed;
};

struct PairArgs {
  Epilogue epi;
  uint32_t* status;
  float* part;             // fp32 partial results [parts][I][J], or null
  int I, J;
  int tiles_i, tiles_j;    // tiles
  int tiles, parts;        // tiles of all parts
  int nkb, per;            // blocks of 64 of r, of a part
  long long wait_limit;
  int64_t stall_at;        // test injection: the producers stop before this ring entry (-1: never)
};

struct Tile {
  int i0, j0, kb, n, part;  // first row and column; first block of r and their number
};
// The walk over the tiles: parts one after the other; in a part bands of eight tile rows, in a band column after column, the
// row index fastest, so that the tiles in flight (76 pairs) read a square of some eight rows and ten columns of operand
// tiles. Kept as a position, not found by divisions (four of them took a sixth of a short tile's epilogue).
template <bool kWide>
struct Walk {
  static constexpr int kBand = 8;
  int t = 0, part = 0, band = 0, in = 0;  // the tile, its part, the first row of its band, its place in the band
  __device__ __forceinline__ Walk(int first, const PairArgs& a) { step(first, a); }
  __device__ __forceinline__ void step(int n, const PairArgs& a) {
    t += n;
    in += n;
    while (t < a.tiles) {
      const int size = min(kBand, a.tiles_i - band) * a.tiles_j;
      if (in < size) break;
      in -= size;
      if ((band += kBand) >= a.tiles_i) {
        band = 0;
        ++part;
      }
    }
  }
  __device__ __forceinline__ bool more(const PairArgs& a) const { return t < a.tiles; }
  __device__ __forceinline__ Tile tile(const PairArgs& a) const {
    const int rows = min(kBand, a.tiles_i - band);
    const int j = rows == kBand ? in / kBand : in / rows;
    Tile w;
    w.i0 = (band + in - j * rows) * 2 * BM;
    w.j0 = j * Form<kWide>::kColumns;
    w.part = part;
    w.kb = part * a.per;
    w.n = min(a.per, a.nkb - w.kb);
    return w;
  }
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// waits for the loads from tensor memory; what they read is not touched before
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}

// kAOuter, kBOuter: whether r is the outermost dimension of the operand in memory
template <bool kAOuter, bool kBOuter, bool kF16, bool kWide>
__global__ void __launch_bounds__(kThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                       const __grid_constant__ CUtensorMap tm_y, const __grid_constant__ CUtensorMap tm_z,
                       const __grid_constant__ CUtensorMap tm_r, const PairArgs args) {
  using F = Form<kWide>;
  constexpr int STAGES = F::kStages;
  extern __shared__ uint8_t smem_raw[];
  PairSmem<kWide>& s = *reinterpret_cast<PairSmem<kWide>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const bool leader = crank == 0;
  const int pair_id = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
  const Epilogue& p = args.epi;

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.tmem_full[i], 1);
      mbar_init(&s.tmem_empty[i], 2 * kEpiWarps);
      for (int w = 0; w < kEpiWarps; ++w) mbar_init(&s.res_full[w][i], 1);
    }
    s.abort_flag = s.issued = s.consumed = 0u;
    fence_mbar_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  if (warp == 1) {
    tmem_alloc_pair(&s.tmem_base, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();  // both CTAs' barriers are initialised before any remote arrival, commit or copy
  const uint32_t tmem = s.tmem_base;
  // what the kernel before this one wrote is visible from here on
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  auto timeout = [&]() {
    if (args.status != nullptr) atomicOr(args.status, kStatusTimeout);
    s.abort_flag = 1u;
  };

  if (warp == 0) {
    if (lane == 0) {
      uint32_t gj = 0;
      bool stopped = false;
      for (Walk<kWide> at(pair_id, args); at.more(args) && !s.abort_flag && !stopped; at.step(pairs, args)) {
        const Tile w = at.tile(args);
        const int i0 = w.i0 + BM * static_cast<int>(crank);
        for (int i = 0; i < w.n && !s.abort_flag; ++i, ++gj) {
          if (static_cast<int64_t>(gj) == args.stall_at) {
            stopped = true;
            break;
          }
          const int st = gj % STAGES;
          if (gj >= STAGES && !mbar_wait(&s.empty[st], ((gj / STAGES) - 1) & 1, args.wait_limit)) {
            timeout();
            break;
          }
          if (leader) mbar_arrive_expect_tx(&s.full[st], 2 * (1 + F::kHalves) * kHalf);  // both CTAs' copies
          const uint32_t full = cluster_addr(&s.full[st], 0);
          const int r = (w.kb + i) * BK;
          if (kAOuter) {
            tma_load_2d_pair(s.a[st], &tm_a, full, i0, r);
            tma_load_2d_pair(s.a[st] + kBox, &tm_a, full, i0 + 64, r);
          } else {
            tma_load_2d_pair(s.a[st], &tm_a, full, r, i0);
          }
#pragma unroll
          for (int h = 0; h < F::kHalves; ++h) {  // this CTA's 128 columns of each 256
            uint8_t* pb = s.b[st] + h * kHalf;
            const int j0 = w.j0 + BN * h + 128 * static_cast<int>(crank);
            if (kBOuter) {
              tma_load_2d_pair(pb, &tm_b, full, j0, r);
              tma_load_2d_pair(pb + kBox, &tm_b, full, j0 + 64, r);
            } else {
              tma_load_2d_pair(pb, &tm_b, full, r, j0);
            }
          }
          s.issued = gj + 1;
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      const uint32_t idesc = idesc_f32(2 * BM, BN, kAOuter, kBOuter, kF16);
      auto commit2 = [](uint64_t* bar) {  // to the barrier at the same offset in both CTAs
        umma_commit_pair(cluster_addr(bar, 0));
        umma_commit_pair(cluster_addr(bar, 1));
      };
      uint32_t gj = 0, it = 0;
      bool ok = true;
      for (Walk<kWide> at(pair_id, args); at.more(args) && ok; at.step(pairs, args), ++it) {
        const Tile w = at.tile(args);
        const uint32_t buf = it % F::kBuffers;
        if (it >= F::kBuffers) {
          if (!mbar_wait(&s.tmem_empty[buf], (it / F::kBuffers - 1) & 1, args.wait_limit)) {
            timeout();
            break;
          }
          tc_fence_after();
        }
        const uint32_t d = tmem + buf * BN;
        for (int i = 0; i < w.n; ++i, ++gj) {
          const int st = gj % STAGES;
          if (!mbar_wait(&s.full[st], (gj / STAGES) & 1, args.wait_limit)) {
            timeout();
            ok = false;
            break;
          }
          s.consumed = gj + 1;
          tc_fence_after();
          const uint32_t pa = smem_u32(s.a[st]), pb = smem_u32(s.b[st]);
#pragma unroll
          for (int k = 0; k < BK / 16; ++k) {
            const uint64_t da = kAOuter ? smem_desc(pa + 2048 * k, kBox, 1024) : smem_desc(pa + 32 * k, 16, 1024);
#pragma unroll
            for (int h = 0; h < F::kHalves; ++h) {
              const uint32_t ph = pb + h * kHalf;
              const uint64_t db = kBOuter ? smem_desc(ph + 2048 * k, kBox, 1024) : smem_desc(ph + 32 * k, 16, 1024);
              umma_pair(d + h * BN, da, db, idesc, (i > 0 || k > 0) ? 1u : 0u);
            }
          }
          commit2(&s.empty[st]);
        }
        if (ok) commit2(&s.tmem_full[buf]);
      }
    }
  } else {
    const int q = warp & 3;            // TMEM lane quarter this warp may read
    const int e = warp - 2, half = e >> 2;
    const bool add = p.residual != nullptr && args.part == nullptr;
    const bool ahead = add && !kWide;  // the residual comes by TMA, two blocks ahead; in wide tiles by loads
    constexpr int kMine = F::kColumns / 2;  // columns of this warp
    bool dead = false;
    uint32_t it = 0, nb = 0;           // tiles, staged blocks
    // the residual's blocks of 32 columns, four a tile: two of them are under way
    uint32_t nf = 0, nr = 0;           // asked for, read
    Walk<kWide> ft(pair_id, args);     // the tile of the next one
    auto fetch = [&]() {
      if (!ft.more(args)) return;
      if (lane == 0) {
        const Tile w = ft.tile(args);
        uint64_t* bar = &s.res_full[e][nf & 1];
        mbar_arrive_expect_tx(bar, kRes);
        tma_load_2d(s.stage[e] + kOut + (nf & 1) * kRes, &tm_r, bar, w.j0 + half * 128 + (nf & 3) * 32,
                    w.i0 + BM * static_cast<int>(crank) + q * 32);
      }
      if ((++nf & 3) == 0) ft.step(pairs, args);
    };
    if (ahead) {
      fetch();
      fetch();
    }
    // the next block for a store, which the store that used it has read
    auto staged = [&]() -> uint8_t* {
      if (lane == 0) {
        if (add || kWide) bulk_wait_read<0>();
        else bulk_wait_read<1>();
      }
      __syncwarp();
      return s.stage[e] + (add || kWide ? 0 : (nb & 1) * kOut);
    };
    auto store = [&](const CUtensorMap* tm, const uint8_t* blk, int col, int row0) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (row0 < args.I) tma_store_2d(tm, blk, col, row0);
        bulk_commit();
      }
      ++nb;
    };
    // the bias of this lane's column in a block of 32 of a tile, as it is in memory: widened where it is used, so that
    // nothing waits for the load before
    auto bias_of = [&](const Tile& w, int c) -> uint32_t {
      const int j = w.j0 + half * kMine + c * 32 + lane;
      if (p.bias == nullptr || j >= args.J) return 0u;
      return p.bias_f32 ? static_cast<const uint32_t*>(p.bias)[j] : static_cast<const uint16_t*>(p.bias)[j];
    };
    Walk<kWide> at(pair_id, args);
    Tile next = at.tile(args);
    uint32_t b0 = bias_of(next, 0), b1 = bias_of(next, 1);  // loaded under the columns before them
    for (bool more = at.more(args); more; ++it) {
      const Tile w = next;
      at.step(pairs, args);
      if ((more = at.more(args))) next = at.tile(args);
      const uint32_t buf = it % F::kBuffers;
      const int row0 = w.i0 + BM * static_cast<int>(crank) + q * 32, col0 = w.j0 + half * kMine;
      bool ready = false;
      if (!dead && !s.abort_flag) {
        ready = mbar_wait(&s.tmem_full[buf], (it / F::kBuffers) & 1, args.wait_limit);
        if (!ready) {
          timeout();
          dead = true;
        }
      }
      tc_fence_after();
      // tcgen05.ld is warp-collective: decide for the whole warp
      if (__all_sync(0xffffffffu, ready && !s.abort_flag)) {
        const uint32_t d = tmem + (static_cast<uint32_t>(q * 32) << 16) + buf * BN + half * kMine;
        const uint32_t swz = lane & 7;           // 128-byte swizzle of this lane's row: 16-byte chunk j ^ swz
        const uint32_t swr = (lane >> 1) & 3;    // 64-byte swizzle
#pragma unroll 1
        for (int c = 0; c < kMine / 32; c += 2) {  // 64 columns at a time
          const int col = col0 + c * 32;
          uint4 res[8] = {};
          if (kWide && add && row0 + lane < args.I) {
            const uint16_t* from = p.residual + static_cast<int64_t>(row0 + lane) * p.ldr + col;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (col + 8 * j < args.J) res[j] = *reinterpret_cast<const uint4*>(from + 8 * j);
          }
          uint32_t v[2][32];
          tmem_ld_32x32b_x32(d + c * 32, v[0]);
          tmem_ld_32x32b_x32(d + c * 32 + 32, v[1]);
          tmem_loaded(v[0]);
          tmem_loaded(v[1]);
          if (args.part != nullptr) {
            const int row = row0 + lane;
            if (row < args.I) {
              float* to = args.part + (static_cast<int64_t>(w.part) * args.I + row) * args.J + col;
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const uint32_t* x = v[j >> 3] + 4 * (j & 7);
                if (col + 4 * j < args.J) reinterpret_cast<uint4*>(to)[j] = make_uint4(x[0], x[1], x[2], x[3]);
              }
            }
            __syncwarp();
            continue;
          }
          float2 f[2][16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            f[0][i] = make_float2(__uint_as_float(v[0][2 * i]), __uint_as_float(v[0][2 * i + 1]));
            f[1][i] = make_float2(__uint_as_float(v[1][2 * i]), __uint_as_float(v[1][2 * i + 1]));
          }
          if (p.bias != nullptr) {  // from each lane's register to all lanes, through shared memory
            float* row = s.bias[e];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t raw = h == 0 ? b0 : b1;
              row[lane] = p.bias_f32 ? __uint_as_float(raw) : widen2<kF16>(raw).x;
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 b = *reinterpret_cast<const float4*>(row + 4 * i);
                f[h][2 * i] = __fadd2_rn(f[h][2 * i], make_float2(b.x, b.y));
                f[h][2 * i + 1] = __fadd2_rn(f[h][2 * i + 1], make_float2(b.z, b.w));
              }
              __syncwarp();
            }
            const bool last = c + 2 == kMine / 32;
            b0 = bias_of(last ? next : w, last ? 0 : c + 2);
            b1 = bias_of(last ? next : w, last ? 1 : c + 3);
          }
          if (p.z != nullptr) {
            uint8_t* blk = staged();
            const uint32_t to = smem_u32(blk) + lane * 128;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float2* x = f[j >> 2] + 4 * (j & 3);
              sts128(to + ((j ^ swz) << 4), make_uint4(narrow2<kF16>(x[0]), narrow2<kF16>(x[1]), narrow2<kF16>(x[2]),
                                                       narrow2<kF16>(x[3])));
            }
            store(&tm_z, blk, col, row0);
          }
          with_act(p.act, [&](auto act) {
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i >> 4][i & 15] = activate<decltype(act)::value>(f[i >> 4][i & 15]);
          });
          if (kWide && add) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float2 r[4];
              widen8<kF16>(res[j], r);
#pragma unroll
              for (int i = 0; i < 4; ++i) f[j >> 2][4 * (j & 3) + i] = __fadd2_rn(f[j >> 2][4 * (j & 3) + i], r[i]);
            }
          }
          if (ahead) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              if (!mbar_wait(&s.res_full[e][nr & 1], (nr >> 1) & 1, args.wait_limit)) {
                timeout();
                dead = true;
              }
              const uint32_t rb = smem_u32(s.stage[e] + kOut + (nr & 1) * kRes) + lane * 64;
              ++nr;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                float2 r[4];
                widen8<kF16>(lds128(rb + ((j ^ swr) << 4)), r);
#pragma unroll
                for (int i = 0; i < 4; ++i) f[k][4 * j + i] = __fadd2_rn(f[k][4 * j + i], r[i]);
              }
              __syncwarp();  // the block has been read by every lane
              fetch();
            }
          }
          uint8_t* blk = staged();
          const uint32_t to = smem_u32(blk) + lane * 128;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2* x = f[j >> 2] + 4 * (j & 3);
            sts128(to + ((j ^ swz) << 4), make_uint4(narrow2<kF16>(x[0]), narrow2<kF16>(x[1]), narrow2<kF16>(x[2]),
                                                     narrow2<kF16>(x[3])));
          }
          store(&tm_y, blk, col, row0);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {  // this warp has read its part of the accumulator: tell the leader's MMA issuer
        if (leader) mbar_arrive(&s.tmem_empty[buf]);
        else mbar_arrive_remote(cluster_addr(&s.tmem_empty[buf], 0));
      }
    }
    if (lane == 0) {
      bulk_wait_all();  // every store has landed before the CTA exits
      for (; ahead && nr < nf; ++nr)  // and every residual block that was asked for
        if (!mbar_wait(&s.res_full[e][nr & 1], (nr >> 1) & 1, args.wait_limit)) break;
    }
  }

  __syncthreads();
  cluster_sync();  // both CTAs are done with their roles: no more remote arrivals or commits
  if (leader && threadIdx.x == 0) {
    const uint32_t peer_abort = ld_cluster_u32(&s.abort_flag, 1);
    if (s.abort_flag || peer_abort) {
      const uint32_t peer_issued = ld_cluster_u32(&s.issued, 1);
      const uint32_t issued = s.issued > peer_issued ? s.issued : peer_issued;
      for (uint32_t i = s.consumed; i < issued; ++i)
        if (!mbar_wait(&s.full[i % STAGES], (i / STAGES) & 1, args.wait_limit)) break;
    }
  }
  cluster_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// out = the sum of the parts in order (+ the old out), rounded once
template <bool kF16>
__global__ void __launch_bounds__(256) linear_parts_kernel(const float4* part, int parts, int64_t n4, uint2* out,
                                                           bool accumulate) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n4;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    float4 s = part[i], t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // 64 in sequence, and these sums
    for (int k = 1; k < parts; ++k) {
      if (k % 64 == 0) {
        t = make_float4(t.x + s.x, t.y + s.y, t.z + s.z, t.w + s.w);
        s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
      const float4 v = part[k * n4 + i];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    s = make_float4(t.x + s.x, t.y + s.y, t.z + s.z, t.w + s.w);
    if (accumulate) {
      const uint2 o = out[i];
      const float2 a = widen2<kF16>(o.x), b = widen2<kF16>(o.y);
      s.x += a.x;
      s.y += a.y;
      s.z += b.x;
      s.w += b.y;
    }
    out[i] = make_uint2(narrow2<kF16>(make_float2(s.x, s.y)), narrow2<kF16>(make_float2(s.z, s.w)));
  }
}

}  // namespace

// A plan with tiles of 256 x 256 or 256 x 512, and an estimate of its time in microseconds.
//   narrow  0.36 us for 64 of r: the rate at which the SMs get 64 KB a pair from L2 (14 TB/s in all), not the tensor
//           cores' (0.27 us); the epilogue runs under the next tile's products
//   wide    0.62 us for twice the products, as a pair's copies of A serve 512 columns (96 KB); the accumulator is the
//           whole of tensor memory, so that the epilogue stops the tensor cores, 3.5 us a tile for a gradient's plain
//           rounding, 9 with bias, activation or residual
// Measured, us, narrow and wide, in short runs of each: forward 16384x14336x4096 1105 and 1056, 4096x4096x14336 285 and 318; dx of
// 4096x4096x14336 300 and 277, of 220000x1024x512 174 and 206; dw of 16384x14336x4096 1160 and 1020, of 2048x4096x4096
// 62 and 48.
PairPlan pair_plan_of(int64_t I, int64_t J, int64_t R, bool gradient, bool cut, bool wide, int sms) {
  PairPlan p;
  p.wide = wide;
  const int64_t columns = wide ? 2 * BN : BN;
  p.tiles_i = (I + 2 * BM - 1) / (2 * BM);
  p.tiles_j = (J + columns - 1) / columns;
  p.nkb = (R + BK - 1) / BK;
  p.parts = 1;
  const int64_t tiles = p.tiles_i * p.tiles_j, pairs = std::max(1, sms / 2);
  // cut where whole tiles leave half of the pairs without work, into parts of 16 blocks or more, and where one accumulator
  // would take more than kMostBlocks
  if (cut && 2 * tiles <= pairs) p.parts = std::max<int64_t>(1, std::min(pairs / tiles, p.nkb / 16));
  if (cut) p.parts = std::max(p.parts, (p.nkb + kMostBlocks - 1) / kMostBlocks);
  p.per = (p.nkb + p.parts - 1) / p.parts;
  p.parts = (p.nkb + p.per - 1) / p.per;
  p.part_bytes = p.parts > 1 ? static_cast<size_t>(p.parts) * I * J * sizeof(float) : 0;
  const double waves = static_cast<double>((tiles * p.parts + pairs - 1) / pairs), per = static_cast<double>(p.per);
  p.us = wide ? waves * (per * 0.62 + (gradient ? 3.5 : 9.0)) + 4.0 : waves * std::max(per * 0.36, 4.0) + 5.5;
  if (p.parts > 1) p.us += 4.0 + static_cast<double>(p.part_bytes) / 3e6;
  return p;
}
PairPlan linear_pair_plan(int64_t I, int64_t J, int64_t R, bool gradient, bool cut, int sms) {
  const PairPlan narrow = pair_plan_of(I, J, R, gradient, cut, false, sms),
                 wide = pair_plan_of(I, J, R, gradient, cut, true, sms);
  return wide.us < narrow.us ? wide : narrow;
}

template <bool kAOuter, bool kBOuter>
cudaError_t launch_linear_pair(const void* A, int64_t lda, const void* B, int64_t ldb, int64_t I, int64_t J, int64_t R,
                        const LinearEpilogue& e, const PairPlan& plan, float* part, cudaStream_t stream) {
  CUtensorMap ma, mb, my, mz, mr;
  const uint64_t i = I, j = J, r = R, sa = lda * 2, sb = ldb * 2;
  const bool ok =
      (kAOuter ? encode_tmap_2d_bf16(&ma, A, i, r, sa, 64, BK) : encode_tmap_2d_bf16(&ma, A, r, i, sa, BK, BM)) &&
      (kBOuter ? encode_tmap_2d_bf16(&mb, B, j, r, sb, 64, BK) : encode_tmap_2d_bf16(&mb, B, r, j, sb, BK, 128)) &&
      encode_tmap_2d_bf16(&my, e.y, j, i, j * 2, 64, 32) &&
      encode_tmap_2d_bf16(&mz, e.z != nullptr ? e.z : e.y, j, i, j * 2, 64, 32) &&
      encode_tmap_2d_bf16(&mr, e.residual != nullptr ? e.residual : e.y, j, i, (e.residual != nullptr ? e.ldr : J) * 2, 32,
                          32, 64);
  if (!ok) return cudaErrorInvalidValue;
  const Injection inj = take_injection(kInjectLinear);
  PairArgs a{};
  a.epi = epilogue_of(e);
  a.status = status_word_ptr();
  a.part = plan.parts > 1 ? part : nullptr;
  a.I = static_cast<int>(I);
  a.J = static_cast<int>(J);
  a.tiles_i = static_cast<int>(plan.tiles_i);
  a.tiles_j = static_cast<int>(plan.tiles_j);
  a.parts = static_cast<int>(plan.parts);
  a.tiles = static_cast<int>(plan.tiles_i * plan.tiles_j * plan.parts);
  a.nkb = static_cast<int>(plan.nkb);
  a.per = static_cast<int>(plan.per);
  a.wait_limit = inj.wait_limit;
  a.stall_at = inj.stall_at;
  static_assert(sizeof(PairSmem<false>) + 1024 <= 232448 && sizeof(PairSmem<true>) + 1024 <= 232448,
                "linear pair kernel shared memory");
  const size_t smem = (plan.wide ? sizeof(PairSmem<true>) : sizeof(PairSmem<false>)) + 1024;
  const auto kernel = plan.wide ? (e.f16 ? linear_pair_kernel<kAOuter, kBOuter, true, true>
                                         : linear_pair_kernel<kAOuter, kBOuter, false, true>)
                                : (e.f16 ? linear_pair_kernel<kAOuter, kBOuter, true, false>
                                         : linear_pair_kernel<kAOuter, kBOuter, false, false>);
  cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  const int pairs = std::max(1, std::min(device_sm_count() / 2, a.tiles));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  err = cudaLaunchKernelEx(&cfg, kernel, ma, mb, my, mz, mr, a);
  if (err != cudaSuccess || plan.parts == 1) return err;
  const int64_t n4 = I * J / 4;
  const auto add = e.f16 ? linear_parts_kernel<true> : linear_parts_kernel<false>;
  add<<<static_cast<unsigned>(std::min<int64_t>((n4 + 255) / 256, 4096)), 256, 0, stream>>>(
      reinterpret_cast<const float4*>(part), a.parts, n4, static_cast<uint2*>(e.y), e.residual != nullptr);
  return cudaGetLastError();
}

template cudaError_t launch_linear_pair<false, true>(const void*, int64_t, const void*, int64_t, int64_t, int64_t, int64_t,
                                              const LinearEpilogue&, const PairPlan&, float*, cudaStream_t);
template cudaError_t launch_linear_pair<false, false>(const void*, int64_t, const void*, int64_t, int64_t, int64_t, int64_t,
                                               const LinearEpilogue&, const PairPlan&, float*, cudaStream_t);
template cudaError_t launch_linear_pair<true, true>(const void*, int64_t, const void*, int64_t, int64_t, int64_t, int64_t,
                                             const LinearEpilogue&, const PairPlan&, float*, cudaStream_t);

}  // namespace swg
