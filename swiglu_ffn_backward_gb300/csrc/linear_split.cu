// The linear layer's products with a small result: few rows (decoding, short batches), or a weight gradient
// with a long reduction. out[c][l] = sum_r A[l, r] B[c, r], where l runs over the contiguous dimension of out
// and c over its rows:
//   forward  y[m][n]:  l = n, c = m, r = k   A = w (r outermost), B = x (r innermost)
//   dx[m][k]:          l = k, c = m, r = n   A = w (r innermost), B = dz (r innermost)
//   dw[k][n]:          l = n, c = k, r = m   A = dz, B = x (r outermost in both)
// so that the weights, which are most of what a small call reads, are the 128-wide operand of the tensor
// instruction (tcgen05.mma M = 128), and the rows of out its N: 16 to 256, as many as there are.
//
// What bounds it: reading w once, for few rows. One tile [128 l x NT c] is shared by a cluster of S blocks, each of
// which takes a part of the reduction, so that all SMs read although there are only N / 128 tiles; the parts are
// added in the cluster through shared memory in the blocks' order (no atomics, no workspace, one launch).
//
// A block: warp 0 lane 0 copies operand tiles (64 of r) into a ring with TMA, warp 1 lane 0 issues the tensor
// instructions into TMEM; then all warps move the sums from TMEM into the ring's memory, add the cluster's parts, each
// block a share of the tile, and apply the epilogue: 16-byte loads and stores. A programmatic dependent launch: its
// set-up runs beside the end of the kernel before it.
//
// Measured, bf16: 1 x 14336 x 4096 22 us and 77 x 4096 x 14336 25.4 us a call (79 and 70% of the copy rate, on one w of 117
// MB, a part of which L2 still holds); with three w's in turn 24.1 and 26.7 us (72 and 66%). 257 x 512 x 1024 with
// everything in L2 6.2 us, which is three launches' latencies and no rate.
//
// Every wait is bounded: a block whose wait ran out sets the status word, issues nothing more, waits (bounded) for
// its copies and products in flight and goes through the cluster's barriers like the others.
#include <algorithm>

#include "linear.cuh"

namespace swg {
namespace {

using namespace lin;

constexpr int kLanes = 128;               // of l in a tile
constexpr int kRed = 64;                  // of r in a stage
constexpr int kABytes = kLanes * kRed * 2;
constexpr int kMaxStages = 16;
constexpr int kThreads = 256;
constexpr int kBoxBytes = 64 * kRed * 2;  // a box of 64 x 64 elements
constexpr int kMaxSplit = 8;              // portable cluster size
constexpr int kMostRing = 196 * 1024;     // bytes of a ring

struct SplitArgs {
  Epilogue epi;
  uint32_t* status;
  int L, C;              // sizes of l and c
  int NT;                // c in a tile: a multiple of 16 (of 64 where r is B's outermost dimension), up to 256
  int tiles_l, tiles_c;
  int nkb, S;            // blocks of 64 of r; blocks of a cluster
  int stages;
  long long wait_limit;
  int64_t stall_at;      // test injection: the producer of a cluster's last block stops there (-1: never)
};

struct SplitControl {
  uint64_t full[kMaxStages], empty[kMaxStages], done;
  uint32_t tmem_base;
  volatile uint32_t abort_flag, issued, consumed;
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {  // volatile: it stays between the cluster's barriers
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

// kAOuter, kBOuter: whether r is the outermost dimension of the operand in memory
template <bool kAOuter, bool kBOuter, bool kF16>
__global__ void __launch_bounds__(kThreads, 2)
    linear_split_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                        const SplitArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ SplitControl s;
  uint8_t* const ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = a.S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / a.S;
  const int l0 = (tile % a.tiles_l) * kLanes, c0 = (tile / a.tiles_l) * a.NT;
  const int stage_bytes = kABytes + a.NT * kRed * 2;
  // this block's part of the reduction: at least one block of 64
  const int kb0 = static_cast<int>(static_cast<int64_t>(a.nkb) * rank / a.S);
  const int n = static_cast<int>(static_cast<int64_t>(a.nkb) * (rank + 1) / a.S) - kb0;
  const uint32_t tmem_cols = a.NT <= 32 ? 32 : a.NT <= 64 ? 64 : a.NT <= 128 ? 128 : 256;

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    mbar_init(&s.done, 1);
    s.abort_flag = s.issued = s.consumed = 0u;
    fence_mbar_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  if (warp == 1) {
    tmem_alloc(&s.tmem_base, tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  // everything above ran beside the end of the kernel before this one; its writes are visible from here on
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  auto timeout = [&]() {
    if (a.status != nullptr) atomicOr(a.status, kStatusTimeout);
    s.abort_flag = 1u;
  };

  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < n && !s.abort_flag; ++i) {
        if (rank == a.S - 1 && i == a.stall_at) break;
        const int st = i % a.stages;
        if (i >= a.stages && !mbar_wait(&s.empty[st], ((i / a.stages) - 1) & 1, a.wait_limit)) {
          timeout();
          break;
        }
        mbar_arrive_expect_tx(&s.full[st], stage_bytes);
        uint8_t *pa = ring + st * stage_bytes, *pb = pa + kABytes;
        const int r = (kb0 + i) * kRed;
        if (kAOuter) {
          tma_load_2d(pa, &tm_a, &s.full[st], l0, r);
          tma_load_2d(pa + kBoxBytes, &tm_a, &s.full[st], l0 + 64, r);
        } else {
          tma_load_2d(pa, &tm_a, &s.full[st], r, l0);
        }
        if (kBOuter) {
          for (int j = 0; j < a.NT / 64; ++j) tma_load_2d(pb + j * kBoxBytes, &tm_b, &s.full[st], c0 + 64 * j, r);
        } else {
          tma_load_2d(pb, &tm_b, &s.full[st], r, c0);
        }
        s.issued = i + 1;
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_f32(kLanes, a.NT, kAOuter, kBOuter, kF16);
      for (int i = 0; i < n; ++i) {
        const int st = i % a.stages;
        if (!mbar_wait(&s.full[st], (i / a.stages) & 1, a.wait_limit)) {
          timeout();
          break;
        }
        s.consumed = i + 1;
        tc_fence_after();
        const uint32_t pa = smem_u32(ring + st * stage_bytes), pb = pa + kABytes;
#pragma unroll
        for (int k = 0; k < kRed / 16; ++k) {
          const uint64_t da = kAOuter ? smem_desc(pa + 2048 * k, kBoxBytes, 1024) : smem_desc(pa + 32 * k, 16, 1024);
          const uint64_t db = kBOuter ? smem_desc(pb + 2048 * k, kBoxBytes, 1024) : smem_desc(pb + 32 * k, 16, 1024);
          umma_bf16(tmem, da, db, idesc, (i > 0 || k > 0) ? 1u : 0u);
        }
        umma_commit(&s.empty[st]);
      }
      umma_commit(&s.done);  // also after a timeout: what was issued has to be done before TMEM and the ring are reused
    }
  }
  // every thread waits for the products, and so for the copies that they read: as long as they come on
  __syncwarp();
  uint32_t seen = ~0u;
  while (!mbar_wait(&s.done, 0, a.wait_limit)) {
    const uint32_t now = s.consumed;
    if (now == seen) {
      timeout();
      break;
    }
    seen = now;
  }
  __syncthreads();
  if (s.abort_flag) {  // copies that nothing reads
    if (threadIdx.x == 0)
      for (uint32_t i = s.consumed; i < s.issued; ++i)
        if (!mbar_wait(&s.full[i % a.stages], (i / a.stages) & 1, a.wait_limit)) break;
    __syncthreads();
  }
  // the sums into the ring's place, [c][l]
  float* const part = reinterpret_cast<float*>(ring);
  const int cols = min(a.NT, a.C - c0);
  tc_fence_after();
  {
    const int q = warp & 3;  // TMEM lane quarter
    for (int c = (warp >> 2) * 32; c < cols; c += 64) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(q * 32) << 16) + c, v);
      tmem_ld_wait();
      float* to = part + c * kLanes + q * 32 + lane;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (c + j < cols) to[j * kLanes] = __uint_as_float(v[j]);
    }
  }
  tc_fence_before();
  if (a.S > 1) cluster_sync();
  else __syncthreads();
  // this block's share of the tile: vectors of eight elements of a row
  uint32_t peers[kMaxSplit];
#pragma unroll
  for (int i = 0; i < kMaxSplit; ++i) peers[i] = i < a.S && a.S > 1 ? cluster_addr(part, i) : smem_u32(part);
  const Epilogue& p = a.epi;
  with_act(p.act, [&](auto act) {
    for (int i = rank * kThreads + static_cast<int>(threadIdx.x); i < cols * (kLanes / 8); i += a.S * kThreads) {
      const int c = i / (kLanes / 8), l = (i % (kLanes / 8)) * 8;
      if (l0 + l >= a.L) continue;
      const int64_t row = c0 + c, at = row * a.L + l0 + l;
      uint4 res = make_uint4(0u, 0u, 0u, 0u);
      if (p.residual != nullptr) res = *reinterpret_cast<const uint4*>(p.residual + row * p.ldr + l0 + l);
      const uint32_t off = static_cast<uint32_t>(c * kLanes + l) * sizeof(float);
      // all parts' loads are under way at once
      float4 x[kMaxSplit], y[kMaxSplit];
#pragma unroll
      for (int k = 0; k < kMaxSplit; ++k) {
        if (k < a.S) {
          x[k] = ld_cluster_f4(peers[k] + off);
          y[k] = ld_cluster_f4(peers[k] + off + 16);
        }
      }
      float2 v[4] = {make_float2(x[0].x, x[0].y), make_float2(x[0].z, x[0].w), make_float2(y[0].x, y[0].y),
                     make_float2(y[0].z, y[0].w)};
#pragma unroll
      for (int k = 1; k < kMaxSplit; ++k) {
        if (k < a.S) {
          v[0] = __fadd2_rn(v[0], make_float2(x[k].x, x[k].y));
          v[1] = __fadd2_rn(v[1], make_float2(x[k].z, x[k].w));
          v[2] = __fadd2_rn(v[2], make_float2(y[k].x, y[k].y));
          v[3] = __fadd2_rn(v[3], make_float2(y[k].z, y[k].w));
        }
      }
      add_bias<kF16>(p, l0 + l, a.L, v);
      if (p.z != nullptr) *reinterpret_cast<uint4*>(p.z + at) = narrow8<kF16>(v);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = activate<decltype(act)::value>(v[e]);
      if (p.residual != nullptr) {
        float2 r[4];
        widen8<kF16>(res, r);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __fadd2_rn(v[e], r[e]);
      }
      *reinterpret_cast<uint4*>(p.y + at) = narrow8<kF16>(v);
    }
  });
  if (a.S > 1) cluster_sync();  // no block leaves while another reads its sums
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols);
  }
}

// What a product costs with tiles of 128 x NT, S blocks each, in microseconds: estimates that order the choices, from
// the rates of the tensor cores (0.36 us for 64 of r in a 128 x 256 tile on one SM), of HBM and of L2, the copies under
// way in a ring, and from what a block's start, its epilogue and the exchange in a cluster take. Measured (w from HBM):
// 1 x 14336 x 4096 by 16/6 (NT/S) 22.0 us, 16/4 24.7, 16/2 43; 77 x 4096 x 14336 by 80/2 23.7, 80/1 30, 48/2 39 (two waves);
// 257 x 512 x 1024 by 48/1 6.2, 256/8 17.6 (eight blocks of 200 KB a cluster: two waves).
struct SplitPlan {
  int NT, S, stages, per_sm, tiles_l, tiles_c, nkb;
  int64_t tiles;
  double us;
};
SplitPlan split_cost(int64_t L, int64_t C, int64_t R, int NT, int S, int per_sm, int sms) {
  SplitPlan p;
  p.NT = NT;
  p.S = S;
  p.tiles_l = static_cast<int>((L + kLanes - 1) / kLanes);
  p.tiles_c = static_cast<int>((C + NT - 1) / NT);
  p.tiles = static_cast<int64_t>(p.tiles_l) * p.tiles_c;
  p.nkb = static_cast<int>((R + kRed - 1) / kRed);
  const int stage = kABytes + NT * kRed * 2;
  p.per_sm = per_sm;
  p.stages = std::min(kMaxStages, (p.per_sm == 2 ? 108 * 1024 : kMostRing) / stage);
  // blocks that run at once, of 152 and 304: a cluster's lie in one part of the device (cudaOccupancyMaxActiveClusters)
  constexpr int kRoom[2][kMaxSplit] = {{152, 152, 138, 144, 140, 138, 105, 120}, {304, 304, 291, 296, 290, 276, 266, 288}};
  const int64_t blocks = p.tiles * S;
  const int64_t slots = std::max<int64_t>(S, static_cast<int64_t>(kRoom[p.per_sm - 1][S - 1]) * sms / 152);
  const double waves = static_cast<double>((blocks + slots - 1) / slots);
  const double on_sm = static_cast<double>(std::min<int64_t>(p.per_sm, (blocks + sms - 1) / sms));
  const double kb = static_cast<double>((p.nkb + S - 1) / S);
  const double tensor = waves * on_sm * kb * std::max(NT, 96) / 256.0 * 0.36;
  // what several tiles along c read of A comes from L2 in part
  const double again = std::min(2.0, 1.0 + 0.3 * (p.tiles_c - 1));
  // 64 of r: A at most at 48 KB/us a block and 65 an SM, whatever the ring's depth, everything at 130 an SM, and the
  // ring's copies have to cover their latency
  const double from_hbm = kABytes * again / p.tiles_c;
  const double block = std::max(on_sm > 1 ? from_hbm * 2.0 / 65e3 : from_hbm / 48e3, on_sm * stage / 130e3);
  const double stream = waves * kb * std::max(block, (1.0 + 0.7 * kABytes / stage) / p.stages);
  const double l2 = static_cast<double>(p.tiles) * (kLanes + NT) * R * 2 / 14e6;
  const double hbm = (static_cast<double>(p.tiles_l) * kLanes * again + static_cast<double>(C)) * R * 2 /
                     6.5e6;
  const double finish = 1.0 + 0.02 * NT + (S > 1 ? 0.5 + 0.007 * NT * S : 0.0);
  p.us = std::max(std::max(tensor, stream), std::max(l2, hbm)) + waves * (2.5 + finish);
  return p;
}
// The cheapest of the tiles that cover C evenly and of the cluster sizes.
SplitPlan split_search(int64_t L, int64_t C, int64_t R, bool b_outer, int sms) {
  const int unit = b_outer ? 64 : 16;
  const int64_t nkb = (R + kRed - 1) / kRed, least = (C + 255) / 256;
  SplitPlan best;
  best.us = -1.0;
  int last = 0;
  for (int64_t n = least; n < least + 8; ++n) {  // tiles along c
    int NT = static_cast<int>(((C + n - 1) / n + unit - 1) / unit * unit);
    if (NT > 128) NT = 256;  // 160 to 208 took as long for 64 of r (200 x 4096 x 14336 34.8 us by 208, 32.7 by 256)
    if (NT == last) continue;
    last = NT;
    for (int S = 1; S <= kMaxSplit && S <= nkb; ++S) {
      for (int per_sm = 1; per_sm <= (NT <= 128 ? 2 : 1); ++per_sm) {  // blocks an SM: with three stages or more each
        const SplitPlan p = split_cost(L, C, R, NT, S, per_sm, sms);
        if (best.us < 0.0 || p.us < best.us) best = p;
      }
    }
  }
  return best;
}

// The same, remembered for the sizes that a thread used last (a search takes some 8 us of the host, as much as a small
// product): a function of the sizes alone.
SplitPlan split_plan(int64_t L, int64_t C, int64_t R, bool b_outer, int sms) {
  struct Entry {
    int64_t L = -1, C, R;
    int sms;
    bool b_outer;
    SplitPlan plan;
  };
  constexpr uint64_t kEntries = 64;
  static thread_local Entry entries[kEntries];
  const uint64_t h = (static_cast<uint64_t>(L) * 0x9e3779b97f4a7c15ull ^ static_cast<uint64_t>(C) * 0xc2b2ae3d27d4eb4full ^
                      static_cast<uint64_t>(R) * 0x165667b19e3779f9ull) + (b_outer ? 1u : 0u);
  Entry& e = entries[(h ^ (h >> 32)) % kEntries];
  if (e.L != L || e.C != C || e.R != R || e.sms != sms || e.b_outer != b_outer) {
    e.plan = split_search(L, C, R, b_outer, sms);
    e.L = L;
    e.C = C;
    e.R = R;
    e.sms = sms;
    e.b_outer = b_outer;
  }
  return e.plan;
}

template <bool kAOuter, bool kBOuter, bool kF16>
cudaError_t launch_split_of(const void* A, int64_t lda, const void* B, int64_t ldb, int64_t L, int64_t C, int64_t R,
                         const Epilogue& epi, cudaStream_t stream) {
  const SplitPlan p = split_plan(L, C, R, kBOuter, device_sm_count());
  CUtensorMap ma, mb;
  const uint64_t l = L, c = C, r = R, sa = lda * 2, sb = ldb * 2;
  if (!(kAOuter ? encode_tmap_2d_bf16(&ma, A, l, r, sa, 64, kRed) : encode_tmap_2d_bf16(&ma, A, r, l, sa, kRed, kLanes)) ||
      !(kBOuter ? encode_tmap_2d_bf16(&mb, B, c, r, sb, 64, kRed) : encode_tmap_2d_bf16(&mb, B, r, c, sb, kRed, p.NT)))
    return cudaErrorInvalidValue;
  const Injection inj = take_injection(kInjectLinearSplit);
  const SplitArgs a{epi,       status_word_ptr(), static_cast<int>(L), static_cast<int>(C), p.NT,          p.tiles_l,
                    p.tiles_c, p.nkb,             p.S,                 p.stages,            inj.wait_limit, inj.stall_at};
  const size_t smem = static_cast<size_t>(p.stages) * (kABytes + p.NT * kRed * 2) + 1024;
  const auto kernel = linear_split_kernel<kAOuter, kBOuter, kF16>;
  // any plan's limit, not this one's: the limit is the kernel's, so a smaller one would fail the launch of another host
  // thread's larger plan
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostRing + 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.tiles * p.S));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.S);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, ma, mb, a);
}

template <bool kAOuter, bool kBOuter>
cudaError_t launch_split(const void* A, int64_t lda, const void* B, int64_t ldb, int64_t L, int64_t C, int64_t R,
                         const LinearEpilogue& e, cudaStream_t stream) {
  const Epilogue epi = epilogue_of(e);
  return e.f16 ? launch_split_of<kAOuter, kBOuter, true>(A, lda, B, ldb, L, C, R, epi, stream)
               : launch_split_of<kAOuter, kBOuter, false>(A, lda, B, ldb, L, C, R, epi, stream);
}

// Whether the kernel on CTA pairs takes a product: by the estimates of both, and for dw (b_outer) where a block here would
// take too many rows in one accumulator.
bool use_pairs(const PairPlan& p, int64_t L, int64_t C, int64_t R, bool b_outer, int sms) {
  if (C <= 128 && !b_outer) return false;  // half of a tile's rows and more would be empty
  const SplitPlan s = split_plan(L, C, R, b_outer, sms);
  if (b_outer && (s.nkb + s.S - 1) / s.S > kMostBlocks) return true;
  return C > 128 && p.us < s.us;
}

}  // namespace

cudaError_t launch_linear_fwd(const void* x, const void* w, const LinearEpilogue& epi, int64_t M, int64_t K, int64_t N,
                              int64_t ldx, cudaStream_t stream) {
  const int sms = device_sm_count();
  const PairPlan p = linear_pair_plan(M, N, K, false, false, sms);
  if (use_pairs(p, N, M, K, false, sms))
    return launch_linear_pair<false, true>(x, ldx, w, N, M, N, K, epi, p, nullptr, stream);
  return launch_split<true, false>(w, N, x, ldx, N, M, K, epi, stream);
}

cudaError_t launch_linear_dx(const void* dz, const void* w, const LinearEpilogue& epi, int64_t M, int64_t K, int64_t N,
                             int64_t lddz, cudaStream_t stream) {
  const int sms = device_sm_count();
  const PairPlan p = linear_pair_plan(M, K, N, true, false, sms);
  if (use_pairs(p, K, M, N, false, sms))
    return launch_linear_pair<false, false>(dz, lddz, w, N, M, K, N, epi, p, nullptr, stream);
  return launch_split<false, false>(w, N, dz, lddz, K, M, N, epi, stream);
}

size_t linear_dw_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  const int sms = device_sm_count();
  const PairPlan p = linear_pair_plan(K, N, M, true, true, sms);
  return use_pairs(p, N, K, M, true, sms) ? p.part_bytes : 0;
}

cudaError_t launch_linear_dw(const void* x, const void* dz, const LinearEpilogue& epi, int64_t M, int64_t K, int64_t N,
                             int64_t ldx, int64_t lddz, float* part, cudaStream_t stream) {
  const int sms = device_sm_count();
  const PairPlan p = linear_pair_plan(K, N, M, true, true, sms);
  if (use_pairs(p, N, K, M, true, sms))
    return launch_linear_pair<true, true>(x, ldx, dz, lddz, K, N, M, epi, p, part, stream);
  return launch_split<true, true>(dz, lddz, x, ldx, N, K, M, epi, stream);
}

}  // namespace swg
