// What the forward and the backward of the norms between blocks share: rows that come through a ring in shared
// memory, sums over a group of warps, and the sizes of groups, clusters and rings.
#pragma once

#include <algorithm>

#include "row_vectors.cuh"

namespace swg {
namespace bn {

using namespace row;

constexpr int kMaxThreads = 1024;  // of the kernels for longest rows
constexpr int kBlock = 256;        // threads of a block, unless a row takes more
constexpr int kMaxGroup = 512;     // threads of a group, and of a block

// 1 / sqrt(x): rsqrtf with a Newton step, to about an ulp, as its error is a whole row's (0 for infinity)
__device__ __forceinline__ float inverse_root(float x) {
  const float r = rsqrtf(x), e = fmaf(-x * r, r, 1.0f);
  return e == e ? fmaf(0.5f * r, e, r) : r;
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
template <int kTensors, bool kMended>  // kMended: the readers write into the stages
struct RowRing {
  uint64_t* full;
  unsigned char* buf;
  int stages, stage_bytes, at = 0;  // stage of the row that is read next
  uint32_t parity = 0;
  int64_t issued = 0;
  Patience wait;
  __device__ __forceinline__ RowRing(unsigned char* smem, uint64_t* bars, const RingPlan& p, int group, const Stall& stall)
      : full(bars + group * kMaxStages), buf(smem + group * p.group_bytes), stages(p.stages), stage_bytes(p.stage_bytes),
        wait(stall.limit) {}
  __device__ __forceinline__ void init() {
    for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
  }
  // by the group's first thread: the next row's tensors, `bytes` of each from `from` (null: none) into the stage's
  // slots of `slot` bytes
  __device__ __forceinline__ void issue(const void* const (&from)[kTensors], const uint32_t (&bytes)[kTensors], int slot,
                                        int64_t stall_at, int offset = 0) {  // offset: of the first byte in the slots
    if (wait.lost() || issued == stall_at) return;
    const int st = static_cast<int>(issued % stages);
    if (kMended) fence_proxy_async_smem();  // the group has written into the stage
    uint32_t all = 0;
#pragma unroll
    for (int i = 0; i < kTensors; ++i) all += from[i] != nullptr ? bytes[i] : 0u;
    mbar_arrive_expect_tx(&full[st], all);
#pragma unroll
    for (int i = 0; i < kTensors; ++i)
      if (from[i] != nullptr && bytes[i] > 0) bulk_g2s(buf + st * stage_bytes + i * slot + offset, from[i], bytes[i], &full[st]);
    ++issued;
  }
  // the stage of the next row, landed
  __device__ __forceinline__ unsigned char* next() {
    wait(&full[at], parity);
    unsigned char* p = buf + at * stage_bytes;
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
// Ragged rows in a ring: a row is copied as the 16-byte vectors that it touches, with elements of its neighbours, which
// the readers clear. Only the tensor's own first and last vector may reach beyond it: they are not copied where they do,
// but loaded element by element. This asks that all tensors' rows lie on the same offsets within 16 bytes.
struct Span {
  int first, count;  // of a block's vectors, those that are copied
};
// row r of M, whose n vectors begin `shift` elements before it and end `over` behind it; the block has those from n0 on
__device__ __forceinline__ Span span_of(int64_t r, int64_t M, int n, int n0, int mine, int shift, int over) {
  Span s{0, mine};
  if (r == 0 && n0 == 0 && shift > 0) {
    s.first = 1;
    --s.count;
  }
  if (r == M - 1 && n0 + mine == n && over > 0) --s.count;
  return Span{s.first, max(s.count, 0)};
}
__device__ __forceinline__ Raw ld_stage(const unsigned char* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  return Raw{{u.x, u.y, u.z, u.w}};
}
// By the thread that reads it: such a first or last vector in a stage, of row r from column j on, with zeros in place of
// the neighbours' elements, and with the row's own where it was not copied. The threads of a group wait for the one that
// does this, so it is a few operations on words.
template <typename T>
__device__ __forceinline__ void mend_edge(unsigned char* p, const Rows<T>& rows, int64_t r, int64_t M, int j, int N) {
  Raw v = ld_stage(p);
  if ((r == 0 && j < 0) || (r == M - 1 && j + kElems<T> > N)) v = load_columns<T, true>(rows, r, j, N);
  clear_others<T>(v, j, N);
  st_raw(p, v);
}
// an output's vector at column j; of a first or last one the row's elements
template <typename T, bool kRagged>
__device__ __forceinline__ void store_vector(T* row, int j, int N, bool edge, const Raw& v) {
  if (!kRagged || !edge) {
    st_raw(row + j, v);
    return;
  }
  const int lo = max(0, -j), hi = min(kElems<T>, N - j);
#pragma unroll
  for (int e = 0; e < kElems<T>; ++e) {
    if (e < lo || e >= hi) continue;
    if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t*>(row + j)[e] = v.w[e];
    else reinterpret_cast<uint16_t*>(row + j)[e] = static_cast<uint16_t>(v.w[e / 2] >> (16 * (e % 2)));
  }
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

// ---- host
// whether ragged rows can come through a ring: every tensor's rows lie on the same offsets within 16 bytes as the dense
// rows of N elements from `out` on
inline bool same_offsets(int64_t M, int64_t N, int es, const void* out, std::initializer_list<const void*> ptrs,
                         std::initializer_list<int64_t> lds) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(out) % 16;
  bool ok = N >= 16;
  for (const void* p : ptrs) ok = ok && (p == nullptr || reinterpret_cast<uintptr_t>(p) % 16 == at);
  for (int64_t ld : lds) ok = ok && (M <= 1 || (ld >= N && (ld - N) * es % 16 == 0));
  return ok;
}
// Rows shared by a cluster: S blocks of G threads, R vectors each
struct Shared {
  int S, G;
};
inline Shared share_row(int64_t n, int R) {
  const int64_t threads = (n + R - 1) / R;
  const int S = static_cast<int>(threads <= kMaxCluster * kBlock ? (threads + kBlock - 1) / kBlock : kMaxCluster);
  return Shared{S, static_cast<int>((threads + 32 * S - 1) / (32 * S)) * 32};
}

// The ring of a group: as many rows of `row` bytes as fit beside one another in the memory of `blocks` blocks an SM,
// `groups` groups each.
constexpr int64_t kRingMemory = 220 * 1024;  // of an SM's 228 KB: what is static and 1 KB a block stay free
inline RingPlan ring_plan(int64_t row, int blocks, int groups) {
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

}  // namespace bn
}  // namespace swg
