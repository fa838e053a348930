// Device helpers shared by the row-wise operators (layer norm, token log probabilities,
// distillation): element conversions, block reductions, and the order of a row's best logits.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "swg_device.cuh"

namespace swg {
namespace row {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// an element of a tensor whose type is known at run time (SWG_F32, SWG_F16, SWG_BF16)
__device__ __forceinline__ float load_any(const void* p, int64_t i, int dtype) {
  if (dtype == 0) return static_cast<const float*>(p)[i];
  if (dtype == 1) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void store_any(void* p, int64_t i, int dtype, float v) {
  if (dtype == 0) static_cast<float*>(p)[i] = v;
  else if (dtype == 1) static_cast<__half*>(p)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}
// an index of a tensor of 32- or 64-bit integers
__device__ __forceinline__ int64_t load_index(const void* p, int64_t i, bool wide) {
  return wide ? static_cast<const int64_t*>(p)[i] : static_cast<int64_t>(static_cast<const int32_t*>(p)[i]);
}

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {  // one instruction, in place of five shuffles in turn
  asm volatile("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(v));
  return v;
}

// The block's sum: every thread gets it, added in a fixed order. `buf` holds one value a warp; the barriers
// around it let a caller use it again at once.
__device__ __forceinline__ float block_sum(float v, float* buf) {
  const int warps = static_cast<int>(blockDim.x + 31) >> 5;
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = buf[0];
  for (int w = 1; w < warps; ++w) r += buf[w];
  __syncthreads();
  return r;
}

// The order of a row's alternatives: larger logits first, equal ones by the lower index; a NaN counts
// as -inf and -0 as +0. One unsigned 64-bit key for each (logit, index): the better one is larger, and
// no two of a row are equal. Key 0 is below every element's.
__device__ __forceinline__ uint64_t rank_key(float z, uint32_t index) {
  z = (z == z ? z : neg_inf()) + 0.0f;
  const uint32_t u = __float_as_uint(z);
  const uint32_t ord = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return (static_cast<uint64_t>(ord) << 32) | (0xffffffffu - index);
}
__device__ __forceinline__ uint32_t rank_index(uint64_t key) { return 0xffffffffu - static_cast<uint32_t>(key); }
__device__ __forceinline__ float rank_logit(uint64_t key) {
  const uint32_t ord = static_cast<uint32_t>(key >> 32);
  return __uint_as_float((ord & 0x80000000u) ? (ord & 0x7fffffffu) : ~ord);
}

}  // namespace row
}  // namespace swg
