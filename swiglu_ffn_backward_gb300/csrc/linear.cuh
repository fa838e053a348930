// What the kernels of the linear layer share: its activations and their gradients in fp32, the narrowing
// to its two element types, and the arguments of an epilogue.
#pragma once

#include "row_ops.cuh"
#include "swg_device.cuh"
#include "swg_launch.h"

namespace swg {
namespace lin {

// Phi(x) and e^{-x^2/2}. For the smaller tail, Phi(-|x|) = e^{-x^2/2} t Q(t) with t = 1 / (1 + |x| / (2 sqrt 2)):
// Q is a polynomial of degree 6 fitted to erfcx(|x| / sqrt 2) / (2 t) for the least relative error (1.2e-6 up to
// |x| = 13.5, where e^{-x^2/2} leaves fp32), so that x Phi(x) keeps its relative accuracy in the negative tail,
// where 1 + erf would cancel.
struct Gauss {
  float cdf, e;
};
__device__ __forceinline__ Gauss gauss(float x) {
  Gauss g;
  g.e = ex2_approx(-(x * x) * (0.5f * kLog2e));
  const float t = rcp_approx(fmaf(fabsf(x), 0.35355339059327373f, 1.0f));
  float q = 0.04446815699338913f;
  q = fmaf(q, t, -0.179658904671669f);
  q = fmaf(q, t, 0.19641998410224915f);
  q = fmaf(q, t, 0.017663639038801193f);
  q = fmaf(q, t, 0.14123354852199554f);
  q = fmaf(q, t, 0.1387006789445877f);
  q = fmaf(q, t, 0.14117228984832764f);
  const float tail = q * t * g.e;
  g.cdf = x >= 0.0f ? 1.0f - tail : tail;
  return g;
}

// f(z) of an activation (swg_act); kActNone: z itself
constexpr int kActNone = kLinearNoAct;
__device__ __forceinline__ float2 activate(float2 z, int act) {
  if (act == 0) return __fmul2_rn(z, sigmoid_pair2(z).s);
  if (act == 1) return make_float2(z.x * gauss(z.x).cdf, z.y * gauss(z.y).cdf);
  if (act == 2) {
    auto f = [](float v) { return v <= -3.0f ? 0.0f : (v < 3.0f ? v * fmaf(v, 1.0f / 6.0f, 0.5f) : v); };
    return make_float2(f(z.x), f(z.y));
  }
  return z;
}
// f'(z)
__device__ __forceinline__ float2 activate_grad(float2 z, int act) {
  if (act == 0) {
    const Sig2 q = sigmoid_pair2(z);
    return __fmul2_rn(q.s, __ffma2_rn(z, q.sc, make_float2(1.0f, 1.0f)));
  }
  if (act == 1) {
    const Gauss a = gauss(z.x), b = gauss(z.y);
    return make_float2(fmaf(z.x, 0.39894228040143268f * a.e, a.cdf), fmaf(z.y, 0.39894228040143268f * b.e, b.cdf));
  }
  if (act == 2) {
    auto f = [](float v) { return v <= -3.0f ? 0.0f : (v < 3.0f ? fmaf(v, 1.0f / 3.0f, 0.5f) : 1.0f); };
    return make_float2(f(z.x), f(z.y));
  }
  return make_float2(1.0f, 1.0f);
}

// two elements of a packed word of fp16 (f16) or bf16, widened; two fp32 rounded to one
__device__ __forceinline__ float2 widen2(uint32_t u, bool f16) {
  if (f16) return __half22float2(*reinterpret_cast<const __half2*>(&u));
  return bf16x2_to_f2(u);
}
__device__ __forceinline__ uint32_t narrow2(float2 v, bool f16) {
  if (f16) {
    const __half2 h = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  return pack_bf16x2(v.x, v.y);
}
// eight elements
__device__ __forceinline__ void widen8(const uint4& u, bool f16, float2 (&v)[4]) {
  v[0] = widen2(u.x, f16);
  v[1] = widen2(u.y, f16);
  v[2] = widen2(u.z, f16);
  v[3] = widen2(u.w, f16);
}
__device__ __forceinline__ uint4 narrow8(const float2 (&v)[4], bool f16) {
  return make_uint4(narrow2(v[0], f16), narrow2(v[1], f16), narrow2(v[2], f16), narrow2(v[3], f16));
}

// What happens to a product's elements before they are stored: z = sum + bias, y = f(z) + residual.
struct Epilogue {
  const void* bias;          // [columns] of the element type or fp32, or null
  const uint16_t* residual;  // rows ldr apart, or null; may be y itself
  uint16_t* y;               // rows of `columns` elements
  uint16_t* z;               // the same, or null
  int64_t ldr;
  int act;
  bool f16, bias_f32;
};
__device__ __forceinline__ void add_bias(const Epilogue& p, int64_t n, float2 (&v)[4]) {
  if (p.bias == nullptr) return;
  if (p.bias_f32) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.bias) + n));
    const float4 b = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.bias) + n + 4));
    v[0] = __fadd2_rn(v[0], make_float2(a.x, a.y));
    v[1] = __fadd2_rn(v[1], make_float2(a.z, a.w));
    v[2] = __fadd2_rn(v[2], make_float2(b.x, b.y));
    v[3] = __fadd2_rn(v[3], make_float2(b.z, b.w));
  } else {
    float2 b[4];
    widen8(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.bias) + n)), p.f16, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __fadd2_rn(v[i], b[i]);
  }
}

// instruction descriptor of kind::f16 with both operands fp16 (f16) or bf16 and fp32 sums
__host__ __device__ constexpr uint32_t idesc_f32(int m, int n, bool a_mn, bool b_mn, bool f16) {
  return f16 ? idesc_bf16_f32(m, n, a_mn, b_mn) & ~((1u << 7) | (1u << 10)) : idesc_bf16_f32(m, n, a_mn, b_mn);
}

}  // namespace lin
}  // namespace swg
