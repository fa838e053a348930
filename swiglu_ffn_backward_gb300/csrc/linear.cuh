// What the kernels of the linear layer share: its activations and their gradients in fp32, the narrowing
// to its two element types, and the arguments of an epilogue.
#pragma once

#include "row_ops.cuh"
#include "swg_device.cuh"
#include "swg_launch.h"

namespace swg {
namespace lin {

// Phi(x) and e^{-x^2/2} of two elements. For the smaller tail, Phi(-|x|) = e^{-x^2/2} t Q(t) with t = 1 / (1 + |x| / (2
// sqrt 2)): Q is a polynomial of degree 6 fitted to erfcx(|x| / sqrt 2) / (2 t) for the least relative error (1.2e-6 up to
// |x| = 13.5, where e^{-x^2/2} leaves fp32), so that x Phi(x) keeps its relative accuracy in the negative tail, where
// 1 + erf would cancel.
struct Gauss2 {
  float2 cdf, e, tail;
};
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ Gauss2 gauss2(float2 x) {
  Gauss2 g;
  const float2 a = __fmul2_rn(__fmul2_rn(x, x), both(-0.5f * kLog2e));
  g.e = make_float2(ex2_approx(a.x), ex2_approx(a.y));
  const float2 d = __ffma2_rn(make_float2(fabsf(x.x), fabsf(x.y)), both(0.35355339059327373f), both(1.0f));
  const float2 t = make_float2(rcp_approx(d.x), rcp_approx(d.y));
  float2 q = __ffma2_rn(both(0.04446815699338913f), t, both(-0.179658904671669f));
  q = __ffma2_rn(q, t, both(0.19641998410224915f));
  q = __ffma2_rn(q, t, both(0.017663639038801193f));
  q = __ffma2_rn(q, t, both(0.14123354852199554f));
  q = __ffma2_rn(q, t, both(0.1387006789445877f));
  q = __ffma2_rn(q, t, both(0.14117228984832764f));
  g.tail = __fmul2_rn(__fmul2_rn(q, t), g.e);
  g.cdf = make_float2(x.x >= 0.0f ? 1.0f - g.tail.x : g.tail.x, x.y >= 0.0f ? 1.0f - g.tail.y : g.tail.y);
  return g;
}

// f(z) of an activation (swg_act); kActNone: z itself
constexpr int kActNone = kLinearNoAct;
template <int kAct>
__device__ __forceinline__ float2 activate(float2 z) {
  if constexpr (kAct == 0) return __fmul2_rn(z, sigmoid_pair2(z).s);
  if constexpr (kAct == 1) {  // z Phi(z) = max(z, 0) - |z| Phi(-|z|); |z| held finite, as Phi(-inf) is 0
    const float2 m = make_float2(fmaxf(z.x, 0.0f), fmaxf(z.y, 0.0f));
    const float2 n = make_float2(-fminf(fabsf(z.x), 3e38f), -fminf(fabsf(z.y), 3e38f));
    return __ffma2_rn(n, gauss2(z).tail, m);
  }
  if constexpr (kAct == 2) {
    auto f = [](float v) { return v <= -3.0f ? 0.0f : (v < 3.0f ? v * fmaf(v, 1.0f / 6.0f, 0.5f) : v); };
    return make_float2(f(z.x), f(z.y));
  }
  return z;
}
// f'(z)
template <int kAct>
__device__ __forceinline__ float2 activate_grad(float2 z) {
  if constexpr (kAct == 0) {
    const Sig2 q = sigmoid_pair2(z);
    return __fmul2_rn(q.s, __ffma2_rn(z, q.sc, both(1.0f)));
  }
  if constexpr (kAct == 1) {
    const Gauss2 g = gauss2(z);
    return __ffma2_rn(z, __fmul2_rn(both(0.39894228040143268f), g.e), g.cdf);
  }
  if constexpr (kAct == 2) {
    auto f = [](float v) { return v <= -3.0f ? 0.0f : (v < 3.0f ? fmaf(v, 1.0f / 3.0f, 0.5f) : 1.0f); };
    return make_float2(f(z.x), f(z.y));
  }
  return both(1.0f);
}
// f(the activation as a constant): one copy of the code for each, outside the loops over elements
template <int kAct>
struct ActIs {
  static constexpr int value = kAct;
};
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
  if (act == kActNone) f(ActIs<kActNone>());
  else if (act == 0) f(ActIs<0>());
  else if (act == 1) f(ActIs<1>());
  else f(ActIs<2>());
}

// two elements of a packed word of fp16 (kF16) or bf16, widened; two fp32 rounded to one
template <bool kF16>
__device__ __forceinline__ float2 widen2(uint32_t u) {
  if constexpr (kF16) return __half22float2(*reinterpret_cast<const __half2*>(&u));
  return bf16x2_to_f2(u);
}
template <bool kF16>
__device__ __forceinline__ uint32_t narrow2(float2 v) {
  if constexpr (kF16) {
    const __half2 h = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  return pack_bf16x2(v.x, v.y);
}
// eight elements
template <bool kF16>
__device__ __forceinline__ void widen8(const uint4& u, float2 (&v)[4]) {
  v[0] = widen2<kF16>(u.x);
  v[1] = widen2<kF16>(u.y);
  v[2] = widen2<kF16>(u.z);
  v[3] = widen2<kF16>(u.w);
}
template <bool kF16>
__device__ __forceinline__ uint4 narrow8(const float2 (&v)[4]) {
  return make_uint4(narrow2<kF16>(v[0]), narrow2<kF16>(v[1]), narrow2<kF16>(v[2]), narrow2<kF16>(v[3]));
}

// What happens to a product's elements before they are stored: z = sum + bias, y = f(z) + residual.
struct Epilogue {
  const void* bias;          // [columns] of the element type or fp32, or null
  const uint16_t* residual;  // rows ldr apart, or null; may be y itself
  uint16_t* y;               // rows of `columns` elements
  uint16_t* z;               // the same, or null
  int64_t ldr;
  int act;
  bool bias_f32;
};
inline Epilogue epilogue_of(const LinearEpilogue& e) {
  return Epilogue{e.bias, static_cast<const uint16_t*>(e.residual), static_cast<uint16_t*>(e.y),
                  static_cast<uint16_t*>(e.z), e.ldr, e.act, e.bias_f32};
}
// the bias of eight columns from n on, added; 0 beyond `columns`
template <bool kF16>
__device__ __forceinline__ void add_bias(const Epilogue& p, int64_t n, int64_t columns, float2 (&v)[4]) {
  if (p.bias == nullptr || n >= columns) return;
  if (p.bias_f32) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.bias) + n));
    const float4 b = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.bias) + n + 4));
    v[0] = __fadd2_rn(v[0], make_float2(a.x, a.y));
    v[1] = __fadd2_rn(v[1], make_float2(a.z, a.w));
    v[2] = __fadd2_rn(v[2], make_float2(b.x, b.y));
    v[3] = __fadd2_rn(v[3], make_float2(b.z, b.w));
  } else {
    float2 b[4];
    widen8<kF16>(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.bias) + n)), b);
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
