// Activations and their derivatives in fp32, shared by the gated SiLU and the linear layer's epilogue.
#pragma once

#include "tdx_rows.cuh"

namespace tdx {

// 2^x and 1/x by the special-function unit (2 and 1 ulp), subnormal results 0
__device__ __forceinline__ float power_of_2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// a * sigmoid(a) of two values; sigmoid(a) and 1 - sigmoid(a). For fp32 results (kExact) with expf and the IEEE
// quotient, which costs nothing there (65536 x 2048 fp32 224 us either way). For the others exp(-a) = 2^(-a log2 e)
// and the reciprocal are approximate: within 2^-22 * (4 + |a|) relative, |a| < 89, which a rounding to 8 bits hides;
// with the exact forms that kernel is bound by issue slots (262144 x 2048 bf16, one vector per thread: 669 us). The
// divisor is taken times 1/16, so that its reciprocal is no subnormal where exp(-a) is below fp32's largest.
// exp(-a) = inf gives -0 and 0, as the exact quotient does.
constexpr float kLog2e = 1.44269504f, kPart = 0.0625f;
template <bool kExact>
__device__ __forceinline__ f32x2 silu(f32x2 a) {
  if (kExact) return pair(first(a) / (1.0f + expf(-first(a))), second(a) / (1.0f + expf(-second(a))));
  const f32x2 z = mul2(a, pair(-kLog2e, -kLog2e)), part = pair(kPart, kPart);
  const f32x2 d = fma2(pair(power_of_2(first(z)), power_of_2(second(z))), part, part);
  return mul2(mul2(a, part), pair(reciprocal(first(d)), reciprocal(second(d))));
}
template <bool kExact>
__device__ __forceinline__ float sigmoid(float a, float* rest) {
  if (kExact) {
    const float e = expf(-a), s = 1.0f / (1.0f + e);
    *rest = e < INFINITY ? e * s : 1.0f;   // 1 - s without the difference's cancellation
    return s;
  }
  const float s = kPart * reciprocal(fmaf(power_of_2(-kLog2e * a), kPart, kPart));
  *rest = 1.0f - s;
  return s;
}

// a * sigmoid(b) of one value, as silu above
template <bool kExact>
__device__ __forceinline__ float times_sigmoid(float a, float b) {
  if (kExact) return a / (1.0f + expf(-b));
  return a * kPart * reciprocal(fmaf(power_of_2(-kLog2e * b), kPart, kPart));
}

// GELU with tanh: 0.5 a (1 + tanh(w / 2)) = a * sigmoid(w), w = 2 sqrt(2 / pi) (a + 0.044715 a^3): the sum with
// tanh would cancel for a < 0
constexpr float kGelu2 = 1.59576912f, kGeluCube = 0.044715f, kHalfRoot = 0.70710678f, kInvRoot2Pi = 0.39894228f;
__device__ __forceinline__ float gelu_arg(float a) { return kGelu2 * a * fmaf(kGeluCube * a, a, 1.0f); }

// One value, exact forms and GELU with the error function: called, not unrolled. (The epilogues run these once per
// column; unrolled for every activation they filled the instruction cache.)
static __device__ __noinline__ float act_exact(tdx_activation act, float v) {
  if (act == TDX_ACT_GELU) return 0.5f * v * erfcf(-kHalfRoot * v);
  return times_sigmoid<true>(v, act == TDX_ACT_GELU_TANH ? gelu_arg(v) : v);
}

// One activation over N values (the gate's alone for TDX_ACT_SWIGLU). Exact forms for fp32 results; the
// approximate ones err by 2^-22 * (4 + |exponent|) relative, which a rounding to 8 bits hides.
template <int N>
__device__ __forceinline__ void act_forward(tdx_activation act, bool exact, float (&v)[N]) {
  if (act == TDX_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];   // a NaN stays one
  } else if (exact || act == TDX_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = act_exact(act, v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = times_sigmoid<false>(v[i], act == TDX_ACT_GELU_TANH ? gelu_arg(v[i]) : v[i]);
  }
}

// The approximate forms of two values: RELU, GELU_TANH and SILU (the gate of SWIGLU)
__device__ __forceinline__ f32x2 act_pair(tdx_activation act, f32x2 v) {
  if (act == TDX_ACT_RELU) return pair(first(v) < 0.0f ? 0.0f : first(v), second(v) < 0.0f ? 0.0f : second(v));
  f32x2 z = pair(-kLog2e, -kLog2e);
  if (act == TDX_ACT_GELU_TANH)
    z = fma2(mul2(v, v), pair(-kLog2e * kGelu2 * kGeluCube, -kLog2e * kGelu2 * kGeluCube), pair(-kLog2e * kGelu2, -kLog2e * kGelu2));
  z = mul2(z, v);
  const f32x2 part = pair(kPart, kPart);
  const f32x2 d = fma2(pair(power_of_2(first(z)), power_of_2(second(z))), part, part);
  return mul2(mul2(v, part), pair(reciprocal(first(d)), reciprocal(second(d))));
}

}  // namespace tdx
