// The expert activation and its derivative on fp32 values, for the operators that stand outside the GEMM
// epilogues.  FAST: where the result is rounded to bf16 (half a step is 2^-9 relative); otherwise with
// the accurate functions of the CUDA math library.
//   GELU(u) = u Phi(u), GELU'(u) = Phi(u) + u phi(u);  SiLU(u) = u s, SiLU'(u) = s (1 + u (1 - s)), s = sigmoid(u)
#pragma once
#include "moe_internal.cuh"

namespace moe {

// The special-function unit's power of two and reciprocal, results below 2^-126 flushed to zero (2 units in the last
// place or so; without the flush each takes three more instructions).
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2E = 1.4426950408889634f;

// Phi(u) and exp(-u^2 / 2) together.  FAST: with x = |u| / sqrt 2 and t = 1 / (1 + 0.45 x),
//   erfc(x) / 2 = exp(-x^2) t (c1 + c2 t + ... + c6 t^5),
// coefficients fitted to erfc(x) exp(x^2) / 2 on [0, 20] by reweighted least squares on the relative error,
// which stays below 1e-5 over the whole range (so that small values of the far tail keep their digits).
template <bool FAST>
__device__ __forceinline__ float normal_cdf_exp(float u, float& ex) {
  if constexpr (FAST) {
    const float x = fabsf(u) * 0.70710678118654752f;
    const float t = fast_rcp(fmaf(0.45f, x, 1.f));
    float q = fmaf(t, -0.06796646f, 0.14623705f);
    q = fmaf(t, q, 0.04459168f);
    q = fmaf(t, q, 0.124316f);
    q = fmaf(t, q, 0.12583096f);
    q = fmaf(t, q, 0.12698601f);
    ex = fast_exp2(x * x * -kLog2E);
    const float half_erfc = q * t * ex;
    return u >= 0.f ? 1.f - half_erfc : half_erfc;
  } else {
    ex = expf(-0.5f * u * u);
    return 0.5f * erfcf(u * -0.70710678118654752f);
  }
}
template <bool FAST>
__device__ __forceinline__ float sigmoid(float u) {
  if constexpr (FAST) return fast_rcp(1.f + fast_exp2(u * -kLog2E));
  else return 1.f / (1.f + expf(-u));
}

// act(u); ACT is a moe_activation_t, MOE_ACT_NONE the identity
template <int ACT, bool FAST>
__device__ __forceinline__ float activate(float u) {
  if constexpr (ACT == MOE_ACT_GELU) {
    float ex;
    return u * normal_cdf_exp<FAST>(u, ex);
  } else if constexpr (ACT == MOE_ACT_SILU) {
    return u * sigmoid<FAST>(u);
  } else {
    return u;
  }
}
// act(u), and act'(u) into d
template <int ACT, bool FAST>
__device__ __forceinline__ float activate_grad(float u, float& d) {
  if constexpr (ACT == MOE_ACT_GELU) {
    float ex;
    const float phi = normal_cdf_exp<FAST>(u, ex);
    d = fmaf(u * 0.3989422804014327f, ex, phi);
    return u * phi;
  } else if constexpr (ACT == MOE_ACT_SILU) {
    const float s = sigmoid<FAST>(u);
    d = s * fmaf(u, 1.f - s, 1.f);
    return u * s;
  } else {
    d = 1.f;
    return u;
  }
}

}  // namespace moe
