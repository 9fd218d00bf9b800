// Arithmetic that the bf16 products' kernels share: activations, their
// derivatives, bf16 pairs.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "moe_train.h"

namespace moe {
namespace lin {

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 2^v within 2^-22 of itself, and 1 / v within 2^-23; results below 2^-126 are 0.
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// The product with log2(e) is off by 2^-24 of itself, exp(-v) by 2^-23.5 |v| of
// itself, and the sigmoid by s (1 - s) of that: 2^-22 in all.
__device__ __forceinline__ float sigmoid(float v) {
  return reciprocal(1.0f + exp2_fast(v * -1.4426950408889634f));
}
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }
__device__ __forceinline__ float silu_slope(float v) {
  const float s = sigmoid(v);
  return s * fmaf(v, 1.0f - s, 1.0f);
}
__device__ __forceinline__ float relu(float v) { return v > 0.0f || v != v ? v : 0.0f; }

// The normal distribution function P(v) = (1 + erf(v / sqrt 2)) / 2, and exp(-v^2 / 2),
// which it needs: erf by formula 7.1.26 of Abramowitz and Stegun, Handbook of
// Mathematical Functions (absolute error 1.5e-7), from v's side of zero, so that 1 - P
// and P keep their digits where they are small.  (The library's erff and expf together
// took three times the instructions, and a gradient through GELU of 40 experts' 3003
// rows, N 1416, K 2320, 76 us instead of 64.)
__device__ __forceinline__ float normal(float v, float& e) {
  const float x = fabsf(v);
  e = exp2_fast(v * v * -0.72134752044448170f);
  const float t = reciprocal(fmaf(0.3275911f * 0.70710678118654752f, x, 1.0f));
  float q = fmaf(t, 1.061405429f, -1.453152027f);
  q = fmaf(t, q, 1.421413741f);
  q = fmaf(t, q, -0.284496736f);
  q = fmaf(t, q, 0.254829592f);
  q *= 0.5f * t * e;
  return v < 0.0f ? q : 1.0f - q;
}
__device__ __forceinline__ float gelu(float v) {
  float e;
  return v * normal(v, e);
}
__device__ __forceinline__ float gelu_slope(float v) {
  float e;
  const float p = normal(v, e);
  return fmaf(v * 0.39894228040143268f, e, p);
}

// One value of MOE_ACT_* but MOE_ACT_SWIGLU.
__device__ __forceinline__ float act_value(int act, float v) {
  if (act == MOE_ACT_RELU) return relu(v);
  if (act == MOE_ACT_GELU) return gelu(v);
  if (act == MOE_ACT_SILU) return silu(v);
  return v;
}
// g times its derivative at v.
__device__ __forceinline__ float act_through(int act, float g, float v) {
  if (act == MOE_ACT_RELU) return v > 0.0f ? g : 0.0f;
  if (act == MOE_ACT_GELU) return g * gelu_slope(v);
  if (act == MOE_ACT_SILU) return g * silu_slope(v);
  return g;
}
// The derivatives of SiLU(gate) * up, times g, in the place of gate and up.
__device__ __forceinline__ void swiglu_through(float g, float& gate, float& up) {
  const float sig = sigmoid(gate);
  const float d_up = g * (gate * sig);
  gate = g * up * (sig * fmaf(gate, 1.0f - sig, 1.0f));
  up = d_up;
}

}  // namespace lin
}  // namespace moe
