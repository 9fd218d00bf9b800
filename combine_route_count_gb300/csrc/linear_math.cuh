// Arithmetic that the bf16 products' kernels share: activations, their
// derivatives, bf16 pairs.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "moe_train.h"
#include "tcgen05.cuh"

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
// From s = sigmoid(v).
__device__ __forceinline__ float silu_slope(float v, float s) { return s * fmaf(v, 1.0f - s, 1.0f); }
__device__ __forceinline__ float relu(float v) { return v > 0.0f || v != v ? v : 0.0f; }

// The normal distribution function P(v) = (1 + erf(v / sqrt 2)) / 2, and exp(-v^2 / 2),
// which it needs: erf by formula 7.1.26 of Abramowitz and Stegun, Handbook of
// Mathematical Functions (absolute error 1.5e-7), from v's side of zero, so that 1 - P
// and P keep their digits where they are small.  (The library's erff and expf together
// took three times the instructions, and a gradient through GELU of 40 experts' 3003
// rows, N 1416, K 2320, 76 us instead of 64.)
constexpr float kErfP = 0.3275911f * 0.70710678118654752f;
constexpr float kErf0 = 0.5f * 0.254829592f, kErf1 = 0.5f * -0.284496736f, kErf2 = 0.5f * 1.421413741f,
                kErf3 = 0.5f * -1.453152027f, kErf4 = 0.5f * 1.061405429f;
constexpr float kHalfLog2e = 0.72134752044448170f, kInvSqrt2Pi = 0.39894228040143268f;
__device__ __forceinline__ float normal(float v, float& e) {
  e = exp2_fast(v * v * -kHalfLog2e);
  const float t = reciprocal(fmaf(kErfP, fabsf(v), 1.0f));
  float q = fmaf(t, kErf4, kErf3);
  q = fmaf(t, q, kErf2);
  q = fmaf(t, q, kErf1);
  q = fmaf(t, q, kErf0);
  q *= t * e;
  return v < 0.0f ? q : 1.0f - q;
}
__device__ __forceinline__ float gelu(float v) {
  float e;
  return v * normal(v, e);
}
__device__ __forceinline__ float gelu_slope(float v) {
  float e;
  const float p = normal(v, e);
  return fmaf(v * kInvSqrt2Pi, e, p);
}

// ---- the same for two values, with the instructions that do two at a time ----------
// An activation over a tile is bound by instructions: eight warps, 32768 values.
struct Two {
  unsigned long long v;
  __device__ __forceinline__ Two(float a, float b) : v(tc::pack2(a, b)) {}
  __device__ __forceinline__ explicit Two(unsigned long long both) : v(both) {}
  __device__ __forceinline__ float lo() const { return tc::lo2(v); }
  __device__ __forceinline__ float hi() const { return tc::hi2(v); }
};
__device__ __forceinline__ Two operator*(Two a, Two b) { return Two(tc::mul2(a.v, b.v)); }
__device__ __forceinline__ Two operator*(Two a, float b) { return a * Two(b, b); }
__device__ __forceinline__ Two fma(Two a, Two b, Two c) { return Two(tc::fma2(a.v, b.v, c.v)); }
__device__ __forceinline__ Two fma(Two a, Two b, float c) { return fma(a, b, Two(c, c)); }

__device__ __forceinline__ Two sigmoid(Two v) {
  const Two a = v * -1.4426950408889634f;
  return Two(reciprocal(1.0f + exp2_fast(a.lo())), reciprocal(1.0f + exp2_fast(a.hi())));
}
// From s = sigmoid(v).
__device__ __forceinline__ Two silu_slope(Two v, Two s) { return s * fma(v, fma(s, Two(-1.0f, -1.0f), 1.0f), 1.0f); }
__device__ __forceinline__ Two normal(Two v, Two& e) {
  const Two a = v * v * -kHalfLog2e;
  e = Two(exp2_fast(a.lo()), exp2_fast(a.hi()));
  const Two t(reciprocal(fmaf(kErfP, fabsf(v.lo()), 1.0f)), reciprocal(fmaf(kErfP, fabsf(v.hi()), 1.0f)));
  Two q = fma(t, Two(kErf4, kErf4), kErf3);
  q = fma(t, q, kErf2);
  q = fma(t, q, kErf1);
  q = fma(t, q, kErf0);
  q = q * (t * e);
  return Two(v.lo() < 0.0f ? q.lo() : 1.0f - q.lo(), v.hi() < 0.0f ? q.hi() : 1.0f - q.hi());
}
__device__ __forceinline__ Two gelu_slope(Two v) {
  Two e(0.0f, 0.0f);
  const Two p = normal(v, e);
  return fma(v * kInvSqrt2Pi, e, p);
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
  if (act == MOE_ACT_SILU) return g * silu_slope(v, sigmoid(v));
  return g;
}
__device__ __forceinline__ Two act_value(int act, Two v) {
  if (act == MOE_ACT_RELU) return Two(relu(v.lo()), relu(v.hi()));
  if (act == MOE_ACT_GELU) {
    Two e(0.0f, 0.0f);
    return v * normal(v, e);
  }
  if (act == MOE_ACT_SILU) return v * sigmoid(v);
  return v;
}
__device__ __forceinline__ Two act_through(int act, Two g, Two v) {
  if (act == MOE_ACT_RELU) return Two(v.lo() > 0.0f ? g.lo() : 0.0f, v.hi() > 0.0f ? g.hi() : 0.0f);
  if (act == MOE_ACT_GELU) return g * gelu_slope(v);
  if (act == MOE_ACT_SILU) return g * silu_slope(v, sigmoid(v));
  return g;
}
// The derivatives of SiLU(gate) * up, times g, in the place of gate and up.
__device__ __forceinline__ void swiglu_through(Two g, Two& gate, Two& up) {
  const Two s = sigmoid(gate), d_up = g * (gate * s);
  gate = g * up * silu_slope(gate, s);
  up = d_up;
}

}  // namespace lin
}  // namespace moe
