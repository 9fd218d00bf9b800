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

// Quotients by a denominator beyond 2^126 become 0; they are below 2^-119 of the numerator there.
__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.0f, 1.0f + expf(-v)); }
__device__ __forceinline__ float silu(float v) { return __fdividef(v, 1.0f + expf(-v)); }
__device__ __forceinline__ float silu_slope(float v) {
  const float s = sigmoid(v);
  return s * fmaf(v, 1.0f - s, 1.0f);
}
__device__ __forceinline__ float relu(float v) { return v > 0.0f || v != v ? v : 0.0f; }
// erf at v / sqrt 2.  For v far below zero 1 + erf loses its digits: the value is off
// by 2^-24 of |v|, not of itself.
__device__ __forceinline__ float gelu(float v) { return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f)); }
__device__ __forceinline__ float gelu_slope(float v) {
  const float density = 0.39894228040143268f * expf(-0.5f * v * v);
  return fmaf(v, density, 0.5f * (1.0f + erff(v * 0.70710678118654752f)));
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
