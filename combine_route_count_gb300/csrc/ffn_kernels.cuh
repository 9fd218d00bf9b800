// Internal interface between the C ABI of the feed-forward operators
// (ffn_abi.cu) and their kernels.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "moe_ffn.h"
#include "moe_kernels.cuh"

namespace moe {

// A block whose largest magnitude is smaller counts as this large when its
// scale is taken, so that 1 / scale stays finite.
constexpr float kTinyAmax = 0x1p-100f;

// ---- add_rms_norm_fp8: residual addition, RMS norm, quantisation -----------
struct AddNormParams {
  const uint8_t* x;         // bf16 [T, H]
  const uint8_t* residual;  // bf16 [T, H] or null
  const uint8_t* weight;    // bf16 or float32 [H]
  uint8_t* residual_out;    // bf16 [T, H], null with residual
  uint8_t* y;               // bf16 [T, H] or null
  uint8_t* xq;              // E4M3 [T, H]
  float* x_scales;          // [T, H/128]
  int64_t T;
  int32_t H;
  float eps;
};
cudaError_t launch_add_norm_fp8(const AddNormParams& p, bool weight_f32, int sms, cudaStream_t stream);

}  // namespace moe
