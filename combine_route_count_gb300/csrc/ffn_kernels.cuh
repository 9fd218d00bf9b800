// Internal interface between the C ABI of the feed-forward operators
// (ffn_abi.cu) and their kernels.
#pragma once

#include <cuda.h>
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

// ---- expert_gemm: grouped block-scaled E4M3 products ------------------------
struct ExpertGemmParams {
  CUtensorMap a;            // E4M3 [rows, K], boxes of 128 x 128
  CUtensorMap w;            // E4M3 [E * w_rows, K], boxes of 128 x 128
  const float* a_scales;    // [rows, kblocks]
  const float* w_scales;    // [E, w_blocks, kblocks]
  const int32_t* offsets;   // [E+1] first row of each expert, or null: all rows are expert 0's
  void* out;                // bf16 or float32 [rows, N]; glu: E4M3 [rows, N]
  float* h_scales;          // glu: [rows, N/128]
  int32_t* status;          // may be null
  int64_t rows;
  int32_t kblocks, N, n_tiles, E;
  int32_t w_rows;           // weight rows of one expert: N, glu: 2N (gate rows, then up rows)
  int32_t w_blocks;         // ceil(w_rows / 128)
};
// Columns of out that one tile covers.
int expert_gemm_n_tile(bool glu);
cudaError_t launch_expert_gemm(const ExpertGemmParams& p, bool glu, bool f32, int sms, cudaStream_t stream);

}  // namespace moe
