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

// A load that stays where it is written, behind the grid's dependency wait: for
// data that the kernel before this one may have written.
__device__ __forceinline__ float ld_f32(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}

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
  CUtensorMap w;            // E4M3 [E * w_rows, K], boxes of 128 x 128, glu: 64 rows
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
  uint32_t test_drop;       // the number of a load that each CTA leaves out; UINT32_MAX: none
};
// Columns of out that one tile covers.
int expert_gemm_n_tile(bool glu);
cudaError_t launch_expert_gemm(const ExpertGemmParams& p, bool glu, bool f32, int sms, cudaStream_t stream);

// ---- decode_layer: products of few rows with many weights ----------------------
constexpr int kFewTokens = MOE_DECODE_MAX_TOKENS;  // of launch_decode_layer
constexpr int kFewDenseRows = 32;                // of launch_few_rows
constexpr int kFewChunk = 16;
struct DecodeParams {
  CUtensorMap w13_map;      // E4M3 [E * 2I, H], boxes of 128 rows (all boxes 128 wide)
  CUtensorMap x_map;        // E4M3 [T, H], boxes of one row (gathered) or of kFewChunk rows
  CUtensorMap w2_map;       // E4M3 [E * H, I], boxes of 128 rows
  CUtensorMap h_map;        // E4M3 [T*K, I], boxes of kFewChunk rows
  const float* x_scales;    // [T, H/128]
  const int32_t* topk_idx;  // [T, K]
  const float* topk_w;      // [T, K]
  const int32_t* offsets;   // launch_row_groups: [E+1] first row of each expert, or null (E = 1)
  const float* w13_scales;  // [E, 2I/128, H/128]
  const float* w2_scales;   // [E, out_blocks, h_blocks]
  uint8_t* hq;              // workspace: E4M3 [T*K, I], rows ordered by (expert, token)
  float* h_scales;          // workspace: [T*K, h_blocks]
  void* out;                // [T, H], bf16 or float32
  int32_t* status;          // may be null but in launch_decode_layer
  int32_t T, H, K, E, I;
  int32_t h_blocks, out_blocks;  // ceil(I/128), ceil(H/128)
  bool out_f32;
  uint32_t test_drop;       // as in ExpertGemmParams
};
cudaError_t launch_decode_layer(const DecodeParams& p, int sms, cudaStream_t stream);
// One dense product of T <= kFewDenseRows rows: out [T, H] = h [T, I] . w2 [H, I]^T,
// from w2_map, h_map and the scales (K = E = 1).
cudaError_t launch_few_rows(const DecodeParams& p, int sms, cudaStream_t stream);
// Products of T rows, grouped by E experts (K = 1): out [T, I] =
// x [T, H] . w13 [e, I, H]^T, or (glu) hq, h_scales from w13 [e, 2I, H]; x_map
// with boxes of kFewChunk rows.
cudaError_t launch_row_groups(const DecodeParams& p, bool glu, int sms, cudaStream_t stream);

}  // namespace moe
