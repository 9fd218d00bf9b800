// Internal interface between the C ABI of the training operators (train_abi.cu)
// and their kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "moe_kernels.cuh"
#include "moe_train.h"

namespace moe {

// ---- router: choice, weights and their gradient ------------------------------
struct RouterParams {
  const void* logits;        // bf16 or float32 [T, E]
  const float* bias;         // [E] or null
  int32_t* idx;              // [T, K], written forward, read backward
  float* w;                  // [T, K], forward
  const float* dw;           // [T, K], backward
  void* d_logits;            // [T, E], backward
  int64_t T;
  int32_t E, K;
  float scale;
  bool f32;                  // the logits' type
};
cudaError_t launch_router(const RouterParams& p, bool sigmoid, bool normalize, bool backward, cudaStream_t stream);

// ---- gradients of combine and dispatch ----------------------------------------
struct CombineGradParams {
  const uint8_t* d_out;      // bf16 [T, H]
  const uint8_t* y;          // bf16 [rows, H] or null
  const float* w;            // [T, K]
  const int32_t* slot_row;   // [T, K]
  uint8_t* dy;               // bf16 [rows, H]; may be y
  float* dw;                 // [T, K], null with y
  int64_t T, rows;
  int32_t H, K;
};
cudaError_t launch_combine_grad(const CombineGradParams& p, cudaStream_t stream);

struct DispatchGradParams {
  const uint8_t* de;         // bf16 [rows, H]
  const int32_t* slot_row;   // [T, K]
  const uint8_t* add;        // bf16 [T, H] or null
  uint8_t* dx;               // bf16 [T, H]; may be add
  int64_t T, rows;
  int32_t H, K;
};
cudaError_t launch_dispatch_grad(const DispatchGradParams& p, cudaStream_t stream);

// ---- expert_linear: grouped bf16 products and their gradients --------------------
struct LinearParams {
  CUtensorMap a;             // forward, input: [rows, kc] in boxes of 64 x 128 rows; weight: dy [rows, M], 64 x 64
  CUtensorMap b;             // forward: w [E, w_rows, kc], 64 x 128; input: w [E, kc, N], 64 x 64; weight: a [rows, N], 64 x 64
  const int32_t* offsets;    // [E+1] first row of each expert, or null: all rows are expert 0's
  const void* bias;          // forward: bf16 or float32 [E, bias_cols], or null
  void* residual;            // forward: bf16 [rows, N] or null
  void* pre;                 // forward: bf16 [rows, N], glu [rows, 2N], written, or null; input: read
  void* out;                 // forward: [rows, N]; input: bf16 [rows, N], glu [rows, 2N]; weight: [E, M, N]
  const uint8_t* dy;         // weight: as in a, for db
  float* db;                 // weight: [E, M] or null
  int32_t* status;           // may be null
  int64_t rows;
  int32_t N, n_tiles;        // columns of the product (glu forward: of h)
  int32_t M, m_tiles;        // weight: rows of an expert's matrix
  int32_t kc;                // length of the summed axis (weight: the expert's rows instead)
  int32_t E, act, bias_cols;
  int32_t split;             // CTAs that share a tile's sum: 1, 2, 4 or 8
  bool narrow;               // tiles of 128 columns (not glu forward; split 1, no pairs)
  bool bias_f32, out_f32, accumulate;
  uint32_t test_drop;        // the number of a load that each CTA leaves out; UINT32_MAX: none
};
int linear_n_tile(bool glu, bool narrow);  // columns of out that one tile covers (glu: forward)
int linear_m_tile(bool pair);
cudaError_t launch_linear(const LinearParams& p, bool glu, bool f32, bool pair, int sms, cudaStream_t stream);
cudaError_t launch_linear_input(const LinearParams& p, bool glu, bool pair, int sms, cudaStream_t stream);
cudaError_t launch_linear_weight(const LinearParams& p, bool f32, bool pair, int sms, cudaStream_t stream);

// The same for few rows (forward, input): a in boxes of 64 x kFewLinearRows, n_tiles
// of 128 columns, the summed axis split over `ranks` CTAs (1, 2, 4 or 8).
constexpr int kFewLinearRows = 32;
// The most groups of up to kFewLinearRows rows that the rows of `ragged` experts can make (0:
// one matrix, all rows).
inline int64_t few_linear_units(int64_t rows, int32_t ragged) {
  if (ragged == 0) return (rows + kFewLinearRows - 1) / kFewLinearRows;
  return (rows < ragged ? rows : ragged) + rows / kFewLinearRows;
}
cudaError_t launch_few_linear(const LinearParams& p, bool input, bool gate, int ranks, cudaStream_t stream);

}  // namespace moe
