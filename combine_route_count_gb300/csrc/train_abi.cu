// The C ABI of the training operators (declared in include/moe_train.h):
// argument checks and launches.

#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "abi_host.cuh"
#include "ffn_kernels.cuh"
#include "moe_train.h"
#include "train_kernels.cuh"

namespace {

using moe::aligned;
using moe::guarded;
using moe::launched;
using moe::NvtxRange;
using moe::sm_count;

constexpr int32_t kMaxSize = 1 << 30;  // of n and k: a tile's end past the last column, and twice that, are int32

bool type_ok(int type) { return type == MOE_TYPE_BF16 || type == MOE_TYPE_F32; }

bool router_ok(int logits_type, int64_t T, int32_t E, int32_t K, int score, float scale) {
  return type_ok(logits_type) && T >= 0 && T <= INT_MAX && E >= 1 && E <= MOE_MAX_EXPERTS && K >= 1 &&
         K <= MOE_MAX_TOP_K && K <= E && (score == MOE_SCORE_SOFTMAX || score == MOE_SCORE_SIGMOID) &&
         std::isfinite(scale);
}

bool moves_ok(int64_t T, int32_t H, int32_t K, int64_t rows) {
  return T >= 0 && H > 0 && H % 8 == 0 && K >= 1 && K <= MOE_MAX_TOP_K && T * K <= INT_MAX && T <= INT_MAX &&
         rows >= 0 && rows <= INT_MAX;
}

// bf16 matrix [rows, cols] as a tensor map of box_rows x 64 boxes.
bool encode_rows(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  return moe::encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, 2, dims, strides, box);
}

// bf16 weights [E, n, k] as a tensor map of box_rows x 64 boxes of one expert.
bool encode_weights(CUtensorMap* map, const void* base, int32_t E, int32_t n, int32_t k, int box_rows) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(E)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(k) * 2, static_cast<cuuint64_t>(k) * 2 * n};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  return moe::encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, 3, dims, strides, box);
}

bool product_ok(int64_t rows, int32_t n, int32_t k, int32_t E, const int32_t* offsets, const int32_t* status) {
  return rows >= 0 && rows <= INT_MAX - 256 && n > 0 && n % 8 == 0 && n <= kMaxSize && k > 0 && k % 8 == 0 &&
         k <= kMaxSize && E >= 1 && E <= MOE_MAX_EXPERTS && (offsets || E == 1) && aligned(offsets, 4) &&
         aligned(status, 4);
}

int32_t tiles(int32_t n, int32_t tile) { return (n + tile - 1) / tile; }

// Which kernel a product takes, from what the host knows: the mean of the experts' rows.
//
// Tiles by pairs of CTAs (256 x 256, half the operand traffic of two tiles of 128 x
// 256) from a mean of 256 rows an expert on; below it half of such a tile is empty.  us,
// single CTAs / pairs, N = K = 4096 but where said:
//   forward  8 experts: 50.6 / 53.9 at a mean of 128, 63.3 / 56.5 at 256, 173 / 149 at
//            1024; 64 experts, N 2816, K 2048, swiglu: 126 / 136 at 128, 158 / 142 at
//            256, under a skewed router 176 / 178; 1 expert: 161 / 141 at 8192 rows
//   by rows  8 experts 60.7 / 53.9 at 256; K 8192, swiglu: 381 / 332 at 1024
//   by weights  1 expert: 10.5 / 11.7 at 128 rows, 27.1 / 24.8 at 1024, 176 / 156 at
//            8192; 256 experts, N = K = 2048: 371 / 442 at 128 (bound by what it writes)
bool takes_pairs(int64_t rows, int32_t E) { return rows >= 256 * static_cast<int64_t>(E); }

// CTAs that share a tile of the few-row kernel; 0: not the few-row kernel.  It is
// for a mean of up to 4 rows an expert, and for calls whose tiles leave most SMs without
// work: two or more of its CTAs a tile fit on the GPU at once, whatever the rows.  (With one
// each, a long axis and many rows it reads the weights for every 32 of them: 5925 rows, N 176,
// K 6952, swiglu: 115 instead of 44.)  us, tile kernel / 1 / 2 / 4 / 8 CTAs a tile of 128
// columns (56 of them for N 7168; few_linear_units times that many for the rows):
//   N 7168, K 2048: 16.1 / 11.7 / 10.7 / 10.1 / 14.3 at 1 row, 16.1 / 13.3 / 11.7 / 11.4 /
//   17.2 at 32, 16.2 / 13.5 / 12.0 / 17.4 / 29 at 64, 16.6 / 13.8 / 19.5 / 29 / 48 at 128
//   (224 tiles), 15.8 / 24 / 30 / 48 / - at 256; N 2048, K 7168: 42 / 27 / 17.3 / 12.5 / 11.2 at
//   16; N = K = 4096: 17.8 (a split sum) / 18.3 / 14.9 / 21 / - at 128, 18.3 / 20.3 / 26 / 38 / -
//   at 256 (256 tiles); 8 experts, N = K = 1024: 11.3 / 8.9 / 8.6 / 8.8 / 13.7 at 64 rows,
//   11.2 / 10.5 / 11.1 / 16.8 / 30 at 512 (192 tiles); N 128, K 4096, 4096 rows (128 tiles): 15.2 (a
//   split sum) / 17.0 / 12.6 / 17.4 / -
// and, tile kernel / 1 CTA a tile, by the mean of the rows, 64 experts, N 2816, K 2048, swiglu:
//   116 / 112 at 2, 116 / 111 at 4 (skewed router 94.5 / 90), 116 / 113 at 8 (97 / 98); N 2048, K
//   1408: 63 / 63 at 8 (52 / 54), 64 / 65 at 16; 194 experts, N 4464, K 408, gelu, 14 rows: 22 / 15
int few_ranks(int64_t rows, int32_t ragged, int32_t cols, int32_t kc, int sms) {
  const int64_t all = moe::few_linear_units(rows, ragged) * tiles(cols, 128);
  int ranks = 1;
  while (ranks < 8 && all * ranks * 2 <= 2 * sms && ranks * 2 <= tiles(kc, 64)) ranks *= 2;
  return all <= sms || rows <= 4 * static_cast<int64_t>(ragged) ? ranks : 0;
}

// The most row tiles that `ragged` experts' rows make (0: one matrix).
int64_t row_tiles(int64_t rows, int32_t ragged) {
  return (rows + moe::linear_m_tile(false) - 1) / moe::linear_m_tile(false) + ragged;
}

// CTAs that share the sum of a tile, for calls with few tiles and a long summed axis
// (kc; by weights the mean of the experts' rows).  Sharing costs about 8 us, so a CTA keeps
// 12 blocks of 64 or more, and at most 128 CTAs take part (of clusters of 8, 96: more
// are not resident at once).  us, 1 / 2 / 4 / 8 CTAs a tile:
//   forward  N = K = 4096: 26.8 / 22.2 / 17.8 / 28.3 at 128 rows (16 tiles), 26.9 / 22.7 /
//            33 / 64 at 512; 2048 rows, N = K = 1024: 9.9 / 13.1 / 22.7 / 52
//   by rows  256 rows, N = K = 4096: 25.6 / 21.3 / 17.6 / 38
//   by weights  16384 rows, N = K = 512: 72 / 44 / 26.3 / 19.2; 8192 rows, N = K = 1024: 38.5 /
//            27 / 19.8 / 42, 2048: 45 / 58 / 77 / 128; 1024 rows, 1024: 8.9 / 12.1 / 11.2 / 29
int split_of(int64_t most_tiles, int64_t kc) {
  int split = 1;
  while (split < 8 && most_tiles * split * 2 <= (split == 4 ? 96 : 128) && kc / 64 >= 12 * split * 2) split *= 2;
  return split;
}

// What tiles of which shape a product of `most_row_tiles` x cols takes, into p; whether by pairs.
//
// Tiles of 128 columns (narrow) where all of them fit on the SMs at once: twice the CTAs, and six
// stages on their way instead of four, which is what a call without other work on its SMs waits
// for; two CTAs to a sum gain less.  us, one CTA a tile of 256 columns / of 128 / pairs / a sum
// split over 2 / 4:
//   forward  N = K = 4096, 256 rows: 27.2 / 18.2 / 23.8 / 22.4 / 18.6, 512: 27.2 / 18.9 / 24.0 /
//            23.1 / 33; 2048 rows, N = K = 1024: 9.9 / 7.9 / 10.7 / 13.3 / 22.8
//   by rows  589 rows, 2400 x 408: 22.1 / 14.6 / 17.2 / 18.7 / 14.1
//   by weights  1024 rows, N = K = 1024: 8.9 / 7.3 / 9.9 / 12.1 / 11.2; 6758 rows, 1376 x 280: 54 /
//            34.5 / 37 / 34.5 / 22.5
// and with several rounds of tiles: 40 experts' 3003 rows, 1416 x 2320, gelu: 62.8 / 70.1; 256
// experts' dw, 128 rows, N = K = 2048: 388 / 448; forward 256 experts, 8192 rows: 324 / 322.
bool choose_tiles(moe::LinearParams& p, int64_t most_row_tiles, int32_t cols, int64_t kc, bool glu, bool pairs, int sms) {
  p.n_tiles = tiles(cols, moe::linear_n_tile(glu, false));
  const int64_t most = most_row_tiles * p.n_tiles;
  p.split = split_of(most, kc);
  if (p.split > (glu ? 1 : 2)) return false;
  if (!glu) p.split = 1;
  if (!glu && 2 * most <= sms) {
    p.narrow = true;
    p.n_tiles = tiles(cols, moe::linear_n_tile(false, true));
    return false;
  }
  return pairs;
}

}  // namespace

#define MOE_API extern "C" __attribute__((visibility("default")))

MOE_API int moe_router_topk(const void* logits, int logits_type, const float* bias, int64_t num_tokens,
                            int32_t num_experts, int32_t top_k, int score, int normalize, float scale,
                            int32_t* topk_idx, float* topk_w, void* stream) {
  NvtxRange nvtx_range("moe_router_topk");
  if (!router_ok(logits_type, num_tokens, num_experts, top_k, score, scale)) return MOE_EINVAL;
  if (bias && score != MOE_SCORE_SIGMOID) return MOE_EINVAL;
  if (num_tokens == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_w) return MOE_EINVAL;
  if (!aligned(logits, logits_type == MOE_TYPE_F32 ? 4 : 2) || !aligned(bias, 4) || !aligned(topk_idx, 4) ||
      !aligned(topk_w, 4))
    return MOE_EINVAL;
  return guarded([&] {
    moe::RouterParams p = {};
    p.logits = logits;
    p.bias = bias;
    p.idx = topk_idx;
    p.w = topk_w;
    p.T = num_tokens;
    p.E = num_experts;
    p.K = top_k;
    p.scale = scale;
    p.f32 = logits_type == MOE_TYPE_F32;
    return launched(moe::launch_router(p, score == MOE_SCORE_SIGMOID, normalize != 0, false,
                                       static_cast<cudaStream_t>(stream)));
  });
}

MOE_API int moe_router_topk_backward(const void* logits, int logits_type, const int32_t* topk_idx,
                                     const float* d_topk_w, int64_t num_tokens, int32_t num_experts, int32_t top_k,
                                     int score, int normalize, float scale, void* d_logits, void* stream) {
  NvtxRange nvtx_range("moe_router_topk_backward");
  if (!router_ok(logits_type, num_tokens, num_experts, top_k, score, scale)) return MOE_EINVAL;
  if (num_tokens == 0) return MOE_OK;
  if (!logits || !topk_idx || !d_topk_w || !d_logits) return MOE_EINVAL;
  const size_t size = logits_type == MOE_TYPE_F32 ? 4 : 2;
  if (!aligned(logits, size) || !aligned(topk_idx, 4) || !aligned(d_topk_w, 4) || !aligned(d_logits, size))
    return MOE_EINVAL;
  return guarded([&] {
    moe::RouterParams p = {};
    p.logits = logits;
    p.idx = const_cast<int32_t*>(topk_idx);  // read only by the gradient
    p.dw = d_topk_w;
    p.d_logits = d_logits;
    p.T = num_tokens;
    p.E = num_experts;
    p.K = top_k;
    p.scale = scale;
    p.f32 = logits_type == MOE_TYPE_F32;
    return launched(moe::launch_router(p, score == MOE_SCORE_SIGMOID, normalize != 0, true,
                                       static_cast<cudaStream_t>(stream)));
  });
}

MOE_API int moe_combine_backward(const void* d_out, const void* expert_y, const float* topk_w,
                                 const int32_t* slot_row, int64_t num_tokens, int32_t hidden, int32_t top_k,
                                 int64_t rows, void* d_expert_y, float* d_topk_w, void* stream) {
  NvtxRange nvtx_range("moe_combine_backward");
  if (!moves_ok(num_tokens, hidden, top_k, rows)) return MOE_EINVAL;
  if (num_tokens == 0) return MOE_OK;
  if (!d_out || !topk_w || !slot_row || !d_expert_y || !expert_y != !d_topk_w) return MOE_EINVAL;
  if (!aligned(d_out, 16) || !aligned(expert_y, 16) || !aligned(topk_w, 4) || !aligned(slot_row, 4) ||
      !aligned(d_expert_y, 16) || !aligned(d_topk_w, 4))
    return MOE_EINVAL;
  return guarded([&] {
    moe::CombineGradParams p = {};
    p.d_out = static_cast<const uint8_t*>(d_out);
    p.y = static_cast<const uint8_t*>(expert_y);
    p.w = topk_w;
    p.slot_row = slot_row;
    p.dy = static_cast<uint8_t*>(d_expert_y);
    p.dw = d_topk_w;
    p.T = num_tokens;
    p.rows = rows;
    p.H = hidden;
    p.K = top_k;
    return launched(moe::launch_combine_grad(p, static_cast<cudaStream_t>(stream)));
  });
}

MOE_API int moe_dispatch_backward(const void* d_expert_x, const int32_t* slot_row, const void* add,
                                  int64_t num_tokens, int32_t hidden, int32_t top_k, int64_t rows, void* d_x,
                                  void* stream) {
  NvtxRange nvtx_range("moe_dispatch_backward");
  if (!moves_ok(num_tokens, hidden, top_k, rows)) return MOE_EINVAL;
  if (num_tokens == 0) return MOE_OK;
  if ((!d_expert_x && rows > 0) || !slot_row || !d_x) return MOE_EINVAL;
  if (!aligned(d_expert_x, 16) || !aligned(slot_row, 4) || !aligned(add, 16) || !aligned(d_x, 16)) return MOE_EINVAL;
  return guarded([&] {
    moe::DispatchGradParams p = {};
    p.de = static_cast<const uint8_t*>(d_expert_x);
    p.slot_row = slot_row;
    p.add = static_cast<const uint8_t*>(add);
    p.dx = static_cast<uint8_t*>(d_x);
    p.T = num_tokens;
    p.rows = rows;
    p.H = hidden;
    p.K = top_k;
    return launched(moe::launch_dispatch_grad(p, static_cast<cudaStream_t>(stream)));
  });
}

MOE_API int moe_expert_linear(const void* a, int64_t rows, int32_t k, const void* w, int32_t n, int32_t num_experts,
                              const int32_t* expert_offsets, const void* bias, int bias_type, int activation,
                              const void* residual, void* pre, void* out, int out_type, int32_t* status,
                              void* stream) {
  NvtxRange nvtx_range("moe_expert_linear");
  const bool glu = activation == MOE_ACT_SWIGLU;
  if (!product_ok(rows, n, k, num_experts, expert_offsets, status)) return MOE_EINVAL;
  if (activation < MOE_ACT_NONE || activation > MOE_ACT_SWIGLU || (glu && n % 16 != 0) || !type_ok(out_type) ||
      (bias && !type_ok(bias_type)))
    return MOE_EINVAL;
  if (rows == 0) return MOE_OK;
  if (!a || !w || !out) return MOE_EINVAL;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(bias, 16) || !aligned(residual, 16) || !aligned(pre, 16) ||
      !aligned(out, 16))
    return MOE_EINVAL;
  if (residual == out && out_type != MOE_TYPE_BF16) return MOE_EINVAL;
  return guarded([&] {
    const int sms = sm_count();
    if (sms <= 0) return static_cast<int>(MOE_ECUDA);
    const int ranks = few_ranks(rows, expert_offsets ? num_experts : 0, glu ? n / 2 : n, k, sms);
    moe::LinearParams p = {};
    if (!encode_rows(&p.a, a, rows, k, ranks > 0 ? moe::kFewLinearRows : 128) || !encode_weights(&p.b, w, num_experts, n, k, 128))
      return static_cast<int>(MOE_ECUDA);
    p.offsets = expert_offsets;
    p.bias = bias;
    p.residual = const_cast<void*>(residual);
    p.pre = pre;
    p.out = out;
    p.status = status;
    p.rows = rows;
    p.N = glu ? n / 2 : n;
    p.kc = k;
    p.E = num_experts;
    p.act = activation;
    p.bias_cols = n;
    p.bias_f32 = bias_type == MOE_TYPE_F32;
    p.out_f32 = out_type == MOE_TYPE_F32;
    p.test_drop = moe::test_drop();
    const cudaStream_t on = static_cast<cudaStream_t>(stream);
    if (ranks > 0) {
      p.n_tiles = tiles(p.N, 128);
      return launched(moe::launch_few_linear(p, false, glu, ranks, on));
    }
    const bool pair = choose_tiles(p, row_tiles(rows, expert_offsets ? num_experts : 0), p.N, k, glu,
                                   takes_pairs(rows, num_experts), sms);
    return launched(moe::launch_linear(p, glu, out_type == MOE_TYPE_F32, pair, sms, on));
  });
}

MOE_API int moe_expert_linear_backward_input(const void* dy, int64_t rows, int32_t n, const void* w, int32_t k,
                                             int32_t num_experts, const int32_t* expert_offsets, int activation,
                                             const void* pre, void* dx, int32_t* status, void* stream) {
  NvtxRange nvtx_range("moe_expert_linear_backward_input");
  if (!product_ok(rows, n, k, num_experts, expert_offsets, status)) return MOE_EINVAL;
  if (activation < MOE_ACT_NONE || activation > MOE_ACT_SWIGLU) return MOE_EINVAL;
  if (rows == 0) return MOE_OK;
  if (!dy || !w || !dx || !pre != (activation == MOE_ACT_NONE)) return MOE_EINVAL;
  if (!aligned(dy, 16) || !aligned(w, 16) || !aligned(pre, 16) || !aligned(dx, 16)) return MOE_EINVAL;
  return guarded([&] {
    const int sms = sm_count();
    if (sms <= 0) return static_cast<int>(MOE_ECUDA);
    const int ranks = few_ranks(rows, expert_offsets ? num_experts : 0, k, n, sms);
    moe::LinearParams p = {};
    if (!encode_rows(&p.a, dy, rows, n, ranks > 0 ? moe::kFewLinearRows : 128) || !encode_weights(&p.b, w, num_experts, n, k, 64))
      return static_cast<int>(MOE_ECUDA);
    p.offsets = expert_offsets;
    p.pre = const_cast<void*>(pre);
    p.out = dx;
    p.status = status;
    p.rows = rows;
    p.N = k;
    p.kc = n;
    p.E = num_experts;
    p.act = activation;
    p.test_drop = moe::test_drop();
    const cudaStream_t on = static_cast<cudaStream_t>(stream);
    if (ranks > 0) {
      p.n_tiles = tiles(k, 128);
      return launched(moe::launch_few_linear(p, true, false, ranks, on));
    }
    const bool pair = choose_tiles(p, row_tiles(rows, expert_offsets ? num_experts : 0), k, n, false,
                                   takes_pairs(rows, num_experts), sms);
    return launched(moe::launch_linear_input(p, activation == MOE_ACT_SWIGLU, pair, sms, on));
  });
}

MOE_API int moe_expert_linear_backward_weight(const void* dy, int64_t rows, int32_t n, const void* a, int32_t k,
                                              int32_t num_experts, const int32_t* expert_offsets, void* dw,
                                              int dw_type, float* db, int accumulate, int32_t* status, void* stream) {
  NvtxRange nvtx_range("moe_expert_linear_backward_weight");
  if (!product_ok(rows, n, k, num_experts, expert_offsets, status) || !type_ok(dw_type) || !dw || !aligned(dw, 16) ||
      !aligned(db, 16))
    return MOE_EINVAL;
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (accumulate) return MOE_OK;
    const size_t elements = static_cast<size_t>(num_experts) * n;
    cudaError_t err = cudaMemsetAsync(dw, 0, elements * k * (dw_type == MOE_TYPE_F32 ? 4 : 2), on);
    if (err == cudaSuccess && db) err = cudaMemsetAsync(db, 0, elements * sizeof(float), on);
    return launched(err);
  }
  if (!dy || !a || !aligned(dy, 16) || !aligned(a, 16)) return MOE_EINVAL;
  return guarded([&] {
    const int sms = sm_count();
    if (sms <= 0) return static_cast<int>(MOE_ECUDA);
    moe::LinearParams p = {};
    if (!encode_rows(&p.a, dy, rows, n, 64) || !encode_rows(&p.b, a, rows, k, 64)) return static_cast<int>(MOE_ECUDA);
    p.offsets = expert_offsets;
    p.out = dw;
    p.dy = static_cast<const uint8_t*>(dy);
    p.db = db;
    p.status = status;
    p.rows = rows;
    p.N = k;
    p.M = n;
    p.E = num_experts;
    p.accumulate = accumulate != 0;
    p.test_drop = moe::test_drop();
    const bool pair = choose_tiles(p, static_cast<int64_t>(num_experts) * tiles(n, moe::linear_m_tile(false)), k,
                                   rows / num_experts, false, takes_pairs(rows, num_experts), sms);
    p.m_tiles = tiles(n, moe::linear_m_tile(pair));
    return launched(moe::launch_linear_weight(p, dw_type == MOE_TYPE_F32, pair, sms, on));
  });
}
