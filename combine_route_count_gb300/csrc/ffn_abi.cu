// The C ABI of the feed-forward operators (declared in include/moe_ffn.h):
// argument checks and launches.  Exceptions do not cross it: what can throw
// in the host code below is the allocation of a per-device cache entry.

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include "abi_host.cuh"
#include "ffn_kernels.cuh"
#include "moe_ffn.h"

namespace {

using moe::aligned;
using moe::guarded;
using moe::launched;
using moe::NvtxRange;
using moe::sm_count;
using moe::test_drop;

// moe_ffn_test_drop_load's.
std::atomic<int32_t> g_test_drop{-1};

// E4M3 matrix [rows, cols] as a tensor map of box_rows x 128 boxes.
bool encode_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int box_rows = 128) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols)};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
  return moe::encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, 2, dims, strides, box);
}

// Which kernel a product takes.  The tile kernel (expert_gemm.cu) gives 128
// rows of one expert to a tile and all of K to one CTA, which is what many rows
// want; with few rows its tiles are mostly empty, and with few tiles a long K is
// walked by few SMs.  The few-row kernels (decode_layer.cu) put weight rows in
// the tile's 128 and split K, and read the weights again for every 16 rows of
// an expert.  Measured in us, tile kernel / row groups:
//   glu   E 256, H 7168, inner 1024: 465 / 460 at 2 rows an expert, 538 / 531 at
//         8, 545 / 597 at 16; E 8, H = inner = 4096 (256 tiles): 47 / 47 at 8,
//         47 / 53 at 32; E 8, H = inner = 1024 (64 tiles): 8.3 / 7.9 at 32, 8.2 /
//         8.9 at 64; E 1, H 7168, inner 2048 (16 tiles): 25 / 17 at 64 rows,
//         25 / 20 at 128, 26 / 31 at 256
//   gemm  E 256, N 7168, K 2048: 466 / 467 at 2, 543 / 546 at 8; N 1024, K 7168:
//         274 / 273 at 8, 278 / 285 at 16; E 32, N 512, K 4096: 16.8 / 9.8 at half
//         a row, 18.7 / 17.9 at 8; E 1, N 1024, K 8192 (4 tiles): 25 / 13 at 64
//         rows, 28 / 15 at 128; E 4, N 768, K 5120: 18.3 / 16.9 at 128 (24 tiles),
//         18.4 / 22.4 at 256
// The host knows the mean rows an expert, not their counts, and a skewed router
// costs row groups more.  With many tiles, rows on all / a quarter / one (E 256: on
// 256 / 64 / 8) of the experts:
//   glu   E 64, H 2048, inner 1408: mean 2 62.4 / 59.4, 20.5 / 13.6, 11.4 / 10.7;
//         4 62.6 / 59.7, 20.6 / 13.7, 11.6 / 12.6; 8 63.2 / 60.3, 20.5 / 21.9,
//         11.6 / 18.2
//         E 256, H 7168, inner 1024: mean 2 552 / 549, 154 / 145, 29.8 / 34.3; 8
//         557 / 552, 155 / 154, 32.4 / 103
//   gemm  E 64, N = K = 4096: mean 2 161 / 160, 46.5 / 45.8, 17.0 / 15.4; 4 162 /
//         160, 47.6 / 47.8, 17.0 / 21.5; 8 163 / 163, 47.3 / 57.1, 17.4 / 36.0
// So row groups take a mean of up to 4: beyond it they gain 5 % at most and may
// lose a multiple.  With few tiles, where they take more, they keep their gain
// however the rows lie (E 8, H = inner = 1024, mean 32: 8.3 / 7.3 on 8, 2 or 1
// expert; gemm E 4, N 768, K 5120, mean 128: 18.2 / 16.9 on 4, 18.2 / 16.2 on 1).
// and, for one matrix, tile kernel / few-row product: N 7168, K 2048: 10.1 / 6.1
// at one row, 10.1 / 7.6 at 32; N 2048, K 128: 4.3 / 3.5 at 16.
enum class Product { kTiles, kRowGroups, kFewRows };

Product choose_product(bool glu, bool grouped, int64_t rows, int32_t kblocks, int64_t n_tiles, int32_t E, int sms) {
  if (!glu && !grouped && rows <= moe::kFewDenseRows) return Product::kFewRows;
  const int64_t tiles = (std::min<int64_t>(rows, E) + rows / 128) * n_tiles;
  int64_t most = 4;  // rows an expert
  if (tiles * 4 <= sms) most = 128;
  else if (glu && tiles <= sms) most = 32;
  return rows <= most * E && (glu || kblocks >= 24) ? Product::kRowGroups : Product::kTiles;
}

// What the two grouped products have in common; N: columns of the output.
int expert_product(bool glu, const void* a, const float* a_scales, int64_t rows, int32_t K, const void* w,
                   const float* w_scales, int32_t N, int32_t E, const int32_t* offsets, void* out, float* h_scales,
                   bool f32, int32_t* status, void* stream) {
  const int64_t w_rows = glu ? 2 * static_cast<int64_t>(N) : N;
  if (rows < 0 || rows > INT_MAX - 128 || K <= 0 || K % 16 != 0 || N <= 0 || E < 1 || E > MOE_MAX_EXPERTS)
    return MOE_EINVAL;
  // A tile's end past the last column, and a block's past the last element, are int32 as well.
  if (K > INT_MAX - 127 || w_rows * E > INT_MAX - 255 || (!offsets && E != 1)) return MOE_EINVAL;
  if (rows == 0) return MOE_OK;
  if (!a || !a_scales || !w || !w_scales || !out || (glu && !h_scales)) return MOE_EINVAL;
  if (!aligned(a, 16) || !aligned(a_scales, 4) || !aligned(w, 16) || !aligned(w_scales, 4) || !aligned(offsets, 4) ||
      !aligned(out, 16) || !aligned(h_scales, 4) || !aligned(status, 4))
    return MOE_EINVAL;
  return guarded([&] {
    const int sms = sm_count();
    if (sms <= 0) return static_cast<int>(MOE_ECUDA);
    const int32_t kblocks = (K + MOE_FP8_BLOCK - 1) / MOE_FP8_BLOCK;
    const int32_t n_tiles = (N + moe::expert_gemm_n_tile(glu) - 1) / moe::expert_gemm_n_tile(glu);
    const Product product = choose_product(glu, offsets != nullptr, rows, kblocks, n_tiles, E, sms);
    if (product == Product::kFewRows) {
      moe::DecodeParams p = {};
      if (!encode_map(&p.w2_map, w, N, K) || !encode_map(&p.h_map, a, rows, K, moe::kFewChunk))
        return static_cast<int>(MOE_ECUDA);
      p.w2_scales = w_scales;
      p.h_scales = const_cast<float*>(a_scales);  // read only by launch_few_rows
      p.out = out;
      p.status = status;
      p.T = static_cast<int32_t>(rows);
      p.H = N;
      p.K = p.E = 1;
      p.I = K;
      p.h_blocks = kblocks;
      p.out_blocks = (N + MOE_FP8_BLOCK - 1) / MOE_FP8_BLOCK;
      p.out_f32 = f32;
      p.test_drop = test_drop();
      return launched(moe::launch_few_rows(p, sms, static_cast<cudaStream_t>(stream)));
    }
    if (product == Product::kRowGroups) {
      moe::DecodeParams p = {};
      if (!encode_map(&p.w13_map, w, w_rows * E, K) || !encode_map(&p.x_map, a, rows, K, moe::kFewChunk))
        return static_cast<int>(MOE_ECUDA);
      p.x_scales = a_scales;
      p.w13_scales = w_scales;
      p.offsets = offsets;
      p.hq = static_cast<uint8_t*>(out);
      p.h_scales = h_scales;
      p.out = out;
      p.status = status;
      p.T = static_cast<int32_t>(rows);
      p.H = K;
      p.K = 1;
      p.E = E;
      p.I = N;
      p.out_f32 = f32;
      p.test_drop = test_drop();
      return launched(moe::launch_row_groups(p, glu, sms, static_cast<cudaStream_t>(stream)));
    }
    moe::ExpertGemmParams p = {};
    if (!encode_map(&p.a, a, rows, K) || !encode_map(&p.w, w, w_rows * E, K, glu ? 64 : 128)) return static_cast<int>(MOE_ECUDA);
    p.a_scales = a_scales;
    p.w_scales = w_scales;
    p.offsets = offsets;
    p.out = out;
    p.h_scales = h_scales;
    p.status = status;
    p.rows = rows;
    p.kblocks = kblocks;
    p.N = N;
    p.n_tiles = n_tiles;
    p.E = E;
    p.w_rows = static_cast<int32_t>(w_rows);
    p.w_blocks = static_cast<int32_t>((w_rows + MOE_FP8_BLOCK - 1) / MOE_FP8_BLOCK);
    p.test_drop = test_drop();
    return launched(moe::launch_expert_gemm(p, glu, f32, sms, static_cast<cudaStream_t>(stream)));
  });
}

bool decode_config_ok(const moe_config* c, int32_t inter) {
  return c && moe_validate_config(c) == MOE_OK && c->num_tokens <= MOE_DECODE_MAX_TOKENS &&
         c->hidden % MOE_FP8_BLOCK == 0 && inter > 0 && inter % MOE_FP8_BLOCK == 0 &&
         static_cast<int64_t>(inter) * 2 * c->num_experts <= INT_MAX &&
         static_cast<int64_t>(c->hidden) * c->num_experts <= INT_MAX;
}

size_t decode_codes_bytes(const moe_config* c, int32_t inter) {
  return (static_cast<size_t>(c->num_tokens) * c->top_k * inter + 255) / 256 * 256;
}

size_t decode_workspace(const moe_config* c, int32_t inter) {
  const size_t scales = static_cast<size_t>(c->num_tokens) * c->top_k * (inter / MOE_FP8_BLOCK) * sizeof(float);
  return decode_codes_bytes(c, inter) + (scales + 255) / 256 * 256;
}

}  // namespace

uint32_t moe::test_drop() { return static_cast<uint32_t>(g_test_drop.load(std::memory_order_relaxed)); }

#define MOE_API extern "C" __attribute__((visibility("default")))

MOE_API int moe_add_rms_norm_fp8(const void* x, const void* residual, const void* weight, int weight_type,
                                 int64_t num_tokens, int32_t hidden, float eps, void* residual_out, void* y, void* xq,
                                 float* x_scales, void* stream) {
  NvtxRange nvtx_range("moe_add_rms_norm_fp8");
  if (num_tokens < 0 || num_tokens > INT_MAX || hidden <= 0 || hidden % MOE_FP8_BLOCK != 0 ||
      hidden > MOE_NORM_MAX_HIDDEN)
    return MOE_EINVAL;
  if (weight_type != MOE_TYPE_BF16 && weight_type != MOE_TYPE_F32) return MOE_EINVAL;
  if (!(eps > 0.0f) || std::isinf(eps)) return MOE_EINVAL;
  if (num_tokens == 0) return MOE_OK;
  if (!x || !weight || !xq || !x_scales || !residual != !residual_out) return MOE_EINVAL;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(residual_out, 16) ||
      !aligned(y, 16) || !aligned(xq, 16) || !aligned(x_scales, 4))
    return MOE_EINVAL;
  if (y && y == residual_out) return MOE_EINVAL;
  return guarded([&] {
    const int sms = sm_count();
    if (sms <= 0) return static_cast<int>(MOE_ECUDA);
    moe::AddNormParams p = {};
    p.x = static_cast<const uint8_t*>(x);
    p.residual = static_cast<const uint8_t*>(residual);
    p.weight = static_cast<const uint8_t*>(weight);
    p.residual_out = static_cast<uint8_t*>(residual_out);
    p.y = static_cast<uint8_t*>(y);
    p.xq = static_cast<uint8_t*>(xq);
    p.x_scales = x_scales;
    p.T = num_tokens;
    p.H = hidden;
    p.eps = eps;
    return launched(moe::launch_add_norm_fp8(p, weight_type == MOE_TYPE_F32, sms, static_cast<cudaStream_t>(stream)));
  });
}

MOE_API int moe_expert_gemm_fp8(const void* a, const float* a_scales, int64_t rows, int32_t k, const void* w,
                                const float* w_scales, int32_t n, int32_t num_experts, const int32_t* expert_offsets,
                                void* out, int out_type, int32_t* status, void* stream) {
  NvtxRange nvtx_range("moe_expert_gemm_fp8");
  if (n % 8 != 0 || (out_type != MOE_TYPE_BF16 && out_type != MOE_TYPE_F32)) return MOE_EINVAL;
  return expert_product(false, a, a_scales, rows, k, w, w_scales, n, num_experts, expert_offsets, out, nullptr,
                        out_type == MOE_TYPE_F32, status, stream);
}

MOE_API int moe_expert_glu_fp8(const void* a, const float* a_scales, int64_t rows, int32_t hidden, const void* w13,
                               const float* w13_scales, int32_t inter, int32_t num_experts,
                               const int32_t* expert_offsets, void* hq, float* h_scales, int32_t* status,
                               void* stream) {
  NvtxRange nvtx_range("moe_expert_glu_fp8");
  if (inter % MOE_FP8_BLOCK != 0) return MOE_EINVAL;
  return expert_product(true, a, a_scales, rows, hidden, w13, w13_scales, inter, num_experts, expert_offsets, hq,
                        h_scales, false, status, stream);
}

MOE_API int moe_decode_workspace_bytes(const moe_config* cfg, int32_t inter, size_t* bytes) {
  if (!bytes || !decode_config_ok(cfg, inter)) return MOE_EINVAL;
  *bytes = decode_workspace(cfg, inter);
  return MOE_OK;
}

MOE_API int moe_decode_layer_fp8(const moe_config* cfg, int32_t inter, const void* xq, const float* x_scales,
                                 const int32_t* topk_idx, const float* topk_w, const void* w13,
                                 const float* w13_scales, const void* w2, const float* w2_scales, void* out,
                                 int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange nvtx_range("moe_decode_layer_fp8");
  if (!decode_config_ok(cfg, inter)) return MOE_EINVAL;
  if (cfg->num_tokens == 0) return MOE_OK;
  if (!xq || !x_scales || !topk_idx || !topk_w || !w13 || !w13_scales || !w2 || !w2_scales || !out || !status ||
      !workspace)
    return MOE_EINVAL;
  if (!aligned(xq, 16) || !aligned(x_scales, 4) || !aligned(topk_idx, 4) || !aligned(topk_w, 4) || !aligned(w13, 16) ||
      !aligned(w13_scales, 4) || !aligned(w2, 16) || !aligned(w2_scales, 4) || !aligned(out, 16) ||
      !aligned(status, 4) || !aligned(workspace, 256) || workspace_bytes < decode_workspace(cfg, inter))
    return MOE_EINVAL;
  return guarded([&] {
    const int sms = sm_count();
    if (sms <= 0) return static_cast<int>(MOE_ECUDA);
    moe::DecodeParams p = {};
    if (!encode_map(&p.w13_map, w13, static_cast<int64_t>(cfg->num_experts) * 2 * inter, cfg->hidden) ||
        !encode_map(&p.x_map, xq, cfg->num_tokens, cfg->hidden, 1) ||
        !encode_map(&p.w2_map, w2, static_cast<int64_t>(cfg->num_experts) * cfg->hidden, inter) ||
        !encode_map(&p.h_map, workspace, static_cast<int64_t>(cfg->num_tokens) * cfg->top_k, inter,
                    moe::kFewChunk))
      return static_cast<int>(MOE_ECUDA);
    p.x_scales = x_scales;
    p.topk_idx = topk_idx;
    p.topk_w = topk_w;
    p.w13_scales = w13_scales;
    p.w2_scales = w2_scales;
    p.hq = static_cast<uint8_t*>(workspace);
    p.h_scales = reinterpret_cast<float*>(p.hq + decode_codes_bytes(cfg, inter));
    p.out = out;
    p.status = status;
    p.T = cfg->num_tokens;
    p.H = cfg->hidden;
    p.K = cfg->top_k;
    p.E = cfg->num_experts;
    p.I = inter;
    p.h_blocks = inter / MOE_FP8_BLOCK;
    p.out_blocks = cfg->hidden / MOE_FP8_BLOCK;
    p.test_drop = test_drop();
    return launched(moe::launch_decode_layer(p, sms, static_cast<cudaStream_t>(stream)));
  });
}

MOE_API int moe_ffn_test_drop_load(int32_t load) {
  if (load < -1) return MOE_EINVAL;
  g_test_drop.store(load, std::memory_order_relaxed);
  return MOE_OK;
}
