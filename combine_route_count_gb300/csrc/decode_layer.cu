// A whole expert layer for a few tokens (T <= 64) in two kernels, weights and
// activations block-scaled E4M3:
//
//   decode_glu   h[t,k] = SiLU(W1[e] x[t]) * (W3[e] x[t]),  e = topk_idx[t,k],
//                quantised by blocks of 128 like every payload here
//   decode_down  out[t] = bf16( sum_k topk_w[t,k] * W2[e] h[t,k] )
//
// Bound by memory: the chosen experts' weights are read once (3 * I * H bytes
// each) for a handful of tokens, so what counts is to keep many weight bytes
// in flight all the time and to start early.  The weights go straight from
// global memory into the fragments of mma.sync (16 weight rows x 8 tokens,
// K = 32): a lane's 16-byte loads hold the K elements of its row in an order
// that is not the fragment's, but the token operand is loaded with the same
// order, and a sum does not depend on it.  Shared memory, tensor memory and
// their barriers would only add to the way; the arithmetic (16 x 8 tile of
// which one or two token columns are real) stays far below the load time.
//
// Each 128 of K is summed by four matrix instructions from zero and then added
// with its two scales to float32 accumulators.
//
// Routing: every CTA sorts the T*K (token, expert) pairs itself (a bit per
// token in a mask per expert; a pair's place among its expert's rows is the
// number of lower bits set), about 2 us less than a kernel of its own.
// Malformed routing is seen by every CTA alike: nothing is written but the
// status.
//
// decode_down is launched while decode_glu runs and brings in its first
// weights before it waits for h.  Sums have a fixed order: same inputs, same
// bits.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ffn_kernels.cuh"
#include "fp8_quant.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxPairs = MOE_DECODE_MAX_TOKENS * MOE_MAX_TOP_K;
constexpr int kBlock = MOE_FP8_BLOCK;

// The layer's routing, built by every CTA.  Rows are the pairs ordered by
// (expert, token); expert number a is the a-th that has any.
struct Routing {
  uint32_t mask[MOE_MAX_EXPERTS][2];  // tokens of each expert
  int16_t active[kMaxPairs];          // the experts that have rows, ascending
  int16_t first[kMaxPairs + 1];       // their first rows
  int16_t row_of[MOE_MAX_EXPERTS];    // first row of each expert
  uint8_t token[kMaxPairs];           // of each row
  float weight[kMaxPairs];            // topk_w of each row
  int32_t warp_active[32], warp_rows[32];
  int32_t n_active, bad;
};

__device__ __forceinline__ void build_routing(Routing& r, const DecodeParams& p) {
  const int pairs = p.T * p.K, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) r.bad = 0;
  for (int e = threadIdx.x; e < p.E; e += kThreads) r.mask[e][0] = r.mask[e][1] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += kThreads) {
    const int e = p.topk_idx[i], t = i / p.K;
    if (e < 0 || e >= p.E) {
      r.bad = 1;
    } else {
      const uint32_t bit = 1u << (t & 31);
      if (atomicOr(&r.mask[e][t >> 5], bit) & bit) r.bad = 1;  // repeated within the token
    }
  }
  __syncthreads();
  if (r.bad) return;  // the same for the whole CTA
  const int chunks = (p.E + 31) / 32;
  for (int c = warp; c < chunks; c += kWarps) {
    const int e = c * 32 + lane;
    const int n = e < p.E ? __popc(r.mask[e][0]) + __popc(r.mask[e][1]) : 0;
    const int rows = __reduce_add_sync(0xffffffffu, n);
    const uint32_t some = __ballot_sync(0xffffffffu, n > 0);
    if (lane == 0) {
      r.warp_active[c] = __popc(some);
      r.warp_rows[c] = rows;
    }
  }
  __syncthreads();
  for (int c = warp; c < chunks; c += kWarps) {
    const int e = c * 32 + lane;
    const int n = e < p.E ? __popc(r.mask[e][0]) + __popc(r.mask[e][1]) : 0;
    const int before = lane < c ? r.warp_active[lane] : 0, before_rows = lane < c ? r.warp_rows[lane] : 0;
    const int base = __reduce_add_sync(0xffffffffu, before);
    const int base_row = __reduce_add_sync(0xffffffffu, before_rows);
    const uint32_t some = __ballot_sync(0xffffffffu, n > 0);
    int sum = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += up;
    }
    if (n > 0) {
      const int a = base + __popc(some & ((1u << lane) - 1));
      r.active[a] = static_cast<int16_t>(e);
      r.first[a] = r.row_of[e] = static_cast<int16_t>(base_row + sum - n);
    }
    if (c == chunks - 1 && lane == 0) {
      const int n_active = base + __popc(some);
      r.n_active = n_active;
      r.first[n_active] = static_cast<int16_t>(pairs);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += kThreads) {
    const int e = p.topk_idx[i], t = i / p.K;
    const int low = t < 32 ? __popc(r.mask[e][0] & ((1u << t) - 1))
                           : __popc(r.mask[e][0]) + __popc(r.mask[e][1] & ((1u << (t - 32)) - 1));
    const int row = r.row_of[e] + low;
    r.token[row] = static_cast<uint8_t>(t);
    r.weight[row] = p.topk_w[i];
  }
  __syncthreads();
}

__device__ __forceinline__ uint4 ldg_v4(const uint8_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// Two 16-byte pieces of one row's 128 bytes of K: bytes [16 t, +16) and [64 + 16 t, +16).
struct Piece {
  uint4 a, b;
};
__device__ __forceinline__ uint32_t word(const Piece& f, int i) {
  const uint32_t w[8] = {f.a.x, f.a.y, f.a.z, f.a.w, f.b.x, f.b.y, f.b.z, f.b.w};
  return w[i];
}
__device__ __forceinline__ Piece load_weights(const uint8_t* p) {
  return Piece{ptx::ld_stream_v4(p), ptx::ld_stream_v4(p + 64)};
}

// d[0..3] = (rows g and g + 8) x (tokens 2t, 2t + 1), summed over 128 of K.
__device__ __forceinline__ void mma_128(float* d, const Piece& lo, const Piece& hi, const Piece& x) {
  d[0] = d[1] = d[2] = d[3] = 0.0f;
#pragma unroll
  for (int s = 0; s < 4; ++s)
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(word(lo, 2 * s)), "r"(word(hi, 2 * s)), "r"(word(lo, 2 * s + 1)), "r"(word(hi, 2 * s + 1)),
          "r"(word(x, 2 * s)), "r"(word(x, 2 * s + 1)));
}

// ---- first kernel -----------------------------------------------------------
// Unit: (expert with rows, block of 128 columns of h) = 128 gate and 128 up
// rows of w13; a warp has 16 of each, as two 16-row operands of 8 gate rows
// (fragment rows 0-7) and their 8 up rows (8-15), so that a lane ends up with
// both halves of the same h.  kTiles token tiles of 8 cover T.
template <int kTiles, int kDepth>
__global__ void __launch_bounds__(kThreads, kTiles <= 2 ? 2 : 1) decode_glu_kernel(DecodeParams p) {
  __shared__ Routing r;
  __shared__ float s_amax[kWarps][kTiles * 8];
  ptx::wait_prerequisites();
  // From here on everything earlier in the stream is done, which
  // decode_down's early reads of topk_idx, topk_w and the weights rely on.
  ptx::launch_dependents();
  build_routing(r, p);
  if (r.bad) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int jb = p.I / kBlock, kb_n = p.H / kBlock;
  const int units = r.n_active * jb;

  Piece buf[kDepth][2][2];  // [stage][operand][gate, up]
  const uint8_t* wp;        // this lane's gate row of operand 0
  const int64_t up_off = static_cast<int64_t>(p.I) * p.H, m_off = static_cast<int64_t>(8) * p.H;
  auto point_at = [&](int u) {
    const int a = u / jb, j = u - a * jb;
    wp = p.w13 + (static_cast<int64_t>(r.active[a]) * 2 * p.I + j * kBlock + warp * 16 + g) * p.H + q * 16;
  };
  auto fetch = [&](Piece (*f)[2], int kb) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint8_t* at = wp + m * m_off + kb * kBlock;
      f[m][0] = load_weights(at);
      f[m][1] = load_weights(at + up_off);
    }
  };
  int u = blockIdx.x;
  if (u < units) {
    point_at(u);
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
      if (d < kb_n) fetch(buf[d], d);
  }
  for (; u < units; u += gridDim.x) {
    const int a = u / jb, j = u - a * jb, e = r.active[a];
    const int row0 = r.first[a], n = r.first[a + 1] - row0;
    const float* sg = p.w13_scales + (static_cast<int64_t>(e) * 2 * jb + j) * kb_n;
    const float* su = sg + static_cast<int64_t>(jb) * kb_n;
    // Token rows of this lane: column g of each tile as operand, columns 2q
    // and 2q + 1 as results.  Columns past the expert's rows repeat row 0.
    const uint8_t* x[kTiles];
    const float* sx[kTiles][2];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const int c = i * 8 + g, c0 = i * 8 + 2 * q;
      x[i] = p.xq + static_cast<int64_t>(r.token[row0 + (c < n ? c : 0)]) * p.H + q * 16;
      sx[i][0] = p.x_scales + static_cast<int64_t>(r.token[row0 + (c0 < n ? c0 : 0)]) * kb_n;
      sx[i][1] = p.x_scales + static_cast<int64_t>(r.token[row0 + (c0 + 1 < n ? c0 + 1 : 0)]) * kb_n;
    }
    float acc[kTiles][2][4];
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[i][m][k] = 0.0f;
    for (int kb0 = 0; kb0 < kb_n; kb0 += kDepth) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        const int kb = kb0 + d;
        if (kb < kb_n) {
          const float fg = __ldg(sg + kb), fu = __ldg(su + kb);
#pragma unroll
          for (int i = 0; i < kTiles; ++i) {
            if (i * 8 < n) {
              const Piece xf = {ldg_v4(x[i] + kb * kBlock), ldg_v4(x[i] + kb * kBlock + 64)};
              const float s0 = __ldg(sx[i][0] + kb), s1 = __ldg(sx[i][1] + kb);
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                float v[4];
                mma_128(v, buf[d][m][0], buf[d][m][1], xf);
                acc[i][m][0] = fmaf(v[0], s0 * fg, acc[i][m][0]);
                acc[i][m][1] = fmaf(v[1], s1 * fg, acc[i][m][1]);
                acc[i][m][2] = fmaf(v[2], s0 * fu, acc[i][m][2]);
                acc[i][m][3] = fmaf(v[3], s1 * fu, acc[i][m][3]);
              }
            }
          }
          if (kb + kDepth < kb_n) fetch(buf[d], kb + kDepth);
        }
      }
    }
    if (u + gridDim.x < units) {  // the next unit's weights are on their way during the epilogue
      point_at(u + gridDim.x);
#pragma unroll
      for (int d = 0; d < kDepth; ++d)
        if (d < kb_n) fetch(buf[d], d);
    }
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      if (i * 8 < n) {
        float top0 = 0.0f, top1 = 0.0f;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          float* v = acc[i][m];
          v[0] = v[0] / (1.0f + expf(-v[0])) * v[2];
          v[1] = v[1] / (1.0f + expf(-v[1])) * v[3];
          top0 = fmaxf(top0, fabsf(v[0]));
          top1 = fmaxf(top1, fabsf(v[1]));
        }
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) {
          top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, s));
          top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, s));
        }
        if (g == 0) {
          s_amax[warp][i * 8 + 2 * q] = top0;
          s_amax[warp][i * 8 + 2 * q + 1] = top1;
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = i * 8 + 2 * q + h;
        if (c < n) {
          float amax = 0.0f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) amax = fmaxf(amax, s_amax[w][c]);
          const float scale = amax > 0.0f ? __fdiv_rn(fmaxf(amax, kTinyAmax), 448.0f) : 1.0f;
          const float inv = __fdiv_rn(1.0f, scale);
          uint8_t* dst = p.hq + static_cast<int64_t>(row0 + c) * p.I + j * kBlock + warp * 16 + g;
          const uint32_t two = fp8q::e4m3x2(__fmul_rn(acc[i][0][h], inv), __fmul_rn(acc[i][1][h], inv));
          dst[0] = static_cast<uint8_t>(two);
          dst[8] = static_cast<uint8_t>(two >> 8);
          if (warp == 0 && g == 0) p.h_scales[static_cast<int64_t>(row0 + c) * jb + j] = scale;
        }
      }
    }
    __syncthreads();  // s_amax is read before the next unit writes it
  }
}

// ---- second kernel ------------------------------------------------------------
// A CTA owns 16 columns of out, for every token and expert; its warps share
// the (expert, K block) items evenly, each a contiguous range.  A warp adds
// what an expert gives to its own copy of out's columns in shared memory,
// token by token (an expert has a token at most once: no two lanes meet); the
// copies are added in warp order at the end.
template <int kTiles, int kDepth>
__global__ void __launch_bounds__(kThreads, 2) decode_down_kernel(DecodeParams p) {
  extern __shared__ float s_out[];  // [kWarps][T][16]
  __shared__ Routing r;
  build_routing(r, p);  // topk_idx and topk_w: see the first kernel's launch_dependents
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int kb_n = p.I / kBlock, n0 = blockIdx.x * 16;
  if (r.bad) {
    ptx::wait_prerequisites();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = MOE_EROUTE;
    return;
  }
  const int items = r.n_active * kb_n;
  const int end = static_cast<int>(static_cast<int64_t>(items) * (warp + 1) / kWarps);
  int it = static_cast<int>(static_cast<int64_t>(items) * warp / kWarps);
  // Where the next item to fetch lies.
  int fa = it / kb_n, fk = it - fa * kb_n, fetched = it;
  Piece buf[kDepth][2];
  auto fetch = [&](Piece* f) {
    const uint8_t* w =
        p.w2 + (static_cast<int64_t>(r.active[fa]) * p.H + n0 + g) * p.I + fk * kBlock + q * 16;
    f[0] = load_weights(w);
    f[1] = load_weights(w + static_cast<int64_t>(8) * p.I);
    ++fetched;
    if (++fk == kb_n) fk = 0, ++fa;
  };
#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (fetched < end) fetch(buf[d]);
  float* mine = s_out + warp * p.T * 16;
  for (int i = lane; i < p.T * 16; i += 32) mine[i] = 0.0f;
  __syncwarp();
  ptx::wait_prerequisites();  // hq and h_scales
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = MOE_OK;

  int a = it / kb_n, kb = it - a * kb_n;
  float acc[kTiles][4];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
  while (it < end) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (it < end) {
        const int row0 = r.first[a], n = r.first[a + 1] - row0;
        const float fw = __ldg(p.w2_scales + (static_cast<int64_t>(r.active[a]) * (p.H / kBlock) + n0 / kBlock) * kb_n +
                               kb);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          if (i * 8 < n) {
            const int c = i * 8 + g, c0 = i * 8 + 2 * q;
            const uint8_t* h = p.hq + static_cast<int64_t>(row0 + (c < n ? c : 0)) * p.I + kb * kBlock + q * 16;
            const Piece hf = {ld_v4(h), ld_v4(h + 64)};
            const float s0 = ld_f32(p.h_scales + static_cast<int64_t>(row0 + (c0 < n ? c0 : 0)) * kb_n + kb);
            const float s1 = ld_f32(p.h_scales + static_cast<int64_t>(row0 + (c0 + 1 < n ? c0 + 1 : 0)) * kb_n + kb);
            float v[4];
            mma_128(v, buf[d][0], buf[d][1], hf);
            acc[i][0] = fmaf(v[0], s0 * fw, acc[i][0]);
            acc[i][1] = fmaf(v[1], s1 * fw, acc[i][1]);
            acc[i][2] = fmaf(v[2], s0 * fw, acc[i][2]);
            acc[i][3] = fmaf(v[3], s1 * fw, acc[i][3]);
          }
        }
        if (fetched < end) fetch(buf[d]);
        ++it;
        if (++kb == kb_n || it == end) {  // this warp's part of the expert is complete
#pragma unroll
          for (int i = 0; i < kTiles; ++i) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int c = i * 8 + 2 * q + h;
              if (c < n) {
                const float w = r.weight[row0 + c];
                float* o = mine + r.token[row0 + c] * 16 + g;
                o[0] = fmaf(w, acc[i][h], o[0]);
                o[8] = fmaf(w, acc[i][2 + h], o[8]);
              }
            }
            acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
          }
          if (kb == kb_n) kb = 0, ++a;
          __syncwarp();
        }
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.T * 16; i += kThreads) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += s_out[w * p.T * 16 + i];
    reinterpret_cast<__nv_bfloat16*>(p.out)[static_cast<int64_t>(i >> 4) * p.H + n0 + (i & 15)] =
        __float2bfloat16_rn(sum);
  }
}

template <int kTiles, int kDepthGlu, int kDepthDown>
cudaError_t launch(const DecodeParams& p, int sms, cudaStream_t stream) {
  const int pairs = p.T * p.K;
  auto* glu = decode_glu_kernel<kTiles, kDepthGlu>;
  const int resident = resident_ctas_per_sm(reinterpret_cast<const void*>(glu), kThreads, 0);
  if (resident < 1) return cudaErrorInvalidConfiguration;
  int64_t units = static_cast<int64_t>(pairs < p.E ? pairs : p.E) * (p.I / kBlock);
  const int64_t most = static_cast<int64_t>(sms) * resident;
  if (units > most) units = most;
  cudaError_t err = launch_kernel(glu, dim3(static_cast<unsigned>(units)), dim3(kThreads), 0, stream, true, p);
  if (err != cudaSuccess) return err;
  auto* down = decode_down_kernel<kTiles, kDepthDown>;
  const size_t smem = static_cast<size_t>(kWarps) * p.T * 16 * sizeof(float);
  err = set_kernel_limits(reinterpret_cast<const void*>(down), smem);
  if (err != cudaSuccess) return err;
  return launch_kernel(down, dim3(p.H / 16), dim3(kThreads), smem, stream, true, p);
}

}  // namespace

cudaError_t launch_decode_layer(const DecodeParams& p, int sms, cudaStream_t stream) {
  if (p.T <= 8) return launch<1, 2, 3>(p, sms, stream);
  if (p.T <= 16) return launch<2, 2, 3>(p, sms, stream);
  if (p.T <= 32) return launch<4, 2, 3>(p, sms, stream);
  return launch<8, 2, 3>(p, sms, stream);
}

}  // namespace moe
