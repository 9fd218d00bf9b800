// Residual addition, root-mean-square norm and block-scaled E4M3 quantisation
// of token rows in one pass:
//
//   s = x + residual,  v = s * (1 / sqrt(mean(s^2) + eps)) * weight,
//   scale_b = max(amax_b |v|, 2^-100) / 448 (1 if the block is all zero),
//   q = E4M3(v / scale_b), per block b of 128 elements.
//
// All arithmetic is float32; the row's sum of squares is taken from the
// float32 s, and the codes come from the float32 s * weight without passing
// through bf16 (y and residual_out are separate roundings of v and s).
//
// Bound by memory: with a residual and y, 2+2 bytes in and 2+2+1 out per
// element, a few operations each.  A row has to be known before its first
// output, so it is held in registers between the two: each thread keeps one
// chunk of 16 elements (one 32-byte sector of an input; 8 lanes cover one
// 128-element block, so a block's largest value takes three shuffles and its
// codes leave as one 16-byte store per lane).  Threads of a row only meet
// once, for the sum.  A CTA walks rows b, b+G, ... and loads the next row
// before it waits for the current row's sum.  16384 x 7168 with a residual and y:
// 171 to 174 us, 6.1 TB/s.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ffn_kernels.cuh"
#include "fp8_quant.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

constexpr int kElems = 16;  // elements of one chunk

// A chunk of bf16 is 32 bytes, one sector, moved whole or as two halves.  Whole
// needs 32-byte alignment.  Whole stores are never slower than halves by more
// than noise; whole loads help until the two inputs of a residual are much
// larger than L2.  Measured in us, halves / whole stores / whole loads and stores:
//   no residual, y   8192 x 1024 9.1 / 9.0 / 8.8, 16384 x 7168 102 / 97 / 95,
//                    16384 x 16384 271 / 233 / 220; without y -1 to 5 % from
//                    left to right
//   residual, y      9216 x 1024 15.6 / 15.9 / 15.1, 8192 x 2048 26.9 / 27.4 / 26.5;
//                    from 2^25 elements on: 8192 x 4096 53.1 / 50.9 / 52.5, 8192 x
//                    7168 88.8 / 87.2 / 92.1, 16384 x 7168 176 / 173 / 182, 8192 x
//                    16384 195 / 194 / 203, but 4096 x 12288 77.5 / 71.7 / 70.9
//   residual only    16384 x 1024 21.1 / 21.2 / 20.2, 8192 x 7168 65.7 / 65.3 / 64.1;
//                    from 2^26 on, rows up to 8192: 16384 x 4096 77.7 / 76.3 / 79.8,
//                    8192 x 8192 75.1 / 74.9 / 77.5, 16384 x 8192 147 / 148 / 158;
//                    longer rows: 16384 x 12288 243 / 226 / 213
enum Access { kHalves, kSectorStores, kSectors };

// Which one rows on 32-byte boundaries take.
Access choose_access(bool residual, bool y, int64_t T, int32_t H) {
  const int64_t n = T * H;
  const bool halves_in = residual && (y ? n >= 1 << 25 : n >= 1 << 26 && H <= 8192);
  return halves_in ? kSectorStores : kSectors;
}

struct Chunk {
  uint4 a, b;
};

__device__ __forceinline__ void ld_stream_v8(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p));
}

template <bool kWide>
__device__ __forceinline__ Chunk load_chunk(const uint8_t* p) {
  Chunk c;
  if (kWide) {
    ld_stream_v8(p, c.a, c.b);
    return c;
  }
  c.a = ptx::ld_stream_v4(p);
  c.b = ptx::ld_stream_v4(p + 16);
  return c;
}

__device__ __forceinline__ void widen(const Chunk& c, float* v) {
  const uint32_t w[8] = {c.a.x, c.a.y, c.a.z, c.a.w, c.b.x, c.b.y, c.b.z, c.b.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[2 * j] = fp8q::lo_f(w[j]);
    v[2 * j + 1] = fp8q::hi_f(w[j]);
  }
}

template <bool kWide>
__device__ __forceinline__ void store_bf16(uint8_t* p, const float* v) {
  uint4 o[2];
  uint32_t* w = &o[0].x;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  if (kWide) {
    tc::st_v8(p, o[0], o[1]);
  } else {
    ptx::st_v4(p, o[0]);
    ptx::st_v4(p + 16, o[1]);
  }
}

// s = x (+ residual) of one chunk.
template <bool kResidual>
__device__ __forceinline__ void add_chunk(const Chunk& x, const Chunk& r, float* s) {
  widen(x, s);
  if (kResidual) {
    float add[kElems];
    widen(r, add);
#pragma unroll
    for (int j = 0; j < kElems; ++j) s[j] += add[j];
  }
}

__device__ __forceinline__ float square_sum(const float* s, float sum) {
#pragma unroll
  for (int j = 0; j < kElems; ++j) sum = fmaf(s[j], s[j], sum);
  return sum;
}

// Sum over the CTA's threads of one row, in an order that depends on the row
// length only.  Rows of more than one warp have the CTA to themselves.
__device__ __forceinline__ float row_sum(float sum, float* buf) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  const int warps = blockDim.x >> 5;
  if (warps > 1) {
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0.0f;
    for (int w = 0; w < warps; ++w) sum += buf[w];
  }
  return sum;
}

// Outputs of chunk c of row t from its s.  Every lane of the warp calls it;
// lanes with act = false take part in the shuffles only.
template <bool kResidual, bool kWeightF32, Access kAccess>
__device__ __forceinline__ void finish_chunk(const AddNormParams& p, int64_t t, int c, bool act, const float* s,
                                             float rms) {
  const int64_t at = t * p.H + static_cast<int64_t>(c) * kElems;
  float v[kElems];
#pragma unroll
  for (int j = 0; j < kElems; ++j) v[j] = 0.0f;
  if (act) {
    if (kResidual) store_bf16<kAccess != kHalves>(p.residual_out + at * 2, s);
    if (kWeightF32) {
      const float4* w = reinterpret_cast<const float4*>(p.weight) + c * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 f = __ldg(w + j);
        v[4 * j] = f.x, v[4 * j + 1] = f.y, v[4 * j + 2] = f.z, v[4 * j + 3] = f.w;
      }
    } else {
      const uint4* w = reinterpret_cast<const uint4*>(p.weight) + c * 2;
      widen(Chunk{__ldg(w), __ldg(w + 1)}, v);
    }
#pragma unroll
    for (int j = 0; j < kElems; ++j) v[j] *= s[j];
  }
  // v here is s * weight, still without rms: a block's codes do not depend on
  // its common factor, and every rounding left out is fewer codes that fall to
  // the wrong side.
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < kElems; ++j) amax = fmaxf(amax, fabsf(v[j]));
  // The 8 lanes of one 128-element block are 8 consecutive lanes.
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
  const float top = amax * rms;
  const float scale = amax > 0.0f ? __fdiv_rn(fmaxf(top, kTinyAmax), 448.0f) : 1.0f;
  // Below the floor 448 / amax may be infinite, and so may rms / scale: such a
  // block's values take rms first.
  const bool tiny = fminf(amax, top) < kTinyAmax;
  const float inv = __fdiv_rn(tiny ? 1.0f : 448.0f, tiny ? scale : amax);
  if (__any_sync(0xffffffffu, tiny)) {
#pragma unroll
    for (int j = 0; j < kElems; ++j) v[j] *= tiny ? rms : 1.0f;
    if (tiny) rms = 1.0f;
  }
  if (act) {
    uint4 q;
    uint32_t* o = &q.x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float* e = v + 4 * j;
      o[j] = fp8q::e4m3x2(__fmul_rn(e[0], inv), __fmul_rn(e[1], inv)) |
             (fp8q::e4m3x2(__fmul_rn(e[2], inv), __fmul_rn(e[3], inv)) << 16);
    }
    ptx::st_v4(p.xq + at, q);
    if (p.y) {
#pragma unroll
      for (int j = 0; j < kElems; ++j) v[j] *= rms;
      store_bf16<kAccess != kHalves>(p.y + at * 2, v);
    }
    if ((c & 7) == 0) p.x_scales[t * (p.H / MOE_FP8_BLOCK) + (c >> 3)] = scale;
  }
}

// Rows of at most 1024 chunks: one chunk a thread.  A row is shared
// by blockDim.x threads (a multiple of 32); blockDim.y rows of one warp each
// share a CTA.  x is read with non-coherent loads before anything of the same
// row is written, and by the thread that writes the same columns, so outputs
// may replace inputs row by row.
template <bool kResidual, bool kWeightF32, Access kAccess>
__global__ void __launch_bounds__(1024) add_norm_fp8_kernel(AddNormParams p, int chunks) {
  __shared__ float s_sum[2][32];
  ptx::wait_prerequisites();
  const int c = threadIdx.x;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.y;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const float inv_h = 1.0f / static_cast<float>(p.H);
  const Chunk zero = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  Chunk x = zero, r = zero;
  auto load_row = [&](int64_t t) {
    if (c < chunks && t < p.T) {
      const int64_t at = (t * p.H + static_cast<int64_t>(c) * kElems) * 2;
      x = load_chunk<kAccess == kSectors>(p.x + at);
      if (kResidual) r = load_chunk<kAccess == kSectors>(p.residual + at);
    }
  };
  // Every thread makes the same number of rounds, so all reach the barrier.
  const int64_t rounds = (p.T + stride - 1) / stride;
  load_row(first);
  for (int64_t n = 0; n < rounds; ++n) {
    const int64_t t = first + n * stride;
    float s[kElems];
    add_chunk<kResidual>(x, r, s);
    float sum = square_sum(s, 0.0f);  // threads without a chunk hold zeros
    if (n + 1 < rounds) load_row(t + stride);
    // Two buffers in turn: a warp that is a round ahead cannot overwrite sums
    // still being read, because a barrier lies between.
    sum = row_sum(sum, s_sum[n & 1]);
    finish_chunk<kResidual, kWeightF32, kAccess>(p, t, c, c < chunks && t < p.T, s, __frsqrt_rn(fmaf(sum, inv_h, p.eps)));
  }
}

// Longer rows: 1024 threads walk the row twice, the second time from the
// caches.  A thread reads its own columns again before it writes them.  With y,
// 4096 rows: of 32768 228 us (0.79 of the copy rate's floor) with a residual, 171
// (0.59) without; of 65536 424 (0.85) and 295 (0.68); of 16512 156 (0.58) and 119
// (0.43), where only 8 threads of 1024 have work in the second step of a walk.
template <bool kResidual, bool kWeightF32, Access kAccess>
__global__ void __launch_bounds__(1024) add_norm_fp8_long_kernel(AddNormParams p, int chunks) {
  __shared__ float s_sum[2][32];
  ptx::wait_prerequisites();
  const float inv_h = 1.0f / static_cast<float>(p.H);
  const int chunks_up = (chunks + 31) / 32 * 32;  // whole warps reach the shuffles
  int n = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, ++n) {
    float s[kElems];
    auto load = [&](int c) {
      const int64_t at = (t * p.H + static_cast<int64_t>(c) * kElems) * 2;
      const Chunk x = load_chunk<kAccess == kSectors>(p.x + at);
      add_chunk<kResidual>(x, kResidual ? load_chunk<kAccess == kSectors>(p.residual + at) : x, s);
    };
    float sum = 0.0f;
    for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
      load(c);
      sum = square_sum(s, sum);
    }
    sum = row_sum(sum, s_sum[n & 1]);
    const float rms = __frsqrt_rn(fmaf(sum, inv_h, p.eps));
    for (int c = threadIdx.x; c < chunks_up; c += blockDim.x) {
      if (c < chunks) load(c);
      finish_chunk<kResidual, kWeightF32, kAccess>(p, t, c, c < chunks, s, rms);
    }
  }
}

template <bool kResidual, bool kWeightF32, Access kAccess>
cudaError_t launch(const AddNormParams& p, int sms, cudaStream_t stream) {
  const int chunks = p.H / kElems;
  const bool one = chunks <= 1024;
  auto* kernel = one ? add_norm_fp8_kernel<kResidual, kWeightF32, kAccess> : add_norm_fp8_long_kernel<kResidual, kWeightF32, kAccess>;
  const int row_threads = one ? (chunks + 31) / 32 * 32 : 1024;
  const int rows = row_threads == 32 ? 8 : 1;
  const int resident = resident_ctas_per_sm(reinterpret_cast<const void*>(kernel), row_threads * rows, 0);
  if (resident < 1) return cudaErrorInvalidConfiguration;
  int64_t grid = (p.T + rows - 1) / rows;
  const int64_t most = static_cast<int64_t>(sms) * resident;
  if (grid > most) grid = most;
  return launch_kernel(kernel, dim3(static_cast<unsigned>(grid)), dim3(row_threads, rows), 0, stream, true, p, chunks);
}

template <Access kAccess>
cudaError_t launch_access(const AddNormParams& p, bool weight_f32, int sms, cudaStream_t stream) {
  if (kAccess == kSectorStores || p.residual)
    return weight_f32 ? launch<true, true, kAccess>(p, sms, stream) : launch<true, false, kAccess>(p, sms, stream);
  if constexpr (kAccess != kSectorStores)
    return weight_f32 ? launch<false, true, kAccess>(p, sms, stream) : launch<false, false, kAccess>(p, sms, stream);
}

}  // namespace

cudaError_t launch_add_norm_fp8(const AddNormParams& p, bool weight_f32, int sms, cudaStream_t stream) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.residual) |
                       reinterpret_cast<uintptr_t>(p.residual_out) | reinterpret_cast<uintptr_t>(p.y);
  if (at % 32 != 0) return launch_access<kHalves>(p, weight_f32, sms, stream);
  return choose_access(p.residual, p.y, p.T, p.H) == kSectorStores
             ? launch_access<kSectorStores>(p, weight_f32, sms, stream)
             : launch_access<kSectors>(p, weight_f32, sms, stream);
}

}  // namespace moe
