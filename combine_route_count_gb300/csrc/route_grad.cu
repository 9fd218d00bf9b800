// Gradients of the two moves of an expert layer, over the dispatch's slot_row:
//
//   combine_grad   dy[slot_row[t,k]] = bf16(w[t,k] * g[t]),  dw[t,k] = <g[t], y[slot_row[t,k]]>
//   dispatch_grad  dx[t] = bf16(sum_k de[slot_row[t,k]] + add[t])
//
// Both are bound by memory: (1 + 2 K) and K + 1 (+ 1) rows a token.  4096 tokens, H 7168,
// K 8: combine_grad 152 us, 6.56 TB/s; dispatch_grad 76.4 us, 6.92 TB/s; 16384 tokens 587 us
// (6.80 TB/s) and 311 us (6.80 TB/s).

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ptx.cuh"
#include "train_kernels.cuh"

namespace moe {
namespace {

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ float dot8(uint4 a, uint4 b, float s) {
  s = fmaf(lo(a.x), lo(b.x), s);
  s = fmaf(hi(a.x), hi(b.x), s);
  s = fmaf(lo(a.y), lo(b.y), s);
  s = fmaf(hi(a.y), hi(b.y), s);
  s = fmaf(lo(a.z), lo(b.z), s);
  s = fmaf(hi(a.z), hi(b.z), s);
  s = fmaf(lo(a.w), lo(b.w), s);
  return fmaf(hi(a.w), hi(b.w), s);
}
__device__ __forceinline__ uint4 scaled(uint4 a, float w) {
  return make_uint4(bf16x2(w * lo(a.x), w * hi(a.x)), bf16x2(w * lo(a.y), w * hi(a.y)),
                    bf16x2(w * lo(a.z), w * hi(a.z)), bf16x2(w * lo(a.w), w * hi(a.w)));
}

// y may be dy: a plain load, in the thread that writes the same 16 bytes later.
__device__ __forceinline__ uint4 ld_v4(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

constexpr int kMaxWarps = 8;

// Sums of K values over the kGroup lanes of a group.  While there are several, two
// lanes swap halves of them and go on with one half each; so a lane ends with kLeft sums,
// those from `first` on, and where lanes outnumber sums the ones with `writes` have them.
template <int K, int kGroup>
struct GroupSums {
  static constexpr int kLeft = K > kGroup ? K / kGroup : 1;
  int first;
  bool writes;
  __device__ __forceinline__ explicit GroupSums(float (&v)[K], int lane) : first(0), writes(true) {
    int n = K;
#pragma unroll
    for (int d = kGroup / 2; d > 0; d /= 2) {
      const bool upper = lane & d;
      if (n > 1) {
        n /= 2;
        if (upper) first += n;
#pragma unroll
        for (int j = 0; j < K / 2; ++j)
          if (j < n) {
            const float got = __shfl_xor_sync(0xffffffffu, upper ? v[j] : v[j + n], d);
            v[j] = (upper ? v[j + n] : v[j]) + got;
          }
      } else {
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], d);
        writes = writes && !upper;
      }
    }
  }
};

// kGroup lanes, or (0) the whole block, take a token: a thread reads 16 bytes of g[t]
// and of the token's K rows, and writes 16 bytes of each.
template <int KMAX, bool kDots, int kGroup>
__global__ void __launch_bounds__(kMaxWarps * 32) combine_grad_kernel(CombineGradParams p) {
  __shared__ float s_dot[kGroup ? 1 : kMaxWarps][KMAX];
  ptx::wait_prerequisites();
  ptx::launch_dependents();
  const int group = kGroup ? kGroup : blockDim.x;
  const int64_t t = kGroup ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / group) + threadIdx.x / group : blockIdx.x;
  const int K = p.K, at = threadIdx.x % group;
  const bool here = t < p.T;  // the last block may have fewer tokens
  const int64_t row_bytes = static_cast<int64_t>(p.H) * 2;
  int32_t row[KMAX];
  float w[KMAX], dot[KMAX];
#pragma unroll
  for (int k = 0; k < KMAX; ++k) {
    row[k] = -1;
    dot[k] = 0.0f;
    if (k < K && here) {
      row[k] = __ldg(p.slot_row + t * K + k);
      if (row[k] >= p.rows) row[k] = -1;
      w[k] = __ldg(p.w + t * K + k);
    }
  }
  for (int64_t c = static_cast<int64_t>(at) * 16; here && c < row_bytes; c += group * 16) {
    const uint4 g = ptx::ld_stream_v4(p.d_out + t * row_bytes + c);
    uint4 v[KMAX];
    if (kDots) {
#pragma unroll
      for (int k = 0; k < KMAX; ++k)
        if (row[k] >= 0) v[k] = ld_v4(p.y + row[k] * row_bytes + c);
    }
#pragma unroll
    for (int k = 0; k < KMAX; ++k) {
      if (row[k] >= 0) {
        if (kDots) dot[k] = dot8(g, v[k], dot[k]);
        ptx::st_v4(p.dy + row[k] * row_bytes + c, scaled(g, w[k]));
      }
    }
  }
  if (!kDots) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const GroupSums<KMAX, kGroup ? kGroup : 32> sums(dot, lane);
#pragma unroll
  for (int j = 0; j < sums.kLeft; ++j) {
    const int k = sums.first + j;
    if (!sums.writes || k >= K) continue;
    if (kGroup == 0) s_dot[warp][k] = dot[j];
    else if (here) p.dw[t * K + k] = dot[j];
  }
  if (kGroup) return;
  __syncthreads();
  if (threadIdx.x < K) {
    float sum = 0.0f;
    for (int i = 0; i < group / 32; ++i) sum += s_dot[i][threadIdx.x];
    p.dw[t * K + threadIdx.x] = sum;
  }
}

template <int KMAX, bool kDots>
cudaError_t launch_combine_grad_k(const CombineGradParams& p, cudaStream_t stream) {
  const int chunks = p.H / 8;
  if (chunks <= 64) {
    // Rows of up to 256 bytes: 8 lanes a token; up to 1024: a warp.  16384 tokens of 8 x 64
    // elements: 6.7 us, a warp each 23.2.
    const int group = chunks <= 16 ? 8 : 32;
    int threads = 32;  // few tokens: many blocks
    while (threads < kMaxWarps * 32 && p.T * group > static_cast<int64_t>(threads) * 1024) threads *= 2;
    const int64_t blocks = (p.T * group + threads - 1) / threads;
    auto* kernel = group == 8 ? combine_grad_kernel<KMAX, kDots, 8> : combine_grad_kernel<KMAX, kDots, 32>;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, stream, true, p);
  }
  // A block a token.  us with blocks of up to 64 / 128 / 256 threads: 4096 tokens of 8 x 7168
  // 157 / 153 / 152, 16384 tokens 599 / 592 / 587, 1024 tokens 45.1 / 47.0 / 43.3.
  // With few tokens every thread has one chunk, or as few as there are threads for.
  int threads = 64;
  while (threads < kMaxWarps * 32 && threads * (p.T <= 256 ? 1 : 4) < chunks) threads *= 2;
  return launch_kernel(combine_grad_kernel<KMAX, kDots, 0>, dim3(static_cast<unsigned>(p.T)), dim3(threads), 0, stream,
                       true, p);
}

template <int KMAX>
cudaError_t launch_combine_grad_k(const CombineGradParams& p, cudaStream_t stream) {
  return p.dw ? launch_combine_grad_k<KMAX, true>(p, stream) : launch_combine_grad_k<KMAX, false>(p, stream);
}

__device__ __forceinline__ void add8(float (&a)[8], uint4 v) {
  a[0] += lo(v.x);
  a[1] += hi(v.x);
  a[2] += lo(v.y);
  a[3] += hi(v.y);
  a[4] += lo(v.z);
  a[5] += hi(v.z);
  a[6] += lo(v.w);
  a[7] += hi(v.w);
}

constexpr int kSumThreads = 256;

// A thread takes 16 bytes of one token's row: its K loads are in flight together.
template <int KMAX>
__global__ void __launch_bounds__(kSumThreads) dispatch_grad_kernel(DispatchGradParams p) {
  ptx::wait_prerequisites();
  ptx::launch_dependents();
  const int K = p.K;
  const int64_t chunks = p.H / 8;
  const int64_t g = static_cast<int64_t>(blockIdx.x) * kSumThreads + threadIdx.x;
  const int64_t t = g / chunks, c = (g - t * chunks) * 16;
  if (t >= p.T) return;
  const int64_t row_bytes = static_cast<int64_t>(p.H) * 2;
  uint4 v[KMAX];
  int32_t row[KMAX];
#pragma unroll
  for (int k = 0; k < KMAX; ++k) {
    row[k] = k < K ? __ldg(p.slot_row + t * K + k) : -1;
    if (row[k] >= p.rows) row[k] = -1;
    if (row[k] >= 0) v[k] = ptx::ld_stream_v4(p.de + row[k] * row_bytes + c);
  }
  uint4 more;
  if (p.add) more = ld_v4(p.add + t * row_bytes + c);
  float a[8] = {};
#pragma unroll
  for (int k = 0; k < KMAX; ++k)
    if (row[k] >= 0) add8(a, v[k]);
  if (p.add) add8(a, more);
  ptx::st_v4(p.dx + t * row_bytes + c,
             make_uint4(bf16x2(a[0], a[1]), bf16x2(a[2], a[3]), bf16x2(a[4], a[5]), bf16x2(a[6], a[7])));
}

template <int KMAX>
cudaError_t launch_dispatch_grad_k(const DispatchGradParams& p, cudaStream_t stream) {
  const int64_t threads = p.T * (p.H / 8);
  const int64_t blocks = (threads + kSumThreads - 1) / kSumThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_kernel(dispatch_grad_kernel<KMAX>, dim3(static_cast<unsigned>(blocks)), dim3(kSumThreads), 0, stream,
                       true, p);
}

}  // namespace

cudaError_t launch_combine_grad(const CombineGradParams& p, cudaStream_t stream) {
  if (p.K <= 2) return launch_combine_grad_k<2>(p, stream);
  if (p.K <= 4) return launch_combine_grad_k<4>(p, stream);
  if (p.K <= 8) return launch_combine_grad_k<8>(p, stream);
  return launch_combine_grad_k<16>(p, stream);
}

cudaError_t launch_dispatch_grad(const DispatchGradParams& p, cudaStream_t stream) {
  if (p.K <= 2) return launch_dispatch_grad_k<2>(p, stream);
  if (p.K <= 4) return launch_dispatch_grad_k<4>(p, stream);
  if (p.K <= 8) return launch_dispatch_grad_k<8>(p, stream);
  return launch_dispatch_grad_k<16>(p, stream);
}

}  // namespace moe
