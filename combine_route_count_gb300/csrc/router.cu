// The router: choice of experts, their weights, and the gradient by the logits.
//
//   key = z, or sigmoid(z) + bias;   idx = the K largest keys, lower index first among equals
//   w_k = scale * p_k  or  scale * p_k / sum_j p_j,   p = softmax(z) or sigmoid(z)
//
// A warp takes a token, a lane every 32nd expert.  A choice is a maximum over the
// warp of the keys as ordered integers, K times.  Without a bias the keys are the
// logits, so the choice is exact.  With one the keys are float32 sums, off by
// about 2^-21: where several keys lie that close to the largest, those few are
// computed again in 64 bits.
//
// Normalised weights divide by the largest chosen score first, so that they
// neither overflow nor vanish however small the scores are:
//   softmax  p_k ~ exp(z_k - M),  M the largest chosen logit
//   sigmoid  p_k ~ exp(min(z_k, 0) - M) / (1 + exp(-|z_k|)),  M the largest min(z, 0)
//
// The gradient, with L_k = log p_k (d w_k / d L_j = w_k (delta_kj - [normalised] w_j / scale)):
//   u_k  = w_k * (dw_k - [normalised] sum_j dw_j w_j / scale)
//   dz_e = sum_k u_k * d L_k / d z_e:  softmax u_e - p_e sum_k u_k (the sum is 0
//   when normalised), sigmoid u_e * (1 - p_e)

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ptx.cuh"
#include "train_kernels.cuh"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 4;

__device__ __forceinline__ float load(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load(const __nv_bfloat16* p) {
  return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p))) << 16);
}
__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
  return v;
}

// Floats as integers in the same order; -0 as 0, NaN below -inf, nothing at 0
// (which stands for an expert that is taken or does not exist).
__device__ __forceinline__ uint32_t ordered(float v) {
  if (v != v) return 1;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }
// exp(a - b), 0 for a = -inf whatever b is.
__device__ __forceinline__ float exp_from(float a, float b) { return a == -INFINITY ? 0.0f : expf(a - b); }

// The scores of the chosen experts, up to a common factor where they are going
// to be normalised.  z: the logit of the lane's choice (lanes < K).
template <bool kSigmoid>
__device__ __forceinline__ float share(float z, bool chosen) {
  const float e = kSigmoid ? fminf(z, 0.0f) : z;
  const float top = warp_max(chosen ? e : -INFINITY);
  float s = chosen ? exp_from(e, top) : 0.0f;
  if (kSigmoid) s = __fdiv_rn(s, 1.0f + expf(-fabsf(z)));
  const float sum = warp_sum(chosen ? s : 0.0f);
  return sum > 0.0f ? __fdiv_rn(s, sum) : (sum == 0.0f ? 0.0f : sum);
}

// exp(z - top) over the sum of it, 0 in a row without a finite logit.
template <int N>
__device__ __forceinline__ void softmax_stats(const float (&z)[N], int lane, int E, float& top, float& inv) {
  top = -INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i * 32 + lane < E) top = fmaxf(top, z[i]);
  top = warp_max(top);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i * 32 + lane < E) sum += exp_from(z[i], top);
  sum = warp_sum(sum);
  inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
}

template <class T, int N, bool kSigmoid, bool kNormalize, bool kBias>
__global__ void __launch_bounds__(kWarps * 32) router_kernel(RouterParams p) {
  ptx::wait_prerequisites();
  ptx::launch_dependents();
  const int lane = threadIdx.x & 31, E = p.E, K = p.K;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const T* row = static_cast<const T*>(p.logits) + t * E;
  float z[N];
  uint32_t key[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = i * 32 + lane;
    z[i] = e < E ? load(row + e) : -INFINITY;
    key[i] = 0;
    if (e < E) key[i] = ordered(kBias ? sigmoid(z[i]) + __ldg(p.bias + e) : z[i]);
  }
  int mine = 0;  // lane k: choice k
  for (int k = 0; k < K; ++k) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) best = max(best, key[i]);
    best = __reduce_max_sync(kAll, best);
    int e = 0x7fffffff;
#pragma unroll
    for (int i = N - 1; i >= 0; --i)
      if (key[i] == best) e = i * 32 + lane;
    e = __reduce_min_sync(kAll, e);
    if (kBias) {
      // Float32 keys are off by at most 4 * 2^-24 of the score (<= 1) and half a
      // step of the sum, two of them by twice that.
      const float m = from_ordered(best);
      const float near = m - (0x1p-19f + 0x1p-21f * fabsf(m));
      const uint32_t from = isfinite(near) ? ordered(near) : best;
      int close = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) close += key[i] >= from;
      if (__reduce_add_sync(kAll, close) > 1) {
        double top = -INFINITY;
        int at = 0x7fffffff;
#pragma unroll 1
        for (int i = 0; i < N; ++i) {
          const int c = i * 32 + lane;
          uint32_t this_key = 0;
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (j == i) this_key = key[j];
          if (c < E && this_key >= from) {
            const double exact = 1.0 / (1.0 + exp(-static_cast<double>(load(row + c)))) + __ldg(p.bias + c);
            if (exact > top) {
              top = exact;
              at = c;
            }
          }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
          const double other = __shfl_xor_sync(kAll, top, d);
          const int other_at = __shfl_xor_sync(kAll, at, d);
          if (other > top || (other == top && other_at < at)) {
            top = other;
            at = other_at;
          }
        }
        if (at < E) e = at;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e == i * 32 + lane) key[i] = 0;
    if (lane == k) mine = e;
  }
  const bool chosen = lane < K;
  const float zk = chosen ? load(row + mine) : 0.0f;
  float w;
  if (kNormalize) {
    w = share<kSigmoid>(zk, chosen);
  } else if (kSigmoid) {
    w = sigmoid(zk);
  } else {
    float top, inv;
    softmax_stats(z, lane, E, top, inv);
    w = exp_from(zk, top) * inv;
  }
  if (chosen) {
    p.idx[t * K + lane] = mine;
    p.w[t * K + lane] = p.scale * w;
  }
}

template <class T, int N, bool kSigmoid, bool kNormalize>
__global__ void __launch_bounds__(kWarps * 32) router_grad_kernel(RouterParams p) {
  ptx::wait_prerequisites();
  ptx::launch_dependents();
  const int lane = threadIdx.x & 31, E = p.E, K = p.K;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const T* row = static_cast<const T*>(p.logits) + t * E;
  T* out = static_cast<T*>(p.d_logits) + t * E;
  constexpr bool kDense = !kSigmoid && !kNormalize;
  float z[kDense ? N : 1], top = 0.0f, inv = 0.0f;
  if constexpr (kDense) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = i * 32 + lane < E ? load(row + i * 32 + lane) : -INFINITY;
    softmax_stats(z, lane, E, top, inv);
  }
  const int e = lane < K ? __ldg(p.idx + t * K + lane) : -1;
  const bool chosen = e >= 0 && e < E;
  const float zk = chosen ? load(row + e) : 0.0f;
  const float dw = chosen ? p.scale * __ldg(p.dw + t * K + lane) : 0.0f;
  float u;
  if (kNormalize) {
    const float w = share<kSigmoid>(zk, chosen);
    u = w * (dw - warp_sum(w * dw));
  } else {
    u = dw * (kSigmoid ? sigmoid(zk) : exp_from(zk, top) * inv);
  }
  if (!chosen) u = 0.0f;
  // The same expert named twice counts twice.
  float sum_here = 0.0f;
  for (int k = 0; k < K; ++k) {
    const int other = __shfl_sync(kAll, e, k);
    const float v = __shfl_sync(kAll, u, k);
    if (other == e) sum_here += v;
  }
  float d = sum_here;
  if (kSigmoid) d *= sigmoid(-zk);
  if constexpr (kDense) {
    const float all = warp_sum(u);
    d -= exp_from(zk, top) * inv * all;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i * 32 + lane < E) store(out + i * 32 + lane, -(exp_from(z[i], top) * inv) * all);
  } else {
    for (int i = lane; i < E; i += 32) store(out + i, 0.0f);
  }
  __syncwarp();  // the chosen ones' values come last
  if (chosen) store(out + e, d);
}

template <class T, int N>
cudaError_t launch_n(const RouterParams& p, bool sigmoid, bool normalize, bool backward, cudaStream_t stream) {
  void (*kernel)(RouterParams);
  if (backward)
    kernel = sigmoid ? (normalize ? router_grad_kernel<T, N, true, true> : router_grad_kernel<T, N, true, false>)
                     : (normalize ? router_grad_kernel<T, N, false, true> : router_grad_kernel<T, N, false, false>);
  else if (!sigmoid)
    kernel = normalize ? router_kernel<T, N, false, true, false> : router_kernel<T, N, false, false, false>;
  else if (p.bias)
    kernel = normalize ? router_kernel<T, N, true, true, true> : router_kernel<T, N, true, false, true>;
  else
    kernel = normalize ? router_kernel<T, N, true, true, false> : router_kernel<T, N, true, false, false>;
  return launch_kernel(kernel, dim3(static_cast<unsigned>((p.T + kWarps - 1) / kWarps)), dim3(kWarps * 32), 0, stream,
                       true, p);
}

template <class T>
cudaError_t launch_t(const RouterParams& p, bool sigmoid, bool normalize, bool backward, cudaStream_t stream) {
  if (p.E <= 64) return launch_n<T, 2>(p, sigmoid, normalize, backward, stream);
  if (p.E <= 256) return launch_n<T, 8>(p, sigmoid, normalize, backward, stream);
  if (p.E <= 512) return launch_n<T, 16>(p, sigmoid, normalize, backward, stream);
  return launch_n<T, 32>(p, sigmoid, normalize, backward, stream);
}

}  // namespace

cudaError_t launch_router(const RouterParams& p, bool f32, bool sigmoid, bool normalize, bool backward,
                          cudaStream_t stream) {
  return f32 ? launch_t<float>(p, sigmoid, normalize, backward, stream)
             : launch_t<__nv_bfloat16>(p, sigmoid, normalize, backward, stream);
}

}  // namespace moe
