// The router: choice of experts, their weights, and the gradient by the logits.
//
//   key = z, or sigmoid(z) + bias;   idx = the K largest keys, lower index first among equals
//   w_k = scale * p_k  or  scale * p_k / sum_j p_j,   p = softmax(z) or sigmoid(z)
//
// A warp takes a token, a lane every 32nd expert.  A choice is a maximum over the
// warp of the keys as ordered integers, K times; a lane knows the two largest of its
// own, and looks for the next two when both are taken.  Without a bias the keys are the
// logits, so the choice is exact.  With one the keys are float32 sums, off by up to
// 2^-20: K + 1 choices are made, and where two of them in a row lie closer together than
// that can tell, the token's choice is made again (choose_exactly), and of all keys so
// close to the largest the largest is found in 64 bits.
//
// Bound by instructions: 16384 tokens, 384 experts, 8 chosen: 14.7 us forward (20.4 with a bias), 8.8 the
// gradient of every logit; their bytes take 3.9 and 7.5.
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

// Floats as integers in the same order; -0 as 0, NaN as -inf, nothing at 0 (which
// stands for an expert that is taken or does not exist).
__device__ __forceinline__ uint32_t ordered(float v) {
  const int32_t b = __float_as_int(fmaxf(v + 0.0f, -INFINITY));
  return static_cast<uint32_t>(b ^ ((b >> 31) | static_cast<int32_t>(0x80000000)));
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

// 2^v within 2^-22 of itself, 0 below 2^-126.
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

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

// z becomes exp(z - top); 1 / their sum, 0 in a row without a finite logit.  The
// product with log2(e) is off by 2^-24 of itself, so a term by 2^-24 (1.5 (top - z) + 4)
// of itself: nothing in the sum, where such terms are small.
template <int N>
__device__ __forceinline__ float softmax_terms(float (&z)[N], float& top) {
  top = -INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, z[i]);
  top = warp_max(top);
  const float from = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    z[i] = exp2_fast((z[i] - from) * kLog2e);
    sum += z[i];
  }
  sum = warp_sum(sum);
  return sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
}

// The two largest keys of a lane that are not taken (0: none), lower places first among equals.
template <bool kTaken, int N>
__device__ __forceinline__ void two_largest(const uint32_t (&key)[N], uint32_t taken, uint32_t& k1, int& i1,
                                            uint32_t& k2, int& i2) {
  k1 = k2 = 0;
  i1 = i2 = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t k = kTaken && ((taken >> i) & 1) ? 0 : key[i];
    const bool first = k > k1, second = k > k2;
    k2 = first ? k1 : second ? k : k2;
    i2 = first ? i1 : second ? i : i2;
    k1 = first ? k : k1;
    i1 = first ? i : i1;
  }
}

// Two keys of at most m are told apart by float32 if they differ by more: a score
// (<= 1) is off by less than 2^-21 (exp2_fast, a sum, a reciprocal: 8 half steps), the sum
// with the bias by half a step, two keys by twice that.
__device__ __forceinline__ float key_error(float m) { return 0x1p-19f + 0x1p-21f * fabsf(m); }

// Lane k's choice k where float32 keys lie too close together: of the keys near the
// largest the largest in 64 bits.
template <class T, int N>
__device__ __noinline__ int choose_exactly(const T* row, const float* bias, int E, int K) {
  const int lane = threadIdx.x & 31;
  uint32_t key[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = i * 32 + lane;
    key[i] = e < E ? ordered(sigmoid(load(row + e)) + __ldg(bias + e)) : 0;
  }
  int mine = 0;
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
    const float m = from_ordered(best), near = m - key_error(m);
    const uint32_t from = isfinite(near) ? ordered(near) : best;
    int close = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) close += key[i] >= from;
    // 64 bits only where there is something to tell apart: they take a microsecond.
    if (__reduce_add_sync(kAll, close) > 1) {
      double top = -INFINITY;
      int at = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = i * 32 + lane;
        if (key[i] >= from && c < E) {
          const double exact = 1.0 / (1.0 + exp(-static_cast<double>(load(row + c)))) + __ldg(bias + c);
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
      if (at < E) e = at;  // else all of them are NaN
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e == i * 32 + lane) key[i] = 0;
    if (lane == k) mine = e;
  }
  return mine;
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
  for (int i = 0; i < N; ++i) z[i] = i * 32 + lane < E ? load(row + i * 32 + lane) : -INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = i * 32 + lane;
    key[i] = 0;
    if (e < E)
      key[i] = ordered(kBias ? __fdividef(1.0f, 1.0f + exp2_fast(-z[i] * kLog2e)) + __ldg(p.bias + e) : z[i]);
  }
  uint32_t taken = 0, k1, k2;
  int i1, i2;
  two_largest<false>(key, taken, k1, i1, k2, i2);
  bool second = true;  // whether k2 is known
  int mine = 0;        // lane k: choice k
  bool close = false;
  float before = 0.0f;
  for (int k = 0; k < (kBias ? K + 1 : K); ++k) {
    const uint32_t best = __reduce_max_sync(kAll, k1);
    if (kBias) {
      const float m = from_ordered(best);  // after the last expert there is nothing (0)
      close |= k > 0 && best > 0 && !(before - m > key_error(before));
      before = m;
      if (k == K) break;
    }
    const unsigned lanes = __ballot_sync(kAll, k1 == best);
    int e = i1 * 32 + lane;
    if (lanes & (lanes - 1)) e = __reduce_min_sync(kAll, k1 == best ? e : 0x7fffffff);
    else e = __shfl_sync(kAll, e, __ffs(lanes) - 1);
    if (lane == k) mine = e;
    if (k1 == best && e == i1 * 32 + lane) {
      taken |= 1u << i1;
      k1 = k2;
      i1 = i2;
      if (!second) two_largest<true>(key, taken, k1, i1, k2, i2);
      second = !second;
    }
  }
  if (kBias && close) mine = choose_exactly<T, N>(row, p.bias, E, K);
  const bool chosen = lane < K;
  const float zk = chosen ? load(row + mine) : 0.0f;
  float w;
  if (kNormalize) {
    w = share<kSigmoid>(zk, chosen);
  } else if (kSigmoid) {
    w = sigmoid(zk);
  } else {
    float top;
    const float inv = softmax_terms(z, top);
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
    inv = softmax_terms(z, top);
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
  float d = u;
  const unsigned same = __match_any_sync(kAll, chosen ? e : -1 - lane);
  if (__any_sync(kAll, (same & (same - 1)) != 0)) {  // the same expert named twice counts twice
    d = 0.0f;
    for (int k = 0; k < K; ++k) {
      const float v = __shfl_sync(kAll, u, k);
      if ((same >> k) & 1) d += v;
    }
  }
  if (kSigmoid) d *= sigmoid(-zk);
  if constexpr (kDense) {
    const float all = warp_sum(u);
    d -= exp_from(zk, top) * inv * all;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i * 32 + lane < E) store(out + i * 32 + lane, -(z[i] * inv) * all);
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
  if (p.E <= 128) return launch_n<T, 4>(p, sigmoid, normalize, backward, stream);
  if (p.E <= 256) return launch_n<T, 8>(p, sigmoid, normalize, backward, stream);
  if (p.E <= 384) return launch_n<T, 12>(p, sigmoid, normalize, backward, stream);
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
