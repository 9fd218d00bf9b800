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

// Logit i of the call, of either type.
__device__ __forceinline__ float load(const RouterParams& p, int64_t i) {
  if (p.f32) return __ldg(static_cast<const float*>(p.logits) + i);
  return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const unsigned short*>(p.logits) + i)) << 16);
}
__device__ __forceinline__ void store(const RouterParams& p, int64_t i, float v) {
  if (p.f32) static_cast<float*>(p.d_logits)[i] = v;
  else static_cast<__nv_bfloat16*>(p.d_logits)[i] = __float2bfloat16_rn(v);
}
// A lane's logits of the token whose first one is number `row`: every G-th.
template <int G, int N>
__device__ __forceinline__ void load_row(const RouterParams& p, int64_t row, int lane, float (&z)[N]) {
  if (p.f32) {
    const float* from = static_cast<const float*>(p.logits) + row;
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = i * G + lane < p.E ? __ldg(from + i * G + lane) : -INFINITY;
  } else {
    const unsigned short* from = static_cast<const unsigned short*>(p.logits) + row;
#pragma unroll
    for (int i = 0; i < N; ++i)
      z[i] = i * G + lane < p.E ? __uint_as_float(static_cast<uint32_t>(__ldg(from + i * G + lane)) << 16) : -INFINITY;
  }
}

// Over the G lanes of a token; the whole warp calls them together.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int d = G / 2; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int d = G / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
  return v;
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  if constexpr (G == 32) {
    return __reduce_max_sync(kAll, v);
  } else {
#pragma unroll
    for (int d = G / 2; d > 0; d >>= 1) v = max(v, __shfl_xor_sync(kAll, v, d));
    return v;
  }
}
template <int G>
__device__ __forceinline__ int group_min(int v) {
  if constexpr (G == 32) {
    return __reduce_min_sync(kAll, v);
  } else {
#pragma unroll
    for (int d = G / 2; d > 0; d >>= 1) v = min(v, __shfl_xor_sync(kAll, v, d));
    return v;
  }
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
template <bool kSigmoid, int G>
__device__ __forceinline__ float share(float z, bool chosen) {
  const float e = kSigmoid ? fminf(z, 0.0f) : z;
  const float top = group_max<G>(chosen ? e : -INFINITY);
  float s = chosen ? exp_from(e, top) : 0.0f;
  if (kSigmoid) s = __fdiv_rn(s, 1.0f + expf(-fabsf(z)));
  const float sum = group_sum<G>(chosen ? s : 0.0f);
  return sum > 0.0f ? __fdiv_rn(s, sum) : (sum == 0.0f ? 0.0f : sum);
}

// z becomes exp(z - top); 1 / their sum, 0 in a row without a finite logit.  The
// product with log2(e) is off by 2^-24 of itself, so a term by 2^-24 (1.5 (top - z) + 4)
// of itself: nothing in the sum, where such terms are small.
template <int G, int N>
__device__ __forceinline__ float softmax_terms(float (&z)[N], float& top) {
  top = -INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, z[i]);
  top = group_max<G>(top);
  const float from = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    z[i] = exp2_fast((z[i] - from) * kLog2e);
    sum += z[i];
  }
  sum = group_sum<G>(sum);
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
template <int G, int N>
__device__ __noinline__ int choose_exactly(const RouterParams& p, int64_t row, int lane) {
  float z[N];
  load_row<G>(p, row, lane, z);
  uint32_t key[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = i * G + lane;
    key[i] = e < p.E ? ordered(sigmoid(z[i]) + __ldg(p.bias + e)) : 0;
  }
  int mine = 0;
  for (int k = 0; k < p.K; ++k) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) best = max(best, key[i]);
    best = group_max<G>(best);
    int e = 0x7fffffff;
#pragma unroll
    for (int i = N - 1; i >= 0; --i)
      if (key[i] == best) e = i * G + lane;
    e = group_min<G>(e);
    const float m = from_ordered(best), near = m - key_error(m);
    const uint32_t from = isfinite(near) ? ordered(near) : best;
    uint32_t close = 0;  // a bit for each of the lane's keys near the largest
#pragma unroll
    for (int i = 0; i < N; ++i) close |= static_cast<uint32_t>(key[i] >= from) << i;
    // 64 bits only where there is something to tell apart: they take a microsecond.
    if (__any_sync(kAll, group_sum<G>(static_cast<float>(__popc(close))) > 1.0f)) {
      double top = -INFINITY;
      int at = 0x7fffffff;
      for (; close; close &= close - 1) {
        const int c = (__ffs(close) - 1) * G + lane;
        if (c < p.E) {
          const double exact = 1.0 / (1.0 + exp(-static_cast<double>(load(p, row + c)))) + __ldg(p.bias + c);
          if (exact > top) {
            top = exact;
            at = c;
          }
        }
      }
      __syncwarp();
#pragma unroll
      for (int d = G / 2; d > 0; d >>= 1) {
        const double other = __shfl_xor_sync(kAll, top, d);
        const int other_at = __shfl_xor_sync(kAll, at, d);
        if (other > top || (other == top && other_at < at)) {
          top = other;
          at = other_at;
        }
      }
      if (at < p.E) e = at;  // else all of them are NaN
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e == i * G + lane) key[i] = 0;
    if (lane == k) mine = e;
  }
  return mine;
}

// This lane's token and place among its G lanes; behind the last token a group does the
// last one again and keeps it to itself.
template <int G>
struct Place {
  int lane, base;
  int64_t t;
  bool here;
  __device__ __forceinline__ explicit Place(int64_t T) {
    lane = threadIdx.x % G;
    base = (threadIdx.x & 31) - lane;
    t = (static_cast<int64_t>(blockIdx.x) * (kWarps * 32) + threadIdx.x) / G;
    here = t < T;
    if (!here) t = T - 1;
  }
};

// G lanes a token, N logits a lane, K <= G.
template <int G, int N, bool kSigmoid, bool kNormalize, bool kBias>
__global__ void __launch_bounds__(kWarps * 32) router_kernel(const __grid_constant__ RouterParams p) {
  ptx::wait_prerequisites();
  ptx::launch_dependents();
  const Place<G> at(p.T);
  const int lane = at.lane, E = p.E, K = p.K;
  const int64_t row = at.t * E;
  float z[N];
  load_row<G>(p, row, lane, z);
  uint32_t key[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = i * G + lane;
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
    const uint32_t best = group_max<G>(k1);
    if (kBias) {
      const float m = from_ordered(best);  // after the last expert there is nothing (0)
      close |= k > 0 && best > 0 && !(before - m > key_error(before));
      before = m;
      if (k == K) break;
    }
    int e = i1 * G + lane;
    if (G == 32) {
      const unsigned lanes = __ballot_sync(kAll, k1 == best);
      if (lanes & (lanes - 1)) e = group_min<G>(k1 == best ? e : 0x7fffffff);
      else e = __shfl_sync(kAll, e, __ffs(lanes) - 1);
    } else {
      e = group_min<G>(k1 == best ? e : 0x7fffffff);
    }
    if (lane == k) mine = e;
    if (k1 == best && e == i1 * G + lane) {
      taken |= 1u << i1;
      k1 = k2;
      i1 = i2;
      if (!second) two_largest<true>(key, taken, k1, i1, k2, i2);
      second = !second;
    }
  }
  if (kBias && __any_sync(kAll, close)) mine = choose_exactly<G, N>(p, row, lane);
  const bool chosen = lane < K;
  const float zk = chosen ? load(p, row + mine) : 0.0f;
  float w;
  if (kNormalize) {
    w = share<kSigmoid, G>(zk, chosen);
  } else if (kSigmoid) {
    w = sigmoid(zk);
  } else {
    float top;
    const float inv = softmax_terms<G>(z, top);
    w = exp_from(zk, top) * inv;
  }
  if (chosen && at.here) {
    p.idx[at.t * K + lane] = mine;
    p.w[at.t * K + lane] = p.scale * w;
  }
}

template <int G, int N, bool kSigmoid, bool kNormalize>
__global__ void __launch_bounds__(kWarps * 32) router_grad_kernel(const __grid_constant__ RouterParams p) {
  ptx::wait_prerequisites();
  ptx::launch_dependents();
  const Place<G> at(p.T);
  const int lane = at.lane, E = p.E, K = p.K;
  const int64_t row = at.t * E;
  constexpr bool kDense = !kSigmoid && !kNormalize;
  float z[kDense ? N : 1], top = 0.0f, inv = 0.0f;
  if constexpr (kDense) {
    load_row<G>(p, row, lane, z);
    inv = softmax_terms<G>(z, top);
  }
  const int e = lane < K ? __ldg(p.idx + at.t * K + lane) : -1;
  const bool chosen = e >= 0 && e < E;
  const float zk = chosen ? load(p, row + e) : 0.0f;
  const float dw = chosen ? p.scale * __ldg(p.dw + at.t * K + lane) : 0.0f;
  float u;
  if (kNormalize) {
    const float w = share<kSigmoid, G>(zk, chosen);
    u = w * (dw - group_sum<G>(w * dw));
  } else {
    u = dw * (kSigmoid ? sigmoid(zk) : exp_from(zk, top) * inv);
  }
  if (!chosen) u = 0.0f;
  float d = u;
  const unsigned same = __match_any_sync(kAll, chosen ? e + at.base * MOE_MAX_EXPERTS : -1 - lane - at.base);
  if (__any_sync(kAll, (same & (same - 1)) != 0)) {  // the same expert named twice counts twice
    d = 0.0f;
    for (int k = 0; k < K; ++k) {
      const float v = __shfl_sync(kAll, u, k, G);
      if ((same >> (at.base + k)) & 1) d += v;
    }
  }
  if (kSigmoid) d *= sigmoid(-zk);
  if constexpr (kDense) {
    const float all = group_sum<G>(u);
    d -= exp_from(zk, top) * inv * all;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at.here && i * G + lane < E) store(p, row + i * G + lane, -(z[i] * inv) * all);
  } else {
    for (int i = lane; at.here && i < E; i += G) store(p, row + i, 0.0f);
  }
  __syncwarp();  // the chosen ones' values come last
  if (chosen && at.here) store(p, row + e, d);
}

template <int G, int N>
cudaError_t launch_n(const RouterParams& p, bool sigmoid, bool normalize, bool backward, cudaStream_t stream) {
  void (*kernel)(const RouterParams);
  if (backward)
    kernel = sigmoid ? (normalize ? router_grad_kernel<G, N, true, true> : router_grad_kernel<G, N, true, false>)
                     : (normalize ? router_grad_kernel<G, N, false, true> : router_grad_kernel<G, N, false, false>);
  else if (!sigmoid)
    kernel = normalize ? router_kernel<G, N, false, true, false> : router_kernel<G, N, false, false, false>;
  else if (p.bias)
    kernel = normalize ? router_kernel<G, N, true, true, true> : router_kernel<G, N, true, false, true>;
  else
    kernel = normalize ? router_kernel<G, N, true, true, false> : router_kernel<G, N, true, false, false>;
  const int64_t tokens = kWarps * 32 / G;  // a block
  return launch_kernel(kernel, dim3(static_cast<unsigned>((p.T + tokens - 1) / tokens)), dim3(kWarps * 32), 0, stream,
                       true, p);
}

}  // namespace

// Up to 64 experts do not fill a warp: 8 or 16 lanes a token.  15503 tokens, 34 experts, 14
// chosen, with gradient: 18.4 us, a warp each 21.0; 16384 tokens, 64 experts, 6 chosen: 8.1 forward.
cudaError_t launch_router(const RouterParams& p, bool sigmoid, bool normalize, bool backward, cudaStream_t stream) {
  if (p.E <= 16 && p.K <= 8) return launch_n<8, 2>(p, sigmoid, normalize, backward, stream);
  if (p.E <= 64 && p.K <= 8) return launch_n<8, 8>(p, sigmoid, normalize, backward, stream);
  if (p.E <= 64) return launch_n<16, 4>(p, sigmoid, normalize, backward, stream);
  if (p.E <= 128) return launch_n<32, 4>(p, sigmoid, normalize, backward, stream);
  if (p.E <= 256) return launch_n<32, 8>(p, sigmoid, normalize, backward, stream);
  if (p.E <= 384) return launch_n<32, 12>(p, sigmoid, normalize, backward, stream);
  if (p.E <= 512) return launch_n<32, 16>(p, sigmoid, normalize, backward, stream);
  return launch_n<32, 32>(p, sigmoid, normalize, backward, stream);
}

}  // namespace moe
