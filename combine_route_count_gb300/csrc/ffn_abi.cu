// The C ABI of the feed-forward operators (declared in include/moe_ffn.h):
// argument checks and launches.  Exceptions do not cross it: what can throw
// in the host code below is the allocation of a per-device cache entry.

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "ffn_kernels.cuh"
#include "moe_ffn.h"

namespace {

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// SM count of the current device, asked once per device (0: the query failed).
int sm_count() {
  static int known[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) {
    const int n = __atomic_load_n(&known[dev], __ATOMIC_RELAXED);
    if (n > 0) return n;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) __atomic_store_n(&known[dev], n, __ATOMIC_RELAXED);
  return n;
}

template <class F>
int guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return MOE_ECUDA;
  }
}

int launched(cudaError_t err) {
  if (err == cudaSuccess) return MOE_OK;
  cudaGetLastError();  // a refused launch is reported here, not by a later call
  return MOE_ECUDA;
}

}  // namespace

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
