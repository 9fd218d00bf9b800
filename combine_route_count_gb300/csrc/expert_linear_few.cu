// The products of expert_linear.cu for few rows: forward and input.
//
// Bound by memory: the weights are read once for a few rows, so what counts is to
// have every SM load from the start.  A tile of expert_linear.cu is 256 columns of
// out and all of the summed axis, 28 tiles of N = 7168: 28 SMs at work.  Here 128
// weight rows (input: columns) are the 128 rows of the matrix instruction and up
// to 32 rows of the expert its columns, and the summed axis is split over a
// cluster of up to 8 CTAs, whose sums are exchanged through distributed shared
// memory and added in rank order.  Two CTAs share an SM.
//
// A thread of the epilogue owns one column of out.  Operands, bounds of the summed
// axis and waits as in expert_linear.cu.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ffn_kernels.cuh"
#include "linear_math.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "train_kernels.cuh"

namespace moe {
namespace {

using namespace lin;

constexpr int kCols = 128, kBlockK = 64;  // columns of out a CTA, summed axis a stage
constexpr int kRows = kFewLinearRows;     // rows of an expert a CTA
constexpr int kWBytes = kCols * kBlockK * 2, kABytes = kRows * kBlockK * 2;
constexpr int kChunkBytes = 64 * kBlockK * 2;  // a box of 64 x 64
constexpr int kMaxStages = 8;
constexpr int kThreads = 192;  // warps 0-3: epilogue
constexpr int kTmaWarp = 4, kMmaWarp = 5;
constexpr int kMaxRanks = 8;
constexpr int kPitch = kCols + 4;  // floats from one row's sums to the next
static_assert(MOE_MAX_EXPERTS * sizeof(int2) <= kWBytes, "the table of the experts' rows fits in a stage");

__host__ __device__ constexpr int stage_bytes(bool two) { return (two ? 2 : 1) * kWBytes + kABytes; }
__host__ __device__ constexpr int stage_count(bool two) { return two ? 3 : 5; }

// Four neighbouring columns.
struct Four {
  float v[4];
  __device__ __forceinline__ explicit Four(float a) : v{a, a, a, a} {}
  __device__ __forceinline__ explicit Four(float4 q) : v{q.x, q.y, q.z, q.w} {}
  static __device__ __forceinline__ Four f32(const void* p, int64_t i) {
    return Four(*reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
  }
  static __device__ __forceinline__ Four bf16(const void* p, int64_t i) {
    const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    return Four(make_float4(bf_lo(q.x), bf_hi(q.x), bf_lo(q.y), bf_hi(q.y)));
  }
  __device__ __forceinline__ void store_bf16(void* p, int64_t i) const {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
  }
  __device__ __forceinline__ Four operator+(const Four& o) const {
    return Four(make_float4(v[0] + o.v[0], v[1] + o.v[1], v[2] + o.v[2], v[3] + o.v[3]));
  }
};

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full;
  uint32_t tmem;
  int gave_up;
  int unit[3];  // expert, first row, rows
};

// kGate: forward with MOE_ACT_SWIGLU, gate and up columns side by side.
template <bool kInput, bool kGate>
__global__ void __launch_bounds__(kThreads, 2) few_linear_kernel(const __grid_constant__ LinearParams p, int ranks) {
  constexpr int kStages = stage_count(kGate), kStageBytes = stage_bytes(kGate);
  constexpr uint32_t kTmemColumns = kGate ? 2 * kRows : kRows;
  extern __shared__ uint8_t s_raw[];
  __shared__ Shared s;
  uint8_t* stages = s_raw + ((1024 - (ptx::smem_addr(s_raw) & 1023)) & 1023);
  float* sums = reinterpret_cast<float*>(stages);  // [gate, up][row][column], when the stages are done with
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = ranks > 1 ? static_cast<int>(tc::cluster_rank()) : 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&s.full[i], 1);
      ptx::mbar_init(&s.empty[i], 1);
    }
    ptx::mbar_init(&s.acc_full, 1);
    ptx::mbar_fence_init();
    s.gave_up = 0;
  }
  if (warp == kMmaWarp) tc::tmem_alloc(&s.tmem, kTmemColumns);
  if (threadIdx.x == kTmaWarp * 32) {
    tc::tma_prefetch_map(&p.a);
    tc::tma_prefetch_map(&p.b);
  }
  ptx::wait_prerequisites();
  ptx::launch_dependents();
  // Unit (expert, 32 of its rows) number u: the experts' rows are counted off until it is reached.
  const unsigned cluster = blockIdx.x / ranks;
  const int tile = static_cast<int>(cluster % p.n_tiles), u = static_cast<int>(cluster / p.n_tiles);
  // (The table lies where the first stage will: the threads that use it say so to the loads.)
  int2* table = reinterpret_cast<int2*>(stages);
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    const int rows = static_cast<int>(p.rows);
    int2 r = make_int2(0, rows);
    if (p.offsets) {  // clamped: a damaged table cannot lead outside the buffers
      r.x = min(max(p.offsets[e], 0), rows);
      r.y = min(max(p.offsets[e + 1], r.x), rows);
    }
    table[e] = r;
  }
  __syncthreads();
  if (warp == 0) {
    int e_found = -1, lo_found = 0, hi_found = 0, before = 0;
    for (int e0 = 0; e0 < p.E && e_found < 0; e0 += 32) {
      const int2 r = e0 + lane < p.E ? table[e0 + lane] : make_int2(0, 0);
      const int own = (r.y - r.x + kRows - 1) / kRows;
      int sum = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += up;
      }
      const int first = before + sum - own;
      const unsigned here = __ballot_sync(0xffffffffu, u >= first && u < first + own);
      if (here) {
        const int from = __ffs(here) - 1;
        e_found = e0 + from;
        lo_found = __shfl_sync(0xffffffffu, r.x + (u - first) * kRows, from);
        hi_found = __shfl_sync(0xffffffffu, r.y, from);
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) {
      s.unit[0] = e_found;
      s.unit[1] = lo_found;
      s.unit[2] = min(kRows, hi_found - lo_found);
    }
  }
  tc::fence_async_shared();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const int e = s.unit[0], row0 = s.unit[1], rows = s.unit[2];
  const uint32_t tmem = s.tmem, tmem_u = __shfl_sync(0xffffffffu, tmem, 0);
  // This rank's part of the summed axis (the same in every CTA of the cluster whether there is a unit).
  const int kblocks = (p.kc + kBlockK - 1) / kBlockK;
  const int kb0 = static_cast<int>(static_cast<int64_t>(kblocks) * rank / ranks);
  const int kb1 = static_cast<int>(static_cast<int64_t>(kblocks) * (rank + 1) / ranks);
  const int col0 = tile * kCols;

  if (e >= 0) {
    if (warp == kTmaWarp) {
      bool ok = true;
      int it = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int st = it % kStages;
        ok = it < kStages || tc::wait(&s.empty[st], (it / kStages - 1) & 1, &s.gave_up);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint8_t *w = stages + st * kStageBytes, *a = w + kStageBytes - kABytes;
        if (tc::elect() && static_cast<uint32_t>(it) != p.test_drop) {
          ptx::mbar_arrive_expect_tx(&s.full[st], kStageBytes);
          const uint32_t bar = ptx::smem_addr(&s.full[st]);
          const int k = kb * kBlockK;
          if (kInput) {
            tc::tma_load_3d(w, &p.b, col0, k, e, bar);
            tc::tma_load_3d(w + kChunkBytes, &p.b, col0 + 64, k, e, bar);
          } else {
            tc::tma_load_3d(w, &p.b, k, col0, e, bar);
            if (kGate) tc::tma_load_3d(w + kWBytes, &p.b, k, p.N + col0, e, bar);
          }
          tc::tma_load_2d(a, &p.a, k, row0, bar);
        }
        __syncwarp();
      }
      // Loads in flight write to this CTA's shared memory: it does not end before them.
      const unsigned long long start = tc::now_ns();
      for (int j = it > kStages ? it - kStages : 0; j < it; ++j)
        if (static_cast<uint32_t>(j) != p.test_drop) tc::settle(&s.full[j % kStages], (j / kStages) & 1, start);
    } else if (warp == kMmaWarp) {
      constexpr uint32_t kInstr = tc::instr_desc_bf16(kCols, kRows, kInput, false);
      constexpr uint64_t kStepW = (kInput ? 2048 : 32) >> 4;
      bool ok = true;
      int it = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int st = it % kStages;
        ok = tc::wait(&s.full[st], (it / kStages) & 1, &s.gave_up);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc::fence_after();
        const uint8_t* w_tile = stages + st * kStageBytes;
        const uint64_t w = kInput ? tc::smem_desc_mn(w_tile) : tc::smem_desc(w_tile);
        const uint64_t up = tc::smem_desc(w_tile + kWBytes);
        const uint64_t a = tc::smem_desc(w_tile + kStageBytes - kABytes);
        if (tc::elect()) {
#pragma unroll
          for (int k = 0; k < kBlockK / 16; ++k) {
            tc::mma_f16(tmem_u, w + kStepW * k, a + 2 * k, kInstr, kb > kb0 || k > 0);
            if (kGate) tc::mma_f16(tmem_u + kRows, up + kStepW * k, a + 2 * k, kInstr, kb > kb0 || k > 0);
          }
          tc::commit(&s.empty[st]);
        }
        __syncwarp();
      }
      // Also where a wait gave up: nothing may be in flight when the CTA ends.
      if (tc::elect()) tc::commit(&s.acc_full);
      __syncwarp();
      tc::settle(&s.acc_full, 0, tc::now_ns());
    }
  }
  __syncthreads();
  // Every load and product of this CTA is over.
  tc::fence_after();
  constexpr int kSums = kGate ? 2 : 1;
  if (e >= 0 && warp < 4) {
    float v[kSums][kRows];
#pragma unroll
    for (int h = 0; h < kSums; ++h)
      tc::tmem_load_32(tmem + (static_cast<uint32_t>(warp * 32) << 16) + h * kRows, reinterpret_cast<uint32_t*>(v[h]));
    tc::wait_loads();
#pragma unroll
    for (int h = 0; h < kSums; ++h)
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        if (r < rows) sums[(h * kRows + r) * kPitch + threadIdx.x] = v[h][r];
  }
  tc::fence_before();
  if (ranks > 1) tc::cluster_sync();
  else __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::tmem_free(tmem, kTmemColumns);
  if (threadIdx.x == 0 && s.gave_up && p.status) atomicCAS(p.status, MOE_OK, MOE_ETIMEDOUT);

  if (e >= 0) {
    // A rank's share: 128 / ranks columns of every row, four at a time; what else they need
    // is on its way while the sums are read.  (One loop for all: 32 rows unrolled were more
    // code than the instruction cache takes, 4 us.  us, N 7168, K 2048, one token with bias
    // and residual, and 32 rows: four columns one after the other 9.6, 12.7; one column at a
    // time 9.0, 14.7; so 8.9, 11.6.)
    const int quads = kCols / ranks / 4;
    const int64_t wide = p.N;
    const bool halves = kGate || (kInput && p.act == MOE_ACT_SWIGLU);
#pragma unroll 1
    for (int i = threadIdx.x; i < quads * rows; i += kThreads) {
      const int r = i / quads, c = rank * (kCols / ranks) + i % quads * 4, col = col0 + c;
      if (col >= p.N) continue;  // N is a multiple of 8
      const int64_t row = row0 + r, at = row * wide + col;
      const int64_t at_pre = halves ? row * 2 * wide + col : at;
      const Four none(0.0f);
      Four b0 = none, b1 = none, more = none, pre0 = none, pre1 = none;
      if (kInput) {
        if (p.pre) pre0 = Four::bf16(p.pre, at_pre);
        if (halves) pre1 = Four::bf16(p.pre, at_pre + wide);
      } else {
        const int64_t b = static_cast<int64_t>(e) * p.bias_cols + col;
        if (p.bias) b0 = p.bias_f32 ? Four::f32(p.bias, b) : Four::bf16(p.bias, b);
        if (kGate && p.bias) b1 = p.bias_f32 ? Four::f32(p.bias, b + p.N) : Four::bf16(p.bias, b + p.N);
        if (p.residual) more = Four::bf16(p.residual, at);
      }
      Four x = none, y = none;
#pragma unroll
      for (int h = 0; h < kSums; ++h) {
        const float* from = sums + (h * kRows + r) * kPitch + c;
        float4 v[kMaxRanks];
#pragma unroll
        for (int q = 0; q < kMaxRanks; ++q)
          if (q < ranks) v[q] = ranks > 1 ? tc::ld_cluster_v4(tc::at_rank(from, q)) : *reinterpret_cast<const float4*>(from);
        Four& to = h ? y : x;
#pragma unroll
        for (int q = 0; q < kMaxRanks; ++q)
          if (q < ranks) to = q ? to + Four(v[q]) : Four(v[0]);
      }
      if (kInput) {
        if (halves) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            Two gate(pre0.v[2 * j], pre0.v[2 * j + 1]), up(pre1.v[2 * j], pre1.v[2 * j + 1]);
            swiglu_through(Two(x.v[2 * j], x.v[2 * j + 1]), gate, up);
            x.v[2 * j] = gate.lo(), x.v[2 * j + 1] = gate.hi();
            y.v[2 * j] = up.lo(), y.v[2 * j + 1] = up.hi();
          }
          y.store_bf16(p.out, at_pre + wide);
        } else if (p.act != MOE_ACT_NONE) {
#pragma unroll
          for (int j = 0; j < 4; ++j) x.v[j] = act_through(p.act, x.v[j], pre0.v[j]);
        }
        x.store_bf16(p.out, at_pre);
        continue;
      }
      if (p.bias) {
        x = x + b0;
        y = y + b1;
      }
      if (p.pre) {
        x.store_bf16(p.pre, at_pre);
        if (kGate) y.store_bf16(p.pre, at_pre + wide);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) x.v[j] = kGate ? silu(x.v[j]) * y.v[j] : act_value(p.act, x.v[j]);
      if (p.residual) x = x + more;
      if (p.out_f32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(x.v[0], x.v[1], x.v[2], x.v[3]);
      else x.store_bf16(p.out, at);
    }
  }
  if (ranks > 1) tc::cluster_sync();  // no CTA leaves while its shared memory is being read
}

template <bool kInput, bool kGate>
cudaError_t launch(const LinearParams& p, int ranks, cudaStream_t stream) {
  const size_t smem = 1024 + static_cast<size_t>(stage_count(kGate)) * stage_bytes(kGate);
  auto* kernel = few_linear_kernel<kInput, kGate>;
  cudaError_t err = set_kernel_limits(reinterpret_cast<const void*>(kernel), smem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(few_linear_units(p.rows, p.offsets ? p.E : 0) * p.n_tiles * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ranks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, ranks);
}

}  // namespace

cudaError_t launch_few_linear(const LinearParams& p, bool input, bool gate, int ranks, cudaStream_t stream) {
  if (input) return launch<true, false>(p, ranks, stream);
  return gate ? launch<false, true>(p, ranks, stream) : launch<false, false>(p, ranks, stream);
}

}  // namespace moe
