// The experts' products on grouped rows, block-scaled E4M3 operands, on the
// 5th-generation tensor core:
//
//   P[i, n] = sum_b sa[i, b] * sw[e, n / 128, b] * sum_{k in block b} a[i, k] * w[e, n, k]
//
// for every row i of expert e (rows [offsets[e], offsets[e+1])), blocks b of
// 128 along K.  Two epilogues: P itself as bf16 or float32 rows
// (moe_expert_gemm_fp8), and, with w's rows the gate rows followed by the up
// rows, h = SiLU(P_gate) * P_up quantised again by blocks of 128
// (moe_expert_glu_fp8).
//
// The scales differ from block to block of K, so a block's product cannot be
// left to accumulate in tensor memory: each block of K = 128 (four matrix
// instructions) goes to a tensor-memory buffer of its own, and the epilogue
// warps add it, scaled, to float32 accumulators in registers while the tensor
// core fills other buffers.
//
// One CTA per SM, tile 128 rows x 256 columns (glu: 128 gate + 128 up columns,
// 128 columns of h), 12 warps: two epilogue groups of four, each with half of
// the columns (glu: 64 gate columns and their up columns), one TMA warp, one
// matrix warp, two that only fill their group.  A thread of the epilogue owns
// one row and 128 columns, added two at a time.  Operands arrive by tiled TMA
// into kStages stages of 48 KiB with the 128-byte swizzle that the matrix
// instruction reads.  Rows past the end of an expert and columns past N are
// computed and not stored: rows and columns do not mix.
//
// What bounds large products is the way of a buffer: from the last matrix
// instruction over a barrier to the epilogue, out of tensor memory, and over a
// barrier back takes 700 to 1000 cycles, 128 x 256 x 128 of matrix work 512.
// With two buffers of 256 columns a K block took 1190 cycles.  So each half of
// the columns has its own two buffers of 128, and four are on their way at a
// time: on zeros, at 2070 MHz and in 8 whole rounds of tiles, 660 cycles a K block
// up to K = 1024, 720 to 2048 and 740 to 780 beyond, and about 4700 a tile beside
// them (its end, and its share of the launch).  8192 rows, N 7168, K 4096: 164 us
// on zeros (2.93 PFLOP/s); on random values 179 us in bursts of 20 calls and 199
// to 204 call after call, where the power limit holds the SMs at 1690 MHz: 164 us
// at that clock are 201.  So at the full clock the buffers' way is the bound,
// and in a long run the power.  Leaving out half of the operand loads changed
// neither.
//
// Tiles are dealt out statically (tile b, b+G, ...), rows fastest, so that the
// CTAs at work at one time share weight columns in L2.  Waits are bounded (2 s)
// and report MOE_ETIMEDOUT.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ffn_kernels.cuh"
#include "fp8_quant.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

constexpr int kTileM = 128, kTileN = 256, kBlockK = MOE_FP8_BLOCK;
constexpr int kStages = 4;
constexpr int kABytes = kTileM * kBlockK, kBBytes = kTileN * kBlockK;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kEpilogueWarps = 8;
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 384;
// Registers a thread: 168 at launch (65536 / 384), of which the last group gives
// up what the epilogue's two take: 256 * 216 + 128 * 72 = 384 * 168.
constexpr int kRegsEpilogue = 216, kRegsRest = 72;
constexpr uint32_t kTmemColumns = 512;
constexpr int kCols = 128;  // accumulators of one epilogue thread

struct Shared {
  uint64_t full[kStages], empty[kStages];
  uint64_t acc_full[2][2], acc_empty[2][2];  // [half of the columns][buffer]
  uint64_t amax_ready[2];
  uint64_t drained;
  uint32_t tmem;
  int gave_up;
  float amax[2][2][kTileM];  // [tile parity][half of the columns][row]
};

// Per expert: where its rows begin and end, and how many row tiles come before it.
struct Groups {
  int32_t *lo, *hi, *start;
};

struct Tile {
  int e, row0, rows, n;  // expert, first row, rows of the tile that exist, column tile
};

__device__ __forceinline__ Tile find_tile(const Groups& g, int E, int n_tiles, int64_t t) {
  int lo = 0, hi = E;  // largest e with start[e] * n_tiles <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (static_cast<int64_t>(g.start[mid]) * n_tiles <= t) lo = mid;
    else hi = mid;
  }
  const int m_tiles = g.start[lo + 1] - g.start[lo];
  const int local = static_cast<int>(t - static_cast<int64_t>(g.start[lo]) * n_tiles);
  Tile r;
  r.e = lo;
  r.n = local / m_tiles;
  r.row0 = g.lo[lo] + (local - r.n * m_tiles) * kTileM;
  r.rows = min(kTileM, g.hi[lo] - r.row0);
  return r;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Lane i of four holds units u[0..3] of row i; after it, unit i of rows 0..3.
template <int kWords>
__device__ __forceinline__ void transpose_4(uint32_t (&u)[4][kWords], int lane) {
#pragma unroll
  for (int d = 1; d < 4; d *= 2) {
    const bool upper = lane & d;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & d) continue;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? u[j][i] : u[j + d][i], d);
        u[j][i] = upper ? got : u[j][i];
        u[j + d][i] = upper ? u[j + d][i] : got;
      }
    }
  }
}

template <bool kGlu, bool kF32>
__global__ void __launch_bounds__(kThreads, 1) expert_gemm_kernel(const __grid_constant__ ExpertGemmParams p) {
  extern __shared__ uint8_t s_raw[];
  __shared__ Shared s;
  uint8_t* stages = s_raw + ((1024 - (ptx::smem_addr(s_raw) & 1023)) & 1023);
  Groups g;
  g.lo = reinterpret_cast<int32_t*>(stages + kStages * kStageBytes);
  g.hi = g.lo + p.E;
  g.start = g.hi + p.E;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&s.full[i], 1);
      ptx::mbar_init(&s.empty[i], 2);  // both matrix warps
    }
    for (int i = 0; i < 2; ++i) {
      for (int h = 0; h < 2; ++h) {
        ptx::mbar_init(&s.acc_full[h][i], 1);
        ptx::mbar_init(&s.acc_empty[h][i], kEpilogueWarps / 2);
      }
      ptx::mbar_init(&s.amax_ready[i], kEpilogueWarps);
    }
    ptx::mbar_init(&s.drained, 2);
    ptx::mbar_fence_init();
    s.gave_up = 0;
  }
  if (warp == kMmaWarp) tc::tmem_alloc(&s.tmem, kTmemColumns);
  if (threadIdx.x == kTmaWarp * 32) {
    tc::tma_prefetch_map(&p.a);
    tc::tma_prefetch_map(&p.w);
  }
  ptx::wait_prerequisites();
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    const int rows = static_cast<int>(p.rows);
    int lo = 0, hi = rows;
    if (p.offsets) {  // clamped: a damaged table cannot lead outside the buffers
      lo = min(max(p.offsets[e], 0), rows);
      hi = min(max(p.offsets[e + 1], lo), rows);
    }
    g.lo[e] = lo;
    g.hi[e] = hi;
  }
  __syncthreads();
  if (warp == 0) {
    int before = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const int own = e < p.E ? (g.hi[e] - g.lo[e] + kTileM - 1) / kTileM : 0;
      int sum = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += up;
      }
      if (e < p.E) g.start[e] = before + sum - own;
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) g.start[p.E] = before;
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const int64_t tiles = static_cast<int64_t>(g.start[p.E]) * p.n_tiles;
  const uint32_t tmem = s.tmem, tmem_u = __shfl_sync(0xffffffffu, tmem, 0);
  const int kblocks = p.kblocks;

  if (warp >= kEpilogueWarps) {
    tc::fewer_registers<kRegsRest>();
    if (warp == kTmaWarp) {
      uint32_t it = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const Tile tile = find_tile(g, p.E, p.n_tiles, t);
        const int w0 = tile.e * p.w_rows + tile.n * (kGlu ? kTileN / 2 : kTileN);
        for (int kb = 0; kb < kblocks; ++kb, ++it) {
          const int st = it % kStages;
          ok = it < kStages || tc::wait(&s.empty[st], (it / kStages - 1) & 1, &s.gave_up);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          uint8_t* a = stages + st * kStageBytes;
          if (tc::elect() && it != p.test_drop) {
            ptx::mbar_arrive_expect_tx(&s.full[st], kStageBytes);
            tc::tma_load_2d(a, &p.a, kb * kBlockK, tile.row0, &s.full[st]);
            // The first half of the columns, then the second; glu (boxes of 64
            // rows): 64 gate rows and their up rows each.
            uint8_t* b = a + kABytes;
            if (kGlu) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                tc::tma_load_2d(b + q * (kBBytes / 4), &p.w, kb * kBlockK, w0 + (q & 1) * p.N + (q >> 1) * 64,
                                &s.full[st]);
            } else {
              tc::tma_load_2d(b, &p.w, kb * kBlockK, w0, &s.full[st]);
              tc::tma_load_2d(b + kBBytes / 2, &p.w, kb * kBlockK, w0 + kTileN / 2, &s.full[st]);
            }
          }
          __syncwarp();
        }
      }
      // Loads in flight write to this CTA's shared memory: it does not end before
      // them, whichever warp gave up.
      const unsigned long long start = tc::now_ns();
      for (uint32_t j = it > kStages ? it - kStages : 0; j < it; ++j)
        if (j != p.test_drop) tc::settle(&s.full[j % kStages], (j / kStages) & 1, start);
    }
    if (warp == kMmaWarp || warp == kMmaWarp + 1) {
      constexpr uint32_t kInstr = tc::instr_desc_e4m3(kTileM, kTileN / 2);
      const int h = warp - kMmaWarp;
      uint32_t it = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        for (int kb = 0; kb < kblocks; ++kb, ++it) {
          const int st = it % kStages, buf = it & 1;
          ok = (it < 2 || tc::wait(&s.acc_empty[h][buf], (it / 2 - 1) & 1, &s.gave_up)) &&
               tc::wait(&s.full[st], (it / kStages) & 1, &s.gave_up);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc::fence_after();
          const uint64_t a = tc::smem_desc(stages + st * kStageBytes);
          const uint64_t b = tc::smem_desc(stages + st * kStageBytes + kABytes + h * (kBBytes / 2));
          if (tc::elect()) {
#pragma unroll
            for (int k = 0; k < kBlockK / 32; ++k)
              tc::mma_e4m3(tmem_u + h * kTileN + buf * kCols, a + 2 * k, b + 2 * k, kInstr, k > 0);
            tc::commit(&s.acc_full[h][buf]);
            tc::commit(&s.empty[st]);
          }
          __syncwarp();
        }
      }
      // Nothing may be in flight when the tensor memory is freed.
      if (tc::elect()) tc::commit(&s.drained);
      __syncwarp();
      tc::settle(&s.drained, 0, tc::now_ns());
    }
  } else {
    tc::more_registers<kRegsEpilogue>();
    const int half = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    uint32_t it = 0;
    int parity = 0, round = 0;
    bool ok = true;
    // Rows that begin on 32-byte boundaries are stored by whole sectors, four
    // lanes side by side.  (A lane a row: 32 lines an instruction, and the
    // experts' second products, 128 rows each, take 870 us instead of 765.)
    const bool wide = ((reinterpret_cast<uintptr_t>(p.out) | static_cast<uintptr_t>(p.N) * (kF32 ? 4 : 2)) & 31) == 0;
    for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++round) {
      const Tile tile = find_tile(g, p.E, p.n_tiles, t);
      const bool act = r < tile.rows;
      const int64_t row = tile.row0 + (act ? r : 0);
      const float* sa = p.a_scales + row * kblocks;
      // The block rows of w's scales that this thread's columns lie in.
      const float* sw = p.w_scales + static_cast<int64_t>(tile.e) * p.w_blocks * kblocks;
      const float *sw0, *sw1;
      if (kGlu) {
        sw0 = sw + static_cast<int64_t>(tile.n) * kblocks;
        sw1 = sw0 + static_cast<int64_t>(p.N / kBlockK) * kblocks;
      } else {
        sw0 = sw1 = sw + static_cast<int64_t>(min(tile.n * 2 + half, p.w_blocks - 1)) * kblocks;
      }
      unsigned long long acc[kCols / 2];
#pragma unroll
      for (int j = 0; j < kCols / 2; ++j) acc[j] = 0;
      // A warp none of whose rows exist only passes the buffers on.
      const bool some = (warp & 3) * 32 < tile.rows;
      float next_a = *sa, next_0 = *sw0, next_1 = kGlu ? *sw1 : 0.0f;  // scales, a block ahead
      for (int kb = 0; kb < kblocks; ++kb, ++it) {
        const float f0 = next_a * next_0, f1 = kGlu ? next_a * next_1 : f0;
        const unsigned long long scale0 = tc::pack2(f0, f0), scale1 = tc::pack2(f1, f1);
        if (kb + 1 < kblocks) {
          next_a = *++sa;
          next_0 = *++sw0;
          if (kGlu) next_1 = *++sw1;
        }
        const int buf = it & 1;
        ok = tc::wait(&s.acc_full[half][buf], (it / 2) & 1, &s.gave_up);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc::fence_after();
        if (some) {
          const uint32_t from = lanes + half * kTileN + buf * kCols;
          uint32_t v[2][32];
          tc::tmem_load_32(from, v[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tc::wait_loads();
            if (c < 3) {
              tc::tmem_load_32(from + (c + 1) * 32, v[(c + 1) & 1]);
            } else {
              tc::fence_before();
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(&s.acc_empty[half][buf]);
            }
            const uint32_t* d = v[c & 1];
#pragma unroll
            for (int j = 0; j < 16; ++j)
              acc[c * 16 + j] = tc::fma2(tc::pack2(__uint_as_float(d[2 * j]), __uint_as_float(d[2 * j + 1])),
                                         c < 2 ? scale0 : scale1, acc[c * 16 + j]);
          }
        } else {
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&s.acc_empty[half][buf]);
        }
      }
      if (!ok) break;
      if (kGlu) {
        float h[kCols / 2];
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < kCols / 2; ++j) {
          const float gate = j & 1 ? tc::hi2(acc[j / 2]) : tc::lo2(acc[j / 2]);
          const float up = j & 1 ? tc::hi2(acc[kCols / 4 + j / 2]) : tc::lo2(acc[kCols / 4 + j / 2]);
          // Of a denominator beyond 2^126 the quotient becomes 0; it is below 2^-119 there.
          h[j] = __fdividef(gate, 1.0f + expf(-gate)) * up;
          amax = fmaxf(amax, fabsf(h[j]));
        }
        // The other half of the row's 128 columns is another warp's.  The two
        // copies alternate, so a warp one tile ahead does not overwrite.
        parity = round & 1;
        s.amax[parity][half][r] = amax;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&s.amax_ready[parity]);
        ok = tc::wait(&s.amax_ready[parity], (round >> 1) & 1, &s.gave_up);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        amax = fmaxf(amax, s.amax[parity][half ^ 1][r]);
        const float scale = amax > 0.0f ? __fdiv_rn(fmaxf(amax, kTinyAmax), 448.0f) : 1.0f;
        const float inv = __fdiv_rn(1.0f, scale);
        // Four lanes store 64 bytes of a row together.
        uint32_t u[4][4];
#pragma unroll
        for (int c = 0; c < kCols / 2; c += 4)
          u[c / 16][c / 4 & 3] = fp8q::e4m3x2(__fmul_rn(h[c], inv), __fmul_rn(h[c + 1], inv)) |
                                 (fp8q::e4m3x2(__fmul_rn(h[c + 2], inv), __fmul_rn(h[c + 3], inv)) << 16);
        transpose_4(u, lane);
        const int r0 = r & ~3;
        uint8_t* dst = static_cast<uint8_t*>(p.out) + static_cast<int64_t>(tile.row0 + r0) * p.N + tile.n * kBlockK +
                       half * (kCols / 2) + (lane & 3) * 16;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (r0 + k < tile.rows)
            ptx::st_v4(dst + static_cast<int64_t>(k) * p.N, make_uint4(u[k][0], u[k][1], u[k][2], u[k][3]));
        if (act && half == 0) p.h_scales[row * (p.N / kBlockK) + tile.n] = scale;
      } else if (some) {
        // Four lanes store 128 bytes of a row together, 32 each.
        constexpr int kStep = kF32 ? 8 : 16;  // columns of 32 bytes
        const int n0 = tile.n * kTileN + half * kCols + (lane & 3) * kStep, r0 = r & ~3;
        const int64_t stride = static_cast<int64_t>(p.N) * (kF32 ? 4 : 2);
        uint8_t* dst = static_cast<uint8_t*>(p.out) + (tile.row0 + r0) * stride + static_cast<int64_t>(n0) * (kF32 ? 4 : 2);
#pragma unroll
        for (int c = 0; c < kCols; c += 4 * kStep) {
          uint32_t u[4][8];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (kF32) u[i / 8][i & 7] = static_cast<uint32_t>(acc[(c + i) / 2] >> (i & 1 ? 32 : 0));
            else u[i / 8][i & 7] = bf16x2(tc::lo2(acc[c / 2 + i]), tc::hi2(acc[c / 2 + i]));
          }
          transpose_4(u, lane);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint8_t* to = dst + k * stride + c * (kF32 ? 4 : 2);
            const uint4 q0 = make_uint4(u[k][0], u[k][1], u[k][2], u[k][3]);
            const uint4 q1 = make_uint4(u[k][4], u[k][5], u[k][6], u[k][7]);
            if (r0 + k < tile.rows) {
              if (wide && n0 + c + kStep <= p.N) {
                tc::st_v8(to, q0, q1);
              } else {  // N is a multiple of 8
                if (n0 + c < p.N) ptx::st_v4(to, q0);
                if (n0 + c + kStep / 2 < p.N) ptx::st_v4(to + 16, q1);
              }
            }
          }
        }
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (threadIdx.x == 0 && s.gave_up && p.status) atomicCAS(p.status, MOE_OK, MOE_ETIMEDOUT);
  if (warp == kMmaWarp) tc::tmem_free(tmem, kTmemColumns);
}

template <bool kGlu, bool kF32>
cudaError_t launch(const ExpertGemmParams& p, int sms, cudaStream_t stream) {
  const size_t smem = 1024 + kStages * kStageBytes + (3 * static_cast<size_t>(p.E) + 1) * sizeof(int32_t);
  auto* kernel = expert_gemm_kernel<kGlu, kF32>;
  cudaError_t err = set_kernel_limits(reinterpret_cast<const void*>(kernel), smem);
  if (err != cudaSuccess) return err;
  // Every expert may add one partly filled row tile.
  int64_t most = ((p.rows + kTileM - 1) / kTileM + (p.offsets ? p.E : 0)) * p.n_tiles;
  if (most > sms) most = sms;
  return launch_kernel(kernel, dim3(static_cast<unsigned>(most)), dim3(kThreads), smem, stream, true, p);
}

}  // namespace

int expert_gemm_n_tile(bool glu) { return glu ? kTileN / 2 : kTileN; }

cudaError_t launch_expert_gemm(const ExpertGemmParams& p, bool glu, bool f32, int sms, cudaStream_t stream) {
  if (glu) return launch<true, false>(p, sms, stream);
  return f32 ? launch<false, true>(p, sms, stream) : launch<false, false>(p, sms, stream);
}

}  // namespace moe
