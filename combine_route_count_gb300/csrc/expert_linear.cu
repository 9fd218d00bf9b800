// The bf16 products of an expert layer and their gradients, on the 5th-generation
// tensor core.  Three products of one shape, out = A x B summed over kc:
//
//              out [rows of a tile, columns]      summed over        A          B
//   forward    [rows of expert e, N]              K                  a          w[e]
//   input      [rows of expert e, K]              N                  dy         w[e], by its other axis
//   weight     [N, K] of expert e                 rows of expert e   dy, a: both by their other axis
//
// "By its other axis": the axis that is summed over is not the contiguous one.  The
// matrix instruction takes such operands as they lie (MN-major): TMA boxes of 64
// columns x 64 summed rows, no transposition anywhere.
//
// One CTA per SM, tile 128 x 256, 64 of the summed axis a stage, 4 stages of 48
// KiB by tiled TMA (128-byte swizzle).  With many rows an expert two CTAs (a cluster)
// share a tile of 256 x 256: one issues the products of both (cta_group::2), each
// holds half of either operand, 6 stages of 32 KiB, so that a product of 256 x 256 x 64
// takes 64 KiB out of L2 instead of 96.  Where there are few tiles, they have 128 columns
// and 6 stages of 32 KiB; where the summed axis is long as well,
// up to 8 CTAs (a cluster) split the axis of one tile, read one another's sums through
// distributed shared memory and each finish a part of the tile.  12 warps: eight for the epilogue (two
// groups of four, each with half of the columns), one for TMA, one for the matrix
// instructions, two for the bias gradient, which they sum from memory (from L2: the
// tiles read the same rows; 3 % more time than without).  A tile's sum stays in tensor memory:
// two buffers of 256 columns, so that one tile's epilogue runs under the next
// one's products.
//
// Rows past the end of an expert and columns past the last are computed and not
// stored.  What is summed over must end exactly: past the end of K or N the tensor
// maps give zeros (w is a map of three dimensions, so that they end with the
// expert); rows past the end of an expert belong to the next one, and the matrix
// warp overwrites them with zeros in the last stage.
//
// What bounds it: at many rows the tensor cores.  8192 rows, N = K = 4096: forward 143
// us, 1923 TFLOP/s, what a library's plain product takes in a burst (single CTAs 162);
// by rows 142, by weights 157.  Call after call the power limit holds the SMs at 1350 to
// 1700 MHz, and these times grow by a tenth to a fifth.  At few rows an expert the bytes
// of the weights.
//
// Tiles are dealt out statically (tile b, b+G, ...).  Waits are bounded (2 s) and
// report MOE_ETIMEDOUT.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <map>
#include <mutex>
#include <utility>

#include "ffn_kernels.cuh"
#include "linear_math.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "train_kernels.cuh"

namespace moe {
namespace {

using namespace lin;

enum Mode { kForward, kInput, kWeight };
// Who works on a tile: one CTA (on half as many columns: kNarrow), a pair of them, or
// several that split the summed axis.
enum Team { kAlone, kNarrow, kPairs, kSplit };

constexpr int kTileM = 128, kBlockK = 64;  // kTileM: rows of one CTA
__host__ __device__ constexpr int tile_n(Team team) { return team == kNarrow ? 128 : 256; }
constexpr int kABytes = kTileM * kBlockK * 2;
constexpr int kChunkBytes = 64 * kBlockK * 2;  // a box of 64 x 64
// Of one CTA: alone it holds all of B's columns, in a pair half of them.
__host__ __device__ constexpr int b_columns(Team team) { return team == kPairs ? tile_n(team) / 2 : tile_n(team); }
__host__ __device__ constexpr int stage_bytes(Team team) { return kABytes + b_columns(team) * kBlockK * 2; }
__host__ __device__ constexpr int stage_count(Team team) { return b_columns(team) == 128 ? 6 : 4; }
constexpr int kMaxStages = 6;
constexpr int kEpilogueWarps = 8;
constexpr int kTmaWarp = 8, kMmaWarp = 9, kBiasWarp = 10;
constexpr int kThreads = 384;
constexpr int kLoads = 24;  // of a lane of the bias warps on their way: under load one takes microseconds
constexpr uint32_t kTmemColumns = 512;
constexpr int kUnit = 64;  // columns that an epilogue warp works on at a time
constexpr int kMaxSplit = 8;
constexpr int kPitch = tile_n(kSplit) + 4;  // floats from one row's sums to the next, where they are split

struct Shared {
  alignas(16) float bias[kEpilogueWarps][2 * kUnit];  // of each epilogue warp's columns
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t tail_full[kMaxStages];  // pair, second CTA: its half of an expert's last stage is there
  uint64_t tail_clear[kMaxStages]; // pair, first CTA: and ends in zeros
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drained;
  uint32_t tmem;
  int gave_up;
};

// Per expert: where its rows begin and end, and how many row tiles come before it.
struct Groups {
  int32_t *lo, *hi, *start;
};

struct Tile {
  int e;
  int row0, rows;  // first row of out and how many exist (weight: of the expert's matrix)
  int n;           // column tile
  int k0, kc;      // the summed axis: where it begins, how long it is
};

// Tiles are counted in 32 bits (the host refuses calls with more).
template <Mode kMode>
__device__ __forceinline__ uint32_t tile_count(const Groups& g, const LinearParams& p) {
  if (kMode == kWeight) return static_cast<uint32_t>(p.E) * p.m_tiles * p.n_tiles;
  return static_cast<uint32_t>(g.start[p.E]) * p.n_tiles;
}

// Row tile (returned) and column tile of an expert's tile number t.  Bands of 2048
// rows, inside a band rows fastest: the tiles at work at one time cover about as many
// rows as columns, which share the operands in L2.  (All of 8192 rows first: 203 us
// instead of 153 for the gradient by rows, N = K = 4096, whose weights were then read in
// strips of a few hundred bytes.)  The gradient by weights has its bands along the
// columns, so that whole rows of dw are written at a time: 170 us / 157 with N = K = 4096,
// 440 / 370 where the writes are all (256 experts of 128 rows, N = K = 2048).
template <int kRows>
__device__ __forceinline__ int place(uint32_t t, uint32_t m_tiles, uint32_t n_tiles, int& n) {
  constexpr uint32_t kBand = 2048 / kRows;
  const uint32_t band = t / kBand / n_tiles;
  const uint32_t height = min(kBand, m_tiles - band * kBand);
  const uint32_t in_band = t - band * kBand * n_tiles;
  const uint32_t column = height == kBand ? in_band / kBand : in_band / height;
  n = static_cast<int>(column);
  return static_cast<int>(band * kBand + in_band - column * height);
}

// What CTA `rank` of a pair has of tile t (rank 0: of a CTA alone).  Rows may be none.
template <Mode kMode, bool kPair, int kN>
__device__ __forceinline__ Tile find_tile(const Groups& g, const LinearParams& p, uint32_t t, int rank) {
  constexpr int kRows = kPair ? 2 * kTileM : kTileM;
  Tile r;
  if (kMode == kWeight) {
    const uint32_t per = static_cast<uint32_t>(p.m_tiles) * p.n_tiles;
    r.e = static_cast<int>(t / per);
    const uint32_t local = t - r.e * per;
    int m;
    r.n = place<kN>(local, p.n_tiles, p.m_tiles, m);  // bands of 2048 columns, columns fastest
    r.row0 = m * kRows + rank * kTileM;
    r.rows = min(kTileM, p.M - r.row0);
    r.k0 = g.lo[r.e];
    r.kc = g.hi[r.e] - r.k0;
    return r;
  }
  int lo = 0, hi = p.E;  // largest e with start[e] * n_tiles <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (static_cast<uint32_t>(g.start[mid]) * p.n_tiles <= t) lo = mid;
    else hi = mid;
  }
  const int m_tiles = g.start[lo + 1] - g.start[lo];
  const uint32_t local = t - static_cast<uint32_t>(g.start[lo]) * p.n_tiles;
  r.e = lo;
  r.row0 = g.lo[lo] + place<kRows>(local, m_tiles, p.n_tiles, r.n) * kRows + rank * kTileM;
  r.rows = min(kTileM, g.hi[lo] - r.row0);
  r.k0 = 0;
  r.kc = p.kc;
  return r;
}

// The tiles of a CTA one after the other, for a whole warp: every lane looks for one of
// the next 32, which are then handed round.  (Looked for one at a time: through 8
// experts' gate, N 4096, K 8192, 340 us instead of 334; 256 experts' dw, 381 instead of 369.)
template <Mode kMode, bool kPair, int kN>
struct Walk {
  uint32_t first, step, tiles;
  int rank;
  Tile mine;

  // Number i; i goes up by one from call to call, first + i * step < tiles.
  __device__ __forceinline__ Tile get(const Groups& g, const LinearParams& p, uint32_t i, int lane) {
    if (i % 32 == 0) mine = find_tile<kMode, kPair, kN>(g, p, min(first + (i + lane) * step, tiles - 1), rank);
    const int from = i % 32;
    Tile r;
    r.e = __shfl_sync(0xffffffffu, mine.e, from);
    r.row0 = __shfl_sync(0xffffffffu, mine.row0, from);
    r.rows = __shfl_sync(0xffffffffu, mine.rows, from);
    r.n = __shfl_sync(0xffffffffu, mine.n, from);
    r.k0 = __shfl_sync(0xffffffffu, mine.k0, from);
    r.kc = __shfl_sync(0xffffffffu, mine.kc, from);
    return r;
  }
};

__device__ __forceinline__ int blocks_of(int kc) { return (kc + kBlockK - 1) / kBlockK; }
// Where share `part` of `parts` of them begins.
__device__ __forceinline__ int share(int kblocks, int part, int parts) {
  return parts == 1 ? part * kblocks : static_cast<int>(static_cast<int64_t>(kblocks) * part / parts);
}

// ---- rows in and out of the epilogue ------------------------------------------
// A lane holds 128 bytes of its own row; four lanes move 128 bytes of one row
// together, 32 each, for their four rows in turn.

// Lane i of four holds units u[0..3] of row i; after it, unit i of rows 0..3.  Its own inverse.
__device__ __forceinline__ void transpose_4(uint32_t (&u)[4][8], int lane) {
#pragma unroll
  for (int d = 1; d < 4; d *= 2) {
    const bool upper = lane & d;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & d) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? u[j][i] : u[j + d][i], d);
        u[j][i] = upper ? got : u[j][i];
        u[j + d][i] = upper ? u[j + d][i] : got;
      }
    }
  }
}

struct Rows {
  uint8_t* at;      // the lane's 32 bytes of the first of its four rows
  int64_t stride;   // bytes of a row
  int rows;         // of the four, how many exist
  int left;         // bytes of the row from `at` on (a multiple of 16; may be negative)
  bool wide;        // rows begin on 32-byte boundaries
};

// 128 bytes from byte `col` on of the rows of this warp (32 rows from r0 on).
__device__ __forceinline__ Rows rows_at(void* base, int64_t row, int64_t stride, int64_t col, int rows, int lane) {
  Rows r;
  const int64_t byte = col + (lane & 3) * 32;
  r.at = static_cast<uint8_t*>(base) + (row + (lane & ~3)) * stride + byte;
  r.stride = stride;
  r.rows = rows - (lane & ~3);
  const int64_t left = stride - byte;
  r.left = left > 32 ? 32 : static_cast<int>(left);
  r.wide = ((reinterpret_cast<uintptr_t>(base) | static_cast<uintptr_t>(stride) | static_cast<uintptr_t>(col)) & 31) == 0;
  return r;
}

__device__ __forceinline__ void store_rows(const Rows& r, uint32_t (&u)[4][8], int lane) {
  transpose_4(u, lane);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k >= r.rows) continue;
    uint8_t* to = r.at + k * r.stride;
    const uint4 q0 = make_uint4(u[k][0], u[k][1], u[k][2], u[k][3]);
    const uint4 q1 = make_uint4(u[k][4], u[k][5], u[k][6], u[k][7]);
    if (r.wide && r.left >= 32) {
      tc::st_v8(to, q0, q1);
    } else {
      if (r.left >= 16) ptx::st_v4(to, q0);
      if (r.left >= 32) ptx::st_v4(to + 16, q1);
    }
  }
}

__device__ __forceinline__ uint4 ld_v4(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// The loads alone; transpose_4 then gives every lane its own row.
__device__ __forceinline__ void fetch_rows(const Rows& r, uint32_t (&u)[4][8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint4 q0 = make_uint4(0, 0, 0, 0), q1 = q0;
    if (k < r.rows) {
      const uint8_t* from = r.at + k * r.stride;
      if (r.wide && r.left >= 32) {
        tc::ld_v8(from, q0, q1);
      } else {
        if (r.left >= 16) q0 = ld_v4(from);
        if (r.left >= 32) q1 = ld_v4(from + 16);
      }
    }
    u[k][0] = q0.x, u[k][1] = q0.y, u[k][2] = q0.z, u[k][3] = q0.w;
    u[k][4] = q1.x, u[k][5] = q1.y, u[k][6] = q1.z, u[k][7] = q1.w;
  }
}

// 64 float32 columns of a row out as bf16 or float32.
__device__ __forceinline__ void store_bf16(const Rows& r, const float (&v)[kUnit], int lane) {
  uint32_t u[4][8];
#pragma unroll
  for (int i = 0; i < 32; ++i) u[i / 8][i & 7] = bf16x2(v[2 * i], v[2 * i + 1]);
  store_rows(r, u, lane);
}
__device__ __forceinline__ void store_f32(Rows r, const float (&v)[kUnit], int lane, int64_t bytes_left) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t u[4][8];
#pragma unroll
    for (int i = 0; i < 32; ++i) u[i / 8][i & 7] = __float_as_uint(v[h * 32 + i]);
    const int64_t left = bytes_left - h * 128 - (lane & 3) * 32;
    r.left = left > 32 ? 32 : static_cast<int>(left);
    store_rows(r, u, lane);
    r.at += 128;
  }
}
__device__ __forceinline__ void add_packed(const uint32_t (&u)[4][8], float (&v)[kUnit]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v[2 * i] += bf_lo(u[i / 8][i & 7]);
    v[2 * i + 1] += bf_hi(u[i / 8][i & 7]);
  }
}
__device__ __forceinline__ void load_f32(Rows r, float (&v)[kUnit], int lane, int64_t bytes_left) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t u[4][8];
    const int64_t left = bytes_left - h * 128 - (lane & 3) * 32;
    r.left = left > 32 ? 32 : static_cast<int>(left);
    fetch_rows(r, u);
    transpose_4(u, lane);
    r.at += 128;
#pragma unroll
    for (int i = 0; i < 32; ++i) v[h * 32 + i] = __uint_as_float(u[i / 8][i & 7]);
  }
}

// The kind of activation is asked for once for all 64 columns.
template <int kAct>
__device__ __forceinline__ void activate_all(float (&v)[kUnit]) {
#pragma unroll
  for (int i = 0; i < kUnit; i += 2) {
    const Two r = act_value(kAct, Two(v[i], v[i + 1]));
    v[i] = r.lo();
    v[i + 1] = r.hi();
  }
}
__device__ __forceinline__ void activate(int act, float (&v)[kUnit]) {
  if (act == MOE_ACT_RELU) activate_all<MOE_ACT_RELU>(v);
  else if (act == MOE_ACT_GELU) activate_all<MOE_ACT_GELU>(v);
  else if (act == MOE_ACT_SILU) activate_all<MOE_ACT_SILU>(v);
}
// g times the derivative at the packed values.
template <int kAct>
__device__ __forceinline__ void through_one(float (&g)[kUnit], const uint32_t (&u)[4][8]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const Two r = act_through(kAct, Two(g[2 * i], g[2 * i + 1]), Two(bf_lo(u[i / 8][i & 7]), bf_hi(u[i / 8][i & 7])));
    g[2 * i] = r.lo();
    g[2 * i + 1] = r.hi();
  }
}
__device__ __forceinline__ void through(int act, float (&g)[kUnit], const uint32_t (&u)[4][8]) {
  if (act == MOE_ACT_RELU) through_one<MOE_ACT_RELU>(g, u);
  else if (act == MOE_ACT_GELU) through_one<MOE_ACT_GELU>(g, u);
  else if (act == MOE_ACT_SILU) through_one<MOE_ACT_SILU>(g, u);
}

// 64 columns of this warp's lanes.  The last columns of a matrix may be
// missing in the tile's operand: they are zeros.
__device__ __forceinline__ void load_acc(uint32_t from, float (&v)[kUnit]) {
  tc::tmem_load_32(from, reinterpret_cast<uint32_t*>(v));
  tc::tmem_load_32(from + 32, reinterpret_cast<uint32_t*>(v) + 32);
  tc::wait_loads();
}

// Four columns of the bias from `col` on (0 past the last).
__device__ __forceinline__ float4 bias_at(const LinearParams& p, int e, int col) {
  if (col >= p.bias_cols) return make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // bias_cols is a multiple of 8
  const int64_t at = static_cast<int64_t>(e) * p.bias_cols + col;
  if (p.bias_f32) return __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.bias) + at));
  const uint2 q = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.bias) + at));
  return make_float4(bf_lo(q.x), bf_hi(q.x), bf_lo(q.y), bf_hi(q.y));
}
// 64 columns of it added, from shared memory: the same for every lane.
__device__ __forceinline__ void add_bias(const float* bias, float (&v)[kUnit]) {
#pragma unroll
  for (int i = 0; i < kUnit; i += 4) {
    const float4 q = *reinterpret_cast<const float4*>(bias + i);
    v[i] += q.x, v[i + 1] += q.y, v[i + 2] += q.z, v[i + 3] += q.w;
  }
}

// Asks L2 for what epilogue will read of this warp's rows (residual, pre), a tile
// ahead.
template <Mode kMode, bool kGlu, int kN>
__device__ __forceinline__ void prefetch_rows(const LinearParams& p, const Tile& tile, int half, int sub, int lane) {
  const void* base = kMode == kForward ? p.residual : p.pre;
  if (lane >= tile.rows - sub) return;
  // Glu: forward 64 columns of h, input both halves of pre.
  constexpr bool kWide = kMode == kInput && kGlu;
  const int col = tile.n * (kMode == kForward && kGlu ? kN / 2 : kN) +
                  half * (kMode == kForward && kGlu ? kUnit : kN / 2);
  const uint8_t* row = static_cast<const uint8_t*>(base) +
                       static_cast<int64_t>(tile.row0 + sub + lane) * p.N * (kWide ? 4 : 2) + static_cast<int64_t>(col) * 2;
  // Rows need not begin with a line: the last element's line is asked for too.
  constexpr int kColumns = kMode == kForward && kGlu ? kUnit : kN / 2;
#pragma unroll
  for (int i = 0; i <= kColumns; i += 64) {
    const int c = min(min(i, kColumns - 1), p.N - 1 - col);
    if (c < 0) break;
    ptx::prefetch_l2(row + c * 2);
    if (kWide) ptx::prefetch_l2(row + (static_cast<int64_t>(p.N) + c) * 2);
  }
}

// Whether epilogue reads rows 64 columns at a time, the next ones while it works on these.
template <Mode kMode, bool kGlu>
__device__ __forceinline__ bool reads_ahead(const LinearParams& p) {
  return !kGlu && ((kMode == kForward && p.residual) || (kMode == kInput && p.act != MOE_ACT_NONE));
}
// Columns 64 q .. of a tile's part of them, if this warp has any.
template <Mode kMode, int kN>
__device__ __forceinline__ void fetch_unit(const LinearParams& p, const Tile& tile, int half, int sub, int lane, int q,
                                           uint32_t (&raw)[4][8]) {
  const int col = tile.n * kN + half * (kN / 2) + q * kUnit, rows = tile.rows - sub;
  if (rows > 0 && col < p.N)
    fetch_rows(rows_at(kMode == kForward ? p.residual : p.pre, tile.row0 + sub, static_cast<int64_t>(p.N) * 2,
                       static_cast<int64_t>(col) * 2, rows, lane),
               raw);
}

// What becomes of a tile's sums: this warp's 32 rows (from sub on) and half of the
// columns.  load(column, v, last) waits for the sums and gets 64 of them; it is called
// for all of them even where the warp has no rows (some is false), but not where there
// are no sums (any is false: zeros).  False: the wait gave up.  raw: what fetch_unit gave
// for the first columns, and with `more` in the end for those of `next`; bias: this
// warp's 128 floats of shared memory.
template <Mode kMode, bool kGlu, bool kF32, int kN, class Load>
__device__ __forceinline__ bool epilogue(const LinearParams& p, const Tile& tile, const Tile& next, bool more, int half,
                                         int sub, int lane, bool any, bool some, uint32_t (&raw)[4][8], float* bias,
                                         Load&& load) {
  const int rows = tile.rows - sub;
  const int64_t row = tile.row0 + sub;
  constexpr bool kGate = kMode == kForward && kGlu;  // 64 columns of h: 64 of the gate, 64 up
  const int col0 = kGate ? tile.n * (kN / 2) + half * kUnit : tile.n * kN + half * (kN / 2);
  const int64_t stride = static_cast<int64_t>(p.N) * 2;
  some = some && col0 < p.N;
  const bool adds = kMode == kForward && p.residual, turns = kMode == kInput && !kGlu && p.act != MOE_ACT_NONE;
  if (kMode == kForward && p.bias) {
    __syncwarp();
    const int c = kGate ? (lane < 16 ? 0 : p.N - kUnit) + col0 + lane * 4 : col0 + lane * 4;
    *reinterpret_cast<float4*>(bias + lane * 4) = bias_at(p, tile.e, c);
    __syncwarp();
  }
  if constexpr (kGate) {
    float v[kUnit], up[kUnit];
    if (!load(half * kUnit, v, false) || !load(kN / 2 + half * kUnit, up, true)) return false;
    if (!some) return true;
    if (p.bias) {
      add_bias(bias, v);
      add_bias(bias + kUnit, up);
    }
    if (p.pre) {
      Rows r = rows_at(p.pre, row, 2 * stride, static_cast<int64_t>(col0) * 2, rows, lane);
      const int left = min(32, (p.N - col0) * 2 - (lane & 3) * 32);  // the first half ends where the second begins
      r.left = left;
      store_bf16(r, v, lane);
      r = rows_at(p.pre, row, 2 * stride, stride + static_cast<int64_t>(col0) * 2, rows, lane);
      r.left = left;
      store_bf16(r, up, lane);
    }
#pragma unroll
    for (int i = 0; i < kUnit; i += 2) {
      const Two r = act_value(MOE_ACT_SILU, Two(v[i], v[i + 1])) * Two(up[i], up[i + 1]);
      v[i] = r.lo();
      v[i + 1] = r.hi();
    }
    if (adds) {
      fetch_rows(rows_at(p.residual, row, stride, static_cast<int64_t>(col0) * 2, rows, lane), raw);
      transpose_4(raw, lane);
      add_packed(raw, v);
    }
    constexpr int kSize = kF32 ? 4 : 2;
    const Rows r =
        rows_at(p.out, row, static_cast<int64_t>(p.N) * kSize, static_cast<int64_t>(col0) * kSize, rows, lane);
    if (kF32) store_f32(r, v, lane, static_cast<int64_t>(p.N - col0) * 4);
    else store_bf16(r, v, lane);
  } else if constexpr (kMode == kInput && kGlu) {
#pragma unroll 1
    for (int q = 0; q < kN / 2 / kUnit; ++q) {
      const int64_t byte = static_cast<int64_t>(col0 + q * kUnit) * 2;
      const bool here = some && col0 + q * kUnit < p.N;
      Rows at = rows_at(p.pre, row, 2 * stride, byte, rows, lane);
      const Rows at_up = rows_at(p.pre, row, 2 * stride, stride + byte, rows, lane);
      at.left = at_up.left;  // the row's first half ends where the second begins
      uint32_t up[4][8];     // gate: raw
      if (here) {
        fetch_rows(at, raw);
        fetch_rows(at_up, up);
      }
      float v[kUnit] = {};
      if (any && !load(half * (kN / 2) + q * kUnit, v, q == kN / 2 / kUnit - 1)) return false;
      if (!here) continue;
      transpose_4(raw, lane);
      transpose_4(up, lane);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        uint32_t &g2 = raw[i / 8][i & 7], &u2 = up[i / 8][i & 7];
        Two gate(bf_lo(g2), bf_hi(g2)), u(bf_lo(u2), bf_hi(u2));
        swiglu_through(Two(v[2 * i], v[2 * i + 1]), gate, u);
        g2 = bf16x2(gate.lo(), gate.hi());
        u2 = bf16x2(u.lo(), u.hi());
      }
      Rows to = rows_at(p.out, row, 2 * stride, byte, rows, lane);
      to.left = at.left;
      store_rows(to, raw, lane);
      store_rows(rows_at(p.out, row, 2 * stride, stride + byte, rows, lane), up, lane);
    }
  } else {
#pragma unroll 1
    for (int q = 0; q < kN / 2 / kUnit; ++q) {
      const int col = col0 + q * kUnit;
      float v[kUnit] = {};
      if (any && !load(half * (kN / 2) + q * kUnit, v, q == kN / 2 / kUnit - 1)) return false;
      const bool here = some && col < p.N;
      const int64_t byte = static_cast<int64_t>(col) * 2;
      if (here) {
        if (kMode == kForward) {
          if (p.bias) add_bias(bias + q * kUnit, v);
          if (p.pre) store_bf16(rows_at(p.pre, row, stride, byte, rows, lane), v, lane);
          activate(p.act, v);
        }
        if (adds || turns) transpose_4(raw, lane);
        if (adds) add_packed(raw, v);
        if (turns) through(p.act, v, raw);
      }
      if (adds || turns) {
        if (q + 1 < kN / 2 / kUnit) fetch_unit<kMode, kN>(p, tile, half, sub, lane, q + 1, raw);
        else if (more) fetch_unit<kMode, kN>(p, next, half, sub, lane, 0, raw);
      }
      if (!here) continue;
      if (kMode != kWeight) {
        if (kF32) store_f32(rows_at(p.out, row, 2 * stride, 2 * byte, rows, lane), v, lane, 2 * (stride - byte));
        else store_bf16(rows_at(p.out, row, stride, byte, rows, lane), v, lane);
        continue;
      }
      if (p.accumulate && !any) continue;
      const int64_t out_row = static_cast<int64_t>(tile.e) * p.M + row;
      if (kF32) {
        const Rows at = rows_at(p.out, out_row, 2 * stride, 2 * byte, rows, lane);
        if (p.accumulate) {
          float old[kUnit];
          load_f32(at, old, lane, 2 * (stride - byte));
#pragma unroll
          for (int i = 0; i < kUnit; ++i) v[i] += old[i];
        }
        store_f32(at, v, lane, 2 * (stride - byte));
      } else {
        const Rows at = rows_at(p.out, out_row, stride, byte, rows, lane);
        if (p.accumulate) {
          fetch_rows(at, raw);
          transpose_4(raw, lane);
          add_packed(raw, v);
        }
        store_bf16(at, v, lane);
      }
    }
  }
  return true;
}

template <bool kPair>
__device__ __forceinline__ void load_2d(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if (kPair) tc::tma_load_2d_pair(dst, map, x, y, bar);
  else tc::tma_load_2d(dst, map, x, y, bar);
}
template <bool kPair>
__device__ __forceinline__ void load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  if (kPair) tc::tma_load_3d_pair(dst, map, x, y, z, bar);
  else tc::tma_load_3d(dst, map, x, y, z, bar);
}

// An accumulator buffer is read: the CTA that issues the products may have it again.
template <bool kPair>
__device__ __forceinline__ void release(uint64_t* acc_empty) {
  if (kPair) tc::mbar_arrive_at(tc::at_rank(acc_empty, 0));
  else tc::mbar_arrive(acc_empty);
}

// Rows from `first` on of a stage's boxes, which belong to the next expert, become
// zeros in both operands (0 x infinity is no zero).  Whole warp.
__device__ __forceinline__ void clear_rows(uint8_t* stage, int bytes, int first, int lane) {
#pragma unroll 1
  for (int c = 0; c < bytes; c += kChunkBytes)
    for (int i = first * 8 + lane; i < kBlockK * 8; i += 32)
      *reinterpret_cast<uint4*>(stage + c + i * 16) = make_uint4(0, 0, 0, 0);
  tc::fence_async_shared();
  __syncwarp();
}

template <Mode kMode, bool kGlu, bool kF32, Team kTeam>
__global__ void __launch_bounds__(kThreads, 1) expert_linear_kernel(const __grid_constant__ LinearParams p) {
  constexpr bool kPair = kTeam == kPairs;
  constexpr int kStages = stage_count(kTeam), kStageBytes = stage_bytes(kTeam), kBColumns = b_columns(kTeam);
  constexpr int kN = tile_n(kTeam);
  extern __shared__ uint8_t s_raw[];
  __shared__ Shared s;
  uint8_t* stages = s_raw + ((1024 - (ptx::smem_addr(s_raw) & 1023)) & 1023);
  float* parts_at = reinterpret_cast<float*>(stages);  // split: the tile's sums, when the stages are done with
  Groups g;
  g.lo = reinterpret_cast<int32_t*>(stages + kStages * kStageBytes);
  g.hi = g.lo + p.E;
  g.start = g.hi + p.E;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = kPair ? tc::cluster_rank() : 0;
  // Split: one tile a cluster, whose CTA number `part` sums part / parts of the axis.
  const int part = kTeam == kSplit ? tc::cluster_rank() : 0, parts = kTeam == kSplit ? p.split : 1;
  const int team = kPair ? 2 : parts;
  const uint32_t first_tile = blockIdx.x / team, tile_step = gridDim.x / team;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&s.full[i], 1);
      ptx::mbar_init(&s.empty[i], 1);
      ptx::mbar_init(&s.tail_full[i], 1);
      ptx::mbar_init(&s.tail_clear[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&s.acc_full[i], 1);
      ptx::mbar_init(&s.acc_empty[i], kPair ? 2 * kEpilogueWarps : kEpilogueWarps);
    }
    ptx::mbar_init(&s.drained, 1);
    ptx::mbar_fence_init();
    s.gave_up = 0;
  }
  if (warp == kMmaWarp) {
    if (kPair) tc::tmem_alloc_pair(&s.tmem, kTmemColumns);
    else tc::tmem_alloc(&s.tmem, kTmemColumns);
  }
  if (threadIdx.x == kTmaWarp * 32) {
    tc::tma_prefetch_map(&p.a);
    tc::tma_prefetch_map(&p.b);
  }
  ptx::wait_prerequisites();
  ptx::launch_dependents();
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
  if (kMode != kWeight && warp == 0) {
    constexpr int kRows = kPair ? 2 * kTileM : kTileM;
    int before = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      const int own = e < p.E ? (g.hi[e] - g.lo[e] + kRows - 1) / kRows : 0;
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
  if (kPair) tc::cluster_sync();  // the other CTA's barriers are ready too
  else __syncthreads();
  tc::fence_after();
  const uint32_t tiles = tile_count<kMode>(g, p);
  Walk<kMode, kPair, kN> walk = {first_tile, tile_step, tiles, rank};
  const uint32_t tmem = s.tmem, tmem_u = __shfl_sync(0xffffffffu, tmem, 0);

  if (warp == kTmaWarp) {
    uint32_t it = 0;
    bool ok = true;
    uint32_t i = 0;
    for (uint32_t t = first_tile; ok && t < tiles; t += tile_step) {
      const Tile tile = walk.get(g, p, i++, lane);
      const int kblocks = blocks_of(tile.kc), kb0 = share(kblocks, part, parts), kb1 = share(kblocks, part + 1, parts);
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int st = it % kStages;
        ok = it < kStages || tc::wait(&s.empty[st], (it / kStages - 1) & 1, &s.gave_up);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint8_t *a = stages + st * kStageBytes, *b = a + kABytes;
        // A pair's loads are all counted by the first CTA, which issues the products;
        // but the second one's part of a stage that it has to clear by itself.
        const bool own = kPair && kMode == kWeight && kb == kblocks - 1 && tile.kc % kBlockK != 0;
        uint64_t* expects = own && rank == 1 ? &s.tail_full[st] : &s.full[st];
        const uint32_t bar = kPair && !own ? tc::at_rank(expects, 0) : ptx::smem_addr(expects);
        if (tc::elect() && it != p.test_drop) {
          if (rank == 0 || own) ptx::mbar_arrive_expect_tx(expects, kPair && !own ? 2 * kStageBytes : kStageBytes);
          const int k = tile.k0 + kb * kBlockK;
          if (kMode == kWeight) {
#pragma unroll
            for (int q = 0; q < kTileM / 64; ++q) load_2d<kPair>(a + q * kChunkBytes, &p.a, tile.row0 + q * 64, k, bar);
#pragma unroll
            for (int q = 0; q < kBColumns / 64; ++q)
              load_2d<kPair>(b + q * kChunkBytes, &p.b, tile.n * kN + rank * kBColumns + q * 64, k, bar);
          } else {
            load_2d<kPair>(a, &p.a, k, tile.row0, bar);
            if (kMode == kForward) {
              // Boxes of 128: the first and the second half of the columns (glu: gate, up).
              const int n0 = tile.n * (kGlu ? kN / 2 : kN), n1 = n0 + (kGlu ? p.N : kN / 2);
              load_3d<kPair>(b, &p.b, k, rank == 0 ? n0 : n1, tile.e, bar);
              if (kBColumns == 256) load_3d<kPair>(b + 128 * kBlockK * 2, &p.b, k, n1, tile.e, bar);
            } else {
#pragma unroll
              for (int q = 0; q < kBColumns / 64; ++q)
                load_3d<kPair>(b + q * kChunkBytes, &p.b, tile.n * kN + rank * kBColumns + q * 64, k, tile.e, bar);
            }
          }
        }
        __syncwarp();
      }
    }
    // Loads in flight write to this CTA's shared memory: it does not end before
    // them, whichever warp gave up.
    const unsigned long long start = tc::now_ns();
    if (rank == 0)
      for (uint32_t j = it > kStages ? it - kStages : 0; j < it; ++j)
        if (j != p.test_drop) tc::settle(&s.full[j % kStages], (j / kStages) & 1, start);
    // A pair's second CTA knows its loads by their stages being free again, and
    // that is an arrival from afar in either.
    if (kPair)
      for (uint32_t j = it > kStages ? it - kStages : 0; j < it; ++j)
        tc::settle(&s.empty[j % kStages], (j / kStages) & 1, start);
  } else if (warp == kMmaWarp && rank == 0) {
    constexpr uint32_t kInstr =
        tc::instr_desc_bf16(kPair ? 2 * kTileM : kTileM, kN, kMode == kWeight, kMode != kForward);
    uint32_t i = 0, it = 0, round = 0, tails = 0;  // tails: parity of tail_clear, a bit a stage
    bool ok = true;
    for (uint32_t t = first_tile; ok && t < tiles; t += tile_step) {
      Tile tile;
      tile.kc = p.kc;
      if (kMode == kWeight) tile = walk.get(g, p, i++, lane);
      const int kblocks = blocks_of(tile.kc), kb0 = share(kblocks, part, parts), kb1 = share(kblocks, part + 1, parts);
      if (kb0 == kb1) continue;
      const int buf = round & 1;
      ok = round < 2 || tc::wait(&s.acc_empty[buf], (round / 2 - 1) & 1, &s.gave_up);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int st = it % kStages;
        ok = tc::wait(&s.full[st], (it / kStages) & 1, &s.gave_up);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint8_t* a_tile = stages + st * kStageBytes;
        if (kMode == kWeight && kb == kblocks - 1 && tile.kc % kBlockK != 0) {
          clear_rows(a_tile, kStageBytes, tile.kc % kBlockK, lane);
          if (kPair) {
            ok = tc::wait_cluster(&s.tail_clear[st], (tails >> st) & 1, &s.gave_up);
            tails ^= 1u << st;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
        }
        tc::fence_after();
        const uint64_t a = kMode == kWeight ? tc::smem_desc_mn(a_tile) : tc::smem_desc(a_tile);
        const uint64_t b = kMode != kForward ? tc::smem_desc_mn(a_tile + kABytes) : tc::smem_desc(a_tile + kABytes);
        // 16 further along the summed axis: 32 bytes, or 16 rows of 128.
        constexpr uint64_t kStepA = (kMode == kWeight ? 2048 : 32) >> 4;
        constexpr uint64_t kStepB = (kMode != kForward ? 2048 : 32) >> 4;
        if (tc::elect()) {
#pragma unroll
          for (int k = 0; k < kBlockK / 16; ++k) {
            const uint32_t d = tmem_u + buf * kN;
            if (kPair) tc::mma_f16_pair(d, a + kStepA * k, b + kStepB * k, kInstr, kb > kb0 || k > 0);
            else tc::mma_f16(d, a + kStepA * k, b + kStepB * k, kInstr, kb > kb0 || k > 0);
          }
          if (kPair) tc::commit_pair(&s.empty[st]);
          else tc::commit(&s.empty[st]);
          if (kb == kb1 - 1) {
            if (kPair) tc::commit_pair(&s.acc_full[buf]);
            else tc::commit(&s.acc_full[buf]);
          }
        }
        __syncwarp();
      }
      ++round;
    }
    // Nothing may be in flight when the tensor memory is freed.
    if (tc::elect()) {
      if (kPair) tc::commit_pair(&s.drained);
      else tc::commit(&s.drained);
    }
    __syncwarp();
    tc::settle(&s.drained, 0, tc::now_ns());
  } else if (warp == kMmaWarp) {
    // The second CTA of a pair clears its half of an expert's last stage.
    if (kMode == kWeight) {
      uint32_t i = 0, it = 0, tails = 0;
      bool ok = true;
      for (uint32_t t = first_tile; ok && t < tiles; t += tile_step) {
        const Tile tile = walk.get(g, p, i++, lane);
        it += blocks_of(tile.kc);
        if (tile.kc % kBlockK == 0) continue;
        const int st = (it - 1) % kStages;
        ok = tc::wait(&s.tail_full[st], (tails >> st) & 1, &s.gave_up);
        tails ^= 1u << st;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        clear_rows(stages + st * kStageBytes, kStageBytes, tile.kc % kBlockK, lane);
        if (lane == 0) tc::mbar_release_at(tc::at_rank(&s.tail_clear[st], 0));
        __syncwarp();
      }
    }
    tc::settle(&s.drained, 0, tc::now_ns());
  } else if (warp >= kBiasWarp) {
    if (kMode == kWeight && p.db) {
      // An expert's 128 columns of dy a CTA at a time, 64 a warp, a lane 8 of them in
      // every fourth row.
      const int piece = lane & 7, first = lane >> 3;
      const uint32_t blocks = (p.M + 127) / 128, units = blocks * p.E;
      for (uint32_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int e = static_cast<int>(u / blocks);
        const int col = static_cast<int>(u - e * blocks) * 128 + (warp - kBiasWarp) * 64 + piece * 8;
        const int rows = g.hi[e] - g.lo[e];
        if (p.accumulate && rows == 0) continue;
        const uint8_t* from = p.dy + (static_cast<int64_t>(g.lo[e]) * p.M + col) * 2;
        const int64_t stride = static_cast<int64_t>(p.M) * 2;
        const bool some = col < p.M;  // M is a multiple of 8
        float sum[8] = {};
        for (int r0 = 0; r0 < rows; r0 += 4 * kLoads) {
          uint4 v[kLoads];
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            const int r = r0 + 4 * i + first;
            v[i] = some && r < rows ? ptx::ld_stream_v4(from + r * stride) : make_uint4(0, 0, 0, 0);
          }
          float part[8] = {};
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            part[0] += bf_lo(v[i].x), part[1] += bf_hi(v[i].x), part[2] += bf_lo(v[i].y), part[3] += bf_hi(v[i].y);
            part[4] += bf_lo(v[i].z), part[5] += bf_hi(v[i].z), part[6] += bf_lo(v[i].w), part[7] += bf_hi(v[i].w);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] += part[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 8);
          sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 16);
        }
        if (first == 0 && some) {
          float4* to = reinterpret_cast<float4*>(p.db + static_cast<int64_t>(e) * p.M + col);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float4 v = make_float4(sum[4 * h], sum[4 * h + 1], sum[4 * h + 2], sum[4 * h + 3]);
            if (p.accumulate) {
              const float4 old = to[h];
              v.x += old.x, v.y += old.y, v.z += old.z, v.w += old.w;
            }
            to[h] = v;
          }
        }
      }
    }
  } else {
    const int half = warp >> 2, sub = (warp & 3) * 32;  // this warp's rows begin at sub
    const uint32_t lanes = tmem + (static_cast<uint32_t>(sub) << 16);
    uint32_t round = 0, raw[4][8];
    bool ok = true;
    const bool ahead = reads_ahead<kMode, kGlu>(p);
    // Only where a sum is too short to hide those reads.  us with / without: residual, N 2048
    // 35 / 40 at K = 128, 41.4 / 43.9 at 512, 55 / 54 at 1024; through SiLU, 63810 rows, K 4368
    // of N 208: 363 / 421; through the gate of 8 experts, N 4096: 358 / 340.
    const bool reads = (kMode == kForward ? p.residual : kMode == kInput ? p.pre : nullptr) && p.kc <= 512;
    Tile next;
    uint32_t number = 0;
    if (first_tile < tiles) next = walk.get(g, p, number++, lane);
    if (ahead && kTeam != kSplit && first_tile < tiles) fetch_unit<kMode, kN>(p, next, half, sub, lane, 0, raw);
    for (uint32_t t = first_tile; ok && t < tiles; t += tile_step) {
      const Tile tile = next;
      const bool more = kTeam != kSplit && t + tile_step < tiles;
      if (more) next = walk.get(g, p, number++, lane);
      const int kblocks = blocks_of(tile.kc);
      const bool any = kblocks > 0;  // whether there is a sum at all (weight: the expert has rows)
      const bool sums = share(kblocks, part, parts) < share(kblocks, part + 1, parts);
      const int buf = round & 1;
      const uint32_t acc = lanes + buf * kN;
      bool waits = sums;
      auto sums_are_there = [&] {
        if (waits) {
          waits = false;
          ok = __all_sync(0xffffffffu, tc::wait(&s.acc_full[buf], (round / 2) & 1, &s.gave_up));
          tc::fence_after();
          ++round;
        }
        return ok;
      };
      if (kTeam == kSplit) {
        // This CTA's part of the sums, for the others to read.
        float* to = parts_at + (sub + lane) * kPitch + half * (kN / 2);
        if (any && sums_are_there()) {
#pragma unroll 1
          for (int q = 0; q < kN / 2 / kUnit; ++q) {
            float v[kUnit] = {};
            if (sums) load_acc(acc + half * (kN / 2) + q * kUnit, v);
#pragma unroll
            for (int i = 0; i < kUnit; i += 4)
              *reinterpret_cast<float4*>(to + q * kUnit + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          }
        }
        break;
      }
      if (reads && more) prefetch_rows<kMode, kGlu, kN>(p, next, half, sub, lane);
      // A warp none of whose rows exist only passes the buffer on.
      epilogue<kMode, kGlu, kF32, kN>(p, tile, next, more, half, sub, lane, any, sub < tile.rows, raw, s.bias[warp],
                                  [&](int column, float(&v)[kUnit], bool last) {
                                    if (!sums_are_there()) return false;
                                    if (sub < tile.rows) load_acc(acc + column, v);
                                    if (last) {
                                      tc::fence_before();
                                      __syncwarp();
                                      if (lane == 0) release<kPair>(&s.acc_empty[buf]);
                                    }
                                    return true;
                                  });
    }
  }
  if (kTeam == kSplit) {
    tc::fence_before();
    tc::cluster_sync();
    if (warp < kEpilogueWarps && first_tile < tiles) {
      // Every CTA finishes the blocks of 32 rows x half of the columns whose warp's number
      // falls to it: adds the parts in order, the eight warps together, then writes them out.
      const Tile tile = find_tile<kMode, kPair, kN>(g, p, first_tile, rank);
      const bool any = tile.kc > 0;
      if (any) {
        const int mine = kEpilogueWarps / parts;  // 1 to 4 blocks, part, part + parts, ...
        for (int i = threadIdx.x; i < mine * 32 * 32; i += kEpilogueWarps * 32) {
          const int block = part + (i >> 10) * parts, r = (block & 3) * 32 + ((i >> 5) & 31);
          // Glu: 64 gate columns and the 64 up columns that belong to them.
          const int quad = (i & 31) * 4, h = block >> 2;
          const int c = kMode == kForward && kGlu ? (quad >> 6) * (kN / 2) + h * kUnit + (quad & 63)
                                                  : h * (kN / 2) + quad;
          float* at = parts_at + r * kPitch + c;
          float4 v[kMaxSplit];
#pragma unroll
          for (int q = 0; q < kMaxSplit; ++q)
            if (q < parts) v[q] = tc::ld_cluster_v4(tc::at_rank(at, q));
#pragma unroll
          for (int q = 1; q < kMaxSplit; ++q)
            if (q < parts) {
              v[0].x += v[q].x;
              v[0].y += v[q].y;
              v[0].z += v[q].z;
              v[0].w += v[q].w;
            }
          *reinterpret_cast<float4*>(at) = v[0];
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kEpilogueWarps * 32) : "memory");
      const int half = warp >> 2, sub = (warp & 3) * 32;
      if (warp % parts == part) {
        uint32_t raw[4][8];
        if (reads_ahead<kMode, kGlu>(p)) fetch_unit<kMode, kN>(p, tile, half, sub, lane, 0, raw);
        epilogue<kMode, kGlu, kF32, kN>(p, tile, tile, false, half, sub, lane, any, sub < tile.rows, raw, s.bias[warp],
                                    [&](int column, float(&v)[kUnit], bool) {
                                      const float* from = parts_at + (sub + lane) * kPitch + column;
#pragma unroll
                                      for (int i = 0; i < kUnit; i += 4) {
                                        const float4 q = *reinterpret_cast<const float4*>(from + i);
                                        v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
                                      }
                                      return true;
                                    });
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  // Pair: products read the other CTA's shared memory, arrivals reach it; split: sums are read.
  if (kTeam == kPairs || kTeam == kSplit) tc::cluster_sync();
  tc::fence_after();
  if (threadIdx.x == 0 && s.gave_up && p.status) atomicCAS(p.status, MOE_OK, MOE_ETIMEDOUT);
  if (warp == kMmaWarp) {
    if (kPair) tc::tmem_free_pair(tmem, kTmemColumns);
    else tc::tmem_free(tmem, kTmemColumns);
  }
  if (kPair) tc::cluster_sync();
}

// Pairs of CTAs that are resident at a time (a pair's two share a GPC, so not every
// SM need be used), asked for once per device and kernel; 0: the query failed.
int resident_pairs(const void* kernel, size_t smem) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  static std::mutex mu;
  static std::map<std::pair<int, const void*>, int> known;
  std::lock_guard<std::mutex> lock(mu);
  auto it = known.find({dev, kernel});
  if (it != known.end()) return it->second;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  known[{dev, kernel}] = n;
  return n;
}

template <Mode kMode, bool kGlu, bool kF32, Team kTeam>
cudaError_t launch(const LinearParams& p, int sms, cudaStream_t stream) {
  constexpr bool kPair = kTeam == kPairs;
  // The most tables that any call has, so that what fits is the same for all.
  const size_t smem = 1024 + stage_count(kTeam) * stage_bytes(kTeam) + (3 * MOE_MAX_EXPERTS + 1) * sizeof(int32_t);
  auto* kernel = expert_linear_kernel<kMode, kGlu, kF32, kTeam>;
  cudaError_t err = set_kernel_limits(reinterpret_cast<const void*>(kernel), smem);
  if (err != cudaSuccess) return err;
  // Every expert may add one partly filled row tile.
  constexpr int kRows = kPair ? 2 * kTileM : kTileM;
  const int64_t m_tiles = kMode == kWeight ? static_cast<int64_t>(p.E) * p.m_tiles
                                           : (p.rows + kRows - 1) / kRows + (p.offsets ? p.E : 0);
  const int64_t tiles = m_tiles * p.n_tiles;
  if (tiles > INT_MAX / kMaxSplit) return cudaErrorInvalidValue;
  int64_t teams = tiles, team = 1;  // split: a cluster for each tile there may be
  if (kTeam == kAlone || kTeam == kNarrow) {
    teams = tiles < sms ? tiles : sms;
  } else if (kTeam == kPairs) {
    const int pairs = resident_pairs(reinterpret_cast<const void*>(kernel), smem);
    if (pairs <= 0) return cudaErrorInvalidConfiguration;
    teams = tiles < pairs ? tiles : pairs;
    team = 2;
  } else {
    team = p.split;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(teams * team));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(team);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kTeam == kAlone || kTeam == kNarrow ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <Mode kMode, bool kGlu, bool kF32>
cudaError_t launch(const LinearParams& p, bool pair, int sms, cudaStream_t stream) {
  if (p.split > 1) return launch<kMode, kGlu, kF32, kSplit>(p, sms, stream);
  if constexpr (kMode != kForward || !kGlu)  // (64 gate and 64 up columns would be half units)
    if (p.narrow) return launch<kMode, kGlu, kF32, kNarrow>(p, sms, stream);
  return pair ? launch<kMode, kGlu, kF32, kPairs>(p, sms, stream) : launch<kMode, kGlu, kF32, kAlone>(p, sms, stream);
}

}  // namespace

int linear_n_tile(bool glu, bool narrow) { return glu || narrow ? 128 : 256; }
int linear_m_tile(bool pair) { return pair ? 2 * kTileM : kTileM; }

cudaError_t launch_linear(const LinearParams& p, bool glu, bool f32, bool pair, int sms, cudaStream_t stream) {
  if (glu)
    return f32 ? launch<kForward, true, true>(p, pair, sms, stream) : launch<kForward, true, false>(p, pair, sms, stream);
  return f32 ? launch<kForward, false, true>(p, pair, sms, stream) : launch<kForward, false, false>(p, pair, sms, stream);
}

cudaError_t launch_linear_input(const LinearParams& p, bool glu, bool pair, int sms, cudaStream_t stream) {
  return glu ? launch<kInput, true, false>(p, pair, sms, stream) : launch<kInput, false, false>(p, pair, sms, stream);
}

cudaError_t launch_linear_weight(const LinearParams& p, bool f32, bool pair, int sms, cudaStream_t stream) {
  return f32 ? launch<kWeight, false, true>(p, pair, sms, stream) : launch<kWeight, false, false>(p, pair, sms, stream);
}

}  // namespace moe
