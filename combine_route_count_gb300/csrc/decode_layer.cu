// Products of few rows with many weights, on the 5th-generation tensor core:
//
//   row_groups   decode: h[t,k] = SiLU(W1[e] x[t]) * (W3[e] x[t]),  e = topk_idx[t,k],
//                quantised by blocks of 128 like every payload here
//                glu, gemm: the products of expert_gemm.cu for grouped rows,
//                where an expert has a few
//   few_rows     decode: out[t] = bf16( sum_k topk_w[t,k] * W2[e] h[t,k] )
//                dense:  out[i] = W a[i], one weight matrix, up to 32 rows
//
// The decode forms are a whole expert layer for up to 64 tokens in two kernels
// (moe_decode_layer_fp8).  The others serve moe_expert_glu_fp8 and
// moe_expert_gemm_fp8 where experts have few rows or there are few tiles.
//
// Bound by memory: the weights are read once for a few rows, so what counts is
// to keep many weight bytes in flight on every SM and to start early.  Weight
// tiles of 128 rows x 128 of K arrive by tiled TMA in a ring of stages, with
// the token rows' block beside them, and are the 128-row operand of tcgen05.mma;
// 16 or 32 rows of one expert are its columns.  A thread of the epilogue
// warps owns one weight row and a column per token row; each K block's product
// is scaled and added to its float32 registers as in expert_gemm.cu.  An
// earlier form loaded the weights straight into mma.sync fragments: its register
// stages kept too little in flight (one token, 8 of 256 experts, H 7168, inner
// 2048: 95 us, 45 % of DRAM busy).  Now: 62 to 63 us, 5.6 TB/s; 37 tokens, 6 of 64
// experts, H 4096, inner 1408: 156 to 164 us, 6.7 TB/s; glu of 512 rows over 256
// experts, H 7168, inner 1024: 466 to 485 us, 6.8 TB/s.
//
// row_groups gathers the x rows of an expert's tokens (TMA gather of four rows
// at a time); few_rows reads rows of h, which row_groups writes ordered by
// (expert, token).
//
// Spread over the SMs: row_groups' unit is 128 columns of one expert's h; few
// units are split along K over a cluster.  few_rows gives 128 columns of out to
// a cluster, which shares that tile's (expert, K block) items; partial sums are
// exchanged through distributed shared memory and added in rank order.  Sums
// have a fixed order: same inputs, same bits.
//
// Routing: every CTA sorts the T*K (token, expert) pairs itself (a bit per
// token in a mask per expert; a pair's place among its expert's rows is the
// number of lower bits set).  Malformed routing is seen by every CTA alike:
// nothing is written but the status.
//
// few_rows is launched while row_groups runs and brings in its first weights
// before it waits for h.  Waits are bounded (2 s) and report MOE_ETIMEDOUT.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <map>
#include <mutex>
#include <utility>

#include "ffn_kernels.cuh"
#include "fp8_quant.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

constexpr int kBlock = MOE_FP8_BLOCK;
constexpr int kTileBytes = 128 * kBlock;  // 128 weight rows x 128 of K
constexpr int kChunk = kFewChunk;         // token rows are handled 16 at a time
constexpr int kMaxStages = 12;
constexpr int kMaxBufs = 4;               // tensor-memory buffers, each for one turn
__host__ __device__ constexpr int bufs(int columns) { return columns == 16 ? 4 : 2; }
constexpr int kMaxRanks = 4;              // CTAs of a cluster in few_rows
constexpr int kTmaWarp = 4, kMmaWarp = 5;  // warps 0-3: epilogue
constexpr int kThreads = 192;

// A float of CTA `rank`'s shared memory, at the place that `p` has in this CTA's.
__device__ __forceinline__ float ld_cluster(const float* p, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(tc::at_rank(p, rank)) : "memory");
  return v;
}

__device__ __forceinline__ float4 ld_cluster_v4(const float* p, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(tc::at_rank(p, rank))
               : "memory");
  return v;
}

// ---- routing -------------------------------------------------------------------
// Rows are the pairs ordered by (expert, token).  An expert with more rows than
// a tile has columns (kN) appears several times in the list of those at work,
// with up to kN of its rows each: its weights are then read again, mostly from
// L2.  (A variant with 64 columns for 64 tokens needed registers for all of
// them whatever an expert had, and was slower on the usual experts.)
struct Routing {
  int32_t* active;   // the experts at work, ascending
  int32_t* first;    // their first rows
  int32_t* count;    // how many rows, 1 .. kN
  int32_t* token;    // of each row
  float* weight;     // topk_w of each row
  // scratch, free after build_routing
  uint32_t* mask;    // [E][2]
  int32_t* row_of;   // [E]
};
struct RoutingShared {
  int32_t warp_active[32], warp_rows[32];
  int32_t n_active, bad;
  int32_t most_rows;  // of one expert
};

__host__ __device__ inline int max_active(int pairs, int E, int kN) { return (pairs < E ? pairs : E) + pairs / kN; }
__host__ __device__ inline int routing_bytes(int pairs, int E, int kN, bool by_token) {
  const int a = max_active(pairs, E, kN);
  return (a * 12 + (by_token ? pairs * 8 : 0) + 15) / 16 * 16;
}

// What build_routing needs besides lies at the start of the ring, before any load.
static_assert(MOE_MAX_EXPERTS * 12 <= kTileBytes && 32 * 8 <= kTileBytes, "scratch fits in one stage");

__device__ __forceinline__ Routing routing_at(uint8_t* smem, uint8_t* scratch, int pairs, int E, int kN) {
  const int a = max_active(pairs, E, kN);
  Routing r;
  r.active = reinterpret_cast<int32_t*>(smem);
  r.first = r.active + a;
  r.count = r.first + a;
  r.token = r.count + a;
  r.weight = reinterpret_cast<float*>(r.token + pairs);
  r.mask = reinterpret_cast<uint32_t*>(scratch);
  r.row_of = reinterpret_cast<int32_t*>(r.mask + 2 * E);
  return r;
}

// Called by the whole CTA; ends with a barrier.  For at most 32 pairs: every
// pair counts the pairs before it, which spares the per-expert masks and their
// scan (8 pairs of 256 experts: 1.6 instead of 2.1 us from the launch's wait;
// with 128 pairs the counting takes 6.8 us).
__device__ __forceinline__ void build_routing_small(const Routing& r, RoutingShared& s, const DecodeParams& p, int kN) {
  const int pairs = p.T * p.K, i = threadIdx.x;
  int32_t* expert = reinterpret_cast<int32_t*>(r.mask);  // [pairs]
  int32_t* heads = expert + pairs;                       // [pairs] whether the pair begins a list entry
  int e = 0;
  float w = 0.0f;
  if (i < pairs) {
    e = p.topk_idx[i];
    w = p.topk_w[i];
    expert[i] = e;
  }
  if (i == 0) s.bad = 0, s.most_rows = 1;
  __syncthreads();
  int row = 0;
  bool head = false;  // the first of its expert's rows in a list entry
  if (i < pairs) {
    const int t0 = i / p.K * p.K;  // the token's first pair
    int before_me = 0;
    if (e < 0 || e >= p.E) s.bad = 1;
    for (int j = 0; j < pairs; ++j) {
      const int other = expert[j];
      const bool before = other == e && j < i;
      row += other < e || before;
      before_me += before;
      if (before && j >= t0) s.bad = 1;  // repeated within the token
    }
    head = before_me % kN == 0;
    heads[i] = head;
    atomicMax(&s.most_rows, min(before_me + 1, kN));
  }
  __syncthreads();
  if (s.bad) return;  // the same for the whole CTA
  if (i < pairs) {
    r.token[row] = i / p.K;
    r.weight[row] = w;
    int a = 0;
    for (int j = 0; j < pairs; ++j) a += heads[j] && (expert[j] < e || (expert[j] == e && j < i));
    if (head) {
      int rest = 0;  // of the expert's pairs, from this one on
      for (int j = i; j < pairs; ++j) rest += expert[j] == e;
      r.active[a] = e;
      r.first[a] = row;
      r.count[a] = min(rest, kN);
    }
    if (row == pairs - 1) s.n_active = head ? a + 1 : a;  // of the last entry
  }
  __syncthreads();
}

__device__ __forceinline__ void build_routing(const Routing& r, RoutingShared& s, const DecodeParams& p, int kN) {
  const int pairs = p.T * p.K, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (pairs <= 32) {
    build_routing_small(r, s, p, kN);
    return;
  }
  constexpr int kMost = (kFewTokens * MOE_MAX_TOP_K + kThreads - 1) / kThreads;
  int expert[kMost];
  float weight[kMost];
#pragma unroll
  for (int m = 0; m < kMost; ++m) {
    const int i = threadIdx.x + m * kThreads;
    expert[m] = i < pairs ? p.topk_idx[i] : 0;
    weight[m] = i < pairs ? p.topk_w[i] : 0.0f;
  }
  if (threadIdx.x == 0) s.bad = 0, s.most_rows = 1;
  for (int e = threadIdx.x; e < 2 * p.E; e += kThreads) r.mask[e] = 0;
  __syncthreads();
#pragma unroll
  for (int m = 0; m < kMost; ++m) {
    const int i = threadIdx.x + m * kThreads, e = expert[m], t = i / p.K;
    if (i < pairs) {
      if (e < 0 || e >= p.E) {
        s.bad = 1;
      } else {
        const uint32_t bit = 1u << (t & 31);
        if (atomicOr(&r.mask[2 * e + (t >> 5)], bit) & bit) s.bad = 1;  // repeated within the token
      }
    }
  }
  __syncthreads();
  if (s.bad) return;  // the same for the whole CTA
  const int chunks = (p.E + 31) / 32;
  for (int c = warp; c < chunks; c += kThreads / 32) {
    const int e = c * 32 + lane;
    const int n = e < p.E ? __popc(r.mask[2 * e]) + __popc(r.mask[2 * e + 1]) : 0;
    const int rows = __reduce_add_sync(0xffffffffu, n), most = __reduce_max_sync(0xffffffffu, n);
    const int entries = __reduce_add_sync(0xffffffffu, (n + kN - 1) / kN);
    if (lane == 0) {
      atomicMax(&s.most_rows, min(most, kN));
      s.warp_active[c] = entries;
      s.warp_rows[c] = rows;
    }
  }
  __syncthreads();
  for (int c = warp; c < chunks; c += kThreads / 32) {
    const int e = c * 32 + lane;
    const int n = e < p.E ? __popc(r.mask[2 * e]) + __popc(r.mask[2 * e + 1]) : 0;
    const int base = __reduce_add_sync(0xffffffffu, lane < c ? s.warp_active[lane] : 0);
    const int base_row = __reduce_add_sync(0xffffffffu, lane < c ? s.warp_rows[lane] : 0);
    const int entries = (n + kN - 1) / kN;
    int sum = n << 16 | entries;  // both running sums at once: at most 1024 rows
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += up;
    }
    if (n > 0) {
      const int a = base + (sum & 0xffff) - entries, row = base_row + (sum >> 16) - n;
      r.row_of[e] = row;
      for (int k = 0; k < entries; ++k) {
        r.active[a + k] = e;
        r.first[a + k] = row + k * kN;
        r.count[a + k] = min(n - k * kN, kN);
      }
    }
    if (c == chunks - 1 && lane == 31) s.n_active = base + (sum & 0xffff);
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < kMost; ++m) {
    const int i = threadIdx.x + m * kThreads, e = expert[m], t = i / p.K;
    if (i < pairs) {
      const uint64_t mask = static_cast<uint64_t>(r.mask[2 * e + 1]) << 32 | r.mask[2 * e];
      const int row = r.row_of[e] + __popcll(mask & ((1ull << t) - 1));
      r.token[row] = t;
      r.weight[row] = weight[m];
    }
  }
  __syncthreads();
}

// The same list for rows that come grouped: expert e's are [offsets[e], offsets[e+1]).
__device__ __forceinline__ void build_groups(const Routing& r, RoutingShared& s, const DecodeParams& p, int kN) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, chunks = (p.E + 31) / 32;
  if (threadIdx.x == 0) s.bad = 0, s.most_rows = 1;
  // Clamped: a damaged table cannot lead outside the buffers.
  auto rows_of = [&](int e, int& lo) {
    lo = 0;
    if (e >= p.E) return 0;
    if (!p.offsets) return p.T;  // one expert
    lo = min(max(p.offsets[e], 0), p.T);
    return min(max(p.offsets[e + 1], lo), p.T) - lo;
  };
  __syncthreads();
  for (int c = warp; c < chunks; c += kThreads / 32) {
    int lo;
    const int n = rows_of(c * 32 + lane, lo);
    const int entries = __reduce_add_sync(0xffffffffu, (n + kN - 1) / kN), most = __reduce_max_sync(0xffffffffu, n);
    if (lane == 0) {
      atomicMax(&s.most_rows, min(most, kN));
      s.warp_active[c] = entries;
    }
  }
  __syncthreads();
  // Offsets out of order may give rows to several experts: no more entries
  // than the list has room for.
  const int room = max_active(p.T, p.E, kN);
  for (int c = warp; c < chunks; c += kThreads / 32) {
    int lo;
    const int e = c * 32 + lane, n = rows_of(e, lo), entries = (n + kN - 1) / kN;
    const int base = __reduce_add_sync(0xffffffffu, lane < c ? s.warp_active[lane] : 0);
    int sum = entries;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += up;
    }
    for (int k = 0; k < entries; ++k) {
      const int a = base + sum - entries + k;
      if (a < room) {
        r.active[a] = e;
        r.first[a] = lo + k * kN;
        r.count[a] = min(n - k * kN, kN);
      }
    }
    if (c == chunks - 1 && lane == 31) s.n_active = min(base + sum, room);
  }
  __syncthreads();
}

// ---- what the kernels share ---------------------------------------------------
struct Barriers {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[kMaxBufs], acc_empty[kMaxBufs];
  uint64_t drained;
  uint32_t tmem;
  int gave_up;
};

__device__ __forceinline__ void init_barriers(Barriers& b) {
  for (int i = 0; i < kMaxStages; ++i) {
    ptx::mbar_init(&b.full[i], 1);
    ptx::mbar_init(&b.empty[i], 1);
  }
  for (int i = 0; i < kMaxBufs; ++i) {
    ptx::mbar_init(&b.acc_full[i], 1);
    ptx::mbar_init(&b.acc_empty[i], 4);
  }
  ptx::mbar_init(&b.drained, 1);
  b.gave_up = 0;
}

// A place in the ring and how often it has been passed, counted without
// divisions: one thread issues all loads, another all matrix instructions, and
// each has to keep up with the memory.
struct Place {
  uint32_t st = 0, phase = 0;
  __device__ __forceinline__ void next(uint32_t stages) {
    if (++st == stages) st = 0, phase ^= 1;
  }
};

// The scratch that build_routing wrote lies where TMA will write next.
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async;" ::: "memory"); }

// Waits (bounded) for the loads of iterations [it - stages, it), which may still
// be in flight: they write to this CTA's shared memory, so it does not end or use
// the ring otherwise before them, whichever warp gave up.
__device__ __forceinline__ void drain_loads(Barriers& b, uint32_t it, uint32_t stages, uint32_t test_drop) {
  const unsigned long long start = tc::now_ns();
  for (uint32_t j = it > stages ? it - stages : 0; j < it; ++j)
    if (j != test_drop) tc::settle(&b.full[j % stages], (j / stages) & 1, start);
}

__device__ __forceinline__ int chunks_of(int rows) { return (rows + kChunk - 1) / kChunk; }

// One thread issues 128 weight rows x 16 * chunks token rows over 128 of K.
__device__ __forceinline__ void mma_tile(uint32_t tmem, const uint8_t* w, const uint8_t* x, int chunks) {
  const uint32_t instr = tc::instr_desc_e4m3(128, chunks * kChunk);
  const uint64_t wd = tc::smem_desc(w), xd = tc::smem_desc(x);
#pragma unroll
  for (int k = 0; k < kBlock / 32; ++k) tc::mma_e4m3(tmem, wd + 2 * k, xd + 2 * k, instr, k > 0);
}

__device__ __forceinline__ void finish_mma(Barriers& b) {  // nothing in flight when the tensor memory is freed
  if (tc::elect()) tc::commit(&b.drained);
  __syncwarp();
  tc::settle(&b.drained, 0, tc::now_ns());
}

__device__ __forceinline__ void store_out(const DecodeParams& p, int64_t to, float v) {
  if (p.out_f32) reinterpret_cast<float*>(p.out)[to] = v;
  else reinterpret_cast<__nv_bfloat16*>(p.out)[to] = __float2bfloat16_rn(v);
}

// Four columns of a row of out, whose rows are a multiple of 8 long.
__device__ __forceinline__ void store_out_4(const DecodeParams& p, int t, int column, float4 v) {
  const int64_t to = static_cast<int64_t>(t) * p.H + column;
  if (p.out_f32) {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + to) = v;
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    uint2 o = {*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi)};
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + to) = o;
  }
}

__host__ __device__ constexpr uint32_t tmem_columns(int n) { return n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : 256; }

// acc[c] += v[c] * scale[c] * f for 16 columns; scale in shared memory.
__device__ __forceinline__ void add_scaled(const uint32_t* v, const float* scale, unsigned long long ff,
                                           unsigned long long* acc) {
#pragma unroll
  for (int j = 0; j < kChunk; j += 4) {
    const float4 s = *reinterpret_cast<const float4*>(scale + j);
    acc[j / 2] = tc::fma2(tc::pack2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])),
                          tc::mul2(tc::pack2(s.x, s.y), ff), acc[j / 2]);
    acc[j / 2 + 1] = tc::fma2(tc::pack2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])),
                              tc::mul2(tc::pack2(s.z, s.w), ff), acc[j / 2 + 1]);
  }
}

// ---- first kernel -----------------------------------------------------------
// Unit: (expert number a, block j of 128 columns of h).  A thread of the
// epilogue owns column j * 128 + threadIdx.x of h.  Two CTAs share an SM: one
// CTA's routing and epilogues pass while the other streams.  The units that
// are left when every CTA has had the same number are split along K over
// groups of 2, 4 or 8 CTAs of a cluster, as far as the CTAs go.
// (gemm: 256 columns of the product, two a thread.)
enum Form { kDecode, kGlu, kGemm };
template <int kN, Form kForm>
__global__ void __launch_bounds__(kThreads, 2) row_groups_kernel(const __grid_constant__ DecodeParams p,
                                                                 uint32_t ring_bytes, uint32_t ranks) {
  extern __shared__ uint8_t s_raw[];
  __shared__ Barriers b;
  __shared__ uint64_t amax_ready[2];
  __shared__ RoutingShared rs;
  __shared__ __align__(16) float s_scale[4][2][kN];
  __shared__ __align__(16) float s_amax[2][kN][4];
  constexpr uint32_t kBufs = bufs(kN), kColumns = tmem_columns(kBufs * 2 * kN);
  uint8_t* ring = s_raw + ((1024 - (ptx::smem_addr(s_raw) & 1023)) & 1023);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const Routing r = routing_at(ring + ring_bytes, ring, p.T * p.K, p.E, kN);
  if (threadIdx.x == 0) {
    init_barriers(b);
    ptx::mbar_init(&amax_ready[0], 4);
    ptx::mbar_init(&amax_ready[1], 4);
    ptx::mbar_fence_init();
  }
  if (warp == kMmaWarp) tc::tmem_alloc(&b.tmem, kColumns);
  if (threadIdx.x == kTmaWarp * 32) {
    tc::tma_prefetch_map(&p.w13_map);
    tc::tma_prefetch_map(&p.x_map);
  }
  tc::fence_before();
  __syncthreads();
  ptx::wait_prerequisites();
  // From here on everything earlier in the stream is done, which few_rows'
  // early reads of topk_idx, topk_w and the weights rely on.  This CTA has its
  // tensor memory: CTAs of few_rows, which wait for this grid while they hold
  // theirs, cannot keep it from it.
  if (kForm == kDecode) {
    ptx::launch_dependents();
    build_routing(r, rs, p, kN);
  } else {
    build_groups(r, rs, p, kN);
  }
  tc::fence_after();
  // Stages as large as the fullest expert needs.
  const uint32_t stage_bytes = 2 * kTileBytes + chunks_of(rs.most_rows) * kChunk * kBlock;
  const uint32_t stages = min(ring_bytes / stage_bytes, static_cast<uint32_t>(kMaxStages));
  const int jb = kForm == kGemm ? (p.I + 255) / 256 : p.I / kBlock, kb_all = (p.H + kBlock - 1) / kBlock;
  const int units = rs.bad ? 0 : rs.n_active * jb;
  const int grid = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
  int split = 1;  // CTAs that share one of the last units
  const int whole = units / grid * grid, left = units - whole;
  while (split < static_cast<int>(ranks) && left * split * 2 <= grid) split *= 2;
  // This CTA's units: cta, cta + grid, ... below `whole` (or all, without a
  // split), all of K; then its share of unit `shared`.
  const int end = split > 1 ? whole : units, part = cta % split;
  const int shared = split > 1 && whole + cta / split < units ? whole + cta / split : -1;
  struct Span {
    int u, kb0, kb_n;
  };
  auto first_span = [&]() {
    if (cta < end) return Span{cta, 0, kb_all};
    return Span{shared, part * kb_all / split, (part + 1) * kb_all / split - part * kb_all / split};
  };
  auto next_span = [&](Span v) {  // u < 0: no more
    if (v.u == shared) return Span{-1, 0, 0};
    if (v.u + grid < end) return Span{v.u + grid, 0, kb_all};
    return Span{shared, part * kb_all / split, (part + 1) * kb_all / split - part * kb_all / split};
  };
  if (kForm == kDecode && blockIdx.x == 0 && threadIdx.x == 0) *p.status = rs.bad ? MOE_EROUTE : MOE_OK;
  bool ok = true;

  unsigned long long gate[kN / 2], up[kN / 2];
  int round = 0;  // units this CTA has finished
  // Epilogue warps: h of the unit's token rows from the sums, quantised.
  auto finish = [&](int u, int round) -> bool {
    const int a = u / jb, j = u - a * jb, row0 = r.first[a], n = r.count[a];
    if (kForm == kGemm) {
#pragma unroll
      for (int c0 = 0; c0 < kN; c0 += kChunk) {
        if (c0 < n) {
#pragma unroll
          for (int c = c0; c < c0 + kChunk; ++c) {
            const float v0 = c & 1 ? tc::hi2(gate[c / 2]) : tc::lo2(gate[c / 2]);
            const float v1 = c & 1 ? tc::hi2(up[c / 2]) : tc::lo2(up[c / 2]);
            const int column = j * 256 + static_cast<int>(threadIdx.x);
            const int64_t to = static_cast<int64_t>(row0 + c) * p.I + column;
            if (c < n) {
              if (column < p.I) store_out(p, to, v0);
              if (column + 128 < p.I) store_out(p, to + 128, v1);
            }
          }
        }
      }
      return true;
    }
    float (*amax)[4] = s_amax[round & 1];  // in turn: a warp one unit ahead does not overwrite
#pragma unroll
    for (int c0 = 0; c0 < kN; c0 += kChunk) {
      if (c0 < n) {
        float h[kChunk];
        uint32_t top[kChunk];
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
          const int c = c0 + i;
          const float g = c & 1 ? tc::hi2(gate[c / 2]) : tc::lo2(gate[c / 2]);
          const float v = c & 1 ? tc::hi2(up[c / 2]) : tc::lo2(up[c / 2]);
          // Of a denominator beyond 2^126 the quotient becomes 0; it is below 2^-119 there.
          h[i] = __fdividef(g, 1.0f + expf(-g)) * v;
          top[i] = __float_as_uint(fabsf(h[i]));
        }
#pragma unroll
        for (int i = 0; i < kChunk; ++i) top[i] = __reduce_max_sync(0xffffffffu, top[i]);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
          if (lane == 0) amax[c0 + i][warp] = __uint_as_float(top[i]);
          if (i & 1) gate[(c0 + i) / 2] = tc::pack2(h[i - 1], h[i]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&amax_ready[round & 1]);
    const bool all = tc::wait(&amax_ready[round & 1], (round >> 1) & 1, &b.gave_up);
    if (!__all_sync(0xffffffffu, all)) return false;
    uint8_t* dst = p.hq + static_cast<int64_t>(row0) * p.I + j * kBlock + threadIdx.x;
    // A lane computes the scale of its column of tokens; all use it.
#pragma unroll
    for (int c0 = 0; c0 < kN; c0 += 32) {
      if (c0 < n) {
        const float4 m = *reinterpret_cast<const float4*>(amax[c0 + (lane & (kN < 32 ? kN - 1 : 31))]);
        const float top = fmaxf(fmaxf(m.x, m.y), fmaxf(m.z, m.w));
        const float scale = top > 0.0f ? __fdiv_rn(fmaxf(top, kTinyAmax), 448.0f) : 1.0f;
        const float inv = __fdiv_rn(1.0f, scale);
        if (warp == 0 && c0 + lane < n) p.h_scales[static_cast<int64_t>(row0 + c0 + lane) * jb + j] = scale;
#pragma unroll
        for (int i0 = 0; i0 < 32 && c0 + i0 < kN; i0 += kChunk) {
          if (c0 + i0 < n) {
#pragma unroll
            for (int i = i0; i < i0 + kChunk; ++i) {
              const int c = c0 + i;
              const float h = c & 1 ? tc::hi2(gate[c / 2]) : tc::lo2(gate[c / 2]);
              const float f = __shfl_sync(0xffffffffu, inv, i);
              const uint8_t q = static_cast<uint8_t>(fp8q::e4m3x2(__fmul_rn(h, f), 0.0f));
              if (c < n) dst[static_cast<int64_t>(c) * p.I] = q;
            }
          }
        }
      }
    }
    return true;
  };

  if (warp == kTmaWarp) {
    fence_async_proxy();
    uint32_t it = 0;
    Place at;
    for (Span v = first_span(); ok && v.u >= 0; v = next_span(v)) {
      const int a = v.u / jb, j = v.u - a * jb;
      const int w0 = kForm == kGemm ? r.active[a] * p.I + j * 256 : r.active[a] * 2 * p.I + j * kBlock;
      const int w1 = w0 + (kForm == kGemm ? 128 : p.I);
      const int row0 = r.first[a], n = r.count[a], rows = chunks_of(n) * kChunk;
      int token[kN];  // rows past the expert's last repeat it; their columns are dropped
      if (kForm == kDecode) {
#pragma unroll
        for (int c = 0; c < kN; ++c) token[c] = r.token[row0 + min(c, n - 1)];
      }
      const uint32_t bytes = 2 * kTileBytes + rows * kBlock;
      const int k_end = (v.kb0 + v.kb_n) * kBlock;
      for (int k = v.kb0 * kBlock; k < k_end; k += kBlock, ++it) {
        ok = it < stages || tc::wait(&b.empty[at.st], at.phase ^ 1, &b.gave_up);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (tc::elect() && it != p.test_drop) {
          uint8_t* to = ring + at.st * stage_bytes;
          uint64_t* full = &b.full[at.st];
          ptx::mbar_arrive_expect_tx(full, bytes);
          tc::tma_load_2d(to, &p.w13_map, k, w0, full);
          tc::tma_load_2d(to + kTileBytes, &p.w13_map, k, w1, full);
          if (kForm != kDecode)
            for (int c = 0; c < rows; c += kChunk)
              tc::tma_load_2d(to + 2 * kTileBytes + c * kBlock, &p.x_map, k, row0 + c, full);
#pragma unroll
          for (int c = 0; c < kN; c += 4)
            if (kForm == kDecode && c < rows)
              tc::tma_gather4(to + 2 * kTileBytes + c * kBlock, &p.x_map, k, token[c], token[c + 1], token[c + 2],
                              token[c + 3], full);
        }
        __syncwarp();
        at.next(stages);
      }
    }
    drain_loads(b, it, stages, p.test_drop);
  } else if (warp == kMmaWarp) {
    const uint32_t tmem = __shfl_sync(0xffffffffu, b.tmem, 0);
    uint32_t it = 0;
    Place at;
    for (Span v = first_span(); ok && v.u >= 0; v = next_span(v)) {
      const int a = v.u / jb, chunks = chunks_of(r.count[a]);
      for (int kb = 0; kb < v.kb_n; ++kb, ++it) {
        const uint32_t buf = it % kBufs;
        ok = (it < kBufs || tc::wait(&b.acc_empty[buf], (it / kBufs - 1) & 1, &b.gave_up)) &&
             tc::wait(&b.full[at.st], at.phase, &b.gave_up);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc::fence_after();
        if (tc::elect()) {
          const uint8_t* w = ring + at.st * stage_bytes;
          mma_tile(tmem + buf * 2 * kN, w, w + 2 * kTileBytes, chunks);
          mma_tile(tmem + (buf * 2 + 1) * kN, w + kTileBytes, w + 2 * kTileBytes, chunks);
          tc::commit(&b.acc_full[buf]);
          tc::commit(&b.empty[at.st]);
        }
        __syncwarp();
        at.next(stages);
      }
    }
    finish_mma(b);
  } else {
    const uint32_t lanes = b.tmem + (static_cast<uint32_t>(warp * 32) << 16);
    uint32_t it = 0;
    for (Span v = first_span(); ok && v.u >= 0; v = next_span(v), ++round) {
      const int a = v.u / jb, j = v.u - a * jb, row0 = r.first[a], n = r.count[a];
      // Rows of blocks of the weights' scales that this thread's columns lie in.
      const int blocks = (p.I + kBlock - 1) / kBlock, b0 = kForm == kGemm ? min(2 * j, blocks - 1) : j;
      const int b1 = kForm == kGemm ? min(2 * j + 1, blocks - 1) : jb + j;
      const float* sw = p.w13_scales +
                        static_cast<int64_t>(r.active[a]) * (kForm == kGemm ? blocks : 2 * blocks) * kb_all + v.kb0;
      const float *sg = sw + static_cast<int64_t>(b0) * kb_all, *su = sw + static_cast<int64_t>(b1) * kb_all;
      const float* sx[(kN + 31) / 32];
#pragma unroll
      for (int i = 0; i < (kN + 31) / 32; ++i) {
        const int row = row0 + min(lane + 32 * i, n - 1);
        sx[i] = p.x_scales + static_cast<int64_t>(kForm == kDecode ? r.token[row] : row) * kb_all + v.kb0;
      }
      // The token rows' scales of the next K block are read a block ahead, the
      // weights' of 32 blocks at a time (one a lane), 32 blocks ahead.
      float next[(kN + 31) / 32], lane_g, lane_u, ahead_g = 0.0f, ahead_u = 0.0f;
      auto read = [&](int kb) {
#pragma unroll
        for (int i = 0; i < (kN + 31) / 32; ++i)
          if (32 * i < n) next[i] = sx[i][kb];
      };
      auto read_weights = [&](int kb) {
        if (kb + lane < v.kb_n) ahead_g = sg[kb + lane], ahead_u = su[kb + lane];
      };
      read_weights(0);
      read(0);
#pragma unroll
      for (int c = 0; c < kN / 2; ++c) gate[c] = up[c] = 0;
      for (int kb = 0; kb < v.kb_n; ++kb, ++it) {
        const uint32_t buf = it % kBufs;
        float* scale = s_scale[warp][it & 1];
        if ((kb & 31) == 0) {
          lane_g = ahead_g, lane_u = ahead_u;
          read_weights(kb + 32);
        }
#pragma unroll
        for (int i = 0; i < (kN + 31) / 32; ++i)
          if (32 * i < n && lane + 32 * i < kN) scale[lane + 32 * i] = next[i];
        const float g = __shfl_sync(0xffffffffu, lane_g, kb & 31), u = __shfl_sync(0xffffffffu, lane_u, kb & 31);
        const unsigned long long fg = tc::pack2(g, g), fu = tc::pack2(u, u);
        if (kb + 1 < v.kb_n) read(kb + 1);
        ok = tc::wait(&b.acc_full[buf], (it / kBufs) & 1, &b.gave_up);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        __syncwarp();
        tc::fence_after();
#pragma unroll
        for (int c = 0; c < kN; c += kChunk) {
          if (c < n) {
            uint32_t d[kChunk];
            tc::tmem_load_16(lanes + buf * 2 * kN + c, d);
            tc::wait_loads();
            add_scaled(d, scale + c, fg, gate + c / 2);
            tc::tmem_load_16(lanes + (buf * 2 + 1) * kN + c, d);
            tc::wait_loads();
            add_scaled(d, scale + c, fu, up + c / 2);
          }
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&b.acc_empty[buf]);
      }
      if (v.u == shared) break;  // its sums are not complete
      if (ok) ok = finish(v.u, round);
    }
  }
  if (ranks > 1) {
    // The shared unit's sums meet in the first CTA of its group, through the
    // ring, which is free now: every load has been consumed.
    // [gate, up][token row][column]
    float* sums = reinterpret_cast<float*>(ring);
    const bool mine = warp < kTmaWarp && ok && shared >= 0;
    const int n = shared >= 0 ? r.count[shared / jb] : 0;
    __syncthreads();
    if (mine) {
#pragma unroll
      for (int c = 0; c < kN; c += 8) {
        if (c < n) {
#pragma unroll
          for (int i = c; i < c + 8; ++i) {
            sums[i * 128 + threadIdx.x] = i & 1 ? tc::hi2(gate[i / 2]) : tc::lo2(gate[i / 2]);
            sums[(kN + i) * 128 + threadIdx.x] = i & 1 ? tc::hi2(up[i / 2]) : tc::lo2(up[i / 2]);
          }
        }
      }
    }
    __syncthreads();
    tc::cluster_sync();
    if (mine && part == 0) {
      const uint32_t rank = tc::cluster_rank();
      for (uint32_t q = rank + 1; q < rank + split; ++q) {
#pragma unroll
        for (int c = 0; c < kN; c += 8) {
          if (c < n) {
            float v[16];  // all on their way before the first is needed
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              v[i] = ld_cluster(sums + (c + i) * 128 + threadIdx.x, q);
              v[8 + i] = ld_cluster(sums + (kN + c + i) * 128 + threadIdx.x, q);
            }
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              gate[(c + i) / 2] = tc::add2(gate[(c + i) / 2], tc::pack2(v[i], v[i + 1]));
              up[(c + i) / 2] = tc::add2(up[(c + i) / 2], tc::pack2(v[8 + i], v[9 + i]));
            }
          }
        }
      }
      finish(shared, round);
    }
    __syncthreads();
    tc::cluster_sync();  // no CTA leaves while its shared memory is being read
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (threadIdx.x == 0 && b.gave_up && p.status) atomicCAS(p.status, MOE_OK, MOE_ETIMEDOUT);
  if (warp == kMmaWarp) tc::tmem_free(b.tmem, kColumns);
}

// ---- second kernel ------------------------------------------------------------
// A cluster owns 128 columns of out.  Its CTAs share the (expert, K block)
// items, each a contiguous range; what an expert gives to token t is added to
// the CTA's s_out[t][column] when the CTA's part of that expert is complete
// (dense: one expert, row i is token i with weight 1).  The ring has a stage an
// item; the matrix warp and the epilogue take two items of an expert at a time,
// which halves what a turn costs the epilogue beside its sums.
template <int kN, bool kDense>
__global__ void __launch_bounds__(kThreads, 2)
    few_rows_kernel(const __grid_constant__ DecodeParams p, uint32_t ring_bytes, uint32_t ranks) {
  extern __shared__ uint8_t s_raw[];
  __shared__ Barriers b;
  __shared__ RoutingShared rs;
  __shared__ __align__(16) float s_scale[4][2][2][kN];  // [warp][buffer][item]
  constexpr uint32_t kBufs = bufs(kN), kColumns = tmem_columns(kBufs * 2 * kN);
  uint8_t* ring = s_raw + ((1024 - (ptx::smem_addr(s_raw) & 1023)) & 1023);
  float* s_out = reinterpret_cast<float*>(ring + ring_bytes);  // [T][128]
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  Routing r = {};
  if (threadIdx.x == 0) {
    init_barriers(b);
    ptx::mbar_fence_init();
  }
  if (warp == kMmaWarp) tc::tmem_alloc(&b.tmem, kColumns);
  if (threadIdx.x == kTmaWarp * 32) {
    tc::tma_prefetch_map(&p.w2_map);
    tc::tma_prefetch_map(&p.h_map);
  }
  tc::fence_before();
  if (kDense) {
    if (threadIdx.x == 0) rs.bad = 0, rs.n_active = 1, rs.most_rows = p.T;
    __syncthreads();
  } else {
    r = routing_at(reinterpret_cast<uint8_t*>(s_out + p.T * 128), ring, p.T * p.K, p.E, kN);
    build_routing(r, rs, p, kN);  // topk_idx and topk_w: see the first kernel's launch_dependents
  }
  tc::fence_after();
  const uint32_t stage_bytes = kTileBytes + chunks_of(rs.most_rows) * kChunk * kBlock;
  const uint32_t stages = min(ring_bytes / stage_bytes, static_cast<uint32_t>(kMaxStages));
  const int tile = static_cast<int>(blockIdx.x / ranks);
  const uint32_t rank = ranks > 1 ? tc::cluster_rank() : 0;
  const int kb_n = p.h_blocks;
  const int items = rs.bad ? 0 : rs.n_active * kb_n;
  const int it0 = static_cast<int>(static_cast<int64_t>(items) * rank / ranks);
  const int n = static_cast<int>(static_cast<int64_t>(items) * (rank + 1) / ranks) - it0;
  auto row0_of = [&](int a) { return kDense ? 0 : r.first[a]; };
  auto rows_of = [&](int a) { return kDense ? p.T : r.count[a]; };
  bool ok = true;

  if (warp == kTmaWarp) {
    {
      fence_async_proxy();
      // Weights and rows of an item go to one stage; the first stages get
      // their weights before h is ready, so the two walk separately.
      struct Walk {
        Place at;
        int a, kb, row, rows;
        uint32_t item;
      };
      auto enter = [&](Walk& v) {
        v.row = kDense ? tile * 128 : r.active[v.a] * p.H + tile * 128;
        v.rows = rows_of(v.a);
      };
      auto step = [&](Walk& v) {
        v.at.next(stages);
        ++v.item;
        if (++v.kb == kb_n) {
          v.kb = 0;
          if (++v.a < rs.n_active) enter(v);
        }
      };
      Walk w = {{}, it0 / kb_n, it0 % kb_n, 0, 0, 0};
      if (n > 0) enter(w);
      Walk h = w;
      auto load_w = [&]() {
        if (tc::elect() && w.item != p.test_drop) {
          uint64_t* full = &b.full[w.at.st];
          ptx::mbar_arrive_expect_tx(full, kTileBytes + chunks_of(w.rows) * kChunk * kBlock);
          tc::tma_load_2d(ring + w.at.st * stage_bytes, &p.w2_map, w.kb * kBlock, w.row, full);
        }
        __syncwarp();
        step(w);
      };
      auto load_h = [&]() {
        if (tc::elect() && h.item != p.test_drop) {
          const int row0 = row0_of(h.a);
          for (int c = 0; c < h.rows; c += kChunk)
            tc::tma_load_2d(ring + h.at.st * stage_bytes + kTileBytes + c * kBlock, &p.h_map, h.kb * kBlock, row0 + c,
                            &b.full[h.at.st]);
        }
        __syncwarp();
        step(h);
      };
      const int early = min(n, static_cast<int>(stages));
      if (kDense) ptx::wait_prerequisites();
      for (int i = 0; i < early; ++i) load_w();
      if (!kDense) ptx::wait_prerequisites();  // h
      for (int i = 0; i < early; ++i) load_h();
      int i = early;
      for (; i < n; ++i) {
        ok = tc::wait(&b.empty[w.at.st], w.at.phase ^ 1, &b.gave_up);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        load_w();
        load_h();
      }
      drain_loads(b, i, stages, p.test_drop);
    }
  } else if (warp == kMmaWarp) {
    const uint32_t tmem = __shfl_sync(0xffffffffu, b.tmem, 0);
    int a = it0 / kb_n, kb = it0 - a * kb_n;
    Place at;
    for (uint32_t i = 0, turn = 0; i < static_cast<uint32_t>(n); ++turn) {
      const uint32_t buf = turn % kBufs;
      const int two = i + 1 < static_cast<uint32_t>(n) && kb + 1 < kb_n ? 2 : 1, chunks = chunks_of(rows_of(a));
      ok = turn < kBufs || tc::wait(&b.acc_empty[buf], (turn / kBufs - 1) & 1, &b.gave_up);
      for (int m = 0; m < two; ++m, ++i) {
        ok = ok && tc::wait(&b.full[at.st], at.phase, &b.gave_up);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc::fence_after();
        if (tc::elect()) {
          const uint8_t* w = ring + at.st * stage_bytes;
          mma_tile(tmem + (buf * 2 + m) * kN, w, w + kTileBytes, chunks);
          tc::commit(&b.empty[at.st]);
          if (m + 1 == two) tc::commit(&b.acc_full[buf]);
        }
        __syncwarp();
        at.next(stages);
      }
      if (!ok) break;
      kb += two;
      if (kb == kb_n) kb = 0, ++a;
    }
    finish_mma(b);
  } else {
    float* mine = s_out + threadIdx.x;
    for (int t = 0; t < p.T; ++t) mine[t * 128] = 0.0f;
    ptx::wait_prerequisites();  // h_scales
    const uint32_t lanes = b.tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const float* sw = p.w2_scales + static_cast<int64_t>(tile) * kb_n;
    const int64_t sw_expert = static_cast<int64_t>(p.out_blocks) * kb_n;
    unsigned long long acc[kN / 2];
#pragma unroll
    for (int c = 0; c < kN / 2; ++c) acc[c] = 0;
    int a = it0 / kb_n, kb = it0 - a * kb_n;
    float next[2][(kN + 31) / 32], next_w[2];
    const float *hs[(kN + 31) / 32], *ws;
    int next_rows;
    auto enter = [&](int a) {  // the expert of the next turn's scales
      const int row0 = row0_of(a);
      next_rows = rows_of(a);
#pragma unroll
      for (int i = 0; i < (kN + 31) / 32; ++i)
        hs[i] = p.h_scales + static_cast<int64_t>(row0 + min(lane + 32 * i, next_rows - 1)) * kb_n;
      ws = sw + (kDense ? 0 : r.active[a]) * sw_expert;
    };
    auto read = [&](int kb, int two) {  // the scales of the next turn, a turn ahead
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        if (m < two) {
#pragma unroll
          for (int i = 0; i < (kN + 31) / 32; ++i)
            if (32 * i < next_rows) next[m][i] = ld_f32(hs[i] + kb + m);
          next_w[m] = ld_f32(ws + kb + m);
        }
      }
    };
    int two = n > 1 && kb + 1 < kb_n ? 2 : 1;
    if (n > 0) {
      enter(a);
      read(kb, two);
    }
    for (uint32_t i = 0, turn = 0; static_cast<int>(i) < n; ++turn) {
      const uint32_t buf = turn % kBufs;
      const int row0 = row0_of(a), rows = next_rows, two_now = two;
      unsigned long long f[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        f[m] = tc::pack2(next_w[m], next_w[m]);
#pragma unroll
        for (int c = 0; c < (kN + 31) / 32; ++c)
          if (32 * c < rows && lane + 32 * c < kN) s_scale[warp][turn & 1][m][lane + 32 * c] = next[m][c];
      }
      i += two_now;
      kb += two_now;
      const bool last = kb == kb_n;
      if (last) kb = 0, ++a;
      two = static_cast<int>(i) + 1 < n && kb + 1 < kb_n ? 2 : 1;
      if (static_cast<int>(i) < n) {
        if (last) enter(a);
        read(kb, two);
      }
      ok = tc::wait(&b.acc_full[buf], (turn / kBufs) & 1, &b.gave_up);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      __syncwarp();
      tc::fence_after();
#pragma unroll
      for (int c = 0; c < kN; c += kChunk) {
        if (c < rows) {
          uint32_t v[2][kChunk];
          tc::tmem_load_16(lanes + buf * 2 * kN + c, v[0]);
          if (two_now == 2) tc::tmem_load_16(lanes + (buf * 2 + 1) * kN + c, v[1]);
          tc::wait_loads();
          add_scaled(v[0], s_scale[warp][turn & 1][0] + c, f[0], acc + c / 2);
          if (two_now == 2) add_scaled(v[1], s_scale[warp][turn & 1][1] + c, f[1], acc + c / 2);
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&b.acc_empty[buf]);
      if (last || static_cast<int>(i) == n) {
#pragma unroll
        for (int c0 = 0; c0 < kN; c0 += 8) {
          if (c0 < rows) {
            float* at[8];
            float old[8], weight[8];
            if (!kDense) {  // the token rows of an expert are different tokens
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int row = row0 + min(c0 + i, rows - 1);
                at[i] = mine + r.token[row] * 128;
                weight[i] = r.weight[row];
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) old[i] = *at[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int c = c0 + i;
              const float v = c & 1 ? tc::hi2(acc[c / 2]) : tc::lo2(acc[c / 2]);
              if (c < rows) {
                if (kDense) mine[c * 128] = v;
                else *at[i] = fmaf(weight[i], v, old[i]);
              }
            }
          }
        }
#pragma unroll
        for (int c = 0; c < kN / 2; ++c) acc[c] = 0;
      }
    }
  }
  // Token t's sum is formed by rank t % ranks, in rank order; a warp takes a
  // token, a lane four columns.  One token at a time: this code runs once, and
  // fetching its instructions takes longer than its loads (64 tokens, 8 experts,
  // H 256, inner 512: 13.2 us; four tokens unrolled 13.6, a column a lane 14.5).
  __syncthreads();
  if (ranks > 1) tc::cluster_sync();
  const int column = tile * 128 + lane * 4;
  if (warp < 4 && !rs.bad && !b.gave_up && column < p.H) {
    for (int t = static_cast<int>(rank + warp * ranks); t < p.T; t += 4 * static_cast<int>(ranks)) {
      const float* at = s_out + t * 128 + lane * 4;
      float4 v[kMaxRanks];  // all on their way before the first is needed
#pragma unroll
      for (uint32_t q = 0; q < kMaxRanks; ++q)
        if (q < ranks) v[q] = q == rank ? *reinterpret_cast<const float4*>(at) : ld_cluster_v4(at, q);
      float4 sum = v[0];
#pragma unroll
      for (uint32_t q = 1; q < kMaxRanks; ++q)
        if (q < ranks) sum.x += v[q].x, sum.y += v[q].y, sum.z += v[q].z, sum.w += v[q].w;
      store_out_4(p, t, column, sum);
    }
  }
  __syncthreads();
  if (ranks > 1) tc::cluster_sync();  // no CTA leaves while its shared memory is being read
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (threadIdx.x == 0 && b.gave_up && p.status) atomicCAS(p.status, MOE_OK, MOE_ETIMEDOUT);
  if (warp == kMmaWarp) tc::tmem_free(b.tmem, kColumns);
}

cudaError_t launch_cluster(void (*kernel)(DecodeParams, uint32_t, uint32_t), const DecodeParams& p, size_t rest,
                           size_t ring, uint32_t ranks, unsigned groups, cudaStream_t stream) {
  cudaError_t err = set_kernel_limits(reinterpret_cast<const void*>(kernel), rest + ring);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(groups * ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = rest + ring;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ranks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, static_cast<uint32_t>(ring), ranks);
}

// Dynamic shared memory that a kernel's CTA may have when `per_sm` of them share
// an SM; cached per device and kernel.
size_t smem_budget(const void* kernel, int per_sm) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  static std::mutex mu;
  static std::map<std::pair<int, const void*>, size_t> known;  // static shared memory
  size_t fixed = 0;
  {
    std::lock_guard<std::mutex> lock(mu);
    auto it = known.find({dev, kernel});
    if (it == known.end()) {
      cudaFuncAttributes attr;
      if (cudaFuncGetAttributes(&attr, kernel) != cudaSuccess) return 0;
      // Both kernels want the SM's whole shared memory, so that they can meet on one SM.
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared) != cudaSuccess)
        return 0;
      it = known.emplace(std::make_pair(dev, kernel), attr.sharedSizeBytes).first;
    }
    fixed = it->second;
  }
  constexpr size_t kSm = 228 * 1024, kReserved = 1024;  // of each CTA, the driver's
  return kSm / per_sm - kReserved - fixed;
}

// Clusters of four CTAs of row_groups, two CTAs an SM, that are resident at one
// time: a cluster's CTAs share a GPC, so not every SM can be used.  Asked for
// CTAs that have an SM each and doubled (the query does not count on a second
// CTA).  Cached per device and kernel.
int resident_clusters(void (*kernel)(DecodeParams, uint32_t, uint32_t), size_t smem) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  static std::mutex mu;
  static std::map<std::pair<int, const void*>, int> known;
  std::lock_guard<std::mutex> lock(mu);
  auto it = known.find({dev, reinterpret_cast<const void*>(kernel)});
  if (it != known.end()) return it->second;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(4);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 4;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  known[{dev, reinterpret_cast<const void*>(kernel)}] = 2 * n;
  return 2 * n;
}

template <int kN, Form kForm>
cudaError_t launch_groups(const DecodeParams& p, int sms, cudaStream_t stream) {
  auto* kernel = row_groups_kernel<kN, kForm>;
  const int rows = p.T * p.K;
  const size_t rest = 1024 + routing_bytes(rows, p.E, kN, kForm == kDecode);
  const size_t budget = smem_budget(reinterpret_cast<const void*>(kernel), 2);
  if (budget < rest + 2 * kTileBytes + kN * kBlock) return cudaErrorInvalidConfiguration;
  const cudaError_t err = set_kernel_limits(reinterpret_cast<const void*>(kernel), budget);
  if (err != cudaSuccess) return err;
  const int64_t units =
      static_cast<int64_t>(max_active(rows, p.E, kN)) * (kForm == kGemm ? (p.I + 255) / 256 : p.I / kBlock);
  const int kb_n = (p.H + kBlock - 1) / kBlock;
  uint32_t ranks = 1;
  int64_t groups = units;
  if (units > 2 * sms) {
    // Several rounds: clusters of four, so that the last one can be split.  That
    // costs 1 to 5 % where it finds nothing to split, and pays with a long K: 64
    // tokens of 2, not split / split in us: H 1024, 320 units 46.9 / 54.2, 610
    // 70.3 / 71.5; H 2048, 308 60.6 / 59.0, 320 61.6 / 67.2, 610 91.1 / 92.5; H 4096,
    // 308 90.8 / 85.4, 320 92.0 / 91.6, 360 93.2 / 89.4, 610 117 / 118; H 7168, 308
    // 152 / 140, 320 155 / 149, 610 209 / 210.
    const int clusters = kb_n >= 32 ? std::min(resident_clusters(kernel, budget), 2 * sms / 4) : 0;
    ranks = clusters * 4 >= sms ? 4 : 1;
    groups = ranks > 1 ? clusters : 2 * sms;
  } else {
    // Too few units for two CTAs an SM: split them along K, eight blocks or
    // more each (one token, 128 units: 66.9 us unsplit, 65.1 us in twos).
    while (ranks < 8 && units * ranks <= sms && static_cast<int>(ranks) * 16 <= kb_n) ranks *= 2;
  }
  return launch_cluster(kernel, p, rest, budget - rest, ranks, static_cast<unsigned>(groups), stream);
}

template <int kN, bool kDense>
cudaError_t launch_few(const DecodeParams& p, int sms, cudaStream_t stream) {
  auto* kernel = few_rows_kernel<kN, kDense>;
  const int pairs = p.T * p.K;
  const size_t rest = 1024 + static_cast<size_t>(p.T) * 512 + (kDense ? 0 : routing_bytes(pairs, p.E, kN, true));
  const int64_t tiles = (p.H + 127) / 128;
  const int64_t items = static_cast<int64_t>(kDense ? 1 : max_active(pairs, p.E, kN)) * p.h_blocks;
  // Up to 16 tokens two CTAs share an SM, else their sums leave too little for the
  // rings.  As many CTAs a tile as are resident at once, with four items each or
  // more.  Measured in us, clusters of 1 / 2 / 4: a layer of 8 tokens, 2 of 8 experts,
  // H 256, inner 512 16.9 / 13.6 / 11.7; 64 tokens, 6 of 64, H 4096, inner 1408 314 / 218 /
  // 173; 32 tokens, 1 of 8, H 7168, inner 2048 81.9 / 67.6 / 76.3 (not resident with 4);
  // 8 tokens, 1 of 8, H 16384, inner 512 36.7 / 36.8 / 41.5; dense, 16 rows: N 1024, K
  // 8192 18.8 / 12.6 / 9.0, N 16384, K 4096 15.6 / 15.3 / 19.1, N 256, K 512 (4 items)
  // 4.0 / 4.5 / 4.2, N 2048, K 128 (1 item) 3.3 / 4.4 / 4.4.
  const int per_sm = p.T <= 16 ? 2 : 1;
  uint32_t ranks = 1;
  while (ranks < kMaxRanks && tiles * ranks * 2 <= per_sm * sms && ranks * 2 * 4 <= items) ranks *= 2;
  const size_t stage = kTileBytes + kN * kBlock;
  const size_t budget = smem_budget(reinterpret_cast<const void*>(kernel), tiles * ranks > sms ? per_sm : 1);
  if (budget < rest + stage) return cudaErrorInvalidConfiguration;
  const size_t most = (items + ranks - 1) / ranks * stage;  // a stage for each item
  const size_t ring = std::min(std::min(budget, static_cast<size_t>(227 * 1024 - 8 * 1024)) - rest, most) / 16 * 16;
  return launch_cluster(kernel, p, rest, ring, ranks, static_cast<unsigned>(tiles), stream);
}

}  // namespace

cudaError_t launch_decode_layer(const DecodeParams& p, int sms, cudaStream_t stream) {
  // 16 columns need half of the registers and buffers a turn; an expert with more
  // rows has several entries, and its weights are read again.  Measured in us,
  // 32 / 16 columns, with T * K / E rows an expert on average, routed evenly:
  //   6   2 of 8 experts, H 4096, inner 2048 48.4 / 43.2; 4 of 16, H 4096, inner 1408
  //       53.2 / 53.4; 6 of 64, H 4096, inner 1408 173.8 / 172.5; 8 of 64, H 2048, inner
  //       768 77.3 / 71.5
  //   8   43.5 / 43.3, 53.4 / 53.4, -, 78.1 / 72.3
  //   12  43.8 / 43.8, 55.4 / 55.8; 16: 44.5 / 47.4, 57.3 / 61.9
  // and with all tokens on the same K experts: 6 28.5 / 29.8, 32.1 / 32.9, 47.4 / 49.5,
  // 30.4 / 31.4; 12 31.5 / 32.7, 39.2 / 35.0.
  const bool narrow = p.T <= 16 || p.T * p.K <= 8 * p.E;
  cudaError_t err = narrow ? launch_groups<16, kDecode>(p, sms, stream) : launch_groups<32, kDecode>(p, sms, stream);
  if (err != cudaSuccess) return err;
  return narrow ? launch_few<16, false>(p, sms, stream) : launch_few<32, false>(p, sms, stream);
}

cudaError_t launch_few_rows(const DecodeParams& p, int sms, cudaStream_t stream) {
  return p.T <= 16 ? launch_few<16, true>(p, sms, stream) : launch_few<32, true>(p, sms, stream);
}

cudaError_t launch_row_groups(const DecodeParams& p, bool glu, int sms, cudaStream_t stream) {
  return glu ? launch_groups<16, kGlu>(p, sms, stream) : launch_groups<16, kGemm>(p, sms, stream);
}

}  // namespace moe
