// Attention of every query of a chunk over its own selected blocks: for query
// row x at position p and query head h (KV head g = h / 4)
//     logits_t = scale * q[x][h] . K_t[g],  t in the selected blocks, t <= p
//     out[x][h] = sum_t softmax(logits)_t V_t[g],  lse = log sum_t exp(logits_t)
// with the rows read through the slot table, as sparse_attn.cu does for one
// query per request ("Оффлоадинг KV-кэша Qwen3.8-Flash-Next в RAM через vLLM без
// потери скорости декодирования", section "Механизм гибридного разреженного
// оффлоадинга": attention reads only the selected rows).
//
// Neighbouring queries select mostly the same blocks.  So 64 queries form a
// tile, the union of their blocks is attended densely on the tensor cores, and
// a bit per (query, block) masks the probabilities: a row is read once per tile
// and KV head instead of once per query that selects it (2048 queries over
// 2048 rows of 2 KiB each would read 8.6 GB).  Three kernels:
//  * plan: per tile the ascending list of blocks that any query selects, with
//    a 64-bit mask of the queries that do (bitmaps in shared memory);
//  * split: one CTA per (tile, KV head), or several where tiles are few, each
//    with a share of the tile's list; flash attention over 128 tokens (32 blocks)
//    at a time;
//  * join (where lists are split): log-sum-exp merge of a tile's shares.
//
// Split kernel.  The tile's 64 queries x 4 heads of the group are 256 rows, two
// halves of 128 = the tensor core's M: row = head * 32 + query, so a warp is a
// head and a lane a query.  Per half and 64 tokens: S = Q K^T (8 MMAs of
// K = 16, both operands in shared memory under the 128-byte swizzle), softmax
// by the half's 4 warps (thread = row), P (bf16) over S's own columns of tensor
// memory, O += P V (4 MMAs, P from tensor memory, V as an MN-major operand, so
// that rows lie in shared memory as they come).  Each half has two S tiles in
// turn: while one is in softmax, the other's P V and next S run.  Tensor
// memory: per half O (128 columns) and two S (64 each).
// Warps: 8 softmax, 4 loaders (cp.async of K[g], V[g] of each row, two stages
// of 128 tokens; FP8 codes are turned into f16 on the way, exactly, their scales
// going to the logits and the probabilities), 2 MMA (one per half).  All waits
// are bounded.
//
// The running maximum is each row's own, over the blocks that its query selects
// (a select per block; without it, 5 % faster, a row whose tokens lie far below
// some other query's would lose them).  It is followed lazily: O is rescaled
// only when the maximum has risen by 2^8.  Masked probabilities are 0, but 0
// times a value that is not finite is not: a row whose output is not finite, or
// whose sum has vanished, is computed again over its own tokens alone, by one
// warp in plain fp32 (attend_row), so that a token reaches only the queries that
// select it.
//
// Measured: 2048 BF16 queries, 2048 of 32768 tokens each (34 GFLOP of selected
// pairs; the unions, 2600 blocks here, make 175 of it), 167 us (plan 11, split
// 159): 0.54 of the measured bf16 rate on 128 of 152 SMs, bound by the softmax
// warps' instructions and by the hand-overs between them and the tensor core (the
// schedulers issue in 0.60 of the cycles).  The same with FP8 rows 272 us: the
// loaders' conversions and the products with both scales are added instructions.
// 14 FP8 draft queries of 8 requests (30 MB of rows at most) 31 us (33 with two codes
// a conversion: plan 8, split 27, join 4 each alone): five steps per CTA, each the latency of rows, conversion
// and softmax one after the other.  Not faster: K and V split over the loader warps (310 us at
// 2048 FP8 queries), the next step's codes loaded into the registers just stored
// (321), the idle half's warps on every other 64 tokens of a draft (43 where 39
// was), the dependent kernels' launches triggered early (38 where 38 was).
//
// Rounding: P to bf16 (at most 2^-8 of each term; the tensor core takes no wider
// type beside bf16 rows), and the output to bf16; the sum l is taken from the
// unrounded probabilities, S, O, m and l are fp32.  With FP8 rows P times the V
// scale goes in as f16: off by 2^-11 of itself, or by 2^-25 in units in which the
// largest of the row's products is 2^-6 at least, whatever the scales are and
// whoever else selects what (the reference follows the row's own products).
#include "attn_common.cuh"

namespace qsa {
namespace {

using namespace tc;
using namespace attn;

constexpr int kTileQueries = 64;                  // two halves of 32
constexpr int kStepBlocks = 32, kStepTokens = 4 * kStepBlocks;
constexpr int kSubTokens = kStepTokens / 2;       // tokens of one S tile
constexpr int kSoftWarps = 8, kLoadWarps = 4;
constexpr int kMmaWarps = 2;                      // one per half
constexpr int kThreads = 32 * (kSoftWarps + kLoadWarps + kMmaWarps);     // 448
constexpr int kRoleLoad = kSoftWarps, kRoleMma = kSoftWarps + kLoadWarps;
constexpr int kStages = 2;
constexpr int kPanel = 128 * 128;                 // 128 rows of 64 bf16
constexpr int kQBytes = 2 * 2 * kPanel;           // two halves, two panels of 64 dims
constexpr int kKvBytes = 2 * kPanel;              // K (or V) of a stage: two panels
constexpr int kStageBytes = 2 * kKvBytes;

// What the softmax of a step needs beside S.
struct StepMeta {
  uint32_t mine[2][32];         // [half][query]: bit b, the query selects block b of the step
  uint32_t valid[4];            // bit per token of the step: its row exists
  int32_t block[kStepBlocks];   // block ids
  int32_t special[4];           // per loader warp: a row is missing, or a block reaches past the first query
  uint32_t exps[4];             // FP8, per loader warp: bit e, a row has a V scale with the f16 exponent field e
};
struct __align__(16) Scales {   // FP8 rows
  float k[kStepTokens];         // K scale (times softmax scale and log2 e)
  float v[kStepTokens];         // V scale
  float size[kStepTokens];      // log2 of its size
};
constexpr int kOffKv = kQBytes;
constexpr int kOffMeta = kOffKv + kStages * kStageBytes;
// Metas outlive their K stage (the softmax of step j reads meta j while K of
// step j + 2 comes in), but not by three steps: K of step j + 3 comes after the
// S of step j + 1, that after the P of step j.
constexpr int kMetas = 4;
constexpr int kOffScales = kOffMeta + kMetas * (int)sizeof(StepMeta);
constexpr int kOffBar = kOffScales + kMetas * (int)sizeof(Scales);
// k_full[2], k_empty[2], v_full[2], v_empty[2], then per (half, 64 tokens)
// s_full[4], p_full[4], o_full[4], then q_full, done[2]
constexpr int kNumBars = 4 * kStages + 15;
constexpr int kOffSlot = (kOffBar + 8 * kNumBars + 15) / 16 * 16;
constexpr int kSmemBytes = kOffSlot + 16 + 1024;
static_assert(kSmemBytes <= 227 * 1024 && sizeof(StepMeta) % 16 == 0, "one CTA's shared memory");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColS = 256;        // + 128 per half

constexpr int kPlanThreads = 1024;
constexpr int kPlanWindow = 24576;                // blocks of one bitmap window (192 KiB)
constexpr int kRowFloats = kHeadDim + 2;          // partial of a row: O, m, l
constexpr int kMaxShares = 64;                    // where tiles are split: two tiles per lane
// A share's steps at least, where its tile has them: 4 queries of one request of
// 65536 tokens 26.8, 26.5, 27.6, 29.3 us with 1, 2, 3, 4.
constexpr int kLeastSteps = 2;

struct ChunkAttnParams {
  ChunkDesc c;
  int32_t tile0[kMaxUnits + 1];  // prefix sums of the tiles per unit
  const uint16_t* q;             // [rows][16][128] bf16 bits
  const int32_t* sel;            // [rows][k_max]
  const int32_t* n_sel;          // [rows]
  int32_t k_max;
  int32_t shares;                // CTAs per KV head: the tiles, or more, dealt out by share_of
  float scale_log2;              // |softmax_scale| * log2(e)
  float sign;                    // the scale's sign (goes into Q)
  uint16_t* out;                 // [rows][16][128] bf16 bits
  float* lse;                    // [rows][16] or nullptr
  int32_t cap;                   // list entries per tile (a multiple of 32)
  int32_t* count;                // [tiles]
  int32_t* block;                // [tiles][cap]
  uint32_t* mask;                // [tiles][2][cap]
  int2* dealt;                   // [tiles]: a tile's first share, and how many it has
  float* part;                   // [shares][4][256][kRowFloats]

  __device__ int unit_of_tile(int t) const {
    int lo = 0, hi = c.b.n_units - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tile0[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
  }
};

// ------------------------------------------------------- one row, plain fp32

// One warp, one query row x and head h: online softmax over the row's own
// selected tokens.  (Bad blocks and slots have been reported by the plan and
// the loaders.)  Slow, for values that are not finite only: where one V scale in
// 4096 is infinite, so that nearly every row comes here, 2048 FP8 queries take 47
// ms and 14 draft queries 1.4.
__device__ __noinline__ void attend_row(const ChunkAttnParams& p, int u, int x, int h) {
  const int lane = threadIdx.x & 31, g = h / kGroup;
  const bool fp8 = p.c.b.row_bytes == kRowBytesFp8;
  const int64_t pos = p.c.position(u, x);
  const float f = p.sign * p.scale_log2;
  const uint2 qv = reinterpret_cast<const uint2*>(p.q + ((int64_t)x * kQHeads + h) * kHeadDim)[lane];
  const float q[4] = {bf16_lo(qv.x) * f, bf16_hi(qv.x) * f, bf16_lo(qv.y) * f, bf16_hi(qv.y) * f};
  int nsel = p.n_sel[x];
  if (nsel < 0 || nsel > p.k_max) nsel = 0;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = 0; j < nsel; ++j) {
    const int64_t b = p.sel[(int64_t)x * p.k_max + j];
    if (b < 0 || 4 * b > pos) continue;
    for (int i = 0; i < 4 && 4 * b + i <= pos; ++i) {
      const uint8_t* row = row_source(p.c.b, u, 4 * b + i, kKernChunkAttn);
      if (!row) continue;
      const float4 k = row_values(row, g, lane, fp8);
      float s = fmaf(q[3], k.w, fmaf(q[2], k.z, fmaf(q[1], k.y, q[0] * k.x)));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      const float mn = fmaxf(m, s);
      const float a = mn == -INFINITY ? 1.f : exp2f(m - mn), e = s == -INFINITY ? 0.f : exp2f(s - mn);
      const float4 v = row_values(row, kKvHeads + g, lane, fp8);
      m = mn;
      l = fmaf(l, a, e);
      acc = make_float4(fmaf(acc.x, a, e * v.x), fmaf(acc.y, a, e * v.y), fmaf(acc.z, a, e * v.z),
                        fmaf(acc.w, a, e * v.w));
    }
  }
  const float r = l == 0.f ? 0.f : 1.f / l;      // no tokens: zeros; NaN stays
  reinterpret_cast<uint2*>(p.out + ((int64_t)x * kQHeads + h) * kHeadDim)[lane] =
      make_uint2(pack_bf16(acc.x * r, acc.y * r), pack_bf16(acc.z * r, acc.w * r));
  if (p.lse && lane == 0) p.lse[(int64_t)x * kQHeads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ------------------------------------------------------------------- plan

// One CTA per tile.  In windows of kPlanWindow blocks: a 64-bit query mask per
// block in shared memory, set from the tile's selections (a warp's lanes read
// consecutive entries of one query), then compacted in block order: warp w owns
// a run of blocks, 32 at a time (each lane taking 32 blocks' bits instead would
// read the masks of neighbouring words from one bank: 178 -> 183 us for the
// whole call at 2048 queries).
constexpr int kPlanWarps = kPlanThreads / 32;
__global__ void __launch_bounds__(kPlanThreads, 1) chunk_plan_kernel(const __grid_constant__ ChunkAttnParams p,
                                                                   int window) {
  extern __shared__ __align__(16) uint32_t bits0[];    // [window] queries 0-31, then [window] queries 32-63
  uint32_t* bits1 = bits0 + window;
  __shared__ uint32_t s_warp[kPlanWarps];
  const int tile = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int u = p.unit_of_tile(tile);
  const int i0 = (tile - p.tile0[u]) * kTileQueries;
  const int tokens = p.c.unit_tokens(u);
  const int nq = tokens - i0 < kTileQueries ? tokens - i0 : kTileQueries;
  const int x0 = p.c.row0[u] + i0;
  const int64_t last = p.c.position(u, x0 + nq - 1) / 4;      // the tile's last block
  int32_t* block = p.block + (int64_t)tile * p.cap;
  uint32_t* mask0 = p.mask + (int64_t)tile * 2 * p.cap;
  uint32_t* mask1 = mask0 + p.cap;
  int at = 0;
  for (int64_t w0 = 0; w0 <= last; w0 += window) {
    const int size = last + 1 - w0 < window ? (int)(last + 1 - w0) : window;
    for (int i = tid; i < (size + 3) / 4; i += kPlanThreads) {
      reinterpret_cast<uint4*>(bits0)[i] = make_uint4(0, 0, 0, 0);
      reinterpret_cast<uint4*>(bits1)[i] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    if (w0 == 0) grid_dependency_wait();               // the selection is read from here on
    // a warp takes 256 entries of one query at a time, all loads in flight
    const int turns = (p.k_max + 255) / 256;
    for (int i = warp; i < nq * turns; i += kPlanWarps) {
      const int q = i / turns, j0 = (i % turns) * 256 + lane;
      const int32_t* sel = p.sel + (int64_t)(x0 + q) * p.k_max;
      const int nsel = p.n_sel[x0 + q];
      const bool bad = nsel < 0 || nsel > p.k_max;
      int32_t id[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) id[e] = j0 + 32 * e < p.k_max ? sel[j0 + 32 * e] : 0;
      if (bad) {
        if (w0 == 0 && lane == 0) report_error(p.c.b.err, QSA_ERR_BAD_BLOCK, kKernChunkAttn, nsel);
        continue;
      }
      const int64_t lim = p.c.position(u, x0 + q) / 4;
      uint32_t* bits = q < 32 ? bits0 : bits1;
      const uint32_t bit = 1u << (q & 31);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (j0 + 32 * e >= nsel) continue;
        if (id[e] < 0 || id[e] > lim) {
          if (w0 == 0) report_error(p.c.b.err, QSA_ERR_BAD_BLOCK, kKernChunkAttn, id[e]);
        } else if (id[e] >= w0 && id[e] < w0 + size) {
          atomicOr(bits + (id[e] - w0), bit);
        }
      }
    }
    __syncthreads();
    const int run = ((size + kPlanWarps - 1) / kPlanWarps + 31) / 32 * 32;
    const int b0 = warp * run, b1 = b0 + run < size ? b0 + run : size;
    // 256 blocks at a time, all their words in flight
    constexpr int kTurn = 8;
    uint32_t m0[kTurn], m1[kTurn];
    auto load = [&](int b) {
#pragma unroll
      for (int i = 0; i < kTurn; ++i) {
        const int k = b + 32 * i + lane;
        m0[i] = k < b1 ? bits0[k] : 0u;
        m1[i] = k < b1 ? bits1[k] : 0u;
      }
    };
    uint32_t n = 0;
    for (int b = b0; b < b1; b += 32 * kTurn) {
      load(b);
#pragma unroll
      for (int i = 0; i < kTurn; ++i) n += __popc(__ballot_sync(0xFFFFFFFFu, (m0[i] | m1[i]) != 0));
    }
    if (lane == 0) s_warp[warp] = n;
    __syncthreads();
    uint32_t v = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += y;
    }
    int o = at + (int)(__shfl_sync(0xFFFFFFFFu, v, warp) - n);
    for (int b = b0; b < b1; b += 32 * kTurn) {
      load(b);
#pragma unroll
      for (int k = 0; k < kTurn; ++k) {
        const uint32_t some = __ballot_sync(0xFFFFFFFFu, (m0[k] | m1[k]) != 0);
        if (m0[k] | m1[k]) {
          const int i = o + __popc(some & ((1u << lane) - 1u));
          block[i] = (int32_t)(w0 + b + 32 * k + lane);
          mask0[i] = m0[k];
          mask1[i] = m1[k];
        }
        o += __popc(some);
      }
    }
    at += (int)__shfl_sync(0xFFFFFFFFu, v, 31);
    __syncthreads();
  }
  if (tid == 0) {
    p.count[tile] = at;
    // the unit's planned misses are in their hot rows (launch_hot_complete)
    if (p.c.b.u[u].hot_base >= 0) p.c.b.hot_pend_on[p.c.b.unit_state(u)] = 0;
  }
}
static_assert(kPlanWarps == 32, "one lane per warp in the scan");

// ------------------------------------------------------------------ split

// Which part of which tile share c is: where there are more shares than tiles,
// every tile gets ceil(steps / q) of them (one at least), q the smallest number
// of steps that the shares suffice for, so that the longest share is as short as
// it can be, whatever the lists' lengths.  Whole warps; false: nothing is left
// for share c.
__device__ __forceinline__ bool share_of(const ChunkAttnParams& p, int c, int* tile, int* split, int* n) {
  const int tiles = p.tile0[p.c.b.n_units], lane = threadIdx.x & 31;
  *tile = c;
  *split = 0;
  *n = 1;
  if (p.shares == tiles) return true;
  int steps[2], total = 0, longest = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    steps[i] = lane + 32 * i < tiles ? (p.count[lane + 32 * i] + kStepBlocks - 1) / kStepBlocks : 0;
    total += steps[i];
    longest = steps[i] > longest ? steps[i] : longest;
  }
  total = __reduce_add_sync(0xFFFFFFFFu, total);
  longest = __reduce_max_sync(0xFFFFFFFFu, longest);
  auto shares = [&](int i, int q) {                  // of tile lane + 32 i
    return lane + 32 * i >= tiles ? 0 : (steps[i] > q ? (steps[i] + q - 1) / q : 1);
  };
  int q = (total + p.shares - 1) / p.shares;
  q = q < kLeastSteps ? kLeastSteps : q;
  for (int enough = longest > q ? longest : q; q < enough;) {
    const int mid = (q + enough) / 2;
    if (__reduce_add_sync(0xFFFFFFFFu, shares(0, mid) + shares(1, mid)) <= p.shares) enough = mid;
    else q = mid + 1;
  }
  const int got[2] = {shares(0, q), shares(1, q)};
  int before = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int upto = got[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += y;
    }
    upto += before;
    const uint32_t mine = __ballot_sync(0xFFFFFFFFu, upto > c);
    if (mine) {
      const int l = __ffs(mine) - 1;
      *tile = 32 * i + l;
      *n = __shfl_sync(0xFFFFFFFFu, got[i], l);
      *split = c - (__shfl_sync(0xFFFFFFFFu, upto, l) - *n);
      return true;
    }
    before = __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  return false;
}

// The tokens of 64 c + 4 b .. + 3 of a step that exist and that position pos
// sees, a bit each.
__device__ __forceinline__ uint32_t seen_tokens(const StepMeta& sm, int c, int b, int64_t pos) {
  const int64_t left = pos - 4 * (int64_t)sm.block[16 * c + b];    // tokens of the block that pos sees, - 1
  return (left >= 3 ? 0xFu : (left < 0 ? 0u : (2u << (int)left) - 1u)) & (sm.valid[2 * c + (b >> 3)] >> (4 * (b & 7)));
}

// FP8: the largest logit + log2 (V scale) of a row's tokens among 64, each by its
// own scale (2048 queries where every 64 tokens need it: 272 -> 340 us).  S is read
// from tensor memory for this alone: among the registers of the usual path the
// scales would spill (309 us for rows that never come here).
__device__ __forceinline__ float wide_max(uint32_t colS, const StepMeta& sm, const Scales& sc, int c, uint32_t mine,
                                          bool special, int64_t pos, float f) {
  float most = -INFINITY;
#pragma unroll 1
  for (int b0 = 0; b0 < kSubTokens / 4; b0 += 4) {
    uint32_t x[16];
    ld16(colS + 4u * (uint32_t)b0, x);
    wait_ld();
    reg_fence(x);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int t = kSubTokens * c + 4 * (b0 + b);
      const float4 k = *reinterpret_cast<const float4*>(&sc.k[t]), s = *reinterpret_cast<const float4*>(&sc.size[t]);
      float y[4] = {fmaf(__uint_as_float(x[4 * b]) * k.x, f, s.x), fmaf(__uint_as_float(x[4 * b + 1]) * k.y, f, s.y),
                    fmaf(__uint_as_float(x[4 * b + 2]) * k.z, f, s.z), fmaf(__uint_as_float(x[4 * b + 3]) * k.w, f, s.w)};
      if (special) {
        const uint32_t seen = seen_tokens(sm, c, b0 + b, pos);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!((seen >> i) & 1u)) y[i] = -INFINITY;
      }
      const float top = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
      most = fmaxf(most, (mine >> (b0 + b)) & 1u ? top : -INFINITY);
    }
  }
  return most;
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1) chunk_split_kernel(const __grid_constant__ ChunkAttnParams p) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  StepMeta* meta = reinterpret_cast<StepMeta*>(smem + kOffMeta);
  Scales* scales = reinterpret_cast<Scales*>(smem + kOffScales);
  const uint32_t bars = sb + kOffBar;
  auto k_full = [&](int i) { return bars + 8u * (uint32_t)i; };
  auto k_empty = [&](int i) { return bars + 8u * (uint32_t)(kStages + i); };
  auto v_full = [&](int i) { return bars + 8u * (uint32_t)(2 * kStages + i); };
  auto v_empty = [&](int i) { return bars + 8u * (uint32_t)(3 * kStages + i); };
  auto s_full = [&](int h, int c) { return bars + 8u * (uint32_t)(4 * kStages + 2 * h + c); };
  auto p_full = [&](int h, int c) { return bars + 8u * (uint32_t)(4 * kStages + 4 + 2 * h + c); };
  auto o_full = [&](int h, int c) { return bars + 8u * (uint32_t)(4 * kStages + 8 + 2 * h + c); };
  const uint32_t q_full = bars + 8u * (uint32_t)(4 * kStages + 12);
  auto done = [&](int h) { return bars + 8u * (uint32_t)(4 * kStages + 13 + h); };
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + kOffSlot);
  __shared__ float row_factor[kFp8 ? 256 : 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  ErrorWord* err = p.c.b.err;

  // grid: share x KV head
  const int g = blockIdx.y;
  int tile, split, splits;
  grid_dependency_wait();
  if (!share_of(p, blockIdx.x, &tile, &split, &splits)) return;
  if (g == 0 && split == 0 && tid == 0) p.dealt[tile] = make_int2(blockIdx.x, splits);
  const int u = p.unit_of_tile(tile);
  const int i0 = (tile - p.tile0[u]) * kTileQueries;
  const int tokens = p.c.unit_tokens(u);
  const int nq = tokens - i0 < kTileQueries ? tokens - i0 : kTileQueries;
  const int x0 = p.c.row0[u] + i0;
  const int halves = nq > 32 ? 2 : 1;
  const int64_t pos0 = p.c.position(u, x0);

  if (warp == kRoleMma) {
    tmem_alloc<kTmemCols>(slot);
    if (lane == 0) {
      for (int i = 0; i < kStages; ++i) {
        mbar_init(k_full(i), 32 * kLoadWarps);
        mbar_init(k_empty(i), (uint32_t)halves);
        mbar_init(v_full(i), 32 * kLoadWarps);
        mbar_init(v_empty(i), (uint32_t)halves);
      }
      for (int i = 0; i < 4; ++i) {
        mbar_init(s_full(i >> 1, i & 1), 2);
        mbar_init(p_full(i >> 1, i & 1), 128);
        mbar_init(o_full(i >> 1, i & 1), 1);
      }
      mbar_init(q_full, 32 * kSoftWarps);
      mbar_init(done(0), 1);
      mbar_init(done(1), 1);
      mbar_fence_init();
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *slot;

  // The softmax warps bring Q in, while the loaders begin on K.
  if (warp < kSoftWarps) {
    // ---- Q: row head * 32 + query of each half, two panels of 64 dims.  Against
    // FP8 rows it goes in as f16, beside the K codes, which f16 holds exactly: a
    // row scaled by the power of two that puts its largest element into [2^14,
    // 2^15), the upper end of f16's range, where f16 holds a bf16 element exactly
    // down to 2^-31 of the largest and to 2^-39 of it below; the inverse goes to
    // the logits (row_factor).
    constexpr int kBatch = 4;                        // loads in flight
    for (int i0 = tid; i0 < halves * 128 * 16; i0 += kBatch * 32 * kSoftWarps) {      // (whole warps)
      uint4 in[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int i = i0 + b * 32 * kSoftWarps, c = i & 15, r = (i >> 4) & 127, q = (i >> 11) * 32 + (r & 31);
        in[b] = make_uint4(0, 0, 0, 0);
        if (q < nq)
          in[b] = reinterpret_cast<const uint4*>(p.q + ((int64_t)(x0 + q) * kQHeads + g * kGroup + (r >> 5)) * kHeadDim)[c];
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int i = i0 + b * 32 * kSoftWarps, c = i & 15, r = (i >> 4) & 127, h = i >> 11;
        uint4 v = in[b];
        const uint32_t flip = p.sign < 0.f ? 0x80008000u : 0u;
        v.x ^= flip; v.y ^= flip; v.z ^= flip; v.w ^= flip;
        if (kFp8) {
          uint32_t* w[4] = {&v.x, &v.y, &v.z, &v.w};
          float top = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) top = fmaxf(top, fmaxf(fabsf(bf16_lo(*w[k])), fabsf(bf16_hi(*w[k]))));
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));   // the row's 16 lanes
          int e = 0;
          if (top > 0.f && top < INFINITY) frexpf(top, &e);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __half2 o = __floats2half2_rn(ldexpf(bf16_lo(*w[k]), 15 - e), ldexpf(bf16_hi(*w[k]), 15 - e));
            *w[k] = *reinterpret_cast<const uint32_t*>(&o);
          }
          if (c == 0) row_factor[h * 128 + r] = ldexpf(1.f, e - 15);
        }
        *reinterpret_cast<uint4*>(smem + (h * 2 + (c >> 3)) * kPanel + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
      }
    }
    fence_async_smem();
    mbar_arrive(q_full);
    if (kFp8) asm volatile("bar.sync 1, %0;" ::"n"(32 * kSoftWarps) : "memory");      // row_factor
  }

  const int count = p.count[tile];
  const int all = (count + kStepBlocks - 1) / kStepBlocks;
  const int j0 = (int)((int64_t)all * split / splits), steps = (int)((int64_t)all * (split + 1) / splits) - j0;
  bool ok = true;

  if (warp >= kRoleLoad && warp < kRoleMma) {
    // ---- loaders: warp w brings tokens 32 w .. 32 w + 31 of a step, lane = token
    const int w = warp - kRoleLoad;
    const int32_t* block = p.block + (int64_t)tile * p.cap;
    const uint32_t* mask = p.mask + (int64_t)tile * 2 * p.cap;
    const int32_t* slots = p.c.b.slot_table + p.c.b.unit_row(u);
    const int64_t n = p.c.b.u[u].n;
    // At step j the block id of step j + 3, the slot of step j + 2 and the mask
    // word of step j + 1 are fetched.  Lane = token: block lane / 4 of the
    // warp's eight.
    const int first = j0 * kStepBlocks + 8 * w + (lane >> 2), stop = (j0 + steps) * kStepBlocks;
    auto block_id = [&](int j) {
      const int e = first + j * kStepBlocks;
      return e < stop && e < count ? block[e] : -1;
    };
    auto slot_of = [&](int32_t id) {                 // -2: no such token
      const int64_t t = 4 * (int64_t)id + (lane & 3);
      return id >= 0 && t < n ? slots[t] : -2;
    };
    // masks: loaders 2 and 3 (the schedulers of 0 and 1 have the MMA warps),
    // lane = block of the step
    const int mh = w - 2;
    auto mask_word = [&](int j) {
      const int e = (j0 + j) * kStepBlocks + lane;
      return mh >= 0 && mh < halves && j < steps && e < count ? mask[(int64_t)mh * p.cap + e] : 0u;
    };
    // FP8 rows are loaded into registers, with no copies in flight: rows two
    // steps ahead are on their way from HBM meanwhile (290 -> 282 us at 2048
    // queries; cp.async rows gain nothing from it, 179 -> 186 us)
    auto prefetch = [&](int32_t slot) {
      if (!kFp8 || slot < 0 || (int64_t)slot >= p.c.b.pool_rows) return;
      const uint8_t* r = p.c.b.pool + (int64_t)slot * p.c.b.row_bytes + g * kHeadDim;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(r));
      asm volatile("prefetch.global.L2 [%0];" ::"l"(r + kKvHeads * kHeadDim));
    };
    int32_t id = block_id(0), id_next = block_id(1), id_two = block_id(2);
    int32_t slot_now = slot_of(id), slot_next = slot_of(id_next);
    prefetch(slot_next);
    uint32_t word = mask_word(0);
    for (int j = 0; j < steps && ok; ++j) {
      const int st = j % kStages;
      const uint32_t turn = (uint32_t)(j / kStages - 1) & 1u;
      const int64_t t = 4 * (int64_t)id + (lane & 3);
      const uint8_t* src = nullptr;
      if (slot_now >= 0 && (int64_t)slot_now < p.c.b.pool_rows) {
        src = p.c.b.pool + (int64_t)slot_now * p.c.b.row_bytes;
      } else if (slot_now == -1 && p.c.b.u[u].host_rows) {
        src = p.c.b.u[u].host_rows + t * p.c.b.row_bytes;
      } else if (id >= 0 && t < n) {
        report_error(err, QSA_ERR_BAD_SLOT, kKernChunkAttn, ((int64_t)u << 40) | (t & 0xFFFFFFFFFFll));
      }
      const int32_t slot_two = slot_of(id_two), id_three = block_id(j + 3);
      const uint32_t word_next = mask_word(j + 1);
      if (j >= kStages) ok = mbar_wait_warp(k_empty(st), turn, err, kKernChunkAttn);
      if (!ok) break;
      const uint32_t kdst = kOffKv + st * kStageBytes + 32 * w * 128, vdst = kdst + kKvBytes;
      const uintptr_t from = reinterpret_cast<uintptr_t>(src);
      StepMeta& m = meta[j % kMetas];
      auto write_meta = [&]() {
        const uint32_t there = __ballot_sync(0xFFFFFFFFu, src != nullptr);
        const bool past = id >= 0 && 4 * (int64_t)id + 3 > pos0;
        const bool special = __any_sync(0xFFFFFFFFu, past || (id >= 0 && src == nullptr));
        if (lane == 0) {
          m.valid[w] = there;
          m.special[w] = special;
        }
        if ((lane & 3) == 0) m.block[8 * w + (lane >> 2)] = id;
        if (mh >= 0 && mh < halves) {                // transposed: lane q gets query q's bits of the 32 blocks
          uint32_t mine = 0;
#pragma unroll
          for (int q = 0; q < 32; ++q) {
            const uint32_t b = __ballot_sync(0xFFFFFFFFu, (word >> q) & 1u);
            if (lane == q) mine = b;
          }
          m.mine[mh][lane] = mine;
        }
      };
      if (!kFp8) {
        // 16 lanes copy the 256 bytes of a token's K[g] (or V[g]); two tokens per turn
        // (row r = 2 i + hi; its swizzle takes one of four values per lane)
        const uint32_t c = lane & 15, hi = lane >> 4;
        const uint32_t there = __ballot_sync(0xFFFFFFFFu, src != nullptr) >> hi;
        const uintptr_t at = src ? from : reinterpret_cast<uintptr_t>(p.c.b.pool);
        auto copy = [&](uint32_t dst, int off) {
          const uint32_t to = sb + dst + (c >> 3) * kPanel + hi * 128;
          const int o = off + (int)c * 16;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint8_t* s = reinterpret_cast<const uint8_t*>(__shfl_sync(0xFFFFFFFFu, at, (int)(2 * i + hi)));
            cp_async16(to + i * 256 + ((((c & 7) ^ hi) ^ (2 * i & 7)) << 4), s + o, (there >> (2 * i)) & 1u ? 16u : 0u);
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
        };
        copy(kdst, g * kHeadDim * 2);
        write_meta();
        if (j > 0) {                                 // V of step j - 1 has landed
          asm volatile("cp.async.wait_group 1;" ::: "memory");
          fence_async_smem();
          mbar_arrive(v_full((j - 1) % kStages));
        }
        if (j >= kStages) ok = mbar_wait_warp(v_empty(st), turn, err, kKernChunkAttn);
        if (!ok) break;
        copy(vdst, (kKvHeads + g) * kHeadDim * 2);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        fence_async_smem();
        mbar_arrive(k_full(st));
        if (j + 1 == steps) {
          asm volatile("cp.async.wait_group 0;" ::: "memory");
          fence_async_smem();
          mbar_arrive(v_full(st));
        }
      } else {
        // 8 lanes read the 128 codes of a token's K[g] (or V[g]); four tokens per turn
        const uint32_t c = lane & 7, four = lane >> 3;
        uint4 kv[8], vv[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint8_t* s = reinterpret_cast<const uint8_t*>(__shfl_sync(0xFFFFFFFFu, from, (int)(4 * i + four)));
          kv[i] = s ? *reinterpret_cast<const uint4*>(s + g * kHeadDim + c * 16) : make_uint4(0, 0, 0, 0);
          vv[i] = s ? *reinterpret_cast<const uint4*>(s + (kKvHeads + g) * kHeadDim + c * 16) : make_uint4(0, 0, 0, 0);
        }
        uint16_t kraw = 0, vraw = 0;   // (converted when used: a conversion here would wait for the loads)
        if (src) {
          const uint16_t* sc = reinterpret_cast<const uint16_t*>(src + 2 * kKvHeads * kHeadDim);
          kraw = sc[g];
          vraw = sc[kKvHeads + g];
        }
        write_meta();
        const float ks = __half2float(__ushort_as_half(kraw)), vs = __half2float(__ushort_as_half(vraw));
        scales[j % kMetas].k[32 * w + lane] = ks * p.scale_log2;
        scales[j % kMetas].v[32 * w + lane] = vs;
        scales[j % kMetas].size[32 * w + lane] = log2_size(vs);
        const uint32_t exps = __reduce_or_sync(0xFFFFFFFFu, src ? 1u << ((vraw >> 10) & 31) : 0u);
        if (lane == 0) m.exps[w] = exps;
        // codes 16 c .. +15 are chunks 2 c, 2 c + 1 of the row's 16
        auto store = [&](uint32_t dst, const uint4 (&x)[8]) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t r = 4 * i + four;
            uint8_t* row = smem + dst + (c >> 2) * kPanel + r * 128;
            const uint32_t c0 = (2 * c) & 7;
            *reinterpret_cast<uint4*>(row + ((c0 ^ (r & 7)) << 4)) = codes8_f16(make_uint2(x[i].x, x[i].y));
            *reinterpret_cast<uint4*>(row + (((c0 + 1) ^ (r & 7)) << 4)) = codes8_f16(make_uint2(x[i].z, x[i].w));
          }
          fence_async_smem();
        };
        store(kdst, kv);
        mbar_arrive(k_full(st));
        if (j >= kStages) ok = mbar_wait_warp(v_empty(st), turn, err, kKernChunkAttn);
        if (!ok) break;
        store(vdst, vv);
        mbar_arrive(v_full(st));
      }
      prefetch(slot_two);
      id = id_next;
      id_next = id_two;
      id_two = id_three;
      slot_now = slot_next;
      slot_next = slot_two;
      word = word_next;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  } else if (warp >= kRoleMma && warp - kRoleMma < halves) {
    // ---- MMA warp of half h
    const int h = warp - kRoleMma;
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    const uint32_t colO = tm + kColO + 128u * (uint32_t)h, colS = tm + kColS + 128u * (uint32_t)h;
    const uint32_t is = kFp8 ? idesc_f16(kSubTokens, false) : idesc_bf16(kSubTokens, false);
    const uint32_t io = kFp8 ? idesc_f16(kHeadDim, true) : idesc_bf16(kHeadDim, true);
    const uint64_t qd = desc_sw128(sb + h * 2 * kPanel, 16);
    // S of tokens 64 c .. of the step in K stage st
    auto issue_s = [&](int c, int st) {
      if (elect_one()) {
        const uint64_t b = desc_sw128(sb + kOffKv + st * kStageBytes + c * kSubTokens * 128, 16);
#pragma unroll
        for (int k = 0; k < kHeadDim / 16; ++k) {
          const uint64_t o = (uint64_t)(((k >> 2) * kPanel + (k & 3) * 32) >> 4);
          mma_ss(colS + 64u * (uint32_t)c, qd + o, b + o, is, k != 0);
        }
        mbar_arrive(s_full(h, c));   // passes on the loaders' writes of the meta (waited for with K)
        commit(s_full(h, c));
        if (c == 1) commit(k_empty(st));
      }
      __syncwarp();
    };
    if (steps > 0) {
      ok = mbar_wait_warp(q_full, 0, err, kKernChunkAttn);
      if (ok) ok = mbar_wait_warp(k_full(0), 0, err, kKernChunkAttn);
      if (ok) {
        fence_after();
        issue_s(0, 0);
        issue_s(1, 0);
      }
    }
#pragma unroll 1
    for (int j = 0; j < steps && ok; ++j) {
      const int st = j % kStages, sn = (j + 1) % kStages;
      ok = mbar_wait_warp(v_full(st), (uint32_t)(j / kStages) & 1u, err, kKernChunkAttn);
#pragma unroll 1
      for (int c = 0; c < 2 && ok; ++c) {
        ok = mbar_wait_warp(p_full(h, c), (uint32_t)j & 1u, err, kKernChunkAttn);
        if (!ok) break;
        fence_after();
        if (elect_one()) {
          const uint64_t b = desc_sw128(sb + kOffKv + st * kStageBytes + kKvBytes + c * kSubTokens * 128, kPanel);
#pragma unroll
          for (int k = 0; k < kSubTokens / 16; ++k)
            mma_ts(colO, colS + 64u * (uint32_t)c + 8u * k, b + (uint64_t)(k * 2048 >> 4), io, j > 0 || c > 0 || k > 0);
          commit(o_full(h, c));
          if (c == 1) commit(v_empty(st));
        }
        __syncwarp();
        if (j + 1 < steps) {
          // the next S goes over this P: after its products are complete
          if (c == 0) ok = mbar_wait_warp(k_full(sn), (uint32_t)((j + 1) / kStages) & 1u, err, kKernChunkAttn);
          if (ok) ok = mbar_wait_warp(o_full(h, c), (uint32_t)j & 1u, err, kKernChunkAttn);
          if (!ok) break;
          fence_after();
          issue_s(c, sn);
        }
      }
    }
    // every product is complete before tensor memory is given back
    if (elect_one()) commit(done(h));
    __syncwarp();
    mbar_wait_warp(done(h), 0, err, kKernChunkAttn);
  } else if (warp / 4 < halves) {
    // ---- softmax: thread = row (head warp & 3, query lane) of half h
    const int h = warp >> 2, head = g * kGroup + (warp & 3), q = 32 * h + lane;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t colO = lane_base + kColO + 128u * (uint32_t)h;
    const int64_t pos = pos0 + q;
    // FP8: the K scales hold the softmax scale
    const float f = kFp8 ? row_factor[128 * h + (warp & 3) * 32 + lane] : p.scale_log2;
    const uint64_t f2 = pair(f, f);
    float m = -INFINITY, l = 0.f;                    // in units of log2
#pragma unroll 1
    for (int jc = 0; jc < 2 * steps; ++jc) {
      const int j = jc >> 1, c = jc & 1;             // tokens 64 c .. of step j
      const uint32_t colS = lane_base + kColS + 128u * (uint32_t)h + 64u * (uint32_t)c;
      ok = mbar_wait_warp(s_full(h, c), (uint32_t)j & 1u, err, kKernChunkAttn);
      if (!ok) break;
      fence_after();
      const StepMeta& sm = meta[j % kMetas];
      const Scales& sc = scales[j % kMetas];
      // FP8: probabilities times V scales go in as f16, so the reference follows
      // the largest of these products that the row has, not of the probabilities:
      // log2 of both, x + log2 s.  Where the 64 tokens' scales lie within a factor
      // of 64, s counts as the upper end of that range (`above`); elsewhere (also at
      // zeros, subnormals, infinities and NaN) each as it is, a zero as 2^-100: its
      // token still keeps the sum l in range (and where such tokens outweigh all
      // others, f16's 2^-25 is 2^-117 of the row's weight).
      const uint32_t mine = sm.mine[h][lane] >> (16 * c);
      const bool special = (sm.special[0] | sm.special[1] | sm.special[2] | sm.special[3]) != 0;
      float above = 0.f, most = -INFINITY;
      bool wide = false;
      if (kFp8) {
        const uint32_t exps = sm.exps[2 * c] | sm.exps[2 * c + 1];
        const int high = 31 - __clz(exps);
        above = (float)(high - 14);
        wide = (exps & 0x80000001u) || high - (__ffs(exps) - 1) > 5;
        if (wide) most = wide_max(colS, sm, sc, c, mine, special, pos, f);
      }
      uint32_t v[2][32];
      ld32(colS, v[0]);
      ld32(colS + 32u, v[1]);
      wait_ld();
      reg_fence(v[0]);
      reg_fence(v[1]);
      if (kFp8) {
#pragma unroll
        for (int i = 0; i < kSubTokens; i += 4) {
          const ulonglong2 k4 = *reinterpret_cast<const ulonglong2*>(&sc.k[kSubTokens * c + i]);
          uint32_t* x = &v[i >> 5][i & 31];
          const uint64_t a = mul2(pair(x[0], x[1]), k4.x), b = mul2(pair(x[2], x[3]), k4.y);
          x[0] = (uint32_t)a;
          x[1] = (uint32_t)(a >> 32);
          x[2] = (uint32_t)b;
          x[3] = (uint32_t)(b >> 32);
        }
      }
      // tokens past the query, or without a row, count nowhere: a maximum that
      // they set could leave the row's own products below f16's range
      uint32_t tok[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};  // per token: its row exists and q sees it
      if (special) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          uint32_t seen = sm.valid[2 * c + w];
#pragma unroll 1
          for (int b = 0; b < 8; ++b) {
            const int64_t left = pos - 4 * (int64_t)sm.block[16 * c + 8 * w + b];   // tokens of the block that q sees, - 1
            const uint32_t four = left >= 3 ? 0xFu : (left < 0 ? 0u : (2u << (int)left) - 1u);
            seen &= ~(0xFu << (4 * b)) | (four << (4 * b));
          }
          tok[w] = seen;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!((seen >> i) & 1u)) v[w][i] = __float_as_uint(-INFINITY);
        }
      }
      // ---- maximum over the selected blocks
      auto at = [&](int i) { return __uint_as_float(v[i >> 5][i & 31]); };
      float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int b = 0; b < kSubTokens / 4; ++b) {
        const float top = fmaxf(fmaxf(at(4 * b), at(4 * b + 1)), fmaxf(at(4 * b + 2), at(4 * b + 3)));
        mx4[b & 3] = fmaxf(mx4[b & 3], (mine >> b) & 1u ? top : -INFINITY);
      }
      float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * f;
      if (kFp8) mx = wide ? most : mx + above;
      // the reference goes up only when the maximum has left it 2^8 behind
      const bool up = mx > m + 8.f;                  // true for the first tokens
      if (__any_sync(0xFFFFFFFFu, up)) {
        const float mn = fmaxf(m, mx);
        const float a = mn == -INFINITY ? 1.f : exp2_fast(m - mn);
        m = mn;
        l *= a;
        if (jc > 0) {
          // all products so far have to be complete
          ok = mbar_wait_warp(o_full(h, c ^ 1), (uint32_t)((jc - 1) >> 1) & 1u, err, kKernChunkAttn);
          if (!ok) break;
          fence_after();
#pragma unroll 1
          for (int i = 0; i < kHeadDim; i += 16) {
            uint32_t o[16];
            ld16(colO + (uint32_t)i, o);
            wait_ld();
            reg_fence(o);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
            st16(colO + (uint32_t)i, o);
          }
          wait_st();
        }
      }
      const float ref = m == -INFINITY ? 0.f : m;
      uint64_t l2 = pair(l, 0.f);
      // ---- probabilities, masked, over S's columns
#pragma unroll
      for (int w = 0; w < 2; ++w) {                  // 32 tokens
        uint32_t o[16];
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          // a block that the query does not select: exp2(s f - inf) = 0 (NaN
          // where the logit is not finite: the row is computed again)
          const float add = (mine >> (8 * w + b)) & 1u ? -ref : -INFINITY;
          const uint64_t addend = pair(add, add);
          const uint64_t x01 = fma2(pair(v[w][4 * b], v[w][4 * b + 1]), f2, addend);
          const uint64_t x23 = fma2(pair(v[w][4 * b + 2], v[w][4 * b + 3]), f2, addend);
          float e[4] = {exp2_fast(lo_of(x01)), exp2_fast(hi_of(x01)), exp2_fast(lo_of(x23)), exp2_fast(hi_of(x23))};
          if (special) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!((tok[w] >> (4 * b + i)) & 1u)) e[i] = 0.f;
          }
          l2 = add2(l2, pair(e[0], e[1]));
          l2 = add2(l2, pair(e[2], e[3]));
          if (kFp8) {
            const ulonglong2 v4 = *reinterpret_cast<const ulonglong2*>(&sc.v[kSubTokens * c + 32 * w + 4 * b]);
            const uint64_t a = mul2(pair(e[0], e[1]), v4.x), d = mul2(pair(e[2], e[3]), v4.y);
            e[0] = lo_of(a);
            e[1] = hi_of(a);
            e[2] = lo_of(d);
            e[3] = hi_of(d);
          }
          o[2 * b] = kFp8 ? pack_f16(e[0], e[1]) : pack_bf16(e[0], e[1]);
          o[2 * b + 1] = kFp8 ? pack_f16(e[2], e[3]) : pack_bf16(e[2], e[3]);
        }
        st16(colS + 16u * w, o);
      }
      l = lo_of(l2) + hi_of(l2);
      wait_st();
      fence_before();
      mbar_arrive(p_full(h, c));
    }
    // ---- the row's result
    if (ok && steps > 0) ok = mbar_wait_warp(o_full(h, 1), (uint32_t)(steps - 1) & 1u, err, kKernChunkAttn);
    fence_after();
    const int x = x0 + q;
    const bool mine = ok && q < nq;
    if (splits > 1) {
      float* part = p.part + (((int64_t)blockIdx.x * kKvHeads + g) * 256 + h * 128 + (warp & 3) * 32 + lane) * kRowFloats;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t v[32];
        if (steps > 0) {
          ld32(colO + 32u * c, v);
          wait_ld();
          reg_fence(v);
        }
        if (mine) {
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            *reinterpret_cast<float2*>(part + 32 * c + i) =
                steps > 0 ? make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])) : make_float2(0.f, 0.f);
        }
      }
      if (mine) *reinterpret_cast<float2*>(part + kHeadDim) = make_float2(m, l);
    } else {
      const float r = 1.f / l;
      bool good = l > 0x1p-100f && l < 0x1p125f;     // false for NaN
      uint16_t* out = p.out + ((int64_t)x * kQHeads + head) * kHeadDim;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t v[32];
        if (steps > 0) {
          ld32(colO + 32u * c, v);
          wait_ld();
          reg_fence(v);
        }
        if (mine && steps > 0) {
          float far = 0.f;
#pragma unroll
          for (int i = 0; i < 32; ++i) far = fmaxf(far, isfinite(__uint_as_float(v[i])) ? 0.f : 1.f);
          good = good && far == 0.f;
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            uint4 o;
            o.x = pack_bf16(__uint_as_float(v[i]) * r, __uint_as_float(v[i + 1]) * r);
            o.y = pack_bf16(__uint_as_float(v[i + 2]) * r, __uint_as_float(v[i + 3]) * r);
            o.z = pack_bf16(__uint_as_float(v[i + 4]) * r, __uint_as_float(v[i + 5]) * r);
            o.w = pack_bf16(__uint_as_float(v[i + 6]) * r, __uint_as_float(v[i + 7]) * r);
            *reinterpret_cast<uint4*>(out + 32 * c + i) = o;
          }
        }
      }
      if (mine && good && p.lse) p.lse[(int64_t)x * kQHeads + head] = (m + log2f(l)) * kLn2;
      for (uint32_t again = __ballot_sync(0xFFFFFFFFu, mine && !good); again; again &= again - 1) {
        __syncwarp();
        attend_row(p, u, x0 + 32 * h + __ffs(again) - 1, head);
      }
    }
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kRoleMma) tmem_free<kTmemCols>(tmem);
}

// ------------------------------------------------------------------- join

// One warp per (row, head): lane l holds dims 4 l .. 4 l + 3.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) chunk_join_kernel(const __grid_constant__ ChunkAttnParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
  const int x = (int)(w / kQHeads), head = (int)(w % kQHeads);
  grid_dependency_wait();
  if (x >= p.c.rows()) return;
  const int u = p.c.unit_of_row(x), i = x - p.c.row0[u], tile = p.tile0[u] + i / kTileQueries;
  const int q = i % kTileQueries, row = (q >> 5) * 128 + (head % kGroup) * 32 + (q & 31);
  const int2 dealt = p.dealt[tile];
  const int splits = dealt.y;
  if (splits == 1) return;                           // complete
  const float* part = p.part + (((int64_t)dealt.x * kKvHeads + head / kGroup) * 256 + row) * kRowFloats;
  const int64_t stride = (int64_t)kKvHeads * 256 * kRowFloats;
  // a lane takes two shares' maxima and sums; the first shares' O are on their
  // way with them
  constexpr int kFirst = 16;
  static_assert(kMaxShares == 64, "two shares per lane");
  auto piece = [&](int s) {
    const float* o = part + s * stride + 4 * lane;
    const float2 lo = *reinterpret_cast<const float2*>(o), hi = *reinterpret_cast<const float2*>(o + 2);
    return make_float4(lo.x, lo.y, hi.x, hi.y);
  };
  float4 first[kFirst];
#pragma unroll
  for (int s = 0; s < kFirst; ++s)
    if (s < splits) first[s] = piece(s);
  float2 ml[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    ml[i] = lane + 32 * i < splits ? *reinterpret_cast<const float2*>(part + (lane + 32 * i) * stride + kHeadDim)
                                   : make_float2(-INFINITY, 0.f);
  float m = fmaxf(ml[0].x, ml[1].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  float a[2], l = 0.f;                               // a = 0: nothing selected there
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    a[i] = ml[i].y != 0.f ? exp2f(ml[i].x - m) : 0.f;
    l = fmaf(ml[i].y, a[i], l);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](int s, float4 o) {
    const float w = __shfl_sync(0xFFFFFFFFu, s < 32 ? a[0] : a[1], s & 31);
    if (w != 0.f) acc = make_float4(fmaf(o.x, w, acc.x), fmaf(o.y, w, acc.y), fmaf(o.z, w, acc.z), fmaf(o.w, w, acc.w));
  };
#pragma unroll
  for (int s = 0; s < kFirst; ++s)
    if (s < splits) add(s, first[s]);
#pragma unroll 4
  for (int s = kFirst; s < splits; ++s) add(s, piece(s));
  const bool fine = l > 0x1p-100f && l < 0x1p125f && isfinite(acc.x) && isfinite(acc.y) && isfinite(acc.z) && isfinite(acc.w);
  if (!__all_sync(0xFFFFFFFFu, fine)) {
    attend_row(p, u, x, head);
    return;
  }
  const float r = 1.f / l;
  reinterpret_cast<uint2*>(p.out + ((int64_t)x * kQHeads + head) * kHeadDim)[lane] =
      make_uint2(pack_bf16(acc.x * r, acc.y * r), pack_bf16(acc.z * r, acc.w * r));
  if (p.lse && lane == 0) p.lse[(int64_t)x * kQHeads + head] = (m + log2f(l)) * kLn2;
}

// ------------------------------------------------------------------- host

struct AttnPlan {
  int64_t tiles = 0, cap = 0, nb = 0, shares = 0;
  int64_t off_dealt = 0, off_block = 0, off_mask = 0, off_part = 0, bytes = 0;
};

// Steps of a tile of nq queries of unit u, at most.
int64_t longest_list(const ChunkDesc& c, int u, int64_t nq, int32_t budget_tokens) {
  const int64_t nb = (c.b.u[u].n + 3) / 4, most = nq * (budget_tokens / 4);
  return ((nb < most ? nb : most) + kStepBlocks - 1) / kStepBlocks;
}

AttnPlan make_plan(const ChunkDesc& c, int32_t budget_tokens, int sms, int32_t* tile0) {
  AttnPlan a;
  for (int u = 0; u < c.b.n_units; ++u) {
    if (tile0) tile0[u] = (int32_t)a.tiles;
    if (c.unit_tokens(u) == 0) continue;
    a.tiles += (c.unit_tokens(u) + kTileQueries - 1) / kTileQueries;
    const int64_t nb = (c.b.u[u].n + 3) / 4, most = (int64_t)(c.unit_tokens(u) < kTileQueries ? c.unit_tokens(u) : kTileQueries) * (budget_tokens / 4);
    if (nb > a.nb) a.nb = nb;
    const int64_t cap = nb < most ? nb : most;
    if (cap > a.cap) a.cap = cap;
  }
  if (tile0) tile0[c.b.n_units] = (int32_t)a.tiles;
  a.cap = (a.cap + kStepBlocks - 1) / kStepBlocks * kStepBlocks;
  // Fewer CTAs than SMs: the lists may be split.  The shares are dealt out on the
  // device, by the lists' lengths (share_of).  Whether it pays is judged here by
  // the longest that they can be: not where the longest share stays above 3/4 of
  // the longest list (equal lists and few spare shares: 178 -> 184 us for 32 tiles
  // of 64 queries on 38 shares), since the join comes on top.
  a.shares = a.tiles;
  const int64_t most = sms / kKvHeads < kMaxShares ? sms / kKvHeads : kMaxShares;
  if (a.tiles < most) {
    auto dealt = [&](int64_t q) {                    // shares of at most q steps
      int64_t sum = 0;
      for (int u = 0; u < c.b.n_units; ++u) {
        const int64_t t = c.unit_tokens(u), whole = t / kTileQueries;
        if (whole > 0) sum += whole * ((longest_list(c, u, kTileQueries, budget_tokens) + q - 1) / q);
        if (t % kTileQueries) sum += (longest_list(c, u, t % kTileQueries, budget_tokens) + q - 1) / q;
      }
      return sum;
    };
    const int64_t longest = a.cap / kStepBlocks;
    if (dealt(longest - longest / 4) <= most) {
      a.shares = dealt(kLeastSteps);
      if (a.shares > most) a.shares = most;
    }
  }
  auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
  a.off_dealt = up(4 * a.tiles);
  a.off_block = a.off_dealt + up(8 * a.tiles);
  a.off_mask = a.off_block + up(4 * a.tiles * a.cap);
  a.off_part = a.off_mask + up(8 * a.tiles * a.cap);
  a.bytes = a.off_part + (a.shares > a.tiles ? up(a.shares * kKvHeads * 256 * kRowFloats * 4) : 0);
  return a;
}

}  // namespace

int64_t chunk_attn_workspace(const ChunkDesc& c, int32_t budget_tokens) {
  int sms = 0;
  if (current_sm_count(&sms) != cudaSuccess) return -1;
  const int64_t b = make_plan(c, budget_tokens, sms, nullptr).bytes;
  return b > 256 ? b : 256;
}

cudaError_t launch_chunk_attn(const ChunkDesc& c, const uint16_t* q, const int32_t* sel_blocks,
                              const int32_t* n_sel, int32_t budget_tokens, float softmax_scale,
                              uint16_t* out, float* lse, void* workspace, cudaStream_t s) {
  static PerDeviceOnce setup;
  cudaError_t e = setup.run([] {
    cudaError_t r = prefer_max_shared(chunk_split_kernel<false>, kSmemBytes);
    if (r == cudaSuccess) r = prefer_max_shared(chunk_split_kernel<true>, kSmemBytes);
    if (r == cudaSuccess) r = prefer_max_shared(chunk_plan_kernel, kPlanWindow * 8);
    return r;
  });
  int sms = 0;
  if (e == cudaSuccess) e = current_sm_count(&sms);
  if (e != cudaSuccess) return e;
  ChunkAttnParams p;
  const AttnPlan a = make_plan(c, budget_tokens, sms, p.tile0);
  p.c = c;
  p.q = q;
  p.sel = sel_blocks;
  p.n_sel = n_sel;
  p.k_max = budget_tokens / 4;
  p.shares = (int32_t)a.shares;
  p.scale_log2 = fabsf(softmax_scale) * kLog2e;
  p.sign = softmax_scale < 0.f ? -1.f : 1.f;
  p.out = out;
  p.lse = lse;
  p.cap = (int32_t)a.cap;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.count = reinterpret_cast<int32_t*>(ws);
  p.dealt = reinterpret_cast<int2*>(ws + a.off_dealt);
  p.block = reinterpret_cast<int32_t*>(ws + a.off_block);
  p.mask = reinterpret_cast<uint32_t*>(ws + a.off_mask);
  p.part = reinterpret_cast<float*>(ws + a.off_part);
  e = launch_hot_complete(c.b, s);
  if (e != cudaSuccess) return e;
  const int window = (int)(a.nb < kPlanWindow ? (a.nb + 3) / 4 * 4 : kPlanWindow);
  e = launch_kernel(chunk_plan_kernel, dim3((unsigned)a.tiles), dim3(kPlanThreads), (size_t)window * 8, s, 0, dim3(1),
                    p, window);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)a.shares, kKvHeads);
  e = c.b.row_bytes == kRowBytesFp8
          ? launch_kernel(chunk_split_kernel<true>, grid, dim3(kThreads), kSmemBytes, s, 0, dim3(1), p)
          : launch_kernel(chunk_split_kernel<false>, grid, dim3(kThreads), kSmemBytes, s, 0, dim3(1), p);
  if (e != cudaSuccess || a.shares == a.tiles) return e;
  const int64_t warps = (int64_t)c.rows() * kQHeads;
  return launch_kernel(chunk_join_kernel, dim3((unsigned)((warps + 7) / 8)), dim3(kJoinThreads), 0, s, 0, dim3(1), p);
}

}  // namespace qsa
