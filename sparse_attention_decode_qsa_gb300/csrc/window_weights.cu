// The weight that attention gives each cached token: for token t of a unit
//     weights[t] (+)= sum_x sum_h exp(scale * q[x][h] . K_t[h / 4] - lse[x][h])
// over the chunk's queries x that see t (the window and sinks of dense_attn.cu)
// and all heads h, with the log-sum-exp that the attention returned.  A row
// without tokens (lse = -inf) adds nothing.
//
// Tokens are the rows of the product K Q^T, so that a thread holds one token and
// sums over queries and heads in its own registers: no atomics, no order that
// could change, one store per token.  The queries that see a token are a range of
// the chunk, hence a range of columns.
//
// exp(x - lse) goes through 2^y with y = x log2 e - lse log2 e.  Roundings of
// scale * log2 e and of lse * log2 e would go the same way in all of a row's weights
// (2^-19 of them where logits reach 40), so both are kept in two parts.  The scale's
// second part is added last: x times the first part less the lse is small where there
// is weight, and loses nothing (added to the lse first, it would be lost in the lse's
// last place).  The lse's second part is a factor beside the column.
//
// The tensor core cuts partial sums off where fp32 additions round them, so a logit
// comes out too small in size, by an amount that depends on how its sum grows.  For few
// queries every 16 dims are a product of their own, and the eight are added in fp32.
// For more the sum stays in tensor memory, and kCutOff makes up for the mean.
//
// Measured (device time of a call):
//   8 requests' tokens over 8192 BF16 tokens each (67 MB of keys): 9.4 us, above the
//     measured copy rate (the keys stay in L2 from call to call; 17.0 from cold caches).
//   64 queries over 131072 FP8 tokens (134 M exponentials, 34 GFLOP): 72 us.  BF16
//     rows take 60, 32 queries 56 and 42: codes to bf16 are a part of the bound.  A
//     further turn of 256 tokens costs 1.8 us up to 128 queries and 2.0 beyond, the
//     tensor core 0.6 of it (both operands from shared memory, 66 cycles an MMA); the
//     rest is hand-overs and issue slots (0.54 in use).
//   1024 BF16 queries, windows of 16384 of 32768 tokens (69 GFLOP): 134 us on 136 of 152
//     SMs (128 tokens each; 256 tokens would be 68 CTAs), 1.05 us a turn of 128 x 128.
// Not faster: turns of 256 columns on 128 tokens (127 -> 165 us: with two turns under
// way the loads of Q, products and exponentials came one after the other); a scale per
// row of Q as f16 beside FP8 keys (105 -> 160).
#include <cmath>

#include "dense_common.cuh"

namespace qsa {
namespace {

using namespace tc;
using namespace attn;

// A mean correction of BF16 logits, relative, in the kernel of many queries: no more
// than that, since what is cut off depends on the keys, and a logit that loses nothing
// is then too large by it.  Sums of the weights of logits near 10 (and near 40), off
// from float64 in units of 1e-7, with the correction and without it; the last number
// is a plain fp32 product's:
//   keys at random                                         +2, -8 (-2, -43)      +1
//   all dims alike                                        -14, -27 (-30, -81)    -1
//   the second half of the dims takes most back           -31, -43 (-190, -240)  -4
//   one dim alone                                         +10, -1 (+51, 0)       +1
// FP8 keys go without: -2, -19, -41, -1 (-11, -29, -58, -1).  The kernel of few queries:
// -1, -5, +1, -2 beside BF16 and 0, -3, +14, -1 beside FP8 rows (near 10).
constexpr double kCutOff = 1.1 / 8388608;

struct WeightParams {
  DenseAttn d;
  const uint16_t* q;             // [rows][16][128] bf16 bits
  const float* lse;              // [rows][16]
  float scale_log2, scale_rest;  // softmax_scale * log2(e), in two parts
  float* weights;                // [units][stride]
  int64_t stride;
  int32_t accumulate;
  int32_t few_tokens;            // tokens of a CTA of the few kernel
};

// Whether a query at position pos sees token t.
__device__ __forceinline__ bool sees(const DenseAttn& d, int64_t pos, int64_t t) {
  return t <= pos && (t < d.sinks || t > pos - d.window);
}
// Whether any query of unit u sees token t.
__device__ __forceinline__ bool seen_by_any(const DenseAttn& d, int u, int64_t t) {
  const int n = d.c.unit_tokens(u);
  const int64_t p1 = d.c.b.u[u].n - 1, p0 = p1 - n + 1;
  return n > 0 && t <= p1 && (t < d.sinks || t > p0 - d.window);
}
// -lse in units of log2, and the factor that its rounding leaves.
__device__ __forceinline__ float2 column_of(float lse) {
  const float y = lse * kLog2e;
  const float rest = fmaf(lse, kLog2e, -y) + lse * 1.925963033500e-08f;      // log2(e) past its fp32 value
  return make_float2(-y, isfinite(y) ? exp2f(-rest) : 1.f);
}
__device__ __forceinline__ void store_weight(const WeightParams& p, int u, int64_t t, float w) {
  float* to = p.weights + u * p.stride + t;
  *to = p.accumulate ? *to + w : w;
}

// ------------------------------------------------------------------- few

// Units of at most four queries: one CTA per run of tokens, all KV heads; warp w
// serves KV head w % 4 for the tokens 16 (w / 4) .. + 15 of every step of 32, copied
// by itself into its own ring of three stages, as in dense_attn.cu; S = Q K^T by 16
// mma of m16n8k16 per stage, whose 16 rows are summed over the lanes.  Bound by the
// keys' bytes.
constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32, kFewStages = 3, kFewStep = 32, kFewTokens = 16;
constexpr int kFewMost = 1024;                    // tokens of a CTA at most
template <bool kFp8>
struct FewLayout {
  static constexpr int kVec = kFp8 ? 128 : 256;
  static constexpr int kScales = kFewTokens * kVec;              // FP8: the rows' 8 scales, 16 bytes a token
  static constexpr int kStage = kScales + (kFp8 ? kFewTokens * 16 : 0);
  static constexpr int kSums = kFewWarps * kFewStages * kStage;  // float [4][few_tokens]
  static constexpr int kSmem = kSums + kKvHeads * kFewMost * 4;
};

template <bool kFp8, int kN>
__global__ void __launch_bounds__(kFewThreads, 2) weight_few_kernel(const __grid_constant__ WeightParams p) {
  using L = FewLayout<kFp8>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t there[kFewWarps][kFewStages];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = warp & 3, half = warp >> 2;
  const int r = lane >> 2, j4 = lane & 3;
  const BatchDesc& b = p.d.c.b;
  const int u = blockIdx.y, nq = p.d.c.unit_tokens(u);
  const int64_t n = b.u[u].n, t0 = (int64_t)blockIdx.x * p.few_tokens;
  if (nq > kFewQueries || t0 >= n) return;
  const int64_t t1 = t0 + p.few_tokens < n ? t0 + p.few_tokens : n;
  const int x0 = p.d.c.row0[u];
  const int64_t pos0 = n - nq;
  grid_dependency_wait();
  // steps that some query sees: from the first to the last token it sees here
  const bool all_hidden = nq == 0 || (t0 >= p.d.sinks && t1 - 1 <= pos0 - p.d.window);
  const int steps = all_hidden ? 0 : (int)((t1 - t0 + kFewStep - 1) / kFewStep);

  uint32_t qb[kN][8][2];
  float f[kN][2];
  few_queries<kFp8, kN>(p.q, x0, nq, g, 1.f, qb, f);
  float2 col[kN][2];                                             // columns 8 n + 2 j4 + e: query * 4 + head
  bool live[kN][2];
  int64_t pos[kN];
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    const int qi = 2 * n + (j4 >> 1);
    pos[n] = pos0 + qi;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float lse = qi < nq ? p.lse[(int64_t)(x0 + qi) * kQHeads + g * kGroup + ((2 * j4 + e) & 3)] : -INFINITY;
      live[n][e] = lse != -INFINITY;
      col[n][e] = column_of(lse);
    }
  }
  const int32_t* slots = b.slot_table + b.unit_row(u);
  const uint32_t ring = smem_u32(smem) + warp * kFewStages * L::kStage;
  float* sums = reinterpret_cast<float*>(smem + L::kSums) + g * p.few_tokens;
  const int64_t first = t0 + half * kFewTokens;
  auto token_of = [&](int s) {                                   // lane l < 16: token l of a stage, -1: none that counts
    const int64_t t = first + (int64_t)s * kFewStep + lane;
    return lane < kFewTokens && s < steps && t < t1 && seen_by_any(p.d, u, t) ? t : (int64_t)-1;
  };
  auto slot_of = [&](int s) {
    const int64_t t = token_of(s);
    return t >= 0 ? slots[t] : -2;
  };
  auto issue = [&](int s, int32_t slot) {
    const int64_t t = token_of(s);
    const uint8_t* row = nullptr;
    if (t >= 0) {
      if (slot >= 0 && (int64_t)slot < b.pool_rows) row = b.pool + (int64_t)slot * b.row_bytes;
      else if (slot == -1 && b.u[u].host_rows) row = b.u[u].host_rows + t * b.row_bytes;
      else report_error(b.err, QSA_ERR_BAD_SLOT, kKernWeights, ((int64_t)u << 40) | (t & 0xFFFFFFFFFFll));
    }
    const uint32_t have = __ballot_sync(0xFFFFFFFFu, row != nullptr);
    if (lane == 0) there[warp][s % kFewStages] = have;
    const uint32_t to = ring + (s % kFewStages) * L::kStage;
    constexpr int kLanes = L::kVec / 16;
    const int c = lane % kLanes;
    const uint32_t off = g * L::kVec + c * 16;
    few_copies<32 / kLanes>(b, row, slot, [&](int k, const uint8_t* from) {
      cp_async16(to + k * L::kVec + ((c ^ (k & 7)) << 4), from + off, (have >> k) & 1u ? 16u : 0u);
    });
    if (kFp8 && lane < kFewTokens)
      cp_async16(to + L::kScales + lane * 16, (row ? row : b.pool) + 2 * kKvHeads * kHeadDim, row ? 16u : 0u);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  {
    const int32_t a = slot_of(0), c = slot_of(1);
    issue(0, a);
    issue(1, c);
  }
  int32_t slot_next = slot_of(2);
#pragma unroll 1
  for (int s = 0; s < steps; ++s) {
    const int32_t slot = slot_next;
    slot_next = slot_of(s + 3);
    issue(s + 2, slot);
    asm volatile("cp.async.wait_group 2;" ::: "memory");
    __syncwarp();
    const uint32_t st = ring + (s % kFewStages) * L::kStage;
    const uint32_t have = there[warp][s % kFewStages];
    float x[kN][4];                                              // tokens r (elements 0, 1) and r + 8 (2, 3)
#pragma unroll
    for (int i = 0; i < kN; ++i) x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t ka[4];
      few_keys<kFp8>(st, k, ka);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        float y[4] = {0.f, 0.f, 0.f, 0.f};
        mma16<kFp8>(y, ka, qb[i][k][0], qb[i][k][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[i][e] += y[e];
      }
    }
    float w[2] = {0.f, 0.f};
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
      const int c = r + 8 * hi;
      const int64_t t = first + (int64_t)s * kFewStep + c;
      float ks = 1.f;
      if (kFp8) ks = key_scale_of(*reinterpret_cast<const uint16_t*>(smem + (st - smem_u32(smem)) + L::kScales + c * 16 + 2 * g));
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const bool seen = ((have >> c) & 1u) && sees(p.d, pos[i], t);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float z = x[i][2 * hi + e] * ks * f[i][e];
          const float y = exp2_fast(fmaf(z, p.scale_rest, fmaf(z, p.scale_log2, col[i][e].x))) * col[i][e].y;
          if (seen && live[i][e]) w[hi] += y;
        }
      }
    }
    // sums over the four lanes of a token; lane j4 = 0 keeps token r, j4 = 1 token r + 8
    float v = (j4 & 1 ? w[1] : w[0]) + __shfl_xor_sync(0xFFFFFFFFu, j4 & 1 ? w[0] : w[1], 1);
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
    if (j4 < 2) sums[s * kFewStep + half * kFewTokens + r + 8 * j4] = v;
    __syncwarp();
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(smem + L::kSums);
  for (int i = tid; i < (int)(t1 - t0); i += kFewThreads) {
    if (steps == 0 && p.accumulate) break;
    float w = 0.f;
    if (steps > 0)
      w = (all[i] + all[p.few_tokens + i]) + (all[2 * p.few_tokens + i] + all[3 * p.few_tokens + i]);
    store_weight(p, u, t0 + i, w);
  }
}

// ------------------------------------------------------------------- wide

// Units of more queries: a CTA takes tiles of 128 kTiles tokens (128 = the tensor
// core's M) in turn; a turn is 32 queries x 4 heads of a KV head = 128 columns (N)
// against each 128 tokens, K = 128 dims, both operands in shared memory under the
// 128-byte swizzle.  K[g] of the tile (two buffers, the next head's or tile's on its
// way) stays for all of the chunk's queries, Q streams past from L2: with two tiles of
// 128 it is read half as often, with one there are twice as many tiles to share out.
// Tensor memory: turns of 128 columns per 128 tokens, 512 in all.  Warps: 16 epilogue
// (thread = token), 4 load K, 2 or 3 load Q, 1 MMA; all waits bounded.  FP8 codes
// become bf16, beside which Q stays as it is: f16 would want every row of Q scaled,
// again in every CTA.
constexpr int kEpiWarps = 16, kKeyWarps = 4;
constexpr int kPanel = 128 * 128;                 // 128 rows of 64 16-bit elements
constexpr int kAhead = 4;                         // pieces of FP8 codes that a lane reads ahead (2: 76 us for 72)
constexpr int kTurnQueries = 32, kTurnCols = kTurnQueries * kGroup;
constexpr uint32_t kTmemCols = 512;

template <int kTiles>
struct Wide {
  static constexpr int kTokens = 128 * kTiles;
  static constexpr int kRing = 4 / kTiles;         // turns under way
  static constexpr int kEpiCols = 32 * kTiles;     // of an epilogue warp and turn
  // Query warp w of n has the turns w, w + n, ..  At its turn i - n it has waited for
  // turn i - n - kRing to be done with, so that at turn i it cannot take the phase of
  // turn i - 2 kRing for that of i - kRing: n <= kRing.  (With the MMA warp six warps
  // to a scheduler at most: 80 registers.)
  static constexpr int kQueryWarps = kTiles == 2 ? 2 : 3;
  static constexpr int kThreads = 32 * (kEpiWarps + kKeyWarps + kQueryWarps + 1);
  static constexpr int kRoleKeys = kEpiWarps, kRoleQueries = kRoleKeys + kKeyWarps, kRoleMma = kRoleQueries + kQueryWarps;
  struct __align__(16) Columns {
    float minus[kTurnCols];        // -lse (log2)
    float factor[kTurnCols];       // what its rounding leaves
    int32_t dead, pad[3];          // a column has no weight
  };
  // Columns of turn i are written once the products of turn i - kRing are complete,
  // before which the epilogue of turn i - 2 kRing had left its accumulators.
  static constexpr int kColumns = 2 * kRing;
  static constexpr int kKBytes = kTiles * 2 * kPanel, kQPanel = kTurnCols * 128, kQBytes = 2 * kQPanel;
  static constexpr int kOffQ = 2 * kKBytes, kOffCols = kOffQ + kRing * kQBytes;
  // of two tiles in turn: K scales float [4][kTokens], column parts' sums float [4][128],
  // tokens that count uint32 [8]
  static constexpr int kOffKs = kOffCols + kColumns * (int)sizeof(Columns);
  static constexpr int kOffSum = kOffKs + 2 * kKvHeads * kTokens * 4;
  static constexpr int kOffThere = kOffSum + 2 * 4 * 128 * 4;
  static constexpr int kOffBar = kOffThere + 2 * 32;
  static constexpr int kNumBars = 4 * kRing + 4;   // full, empty, d_full, d_empty [kRing], k_full, k_empty [2]
  static constexpr int kOffSlot = kOffBar + 8 * kNumBars;
  static constexpr int kSmem = kOffSlot + 16 + 1024;
  static_assert(kSmem <= 227 * 1024 && kOffCols % 16 == 0 && kOffBar % 8 == 0 && kQBytes % 1024 == 0, "shared memory");
  static_assert(kQueryWarps <= kRing && kThreads <= 24 * 32, "see above");
};

// Two e4m3 codes (the low 16 bits) as bf16, exactly: their exponent and mantissa at
// the low end of bf16's make 2^-120 times the value (a subnormal code a subnormal),
// which the product puts right.  A NaN code (nan_codes) comes out as 480.
__device__ __forceinline__ uint32_t codes2_bf16(uint32_t two) {
  const uint32_t h = __byte_perm(two, 0, 0x1404);
  const uint32_t x = (h & 0x80008000u) | ((h >> 4) & 0x07F007F0u);
  const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x),
                                   __nv_bfloat162(__ushort_as_bfloat16(0x7B80), __ushort_as_bfloat16(0x7B80)));    // 2^120
  return *reinterpret_cast<const uint32_t*>(&y);
}
// Not 0 where one of four codes is a NaN.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

template <bool kFp8, int kTiles>
__global__ void __launch_bounds__(Wide<kTiles>::kThreads, 1) weight_wide_kernel(const __grid_constant__ WeightParams p) {
  using W = Wide<kTiles>;
  using Columns = typename W::Columns;
  constexpr int kRing = W::kRing, kEpiCols = W::kEpiCols;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  Columns* columns = reinterpret_cast<Columns*>(smem + W::kOffCols);
  const uint32_t bars = sb + W::kOffBar;
  // turns i: buffer i % kRing; heads of K, counted through all tiles: k % 2
  auto full = [&](int i) { return bars + 8u * (uint32_t)(i % kRing); };
  auto empty = [&](int i) { return bars + 8u * (uint32_t)(kRing + i % kRing); };
  auto d_full = [&](int i) { return bars + 8u * (uint32_t)(2 * kRing + i % kRing); };
  auto d_empty = [&](int i) { return bars + 8u * (uint32_t)(3 * kRing + i % kRing); };
  auto k_full = [&](int k) { return bars + 8u * (uint32_t)(4 * kRing + (k & 1)); };
  auto k_empty = [&](int k) { return bars + 8u * (uint32_t)(4 * kRing + 2 + (k & 1)); };
  auto turn_of = [](int i) { return (uint32_t)(i / kRing) & 1u; };
  auto head_of = [](int k) { return (uint32_t)(k >> 1) & 1u; };
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + W::kOffSlot);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const BatchDesc& b = p.d.c.b;
  ErrorWord* err = b.err;
  const int u = blockIdx.y, nq = p.d.c.unit_tokens(u), x0 = p.d.c.row0[u];
  if (nq <= kFewQueries) return;
  const int64_t n = b.u[u].n, pos0 = n - nq;
  grid_dependency_wait();

  // ---- tiles that some query sees: 0 .. front - 1 (sinks) and back .. all - 1
  const int all = (int)((n + W::kTokens - 1) / W::kTokens);
  int64_t newest = pos0 - p.d.window;                  // the newest token that no window has
  if (newest < -1) newest = -1;
  const int back = (int)((newest + 1) / W::kTokens);
  int front = (int)((p.d.sinks + W::kTokens - 1) / W::kTokens);
  if (front > back) front = back;
  const int seen_tiles = front + all - back;
  if (!p.accumulate)
    for (int64_t t = (int64_t)front * W::kTokens + (int64_t)blockIdx.x * W::kThreads + tid; t < (int64_t)back * W::kTokens;
         t += (int64_t)gridDim.x * W::kThreads)
      store_weight(p, u, t, 0.f);
  if ((int)blockIdx.x >= seen_tiles) return;
  // the v-th of them: its tokens t0 .. t1 - 1, and the queries that see any of these
  // (positions t0 .. t1 - 1 + window - 1) in whole turns c0 .. c0 + per - 1 (one at
  // least, which then finds nothing to do)
  struct Range {
    int64_t t0, t1;
    int c0, per;
  };
  auto range_of = [&](int v) {
    Range r;
    r.t0 = (int64_t)(v < front ? v : back + v - front) * W::kTokens;
    r.t1 = r.t0 + W::kTokens < n ? r.t0 + W::kTokens : n;
    int64_t low = r.t0 - pos0, high = r.t0 < p.d.sinks ? nq : r.t1 - 1 + p.d.window - pos0;
    if (low < 0) low = 0;
    if (high > nq) high = nq;
    r.c0 = (int)(low / kTurnQueries);
    r.per = high > low ? (int)((high + kTurnQueries - 1) / kTurnQueries) - r.c0 : 1;
    return r;
  };

  if (warp == W::kRoleMma) {
    tmem_alloc<kTmemCols>(slot);
    if (lane == 0) {
      for (int i = 0; i < kRing; ++i) {
        mbar_init(full(i), 1);
        mbar_init(empty(i), 1);
        mbar_init(d_full(i), 2);
        mbar_init(d_empty(i), kEpiWarps);
      }
      for (int g = 0; g < 2; ++g) {
        mbar_init(k_full(g), 32 * kKeyWarps);
        mbar_init(k_empty(g), 1);
      }
      mbar_fence_init();
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *slot;
  bool ok = true;

  if (warp >= W::kRoleKeys && warp < W::kRoleQueries) {
    // ---- K: warp w has the tokens 32 kTiles w .. of a tile, lane = token of 32.  Step k
    // is head k % 4 of tile k / 4: K of step k + 1 is sent for once step k - 1 has left
    // its buffer, and handed on when it has landed.
    const int w = warp - W::kRoleKeys;
    const int heads = kKvHeads * ((seen_tiles - 1 - (int)blockIdx.x) / (int)gridDim.x + 1);
    const uint8_t* row[kTiles] = {};
    uint32_t exist[kTiles] = {};
    uint2 scales[kTiles] = {};                       // FP8: the tokens' K scales, all heads
    auto send = [&](int k) {
      const int tile = k / kKvHeads, g = k % kKvHeads;
      if (g == 0) {
        const Range r = range_of(blockIdx.x + tile * gridDim.x);
        uint32_t* there = reinterpret_cast<uint32_t*>(smem + W::kOffThere) + 8 * (tile & 1);
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
          const int64_t t = r.t0 + 32 * (kTiles * w + j) + lane;
          row[j] = nullptr;
          if (t < r.t1 && seen_by_any(p.d, u, t)) {
            const int32_t s = b.slot_table[b.unit_row(u) + t];
            if (s >= 0 && (int64_t)s < b.pool_rows) row[j] = b.pool + (int64_t)s * b.row_bytes;
            else if (s == -1 && b.u[u].host_rows) row[j] = b.u[u].host_rows + t * b.row_bytes;
            else report_error(err, QSA_ERR_BAD_SLOT, kKernWeights, ((int64_t)u << 40) | (t & 0xFFFFFFFFFFll));
          }
          exist[j] = __ballot_sync(0xFFFFFFFFu, row[j] != nullptr);
          if (lane == 0) there[kTiles * w + j] = exist[j];
          scales[j] = kFp8 && row[j] ? *reinterpret_cast<const uint2*>(row[j] + 2 * kKvHeads * kHeadDim) : make_uint2(0, 0);
          // the other heads' keys are on their way to L2 meanwhile
          if (row[j]) {
#pragma unroll
            for (int o = 1; o < kKvHeads; ++o)
              asm volatile("prefetch.global.L2 [%0];" ::"l"(row[j] + o * kHeadDim * (kFp8 ? 1 : 2)));
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kTiles; ++j) {
        const int at = 32 * (kTiles * w + j);                    // of the tile's tokens
        const uint32_t dst = sb + (k & 1) * W::kKBytes + (at >> 7) * 2 * kPanel + (at & 127) * 128;
        const uintptr_t from = reinterpret_cast<uintptr_t>(row[j] ? row[j] : b.pool);
        // BF16: 16 lanes a token, 8 in each panel.  FP8: 8 lanes, the codes as they
        // are in the token's row of the second panel
        constexpr int kLanes = kFp8 ? 8 : 16, kPer = 32 / kLanes;
        const uint32_t c = lane % kLanes;
        const uint32_t to = dst + (kFp8 ? kPanel : (c >> 3) * kPanel);
#pragma unroll
        for (int i = 0; i < 32 / kPer; ++i) {
          const uint32_t t = kPer * i + lane / kLanes;
          const uintptr_t a = __shfl_sync(0xFFFFFFFFu, from, (int)t);
          cp_async16(to + t * 128 + (((c & 7) ^ (t & 7)) << 4),
                     reinterpret_cast<const uint8_t*>(a) + g * (kFp8 ? kHeadDim : 2 * kHeadDim) + c * 16,
                     (exist[j] >> t) & 1u ? 16u : 0u);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto hand_on = [&](int k) {                      // (its copies have landed)
      const int g = k % kKvHeads;
      if (kFp8) {
        float* key_scale = reinterpret_cast<float*>(smem + W::kOffKs) + ((k / kKvHeads) & 1) * kKvHeads * W::kTokens;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
          const int at = 32 * (kTiles * w + j);
          uint8_t* panel = smem + (k & 1) * W::kKBytes + (at >> 7) * 2 * kPanel + (at & 127) * 128;
          const uint32_t c = lane & 7;
          uint32_t nan_of = 0;                                   // bit i: of this lane's 16 codes of token 4 i + lane / 8
#pragma unroll 1
          for (int i0 = 0; i0 < 8; i0 += kAhead) {
            uint4 v[kAhead];
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
              const uint32_t t = 4 * (i0 + x) + (lane >> 3);
              v[x] = *reinterpret_cast<const uint4*>(panel + kPanel + t * 128 + ((c ^ (t & 7)) << 4));
            }
            __syncwarp();                                        // (these rows have been read)
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
              const uint32_t t = 4 * (i0 + x) + (lane >> 3), sw = t & 7;
              if (nan_codes(v[x].x) | nan_codes(v[x].y) | nan_codes(v[x].z) | nan_codes(v[x].w)) nan_of |= 1u << (i0 + x);
              // codes 16 c .. + 15 are the chunks 2 c and 2 c + 1 of the row's 16
              uint8_t* to = panel + (c >> 2) * kPanel + t * 128;
              const uint32_t ch = (2 * c) & 7;
              *reinterpret_cast<uint4*>(to + ((ch ^ sw) << 4)) =
                  make_uint4(codes2_bf16(v[x].x), codes2_bf16(v[x].x >> 16), codes2_bf16(v[x].y), codes2_bf16(v[x].y >> 16));
              *reinterpret_cast<uint4*>(to + (((ch + 1) ^ sw) << 4)) =
                  make_uint4(codes2_bf16(v[x].z), codes2_bf16(v[x].z >> 16), codes2_bf16(v[x].w), codes2_bf16(v[x].w >> 16));
            }
          }
          uint32_t bad = 0;                                      // tokens of the 32 with a NaN among their codes
          if (__any_sync(0xFFFFFFFFu, nan_of != 0)) {
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
              const uint32_t which = __ballot_sync(0xFFFFFFFFu, (nan_of >> i) & 1u);
#pragma unroll
              for (int x = 0; x < 4; ++x) bad |= (which >> (8 * x)) & 0xFFu ? 1u << (4 * i + x) : 0u;
            }
          }
          const uint32_t two = g < 2 ? scales[j].x : scales[j].y;
          const float ks = key_scale_of((uint16_t)(g & 1 ? two >> 16 : two & 0xFFFFu));
          key_scale[g * W::kTokens + at + lane] = (bad >> lane) & 1u ? __int_as_float(0x7FC00000) : ks;
        }
      }
      fence_async_smem();
      mbar_arrive(k_full(k));
    };
    send(0);
    send(1);                                         // (a tile has four steps)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    hand_on(0);
#pragma unroll 1
    for (int k = 1; k < heads; ++k) {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      hand_on(k);
      if (k + 1 == heads) break;
      ok = mbar_wait_warp(k_empty(k + 1), head_of(k - 1), err, kKernWeights);
      if (!ok) break;
      send(k + 1);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  } else if (warp >= W::kRoleQueries && warp < W::kRoleMma) {
    // ---- Q: a turn each at a time, so that the next are on their way while one lands;
    // column query * 4 + head
    const int w = warp - W::kRoleQueries;
    int i = 0;
#pragma unroll 1
    for (int v = blockIdx.x; v < seen_tiles && ok; v += gridDim.x) {
      const Range r = range_of(v);
#pragma unroll 1
      for (int j = 0, g = 0, at = 0; j < kKvHeads * r.per && ok; ++j, ++i, ++at) {
        if (at == r.per) at = 0, ++g;
        if (i % W::kQueryWarps != w) continue;
        const int c = r.c0 + at;
        if (i >= kRing) ok = mbar_wait_warp(empty(i), turn_of(i - kRing), err, kKernWeights);
        if (!ok) break;
        const int qa = c * kTurnQueries, have = nq - qa < kTurnQueries ? nq - qa : kTurnQueries;
        const uint32_t dst = sb + W::kOffQ + (i % kRing) * W::kQBytes + ((lane & 15) >> 3) * W::kQPanel;
        // two columns at a time, 16 lanes each: heads 2 (k & 1) + (lane >> 4) of query k / 2
        const uint16_t* from = p.q + ((int64_t)(x0 + qa) * kQHeads + g * kGroup + (lane >> 4)) * kHeadDim + (lane & 15) * 8;
#pragma unroll 8
        for (int k = 0; k < kTurnCols / 2; ++k) {
          const int cc = 2 * k + (lane >> 4);
          const bool there_is = (k >> 1) < have;
          cp_async16(dst + cc * 128 + (((lane & 7) ^ (cc & 7)) << 4),
                     there_is ? from + ((k >> 1) * kQHeads + 2 * (k & 1)) * kHeadDim : p.q, there_is ? 16u : 0u);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        Columns& m = columns[i % W::kColumns];
        bool dead = false;
        for (int col = lane; col < kTurnCols; col += 32) {
          const int q = col / kGroup;
          const float lse = q < have ? p.lse[(int64_t)(x0 + qa + q) * kQHeads + g * kGroup + col % kGroup] : -INFINITY;
          const float2 y = column_of(lse);
          m.minus[col] = y.x;
          m.factor[col] = y.y;
          dead = dead || lse == -INFINITY;
        }
        dead = __any_sync(0xFFFFFFFFu, dead);
        if (lane == 0) m.dead = dead;
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full(i));
      }
    }
  } else if (warp == W::kRoleMma) {
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    int i = 0, k = 0;
#pragma unroll 1
    for (int v = blockIdx.x; v < seen_tiles && ok; v += gridDim.x) {
      const Range r = range_of(v);
#pragma unroll 1
      for (int j = 0, c = 0; j < kKvHeads * r.per && ok; ++j, ++i, ++c) {
        if (c == r.per) c = 0, ++k;
        const int left = (nq - (r.c0 + c) * kTurnQueries) * kGroup;
        const uint32_t cols = left >= kTurnCols ? kTurnCols : (uint32_t)((left + 15) / 16 * 16);
        if (c == 0) ok = mbar_wait_warp(k_full(k), head_of(k), err, kKernWeights);
        if (ok) ok = mbar_wait_warp(full(i), turn_of(i), err, kKernWeights);
        if (ok && i >= kRing) ok = mbar_wait_warp(d_empty(i), turn_of(i - kRing), err, kKernWeights);
        if (!ok) break;
        fence_after();
        if (elect_one()) {
          const uint32_t id = idesc_bf16(cols, false);
          const uint64_t qd = desc_sw128(sb + W::kOffQ + (i % kRing) * W::kQBytes, 16);
#pragma unroll
          for (int m = 0; m < kTiles; ++m) {
            const uint64_t kd = desc_sw128(sb + (k & 1) * W::kKBytes + m * 2 * kPanel, 16);
#pragma unroll
            for (int x = 0; x < kHeadDim / 16; ++x)
              mma_ss(tm + (uint32_t)((i % kRing) * 128 * kTiles + m * kTurnCols), kd + (uint64_t)(((x >> 2) * kPanel + (x & 3) * 32) >> 4),
                     qd + (uint64_t)(((x >> 2) * W::kQPanel + (x & 3) * 32) >> 4), id, x != 0);
          }
          mbar_arrive(d_full(i));                    // passes on the loaders' writes of the columns
          commit(d_full(i));
          commit(empty(i));
          if (c == r.per - 1) commit(k_empty(k));
        }
        __syncwarp();
      }
      ++k;
    }
    // every product is complete before tensor memory is given back
    for (int e = i > kRing ? i - kRing : 0; e < i; ++e) mbar_wait_warp(empty(e), turn_of(e), err, kKernWeights);
  } else {
    // ---- epilogue: thread = token; part `part` of four: of the columns, and with
    // two tiles of 128 of these
    const int part = warp >> 2, at = (kTiles == 2 ? 128 * (part >> 1) : 0) + 32 * (warp & 3) + lane;
    const int first = kEpiCols * (kTiles == 2 ? part & 1 : part);            // its columns of a turn
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(kEpiCols * part);
    int i = 0, odd = 0;                              // odd: the tile's place in what two tiles share
#pragma unroll 1
    for (int v = blockIdx.x; v < seen_tiles; v += gridDim.x, odd ^= 1) {     // (all warps meet in every tile, whatever has run out)
      const Range r = range_of(v);
      const int64_t t = r.t0 + at;
      const float* key_scale = reinterpret_cast<const float*>(smem + W::kOffKs) + odd * kKvHeads * W::kTokens;
      const uint32_t* there = reinterpret_cast<const uint32_t*>(smem + W::kOffThere) + 8 * odd;
      float* part_sum = reinterpret_cast<float*>(smem + W::kOffSum) + odd * 4 * 128;
      // queries that see the token, from the first turn's on
      int64_t low = t - pos0, high = t < p.d.sinks ? nq : t + p.d.window - pos0;
      if (low < 0) low = 0;
      if (high > nq) high = nq;
      const int qlo = (int)low, qhi = (int)(high < 0 ? 0 : high);
      float hi = p.scale_log2, lo = p.scale_rest;
      uint64_t hi2 = pair(hi, hi), lo2 = pair(lo, lo);
      float total = 0.f;
      bool mine = false;
#pragma unroll 1
      for (int j = 0, g = 0, c = 0; j < kKvHeads * r.per; ++j, ++i, ++c) {
        if (c == r.per) c = 0, ++g;
        const int qa = (r.c0 + c) * kTurnQueries;
        if (ok) ok = mbar_wait_warp(d_full(i), turn_of(i), err, kKernWeights);
        if (!ok) break;
        fence_after();
        if (j == 0) mine = (there[at >> 5] >> (at & 31)) & 1u;
        if (kFp8 && c == 0) {                        // times the token's K scale, the rounding into the rest
          const float ks = key_scale[g * W::kTokens + at];
          hi = __fmul_rz(p.scale_log2, ks);          // (both parts of one sign: an infinite logit stays one)
          lo = fmaf(p.scale_rest, ks, fmaf(p.scale_log2, ks, -hi));
          hi2 = pair(hi, hi);
          lo2 = pair(lo, lo);
        }
        const Columns& cm = columns[i % W::kColumns];
        // columns a .. z - 1 count for this token
        int a = (qlo - qa) * kGroup, z = (qhi - qa) * kGroup;
        a = a < 0 ? 0 : (a > kTurnCols ? kTurnCols : a);
        z = z < 0 ? 0 : (z > kTurnCols ? kTurnCols : z);
        const uint32_t d = lane_base + (uint32_t)(i % kRing) * (128u * kTiles);
        uint64_t sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
        // four columns (a query's heads) of a turn
        auto four = [&](uint32_t* x, int cc, ulonglong2& mi, float (&e)[4]) {
          mi = *reinterpret_cast<const ulonglong2*>(&cm.minus[cc]);
          const uint64_t x01 = pair(x[0], x[1]), x23 = pair(x[2], x[3]);
          const uint64_t y01 = fma2(x01, lo2, fma2(x01, hi2, mi.x)), y23 = fma2(x23, lo2, fma2(x23, hi2, mi.y));
          e[0] = exp2_fast(lo_of(y01));
          e[1] = exp2_fast(hi_of(y01));
          e[2] = exp2_fast(lo_of(y23));
          e[3] = exp2_fast(hi_of(y23));
        };
        auto add = [&](int cc, const float (&e)[4]) {
          const ulonglong2 fa = *reinterpret_cast<const ulonglong2*>(&cm.factor[cc]);
          sum[0] = fma2(pair(e[0], e[1]), fa.x, sum[0]);
          sum[1] = fma2(pair(e[2], e[3]), fa.y, sum[1]);
        };
        const bool some = __any_sync(0xFFFFFFFFu, a < z && z > first && a < first + kEpiCols);
        const bool plain = __all_sync(0xFFFFFFFFu, a <= first && z >= first + kEpiCols) && !cm.dead;
#pragma unroll 1
        for (int x = 0; x < kEpiCols && some; x += 32) {
          uint32_t s[32];
          ld32(d + (uint32_t)x, s);
          wait_ld();
          reg_fence(s);
          if (plain) {
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              ulonglong2 mi;
              float e[4];
              four(&s[k], first + x + k, mi, e);
              add(first + x + k, e);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const int cc = first + x + k;
              ulonglong2 mi;
              float e[4];
              four(&s[k], cc, mi, e);
              const bool in = cc >= a && cc < z;
              const float mm[4] = {lo_of(mi.x), hi_of(mi.x), lo_of(mi.y), hi_of(mi.y)};
#pragma unroll
              for (int h = 0; h < 4; ++h)            // (columns without weight, and past the queries: minus is +inf)
                if (!in || mm[h] == INFINITY) e[h] = 0.f;
              add(cc, e);
            }
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(d_empty(i));
        const uint64_t s2 = add2(sum[0], sum[1]);
        total += lo_of(s2) + hi_of(s2);
      }
      part_sum[part * 128 + 32 * (warp & 3) + lane] = total;
      asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
      const float* sums = part_sum + 32 * (warp & 3) + lane;
      if (kTiles == 2 ? (part & 1) == 0 : part == 0) {
        total = kTiles == 2 ? sums[part * 128] + sums[part * 128 + 128] : (sums[0] + sums[128]) + (sums[256] + sums[384]);
        if (ok && t < r.t1) store_weight(p, u, t, mine ? total : 0.f);
      }
    }
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (warp == W::kRoleMma) tmem_free<kTmemCols>(tmem);
}

}  // namespace

cudaError_t launch_window_weights(const DenseAttn& d, const uint16_t* q, const float* lse, float softmax_scale,
                                  float* weights, int64_t stride, bool accumulate, cudaStream_t s) {
  static PerDeviceOnce setup;
  cudaError_t e = setup.run([] {
    cudaError_t r = prefer_max_shared(weight_wide_kernel<false, 1>, Wide<1>::kSmem);
    if (r == cudaSuccess) r = prefer_max_shared(weight_wide_kernel<true, 1>, Wide<1>::kSmem);
    if (r == cudaSuccess) r = prefer_max_shared(weight_wide_kernel<false, 2>, Wide<2>::kSmem);
    if (r == cudaSuccess) r = prefer_max_shared(weight_wide_kernel<true, 2>, Wide<2>::kSmem);
    if (r == cudaSuccess) r = prefer_max_shared(weight_few_kernel<false, 1>, FewLayout<false>::kSmem);
    if (r == cudaSuccess) r = prefer_max_shared(weight_few_kernel<true, 1>, FewLayout<true>::kSmem);
    if (r == cudaSuccess) r = prefer_max_shared(weight_few_kernel<false, 2>, FewLayout<false>::kSmem);
    if (r == cudaSuccess) r = prefer_max_shared(weight_few_kernel<true, 2>, FewLayout<true>::kSmem);
    return r;
  });
  int sms = 0;
  if (e == cudaSuccess) e = current_sm_count(&sms);
  if (e != cudaSuccess) return e;
  WeightParams p;
  p.d = d;
  p.q = q;
  p.lse = lse;
  const bool fp8 = d.c.b.row_bytes == kRowBytesFp8;
  // both parts of one sign, and neither 0: an infinite logit stays one
  auto set_scale = [&](double f) {
    p.scale_log2 = (float)f;
    if (fabs((double)p.scale_log2) > fabs(f)) p.scale_log2 = nextafterf(p.scale_log2, 0.f);
    p.scale_rest = (float)(f - (double)p.scale_log2);
    if (p.scale_rest == 0.f) p.scale_rest = p.scale_log2 * 0x1p-40f;
  };
  const double f = (double)softmax_scale * 1.4426950408889634;
  p.weights = weights;
  p.stride = stride;
  p.accumulate = accumulate;
  int64_t wide = 0, few = 0, few_all = 0;            // the longest contexts; all tokens of few queries
  int wide_units = 0;
  int rows = 0;                                      // queries of a unit of few, at most
  int64_t seen = 0;                                  // tokens that more than a few queries see
  for (int u = 0; u < d.c.b.n_units; ++u) {
    const int64_t n = d.c.b.u[u].n;
    const int nq = d.c.unit_tokens(u);
    if (nq > kFewQueries) {
      wide = n > wide ? n : wide;
      ++wide_units;
      const int64_t low = n - nq - d.window + 1;
      seen += low > 0 ? n - low : n;
    } else {
      few = n > few ? n : few;
      few_all += n;
      rows = nq > rows ? nq : rows;
    }
  }
  if (wide > 0) {
    // tiles of 256 tokens where these fill the device
    const int tiles = seen >= (int64_t)sms * Wide<2>::kTokens ? 2 : 1;
    // as many CTAs as SMs, shared by the units with more than a few queries
    int64_t ctas = (wide + 128 * tiles - 1) / (128 * tiles);
    if (ctas > (sms + wide_units - 1) / wide_units) ctas = (sms + wide_units - 1) / wide_units;
    const dim3 grid((unsigned)ctas, d.c.b.n_units);
    set_scale(fp8 ? f : f * (1 + kCutOff));
    auto* kernel = fp8 ? (tiles == 2 ? weight_wide_kernel<true, 2> : weight_wide_kernel<true, 1>)
                       : (tiles == 2 ? weight_wide_kernel<false, 2> : weight_wide_kernel<false, 1>);
    e = launch_kernel(kernel, grid, dim3(tiles == 2 ? Wide<2>::kThreads : Wide<1>::kThreads), tiles == 2 ? Wide<2>::kSmem : Wide<1>::kSmem, s, 0, dim3(1), p);
  }
  if (e == cudaSuccess && few > 0) {
    // two CTAs on an SM: as many runs of tokens as that, a step of 32 tokens to each warp pair
    int64_t run = (few_all + 2 * sms - 1) / (2 * sms);
    run = (run + kFewStep - 1) / kFewStep * kFewStep;
    run = run < 2 * kFewStep ? 2 * kFewStep : (run > kFewMost ? kFewMost : run);
    p.few_tokens = (int32_t)run;
    set_scale(f);
    auto* kernel = fp8 ? (rows > 2 ? weight_few_kernel<true, 2> : weight_few_kernel<true, 1>)
                       : (rows > 2 ? weight_few_kernel<false, 2> : weight_few_kernel<false, 1>);
    e = launch_kernel(kernel, dim3((unsigned)((few + run - 1) / run), d.c.b.n_units), dim3(kFewThreads),
                      fp8 ? FewLayout<true>::kSmem : FewLayout<false>::kSmem, s, 0, dim3(1), p);
  }
  return e;
}

}  // namespace qsa
