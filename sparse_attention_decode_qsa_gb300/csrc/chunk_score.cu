// Index scores for every query of a chunk: as index_score.cu scores one
// query, each query against the tokens up to its own position
//     S_it = sum_h w_ih * relu(scale_t * sum_d q_i[h][d] * e4m3(code_t[d])),  t <= p_i
// reduced to C4 blocks (max over 4 adjacent tokens; "双卡RTX4090跑通Qwen3-Next：
// 8并发满血长上下文实测", opening explanation of QSA, and "Оффлоадинг KV-кэша
// Qwen3.8-Flash-Next в RAM через vLLM без потери скорости декодирования",
// section "Механизм гибридного разреженного оффлоадинга").
//
// 1024 flops per (query, token): a dense contraction keys[tokens][64] x
// q^T[64][queries x 8 heads], on the tensor cores (tcgen05, kind::f16, fp32
// accumulators) with f16 operands.  An e4m3 code is exact in f16, one
// conversion instruction for two.  A query row (one head) is scaled by a power
// of two until its largest element is in [2^14, 2^15), the upper end of f16's
// range; there f16 holds a bf16 element exactly down to 2^-31 of the largest and
// to 2^-39 of it below; an fp32 query goes in as two pieces (the round-to-nearest
// f16, and that of what is left: 11 bits each), which together are off by at most
// 2^-23 of the element, or 2^-39 of the row's largest.  Products are exact and
// sums are fp32.
//
// Tiling.  A group of 64 queries stays in shared memory as the B operand, four
// tiles of up to 128 columns (16 queries x 8 heads), while the keys stream
// past.  A step is 512 tokens = 128 blocks in four phases: phase k multiplies
// the tokens 4b + k, so that a tensor-memory lane is a block, and the thread
// that owns the lane takes the maximum over the block's four tokens in its
// registers, with no exchange between threads, and stores 32 neighbouring
// blocks per warp.
//
// Warp roles (one CTA per SM, all of tensor memory: four accumulators of
// 128 columns): 2 converter warps, one MMA warp, and 4 epilogue warps per
// accumulator (relu, head weights, scale, maximum), so that an accumulator's
// MMAs run while the others' are read.
// All waits are bounded.  The steps of all groups form one list, cut into
// equal runs, one per CTA; a run that crosses into another group rebuilds B.
//
// Measured: 2048 bf16 queries at the end of 131072 tokens (277 GFLOP) 345 us,
// 0.80 PFLOP/s, 0.41 of the measured bf16 rate; 2048 fp32 queries 417 us; 10 fp32 draft queries of 4 requests of
// 65536 tokens 14 us.  What bounds it is the epilogue's instructions: 8
// saturating products and 4 paired multiply-adds per query and lane against 128
// tensor-core cycles per tile; the schedulers issue in 0.66 of the cycles, and
// the loop without its arithmetic takes 207 us.  The shared-memory port is the next
// limit, busy in 0.7 of the cycles: of a phase's 3500, 1024 for the operands of the
// products and 1340 for the head weights, which every epilogue warp reads in each
// of the four phases (40 M load wavefronts).  Not faster: 128 queries to a
// group (413, registers spill), two sets of 8 warps with two accumulators each
// (357), products per element in place of pairs or maxima in place of saturation
// (359 to 392), an arrival per warp in place of per thread, an earlier release of
// the accumulator, a loop of its own for tokens that every query sees (345 to 376).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "tc_common.cuh"

namespace qsa {
namespace {

using namespace tc;

constexpr int kAccs = 4;                          // tiles, each with its accumulator
constexpr int kAccCols = 512 / kAccs;
constexpr int kTileQueries = kAccCols / kIndexHeads;             // at most, per tile: 16
constexpr int kGroup = kAccs * kTileQueries;      // queries per group: 64
constexpr int kFewQueries = 4;                    // that a single tile takes
constexpr int kEpiWarps = 4;                      // epilogue warps per accumulator
constexpr int kConvWarps = 2;
constexpr int kConvLoads = 512 / (32 * kConvWarps);              // 16-byte loads per lane and phase
// 19 warps: five on a scheduler at most, which leaves 96 registers per thread
constexpr int kThreads = 32 * (kAccs * kEpiWarps + kConvWarps + 1);
constexpr int kRoleConv = kAccs * kEpiWarps, kRoleMma = kRoleConv + kConvWarps;
constexpr int kStepTokens = 512;                  // tokens per step: 128 blocks of 4
constexpr int kABytes = 128 * kIndexDim * 2;      // one phase: 128 tokens of 64 f16
constexpr int kBTile = kAccCols * kIndexDim * 2;  // 16 KiB
constexpr uint32_t kTmemCols = 512;

// Shared memory: the ring of phases (16 KiB each), B (piece by piece, tile by
// tile), head weights, barriers.
template <bool kBf16>
struct Layout {
  static constexpr int kPieces = kBf16 ? 1 : 2;
  static constexpr int kStages = kBf16 ? 6 : 5;
  static constexpr int kOffB = kStages * kABytes;
  static constexpr int kOffW = kOffB + kAccs * kPieces * kBTile;
  static constexpr int kOffBar = kOffW + kGroup * kIndexHeads * 4;
  static constexpr int kNumBars = 2 * kStages + 2 * kAccs + 1;   // a_full, a_empty, d_full, d_empty, done
  static constexpr int kOffSlot = kOffBar + 8 * kNumBars;
  static constexpr int kSmemBytes = kOffSlot + 16 + 1024;        // + alignment to 1024
  static_assert(kSmemBytes <= 227 * 1024, "one CTA's shared memory");
};

struct ChunkScoreParams {
  ChunkDesc c;
  int32_t step0[kMaxUnits + 1];   // prefix sums of the steps per unit
  const void* q_idx;              // [rows][8][64] fp32 or bf16
  const float* w;                 // [rows][8]
  float* blk;                     // [rows][blk_stride]
  int64_t blk_stride;
};

// Steps of the first j groups of a unit whose first query is at position
// `first`: group i sees the steps up to its last query's, (first + (i + 1) G -
// 1) / 512 + 1 of them.  With R = 512 / G and A = (first + G - 1) / G that is
// (A + i) / R + 1, so the sum is closed.  (The unit's last group may hold
// fewer queries and fewer steps; the callers cap it.)
__host__ __device__ __forceinline__ int64_t steps_before(int64_t first, int64_t j) {
  constexpr int64_t G = kGroup, R = kStepTokens / G;
  const int64_t A = (first + G - 1) / G;
  auto S = [](int64_t m) { const int64_t q = m / R; return R * q * (q - 1) / 2 + (m % R) * q; };
  return S(A + j) - S(A) + j;
}
__host__ __device__ __forceinline__ int64_t unit_steps(int64_t n, int64_t tokens) {
  if (tokens == 0) return 0;
  const int64_t groups = (tokens + kGroup - 1) / kGroup;
  return steps_before(n - tokens, groups - 1) + (n - 1) / kStepTokens + 1;
}

// Four codes as f16.
__device__ __forceinline__ uint2 convert4(uint32_t w) {
  const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
  const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
  return make_uint2((uint32_t)a.x | ((uint32_t)a.y << 16), (uint32_t)b.x | ((uint32_t)b.y << 16));
}

// relu(x) * 2^-30 of dot products |x| <= 2^30 (64 elements up to 2^15 by codes up
// to 448), two as a pair: a saturating multiplication, which runs on the
// multiply-add pipe; the one that takes maxima is half as wide.  Products and
// multiply-adds of pairs.
__device__ __forceinline__ uint64_t relu2(uint32_t a, uint32_t b) {
  uint64_t d;
  asm("{\n .reg .f32 x, y;\n mul.sat.f32 x, %1, 0f30800000;\n mul.sat.f32 y, %2, 0f30800000;\n"
      " mov.b64 %0, {x, y};\n}\n"
      : "=l"(d)
      : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// kFew: no group has more than kFewQueries (draft tokens), which all fall into
// one tile.  Its phases then take the four accumulators in turn, and the warps of
// the missing tiles convert too (the kernel alone, with cold caches: 14 bf16
// queries over 8 x 32768 tokens 20.2 -> 16.4 us, 10 fp32 queries over 4 x 65536
// 20.1 -> 16.9, with half of the teams 20).  Run-time choices in one kernel cost
// the full groups 10 %.  One request with five queries takes the call to the
// general form: 8 requests of 32768 tokens with 1, 4, 5, 8, 16, 32 bf16 queries each
// 14.1, 13.6, 17.5, 17.8, 24.0, 27.6 us in a loop.  Both pieces of fp32 queries side by side in one product,
// added in the epilogue, are slower (21.3).
template <bool kBf16, bool kFew>
__global__ void __launch_bounds__(kThreads, 1) chunk_score_kernel(const __grid_constant__ ChunkScoreParams p) {
  using L = Layout<kBf16>;
  constexpr int kPieces = L::kPieces, kStages = L::kStages, kQueries = kFew ? kFewQueries : kTileQueries;
  constexpr int kOffB = L::kOffB, kOffW = L::kOffW, kOffBar = L::kOffBar, kOffSlot = L::kOffSlot;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  float* sw = reinterpret_cast<float*>(smem + kOffW);
  const uint32_t bars = sb + kOffBar;
  auto a_full = [&](int i) { return bars + 8u * (uint32_t)i; };
  auto a_empty = [&](int i) { return bars + 8u * (uint32_t)(kStages + i); };
  auto d_full = [&](int i) { return bars + 8u * (uint32_t)(2 * kStages + i); };
  auto d_empty = [&](int i) { return bars + 8u * (uint32_t)(2 * kStages + kAccs + i); };
  const uint32_t done = bars + 8u * (uint32_t)(2 * kStages + 2 * kAccs);
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + kOffSlot);
  __shared__ int s_fail, s_leader;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  ErrorWord* err = p.c.b.err;

  if (warp == kRoleMma) {
    tmem_alloc<kTmemCols>(slot);
    if (elect_one()) s_leader = lane;          // the lane that issues MMAs
    if (lane == 0) {
      for (int i = 0; i < kStages; ++i) { mbar_init(a_full(i), 32 * kConvWarps); mbar_init(a_empty(i), 1); }
      for (int i = 0; i < kAccs; ++i) { mbar_init(d_full(i), 1); mbar_init(d_empty(i), 32 * kEpiWarps); }
      mbar_init(done, 1);
      mbar_fence_init();
      s_fail = 0;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *slot;
  grid_dependency_wait();

  const int64_t total = p.step0[p.c.b.n_units];
  int64_t at = total * blockIdx.x / gridDim.x;
  const int64_t end = total * (blockIdx.x + 1) / gridDim.x;
  int phase = 0;      // phases streamed by this CTA (ring position)
  int fills = 0;      // epilogue: times its accumulator was filled (kFew: its accumulators, in turn)
  uint32_t used = 0, turn = 0;   // MMA warp, a bit per accumulator: filled before, parity of the next wait
  while (at < end) {
    // ---- the group and its part of the run
    int u = 0;
    {
      int lo = 0, hi = p.c.b.n_units - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.step0[mid] <= at) lo = mid; else hi = mid - 1;
      }
      u = lo;
    }
    const int64_t n = p.c.b.u[u].n;
    const int tokens = p.c.unit_tokens(u);
    const int64_t first = n - tokens, local = at - p.step0[u];
    int grp = 0;
    {
      int lo = 0, hi = (tokens + kGroup - 1) / kGroup - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (steps_before(first, mid) <= local) lo = mid; else hi = mid - 1;
      }
      grp = lo;
    }
    const int nq = tokens - grp * kGroup < kGroup ? tokens - grp * kGroup : kGroup;
    const int64_t pos0 = first + (int64_t)grp * kGroup;             // position of the group's first query
    const int x0 = p.c.row0[u] + grp * kGroup;
    const int64_t s0 = local - steps_before(first, grp);
    const int64_t s_all = (pos0 + nq - 1) / kStepTokens + 1;
    const int64_t s1 = s_all - s0 < end - at ? s_all : s0 + (end - at);
    at += s1 - s0;
    const int64_t row0 = p.c.b.unit_row(u);
    // queries per tile (a multiple of 4: 32 columns) and tiles with queries
    const int qt = ((nq + kAccs - 1) / kAccs + 3) / 4 * 4;
    const int tiles = kFew ? 1 : (nq + qt - 1) / qt;

    // ---- B and the head weights (all threads; the previous run is complete).
    // Row r of a tile is head r & 7 of the tile's query r >> 3, scaled by 2^(15-k)
    // (its largest element is in [2^(k-1), 2^k)); its head weight takes 2^k, the
    // key's scale the rest: 2^30 of relu2 over 2^15.  So a weighted dot product
    // overflows where the score's own terms do.  Rows past the group are 0.
    for (int i = tid; i < tiles * qt * kIndexHeads * (kIndexDim / 8); i += kThreads) {
      const int c = i & 7, r = i >> 3;                         // chunk of 8 places, row over all tiles
      const int q = r >> 3;
      float v[8], top = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = 0.f;
        if (q < nq) {
          const int64_t src = ((int64_t)x0 * kIndexHeads + r) * kIndexDim + 8 * c + e;
          v[e] = kBf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.q_idx)[src])
                       : reinterpret_cast<const float*>(p.q_idx)[src];
        }
        top = fmaxf(top, fabsf(v[e]));
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));   // the row's 8 lanes
      int k = 0;
      if (top > 0.f) frexpf(top, &k);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = ldexpf(v[e], 15 - k);
      if (c == 0) sw[r] = q < nq ? ldexpf(p.w[(int64_t)x0 * kIndexHeads + r], k) : 0.f;
      const int tile = q / qt, tr = r - tile * qt * kIndexHeads;
      uint8_t* dst = smem + kOffB + tile * kBTile + tr * 128 + ((c ^ (tr & 7)) << 4);
#pragma unroll
      for (int pc = 0; pc < kPieces; ++pc) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __half2 b = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
          o[e] = *reinterpret_cast<const uint32_t*>(&b);
          v[2 * e] -= __low2float(b);                          // exact
          v[2 * e + 1] -= __high2float(b);
        }
        *reinterpret_cast<uint4*>(dst + pc * kAccs * kBTile) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    fence_async_smem();
    __syncthreads();

    const int steps = (int)(s1 - s0);
    bool ok = true;
    // teams of kConvWarps converter warps, each with every kTeams-th phase
    constexpr int kTeams = kFew ? 4 : 1;
    const int spare = warp - kEpiWarps;
    const int team = warp >= kRoleConv ? 0 : 1 + spare / kConvWarps;
    if (kFew ? spare >= 0 && warp < kRoleMma && team < kTeams : warp >= kRoleConv && warp < kRoleMma) {
      // ---- converters: 16 codes per lane and load; lanes 4i .. 4i+3 hold one
      // token, a load of a warp 8 blocks, the next phase's loads in flight.  A
      // negative scale turns the code's sign.
      const int wc = (warp >= kRoleConv ? warp - kRoleConv : spare) % kConvWarps, sub = lane >> 2, part = lane & 3;
      const uint8_t* keys = p.c.b.index_keys + row0 * kIndexDim + part * 16;
      const uint16_t* scales = p.c.b.index_scales + row0;
      uint4 v[2][kConvLoads];
      uint32_t negative[2];                                    // bit j: load j's scale is negative
      auto load = [&](int e, int i) {                          // phase i of the run
        const int64_t t0 = (s0 + (i >> 2)) * kStepTokens + 4 * (wc * 8 * kConvLoads + sub) + (i & 3);
        negative[e] = 0;
#pragma unroll
        for (int j = 0; j < kConvLoads; ++j) {
          const int64_t t = t0 + 32 * j;
          const bool in = i < 4 * steps && t < n;
          v[e][j] = in ? __ldg(reinterpret_cast<const uint4*>(keys + t * kIndexDim)) : make_uint4(0, 0, 0, 0);
          negative[e] |= in ? (uint32_t)(__ldg(scales + t) >> 15) << j : 0u;
        }
      };
      const int first_phase = kFew ? team : 0;
      load(0, first_phase);
      load(1, first_phase + kTeams);
#pragma unroll 1
      for (int i0 = first_phase; i0 < 4 * steps && ok; i0 += 2 * kTeams) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (kFew && i0 + e * kTeams >= 4 * steps) break;
          const int ph = phase + i0 + e * kTeams, st = ph % kStages;
          if (ok && ph >= kStages) ok = mbar_wait(a_empty(st), (uint32_t)(ph / kStages - 1) & 1u, err, kKernChunkScore);
          if (!ok) break;
          uint8_t* A = smem + st * kABytes;
#pragma unroll
          for (int j = 0; j < kConvLoads; ++j) {
            const int r = (wc * kConvLoads + j) * 8 + sub;
            const uint32_t flip = (negative[e] >> j) & 1u ? 0x80808080u : 0u;
            const uint2 a = convert4(v[e][j].x ^ flip), b = convert4(v[e][j].y ^ flip);
            const uint2 c = convert4(v[e][j].z ^ flip), d = convert4(v[e][j].w ^ flip);
            *reinterpret_cast<uint4*>(A + r * 128 + (((2 * part) ^ (r & 7)) << 4)) = make_uint4(a.x, a.y, b.x, b.y);
            *reinterpret_cast<uint4*>(A + r * 128 + (((2 * part + 1) ^ (r & 7)) << 4)) =
                make_uint4(c.x, c.y, d.x, d.y);
          }
          load(e, i0 + (e + 2) * kTeams);
          fence_async_smem();
          mbar_arrive(a_full(st));
        }
      }
    } else if (warp == kRoleMma) {
      const uint32_t idesc = idesc_f16((uint32_t)(8 * qt), false);
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      int st = phase % kStages;
      uint32_t lap = (uint32_t)(phase / kStages) & 1u;
#pragma unroll 1
      for (int i = 0; i < 4 * steps && ok; ++i) {
        ok = mbar_wait_warp(a_full(st), lap, err, kKernChunkScore);
#pragma unroll 1
        for (int t = 0; t < tiles && ok; ++t) {
          const int acc = kFew ? i % kAccs : t;
          if ((used >> acc) & 1u) ok = mbar_wait_warp(d_empty(acc), (turn >> acc) & 1u, err, kKernChunkScore);
          if (!ok) break;
          turn ^= ((used >> acc) & 1u) << acc;
          used |= 1u << acc;
          fence_after();
          if (elect_one()) {
            const uint32_t d = tm + (uint32_t)(kAccCols * acc), a = sb + st * kABytes;
            const uint64_t a0 = desc_sw128(a, 16), b0 = desc_sw128(sb + kOffB + t * kBTile, 16);
#pragma unroll
            for (int pc = 0; pc < kPieces; ++pc)
#pragma unroll
              for (int ks = 0; ks < kIndexDim / 16; ++ks)
                mma_ss(d, a0 + 2 * ks, b0 + (uint64_t)(pc * kAccs * kBTile / 16 + 2 * ks), idesc, (pc | ks) != 0);
            commit(d_full(acc));
            if (t == tiles - 1) commit(a_empty(st));
          }
          __syncwarp();
        }
        if (++st == kStages) { st = 0; lap ^= 1u; }
      }
    } else if (warp / kEpiWarps < tiles) {
      // ---- epilogue of one tile: thread = block (tensor-memory lane).  The
      // loops over steps and phases stay rolled: with all phases unrolled the
      // roles' code outgrew the instruction cache.
      const int tile = warp / kEpiWarps, row = (warp & 3) * 32 + lane;
      const int q0 = tile * qt, mine = nq - q0 < qt ? nq - q0 : qt;      // the tile's queries
      const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (kFew ? 0u : (uint32_t)(kAccCols * tile));
      const uint16_t* scales = p.c.b.index_scales + row0;
      const ulonglong2* wq = reinterpret_cast<const ulonglong2*>(sw + q0 * kIndexHeads);
      uint16_t next[4];
      auto load_scales = [&](int64_t s) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t t = s * kStepTokens + 4 * row + k;
          next[k] = t < n ? __ldg(scales + t) : (uint16_t)0;
        }
      };
      load_scales(s0);
#pragma unroll 1
      for (int s = 0; s < steps && ok; ++s) {
        const int64_t b0 = (s0 + s) * (kStepTokens / 4);
        const int64_t t0 = 4 * (b0 + row);                     // the block's first token
        float mag[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) mag[k] = fabsf(__half2float(__ushort_as_half(next[k]))) * 0x1p15f;
        if (s + 1 < steps) load_scales(s0 + s + 1);
        // every token of the step within every query's context?
        const bool whole = (s0 + s + 1) * kStepTokens - 1 <= pos0;
        float best[kQueries];
#pragma unroll
        for (int i = 0; i < kQueries; ++i) best[i] = -INFINITY;
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          const float m = k < 2 ? (k == 0 ? mag[0] : mag[1]) : (k == 2 ? mag[2] : mag[3]);
          const int acc = kFew ? k : tile;
          ok = mbar_wait(d_full(acc), (uint32_t)(kFew ? fills >> 2 : fills) & 1u, err, kKernChunkScore);
          ++fills;
          if (!ok) break;
          fence_after();
          // the tile's queries before `from` do not see this token
          const int64_t from = t0 + k - pos0 - q0;
#pragma unroll
          for (int c = 0; c < kQueries / 4; ++c) {             // four queries: 32 columns
            if (4 * c >= mine) break;
            uint32_t v[32];
            ld32(lane_base + (kFew ? (uint32_t)(kAccCols * k) : 0u) + 32u * (uint32_t)c, v);
            wait_ld();
            reg_fence(v);
            float y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t* x = &v[8 * i];
              const ulonglong2 wa = wq[2 * (4 * c + i)], wb = wq[2 * (4 * c + i) + 1];
              uint64_t sum = mul2(wa.x, relu2(x[0], x[1]));
              sum = fma2(wa.y, relu2(x[2], x[3]), sum);
              sum = fma2(wb.x, relu2(x[4], x[5]), sum);
              sum = fma2(wb.y, relu2(x[6], x[7]), sum);
              y[i] = (__uint_as_float((uint32_t)sum) + __uint_as_float((uint32_t)(sum >> 32))) * m;
            }
            if (!whole) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (4 * c + i < from) y[i] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) best[4 * c + i] = fmaxf(best[4 * c + i], y[i]);
          }
          fence_before();
          mbar_arrive(d_empty(acc));
        }
        if (!ok) break;
        float* o = p.blk + (int64_t)(x0 + q0) * p.blk_stride + b0 + row;
#pragma unroll
        for (int i = 0; i < kQueries; ++i) {
          if (i >= mine) break;
          if (whole || t0 <= pos0 + q0 + i) *o = best[i];
          o += p.blk_stride;
        }
      }
    }
    phase += 4 * steps;
    if (!ok) s_fail = 1;
    fence_before();
    __syncthreads();
    fence_after();
    if (s_fail) break;
  }

  if (warp == kRoleMma) {
    // (chosen by s_leader, not by elect_one(): with that here the prompt case takes
    // 383 us in place of 345, its main loop is compiled differently)
    if (lane == s_leader) {
      commit(done);                 // every MMA issued above is complete once this arrives
      mbar_wait(done, 0, err, kKernChunkScore);
    }
    __syncwarp();
    tmem_free<kTmemCols>(tmem);
  }
}

template <bool kBf16, bool kFew>
cudaError_t launch(ChunkScoreParams& p, cudaStream_t s) {
  constexpr int kSmemBytes = Layout<kBf16>::kSmemBytes;
  static PerDeviceOnce setup;
  cudaError_t e = setup.run([] { return prefer_max_shared(chunk_score_kernel<kBf16, kFew>, kSmemBytes); });
  int sms = 0;
  if (e == cudaSuccess) e = current_sm_count(&sms);
  if (e != cudaSuccess) return e;
  int64_t total = 0;
  for (int u = 0; u < p.c.b.n_units; ++u) {
    p.step0[u] = (int32_t)total;
    total += unit_steps(p.c.b.u[u].n, p.c.unit_tokens(u));
    if (total > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  }
  p.step0[p.c.b.n_units] = (int32_t)total;
  const unsigned grid = (unsigned)(total < sms ? total : sms);
  return launch_kernel(chunk_score_kernel<kBf16, kFew>, dim3(grid), dim3(kThreads), kSmemBytes, s, 0, dim3(1), p);
}

}  // namespace

cudaError_t launch_chunk_score(const ChunkDesc& c, const void* q_idx, bool q_bf16, const float* w,
                               float* blk_scores, int64_t blk_stride, cudaStream_t s) {
  ChunkScoreParams p;
  p.c = c;
  p.q_idx = q_idx;
  p.w = w;
  p.blk = blk_scores;
  p.blk_stride = blk_stride;
  bool few = true;
  for (int u = 0; u < c.b.n_units; ++u) few = few && c.unit_tokens(u) <= kFewQueries;
  if (few) return q_bf16 ? launch<true, true>(p, s) : launch<false, true>(p, s);
  return q_bf16 ? launch<true, false>(p, s) : launch<false, false>(p, s);
}

}  // namespace qsa
