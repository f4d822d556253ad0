// Index scores for every query of a chunk: as index_score.cu scores one
// query, each query against the tokens up to its own position
//     S_it = sum_h w_ih * relu(scale_t * sum_d q_i[h][d] * e4m3(code_t[d])),  t <= p_i
// reduced to C4 blocks (max over 4 adjacent tokens; "双卡RTX4090跑通Qwen3-Next：
// 8并发满血长上下文实测", opening explanation of QSA, and "Оффлоадинг KV-кэша
// Qwen3.8-Flash-Next в RAM через vLLM без потери скорости декодирования",
// section "Механизм гибридного разреженного оффлоадинга").
//
// 1024 flops per (query, token): a dense contraction keys[tokens][64] x
// q^T[64][queries x 8 heads], on the tensor cores (tcgen05, kind::f16, bf16
// operands, fp32 accumulators).  An e4m3 code is exact in bf16; an fp32 query
// goes in as three bf16 pieces (q = p0 + p1 + p2, each the round-to-nearest
// bf16 of what is left: 24 bits), accumulated in the same tile, a bf16 query
// as itself.  So products are exact and sums are fp32.
//
// Tiling.  A group of queries (64 bf16 ones, 32 fp32 ones: what three pieces
// leave room for) stays in shared memory as the B operand, up to 256 columns
// (32 queries x 8 heads) per tile, while the keys stream past.  A step is 512
// tokens = 128 blocks in four phases: phase k multiplies the tokens 4b + k, so
// that a tensor-memory lane is a block, and the thread that owns the lane
// takes the maximum over the block's four tokens in its registers, with no
// exchange between threads, and stores 32 neighbouring blocks per warp.
// The codes are turned into bf16 on the way from global to shared memory:
// exponent and mantissa bits move into place and one multiplication by 2^120
// corrects the bias (subnormal codes included).
//
// Warp roles (one CTA per SM, all of tensor memory: two accumulators of 256
// columns): 8 epilogue warps (relu, head weights, scale, maximum), 4 converter
// warps (a step's codes in flight in registers), one MMA warp.  All waits are
// bounded.  The steps of all groups form one list, cut into equal runs, one
// per CTA; a run that crosses into another group rebuilds B.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tc_common.cuh"

namespace qsa {
namespace {

using namespace tc;

constexpr int kEpiWarps = 8, kConvWarps = 4;
constexpr int kThreads = 32 * (kEpiWarps + kConvWarps + 1);     // 416
constexpr int kRoleConv = kEpiWarps, kRoleMma = kEpiWarps + kConvWarps;
constexpr int kTileQueries = 32;                  // queries per B tile: 256 columns
constexpr int kStepTokens = 512;                  // tokens per step: 128 blocks of 4
constexpr int kABytes = 128 * kIndexDim * 2;      // one phase: 128 tokens of 64 bf16
constexpr int kBTile = 8 * kTileQueries * kIndexDim * 2;        // 32 KiB
constexpr uint32_t kTmemCols = 512;

// Shared memory: the ring of phases (16 KiB each; a step's four stay until
// both tiles have read them), B, head weights, barriers.
template <bool kBf16>
struct Layout {
  static constexpr int kGroup = kBf16 ? 64 : 32;                 // queries per group
  static constexpr int kQTiles = kGroup / kTileQueries;          // accumulators per phase
  static constexpr int kPieces = kBf16 ? 1 : 3;
  static constexpr int kStages = kBf16 ? 8 : 6;
  static constexpr int kOffB = kStages * kABytes;
  static constexpr int kOffW = kOffB + kQTiles * kPieces * kBTile;
  static constexpr int kOffBar = kOffW + kGroup * kIndexHeads * 4;
  static constexpr int kNumBars = 2 * kStages + 4 + 1;           // a_full, a_empty, d_full, d_empty, done
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
template <int G>
__host__ __device__ __forceinline__ int64_t steps_before(int64_t first, int64_t j) {
  constexpr int64_t R = kStepTokens / G;
  const int64_t A = (first + G - 1) / G;
  auto S = [](int64_t m) { const int64_t q = m / R; return R * q * (q - 1) / 2 + (m % R) * q; };
  return S(A + j) - S(A) + j;
}
template <int G>
__host__ __device__ __forceinline__ int64_t unit_steps(int64_t n, int64_t tokens) {
  if (tokens == 0) return 0;
  const int64_t groups = (tokens + G - 1) / G;
  return steps_before<G>(n - tokens, groups - 1) + (n - 1) / kStepTokens + 1;
}

// Two bf16 from two e4m3 codes placed at bits 7-0 and 23-16 of x.
__device__ __forceinline__ uint32_t to_bf16x2(uint32_t magnitude_at_4, uint32_t sign_at_15) {
  const uint32_t raw = magnitude_at_4 | sign_at_15;
  uint32_t out;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(out) : "r"(raw), "r"(0x7B807B80u));   // 2^120 twice
  return out;
}
// Codes c0..c3 of a word as bf16 in the order c0, c2, c1, c3 (B has the same).
__device__ __forceinline__ uint2 convert4(uint32_t w) {
  return make_uint2(to_bf16x2((w & 0x007F007Fu) << 4, (w & 0x00800080u) << 8),
                    to_bf16x2((w & 0x7F007F00u) >> 4, w & 0x80008000u));
}
__device__ __forceinline__ int dim_of(int place) {
  const int r = place & 3;
  return (place & ~3) | (r == 1 ? 2 : r == 2 ? 1 : r);
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads, 1) chunk_score_kernel(const __grid_constant__ ChunkScoreParams p) {
  using L = Layout<kBf16>;
  constexpr int G = L::kGroup, kQTiles = L::kQTiles, kPieces = L::kPieces, kStages = L::kStages;
  constexpr int kOffB = L::kOffB, kOffW = L::kOffW, kOffBar = L::kOffBar, kOffSlot = L::kOffSlot;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  float* sw = reinterpret_cast<float*>(smem + kOffW);
  const uint32_t bars = sb + kOffBar;
  auto a_full = [&](int i) { return bars + 8u * (uint32_t)i; };
  auto a_empty = [&](int i) { return bars + 8u * (uint32_t)(kStages + i); };
  auto d_full = [&](int i) { return bars + 8u * (uint32_t)(2 * kStages + i); };
  auto d_empty = [&](int i) { return bars + 8u * (uint32_t)(2 * kStages + 2 + i); };
  const uint32_t done = bars + 8u * (uint32_t)(2 * kStages + 4);
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + kOffSlot);
  __shared__ int s_fail;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  ErrorWord* err = p.c.b.err;

  if (warp == kRoleMma) {
    tmem_alloc<kTmemCols>(slot);
    if (lane == 0) {
      for (int i = 0; i < kStages; ++i) { mbar_init(a_full(i), 32 * kConvWarps); mbar_init(a_empty(i), 1); }
      for (int i = 0; i < 2; ++i) { mbar_init(d_full(i), 1); mbar_init(d_empty(i), 32 * kEpiWarps); }
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
  int job = 0;        // accumulators filled
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
      int lo = 0, hi = (tokens + G - 1) / G - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (steps_before<G>(first, mid) <= local) lo = mid; else hi = mid - 1;
      }
      grp = lo;
    }
    const int nq = tokens - grp * G < G ? tokens - grp * G : G;
    const int64_t pos0 = first + (int64_t)grp * G;             // position of the group's first query
    const int x0 = p.c.row0[u] + grp * G;
    const int64_t s0 = local - steps_before<G>(first, grp);
    const int64_t s_all = (pos0 + nq - 1) / kStepTokens + 1;
    const int64_t s1 = s_all - s0 < end - at ? s_all : s0 + (end - at);
    at += s1 - s0;
    const int64_t row0 = p.c.b.unit_row(u);
    // columns of each tile: 8 per query, in multiples of 16
    auto tile_cols = [&](int t) {
      const int q = nq - t * kTileQueries;
      return q <= 0 ? 0 : (q >= kTileQueries ? 256 : (8 * q + 15) / 16 * 16);
    };

    // ---- B and the head weights (all threads; the previous run is complete).
    // Row r of a tile is head r & 7 of query r >> 3; rows past the group are 0.
    for (int i = tid; i < G * kIndexHeads * (kIndexDim / 8); i += kThreads) {
      const int c = i & 7, r = i >> 3;                         // chunk of 8 places, row over both tiles
      const int q = r >> 3;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = 0.f;
        if (q < nq) {
          const int64_t src = ((int64_t)x0 * kIndexHeads + r) * kIndexDim + dim_of(8 * c + e);
          v[e] = kBf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.q_idx)[src])
                       : reinterpret_cast<const float*>(p.q_idx)[src];
        }
      }
      const int tile = r >> 8, tr = r & 255;
      uint8_t* dst = smem + kOffB + tile * kBTile + tr * 128 + ((c ^ (tr & 7)) << 4);
#pragma unroll
      for (int pc = 0; pc < kPieces; ++pc) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
          o[e] = *reinterpret_cast<const uint32_t*>(&b);
          v[2 * e] -= __low2float(b);                          // exact
          v[2 * e + 1] -= __high2float(b);
        }
        *reinterpret_cast<uint4*>(dst + pc * kBTile) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    for (int i = tid; i < G * kIndexHeads; i += kThreads)
      sw[i] = i < nq * kIndexHeads ? p.w[(int64_t)x0 * kIndexHeads + i] : 0.f;
    fence_async_smem();
    __syncthreads();

    const int steps = (int)(s1 - s0);
    const int tiles = kQTiles == 2 && nq > kTileQueries ? 2 : 1;
    bool ok = true;
    if (warp >= kRoleConv && warp < kRoleMma) {
      // ---- converters: 16 codes per lane and load; lanes 4i .. 4i+3 hold one
      // token, a warp 32 blocks in four loads per phase, the next phase's
      // loads in flight.  A negative scale turns the code's sign.
      const int wc = warp - kRoleConv, sub = lane >> 2, part = lane & 3;
      const uint8_t* keys = p.c.b.index_keys + row0 * kIndexDim + part * 16;
      const uint16_t* scales = p.c.b.index_scales + row0;
      uint4 v[2][4];
      uint16_t sc[2][4];
      auto load = [&](int e, int i) {                          // phase i of the run
        const int64_t t0 = (s0 + (i >> 2)) * kStepTokens + 4 * (wc * 32 + sub) + (i & 3);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t t = t0 + 32 * j;
          const bool in = i < 4 * steps && t < n;
          v[e][j] = in ? __ldg(reinterpret_cast<const uint4*>(keys + t * kIndexDim)) : make_uint4(0, 0, 0, 0);
          sc[e][j] = in ? __ldg(scales + t) : (uint16_t)0;
        }
      };
      load(0, 0);
      load(1, 1);
#pragma unroll 1
      for (int i0 = 0; i0 < 4 * steps && ok; i0 += 2) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int ph = phase + i0 + e, st = ph % kStages;
          if (ok && ph >= kStages) ok = mbar_wait(a_empty(st), (uint32_t)(ph / kStages - 1) & 1u, err, kKernChunkScore);
          if (!ok) break;
          uint8_t* A = smem + st * kABytes;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = wc * 32 + j * 8 + sub;
            const uint32_t flip = (sc[e][j] & 0x8000u) ? 0x80808080u : 0u;
            const uint2 a = convert4(v[e][j].x ^ flip), b = convert4(v[e][j].y ^ flip);
            const uint2 c = convert4(v[e][j].z ^ flip), d = convert4(v[e][j].w ^ flip);
            *reinterpret_cast<uint4*>(A + r * 128 + (((2 * part) ^ (r & 7)) << 4)) = make_uint4(a.x, a.y, b.x, b.y);
            *reinterpret_cast<uint4*>(A + r * 128 + (((2 * part + 1) ^ (r & 7)) << 4)) =
                make_uint4(c.x, c.y, d.x, d.y);
          }
          load(e, i0 + e + 2);
          fence_async_smem();
          mbar_arrive(a_full(st));
        }
      }
    } else if (warp == kRoleMma) {
      if (lane == 0) {
        int jb = job;
#pragma unroll 1
        for (int s = 0; s < steps && ok; ++s) {
#pragma unroll 1
          for (int i = 0; i < 4 * tiles && ok; ++i, ++jb) {
            const int t = i >> 2, ph = phase + 4 * s + (i & 3), st = ph % kStages, buf = jb & 1;
            if (t == 0) ok = mbar_wait(a_full(st), (uint32_t)(ph / kStages) & 1u, err, kKernChunkScore);
            if (ok && jb >= 2) ok = mbar_wait(d_empty(buf), (uint32_t)(jb / 2 - 1) & 1u, err, kKernChunkScore);
            if (!ok) break;
            fence_after();
            const uint32_t d = tmem + 256u * (uint32_t)buf;
            const uint32_t idesc = idesc_bf16((uint32_t)tile_cols(t), false);
            const uint32_t a = sb + st * kABytes;
#pragma unroll
            for (int pc = 0; pc < kPieces; ++pc) {
              const uint32_t b = sb + kOffB + (t + pc) * kBTile;
#pragma unroll
              for (int ks = 0; ks < kIndexDim / 16; ++ks)
                mma_ss(d, desc_sw128(a + 32 * ks, 16), desc_sw128(b + 32 * ks, 16), idesc, (pc | ks) != 0);
            }
            commit(d_full(buf));
            if (t == tiles - 1) commit(a_empty(st));
          }
        }
      }
      __syncwarp();
    } else {
      // ---- epilogue: thread = block (tensor-memory lane); warps 0-3 take
      // queries 0-15 of a tile, warps 4-7 queries 16-31.  The loops over
      // phases and tiles stay rolled: unrolled, the warp roles' code no longer
      // fits the instruction cache (1573 us against 2048 x 131072 tokens).
      const int half = warp >> 2, row = (warp & 3) * 32 + lane;
      const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 128u * (uint32_t)half;
      const uint16_t* scales = p.c.b.index_scales + row0;
      uint16_t next[4];
      auto load_scales = [&](int64_t s) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t t = s * kStepTokens + 4 * row + k;
          next[k] = t < n ? __ldg(scales + t) : (uint16_t)0;
        }
      };
      load_scales(s0);
      int jb = job;
#pragma unroll 1
      for (int s = 0; s < steps && ok; ++s) {
        const int64_t b0 = (s0 + s) * (kStepTokens / 4);
        const int64_t t0 = 4 * (b0 + row);                     // the block's first token
        float mag[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) mag[k] = fabsf(__half2float(__ushort_as_half(next[k])));
        if (s + 1 < steps) load_scales(s0 + s + 1);
        // every token of the step within every query's context?
        const bool whole = (s0 + s + 1) * kStepTokens - 1 <= pos0;
#pragma unroll 1
        for (int t = 0; t < tiles && ok; ++t) {
          const int q0 = t * kTileQueries + 16 * half;         // this warp's first query
          const float4* wq = reinterpret_cast<const float4*>(sw + q0 * kIndexHeads);
          float best[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) best[i] = -INFINITY;
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            const int buf = jb & 1;
            ok = mbar_wait(d_full(buf), (uint32_t)(jb / 2) & 1u, err, kKernChunkScore);
            ++jb;
            if (!ok) break;
            fence_after();
            const float m = k < 2 ? (k == 0 ? mag[0] : mag[1]) : (k == 2 ? mag[2] : mag[3]);
            const uint32_t dcol = lane_base + 256u * (uint32_t)buf;
            // queries before `from` do not see this token
            const int64_t from = t0 + k - pos0 - q0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {                      // four queries: 32 columns
              if (q0 + 4 * c >= nq) break;
              uint32_t v[32];
              ld32(dcol + 32 * c, v);
              wait_ld();
              reg_fence(v);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 wa = wq[2 * (4 * c + i)], wb = wq[2 * (4 * c + i) + 1];
                const float wh[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
                float y = 0.f;
#pragma unroll
                for (int h = 0; h < 8; ++h) y = fmaf(wh[h], fmaxf(__uint_as_float(v[8 * i + h]), 0.f), y);
                y *= m;
                if (!whole && 4 * c + i < from) y = -INFINITY;
                best[4 * c + i] = fmaxf(best[4 * c + i], y);
              }
            }
            fence_before();
            mbar_arrive(d_empty(buf));
          }
          if (!ok) break;
          float* o = p.blk + (int64_t)(x0 + q0) * p.blk_stride + b0 + row;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (q0 + i < nq && t0 <= pos0 + q0 + i) o[i * p.blk_stride] = best[i];
        }
      }
    }
    phase += 4 * steps;
    job += 4 * steps * tiles;
    if (!ok) s_fail = 1;
    fence_before();
    __syncthreads();
    fence_after();
    if (s_fail) break;
  }

  if (warp == kRoleMma) {
    if (lane == 0) {
      commit(done);                 // every MMA issued above is complete once this arrives
      mbar_wait(done, 0, err, kKernChunkScore);
    }
    __syncwarp();
    tmem_free<kTmemCols>(tmem);
  }
}

template <bool kBf16>
cudaError_t launch(ChunkScoreParams& p, cudaStream_t s) {
  constexpr int G = Layout<kBf16>::kGroup, kSmemBytes = Layout<kBf16>::kSmemBytes;
  static PerDeviceOnce setup;
  cudaError_t e = setup.run([] { return prefer_max_shared(chunk_score_kernel<kBf16>, kSmemBytes); });
  int sms = 0;
  if (e == cudaSuccess) e = current_sm_count(&sms);
  if (e != cudaSuccess) return e;
  int64_t total = 0;
  for (int u = 0; u < p.c.b.n_units; ++u) {
    p.step0[u] = (int32_t)total;
    total += unit_steps<G>(p.c.b.u[u].n, p.c.unit_tokens(u));
    if (total > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  }
  p.step0[p.c.b.n_units] = (int32_t)total;
  const unsigned grid = (unsigned)(total < sms ? total : sms);
  return launch_kernel(chunk_score_kernel<kBf16>, dim3(grid), dim3(kThreads), kSmemBytes, s, 0, dim3(1), p);
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
  return q_bf16 ? launch<true>(p, s) : launch<false>(p, s);
}

}  // namespace qsa
