// Producer side for several tokens at once: store every token of a chunk as
// append_token.cu stores one (66-byte index key and KV row: "Оффлоадинг
// KV-кэша Qwen3.8-Flash-Next в RAM через vLLM без потери скорости
// декодирования", section "Эффективность и память"; placement and slots:
// "双卡RTX4090跑通Qwen3-Next：8并发满血长上下文实测", section
// "显存账本：热缓存卸载省下约84%").
//
// One warp per token, no shared memory and no barrier.  Lane l holds key
// elements 2l, 2l+1 and the row's 16-byte pieces l, l+32, l+64, l+96; an FP8
// row's head vector is 16 pieces, so its absmax is a reduction over half a
// warp.  The kernel moves 2304 bytes in and 2118 (BF16) or 1110 (FP8) bytes
// out per token: 4 x 8191 tokens as FP8 rows (112 MB) take 25 us, 0.67 of the
// measured copy rate (33 with a division per element; the grid's shape and the
// occupancy change nothing); 14 BF16 tokens 3.9 us, a launch's latency.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "qsa_internal.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPieces = kRowBytes / 16 / 32;     // 16-byte pieces of a BF16 row per lane
static_assert(kIndexDim == 64 && kPieces == 4, "two key elements and four row pieces per lane");

struct ChunkAppendParams {
  ChunkDesc c;
  ChunkTargets tg;
  const float* k_new;       // [rows][64]
  const uint8_t* kv_new;    // [rows][2048]
};

// fp16 scale of absmax a (round to nearest even of a / 448, saturating).
__device__ __forceinline__ __half scale_of(float a) { return __float2half_rn(fminf(a / 448.0f, 65504.0f)); }

__device__ __forceinline__ float reciprocal(float f) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(f));
  return r;
}

// e4m3 code of x under scale f > 0.
__device__ __forceinline__ uint32_t code_of(float x, float f) {
  return (uint32_t)(uint8_t)__nv_cvt_float_to_fp8(fminf(fmaxf(x / f, -448.0f), 448.0f), __NV_SATFINITE, __NV_E4M3);
}

// The codes of eight bf16 elements under an fp16 scale f > 0, as their correctly
// rounded quotients x / f would give them.  With r = 1 / f to an ulp or two, q =
// x r and one correction q - r (q f - x), whose remainder is exact, the quotient
// is off by 2^-22 at most, and by nothing where it is a midpoint m of two codes:
// then q f - x = m f d for a d of at most 2^-21, and the correction leaves m (1 -
// d 2^-22), which rounds to m.  Every other quotient is far enough from the
// midpoints: x has 8 bits and m f 16, so x / f differs from m by 2^-16 of it at
// least.  x may be NaN (code of -448, as clamping gives), not infinite.
__device__ __forceinline__ uint2 codes_of(const float (&x)[8], float f, float r) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 q;
    q.x = x[2 * i] * r;
    q.y = x[2 * i + 1] * r;
    q.x = fmaf(-fmaf(q.x, f, -x[2 * i]), r, q.x);    // (these signs keep a zero's own)
    q.y = fmaf(-fmaf(q.y, f, -x[2 * i + 1]), r, q.y);
    q.x = fmaxf(q.x, -448.0f);                       // the conversion takes the upper end
    q.y = fmaxf(q.y, -448.0f);
    c[i] = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

__global__ void __launch_bounds__(kThreads) append_chunk_kernel(const __grid_constant__ ChunkAppendParams p) {
  const int lane = threadIdx.x & 31;
  const int x = blockIdx.x * kWarps + (threadIdx.x >> 5);
  grid_dependency_wait();
  if (x >= p.c.rows()) return;
  const int u = p.c.unit_of_row(x);
  const int64_t n = p.c.b.u[u].n, t = p.c.position(u, x), first = n - p.c.unit_tokens(u);
  const int64_t row = p.c.b.unit_row(u) + t;

  const float2 k = reinterpret_cast<const float2*>(p.k_new + (int64_t)x * kIndexDim)[lane];
  const uint4* src = reinterpret_cast<const uint4*>(p.kv_new + (int64_t)x * kRowBytes);
  uint4 v[kPieces];
#pragma unroll
  for (int j = 0; j < kPieces; ++j) v[j] = src[lane + 32 * j];

  // ---- index key
  float a = fmaxf(fabsf(k.x), fabsf(k.y));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
  const __half s16 = scale_of(a);
  const float sf = __half2float(s16);
  const uint32_t codes = sf > 0.f ? code_of(k.x, sf) | (code_of(k.y, sf) << 8) : 0u;
  reinterpret_cast<uint16_t*>(const_cast<uint8_t*>(p.c.b.index_keys) + row * kIndexDim)[lane] = (uint16_t)codes;
  if (lane == 0)
    const_cast<uint16_t*>(p.c.b.index_scales)[row] = sf > 0.f ? __half_as_ushort(s16) : (uint16_t)0;

  // ---- where the row goes, and the slots
  const int ring = p.tg.ring[u];
  int64_t pool_row = -1;
  if (p.tg.row_base[u] >= 0) {
    if (ring == 0) pool_row = p.tg.row_base[u] + t;
    else if (t >= n - ring) pool_row = p.tg.row_base[u] + t % ring;   // among the newest `ring` tokens
  }
  if (pool_row >= p.c.b.pool_rows) {
    if (lane == 0) report_error(p.c.b.err, QSA_ERR_BAD_SLOT, kKernChunkAppend, pool_row);
    pool_row = -1;
  }
  if (lane == 0) {
    int32_t* slots = p.c.b.slot_table + p.c.b.unit_row(u);
    slots[t] = (int32_t)pool_row;
    // the token that held t's ring row before the chunk (one of the chunk's
    // own tokens writes its slot itself)
    if (ring > 0 && t >= ring && t - ring < first) slots[t - ring] = -1;
  }

  // ---- KV row
  const int32_t rb = p.c.b.row_bytes;
  uint8_t* dst[2] = {pool_row >= 0 ? p.c.b.pool + pool_row * rb : nullptr,
                     p.c.b.u[u].host_rows ? const_cast<uint8_t*>(p.c.b.u[u].host_rows) + t * rb : nullptr};
  if (rb == kRowBytes) {
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      if (!dst[d]) continue;
#pragma unroll
      for (int j = 0; j < kPieces; ++j) reinterpret_cast<uint4*>(dst[d])[lane + 32 * j] = v[j];
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    // piece lane + 32 j: values 8 (lane % 16) .. +7 of head vector 2 j + lane / 16
    // (K heads 0-3, then V heads 0-3)
    const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
    float e[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e[2 * i] = __uint_as_float(w[i] << 16);
      e[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    float va = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) va = fmaxf(va, fabsf(e[i]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) va = fmaxf(va, __shfl_xor_sync(0xFFFFFFFFu, va, o));
    const __half vs = scale_of(va);
    const float vf = __half2float(vs);
    uint2 c8 = make_uint2(0u, 0u);
    if (vf > 0.f && va < INFINITY) {
      c8 = codes_of(e, vf, reciprocal(vf));
    } else if (vf > 0.f) {
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) x = i == k ? e[k] : x;
        const uint32_t c = code_of(x, vf) << (8 * (i & 3));
        if (i < 4) c8.x |= c;
        else c8.y |= c;
      }
    }
    const int hv = 2 * j + (lane >> 4);
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      if (!dst[d]) continue;
      *reinterpret_cast<uint2*>(dst[d] + hv * kHeadDim + (lane & 15) * 8) = c8;
      if ((lane & 15) == 0)
        reinterpret_cast<uint16_t*>(dst[d] + 2 * kKvHeads * kHeadDim)[hv] =
            vf > 0.f ? __half_as_ushort(vs) : (uint16_t)0;
    }
  }
}

}  // namespace

cudaError_t launch_append_chunk(const ChunkDesc& c, const ChunkTargets& tg, const float* k_new,
                                const uint8_t* kv_new, cudaStream_t s) {
  ChunkAppendParams p;
  p.c = c;
  p.tg = tg;
  p.k_new = k_new;
  p.kv_new = kv_new;
  return launch_kernel(append_chunk_kernel, dim3((c.rows() + kWarps - 1) / kWarps), dim3(kThreads), 0, s, 0,
                       dim3(1), p);
}

}  // namespace qsa
