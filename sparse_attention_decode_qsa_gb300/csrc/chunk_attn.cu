// Attention of every query of a chunk over its own selected blocks: for query
// row x at position p and query head h (KV head g = h / 4)
//     logits_t = scale * q[x][h] . K_t[g],  t in the selected blocks, t <= p
//     out[x][h] = sum_t softmax(logits)_t V_t[g],  lse = log sum_t exp(logits_t)
// with the rows read through the slot table, as sparse_attn.cu does for one
// query per request.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "qsa_internal.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct ChunkAttnParams {
  ChunkDesc c;
  const uint16_t* q;        // [rows][16][128] bf16 bits
  const int32_t* sel;       // [rows][k_max]
  const int32_t* n_sel;     // [rows]
  int32_t k_max;
  float scale_log2;         // softmax_scale * log2(e)
  uint16_t* out;            // [rows][16][128] bf16 bits
  float* lse;               // [rows][16] or nullptr
};

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

// Four values at dims 4 lane .. 4 lane + 3 of head vector hv (K heads 0-3,
// then V heads 0-3) of a row.
__device__ __forceinline__ float4 row_values(const uint8_t* row, int hv, int lane, bool fp8) {
  if (!fp8) {
    const uint2 v = reinterpret_cast<const uint2*>(row + hv * kHeadDim * 2)[lane];
    return make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
  }
  const uint32_t c = reinterpret_cast<const uint32_t*>(row + hv * kHeadDim)[lane];
  const float s = __half2float(
      __ushort_as_half(reinterpret_cast<const uint16_t*>(row + 2 * kKvHeads * kHeadDim)[hv]));
  const __half2 a(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xFFFFu), __NV_E4M3));
  const __half2 b(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> 16), __NV_E4M3));
  return make_float4(s * __low2float(a), s * __high2float(a), s * __low2float(b), s * __high2float(b));
}

// One warp, one query row x and head h: online softmax over the row's own
// selected tokens, in fp32.
__device__ void attend_row(const ChunkAttnParams& p, int u, int x, int h) {
  const int lane = threadIdx.x & 31, g = h / kGroup;
  const bool fp8 = p.c.b.row_bytes == kRowBytesFp8;
  const int64_t pos = p.c.position(u, x);
  const uint2 qv = reinterpret_cast<const uint2*>(p.q + ((int64_t)x * kQHeads + h) * kHeadDim)[lane];
  const float q[4] = {bf16_lo(qv.x) * p.scale_log2, bf16_hi(qv.x) * p.scale_log2, bf16_lo(qv.y) * p.scale_log2,
                      bf16_hi(qv.y) * p.scale_log2};
  int nsel = p.n_sel[x];
  if (nsel < 0 || nsel > p.k_max) {
    if (lane == 0 && h == 0) report_error(p.c.b.err, QSA_ERR_BAD_BLOCK, kKernChunkAttn, nsel);
    nsel = 0;
  }
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = 0; j < nsel; ++j) {
    const int64_t b = p.sel[(int64_t)x * p.k_max + j];
    if (b < 0 || 4 * b > pos) {
      if (lane == 0 && h == 0) report_error(p.c.b.err, QSA_ERR_BAD_BLOCK, kKernChunkAttn, b);
      continue;
    }
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
  __nv_bfloat162 o[2] = {__floats2bfloat162_rn(acc.x * r, acc.y * r), __floats2bfloat162_rn(acc.z * r, acc.w * r)};
  reinterpret_cast<uint2*>(p.out + ((int64_t)x * kQHeads + h) * kHeadDim)[lane] = *reinterpret_cast<uint2*>(o);
  if (p.lse && lane == 0) p.lse[(int64_t)x * kQHeads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

__global__ void __launch_bounds__(kThreads) chunk_attn_kernel(const __grid_constant__ ChunkAttnParams p) {
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  grid_dependency_wait();
  const int x = (int)(w / kQHeads);
  if (x >= p.c.rows()) return;
  attend_row(p, p.c.unit_of_row(x), x, (int)(w % kQHeads));
}

}  // namespace

int64_t chunk_attn_workspace(const ChunkDesc&, int32_t) { return 256; }

cudaError_t launch_chunk_attn(const ChunkDesc& c, const uint16_t* q, const int32_t* sel_blocks,
                              const int32_t* n_sel, int32_t budget_tokens, float softmax_scale,
                              uint16_t* out, float* lse, void*, cudaStream_t s) {
  ChunkAttnParams p;
  p.c = c;
  p.q = q;
  p.sel = sel_blocks;
  p.n_sel = n_sel;
  p.k_max = budget_tokens / 4;
  p.scale_log2 = softmax_scale * kLog2e;
  p.out = out;
  p.lse = lse;
  const int64_t warps = (int64_t)c.rows() * kQHeads;
  return launch_kernel(chunk_attn_kernel, dim3((unsigned)((warps + kWarps - 1) / kWarps)), dim3(kThreads), 0, s, 0,
                       dim3(1), p);
}

}  // namespace qsa
