// Index scores for every query of a chunk: as index_score.cu scores one
// query, each query against the tokens up to its own position
//     S_it = sum_h w_ih * relu(scale_t * sum_d q_i[h][d] * e4m3(code_t[d])),  t <= p_i
// reduced to C4 blocks (max over 4 adjacent tokens).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "qsa_internal.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 128;

struct ChunkScoreParams {
  ChunkDesc c;
  const void* q_idx;    // [rows][8][64] fp32 or bf16
  const float* w;       // [rows][8]
  float* blk;           // [rows][blk_stride]
  int64_t blk_stride;
};

// One CTA per (row, 128 blocks); thread = block.
template <bool kBf16>
__global__ void __launch_bounds__(kThreads) chunk_score_kernel(const __grid_constant__ ChunkScoreParams p) {
  __shared__ float q[kIndexHeads * kIndexDim];
  __shared__ float w[kIndexHeads];
  const int x = blockIdx.x, tid = threadIdx.x;
  grid_dependency_wait();
  const int u = p.c.unit_of_row(x);
  const int64_t pos = p.c.position(u, x);
  const int64_t nb = pos / 4 + 1;
  if ((int64_t)blockIdx.y * kThreads >= nb) return;
  for (int i = tid; i < kIndexHeads * kIndexDim; i += kThreads) {
    const int64_t at = (int64_t)x * kIndexHeads * kIndexDim + i;
    q[i] = kBf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.q_idx)[at])
                 : reinterpret_cast<const float*>(p.q_idx)[at];
  }
  if (tid < kIndexHeads) w[tid] = p.w[(int64_t)x * kIndexHeads + tid];
  __syncthreads();
  const int64_t b = (int64_t)blockIdx.y * kThreads + tid;
  if (b >= nb) return;
  float best = -INFINITY;
  for (int i = 0; i < 4 && 4 * b + i <= pos; ++i) {
    const int64_t row = p.c.b.unit_row(u) + 4 * b + i;
    const float sc = __half2float(__ushort_as_half(p.c.b.index_scales[row]));
    const uint8_t* codes = p.c.b.index_keys + row * kIndexDim;
    float y[kIndexHeads] = {};
    for (int d = 0; d < kIndexDim; ++d) {
      const float k = __half2float(__half(__nv_cvt_fp8_to_halfraw(codes[d], __NV_E4M3)));
#pragma unroll
      for (int h = 0; h < kIndexHeads; ++h) y[h] = fmaf(q[h * kIndexDim + d], k, y[h]);
    }
    float s = 0.f;
#pragma unroll
    for (int h = 0; h < kIndexHeads; ++h) s = fmaf(w[h], fmaxf(y[h] * sc, 0.f), s);
    best = fmaxf(best, s);
  }
  p.blk[(int64_t)x * p.blk_stride + b] = best;
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
  int64_t n = 0;
  for (int u = 0; u < c.b.n_units; ++u)
    if (c.unit_tokens(u) > 0 && c.b.u[u].n > n) n = c.b.u[u].n;
  const int64_t nb = (n + 3) / 4;
  if (nb > 65535ll * kThreads) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)c.rows(), (unsigned)((nb + kThreads - 1) / kThreads));
  return launch_kernel(q_bf16 ? chunk_score_kernel<true> : chunk_score_kernel<false>, grid, dim3(kThreads), 0, s, 0,
                       dim3(1), p);
}

}  // namespace qsa
