// The weight that attention gives each cached token: for token t of a unit
//     weights[t] (+)= sum_x sum_h exp(scale * q[x][h] . K_t[h / 4] - lse[x][h])
// over the chunk's queries x that see t (the window and sinks of dense_attn.cu)
// and all heads h, with the log-sum-exp that the attention returned.  A row
// without tokens (lse = -inf) adds nothing.
#include "attn_common.cuh"

namespace qsa {
namespace {

using namespace attn;

struct WeightParams {
  DenseAttn d;
  const uint16_t* q;             // [rows][16][128] bf16 bits
  const float* lse;              // [rows][16]
  float scale_log2;              // softmax_scale * log2(e)
  float* weights;                // [units][stride]
  int64_t stride;
  int32_t accumulate;
};

constexpr int kThreads = 256;
__global__ void __launch_bounds__(kThreads) weight_token_kernel(const __grid_constant__ WeightParams p) {
  const int u = blockIdx.y, lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  grid_dependency_wait();
  const ChunkDesc& c = p.d.c;
  if (t >= c.b.u[u].n) return;
  const bool fp8 = c.b.row_bytes == kRowBytesFp8;
  float sum = 0.f;
  const uint8_t* row = c.unit_tokens(u) > 0 ? row_source(c.b, u, t, kKernWeights) : nullptr;
  if (row) {
    for (int g = 0; g < kKvHeads; ++g) {
      const float4 k = row_values(row, g, lane, fp8);
      for (int x = c.row0[u]; x < c.row0[u + 1]; ++x) {
        const int64_t pos = c.position(u, x);
        if (t > pos || (t >= p.d.sinks && t <= pos - p.d.window)) continue;
        for (int h = g * kGroup; h < (g + 1) * kGroup; ++h) {
          const uint2 w = reinterpret_cast<const uint2*>(p.q + ((int64_t)x * kQHeads + h) * kHeadDim)[lane];
          float s = fmaf(bf16_hi(w.y), k.w, fmaf(bf16_lo(w.y), k.z, fmaf(bf16_hi(w.x), k.y, bf16_lo(w.x) * k.x)));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
          const float lse = p.lse[(int64_t)x * kQHeads + h];
          if (lse != -INFINITY) sum += exp2f(fmaf(s, p.scale_log2, -lse * kLog2e));
        }
      }
    }
  }
  if (lane == 0) {
    float* w = p.weights + u * p.stride + t;
    *w = p.accumulate ? *w + sum : sum;
  }
}

}  // namespace

cudaError_t launch_window_weights(const DenseAttn& d, const uint16_t* q, const float* lse, float softmax_scale,
                                  float* weights, int64_t stride, bool accumulate, cudaStream_t s) {
  WeightParams p;
  p.d = d;
  p.q = q;
  p.lse = lse;
  p.scale_log2 = softmax_scale * kLog2e;
  p.weights = weights;
  p.stride = stride;
  p.accumulate = accumulate;
  int64_t most = 0;
  for (int u = 0; u < d.c.b.n_units; ++u) most = d.c.b.u[u].n > most ? d.c.b.u[u].n : most;
  return launch_kernel(weight_token_kernel, dim3((unsigned)((most + 7) / 8), d.c.b.n_units), dim3(kThreads), 0, s, 0,
                       dim3(1), p);
}

}  // namespace qsa
