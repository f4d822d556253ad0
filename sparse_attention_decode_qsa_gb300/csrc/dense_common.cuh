// Shared by the attention over positions (dense_attn.cu) and the attention weights
// of tokens (window_weights.cu): which tokens a query sees, and fragments of few
// queries for the mma of m16n8k16.
#pragma once

#include "attn_common.cuh"

namespace qsa {
namespace attn {

constexpr int kFewQueries = 4;                    // times four heads of a KV head: the 16 rows of one mma

// Own tokens that any query at the positions p0 .. p1 sees: 0 .. na - 1 (sinks in
// front of the rest, seen by all of them) and from b0 on nb of them.
__host__ __device__ __forceinline__ void own_range(const DenseAttn& d, int64_t p0, int64_t p1, int64_t* na,
                                                   int64_t* b0, int64_t* nb) {
  int64_t low = p0 - d.window + 1;
  if (low < d.own_first) low = d.own_first;
  *na = d.sinks < low ? d.sinks : low;
  *b0 = low;
  *nb = p1 + 1 > low ? p1 + 1 - low : 0;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
template <bool kF16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Q as A fragments: rows query * 4 + head of KV head g, zeros past nq queries; f[i]:
// what a product of row lane / 4 + 8 i is to be multiplied with to be the logit
// times `factor`.  Against FP8 rows as f16, each row scaled by the power of two that
// puts its largest element into [2^14, 2^15) (f16 then holds a bf16 element exactly
// down to 2^-31 of the largest and to 2^-39 of it below), and with its dims in the
// order in which a K word's four codes become two fragments' registers.
template <bool kFp8>
__device__ __forceinline__ void few_queries(const uint16_t* q, int x0, int nq, int g, float factor, uint32_t (&qa)[8][4],
                                            float (&f)[2]) {
  const int lane = threadIdx.x & 31, r = lane >> 2, j4 = lane & 3;
#pragma unroll
  for (int hi = 0; hi < 2; ++hi) {
    const int row = r + 8 * hi, qi = row >> 2;
    const uint16_t* from = q + ((int64_t)(x0 + qi) * kQHeads + g * kGroup + (row & 3)) * kHeadDim;
    const bool have = qi < nq;
    float top = 0.f;
    f[hi] = factor;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t w0 = 0, w1 = 0;
      if (have) {
        if (kFp8) {
          const uint2 v = *reinterpret_cast<const uint2*>(from + 16 * k + 4 * j4);
          w0 = v.x;
          w1 = v.y;
        } else {
          w0 = *reinterpret_cast<const uint32_t*>(from + 16 * k + 2 * j4);
          w1 = *reinterpret_cast<const uint32_t*>(from + 16 * k + 2 * j4 + 8);
        }
      }
      qa[k][hi] = w0;
      qa[k][2 + hi] = w1;
      top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16_lo(w0)), fabsf(bf16_hi(w0))), fmaxf(fabsf(bf16_lo(w1)), fabsf(bf16_hi(w1)))));
    }
    if (kFp8) {
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      const RowScale sc = row_scale(top);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t& w = qa[k][2 * c + hi];
          w = pack_f16(bf16_lo(w) * sc.a * sc.b, bf16_hi(w) * sc.a * sc.b);
        }
      }
      f[hi] *= sc.inverse;
    }
  }
}

// The two B fragments of K-step k for 16 tokens' keys (16-byte chunks at chunk ^
// (row % 8)): {b0, b1} of tokens 0 .. 7, then of tokens 8 .. 15.
template <bool kFp8>
__device__ __forceinline__ void few_keys(uint32_t keys, int k, uint32_t (&kb)[4]) {
  const int lane = threadIdx.x & 31, r = lane >> 2, j4 = lane & 3;
  if (!kFp8) {
    const int tok = ((lane >> 4) << 3) + (lane & 7), c = 2 * k + ((lane >> 3) & 1);
    ldsm4(keys + tok * 256 + ((c ^ (tok & 7)) << 4), kb);
  } else {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      uint32_t w;
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(keys + (8 * n + r) * 128 + ((k ^ r) << 4) + 4 * j4));
      kb[2 * n] = codes2_f16(w & 0xFFFFu);
      kb[2 * n + 1] = codes2_f16(w >> 16);
    }
  }
}

}  // namespace attn
}  // namespace qsa
