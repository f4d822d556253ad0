// Shared by the attention over positions (dense_attn.cu) and the attention weights
// of tokens (window_weights.cu): which tokens a query sees, and fragments of few
// queries for the mma of m16n8k16.
#pragma once

#include "attn_common.cuh"

namespace qsa {
namespace attn {

constexpr int kFewQueries = 4;                    // times four heads of a KV head: two column tiles of an mma

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

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Tokens are the rows of these mma, queries their columns: column query * 4 + head
// of KV head g, kN tiles of eight (two queries each).  A column's statistics then
// lie in the four lanes that hold it in every accumulator.

// Q as B fragments, zeros past nq queries; f[n][e]: what a product of column 8 n + 2
// (lane % 4) + e is to be multiplied with to be the logit times `factor`.  Against
// FP8 rows as f16, each column scaled by the power of two that puts its largest
// element into [2^14, 2^15) (f16 then holds a bf16 element exactly down to 2^-31 of
// the largest and to 2^-39 of it below), and with its dims in the order in which a K
// word's four codes become two registers of a fragment.
template <bool kFp8, int kN>
__device__ __forceinline__ void few_queries(const uint16_t* q, int x0, int nq, int g, float factor,
                                            uint32_t (&qb)[kN][8][2], float (&f)[kN][2]) {
  const int lane = threadIdx.x & 31, r = lane >> 2, j4 = lane & 3;
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    const int qi = 2 * n + (r >> 2);
    const uint16_t* from = q + ((int64_t)(x0 + qi) * kQHeads + g * kGroup + (r & 3)) * kHeadDim;
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint2 v = make_uint2(0, 0);
      if (qi < nq) {
        if (kFp8)
          v = *reinterpret_cast<const uint2*>(from + 16 * k + 4 * j4);
        else
          v = make_uint2(*reinterpret_cast<const uint32_t*>(from + 16 * k + 2 * j4),
                         *reinterpret_cast<const uint32_t*>(from + 16 * k + 2 * j4 + 8));
      }
      qb[n][k][0] = v.x;
      qb[n][k][1] = v.y;
      top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16_lo(v.x)), fabsf(bf16_hi(v.x))), fmaxf(fabsf(bf16_lo(v.y)), fabsf(bf16_hi(v.y)))));
    }
    f[n][0] = f[n][1] = factor;
    if (kFp8) {
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      const RowScale sc = row_scale(top);
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          qb[n][k][c] = pack_f16(bf16_lo(qb[n][k][c]) * sc.a * sc.b, bf16_hi(qb[n][k][c]) * sc.a * sc.b);
#pragma unroll
      for (int e = 0; e < 2; ++e) f[n][e] *= __shfl_sync(0xFFFFFFFFu, sc.inverse, 4 * (2 * j4 + e));
    }
  }
}

// The A fragment of K-step k of 16 tokens' keys (16-byte chunks at chunk ^ (row % 8)).
template <bool kFp8>
__device__ __forceinline__ void few_keys(uint32_t keys, int k, uint32_t (&ka)[4]) {
  const int lane = threadIdx.x & 31, r = lane >> 2, j4 = lane & 3;
  if (!kFp8) {
    const int tok = lane & 15, c = 2 * k + (lane >> 4);
    ldsm4(keys + tok * 256 + ((c ^ (tok & 7)) << 4), ka);
  } else {
#pragma unroll
    for (int n = 0; n < 2; ++n) {                    // tokens r, r + 8
      uint32_t w;
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(keys + (8 * n + r) * 128 + ((k ^ r) << 4) + 4 * j4));
      const uint2 h = codes4_f16(w);
      ka[n] = h.x;
      ka[2 + n] = h.y;
    }
  }
}

// Calls copy(i, address of token i's row) for 16 tokens i; lane l < 16 holds token l's
// row (or nullptr) and its slot.  Rows in the pool need 32 bits of theirs passed on.
template <int kPer, class Copy>
__device__ __forceinline__ void few_copies(const BatchDesc& b, const uint8_t* row, int32_t slot, Copy&& copy) {
  const int lane = threadIdx.x & 31, mine = lane / (32 / kPer);      // kPer tokens a turn
  if (__all_sync(0xFFFFFFFFu, row == nullptr || slot >= 0)) {
    const uint32_t at = row ? (uint32_t)slot : 0u;
#pragma unroll
    for (int i = 0; i < 16; i += kPer) {
      const uint32_t s = __shfl_sync(0xFFFFFFFFu, at, i + mine);
      copy(i + mine, b.pool + (uint64_t)s * (uint32_t)b.row_bytes);
    }
  } else {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row ? row : b.pool);
#pragma unroll
    for (int i = 0; i < 16; i += kPer)
      copy(i + mine, reinterpret_cast<const uint8_t*>(__shfl_sync(0xFFFFFFFFu, at, i + mine)));
  }
}

}  // namespace attn
}  // namespace qsa
