// Arithmetic shared by the attention kernels over chunks: conversions, copies to
// shared memory, pairs of fp32 values, KV rows in either format.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "tc_common.cuh"

namespace qsa {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 b = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A K scale as it goes to the logits, NaN if it is infinite: the codes' product with a
// query has one sign where its terms, each times the scale, have two.
__device__ __forceinline__ float key_scale_of(uint16_t bits) {
  const float s = __half2float(__ushort_as_half(bits));
  return fmaf(s, 0.f, s);
}

// log2 of a V scale's size.
__device__ __forceinline__ float log2_size(float s) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fabsf(s)));
  return fmaxf(y, -100.f);
}

// The power of two that puts a largest size `top` into [2^14, 2^15), as two factors
// (it may be past fp32's range as one), and its inverse; 1 for 0 and values that are
// not finite.
struct RowScale {
  float a, b, inverse;
};
__device__ __forceinline__ RowScale row_scale(float top) {
  int k = 0;
  if (top > 0.f && top < INFINITY) {
    const bool tiny = top < 0x1p-100f;               // (subnormals have no exponent to read)
    const int e = (int)(__float_as_uint(tiny ? top * 0x1p60f : top) >> 23) - 127 - (tiny ? 60 : 0);
    k = 14 - e;                                      // -113 .. 163
  }
  const int h = k >> 1;
  return {__int_as_float((127 + h) << 23), __int_as_float((127 + k - h) << 23),
          __int_as_float((127 - h) << 23) * __int_as_float((127 - k + h) << 23)};
}

// Pairs of fp32 values: one instruction for two multiply-adds or additions.
__device__ __forceinline__ uint64_t pair(uint32_t a, uint32_t b) { return (uint64_t)a | ((uint64_t)b << 32); }
__device__ __forceinline__ uint64_t pair(float a, float b) { return pair(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ float lo_of(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float hi_of(uint64_t x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Four and eight e4m3 codes as f16, exactly.
__device__ __forceinline__ uint2 codes4_f16(uint32_t w) {
  uint2 h;
  asm("{\n .reg .b16 x, y;\n mov.b32 {x, y}, %2;\n cvt.rn.f16x2.e4m3x2 %0, x;\n cvt.rn.f16x2.e4m3x2 %1, y;\n}\n"
      : "=r"(h.x), "=r"(h.y)
      : "r"(w));
  return h;
}
__device__ __forceinline__ uint4 codes8_f16(uint2 w) {
  const uint2 a = codes4_f16(w.x), b = codes4_f16(w.y);
  return make_uint4(a.x, a.y, b.x, b.y);
}

}  // namespace attn
}  // namespace qsa
