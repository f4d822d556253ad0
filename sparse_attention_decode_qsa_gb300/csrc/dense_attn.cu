// Attention of every query of a chunk over tokens that its position alone
// decides, read through the slot table: a window of the newest tokens with the
// context's first ones (sinks), or a prefix that the whole batch shares followed
// by the request's own tokens.  For query row x at position p and head h (KV head
// g = h / 4)
//     logits_t = scale * q[x][h] . K_t[g],  t in V(p)
//     out[x][h] = sum_t softmax(logits)_t V_t[g],  lse = log sum_t exp(logits_t)
//     window:  V(p) = {t <= p : t < sinks or t > p - window}
//     shared:  V(p) = tokens 0 .. P-1 of the prefix's request, and the tokens
//              own_first .. p of the row's own
#include "attn_common.cuh"

namespace qsa {
namespace {

using namespace attn;

struct DenseParams {
  DenseAttn d;
  const uint16_t* q;             // [rows][16][128] bf16 bits
  float scale_log2;              // |softmax_scale| * log2(e)
  float sign;
  uint16_t* out;                 // [rows][16][128] bf16 bits
  float* lse;                    // [rows][16] or nullptr
};

// Own tokens that any query at the positions p0 .. p1 sees: 0 .. na - 1 (sinks in
// front of the rest, seen by all of them) and b0 .. b1 - 1.
__device__ __forceinline__ void own_range(const DenseAttn& d, int64_t p0, int64_t p1, int64_t* na, int64_t* b0,
                                          int64_t* b1) {
  int64_t low = p0 - d.window + 1;
  if (low < d.own_first) low = d.own_first;
  *na = d.sinks < low ? d.sinks : low;
  *b0 = low;
  *b1 = p1 + 1 > low ? p1 + 1 : low;
}

// The row of prefix token t for a row of unit u, nullptr (reported) for a bad slot.
__device__ __forceinline__ const uint8_t* prefix_row(const DenseAttn& d, int u, int64_t t) {
  const BatchDesc& b = d.c.b;
  const int layer = b.u[u].layer;
  const int32_t slot = b.slot_table[((int64_t)d.prefix_req * b.n_layers + layer) * b.ctx_cap + t];
  if (slot >= 0 && (int64_t)slot < b.pool_rows) return b.pool + (int64_t)slot * b.row_bytes;
  if (slot == -1 && d.prefix_host) return d.prefix_host + ((int64_t)layer * d.prefix_stride + t) * b.row_bytes;
  report_error(b.err, QSA_ERR_BAD_SLOT, kKernDenseAttn, t);
  return nullptr;
}

// One warp, one query row x of unit u and head h: online softmax over the row's
// own tokens, plain fp32.
__device__ __noinline__ void attend_row(const DenseParams& p, int u, int x, int h) {
  const int lane = threadIdx.x & 31, g = h / kGroup;
  const bool fp8 = p.d.c.b.row_bytes == kRowBytesFp8;
  const float f = p.sign * p.scale_log2;
  const uint2 qv = reinterpret_cast<const uint2*>(p.q + ((int64_t)x * kQHeads + h) * kHeadDim)[lane];
  const float q[4] = {bf16_lo(qv.x) * f, bf16_hi(qv.x) * f, bf16_lo(qv.y) * f, bf16_hi(qv.y) * f};
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const uint8_t* row) {
    if (!row) return;
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
  };
  for (int64_t t = 0; t < p.d.prefix_len; ++t) add(prefix_row(p.d, u, t));
  const int64_t pos = p.d.c.position(u, x);
  int64_t na, b0, b1;
  own_range(p.d, pos, pos, &na, &b0, &b1);
  for (int64_t t = 0; t < na; ++t) add(row_source(p.d.c.b, u, t, kKernDenseAttn));
  for (int64_t t = b0; t < b1; ++t) add(row_source(p.d.c.b, u, t, kKernDenseAttn));
  const float r = l == 0.f ? 0.f : 1.f / l;      // no tokens: zeros; NaN stays
  reinterpret_cast<uint2*>(p.out + ((int64_t)x * kQHeads + h) * kHeadDim)[lane] =
      make_uint2(pack_bf16(acc.x * r, acc.y * r), pack_bf16(acc.z * r, acc.w * r));
  if (p.lse && lane == 0) p.lse[(int64_t)x * kQHeads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

constexpr int kRowThreads = 256;
__global__ void __launch_bounds__(kRowThreads) dense_row_kernel(const __grid_constant__ DenseParams p) {
  const int64_t w = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int x = (int)(w / kQHeads);
  grid_dependency_wait();
  if (x >= p.d.c.rows()) return;
  attend_row(p, p.d.c.unit_of_row(x), x, (int)(w % kQHeads));
}

}  // namespace

int64_t dense_attn_workspace(const DenseAttn&) { return 256; }

cudaError_t launch_dense_attn(const DenseAttn& d, const uint16_t* q, float softmax_scale, uint16_t* out, float* lse,
                              void* workspace, cudaStream_t s) {
  (void)workspace;
  DenseParams p;
  p.d = d;
  p.q = q;
  p.scale_log2 = fabsf(softmax_scale) * kLog2e;
  p.sign = softmax_scale < 0.f ? -1.f : 1.f;
  p.out = out;
  p.lse = lse;
  const int64_t warps = (int64_t)d.c.rows() * kQHeads;
  return launch_kernel(dense_row_kernel, dim3((unsigned)((warps + 7) / 8)), dim3(kRowThreads), 0, s, 0, dim3(1), p);
}

}  // namespace qsa
