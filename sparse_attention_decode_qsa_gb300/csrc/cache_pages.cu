// Pages of the cache: copying a request's tokens into another request's
// storage (fork), and sliding the live regions of the pool to its front
// (compaction).  The pages ask for both sides of it: logical tokens are kept
// apart from physical slots, and capacity comes back when requests end
// ("双卡RTX4090跑通Qwen3-Next：8并发满血长上下文实测", section
// "显存账本：热缓存卸载省下约84%"), which leaves gaps that only moving rows
// closes.  All three kernels are bound by the bytes they move.
#include "qsa_internal.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// ------------------------------------------------------------------- fork
// One warp per (layer, token): the source row is found through the parent's
// slot table (pool row, or the host history for a cold token) and stored in
// the child's region and / or host history; the token's key, scale and slot go
// with it.  32001 x 12 BF16 rows (1.62 GB in and out) take 227 us, a little above the
// measured copy rate; 1021 x 12 FP8 rows 8 us.
__global__ void __launch_bounds__(kThreads) fork_kernel(const ForkParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  grid_dependency_wait();
  if (w >= p.n_tokens * p.n_layers) return;
  const int64_t l = w / p.n_tokens, t = w % p.n_tokens;
  const int64_t s = ((int64_t)p.src_req * p.n_layers + l) * p.ctx_cap + t;
  const int64_t d = ((int64_t)p.dst_req * p.n_layers + l) * p.ctx_cap + t;
  const int32_t slot = p.slot_table[s];
  const uint8_t* src = nullptr;
  if (slot >= 0 && (int64_t)slot < p.pool_rows) src = p.pool + (int64_t)slot * p.row_bytes;
  else if (slot == -1 && p.src_host) src = p.src_host + (l * p.src_stride + t) * p.row_bytes;
  else if (lane == 0) report_error(p.err, QSA_ERR_BAD_SLOT, kKernFork, t);
  int64_t row = -1;                          // the child's pool row
  if (p.dst_layer_rows > 0 && (!p.dst_ring || t >= p.n_tokens - p.dst_layer_rows))
    row = p.dst_base + l * p.dst_layer_rows + (p.dst_ring ? t % p.dst_layer_rows : t);
  const int chunks = p.row_bytes / 16;       // 128 (BF16) or 65 (FP8)
  uint4 v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (src && lane + 32 * j < chunks) v[j] = reinterpret_cast<const uint4*>(src)[lane + 32 * j];
  if (lane < kIndexDim / 16)
    reinterpret_cast<uint4*>(p.index_keys + d * kIndexDim)[lane] =
        reinterpret_cast<const uint4*>(p.index_keys + s * kIndexDim)[lane];
  if (lane == kIndexDim / 16) p.index_scales[d] = p.index_scales[s];
  if (lane == kIndexDim / 16 + 1) p.slot_table[d] = (int32_t)row;
  if (!src) return;
  uint8_t* pool_dst = row >= 0 ? p.pool + row * p.row_bytes : nullptr;
  uint8_t* host_dst = p.dst_host ? p.dst_host + (l * p.dst_stride + t) * p.row_bytes : nullptr;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (lane + 32 * j >= chunks) continue;
    if (pool_dst) reinterpret_cast<uint4*>(pool_dst)[lane + 32 * j] = v[j];
    if (host_dst) reinterpret_cast<uint4*>(host_dst)[lane + 32 * j] = v[j];
  }
}

// -------------------------------------------------------------- compaction
// Rows [from, from + rows) go down by D = from - to rows; source and
// destination overlap when D < rows.  The move falls apart into independent
// chains: the 16-byte pieces at i, i + S, i + 2S, ... of the source (S = D
// rows in pieces) each overwrite the piece before them in the same chain and
// nothing else.  A thread owns whole chains, so no two threads ever touch the
// same address and no barrier is needed: it loads the next pieces of its
// chains, then stores them where the pieces before them were.  Eight loads are
// in flight per thread: of one chain where the region is long against the gap
// (few chains, long ones), of eight chains side by side where it is not.
constexpr int kDepth = 8;

template <bool kLong>
__global__ void __launch_bounds__(kThreads) move_rows_kernel(uint4* pool, int64_t from, int64_t to, int64_t count) {
  grid_dependency_wait();
  const int64_t S = from - to, chains = S < count ? S : count;
  constexpr int64_t kBlock = (int64_t)kThreads * (kLong ? 1 : kDepth);      // chains of a CTA at a time
  for (int64_t c0 = (int64_t)blockIdx.x * kBlock; c0 < chains; c0 += (int64_t)gridDim.x * kBlock) {
    const int64_t i = c0 + threadIdx.x;
    if (kLong) {
      if (i >= chains) continue;
      for (int64_t k = i; k < count; k += S * kDepth) {
        uint4 v[kDepth];
#pragma unroll
        for (int j = 0; j < kDepth; ++j)
          if (k + j * S < count) v[j] = pool[from + k + j * S];
#pragma unroll
        for (int j = 0; j < kDepth; ++j)
          if (k + j * S < count) pool[to + k + j * S] = v[j];
      }
    } else {
      for (int64_t k = 0; k < count - c0; k += S) {
        uint4 v[kDepth];
#pragma unroll
        for (int j = 0; j < kDepth; ++j) {
          const int64_t c = i + j * kThreads;
          if (c < chains && c + k < count) v[j] = pool[from + c + k];
        }
#pragma unroll
        for (int j = 0; j < kDepth; ++j) {
          const int64_t c = i + j * kThreads;
          if (c < chains && c + k < count) pool[to + c + k] = v[j];
        }
      }
    }
  }
}

__device__ __forceinline__ int32_t remap(const RemapParams& p, int32_t v) {
  if (v < 0) return v;
  // last move whose first row is <= v
  int lo = 0, hi = p.n_moves - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.moves[mid].from <= v) lo = mid; else hi = mid - 1;
  }
  const RowMove m = p.moves[lo];
  return v >= m.from && v < m.from + m.rows ? (int32_t)(v - m.down) : v;
}

// `parts` CTAs per (request, layer).
__global__ void __launch_bounds__(kThreads) remap_kernel(const __grid_constant__ RemapParams p, int parts) {
  grid_dependency_wait();
  const int unit = blockIdx.x / parts, part = blockIdx.x % parts;
  const int r = unit / p.n_layers, l = unit % p.n_layers;
  const int64_t st = (int64_t)p.req[r] * p.n_layers + l;
  int32_t* slots = p.slot_table + st * p.ctx_cap;
  for (int64_t t = (int64_t)part * kThreads + threadIdx.x; t < p.ctx[r]; t += (int64_t)parts * kThreads) {
    const int32_t v = slots[t], w = remap(p, v);
    if (w != v) slots[t] = w;
  }
  if (part == 0) {
    int32_t* pend = p.hot_pend + st * p.pend_stride;
    for (int i = threadIdx.x; i < p.pend_stride; i += kThreads) pend[i] = remap(p, pend[i]);
  }
}

}  // namespace

cudaError_t launch_fork(const ForkParams& p, cudaStream_t s) {
  const int64_t rows = p.n_tokens * p.n_layers;
  return launch_kernel(fork_kernel, dim3((unsigned)((rows + kWarps - 1) / kWarps)), dim3(kThreads), 0, s, 0,
                       dim3(1), p);
}

cudaError_t launch_move_rows(uint8_t* pool, int64_t row_bytes, int64_t from, int64_t to, int64_t rows,
                             cudaStream_t s) {
  const int64_t per = row_bytes / 16;
  const int64_t chains = (from - to < rows ? from - to : rows) * per;
  int sms = 0;
  if (const cudaError_t e = current_sm_count(&sms)) return e;
  // chains side by side once they fill the device eight deep (eight CTAs per SM):
  // 3 x 196608 BF16 rows, each down by as many, 581 -> 379 us
  const bool wide = chains >= (int64_t)sms * 8 * kThreads * kDepth;
  const int64_t block = wide ? (int64_t)kThreads * kDepth : kThreads;
  int64_t blocks = (chains + block - 1) / block;
  if (blocks > sms * 8) blocks = sms * 8;
  return launch_kernel(wide ? move_rows_kernel<false> : move_rows_kernel<true>, dim3((unsigned)blocks), dim3(kThreads), 0,
                       s, 0, dim3(1), reinterpret_cast<uint4*>(pool), from * per, to * per, rows * per);
}

cudaError_t launch_remap(const RemapParams& p, cudaStream_t s) {
  int32_t most = 0;
  for (int i = 0; i < p.n_req; ++i) most = p.ctx[i] > most ? p.ctx[i] : most;
  int parts = (most + kThreads * 8 - 1) / (kThreads * 8);
  parts = parts < 1 ? 1 : (parts > 64 ? 64 : parts);
  return launch_kernel(remap_kernel, dim3((unsigned)(parts * p.n_req * p.n_layers)), dim3(kThreads), 0, s, 0,
                       dim3(1), p, parts);
}

}  // namespace qsa
