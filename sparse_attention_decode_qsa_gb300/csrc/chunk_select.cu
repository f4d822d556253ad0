// Selection for every query of a chunk: per row the K = min(budget/4, nb) best
// of its nb = ceil((p+1)/4) blocks under (score descending, block id
// ascending), in ascending id order, as select_topk.cu selects for one query.
//
// One CTA per row.  Radix select (11, 11, 10 bits) on order-preserving keys
// finds the K-th best key T and how many keys equal to T are kept; then two
// bitmaps in shared memory (keys above T, keys equal to T) are walked in id
// order, in windows of kWindow blocks, which gives the ascending output and
// the tie rule (lowest ids first).
#include "qsa_internal.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kWindow = 262144;      // blocks per window: two bitmaps of 32 KiB

struct ChunkTopkParams {
  ChunkDesc c;
  const float* blk;     // [rows][blk_stride]
  int64_t blk_stride;
  int32_t k_max;
  int32_t* sel;         // [rows][k_max]
  int32_t* n_sel;       // [rows]
};

// Larger float -> larger unsigned key; -0.0 is folded onto +0.0.
__device__ __forceinline__ uint32_t order_key(float f) {
  uint32_t x = __float_as_uint(f);
  if (x == 0x80000000u) x = 0u;
  return (x & 0x80000000u) ? ~x : (x | 0x80000000u);
}

// Exclusive scan of v over the CTA; *total receives the sum.  Called by every
// thread; the closing barrier lets the next call reuse s_warp.
__device__ __forceinline__ uint32_t scan(uint32_t v, uint32_t* total, uint32_t* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  uint32_t before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_warp[w];
    sum += s_warp[w];
  }
  __syncthreads();
  *total = sum;
  return before + x - v;
}

// The bin (from the top) that holds the krem-th largest key of the histogram,
// and the key's rank in it.  Thread t owns the bins kBins-1-4t .. kBins-4-4t.
// The caller has synchronised the histogram; results are valid on return.
__device__ __forceinline__ void find_bin(const uint32_t* hist, uint32_t krem, uint32_t* s_warp, uint32_t* s_bin,
                                         uint32_t* s_rank) {
  static_assert(kBins == 4 * kThreads, "four bins per thread");
  const uint4 c = *reinterpret_cast<const uint4*>(hist + kBins - 4 * (threadIdx.x + 1));
  const uint32_t v[4] = {c.w, c.z, c.y, c.x};
  uint32_t total;
  uint32_t cum = scan(v[0] + v[1] + v[2] + v[3], &total, s_warp);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (cum < krem && krem <= cum + v[j]) {
      *s_bin = kBins - 1 - (4 * threadIdx.x + j);
      *s_rank = krem - cum;
    }
    cum += v[j];
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kThreads) chunk_topk_kernel(const __grid_constant__ ChunkTopkParams p) {
  extern __shared__ __align__(16) uint32_t bits[];     // two bitmaps of a window
  __shared__ __align__(16) uint32_t hist[kBins];
  __shared__ uint32_t s_warp[kWarps], s_bin, s_rank;
  const int x = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const int u = p.c.unit_of_row(x);
  const int64_t nb = p.c.position(u, x) / 4 + 1;
  const int K = nb < p.k_max ? (int)nb : p.k_max;
  const float* s = p.blk + (int64_t)x * p.blk_stride;
  int32_t* sel = p.sel + (int64_t)x * p.k_max;
  grid_dependency_wait();
  if (tid == 0) p.n_sel[x] = K;
  if (K == nb) {                     // the budget covers the context
    for (int i = tid; i < K; i += kThreads) sel[i] = i;
    return;
  }

  // ---- T: the K-th best key, krem: how many keys equal to T are kept
  uint32_t T = 0, mask = 0, krem = (uint32_t)K;
  for (int shift = 21; shift >= 0; shift = shift == 21 ? 10 : shift - 10) {
    const uint32_t digits = shift == 0 ? 1024u : 2048u;
    for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
    __syncthreads();
    for (int64_t i = tid; i < nb; i += kThreads) {
      const uint32_t k = order_key(s[i]);
      if ((k & mask) == T) atomicAdd(&hist[(k >> shift) & (digits - 1)], 1u);
    }
    __syncthreads();
    find_bin(hist, krem, s_warp, &s_bin, &s_rank);
    T |= s_bin << shift;
    mask |= (digits - 1) << shift;
    krem = s_rank;
    __syncthreads();
  }

  // ---- ascending output, window by window
  uint32_t out_at = 0, eq_at = 0;
  const int words_max = (int)((nb < kWindow ? nb : kWindow) + 31) / 32;
  uint32_t* above = bits;
  uint32_t* equal = bits + words_max;
  for (int64_t w0 = 0; w0 < nb; w0 += kWindow) {
    const int count = nb - w0 < kWindow ? (int)(nb - w0) : kWindow;
    const int words = (count + 31) / 32;
    for (int i = tid; i < words * 32; i += kThreads) {      // whole warps
      const uint32_t k = i < count ? order_key(s[w0 + i]) : 0u;
      const uint32_t a = __ballot_sync(0xFFFFFFFFu, i < count && k > T);
      const uint32_t e = __ballot_sync(0xFFFFFFFFu, i < count && k == T);
      if (lane == 0) { above[i / 32] = a; equal[i / 32] = e; }
    }
    __syncthreads();
    const int per = (words + kThreads - 1) / kThreads;
    const int j0 = tid * per, j1 = j0 + per < words ? j0 + per : words;
    uint32_t na = 0, ne = 0;
    for (int j = j0; j < j1; ++j) { na += __popc(above[j]); ne += __popc(equal[j]); }
    uint32_t ta, te;
    uint32_t a_before = out_at + scan(na, &ta, s_warp), e_before = eq_at + scan(ne, &te, s_warp);
    for (int j = j0; j < j1; ++j) {
      const uint32_t a = above[j], e = equal[j];
      for (uint32_t m = a | e; m; m &= m - 1) {
        const int bit = __ffs(m) - 1;
        const uint32_t at = a_before + min(e_before, krem);
        if ((a >> bit) & 1u) {
          if (at < (uint32_t)K) sel[at] = (int32_t)(w0 + 32 * j + bit);
          ++a_before;
        } else {
          if (e_before < krem && at < (uint32_t)K) sel[at] = (int32_t)(w0 + 32 * j + bit);
          ++e_before;
        }
      }
    }
    out_at += ta;
    eq_at += te;
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_chunk_topk(const ChunkDesc& c, const float* blk_scores, int64_t blk_stride,
                              int32_t k_max, int32_t* sel_blocks, int32_t* n_sel, cudaStream_t s) {
  ChunkTopkParams p;
  p.c = c;
  p.blk = blk_scores;
  p.blk_stride = blk_stride;
  p.k_max = k_max;
  p.sel = sel_blocks;
  p.n_sel = n_sel;
  static PerDeviceOnce setup;
  const cudaError_t e = setup.run([] { return prefer_max_shared(chunk_topk_kernel, 2 * kWindow / 8); });
  if (e != cudaSuccess) return e;
  int64_t nb = 0;
  for (int u = 0; u < c.b.n_units; ++u)
    if (c.unit_tokens(u) > 0 && (c.b.u[u].n + 3) / 4 > nb) nb = (c.b.u[u].n + 3) / 4;
  if (nb > kWindow) nb = kWindow;
  return launch_kernel(chunk_topk_kernel, dim3((unsigned)c.rows()), dim3(kThreads), (size_t)((nb + 31) / 32 * 8), s, 0,
                       dim3(1), p);
}

}  // namespace qsa
