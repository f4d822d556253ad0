// Selection for every query of a chunk: per row the K = min(budget/4, nb) best
// of its nb = ceil((p+1)/4) blocks under (score descending, block id
// ascending), in ascending id order, as select_topk.cu selects for one query.
//
// One CTA per row.  A sample of kSample keys (groups of 8 neighbours, spread
// evenly) gives a pivot that a little more than K keys reach, with a margin of
// several standard deviations; one pass over the row collects the keys at or
// above it, with their ids, in shared memory (and their places in a bitmap);
// the rest works on those alone: radix select (11, 11, 10 bits) for the K-th
// best key T and how many keys equal to T are kept, two bitmaps (above T, equal
// to T) walked in id order, which gives the ascending output and the tie rule
// (lowest ids first).  So a row is read once: the kernel is bound by that
// (and not by a histogram of the whole row, whose few crowded bins serialise
// their atomic additions: 222 us for 2048 rows of 32768 scores).
//
// Where the pivot catches fewer than K or more than kCand keys (long runs of
// equal scores), or the row is longer than the bitmaps (kWindow blocks), the
// general path does the radix select on the row itself and walks it in
// windows.
#include "qsa_internal.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kWindow = 262144;      // blocks per window: two bitmaps of 32 KiB
constexpr int kSample = 2048;        // keys of the sample: 4 per thread
constexpr int kCand = 4096;          // candidates in shared memory

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

// Ascending ids of the keys above T and the first krem (lowest ids) of those
// equal to T, from bitmaps of blocks w0 .. w0 + 32 words - 1; out_at and eq_at
// count what earlier windows gave.
__device__ __forceinline__ void write_window(const uint32_t* above, const uint32_t* equal, int words, int64_t w0,
                                             uint32_t krem, int K, int32_t* sel, uint32_t& out_at, uint32_t& eq_at,
                                             uint32_t* s_warp) {
  const int per = (words + kThreads - 1) / kThreads;
  const int j0 = threadIdx.x * per, j1 = j0 + per < words ? j0 + per : words;
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
}

__global__ void __launch_bounds__(kThreads) chunk_topk_kernel(const __grid_constant__ ChunkTopkParams p) {
  extern __shared__ __align__(16) uint32_t bits[];     // two bitmaps of a window
  __shared__ __align__(16) uint32_t hist[kBins];
  __shared__ uint32_t cand_key[kCand];
  __shared__ int32_t cand_id[kCand];
  __shared__ uint32_t s_warp[kWarps], s_bin, s_rank, s_count;
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
  const int words_max = (int)((nb < kWindow ? nb : kWindow) + 31) / 32;
  uint32_t* above = bits;
  uint32_t* equal = bits + words_max;

  // ---- the usual path
  uint32_t found = 0;
  if (nb <= kWindow && K < kCand / 2) {
    const int n = (int)nb;
    if (tid == 0) s_count = 0;
    for (int i = tid; i < words_max; i += kThreads) above[i] = equal[i] = 0;
    // pivot: the key of rank r in the sample.  The number of sample keys among
    // the row's K best has mean K kSample / n = e and a standard deviation
    // below sqrt(e): r = e + 6 sqrt(e) + 8.  A row no longer than the candidate
    // list needs none.
    uint32_t pivot = 0;
    if (n > kCand) {
      const float e = (float)K * kSample / (float)n;
      uint32_t krem = (uint32_t)(e + 6.f * sqrtf(e)) + 8u;
      uint32_t k[kSample / kThreads];
      const int group = tid >> 1, groups = kSample / 8;
      const int64_t at = (int64_t)group * (n - 8) / (groups - 1) + 4 * (tid & 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) k[i] = order_key(s[at + i]);
      uint32_t mask = 0;
#pragma unroll 1
      for (int shift = 21; shift >= 10; shift -= 11) {     // 22 bits are fine enough
        for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((k[i] & mask) == pivot) atomicAdd(&hist[(k[i] >> shift) & 2047u], 1u);
        __syncthreads();
        find_bin(hist, krem, s_warp, &s_bin, &s_rank);
        pivot |= s_bin << shift;
        mask |= 2047u << shift;
        krem = s_rank;
        __syncthreads();
      }
    } else {
      __syncthreads();
    }
    // one pass over the row
    auto take = [&](uint32_t key, int id) {
      if (key >= pivot) {
        const uint32_t c = atomicAdd(&s_count, 1u);
        if (c < (uint32_t)kCand) { cand_key[c] = key; cand_id[c] = id; }
      }
    };
    const int head = (int)((16 - (reinterpret_cast<uintptr_t>(s) & 15)) & 15) / 4;   // to 16-byte loads
    if (tid < head && tid < n) take(order_key(s[tid]), tid);
    const int quads = (n - head) / 4;
    const float4* s4 = reinterpret_cast<const float4*>(s + head);
    constexpr int kBatch = 8;
    for (int q0 = tid; q0 < quads; q0 += kThreads * kBatch) {
      float4 v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int q = q0 + i * kThreads;
        v[i] = q < quads ? __ldcs(s4 + q) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int q = q0 + i * kThreads;
        if (q >= quads) break;
        const uint32_t k0 = order_key(v[i].x), k1 = order_key(v[i].y), k2 = order_key(v[i].z), k3 = order_key(v[i].w);
        if (max(max(k0, k1), max(k2, k3)) >= pivot) {
          const int id = head + 4 * q;
          take(k0, id);
          take(k1, id + 1);
          take(k2, id + 2);
          take(k3, id + 3);
        }
      }
    }
    for (int i = head + 4 * quads + tid; i < n; i += kThreads) take(order_key(s[i]), i);
    __syncthreads();
    found = s_count;
    __syncthreads();
  }

  // ---- T: the K-th best key, krem: how many keys equal to T are kept
  const bool usual = found >= (uint32_t)K && found <= (uint32_t)kCand;
  uint32_t T = 0, mask = 0, krem = (uint32_t)K;
  for (int shift = 21; shift >= 0; shift = shift == 21 ? 10 : shift - 10) {
    const uint32_t digits = shift == 0 ? 1024u : 2048u;
    for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
    __syncthreads();
    if (usual) {
      for (uint32_t i = tid; i < found; i += kThreads) {
        const uint32_t k = cand_key[i];
        if ((k & mask) == T) atomicAdd(&hist[(k >> shift) & (digits - 1)], 1u);
      }
    } else {
      for (int64_t i = tid; i < nb; i += kThreads) {
        const uint32_t k = order_key(s[i]);
        if ((k & mask) == T) atomicAdd(&hist[(k >> shift) & (digits - 1)], 1u);
      }
    }
    __syncthreads();
    find_bin(hist, krem, s_warp, &s_bin, &s_rank);
    T |= s_bin << shift;
    mask |= (digits - 1) << shift;
    krem = s_rank;
    __syncthreads();
  }

  uint32_t out_at = 0, eq_at = 0;
  if (usual) {
    for (uint32_t i = tid; i < found; i += kThreads) {
      const uint32_t k = cand_key[i];
      const int id = cand_id[i];
      if (k > T) atomicOr(&above[id >> 5], 1u << (id & 31));
      else if (k == T) atomicOr(&equal[id >> 5], 1u << (id & 31));
    }
    __syncthreads();
    write_window(above, equal, words_max, 0, krem, K, sel, out_at, eq_at, s_warp);
    return;
  }
  // ---- the general path: the row again, window by window
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
    write_window(above, equal, words, w0, krem, K, sel, out_at, eq_at, s_warp);
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
