// Selection for every query of a chunk: per row the K = min(budget/4, nb) best
// of its nb = ceil((p+1)/4) blocks under (score descending, block id
// ascending), in ascending id order, as select_topk.cu selects for one query.
//
// One CTA per row.  A sample of the row's keys gives a pivot that a little more
// than K keys reach, with a margin of several standard deviations; one pass over
// the row marks the keys at or above it in a bitmap (a ballot per 32 keys); the
// marked ones, a few thousand at most, are fetched again in id order and the
// rest works on those alone: one histogram over their own range and a ranking
// of the few in the K-th key's bin find the K-th best key T and how many keys
// equal to T are kept, and a scan over the candidates writes the ids, which come
// out ascending, lowest ids first among the keys equal to T.  So a row is read
// once, and no histogram sees the whole row, whose few crowded bins would
// serialise their atomic additions (222 us for 2048 rows of 32768 scores;
// collecting the keys themselves during the pass took 153; 95 as it is, 0.43 of
// the copy rate, with four rows to an SM, 100 with three: what is left are the
// short steps after the pass, each a few thousand cycles of latency).  14 rows of
// draft tokens take 16 us, those latencies alone.
//
// Where the pivot catches fewer than K or more than kCand keys (long runs of
// equal scores), or the row is longer than the bitmaps (kWindow blocks), the
// general path does the radix select on the row itself and walks it, window by
// window, with two bitmaps (above T, equal to T).  Budgets from 8192 tokens on
// (K = kCand / 2) take it always.  2048 rows of 32768 blocks: 356 us at a budget of
// 8192, 382 with all scores equal, 169 with scores rounded to halves, where some
// rows take it; 14 rows 64 to 75 us.
#include "qsa_internal.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kWindow = 262144;      // blocks per window: two bitmaps of 32 KiB
constexpr int kCand = 4096;          // candidates in shared memory
constexpr int kLongRow = 32768;      // rows beyond this many blocks take 512 samples, not 256

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

constexpr uint32_t kLeastKey = 0x007FFFFFu;      // of -infinity

__device__ __forceinline__ float order_value(uint32_t key) {      // of order_key
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// The r-th largest (r >= 1) of kSamples keys in shared memory, the smallest key
// with fewer than r above it: every key is compared with all others, kThreads /
// kSamples threads per key.  *pivot starts at the largest key value.
template <int kSamples>
__device__ __forceinline__ void find_pivot(const uint32_t* sample, uint32_t r, uint32_t* pivot) {
  constexpr int kShare = kThreads / kSamples;
  const int part = threadIdx.x % kShare;
  const uint32_t key = sample[threadIdx.x / kShare];
  uint32_t above = 0;
#pragma unroll 8
  for (int j = part * 4; j < kSamples; j += 4 * kShare) {
    const uint4 o = *reinterpret_cast<const uint4*>(sample + j);
    above += (o.x > key) + (o.y > key) + (o.z > key) + (o.w > key);
  }
#pragma unroll
  for (int o = kShare / 2; o > 0; o >>= 1) above += __shfl_xor_sync(0xFFFFFFFFu, above, o);
  if (part == 0 && above < r) atomicMin(pivot, key);
}

__global__ void __launch_bounds__(kThreads, 4) chunk_topk_kernel(const __grid_constant__ ChunkTopkParams p) {
  extern __shared__ __align__(16) uint32_t bits[];     // two bitmaps of a window
  __shared__ __align__(16) uint32_t hist[kBins];
  __shared__ __align__(16) uint32_t cand_key[kCand];
  __shared__ int32_t cand_id[kCand];
  __shared__ uint32_t s_warp[kWarps], s_bin, s_rank, s_pivot, s_max, s_list, s_key[32];
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

  // ---- the usual path: candidates in id order
  uint32_t found = 0, pivot = kLeastKey;
  if (nb <= kWindow && K < kCand / 2) {
    const int n = (int)nb;
    if (tid == 0) { s_max = 0; s_list = 0; s_pivot = n > kCand ? 0xFFFFFFFFu : kLeastKey; }
    for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
    // The number of sample keys among the row's K best has mean e = K samples /
    // n and a standard deviation below sqrt(e): rank r = e + 4 sqrt(e) + 4.  A
    // row no longer than the candidate list needs no pivot.
    if (n > kCand) {
      const int samples = n > kLongRow ? kThreads : kThreads / 2;
      const float e = (float)K * samples / (float)n;
      const uint32_t r = (uint32_t)(e + 4.f * sqrtf(e)) + 4u;        // below samples: K < kCand / 2 < n / 2
      // spread evenly: neighbouring blocks' scores go together
      if (tid < samples) cand_key[tid] = order_key(s[(int64_t)tid * (n - 1) / (samples - 1)]);
      __syncthreads();
      if (samples == kThreads) find_pivot<kThreads>(cand_key, r, &s_pivot);
      else find_pivot<kThreads / 2>(cand_key, r, &s_pivot);
    }
    __syncthreads();
    pivot = s_pivot;
    // one pass over the row: a warp takes 256 neighbouring keys at a time, one
    // bitmap word per 32
    // (the keys' order is the values' own: scores are not NaN)
    constexpr int kBatch = 8;
    const int warp = tid >> 5;
    const float least = order_value(pivot);
    float v[kBatch];
    auto load = [&](int b) {
      if (b + 32 * kBatch <= n) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) v[i] = __ldg(s + b + 32 * i + lane);
      } else {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int id = b + 32 * i + lane;
          v[i] = id < n ? __ldg(s + id) : __uint_as_float(0x7FFFFFFFu);       // NaN: below everything
        }
      }
    };
    load(warp * 32 * kBatch);
    for (int b = warp * 32 * kBatch; b < n; b += kThreads * kBatch) {
      uint32_t word = 0;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, v[i] >= least);
        if (lane == i) word = m;
      }
      load(b + kThreads * kBatch);       // the next ones, in flight
      if (lane < kBatch && b / 32 + lane < words_max) bits[b / 32 + lane] = word;
    }
    __syncthreads();
    // the marked keys, in id order: thread t takes words t per .. t per + per - 1
    const int per = (words_max + kThreads - 1) / kThreads;
    const int j0 = tid * per, j1 = j0 + per < words_max ? j0 + per : words_max;
    uint32_t c = 0;
    for (int j = j0; j < j1; ++j) c += __popc(bits[j]);
    uint32_t at = scan(c, &found, s_warp);
    if (found <= (uint32_t)kCand) {
      for (int j = j0; j < j1; ++j) {
        for (uint32_t m = bits[j]; m; m &= m - 1) cand_id[at++] = 32 * j + __ffs(m) - 1;
      }
      __syncthreads();
      uint32_t top = 0;
      for (uint32_t i = tid; i < found; i += kThreads) {
        const uint32_t k = order_key(__ldg(s + cand_id[i]));
        cand_key[i] = k;
        top = max(top, k);
      }
      top = __reduce_max_sync(0xFFFFFFFFu, top);
      if (lane == 0) atomicMax(&s_max, top);
    }
    __syncthreads();
  }

  // ---- T: the K-th best key, krem: how many keys equal to T are kept
  const bool usual = found >= (uint32_t)K && found <= (uint32_t)kCand;
  uint32_t T = 0, krem = (uint32_t)K;
  bool exact = false;
  if (usual) {
    const uint32_t span = s_max - pivot;
    const int shift = span < 2048u ? 0 : 21 - __clz(span);         // span >> shift < 2048
    for (uint32_t i = tid; i < found; i += kThreads) atomicAdd(&hist[(cand_key[i] - pivot) >> shift], 1u);
    __syncthreads();
    find_bin(hist, krem, s_warp, &s_bin, &s_rank);
    const uint32_t bin = s_bin, in_bin = hist[bin];
    krem = s_rank;
    if (shift == 0) {
      T = pivot + bin;
      exact = true;
    } else if (in_bin <= 32u) {
      for (uint32_t i = tid; i < found; i += kThreads) {
        const uint32_t k = cand_key[i];
        if ((k - pivot) >> shift == bin) s_key[atomicAdd(&s_list, 1u)] = k;
      }
      __syncthreads();
      // every warp ranks them: T is the value with fewer than krem above it and
      // at least krem above or equal
      const uint32_t v = (uint32_t)lane < in_bin ? s_key[lane] : 0u;
      uint32_t gt = 0, eq = 0;
      for (uint32_t j = 0; j < in_bin; ++j) {
        const uint32_t o = __shfl_sync(0xFFFFFFFFu, v, (int)j);
        gt += o > v;
        eq += o == v;
      }
      const uint32_t hit = __ballot_sync(0xFFFFFFFFu, (uint32_t)lane < in_bin && gt < krem && krem <= gt + eq);
      const int src = hit ? __ffs(hit) - 1 : 0;
      T = __shfl_sync(0xFFFFFFFFu, v, src);
      krem -= __shfl_sync(0xFFFFFFFFu, gt, src);
      exact = true;
    }
  }
  if (!exact) {                          // radix select on the candidates, or on the row
    uint32_t mask = 0;
    T = 0;
    krem = (uint32_t)K;
    __syncthreads();
#pragma unroll 1
    for (int shift = 21; shift >= 0; shift = shift == 21 ? 10 : shift - 10) {
      const uint32_t digits = shift == 0 ? 1024u : 2048u;
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
      __syncthreads();
      const int64_t m = usual ? (int64_t)found : nb;
      for (int64_t i = tid; i < m; i += kThreads) {
        const uint32_t k = usual ? cand_key[i] : order_key(s[i]);
        if ((k & mask) == T) atomicAdd(&hist[(k >> shift) & (digits - 1)], 1u);
      }
      __syncthreads();
      find_bin(hist, krem, s_warp, &s_bin, &s_rank);
      T |= s_bin << shift;
      mask |= (digits - 1) << shift;
      krem = s_rank;
      __syncthreads();
    }
  }

  // ---- ids in ascending order
  uint32_t out_at = 0, eq_at = 0;
  if (usual) {
    const int per = ((int)found + kThreads - 1) / kThreads;          // at most 8
    const int i0 = tid * per, i1 = i0 + per < (int)found ? i0 + per : (int)found;
    uint32_t n = 0;                      // keys above T, and (upper half) equal to T
    for (int i = i0; i < i1; ++i) n += (cand_key[i] > T ? 1u : 0u) + (cand_key[i] == T ? 0x10000u : 0u);
    uint32_t total;
    const uint32_t before = scan(n, &total, s_warp);
    uint32_t a = before & 0xFFFFu, e = before >> 16;
    for (int i = i0; i < i1; ++i) {
      const uint32_t k = cand_key[i];
      const uint32_t at = a + min(e, krem);
      if ((k > T || (k == T && e < krem)) && at < (uint32_t)K) sel[at] = cand_id[i];
      a += k > T;
      e += k == T;
    }
    return;
  }
  // the general path: the row again, window by window
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
