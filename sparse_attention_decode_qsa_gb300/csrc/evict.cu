// Eviction of the tokens of a request that attention used least, all layers at
// once, each by its own weights: the first and the last tokens stay, and of the
// rest those with the largest weights (equal weights: the lower position).
//
//  * select: per layer the keep-th largest weight by a radix select over the
//    weights' bits, eight at a time, then the kept positions in ascending order;
//    the kept tokens' new slots; and the list of rows that have to move.
//  * move: those rows, and the kept tokens' keys, scales and weights (the keys
//    and scales into the workspace, since they close up within their own arrays).
//  * close: keys, scales and slots to their places.
//
// Rows move as little as they can.  Logical order lives in the slot table alone,
// so a kept token whose row lies among the region's first `keep` stays where it
// is, and the others, in ascending order of position, take the rows there that
// became free: no row is both read and written, and half of the tokens evicted
// at random moves a quarter of the rows (closing the rows up in order would move
// nearly half, one behind the other).  The request's next tokens find the
// region's rows from `keep` on free, as qsa_append_token expects.
//
// Measured: 12 layers, 32768 -> 16384 BF16 tokens at random: select 23 us (latencies of
// seven cluster barriers and the passes between them), move 67 us (406 MB, 0.90 of the
// measured copy rate), close 7 us.  12 layers, 2047 -> 1021 FP8 tokens: 9 + 8 + 4 us.
#include "qsa_internal.cuh"

namespace qsa {
namespace {

constexpr int kSelectThreads = 512, kSelectWarps = kSelectThreads / 32;
constexpr int kSelectCtas = 8;                    // a cluster per layer

// Descending order of weights as unsigned integers: -0 equals +0, NaN comes last.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Barrier of the cluster: what its threads wrote before (to shared memory or to
// global memory) its threads see afterwards.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The word at `local` in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t cluster_read(const uint32_t* local, uint32_t rank) {
  uint32_t at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(local)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// Whole CTA: exclusive prefix sums over the warps of one value per warp, and the
// total.
__device__ __forceinline__ uint32_t warp_offsets(uint32_t mine, uint32_t* s_warp, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0) s_warp[warp] = mine;
  __syncthreads();
  uint32_t v = lane < kSelectWarps ? s_warp[lane] : 0u;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += y;
  }
  *total = __shfl_sync(0xFFFFFFFFu, v, 31);
  return __shfl_sync(0xFFFFFFFFu, v, warp) - mine;
}
static_assert(kSelectWarps <= 32, "one lane per warp in the scan");

// Whole cluster: the sums of two values over the CTAs before this one (both values
// the same in all threads of a CTA), and over all.  s_pair has been left by the
// readers of an earlier exchange (a cluster barrier lies in between).
__device__ __forceinline__ void cta_offsets(uint32_t a, uint32_t b, uint32_t* s_pair, uint32_t rank, uint32_t* a0,
                                            uint32_t* b0, uint32_t* a_all) {
  if (threadIdx.x == 0) {
    s_pair[0] = a;
    s_pair[1] = b;
  }
  cluster_sync();
  *a0 = *b0 = *a_all = 0;
#pragma unroll
  for (uint32_t r = 0; r < kSelectCtas; ++r) {
    const uint32_t x = cluster_read(s_pair, r), y = cluster_read(s_pair + 1, r);
    *a_all += x;
    if (r < rank) {
      *a0 += x;
      *b0 += y;
    }
  }
}

// One cluster per layer; each CTA has an eighth of the tokens, and then of the kept
// ones.  Per digit every CTA counts its own keys and adds up all CTAs' counts from
// their shared memory: one cluster barrier per digit.  12 layers of 32768 tokens: 50
// us with one CTA per layer, 44 with digits of 11 bits and 1024 threads (the sums over
// 2048 bins of eight CTAs), 41 where every row's bit was an atomic of its own.
__global__ void __launch_bounds__(kSelectThreads, 1) __cluster_dims__(kSelectCtas, 1, 1)
evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ uint32_t hist[4][256], s_warp[kSelectWarps], s_bin[2], s_pair[2][2];
  const int layer = blockIdx.x / kSelectCtas, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  const float* w = p.weights + layer * p.weight_stride;
  // (fewer than 2^31 tokens: places and rows fit 32 bits)
  const uint32_t n = (uint32_t)p.n, keep = (uint32_t)p.keep, lo = (uint32_t)p.first, hi = (uint32_t)(p.n - p.last);      // lo .. hi - 1 compete
  int32_t* kept = p.kept + layer * p.keep;
  const int32_t* slots = p.slot_table + ((int64_t)p.req * p.n_layers + layer) * p.ctx_cap;
  int32_t* new_slot = p.new_slot + layer * p.keep;
  int32_t* holes = p.holes + layer * p.keep;
  uint32_t* used = p.used + layer * p.used_words;
  int2* moves = p.moves + layer * p.keep;
  for (int i = tid; i < 4 * 256; i += kSelectThreads) (&hist[0][0])[i] = 0;
  // runs of whole 32s: of the tokens per CTA and warp, of the kept ones likewise
  auto run_of = [&](uint32_t count, uint32_t* from, uint32_t* to) {
    const uint32_t words = (count + 31) / 32, per = (words + kSelectCtas * kSelectWarps - 1) / (kSelectCtas * kSelectWarps);
    const uint64_t a = (uint64_t)(rank * kSelectWarps + warp) * per * 32, e = a + per * 32;
    *from = a < count ? (uint32_t)a : count;
    *to = e < count ? (uint32_t)e : count;
  };
  uint32_t t0, t1, k0, k1;
  run_of(n, &t0, &t1);
  run_of(keep, &k0, &k1);
  grid_dependency_wait();
  for (int64_t i = (int64_t)rank * kSelectThreads + tid; i < p.used_words; i += kSelectCtas * kSelectThreads) used[i] = 0;
  __syncthreads();

  // eight words of 32 tokens at a time, their loads side by side
  constexpr int kTurn = 8;
  auto load = [&](uint32_t t, float (&v)[kTurn]) {
#pragma unroll
    for (int j = 0; j < kTurn; ++j) v[j] = t + 32 * j + lane < t1 ? w[t + 32 * j + lane] : 0.f;
  };

  // ---- the need-th largest key T, and how many tokens at T stay
  const int64_t need = keep - p.first - p.last;
  uint32_t T = 0, left = (uint32_t)need;
  if (need > 0) {
    uint32_t mask = 0;
#pragma unroll 1
    for (int d = 0; d < 4; ++d) {
      const int shift = 24 - 8 * d;
      for (uint32_t t = t0; t < t1; t += 32 * kTurn) {
        float v[kTurn];
        load(t, v);
#pragma unroll
        for (int j = 0; j < kTurn; ++j) {
          const uint32_t at = t + 32 * j + lane;
          const uint32_t k = weight_key(v[j]);
          if (at < t1 && at >= lo && at < hi && (k & mask) == T) atomicAdd(&hist[d][(k >> shift) & 255u], 1u);
        }
      }
      cluster_sync();
      // bins from the top, one a thread
      uint32_t a = 0;
      if (tid < 256) {
#pragma unroll
        for (uint32_t r = 0; r < kSelectCtas; ++r) a += cluster_read(&hist[d][255 - tid], r);
      }
      uint32_t v = a;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += y;
      }
      uint32_t total;
      const uint32_t before = warp_offsets(__shfl_sync(0xFFFFFFFFu, v, 31), s_warp, &total) + v - a;
      if (before < left && left <= before + a) {
        s_bin[0] = 255 - tid;
        s_bin[1] = left - before;
      }
      __syncthreads();
      T |= s_bin[0] << shift;
      left = s_bin[1];
      mask |= 255u << shift;
    }
  }

  // ---- kept positions, ascending
  auto look = [&](uint32_t t, float v, uint32_t* more, uint32_t* same) {
    const bool there = t < t1, mid = there && t >= lo && t < hi;
    const uint32_t k = weight_key(v);
    *more = __ballot_sync(0xFFFFFFFFu, there && (!mid || (need > 0 && k > T)));
    *same = __ballot_sync(0xFFFFFFFFu, mid && need > 0 && k == T);
  };
  uint32_t more, same, n_more = 0, n_same = 0, all_more, all_same, c_more, c_same, total;
  for (uint32_t t = t0; t < t1; t += 32 * kTurn) {
    float v[kTurn];
    load(t, v);
#pragma unroll
    for (int j = 0; j < kTurn; ++j) {
      look(t + 32 * j + lane, v[j], &more, &same);
      n_more += __popc(more);
      n_same += __popc(same);
    }
  }
  uint32_t b_more = warp_offsets(n_more, s_warp, &all_more), b_same = warp_offsets(n_same, s_warp, &all_same);
  cta_offsets(all_more, all_same, s_pair[0], rank, &c_more, &c_same, &total);
  b_more += c_more;
  b_same += c_same;
  const int32_t base = (int32_t)(p.row_base + layer * p.layer_rows);
  for (uint32_t t = t0; t < t1; t += 32 * kTurn) {
    float v[kTurn];
    int32_t slot[kTurn];
    load(t, v);
#pragma unroll
    for (int j = 0; j < kTurn; ++j) slot[j] = t + 32 * j + lane < t1 ? slots[t + 32 * j + lane] : 0;
#pragma unroll
    for (int j = 0; j < kTurn; ++j) {
      const uint32_t at = t + 32 * j + lane;
      look(at, v[j], &more, &same);
      const uint32_t below = (1u << lane) - 1u, bit = 1u << lane;
      const uint32_t rank_same = b_same + __popc(same & below);
      uint32_t row = keep;                           // of the region, `keep` or more: none of its first `keep`
      if ((more & bit) || ((same & bit) && rank_same < left)) {
        // the token stays: its place, its slot, and its row if that is among the first `keep`
        const uint32_t i = b_more + __popc(more & below) + (rank_same < left ? rank_same : left);
        kept[i] = (int32_t)at;
        new_slot[i] = slot[j];
        if (slot[j] < 0 || (int64_t)slot[j] >= p.pool_rows) report_error(p.err, QSA_ERR_BAD_SLOT, kKernEvict, at);
        row = slot[j] >= base ? (uint32_t)(slot[j] - base) : keep;
      }
      // rows in use: a word of 32 rows at once where the warp's rows lie in one
      const uint32_t low = __ballot_sync(0xFFFFFFFFu, row < keep);
      if (low) {
        const uint32_t word = __shfl_sync(0xFFFFFFFFu, row >> 5, __ffs(low) - 1);
        const bool mine = row < keep;
        if (__all_sync(0xFFFFFFFFu, !mine || (row >> 5) == word)) {
          const uint32_t bits = __reduce_or_sync(0xFFFFFFFFu, mine ? 1u << (row & 31) : 0u);
          if (lane == 0) atomicOr(used + word, bits);
        } else if (mine) {
          atomicOr(used + (row >> 5), 1u << (row & 31));
        }
      }
      b_more += __popc(more);
      b_same += __popc(same);
    }
  }
  __threadfence();
  cluster_sync();

  // ---- the free rows below `keep`, and the kept tokens whose rows have to move there
  const uint32_t layer_rows = (uint32_t)p.layer_rows;
  auto moves_away = [&](int32_t slot) {
    return slot >= base && (uint32_t)(slot - base) >= keep && (uint32_t)(slot - base) < layer_rows;
  };
  // of the 32 kept places (or rows) from i on: free rows, and tokens that move
  auto rows_at = [&](uint32_t i, uint32_t (&open)[kTurn], int32_t (&slot)[kTurn]) {
#pragma unroll
    for (int j = 0; j < kTurn; ++j) {
      const uint32_t at = i + 32 * j;
      open[j] = at < k1 ? ~__ldcg(used + (at >> 5)) : 0u;
      if (at < k1 && k1 - at < 32) open[j] &= (1u << (k1 - at)) - 1u;
      slot[j] = at + lane < k1 ? __ldcg(new_slot + at + lane) : -1;
    }
  };
  uint32_t n_free = 0, n_away = 0, all_free, all_away, c_free, c_away;
  for (uint32_t i = k0; i < k1; i += 32 * kTurn) {
    uint32_t open[kTurn];
    int32_t slot[kTurn];
    rows_at(i, open, slot);
#pragma unroll
    for (int j = 0; j < kTurn; ++j) {
      n_free += __popc(open[j]);
      n_away += __popc(__ballot_sync(0xFFFFFFFFu, moves_away(slot[j])));
    }
  }
  uint32_t b_free = warp_offsets(n_free, s_warp, &all_free), b_away = warp_offsets(n_away, s_warp, &all_away);
  cta_offsets(all_away, all_free, s_pair[1], rank, &c_away, &c_free, &total);
  b_free += c_free;
  b_away += c_away;
  const uint32_t below = (1u << lane) - 1u;
  for (uint32_t i = k0; i < k1; i += 32 * kTurn) {
    uint32_t open[kTurn];
    int32_t slot[kTurn];
    rows_at(i, open, slot);
#pragma unroll
    for (int j = 0; j < kTurn; ++j) {
      if ((open[j] >> lane) & 1u) holes[b_free + __popc(open[j] & below)] = (int32_t)(i + 32 * j + lane);
      b_free += __popc(open[j]);
    }
  }
  __threadfence();
  cluster_sync();
  // (there are no fewer free rows than moving ones: the tokens in rows below
  // `keep` use at most one row each)
  for (uint32_t i = k0; i < k1; i += 32 * kTurn) {
    uint32_t open[kTurn], r[kTurn];
    int32_t slot[kTurn], to[kTurn];
    rows_at(i, open, slot);
#pragma unroll
    for (int j = 0; j < kTurn; ++j) {
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, moves_away(slot[j]));
      r[j] = b_away + __popc(m & below);
      to[j] = moves_away(slot[j]) ? base + (int32_t)__ldcg(holes + r[j]) : 0;
      b_away += __popc(m);
    }
#pragma unroll
    for (int j = 0; j < kTurn; ++j) {
      if (!moves_away(slot[j])) continue;
      moves[r[j]] = make_int2(slot[j], to[j]);
      new_slot[i + 32 * j + lane] = to[j];
    }
  }
  if (tid == 0 && rank == 0) p.n_moves[layer] = (int32_t)total;
}

constexpr int kMoveThreads = 256, kMoveWarps = kMoveThreads / 32;
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictParams p) {
  const int layer = blockIdx.y, lane = threadIdx.x & 31;
  const int64_t warp = (int64_t)blockIdx.x * kMoveWarps + (threadIdx.x >> 5), warps = (int64_t)gridDim.x * kMoveWarps;
  grid_dependency_wait();
  const int32_t* kept = p.kept + layer * p.keep;
  const int2* moves = p.moves + layer * p.keep;
  const int n_moves = p.n_moves[layer];
  const int chunks = p.row_bytes / 16;       // 128 (BF16) or 65 (FP8)
  for (int64_t m = warp; m < n_moves; m += warps) {
    const int2 mv = moves[m];
    const uint4* src = reinterpret_cast<const uint4*>(p.pool + (int64_t)mv.x * p.row_bytes);
    uint4* dst = reinterpret_cast<uint4*>(p.pool + (int64_t)mv.y * p.row_bytes);
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (lane + 32 * j < chunks) v[j] = src[lane + 32 * j];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (lane + 32 * j < chunks) dst[lane + 32 * j] = v[j];
  }
  // keys: four lanes a token
  const int64_t st = ((int64_t)p.req * p.n_layers + layer) * p.ctx_cap;
  const uint4* keys = reinterpret_cast<const uint4*>(p.index_keys + st * kIndexDim);
  uint4* keys_ws = reinterpret_cast<uint4*>(p.keys_ws + layer * p.keep * kIndexDim);
  for (int64_t i = warp * 8 + (lane >> 2); i < p.keep; i += warps * 8)
    keys_ws[4 * i + (lane & 3)] = keys[4 * (int64_t)kept[i] + (lane & 3)];
  for (int64_t i = warp * 32 + lane; i < p.keep; i += warps * 32) {
    const int64_t t = kept[i];
    p.scales_ws[layer * p.keep + i] = p.index_scales[st + t];
    if (p.weights_out) p.weights_out[layer * p.out_stride + i] = p.weights[layer * p.weight_stride + t];
  }
}

__global__ void __launch_bounds__(kMoveThreads) evict_close_kernel(const __grid_constant__ EvictParams p) {
  const int layer = blockIdx.y;
  const int64_t i0 = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x, step = (int64_t)gridDim.x * kMoveThreads;
  grid_dependency_wait();
  const int64_t st = ((int64_t)p.req * p.n_layers + layer) * p.ctx_cap;
  uint4* keys = reinterpret_cast<uint4*>(p.index_keys + st * kIndexDim);
  const uint4* keys_ws = reinterpret_cast<const uint4*>(p.keys_ws + layer * p.keep * kIndexDim);
  for (int64_t i = i0; i < 4 * p.keep; i += step) keys[i] = keys_ws[i];
  for (int64_t i = i0; i < p.keep; i += step) {
    p.index_scales[st + i] = p.scales_ws[layer * p.keep + i];
    p.slot_table[st + i] = p.new_slot[layer * p.keep + i];
  }
}

}  // namespace

int64_t evict_layout(EvictParams* p, void* workspace) {
  const int64_t all = (int64_t)p->n_layers * p->keep;
  const uintptr_t start = reinterpret_cast<uintptr_t>(workspace);
  uintptr_t at = start;
  auto take = [&](int64_t bytes) {
    const uintptr_t r = at;
    at += (bytes + 255) / 256 * 256;
    return r;
  };
  p->used_words = (p->keep + 31) / 32;
  p->n_moves = reinterpret_cast<int32_t*>(take(4 * (int64_t)p->n_layers));
  p->kept = reinterpret_cast<int32_t*>(take(4 * all));
  p->new_slot = reinterpret_cast<int32_t*>(take(4 * all));
  p->holes = reinterpret_cast<int32_t*>(take(4 * all));
  p->used = reinterpret_cast<uint32_t*>(take(4 * p->used_words * p->n_layers));
  p->moves = reinterpret_cast<int2*>(take(8 * all));
  p->keys_ws = reinterpret_cast<uint8_t*>(take(kIndexDim * all));
  p->scales_ws = reinterpret_cast<uint16_t*>(take(2 * all));
  return (int64_t)(at - start);
}

cudaError_t launch_evict(const EvictParams& p, cudaStream_t s) {
  int sms = 0;
  if (const cudaError_t e = current_sm_count(&sms)) return e;
  cudaError_t e = launch_kernel(evict_select_kernel, dim3(p.n_layers * kSelectCtas), dim3(kSelectThreads), 0, s, 0,
                                dim3(1), p);
  if (e != cudaSuccess) return e;
  // eight CTAs per SM over all layers, a row per warp and turn
  int64_t blocks = (p.keep + kMoveWarps - 1) / kMoveWarps;
  const int64_t most = ((int64_t)sms * 8 + p.n_layers - 1) / p.n_layers;
  if (blocks > most) blocks = most;
  e = launch_kernel(evict_move_kernel, dim3((unsigned)blocks, p.n_layers), dim3(kMoveThreads), 0, s, 0, dim3(1), p);
  if (e != cudaSuccess) return e;
  return launch_kernel(evict_close_kernel, dim3((unsigned)blocks, p.n_layers), dim3(kMoveThreads), 0, s, 0, dim3(1), p);
}

}  // namespace qsa
