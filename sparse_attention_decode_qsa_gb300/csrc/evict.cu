// Eviction of the tokens of a request that attention used least, all layers at
// once, each by its own weights: the first and the last tokens stay, and of the
// rest those with the largest weights (equal weights: the lower position).
//
//  * select: per layer the keep-th largest weight by a radix select over the
//    weights' bits (11 + 11 + 10), then the kept positions in ascending order;
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
#include "qsa_internal.cuh"

namespace qsa {
namespace {

constexpr int kSelectThreads = 1024, kSelectWarps = kSelectThreads / 32;

// Descending order of weights as unsigned integers: -0 equals +0, NaN comes last.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Whole CTA: exclusive prefix sums over the warps of one value per warp, and the
// total.
__device__ __forceinline__ uint32_t warp_offsets(uint32_t mine, uint32_t* s_warp, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0) s_warp[warp] = mine;
  __syncthreads();
  uint32_t v = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += y;
  }
  *total = __shfl_sync(0xFFFFFFFFu, v, 31);
  return __shfl_sync(0xFFFFFFFFu, v, warp) - mine;
}
static_assert(kSelectWarps == 32, "one lane per warp in the scan");

__global__ void __launch_bounds__(kSelectThreads, 1) evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ uint32_t hist[2048], s_warp[kSelectWarps], s_bin[2];
  const int layer = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float* w = p.weights + layer * p.weight_stride;
  const int64_t n = p.n, keep = p.keep, lo = p.first, hi = p.n - p.last;      // lo .. hi - 1 compete
  int32_t* kept = p.kept + layer * keep;
  int32_t* slots = p.slot_table + ((int64_t)p.req * p.n_layers + layer) * p.ctx_cap;
  int32_t* new_slot = p.new_slot + layer * keep;
  int32_t* holes = p.holes + layer * keep;
  uint32_t* used = p.used + layer * p.used_words;
  int2* moves = p.moves + layer * keep;
  grid_dependency_wait();

  // ---- the need-th largest key T, and how many tokens at T stay
  const int64_t need = keep - p.first - p.last;
  uint32_t T = 0, left = (uint32_t)need;
  if (need > 0) {
    uint32_t mask = 0;
#pragma unroll
    for (int d = 0; d < 3; ++d) {
      const int shift = d == 0 ? 21 : (d == 1 ? 10 : 0), bits = d == 2 ? 10 : 11;
      for (int i = tid; i < 2048; i += kSelectThreads) hist[i] = 0;
      __syncthreads();
      for (int64_t t = lo + tid; t < hi; t += kSelectThreads) {
        const uint32_t k = weight_key(w[t]);
        if ((k & mask) == T) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
      }
      __syncthreads();
      // bins from the top: thread i has the bins 2047 - 2 i and 2046 - 2 i
      const uint32_t a = hist[2047 - 2 * tid], b = hist[2046 - 2 * tid];
      uint32_t v = a + b;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += y;
      }
      uint32_t total;
      const uint32_t before = warp_offsets(__shfl_sync(0xFFFFFFFFu, v, 31), s_warp, &total) + v - a - b;
      if (before < left && left <= before + a + b) {
        const bool first = left <= before + a;
        s_bin[0] = first ? 2047 - 2 * tid : 2046 - 2 * tid;
        s_bin[1] = left - before - (first ? 0 : a);
      }
      __syncthreads();
      T |= s_bin[0] << shift;
      left = s_bin[1];
      mask |= ((1u << bits) - 1u) << shift;
      __syncthreads();
    }
  }

  // ---- kept positions, ascending: a warp owns a run of tokens
  const int64_t run = ((n + kSelectWarps - 1) / kSelectWarps + 31) / 32 * 32;
  const int64_t t0 = warp * run < n ? warp * run : n, t1 = t0 + run < n ? t0 + run : n;
  auto look = [&](int64_t t, uint32_t* more, uint32_t* same) {
    const bool there = t < t1, mid = there && t >= lo && t < hi;
    const uint32_t k = mid ? weight_key(w[t]) : 0u;
    *more = __ballot_sync(0xFFFFFFFFu, there && (!mid || (need > 0 && k > T)));
    *same = __ballot_sync(0xFFFFFFFFu, mid && need > 0 && k == T);
  };
  uint32_t more, same, n_more = 0, n_same = 0, total;
  for (int64_t t = t0; t < t1; t += 32) {
    look(t + lane, &more, &same);
    n_more += __popc(more);
    n_same += __popc(same);
  }
  uint32_t b_more = warp_offsets(n_more, s_warp, &total), b_same = warp_offsets(n_same, s_warp, &total);
  for (int64_t t = t0; t < t1; t += 32) {
    look(t + lane, &more, &same);
    const uint32_t below = (1u << lane) - 1u, bit = 1u << lane;
    const uint32_t rank = b_same + __popc(same & below);
    if ((more & bit) || ((same & bit) && rank < left))
      kept[b_more + __popc(more & below) + (rank < left ? rank : left)] = (int32_t)(t + lane);
    b_more += __popc(more);
    b_same += __popc(same);
  }
  for (int64_t i = tid; i < p.used_words; i += kSelectThreads) used[i] = 0;
  __syncthreads();

  // ---- rows: those below `keep` that stay in use, then the free ones among them
  const int64_t base = p.row_base + layer * p.layer_rows;
  auto moves_away = [&](int32_t slot) { return slot >= base + keep && slot < base + p.layer_rows; };
  for (int64_t i = tid; i < keep; i += kSelectThreads) {
    const int32_t slot = slots[kept[i]];
    if (slot < 0 || (int64_t)slot >= p.pool_rows) report_error(p.err, QSA_ERR_BAD_SLOT, kKernEvict, kept[i]);
    new_slot[i] = slot;
    const int64_t row = slot - base;
    if (row >= 0 && row < keep) atomicOr(used + (row >> 5), 1u << (row & 31));
  }
  __syncthreads();
  const int64_t run2 = ((keep + kSelectWarps - 1) / kSelectWarps + 31) / 32 * 32;
  const int64_t k0 = warp * run2 < keep ? warp * run2 : keep, k1 = k0 + run2 < keep ? k0 + run2 : keep;
  uint32_t n_free = 0, n_away = 0;
  for (int64_t i = k0; i < k1; i += 32) {
    const bool there = i + lane < k1;
    n_free += __popc(__ballot_sync(0xFFFFFFFFu, there && !((used[i >> 5] >> lane) & 1u)));
    n_away += __popc(__ballot_sync(0xFFFFFFFFu, there && moves_away(new_slot[i + lane])));
  }
  uint32_t b_free = warp_offsets(n_free, s_warp, &total), b_away = warp_offsets(n_away, s_warp, &total);
  const uint32_t below = (1u << lane) - 1u;
  for (int64_t i = k0; i < k1; i += 32) {
    const bool free_row = i + lane < k1 && !((used[i >> 5] >> lane) & 1u);
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, free_row);
    if (free_row) holes[b_free + __popc(m & below)] = (int32_t)(i + lane);
    b_free += __popc(m);
  }
  __syncthreads();
  // (there are no fewer free rows than moving ones: the tokens in rows below
  // `keep` use at most one row each)
  for (int64_t i = k0; i < k1; i += 32) {
    const bool away = i + lane < k1 && moves_away(new_slot[i + lane]);
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, away);
    if (away) {
      const uint32_t r = b_away + __popc(m & below);
      const int32_t to = (int32_t)(base + holes[r]);
      moves[r] = make_int2(new_slot[i + lane], to);
      new_slot[i + lane] = to;
    }
    b_away += __popc(m);
  }
  if (tid == 0) p.n_moves[layer] = (int32_t)total;
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
  cudaError_t e = launch_kernel(evict_select_kernel, dim3(p.n_layers), dim3(kSelectThreads), 0, s, 0, dim3(1), p);
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
