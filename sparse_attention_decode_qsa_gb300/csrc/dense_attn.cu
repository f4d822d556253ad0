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
// A tile is some rows and one list of tokens: the tokens that any of its rows
// sees, cut into shares (of whole steps) where tiles are few.  Tiles of more than
// four queries run on tcgen05 (wide: 64 queries and a KV head per CTA), the others
// on register fragments (few: tokens and dims are the rows of an mma of m16n8k16, four
// KV heads per CTA), since their time is the rows' bytes.  Where the requests of a
// shared prefix have few queries each, the prefix has tiles of its own, over the rows
// of all requests; else every tile reads it in front of its own tokens.  A row's
// pieces are joined by their maxima and sums.
//
// Measured (device time of a call, one behind the other):
//   4096 BF16 queries, window 4096 of 16384 tokens (138 GFLOP): 124 us, 0.58 of the
//     measured bf16 rate over the call, 0.69 while all SMs are at work (256 CTAs on
//     152 SMs are two rounds).  Bound by the hand-overs between softmax and tensor core
//     (issue slots 0.49, tensor pipe 0.55, exponentials 0.28 of the cycles).
//   2 x 1023 FP8 queries over 8191 tokens each (129 GFLOP): 162 us on 128 of 152 SMs;
//     the products with both scales come on top, 2.5 us a step for 1.9.
//   32 requests' tokens, window 4096, FP8 rows (137 MB): 36.9 us, the kernel 34.2 at 4.0
//     TB/s; issue slots 0.51, most of them conversions and addresses, no pipe full.
//   one token, window 1024: 7.2 us, the latency of two launches.
//   64 tokens behind a prefix of 16384, 0.4 K own tokens each (89 MB): 40 us: 19 for the
//     prefix on 128 SMs (four steps a share: 1.9 us each and 10 of set-up, pieces and
//     launch), then 16 for the own tokens, and a join of 35 pieces a row.
//   29 FP8 draft tokens behind 65536 (69 MB): 61 us, 14 steps of 3.3 us a share.
// Not faster: the SMs shared out to prefix and own tokens by their rows (10 us more);
// FP8 codes copied and turned over in place (170 -> 198 us); both halves of a CTA on
// every other step of a small tile (57 -> 76, BF16 44 -> 59); the idle half's warps for
// V (57 -> 60).
//
// Rounding: P to bf16 beside BF16 rows (2^-8 of each term at most; the tensor core
// takes no wider type beside them); beside FP8 rows P times the V scale as f16, 2^-11
// of itself, or 2^-25 in units in which the largest of the row's products is 2^-6 at
// least (the reference follows the row's own products); the output once to bf16.  S, O,
// maxima and sums are fp32, the sums taken from the unrounded probabilities.
#include "dense_common.cuh"

namespace qsa {
namespace {

using namespace tc;
using namespace attn;

constexpr int kTileQueries = 64;                  // wide: two halves of 32
constexpr int kStepTokens = 128;                  // wide
constexpr int kFewStep = 32;                      // few: two halves of 16 tokens
constexpr int kRowFloats = kHeadDim + 4;          // partial of a row and head: O, m, l (16-byte aligned)
constexpr int kMaxShares = 64;                    // of a tile

struct DenseParams {
  DenseAttn d;
  int32_t tile0[kMaxUnits + 1];  // prefix sums of the wide tiles per unit
  int32_t part0[kMaxUnits + 1];  // of the own partial rows per unit: its rows times its most pieces, 0 where every row is written at once
  int32_t join0[kMaxUnits + 1];  // of the rows per unit that have partials
  int32_t grouped;               // 1: the prefix has tiles of its own
  int32_t prefix_pieces;         // of every row, in front of its own ones (0 where not grouped)
  int32_t wide_q, few_q;         // steps of a share
  const uint16_t* q;             // [rows][16][128] bf16 bits
  float scale_log2;              // |softmax_scale| * log2(e)
  float sign;
  uint16_t* out;                 // [rows][16][128] bf16 bits
  float* lse;                    // [rows][16] or nullptr
  float* part;                   // prefix [pieces][rows], then per unit [pieces][its rows], each [16][kRowFloats]
};

// Rows x0 .. x0 + nq - 1 (consecutive positions from pos0 on, where they have own
// tokens) over np tokens of the prefix, the tokens 0 .. na - 1 and b0 .. b0 + nb - 1
// of unit u, in this order.  (Two contexts of fewer than 2^31 tokens each.)
struct Tile {
  int u, x0, nq;
  int32_t pos0;
  uint32_t np, na, b0, total;
};

__host__ __device__ __forceinline__ void own_part(const DenseAttn& d, int64_t p0, int64_t p1, Tile* t) {
  int64_t na, b0, nb;
  own_range(d, p0, p1, &na, &b0, &nb);
  t->na = (uint32_t)na;
  t->b0 = (uint32_t)b0;
  t->total = t->np + (uint32_t)(na + nb);
}

// Own tile of rows i0 .. of unit u.
__host__ __device__ __forceinline__ Tile own_tile(const DenseAttn& d, bool grouped, int u, int i0) {
  Tile t;
  const int left = d.c.unit_tokens(u) - i0;
  t.u = u;
  t.x0 = d.c.row0[u] + i0;
  t.nq = left < kTileQueries ? left : kTileQueries;
  t.pos0 = (int32_t)d.c.position(u, t.x0);
  t.np = grouped ? 0u : (uint32_t)d.prefix_len;
  own_part(d, t.pos0, t.pos0 + t.nq - 1, &t);
  return t;
}

// Tile of the prefix for rows i0 .. of layer l.
__host__ __device__ __forceinline__ Tile prefix_tile(const DenseAttn& d, int l, int i0) {
  Tile t;
  const int layer_rows = d.c.row0[d.n_req];
  t.u = l * d.n_req;
  t.x0 = l * layer_rows + i0;
  t.nq = layer_rows - i0 < kTileQueries ? layer_rows - i0 : kTileQueries;
  t.np = t.total = (uint32_t)d.prefix_len;
  t.pos0 = 0;
  t.na = t.b0 = 0;
  return t;
}

// Shares of a tile: one at least where nothing else writes its rows.  
__host__ __device__ __forceinline__ int shares_of(const Tile& t, int step, int q, bool alone) {
  const uint32_t steps = t.total / step + (t.total % step != 0);
  if (steps == 0) return alone ? 1 : 0;
  return (int)((steps + (uint32_t)q - 1) / (uint32_t)q);
}
// First step of share i of n.
__device__ __forceinline__ uint32_t share_start(uint32_t steps, uint32_t i, uint32_t n) {
  return steps / n * i + steps % n * i / n;          // (n <= kMaxShares: no product leaves 32 bits)
}

// Own pieces of row x of unit u.
__device__ __forceinline__ int own_pieces(const DenseParams& p, int u, int x) {
  const bool few = p.d.c.unit_tokens(u) <= kFewQueries;
  const int i0 = few ? 0 : (x - p.d.c.row0[u]) / kTileQueries * kTileQueries;
  return shares_of(own_tile(p.d, p.grouped, u, i0), few ? kFewStep : kStepTokens, few ? p.few_q : p.wide_q, !p.grouped);
}

// Row x of unit u and head h in piece i of the prefix, or of its own tokens.
__device__ __forceinline__ float* piece_ptr(const DenseParams& p, bool prefix, int u, int i, int x, int h) {
  const int64_t rows = p.d.c.rows();
  const int64_t row = prefix ? i * rows + x
                             : p.prefix_pieces * rows + p.part0[u] + (int64_t)i * p.d.c.unit_tokens(u) + x - p.d.c.row0[u];
  return p.part + (row * kQHeads + h) * kRowFloats;
}

// Where the tokens of a tile lie: slots and host rows of the prefix and of unit u.
struct Source {
  const int32_t* slots;          // own
  const int32_t* prefix_slots;
  const uint8_t* host;
  const uint8_t* prefix_host;
};
__device__ __forceinline__ Source source_of(const DenseAttn& d, int u) {
  const BatchDesc& b = d.c.b;
  const int layer = b.u[u].layer;
  Source s;
  s.slots = b.slot_table + b.unit_row(u);
  s.prefix_slots = b.slot_table + ((int64_t)d.prefix_req * b.n_layers + layer) * b.ctx_cap;
  s.host = b.u[u].host_rows;
  s.prefix_host = d.prefix_host ? d.prefix_host + (int64_t)layer * d.prefix_stride * b.row_bytes : nullptr;
  return s;
}
// The slot of the i-th token of the tile's list; -2 past its end.
__device__ __forceinline__ int32_t slot_at(const Source& s, const Tile& t, uint32_t i) {
  if (i >= t.total) return -2;
  if (i < t.np) return s.prefix_slots[i];
  const uint32_t own = i - t.np;
  return s.slots[own < t.na ? own : t.b0 + own - t.na];
}
// The row behind that slot; nullptr past the end, and (reported) for a bad slot.
__device__ __forceinline__ const uint8_t* row_at(const BatchDesc& b, const Source& s, const Tile& t, uint32_t i,
                                                 int32_t slot) {
  if (slot >= 0 && (int64_t)slot < b.pool_rows) return b.pool + (int64_t)slot * b.row_bytes;
  if (i >= t.total) return nullptr;
  const bool pre = i < t.np;
  const uint32_t own = i - t.np;
  const int64_t tok = pre ? i : (own < t.na ? own : t.b0 + own - t.na);
  const uint8_t* host = pre ? s.prefix_host : s.host;
  if (slot == -1 && host) return host + tok * b.row_bytes;
  report_error(b.err, QSA_ERR_BAD_SLOT, kKernDenseAttn, ((int64_t)t.u << 40) | (tok & 0xFFFFFFFFFFll));
  return nullptr;
}

// One warp, one query row x of unit u and head h: online softmax over the row's
// own tokens, plain fp32, four at a time.  For rows that the tiles cannot compute: 0
// times a value that is not finite is not 0, so that a token which a row does not see
// may have reached it.  Slow, for such values only.
__device__ __noinline__ void attend_row(const DenseParams& p, int u, int x, int h) {
  const int lane = threadIdx.x & 31, g = h / kGroup;
  const BatchDesc& b = p.d.c.b;
  const bool fp8 = b.row_bytes == kRowBytesFp8;
  const float f = p.sign * p.scale_log2;
  const uint2 qv = reinterpret_cast<const uint2*>(p.q + ((int64_t)x * kQHeads + h) * kHeadDim)[lane];
  const float q[4] = {bf16_lo(qv.x) * f, bf16_hi(qv.x) * f, bf16_lo(qv.y) * f, bf16_hi(qv.y) * f};
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  Tile t;
  t.u = u;
  t.np = (uint32_t)p.d.prefix_len;
  const int64_t pos = p.d.c.position(u, x);
  own_part(p.d, pos, pos, &t);
  const Source src = source_of(p.d, u);
  constexpr int kTurn = 4;
  for (uint32_t i = 0; i < t.total; i += kTurn) {
    const uint8_t* row[kTurn];
    float4 k[kTurn], v[kTurn];
    float s[kTurn];
#pragma unroll
    for (int j = 0; j < kTurn; ++j) row[j] = row_at(b, src, t, i + j, slot_at(src, t, i + j));
#pragma unroll
    for (int j = 0; j < kTurn; ++j) {
      k[j] = v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!row[j]) continue;
      k[j] = row_values(row[j], g, lane, fp8);
      v[j] = row_values(row[j], kKvHeads + g, lane, fp8);
    }
#pragma unroll
    for (int j = 0; j < kTurn; ++j) s[j] = fmaf(q[3], k[j].w, fmaf(q[2], k[j].z, fmaf(q[1], k[j].y, q[0] * k[j].x)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int j = 0; j < kTurn; ++j) s[j] += __shfl_xor_sync(0xFFFFFFFFu, s[j], o);
    float mn = m;
#pragma unroll
    for (int j = 0; j < kTurn; ++j) {
      if (!row[j]) s[j] = -INFINITY;
      mn = fmaxf(mn, s[j]);
    }
    const float a = mn == -INFINITY ? 1.f : exp2f(m - mn);
    m = mn;
    l *= a;
    acc = make_float4(acc.x * a, acc.y * a, acc.z * a, acc.w * a);
#pragma unroll
    for (int j = 0; j < kTurn; ++j) {
      if (!row[j]) continue;
      const float e = s[j] == -INFINITY ? 0.f : exp2f(s[j] - mn);
      l += e;
      acc = make_float4(fmaf(e, v[j].x, acc.x), fmaf(e, v[j].y, acc.y), fmaf(e, v[j].z, acc.z), fmaf(e, v[j].w, acc.w));
    }
  }
  const float r = l == 0.f ? 0.f : 1.f / l;      // no tokens: zeros; NaN stays
  reinterpret_cast<uint2*>(p.out + ((int64_t)x * kQHeads + h) * kHeadDim)[lane] =
      make_uint2(pack_bf16(acc.x * r, acc.y * r), pack_bf16(acc.z * r, acc.w * r));
  if (p.lse && lane == 0) p.lse[(int64_t)x * kQHeads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Sums of probabilities, and outputs, that hold: anything else is computed again.
__device__ __forceinline__ bool good_sum(float l) { return l > 0x1p-100f && l < 0x1p125f; }     // false for NaN

// ------------------------------------------------------------------- few

// One CTA: a share of a tile of at most 2 kN queries, all KV heads.  Warp w serves
// KV head w % 4 for the tokens 16 (w / 4) .. + 15 of every step of 32, copied by
// itself into its own ring of three stages (cp.async, K[g] and V[g] alone, 16-byte
// chunks at chunk ^ (row % 8)), so that no barrier is needed while streaming.  Per
// stage S^T = K Q^T and O^T += V^T P^T by mma of m16n8k16, 8 each per 8 columns
// (query * 4 + head): with tokens and dims as the 16 rows, one or two queries fill
// half of what four do, in registers and instructions, and with FP8 rows two CTAs
// share an SM.  P changes sides by a transposing move, V's fragments come by transposing loads; the
// online softmax is in the accumulators' registers.  FP8 codes become f16 on the way
// into registers, exactly: a K word of four codes serves as the dims that the
// fragment asks for, with Q's dims in the same order; V words, transposed as pairs
// of dims, are split into the even dims (the rows 0 .. 7 of a fragment) and the odd.
constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32, kFewStages = 3;
constexpr int kFewTokens = 16;                    // of a warp and step
template <bool kFp8>
struct FewLayout {
  static constexpr int kVec = kFp8 ? 128 : 256;                  // bytes of a head vector
  static constexpr int kV = kFewTokens * kVec;                   // V behind K
  static constexpr int kScales = 2 * kV;                         // FP8: the rows' 8 scales, 16 bytes a token
  static constexpr int kStage = kScales + (kFp8 ? kFewTokens * 16 : 0);
  static constexpr int kSmem = kFewWarps * kFewStages * kStage;
};
static_assert(FewLayout<true>::kSmem >= kKvHeads * 16 * kRowFloats * 4, "room for the halves to come together");

template <bool kFp8, int kN>
__global__ void __launch_bounds__(kFewThreads, kFp8 && kN == 1 ? 2 : 1) dense_few_kernel(const __grid_constant__ DenseParams p) {
  using L = FewLayout<kFp8>;
  constexpr int kStages = kFewStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t there[kFewWarps][kFewStages];                       // tokens of a stage whose row exists
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = warp & 3, half = warp >> 2;
  const BatchDesc& b = p.d.c.b;
  const int r = lane >> 2, j4 = lane & 3;                        // rows r and r + 8, columns 8 n + 2 j4 + e

  // grid: shares x (units, then the prefix at every layer)
  Tile t;
  const bool pre = (int)blockIdx.y >= b.n_units;
  if (pre) {
    t = prefix_tile(p.d, blockIdx.y - b.n_units, 0);
  } else {
    t = own_tile(p.d, p.grouped, blockIdx.y, 0);
  }
  const bool some = pre || (t.nq > 0 && p.d.c.unit_tokens(t.u) <= kFewQueries);
  const int shares = some ? shares_of(t, kFewStep, p.few_q, !p.grouped) : 0;
  // (before any CTA leaves: where all of them do, what follows still follows the kernel before)
  grid_dependency_wait();
  if ((int)blockIdx.x >= shares) return;
  const uint32_t all = t.total / kFewStep + (t.total % kFewStep != 0);
  const uint32_t s0 = share_start(all, blockIdx.x, shares);
  const int steps = (int)(share_start(all, blockIdx.x + 1, shares) - s0);
  const Source src = source_of(p.d, t.u);

  const uint32_t ring = smem_u32(smem) + warp * kStages * L::kStage;
  const uint32_t first = s0 * kFewStep + half * kFewTokens;      // the warp's first token in the tile's list
  // lane l < 16: token l of a stage
  auto slot_of = [&](int s) {
    return lane < kFewTokens && s < steps ? slot_at(src, t, first + s * kFewStep + lane) : -2;
  };
  auto issue = [&](int s, int32_t slot) {
    const uint8_t* row = nullptr;
    if (lane < kFewTokens && s < steps) row = row_at(b, src, t, first + s * kFewStep + lane, slot);
    const uint32_t have = __ballot_sync(0xFFFFFFFFu, row != nullptr);
    if (lane == 0) there[warp][s % kStages] = have;
    const uint32_t to = ring + (s % kStages) * L::kStage;
    // a lane's 16 bytes of K[g] or V[g]: BF16 a token, FP8 two tokens a turn
    constexpr int kPer = kFp8 ? 2 : 1, kLanes = L::kVec / 16;
    const int c = lane % kLanes, v = (lane / kLanes) & 1;
    const uint32_t off = (v ? kKvHeads + g : g) * L::kVec + c * 16;
    few_copies<kPer>(b, row, slot, [&](int k, const uint8_t* from) {
      cp_async16(to + v * L::kV + k * L::kVec + ((c ^ (k & 7)) << 4), from + off, (have >> k) & 1u ? 16u : 0u);
    });
    if (kFp8 && lane < kFewTokens)
      cp_async16(to + L::kScales + lane * 16, (row ? row : b.pool) + 2 * kKvHeads * kHeadDim, row ? 16u : 0u);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int32_t slot_next;
  {
    int32_t a[kStages - 1];
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) a[i] = slot_of(i);
    slot_next = slot_of(kStages - 1);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i, a[i]);
  }
  uint32_t qb[kN][8][2];
  float f[kN][2];
  few_queries<kFp8, kN>(p.q, t.x0, t.nq, g, p.sign * p.scale_log2, qb, f);

  float o[8][kN][4];             // rows of tile i: dims 16 i + r, + 8; FP8: 16 i + 2 r, + 1
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int n = 0; n < kN; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
  float m[kN][2], l[kN][2];      // of the lane's columns, in units of log2; l over its own rows
#pragma unroll
  for (int n = 0; n < kN; ++n) m[n][0] = m[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.f;

  // the newest position that the last query's window leaves out
  const int64_t gone = (int64_t)t.pos0 + t.nq - 1 - p.d.window;
  const int32_t newest = gone < -1 ? -1 : (int32_t)gone;
#pragma unroll 1
  for (int s = 0; s < steps; ++s) {
    const int32_t slot = slot_next;
    slot_next = slot_of(s + kStages);
    issue(s + kStages - 1, slot);                                // its stage was last read at s - 1
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    const uint32_t st = ring + (s % kStages) * L::kStage;
    const uint32_t have = there[warp][s % kStages];
    // ---- S^T = K Q^T: tokens r (elements 0, 1) and r + 8 (2, 3)
    float x[kN][4];
#pragma unroll
    for (int n = 0; n < kN; ++n) x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t ka[4];
      few_keys<kFp8>(st, k, ka);
#pragma unroll
      for (int n = 0; n < kN; ++n) mma16<kFp8>(x[n], ka, qb[n][k][0], qb[n][k][1]);
    }
    float ks[2] = {1.f, 1.f}, vs[2] = {1.f, 1.f}, lv[2] = {0.f, 0.f};        // FP8: scales of tokens r, r + 8
    if (kFp8) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint16_t* sc = reinterpret_cast<const uint16_t*>(smem + (st - smem_u32(smem)) + L::kScales + (r + 8 * i) * 16);
        ks[i] = key_scale_of(sc[g]);
        vs[i] = __half2float(__ushort_as_half(sc[kKvHeads + g]));
        lv[i] = log2_size(vs[i]);
      }
    }
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[n][e] *= kFp8 ? ks[e >> 1] * f[n][e & 1] : f[n][e & 1];
    // ---- tokens without a row, and tokens that a query does not see
    const uint32_t i0 = first + s * kFewStep, front = t.np + t.na;            // (front: seen by every query)
    const int32_t t0 = (int32_t)(t.b0 + i0 - front);             // the first token's position, if it is one of b
    const bool free_of = have == 0xFFFFu && (i0 + kFewTokens <= front ||
                                             (i0 >= front && t0 + kFewTokens - 1 <= t.pos0 && t0 > newest));
    if (!free_of) {
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = r + 8 * (e >> 1);
          const int64_t pos = (int64_t)t.pos0 + 2 * n + ((2 * j4 + (e & 1)) >> 2), tok = (int64_t)t.b0 + i0 + c - front;
          const bool seen = i0 + c < front || (tok <= pos && (tok < p.d.sinks || tok > pos - p.d.window));
          if (!seen || !((have >> c) & 1u)) x[n][e] = -INFINITY;
        }
    }
    // ---- online softmax; the reference follows the largest product of a
    // probability and its V scale (FP8: it has to fit f16)
    float mx[kN][2];
    bool up = false;
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y = fmaxf(x[n][e] + lv[0], x[n][2 + e] + lv[1]);
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, k));
        mx[n][e] = y;
        up = up || y > m[n][e];
      }
    if (__any_sync(0xFFFFFFFFu, up)) {
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mn = fmaxf(m[n][e], mx[n][e]), a = mn == -INFINITY ? 1.f : exp2_fast(m[n][e] - mn);
          m[n][e] = mn;
          l[n][e] *= a;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[i][n][e] *= a;
            o[i][n][2 + e] *= a;
          }
        }
    }
    uint32_t pb[kN][2];                                          // P^T as B fragments
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      float e[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) e[k] = exp2_fast(x[n][k] - (m[n][k & 1] == -INFINITY ? 0.f : m[n][k & 1]));
      l[n][0] += e[0] + e[2];
      l[n][1] += e[1] + e[3];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        pb[n][i] = transpose8x8(kFp8 ? pack_f16(e[2 * i] * vs[i], e[2 * i + 1] * vs[i]) : pack_bf16(e[2 * i], e[2 * i + 1]));
    }
    // ---- O^T += V^T P^T, two chunks of 8 dims (FP8: of 16) per load
    const int tok = lane & 15;                                   // of the transposing loads: rows, then rows + 8
#pragma unroll
    for (int i = 0; i < 8; i += kFp8 ? 2 : 1) {
      uint32_t v[4];
      const int c = kFp8 ? i + (lane >> 4) : 2 * i + (lane >> 4);
      ldsm4_t(st + L::kV + tok * L::kVec + ((c ^ (tok & 7)) << 4), v);
      if (!kFp8) {
        const uint32_t va[4] = {v[0], v[2], v[1], v[3]};
#pragma unroll
        for (int n = 0; n < kN; ++n) mma16<false>(o[i][n], va, pb[n][0], pb[n][1]);
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t va[4];                                        // even dims, odd dims; then tokens + 8
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint2 a = codes4_f16(v[2 * k + h]);
            va[2 * h] = __byte_perm(a.x, a.y, 0x5410);
            va[2 * h + 1] = __byte_perm(a.x, a.y, 0x7632);
          }
#pragma unroll
          for (int n = 0; n < kN; ++n) mma16<true>(o[i + k][n], va, pb[n][0], pb[n][1]);
        }
      }
    }
    __syncwarp();                                                // the stage is refilled in the next turn
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], k);

  // ---- the two halves of a KV head come together, rows [column][dims, m, l]
  __syncthreads();
  float* rows = reinterpret_cast<float*>(smem) + g * 16 * kRowFloats;
  auto each = [&](auto&& fn) {                                   // fn(place, value of the lane's accumulators)
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          fn(rows + (8 * n + 2 * j4 + (e & 1)) * kRowFloats + 16 * i + (kFp8 ? 2 * r + (e >> 1) : r + 8 * (e >> 1)), o[i][n][e],
             n, e & 1);
  };
  if (half == 1) {
    each([&](float* at, float v, int, int) { *at = v; });
    if (r == 0) {
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float2*>(rows + (8 * n + 2 * j4 + e) * kRowFloats + kHeadDim) = make_float2(m[n][e], l[n][e]);
    }
  }
  __syncthreads();
  if (half == 1) return;
  float fa[kN][2], fb[kN][2];
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float* at = rows + (8 * n + 2 * j4 + e) * kRowFloats + kHeadDim;
      const float2 ml = *reinterpret_cast<const float2*>(at);
      const float mn = fmaxf(m[n][e], ml.x);
      fa[n][e] = m[n][e] == -INFINITY ? 0.f : exp2_fast(m[n][e] - mn);
      fb[n][e] = ml.x == -INFINITY ? 0.f : exp2_fast(ml.x - mn);
      __syncwarp();
      if (r == 0) *reinterpret_cast<float2*>(at) = make_float2(mn, fmaf(l[n][e], fa[n][e], ml.y * fb[n][e]));
    }
  each([&](float* at, float v, int n, int e) { *at = fmaf(v, fa[n][e], *at * fb[n][e]); });
  __syncwarp();
  // a row at a time, lane l with dims 4 l .. 4 l + 3
  for (int c = 0; c < kGroup * t.nq; ++c) {
    const int x = t.x0 + (c >> 2), h = g * kGroup + (c & 3);
    const float* at = rows + c * kRowFloats;
    const float2 lo = *reinterpret_cast<const float2*>(at + 4 * lane), hi = *reinterpret_cast<const float2*>(at + 4 * lane + 2);
    const float2 ml = *reinterpret_cast<const float2*>(at + kHeadDim);
    if (shares > 1 || p.grouped) {
      float* to = piece_ptr(p, pre, t.u, blockIdx.x, x, h);
      *reinterpret_cast<float4*>(to + 4 * lane) = make_float4(lo.x, lo.y, hi.x, hi.y);
      if (lane == 0) *reinterpret_cast<float2*>(to + kHeadDim) = ml;
      continue;
    }
    const bool fine = good_sum(ml.y) && isfinite(lo.x) && isfinite(lo.y) && isfinite(hi.x) && isfinite(hi.y);
    if (!__all_sync(0xFFFFFFFFu, fine)) {
      attend_row(p, t.u, x, h);
      continue;
    }
    const float inv = 1.f / ml.y;
    reinterpret_cast<uint2*>(p.out + ((int64_t)x * kQHeads + h) * kHeadDim)[lane] =
        make_uint2(pack_bf16(lo.x * inv, lo.y * inv), pack_bf16(hi.x * inv, hi.y * inv));
    if (lane == 0 && p.lse) p.lse[(int64_t)x * kQHeads + h] = (ml.x + log2f(ml.y)) * kLn2;
  }
}

// ------------------------------------------------------------------- wide

// One CTA: a share of a tile of up to 64 queries and one KV head.  The tile's 64
// queries x 4 heads of the group are 256 rows, two halves of 128 = the tensor
// core's M: row = head * 32 + query, so a warp is a head and a lane a query.  Per
// half and 64 tokens: S = Q K^T (8 MMAs of K = 16, both operands in shared memory
// under the 128-byte swizzle), softmax by the half's 4 warps (thread = row), P over
// S's own columns of tensor memory, O += P V (4 MMAs, P from tensor memory, V as an
// MN-major operand, so that rows lie in shared memory as they come).  Each half has
// two S tiles in turn: while one is in softmax, the other's P V and next S run.
// Warps: 8 softmax, 4 loaders (cp.async of K[g], V[g] of each row, two stages of
// 128 tokens; FP8 codes are turned into f16 on the way, exactly, their scales going
// to the logits and the probabilities), 2 MMA (one per half).  All waits are
// bounded.  Masks are three ranges of positions per row, so 64 tokens' mask is a
// few shifts, and most steps need none.
constexpr int kSubTokens = kStepTokens / 2;       // tokens of one S tile
constexpr int kSoftWarps = 8, kLoadWarps = 4;
constexpr int kMmaWarps = 2;                      // one per half
constexpr int kWideThreads = 32 * (kSoftWarps + kLoadWarps + kMmaWarps);     // 448
constexpr int kRoleLoad = kSoftWarps, kRoleMma = kSoftWarps + kLoadWarps;
constexpr int kStages = 2;
constexpr int kPanel = 128 * 128;                 // 128 rows of 64 16-bit elements
constexpr int kQBytes = 2 * 2 * kPanel;           // two halves, two panels of 64 dims
constexpr int kKvBytes = 2 * kPanel;              // K (or V) of a stage: two panels
constexpr int kStageBytes = 2 * kKvBytes;

// What the softmax of a step needs beside S.
struct StepMeta {
  uint32_t valid[4];            // bit per token of the step: its row exists
  int32_t special[4];           // per loader warp: a row is missing, or not every query sees every token
  uint32_t exps[4];             // FP8, per loader warp: bit e, a row has a V scale with the f16 exponent field e
  uint32_t pad[4];
};
struct __align__(16) Scales {   // FP8 rows
  float k[kStepTokens];         // K scale (times softmax scale and log2 e)
  float v[kStepTokens];         // V scale
  float size[kStepTokens];      // log2 of its size
};
constexpr int kOffKv = kQBytes;
constexpr int kOffMeta = kOffKv + kStages * kStageBytes;
// Metas outlive their K stage (the softmax of step j reads meta j while K of
// step j + 2 comes in), but not by three steps: K of step j + 3 comes after the
// S of step j + 1, that after the P of step j.
constexpr int kMetas = 4;
constexpr int kOffScales = kOffMeta + kMetas * (int)sizeof(StepMeta);
constexpr int kOffBar = kOffScales + kMetas * (int)sizeof(Scales);
// k_full[2], k_empty[2], v_full[2], v_empty[2], then per (half, 64 tokens)
// s_full[4], p_full[4], o_full[4], then q_full, done[2]
constexpr int kNumBars = 4 * kStages + 15;
constexpr int kOffSlot = (kOffBar + 8 * kNumBars + 15) / 16 * 16;
constexpr int kWideSmem = kOffSlot + 16 + 1024;
static_assert(kWideSmem <= 227 * 1024 && sizeof(StepMeta) % 16 == 0, "one CTA's shared memory");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColS = 256;        // + 128 per half

// The lowest k bits.
__device__ __forceinline__ uint64_t low_bits(int64_t k) {
  return k <= 0 ? 0ull : (k >= 64 ? ~0ull : (1ull << k) - 1ull);
}
// Which of the 64 tokens from the i0-th of the tile's list on a query at position
// pos sees (rows that exist or not).
__device__ __forceinline__ uint64_t seen_bits(const DenseAttn& d, const Tile& t, int64_t i0, int64_t pos) {
  const int64_t off = (int64_t)t.np + t.na - i0;               // the first token of the b range
  const int64_t at = off - t.b0;                               // bit of position 0
  const uint64_t in_window = low_bits(pos + 1 + at) & ~low_bits(pos - d.window + 1 + at);
  const uint64_t sinks = low_bits((d.sinks < pos + 1 ? d.sinks : pos + 1) + at);
  return low_bits(off) | in_window | sinks;
}

// FP8: the largest logit + log2 (V scale) of a row's tokens among 64, each by its
// own scale.  S is read from tensor memory for this alone: among the registers of
// the usual path the scales would spill.
__device__ __forceinline__ float wide_max(uint32_t colS, const Scales& sc, int c, uint64_t seen, float f) {
  float most = -INFINITY;
#pragma unroll 1
  for (int b0 = 0; b0 < kSubTokens / 4; b0 += 4) {
    uint32_t x[16];
    ld16(colS + 4u * (uint32_t)b0, x);
    wait_ld();
    reg_fence(x);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int t = kSubTokens * c + 4 * (b0 + b);
      const float4 k = *reinterpret_cast<const float4*>(&sc.k[t]), s = *reinterpret_cast<const float4*>(&sc.size[t]);
      float y[4] = {fmaf(__uint_as_float(x[4 * b]) * k.x, f, s.x), fmaf(__uint_as_float(x[4 * b + 1]) * k.y, f, s.y),
                    fmaf(__uint_as_float(x[4 * b + 2]) * k.z, f, s.z), fmaf(__uint_as_float(x[4 * b + 3]) * k.w, f, s.w)};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!((seen >> (4 * (b0 + b) + i)) & 1u)) y[i] = -INFINITY;
      most = fmaxf(most, fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])));
    }
  }
  return most;
}

template <bool kFp8>
__global__ void __launch_bounds__(kWideThreads, 1) dense_wide_kernel(const __grid_constant__ DenseParams p) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  StepMeta* meta = reinterpret_cast<StepMeta*>(smem + kOffMeta);
  Scales* scales = reinterpret_cast<Scales*>(smem + kOffScales);
  const uint32_t bars = sb + kOffBar;
  auto k_full = [&](int i) { return bars + 8u * (uint32_t)i; };
  auto k_empty = [&](int i) { return bars + 8u * (uint32_t)(kStages + i); };
  auto v_full = [&](int i) { return bars + 8u * (uint32_t)(2 * kStages + i); };
  auto v_empty = [&](int i) { return bars + 8u * (uint32_t)(3 * kStages + i); };
  auto s_full = [&](int h, int c) { return bars + 8u * (uint32_t)(4 * kStages + 2 * h + c); };
  auto p_full = [&](int h, int c) { return bars + 8u * (uint32_t)(4 * kStages + 4 + 2 * h + c); };
  auto o_full = [&](int h, int c) { return bars + 8u * (uint32_t)(4 * kStages + 8 + 2 * h + c); };
  const uint32_t q_full = bars + 8u * (uint32_t)(4 * kStages + 12);
  auto done = [&](int h) { return bars + 8u * (uint32_t)(4 * kStages + 13 + h); };
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + kOffSlot);
  __shared__ float row_factor[kFp8 ? 256 : 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const BatchDesc& b = p.d.c.b;
  ErrorWord* err = b.err;

  // grid: shares x tiles (own ones, a unit's last first, then the prefix's) x KV heads
  const int g = blockIdx.z;
  const int own_tiles = p.tile0[b.n_units];
  const bool pre = (int)blockIdx.y >= own_tiles;
  Tile t;
  if (pre) {
    const int per = (p.d.c.row0[p.d.n_req] + kTileQueries - 1) / kTileQueries, i = blockIdx.y - own_tiles;
    t = prefix_tile(p.d, i / per, (i % per) * kTileQueries);
  } else {
    int lo = 0, hi = b.n_units - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.tile0[mid] <= (int)blockIdx.y) lo = mid; else hi = mid - 1;
    }
    t = own_tile(p.d, p.grouped, lo, (p.tile0[lo + 1] - 1 - (int)blockIdx.y) * kTileQueries);
  }
  const int shares = shares_of(t, kStepTokens, p.wide_q, !p.grouped);
  if ((int)blockIdx.x >= shares) return;
  grid_dependency_wait();
  const int nq = t.nq, x0 = t.x0;
  const int halves = nq > 32 ? 2 : 1;
  const int64_t pos0 = t.pos0;

  if (warp == kRoleMma) {
    tmem_alloc<kTmemCols>(slot);
    if (lane == 0) {
      for (int i = 0; i < kStages; ++i) {
        mbar_init(k_full(i), 32 * kLoadWarps);
        mbar_init(k_empty(i), (uint32_t)halves);
        mbar_init(v_full(i), 32 * kLoadWarps);
        mbar_init(v_empty(i), (uint32_t)halves);
      }
      for (int i = 0; i < 4; ++i) {
        mbar_init(s_full(i >> 1, i & 1), 2);
        mbar_init(p_full(i >> 1, i & 1), 128);
        mbar_init(o_full(i >> 1, i & 1), 1);
      }
      mbar_init(q_full, 32 * kSoftWarps);
      mbar_init(done(0), 1);
      mbar_init(done(1), 1);
      mbar_fence_init();
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *slot;

  // The softmax warps bring Q in, while the loaders begin on K.
  if (warp < kSoftWarps) {
    // ---- Q: row head * 32 + query of each half, two panels of 64 dims.  Against
    // FP8 rows it goes in as f16, beside the K codes, which f16 holds exactly: a
    // row scaled by the power of two that puts its largest element into [2^14,
    // 2^15), the upper end of f16's range, where f16 holds a bf16 element exactly
    // down to 2^-31 of the largest and to 2^-39 of it below; the inverse goes to
    // the logits (row_factor).
    constexpr int kBatch = 4;                        // loads in flight
    for (int i0 = tid; i0 < halves * 128 * 16; i0 += kBatch * 32 * kSoftWarps) {      // (whole warps)
      uint4 in[kBatch];
#pragma unroll
      for (int b4 = 0; b4 < kBatch; ++b4) {
        const int i = i0 + b4 * 32 * kSoftWarps, c = i & 15, r = (i >> 4) & 127, q = (i >> 11) * 32 + (r & 31);
        in[b4] = make_uint4(0, 0, 0, 0);
        if (q < nq)
          in[b4] = reinterpret_cast<const uint4*>(p.q + ((int64_t)(x0 + q) * kQHeads + g * kGroup + (r >> 5)) * kHeadDim)[c];
      }
#pragma unroll
      for (int b4 = 0; b4 < kBatch; ++b4) {
        const int i = i0 + b4 * 32 * kSoftWarps, c = i & 15, r = (i >> 4) & 127, h = i >> 11;
        uint4 v = in[b4];
        const uint32_t flip = p.sign < 0.f ? 0x80008000u : 0u;
        v.x ^= flip; v.y ^= flip; v.z ^= flip; v.w ^= flip;
        if (kFp8) {
          uint32_t* w[4] = {&v.x, &v.y, &v.z, &v.w};
          float top = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) top = fmaxf(top, fmaxf(fabsf(bf16_lo(*w[k])), fabsf(bf16_hi(*w[k]))));
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));   // the row's 16 lanes
          const RowScale rs = row_scale(top);
#pragma unroll
          for (int k = 0; k < 4; ++k) *w[k] = pack_f16(bf16_lo(*w[k]) * rs.a * rs.b, bf16_hi(*w[k]) * rs.a * rs.b);
          if (c == 0) row_factor[h * 128 + r] = rs.inverse;
        }
        *reinterpret_cast<uint4*>(smem + (h * 2 + (c >> 3)) * kPanel + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
      }
    }
    fence_async_smem();
    mbar_arrive(q_full);
    if (kFp8) asm volatile("bar.sync 1, %0;" ::"n"(32 * kSoftWarps) : "memory");      // row_factor
  }

  const uint32_t all = t.total / kStepTokens + (t.total % kStepTokens != 0);
  const uint32_t j0 = share_start(all, blockIdx.x, shares);
  const int steps = (int)(share_start(all, blockIdx.x + 1, shares) - j0);
  bool ok = true;

  if (warp >= kRoleLoad && warp < kRoleMma) {
    // ---- loaders: warp w brings tokens 32 w .. 32 w + 31 of a step, lane = token
    const int w = warp - kRoleLoad;
    const Source src = source_of(p.d, t.u);
    const uint32_t first = j0 * kStepTokens + 32 * w + lane;
    const int64_t last = pos0 + nq - 1;
    auto slot_of = [&](int j) { return j < steps ? slot_at(src, t, first + j * kStepTokens) : -2; };
    // FP8 rows are loaded into registers, with no copies in flight: rows two
    // steps ahead are on their way from HBM meanwhile
    auto prefetch = [&](int32_t s) {
      if (!kFp8 || s < 0 || (int64_t)s >= b.pool_rows) return;
      const uint8_t* r = b.pool + (int64_t)s * b.row_bytes + g * kHeadDim;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(r));
      asm volatile("prefetch.global.L2 [%0];" ::"l"(r + kKvHeads * kHeadDim));
    };
    // at step j the slot of step j + 2 is fetched
    int32_t slot_now = slot_of(0), slot_next = slot_of(1);
    prefetch(slot_next);
    for (int j = 0; j < steps && ok; ++j) {
      const int st = j % kStages;
      const uint32_t turn = (uint32_t)(j / kStages - 1) & 1u;
      const uint32_t i = first + j * kStepTokens;
      const uint8_t* row = row_at(b, src, t, i, slot_now);
      const int32_t slot_two = slot_of(j + 2);
      if (j >= kStages) ok = mbar_wait_warp(k_empty(st), turn, err, kKernDenseAttn);
      if (!ok) break;
      const uint32_t kdst = kOffKv + st * kStageBytes + 32 * w * 128, vdst = kdst + kKvBytes;
      const uintptr_t from = reinterpret_cast<uintptr_t>(row);
      StepMeta& m = meta[j % kMetas];
      auto write_meta = [&]() {
        const uint32_t there = __ballot_sync(0xFFFFFFFFu, row != nullptr);
        const int64_t tok = (int64_t)t.b0 + i - t.np - t.na; // its position, if it is one of b
        const bool some = i >= t.np + t.na && (tok > pos0 || (tok >= p.d.sinks && tok <= last - p.d.window));
        const bool special = __any_sync(0xFFFFFFFFu, some || row == nullptr);
        if (lane == 0) {
          m.valid[w] = there;
          m.special[w] = special;
        }
      };
      if (!kFp8) {
        // 16 lanes copy the 256 bytes of a token's K[g] (or V[g]); two tokens per turn
        // (row r = 2 i + hi; its swizzle takes one of four values per lane)
        const uint32_t c = lane & 15, hi = lane >> 4;
        const uint32_t there = __ballot_sync(0xFFFFFFFFu, row != nullptr) >> hi;
        const uintptr_t at = row ? from : reinterpret_cast<uintptr_t>(b.pool);
        auto copy = [&](uint32_t dst, int off) {
          const uint32_t to = sb + dst + (c >> 3) * kPanel + hi * 128;
          const int o = off + (int)c * 16;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const uint8_t* s = reinterpret_cast<const uint8_t*>(__shfl_sync(0xFFFFFFFFu, at, (int)(2 * k + hi)));
            cp_async16(to + k * 256 + ((((c & 7) ^ hi) ^ (2 * k & 7)) << 4), s + o, (there >> (2 * k)) & 1u ? 16u : 0u);
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
        };
        copy(kdst, g * kHeadDim * 2);
        write_meta();
        if (j > 0) {                                 // V of step j - 1 has landed
          asm volatile("cp.async.wait_group 1;" ::: "memory");
          fence_async_smem();
          mbar_arrive(v_full((j - 1) % kStages));
        }
        if (j >= kStages) ok = mbar_wait_warp(v_empty(st), turn, err, kKernDenseAttn);
        if (!ok) break;
        copy(vdst, (kKvHeads + g) * kHeadDim * 2);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        fence_async_smem();
        mbar_arrive(k_full(st));
        if (j + 1 == steps) {
          asm volatile("cp.async.wait_group 0;" ::: "memory");
          fence_async_smem();
          mbar_arrive(v_full(st));
        }
      } else {
        // 8 lanes read the 128 codes of a token's K[g] (or V[g]); four tokens per turn
        const uint32_t c = lane & 7, four = lane >> 3;
        uint4 kv[8], vv[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint8_t* s = reinterpret_cast<const uint8_t*>(__shfl_sync(0xFFFFFFFFu, from, (int)(4 * k + four)));
          kv[k] = s ? *reinterpret_cast<const uint4*>(s + g * kHeadDim + c * 16) : make_uint4(0, 0, 0, 0);
          vv[k] = s ? *reinterpret_cast<const uint4*>(s + (kKvHeads + g) * kHeadDim + c * 16) : make_uint4(0, 0, 0, 0);
        }
        uint16_t kraw = 0, vraw = 0;   // (converted when used: a conversion here would wait for the loads)
        if (row) {
          const uint16_t* sc = reinterpret_cast<const uint16_t*>(row + 2 * kKvHeads * kHeadDim);
          kraw = sc[g];
          vraw = sc[kKvHeads + g];
        }
        write_meta();
        const float ks = key_scale_of(kraw), vs = __half2float(__ushort_as_half(vraw));
        scales[j % kMetas].k[32 * w + lane] = ks * p.scale_log2;
        scales[j % kMetas].v[32 * w + lane] = vs;
        scales[j % kMetas].size[32 * w + lane] = log2_size(vs);
        const uint32_t exps = __reduce_or_sync(0xFFFFFFFFu, row ? 1u << ((vraw >> 10) & 31) : 0u);
        if (lane == 0) m.exps[w] = exps;
        // codes 16 c .. +15 are chunks 2 c, 2 c + 1 of the row's 16
        auto store = [&](uint32_t dst, const uint4 (&x)[8]) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t r = 4 * k + four;
            uint8_t* to = smem + dst + (c >> 2) * kPanel + r * 128;
            const uint32_t c0 = (2 * c) & 7;
            *reinterpret_cast<uint4*>(to + ((c0 ^ (r & 7)) << 4)) = codes8_f16(make_uint2(x[k].x, x[k].y));
            *reinterpret_cast<uint4*>(to + (((c0 + 1) ^ (r & 7)) << 4)) = codes8_f16(make_uint2(x[k].z, x[k].w));
          }
          fence_async_smem();
        };
        store(kdst, kv);
        mbar_arrive(k_full(st));
        if (j >= kStages) ok = mbar_wait_warp(v_empty(st), turn, err, kKernDenseAttn);
        if (!ok) break;
        store(vdst, vv);
        mbar_arrive(v_full(st));
      }
      prefetch(slot_two);
      slot_now = slot_next;
      slot_next = slot_two;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  } else if (warp >= kRoleMma && warp - kRoleMma < halves) {
    // ---- MMA warp of half h
    const int h = warp - kRoleMma;
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    const uint32_t colO = tm + kColO + 128u * (uint32_t)h, colS = tm + kColS + 128u * (uint32_t)h;
    const uint32_t is = kFp8 ? idesc_f16(kSubTokens, false) : idesc_bf16(kSubTokens, false);
    const uint32_t io = kFp8 ? idesc_f16(kHeadDim, true) : idesc_bf16(kHeadDim, true);
    const uint64_t qd = desc_sw128(sb + h * 2 * kPanel, 16);
    // S of tokens 64 c .. of the step in K stage st
    auto issue_s = [&](int c, int st) {
      if (elect_one()) {
        const uint64_t kd = desc_sw128(sb + kOffKv + st * kStageBytes + c * kSubTokens * 128, 16);
#pragma unroll
        for (int k = 0; k < kHeadDim / 16; ++k) {
          const uint64_t o = (uint64_t)(((k >> 2) * kPanel + (k & 3) * 32) >> 4);
          mma_ss(colS + 64u * (uint32_t)c, qd + o, kd + o, is, k != 0);
        }
        mbar_arrive(s_full(h, c));   // passes on the loaders' writes of the meta (waited for with K)
        commit(s_full(h, c));
        if (c == 1) commit(k_empty(st));
      }
      __syncwarp();
    };
    if (steps > 0) {
      ok = mbar_wait_warp(q_full, 0, err, kKernDenseAttn);
      if (ok) ok = mbar_wait_warp(k_full(0), 0, err, kKernDenseAttn);
      if (ok) {
        fence_after();
        issue_s(0, 0);
        issue_s(1, 0);
      }
    }
#pragma unroll 1
    for (int j = 0; j < steps && ok; ++j) {
      const int st = j % kStages, sn = (j + 1) % kStages;
      ok = mbar_wait_warp(v_full(st), (uint32_t)(j / kStages) & 1u, err, kKernDenseAttn);
#pragma unroll 1
      for (int c = 0; c < 2 && ok; ++c) {
        ok = mbar_wait_warp(p_full(h, c), (uint32_t)j & 1u, err, kKernDenseAttn);
        if (!ok) break;
        fence_after();
        if (elect_one()) {
          const uint64_t vd = desc_sw128(sb + kOffKv + st * kStageBytes + kKvBytes + c * kSubTokens * 128, kPanel);
#pragma unroll
          for (int k = 0; k < kSubTokens / 16; ++k)
            mma_ts(colO, colS + 64u * (uint32_t)c + 8u * k, vd + (uint64_t)(k * 2048 >> 4), io, j > 0 || c > 0 || k > 0);
          commit(o_full(h, c));
          if (c == 1) commit(v_empty(st));
        }
        __syncwarp();
        if (j + 1 < steps) {
          // the next S goes over this P: after its products are complete
          if (c == 0) ok = mbar_wait_warp(k_full(sn), (uint32_t)((j + 1) / kStages) & 1u, err, kKernDenseAttn);
          if (ok) ok = mbar_wait_warp(o_full(h, c), (uint32_t)j & 1u, err, kKernDenseAttn);
          if (!ok) break;
          fence_after();
          issue_s(c, sn);
        }
      }
    }
    // every product is complete before tensor memory is given back
    if (elect_one()) commit(done(h));
    __syncwarp();
    mbar_wait_warp(done(h), 0, err, kKernDenseAttn);
  } else if (warp / 4 < halves) {
    // ---- softmax: thread = row (head warp & 3, query lane) of half h
    const int h = warp >> 2, head = g * kGroup + (warp & 3), q = 32 * h + lane;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t colO = lane_base + kColO + 128u * (uint32_t)h;
    const int64_t pos = pos0 + q;
    // FP8: the K scales hold the softmax scale
    const float f = kFp8 ? row_factor[128 * h + (warp & 3) * 32 + lane] : p.scale_log2;
    const uint64_t f2 = pair(f, f);
    float m = -INFINITY, l = 0.f;                    // in units of log2
#pragma unroll 1
    for (int jc = 0; jc < 2 * steps; ++jc) {
      const int j = jc >> 1, c = jc & 1;             // tokens 64 c .. of step j
      const uint32_t colS = lane_base + kColS + 128u * (uint32_t)h + 64u * (uint32_t)c;
      ok = mbar_wait_warp(s_full(h, c), (uint32_t)j & 1u, err, kKernDenseAttn);
      if (!ok) break;
      fence_after();
      const StepMeta& sm = meta[j % kMetas];
      const Scales& sc = scales[j % kMetas];
      const bool special = (sm.special[0] | sm.special[1] | sm.special[2] | sm.special[3]) != 0;
      uint64_t seen = ~0ull;                         // per token: its row exists and q sees it
      if (special)
        seen = seen_bits(p.d, t, (int64_t)(j0 + j) * kStepTokens + kSubTokens * c, pos) &
               ((uint64_t)sm.valid[2 * c] | ((uint64_t)sm.valid[2 * c + 1] << 32));
      // FP8: probabilities times V scales go in as f16, so the reference follows
      // the largest of these products that the row has, not of the probabilities:
      // log2 of both, x + log2 s.  Where the 64 tokens' scales lie within a factor
      // of 64, s counts as the upper end of that range (`above`); elsewhere (also at
      // zeros, subnormals, infinities and NaN) each as it is, a zero as 2^-100: its
      // token still keeps the sum l in range (and where such tokens outweigh all
      // others, f16's 2^-25 is 2^-117 of the row's weight).
      float above = 0.f, most = -INFINITY;
      bool wide = false;
      if (kFp8) {
        const uint32_t exps = sm.exps[2 * c] | sm.exps[2 * c + 1];
        const int high = 31 - __clz(exps);
        above = (float)(high - 14);
        wide = (exps & 0x80000001u) || high - (__ffs(exps) - 1) > 5;
        if (wide) most = wide_max(colS, sc, c, seen, f);
      }
      uint32_t v[2][32];
      ld32(colS, v[0]);
      ld32(colS + 32u, v[1]);
      wait_ld();
      reg_fence(v[0]);
      reg_fence(v[1]);
      if (kFp8) {
#pragma unroll
        for (int i = 0; i < kSubTokens; i += 4) {
          const ulonglong2 k4 = *reinterpret_cast<const ulonglong2*>(&sc.k[kSubTokens * c + i]);
          uint32_t* x = &v[i >> 5][i & 31];
          const uint64_t a = mul2(pair(x[0], x[1]), k4.x), d = mul2(pair(x[2], x[3]), k4.y);
          x[0] = (uint32_t)a;
          x[1] = (uint32_t)(a >> 32);
          x[2] = (uint32_t)d;
          x[3] = (uint32_t)(d >> 32);
        }
      }
      const uint32_t tok[2] = {(uint32_t)seen, (uint32_t)(seen >> 32)};
      if (special) {
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!((tok[w] >> i) & 1u)) v[w][i] = __float_as_uint(-INFINITY);
      }
      auto at = [&](int i) { return __uint_as_float(v[i >> 5][i & 31]); };
      float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < kSubTokens; i += 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) mx4[k] = fmaxf(mx4[k], fmaxf(at(i + k), at(i + 4 + k)));
      }
      float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * f;
      if (f == 0.f) mx = 0.f;                        // (a scale of 0, beside -inf)
      if (kFp8) mx = wide ? most : mx + above;
      // the reference goes up only when the maximum has left it 2^8 behind
      const bool up = mx > m + 8.f;                  // true for the first tokens
      if (__any_sync(0xFFFFFFFFu, up)) {
        const float mn = fmaxf(m, mx);
        const float a = mn == -INFINITY ? 1.f : exp2_fast(m - mn);
        m = mn;
        l *= a;
        if (jc > 0) {
          // all products so far have to be complete
          ok = mbar_wait_warp(o_full(h, c ^ 1), (uint32_t)((jc - 1) >> 1) & 1u, err, kKernDenseAttn);
          if (!ok) break;
          fence_after();
#pragma unroll 1
          for (int i = 0; i < kHeadDim; i += 16) {
            uint32_t o[16];
            ld16(colO + (uint32_t)i, o);
            wait_ld();
            reg_fence(o);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
            st16(colO + (uint32_t)i, o);
          }
          wait_st();
        }
      }
      const float ref = m == -INFINITY ? 0.f : m;
      const uint64_t addend = pair(-ref, -ref);
      uint64_t l2[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
      // ---- probabilities over S's columns
#pragma unroll
      for (int w = 0; w < 2; ++w) {                  // 32 tokens
        uint32_t o[16];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint64_t x01 = fma2(pair(v[w][4 * k], v[w][4 * k + 1]), f2, addend);
          const uint64_t x23 = fma2(pair(v[w][4 * k + 2], v[w][4 * k + 3]), f2, addend);
          float e[4] = {exp2_fast(lo_of(x01)), exp2_fast(hi_of(x01)), exp2_fast(lo_of(x23)), exp2_fast(hi_of(x23))};
          if (special) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!((tok[w] >> (4 * k + i)) & 1u)) e[i] = 0.f;
          }
          l2[0] = add2(l2[0], pair(e[0], e[1]));
          l2[1] = add2(l2[1], pair(e[2], e[3]));
          if (kFp8) {
            const ulonglong2 v4 = *reinterpret_cast<const ulonglong2*>(&sc.v[kSubTokens * c + 32 * w + 4 * k]);
            const uint64_t a = mul2(pair(e[0], e[1]), v4.x), d = mul2(pair(e[2], e[3]), v4.y);
            e[0] = lo_of(a);
            e[1] = hi_of(a);
            e[2] = lo_of(d);
            e[3] = hi_of(d);
          }
          o[2 * k] = kFp8 ? pack_f16(e[0], e[1]) : pack_bf16(e[0], e[1]);
          o[2 * k + 1] = kFp8 ? pack_f16(e[2], e[3]) : pack_bf16(e[2], e[3]);
        }
        st16(colS + 16u * w, o);
      }
      // the 64 tokens' sum, then the running one: 64 times fewer roundings at its size
      const uint64_t l4 = add2(l2[0], l2[1]);
      l += lo_of(l4) + hi_of(l4);
      wait_st();
      fence_before();
      mbar_arrive(p_full(h, c));
    }
    // ---- the rows' results: from a row to a thread, through the K and V stages once
    // all products are complete, to a row at a time (16-byte chunks at chunk ^ row)
    for (int i = 0; i < halves; ++i) ok = mbar_wait_warp(done(i), 0, err, kKernDenseAttn) && ok;
    fence_after();
    uint8_t* stage = smem + kOffKv + warp * (32 * kHeadDim * 4);
    const int rows = !ok ? 0 : (nq - 32 * h < 32 ? nq - 32 * h : 32);
    if (shares > 1 || p.grouped) {
#pragma unroll 1
      for (int c = 0; c < 4 && ok && steps > 0; ++c) {
        uint32_t v[32];
        ld32(colO + 32u * c, v);
        wait_ld();
        reg_fence(v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4*>(stage + lane * (kHeadDim * 4) + (((8 * c + i) ^ lane) << 4)) =
              make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      }
      __syncwarp();
      float* to = piece_ptr(p, pre, t.u, blockIdx.x, x0 + 32 * h, head);
#pragma unroll 8
      for (int i = 0; i < rows; ++i, to += kQHeads * kRowFloats) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (steps > 0) v = *reinterpret_cast<const float4*>(stage + i * (kHeadDim * 4) + ((lane ^ i) << 4));
        *reinterpret_cast<float4*>(to + 4 * lane) = v;
      }
      if (lane < rows)
        *reinterpret_cast<float2*>(piece_ptr(p, pre, t.u, blockIdx.x, x0 + q, head) + kHeadDim) = make_float2(m, l);
    } else {
      const float inv = 1.f / l;
      bool good = good_sum(l) && steps > 0;
#pragma unroll 1
      for (int c = 0; c < 4 && ok && steps > 0; ++c) {
        uint32_t v[32];
        ld32(colO + 32u * c, v);
        wait_ld();
        reg_fence(v);
        float far = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) far = fmaxf(far, isfinite(__uint_as_float(v[i])) ? 0.f : 1.f);
        good = good && far == 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = pack_bf16(__uint_as_float(v[8 * i + 2 * k]) * inv, __uint_as_float(v[8 * i + 2 * k + 1]) * inv);
          *reinterpret_cast<uint4*>(stage + lane * (kHeadDim * 2) + (((4 * c + i) ^ (lane & 15)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      __syncwarp();
      // 16 lanes a row
      uint16_t* out = p.out + ((int64_t)(x0 + 32 * h) * kQHeads + head) * kHeadDim;
#pragma unroll 8
      for (int i = lane >> 4; i < rows && steps > 0; i += 2)
        reinterpret_cast<uint4*>(out + (int64_t)i * (kQHeads * kHeadDim))[lane & 15] =
            *reinterpret_cast<const uint4*>(stage + i * (kHeadDim * 2) + (((lane & 15) ^ (i & 15)) << 4));
      if (lane < rows && good && p.lse) p.lse[(int64_t)(x0 + q) * kQHeads + head] = (m + log2f(l)) * kLn2;
      for (uint32_t again = __ballot_sync(0xFFFFFFFFu, lane < rows && !good); again; again &= again - 1) {
        __syncwarp();
        attend_row(p, t.u, x0 + 32 * h + __ffs(again) - 1, head);
      }
    }
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kRoleMma) tmem_free<kTmemCols>(tmem);
}

// ------------------------------------------------------------------- join

// kSplit warps per (row, head), each over every kSplit-th piece (eight where there are
// many: their loads are what the join waits for); lane l holds dims 4 l .. 4 l + 3.
// No piece is left out, however small its factor is: a sum or an O that is not finite
// stays one (0 times it is NaN), and the row is computed again.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
template <int kSplit>
__global__ void __launch_bounds__(kJoinThreads) dense_join_kernel(const __grid_constant__ DenseParams p) {
  __shared__ float4 part_o[kSplit > 1 ? kJoinWarps : 1][32];
  __shared__ float2 part_ml[kSplit > 1 ? kJoinWarps : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, s0 = warp % kSplit;
  const int64_t w = (int64_t)blockIdx.x * (kJoinWarps / kSplit) + warp / kSplit;
  const int j = (int)(w / kQHeads), head = (int)(w % kQHeads);              // the j-th row that has partials
  const int units = p.d.c.b.n_units;
  if (j >= p.join0[units]) return;                   // (with kSplit warps the same for the whole CTA)
  int u = 0;
  for (int hi = units - 1; u < hi;) {
    const int mid = (u + hi + 1) >> 1;
    if (p.join0[mid] <= j) u = mid; else hi = mid - 1;
  }
  const int x = p.d.c.row0[u] + j - p.join0[u];
  const int pieces = p.prefix_pieces + own_pieces(p, u, x);
  grid_dependency_wait();
  if (!p.grouped && pieces == 1) return;             // complete
  const float* prefix_part = piece_ptr(p, true, u, 0, x, head);
  const float* own_part = piece_ptr(p, false, u, 0, x, head);
  const int64_t prefix_stride = (int64_t)p.d.c.rows() * kQHeads * kRowFloats;
  const int64_t own_stride = (int64_t)p.d.c.unit_tokens(u) * kQHeads * kRowFloats;
  auto piece = [&](int k) {                          // the k-th of this warp
    const int i = s0 + k * kSplit;
    return i < p.prefix_pieces ? prefix_part + i * prefix_stride : own_part + (i - p.prefix_pieces) * own_stride;
  };
  const int n = pieces > s0 ? (pieces - s0 + kSplit - 1) / kSplit : 0;       // of this warp
  // eight pieces' O, maxima and sums are on their way at a time
  constexpr int kTurn = 8;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < n; k0 += kTurn) {
    float4 o[kTurn];
    float2 ml[kTurn];
#pragma unroll
    for (int k = 0; k < kTurn; ++k) {
      const float* from = piece(k0 + k);
      ml[k] = k0 + k < n ? *reinterpret_cast<const float2*>(from + kHeadDim) : make_float2(-INFINITY, 0.f);
      o[k] = k0 + k < n ? *reinterpret_cast<const float4*>(from + 4 * lane) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float mn = m;
#pragma unroll
    for (int k = 0; k < kTurn; ++k) mn = fmaxf(mn, ml[k].x);
    const float a = l != 0.f ? exp2f(m - mn) : 0.f;
    m = mn;
    l *= a;
    acc = make_float4(acc.x * a, acc.y * a, acc.z * a, acc.w * a);
#pragma unroll
    for (int k = 0; k < kTurn; ++k) {
      const float c = ml[k].y != 0.f ? exp2f(ml[k].x - mn) : 0.f;            // 0: nothing there
      l = fmaf(ml[k].y, c, l);
      acc = make_float4(fmaf(o[k].x, c, acc.x), fmaf(o[k].y, c, acc.y), fmaf(o[k].z, c, acc.z), fmaf(o[k].w, c, acc.w));
    }
  }
  if (kSplit > 1) {
    part_o[warp][lane] = acc;
    if (lane == 0) part_ml[warp] = make_float2(m, l);
    __syncthreads();
    if (s0 != 0) return;
    float mn = -INFINITY;
#pragma unroll
    for (int k = 0; k < kSplit; ++k) mn = fmaxf(mn, part_ml[warp + k].x);
    l = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kSplit; ++k) {
      const float2 ml = part_ml[warp + k];
      const float4 o = part_o[warp + k][lane];
      const float c = ml.y != 0.f ? exp2f(ml.x - mn) : 0.f;
      l = fmaf(ml.y, c, l);
      acc = make_float4(fmaf(o.x, c, acc.x), fmaf(o.y, c, acc.y), fmaf(o.z, c, acc.z), fmaf(o.w, c, acc.w));
    }
    m = mn;
  }
  const bool fine = good_sum(l) && isfinite(acc.x) && isfinite(acc.y) && isfinite(acc.z) && isfinite(acc.w);
  if (!__all_sync(0xFFFFFFFFu, fine)) {
    attend_row(p, u, x, head);
    return;
  }
  const float r = 1.f / l;
  reinterpret_cast<uint2*>(p.out + ((int64_t)x * kQHeads + head) * kHeadDim)[lane] =
      make_uint2(pack_bf16(acc.x * r, acc.y * r), pack_bf16(acc.z * r, acc.w * r));
  if (p.lse && lane == 0) p.lse[(int64_t)x * kQHeads + head] = (m + log2f(l)) * kLn2;
}

// ------------------------------------------------------------------- host

// Grids, shares and the workspace of a call.
struct Plan {
  int grouped = 0;
  int wide_tiles = 0, few_tiles = 0;                 // grid y of the two kernels
  int wide_shares = 0, few_shares = 0;               // grid x
  int wide_q = 1, few_q = 1;
  int few_rows = 0;                                  // queries of a tile of the few kernel, at most
  int64_t pieces = 1;                                // of a row, at most
  int64_t prefix_pieces = 0;
  int join_rows = 0;                                 // rows that have partials
  int64_t bytes = 256;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Steps of a share: the fewest, but `least` at least, for which the shares of all
// tiles (n of them, steps[i] long) are no more than `most`.
int share_steps(const int64_t* steps, int n, int64_t most, int64_t least) {
  int64_t longest = 1;
  for (int i = 0; i < n; ++i) longest = steps[i] > longest ? steps[i] : longest;
  int64_t lo = ceil_div(longest, kMaxShares);
  if (lo < least) lo = least;
  int64_t hi = longest > lo ? longest : lo;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    int64_t sum = 0;
    for (int i = 0; i < n; ++i) sum += ceil_div(steps[i], mid);
    if (sum <= most) hi = mid; else lo = mid + 1;
  }
  // not for less than a quarter of the longest: the join comes on top (measured on one
  // case: 2 x 1023 FP8 queries, 32 tiles of up to 64 steps on 38 shares, 170 us with 63
  // steps a share, 162 with whole tiles)
  return (int)(lo > longest - longest / 4 && longest > lo ? longest : lo);
}

constexpr int kLeastWide = 2, kLeastFew = 1;          // steps of a share at least

// p: receives the prefix sums per unit, or nullptr.
Plan make_plan(const DenseAttn& d, int sms, DenseParams* p) {
  Plan a;
  const int units = d.c.b.n_units, layers = units / d.n_req, layer_rows = d.c.row0[d.n_req];
  int with_rows = 0;                                 // requests
  for (int r = 0; r < d.n_req; ++r) with_rows += d.c.unit_tokens(r) > 0;
  // The prefix has tiles of its own where its tiles of 64 rows are fewer than half
  // of those that the requests alone make.
  a.grouped = d.prefix_len > 0 && with_rows > 1 && layer_rows <= with_rows * (kTileQueries / 2);
  const bool few_prefix = a.grouped && layer_rows <= kFewQueries;
  int own_tiles = 0, few_units = 0;
  // of every tile of the few kernel: the units, and the prefix at every layer (a few
  // prefix has two requests at least, so half as many layers as units at most)
  int64_t few_steps[kMaxUnits + kMaxUnits / 2];
  for (int u = 0; u < units; ++u) {
    const int n = d.c.unit_tokens(u);
    if (p) p->tile0[u] = own_tiles;
    if (n > kFewQueries) own_tiles += (n + kTileQueries - 1) / kTileQueries;
    if (n == 0 || n > kFewQueries) continue;
    a.few_rows = n > a.few_rows ? n : a.few_rows;
    few_steps[few_units++] = ceil_div(own_tile(d, a.grouped, u, 0).total, kFewStep);
  }
  if (p) p->tile0[units] = own_tiles;
  const int per_prefix = a.grouped && !few_prefix ? (layer_rows + kTileQueries - 1) / kTileQueries : 0;
  a.wide_tiles = own_tiles + layers * per_prefix;
  int64_t longest_own = 0, longest = 0;              // wide
  auto each = [&](auto&& fn) {
    for (int u = 0; own_tiles > 0 && u < units; ++u)
      if (d.c.unit_tokens(u) > kFewQueries)
        for (int i = 0; i < d.c.unit_tokens(u); i += kTileQueries)
          fn(ceil_div(own_tile(d, a.grouped, u, i).total, kStepTokens));
  };
  const int64_t prefix_steps = ceil_div(d.prefix_len, kStepTokens), few_prefix_steps = ceil_div(d.prefix_len, kFewStep);
  if (a.wide_tiles > 0) {
    const int64_t most = sms / kKvHeads;
    int64_t steps[128];
    int n = 0;
    const bool split = a.wide_tiles < most && a.wide_tiles <= 128;
    each([&](int64_t s) {
      longest_own = s > longest_own ? s : longest_own;
      if (split) steps[n++] = s;
    });
    longest = per_prefix && prefix_steps > longest_own ? prefix_steps : longest_own;
    if (split) {
      for (int i = 0; i < layers * per_prefix; ++i) steps[n++] = prefix_steps;
      a.wide_q = share_steps(steps, n, most, kLeastWide);
    } else {
      a.wide_q = (int)(longest > 1 ? longest : 1);
    }
    a.wide_shares = (int)ceil_div(longest, a.wide_q);
    if (a.wide_shares == 0) a.wide_shares = 1;       // (rows without any token)
  }
  int64_t longest_few = 0;
  if (few_units > 0) {
    a.few_tiles = units + (few_prefix ? layers : 0);
    for (int i = 0; i < few_units; ++i) longest_few = few_steps[i] > longest_few ? few_steps[i] : longest_few;
    int n = few_units;
    if (few_prefix)
      for (int i = 0; i < layers; ++i) few_steps[n++] = few_prefix_steps;
    if (few_prefix) a.few_rows = layer_rows > a.few_rows ? layer_rows : a.few_rows;
    // (FP8 rows, two queries: two CTAs to an SM)
    a.few_q = share_steps(few_steps, n, a.few_rows <= 2 && d.c.b.row_bytes == kRowBytesFp8 ? 2 * sms : sms, kLeastFew);
    const int64_t most = few_prefix && few_prefix_steps > longest_few ? few_prefix_steps : longest_few;
    a.few_shares = (int)ceil_div(most, a.few_q);
    if (a.few_shares == 0) a.few_shares = 1;
  }
  if (a.grouped) a.prefix_pieces = few_prefix ? ceil_div(few_prefix_steps, a.few_q) : ceil_div(prefix_steps, a.wide_q);
  // partials for the rows that have several pieces alone: a long context of one token
  // beside a prompt's rows, each written at once, has 64 and these none
  int64_t most_own = 0, part_rows = 0;
  for (int u = 0; u < units; ++u) {
    const int n = d.c.unit_tokens(u);
    const bool few = n <= kFewQueries;
    int64_t own = n > 0 ? 1 : 0;                     // pieces of a row, at most
    if (n > 0 && (few ? a.few_shares : a.wide_shares) > 1) {
      for (int i = 0; i < n; i += kTileQueries) {
        const int64_t k = shares_of(own_tile(d, a.grouped, u, i), few ? kFewStep : kStepTokens, few ? a.few_q : a.wide_q, true);
        own = k > own ? k : own;
      }
    }
    if (p) p->part0[u] = (int32_t)part_rows;
    if (p) p->join0[u] = a.join_rows;
    if (!a.grouped && own <= 1) continue;
    part_rows += own * n;
    a.join_rows += n;
    most_own = own > most_own ? own : most_own;
  }
  if (p) p->part0[units] = (int32_t)part_rows;
  if (p) p->join0[units] = a.join_rows;
  a.pieces = most_own + a.prefix_pieces;
  if (a.join_rows > 0) a.bytes = (a.prefix_pieces * d.c.rows() + part_rows) * kQHeads * kRowFloats * 4;
  return a;
}

}  // namespace

int64_t dense_attn_workspace(const DenseAttn& d) {
  int sms = 0;
  if (current_sm_count(&sms) != cudaSuccess) return -1;
  return make_plan(d, sms, nullptr).bytes;
}

cudaError_t launch_dense_attn(const DenseAttn& d, const uint16_t* q, float softmax_scale, uint16_t* out, float* lse,
                              void* workspace, cudaStream_t s) {
  static PerDeviceOnce setup;
  cudaError_t e = setup.run([] {
    cudaError_t r = prefer_max_shared(dense_wide_kernel<false>, kWideSmem);
    if (r == cudaSuccess) r = prefer_max_shared(dense_wide_kernel<true>, kWideSmem);
    if (r == cudaSuccess) r = prefer_max_shared(dense_few_kernel<false, 1>, FewLayout<false>::kSmem);
    if (r == cudaSuccess) r = prefer_max_shared(dense_few_kernel<true, 1>, FewLayout<true>::kSmem);
    if (r == cudaSuccess) r = prefer_max_shared(dense_few_kernel<false, 2>, FewLayout<false>::kSmem);
    if (r == cudaSuccess) r = prefer_max_shared(dense_few_kernel<true, 2>, FewLayout<true>::kSmem);
    return r;
  });
  int sms = 0;
  if (e == cudaSuccess) e = current_sm_count(&sms);
  if (e != cudaSuccess) return e;
  DenseParams p;
  const Plan a = make_plan(d, sms, &p);
  p.d = d;
  p.grouped = a.grouped;
  p.prefix_pieces = (int32_t)a.prefix_pieces;
  p.wide_q = a.wide_q;
  p.few_q = a.few_q;
  p.q = q;
  p.scale_log2 = fabsf(softmax_scale) * kLog2e;
  p.sign = softmax_scale < 0.f ? -1.f : 1.f;
  p.out = out;
  p.lse = lse;
  p.part = static_cast<float*>(workspace);
  const bool fp8 = d.c.b.row_bytes == kRowBytesFp8;
  if (a.wide_tiles > 0) {
    const dim3 grid((unsigned)a.wide_shares, (unsigned)a.wide_tiles, kKvHeads);
    e = launch_kernel(fp8 ? dense_wide_kernel<true> : dense_wide_kernel<false>, grid, dim3(kWideThreads), kWideSmem, s, 0,
                      dim3(1), p);
  }
  if (e == cudaSuccess && a.few_tiles > 0) {
    const dim3 grid((unsigned)a.few_shares, (unsigned)a.few_tiles);
    const int n = a.few_rows > 2 ? 2 : 1;
    auto* kernel = fp8 ? (n == 1 ? dense_few_kernel<true, 1> : dense_few_kernel<true, 2>)
                       : (n == 1 ? dense_few_kernel<false, 1> : dense_few_kernel<false, 2>);
    e = launch_kernel(kernel, grid, dim3(kFewThreads), fp8 ? FewLayout<true>::kSmem : FewLayout<false>::kSmem, s, 0, dim3(1), p);
  }
  if (e != cudaSuccess || a.join_rows == 0) return e;
  const int64_t rows = (int64_t)a.join_rows * kQHeads;
  if (a.pieces > 8)
    return launch_kernel(dense_join_kernel<kJoinWarps>, dim3((unsigned)rows), dim3(kJoinThreads), 0, s, 0, dim3(1), p);
  return launch_kernel(dense_join_kernel<1>, dim3((unsigned)ceil_div(rows, kJoinWarps)), dim3(kJoinThreads), 0, s, 0,
                       dim3(1), p);
}

}  // namespace qsa
