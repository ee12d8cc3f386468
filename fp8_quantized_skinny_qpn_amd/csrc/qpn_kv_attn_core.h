// qpn_kv_attn_core.h -- what attention over the paged caches shares whatever their
// codes are: the split of a call into pieces, masks, running maxima, the products
// of many rows, and the joins of pieces.
//
// Work split.  A segment (request, KV head, tile of rows) is cut into pieces of
// about P pages, one workgroup each.  P comes from the lengths on the device, so
// that ragged requests fill the chip evenly with no host read.  The pieces of a
// cut segment leave their sums in scratch, written through to the device's point
// of coherence, and count themselves in; the last to arrive joins them in
// order (of more than kJoinDirect pieces: in groups, then the groups).
#pragma once

#include <type_traits>

#include "qpn_common.h"
#include "qpn_kv_internal.h"
#include "qpn_kv_lanes.h"

namespace qpn {

namespace {

constexpr int kRsrc = 0x00020000;

constexpr float kMaxSlack = 8.0f;       // how far (log2) a score may pass the running maximum
// Many rows: the FP16 weights carry the page's V scale as a factor vs / vref, which stays
// from 1 on (a smaller one would push weights among FP16's subnormal numbers and cost them
// bits) to this (with the 2^8 above, weights stay below 2^15).  When a page leaves that
// range vref, a power of two, is set anew: to the page's scale's less kScaleBelow.
constexpr float kScaleSlack = 128.0f;
constexpr int kScaleBelow = 3;          // (log2)
constexpr float kScaleLeast = 0x1p-40f; // values of a smaller scale (they are below 2^-31) count as zeros
constexpr float kLowest = -3e38f;     // the running maximum before any score

constexpr int kManyWaves = 8;  // and many rows
// Pages of a piece at least: one for each of the eight wavefronts of few rows.
// (8 rows of 40 + 8 heads over 4099 tokens: 20.3 us with 4, 19.0 with 8, 20.8
// with 16; 256 rows over 4096: 46.3, 46.2, 53.2.)
constexpr int kMinPiecePages = 8;
constexpr int kMaxPieces = 512;    // pieces of a call with cut segments
constexpr int kCounterStep = 8;    // 32-bit words between counters
static_assert((size_t)kMaxPieces * 2 * kCounterStep * 4 <= kKvZeroedBytes, "two counters per piece");

// What differs between the caches, for a kind of arguments A:
//   few_tiles(dim), many_tiles(dim)  16-row tiles: the most of the few-rows form, those of a
//                                    wavefront with many rows
//   apart(tiles, groups, pages)      whether the tiles of few rows are segments of their own, with
//                                    so many requests x KV heads and pages of each at most
//   at_once(n)                       sums of n fragments each that a join loads together
//   kJoinDirect                      pieces joined in one step
//   first_dim<DIM>(d, g)             the first of the four dimensions that lane group g holds of
//                                    the dimension tile d of the second product
template <typename A>
struct KindOf;

struct Form {
  bool many;
  int tiles;
  int rows() const { return 16 * tiles * (many ? kManyWaves : 1); }
};
template <typename A>
Form form_of(int requests, int max_rows, int q_heads, int heads, int dim, int table_width) {
  const int64_t t = ((int64_t)max_rows * (q_heads / heads) + 15) / 16;
  if (t <= KindOf<A>::few_tiles(dim))
    return {false, t < 1 || KindOf<A>::apart(t, (int64_t)requests * heads, table_width) ? 1 : (int)t};
  return {true, t <= kManyWaves ? 1 : KindOf<A>::many_tiles(dim)};
}

struct AttnLaunch {
  int tile_rows;   // rows of a workgroup's segment
  int group;       // query heads of a KV head
  uint32_t inverse;  // ceil(2^32 / group), for row_of
  int target;      // pieces the lengths are cut into
  int slots;       // pieces the scratch has room for (0: segments stay whole)
  float* partial;  // 1.5 slots of partial sums (layout at Slot)
};

// The query row of row `rr` of a segment, rr / group: exact for rr < 2^26, as
// the inverse is less than group <= 64 parts in 2^32 too large.
__device__ __forceinline__ int row_of(const AttnLaunch& l, int rr) {
  return l.group == 1 ? rr : (int)__umulhi((uint32_t)rr, l.inverse);
}

// One request as the kernels see it.
struct Req {
  int row0, rows;          // its rows (0: skipped)
  int seq;                 // tokens it sees at its last row, clamped to the table
  bool bad;                // more tokens than the table has pages for
  int first_page, pages;   // pages any of its rows sees (at least 1 when it has rows)
  int tiles;               // row tiles of a KV head
};

template <typename A>
__device__ __forceinline__ Req request_of(const A& a, const AttnLaunch& l, int r) {
  Req q;
  const int s0 = a.row_start[r], s1 = a.row_start[r + 1];
  const int seq = a.seq_lens[r];
  q.row0 = s0;
  q.rows = s0 >= 0 && s1 > s0 && s1 <= a.rows ? s1 - s0 : 0;
  const int most = a.table_width * kKvPage;  // (below 2^31)
  q.bad = seq > most;
  q.seq = q.bad ? most : seq < 0 ? 0 : seq;
  const int start = a.window > 0 && q.seq - q.rows >= a.window ? q.seq - q.rows + 1 - a.window : 0;
  q.first_page = start / kKvPage;
  const int last = q.seq / kKvPage + (q.seq % kKvPage != 0);
  q.pages = last > q.first_page ? last - q.first_page : 1;
  q.tiles = (int)((uint32_t)(q.rows * l.group + l.tile_rows - 1) / (uint32_t)l.tile_rows);
  return q;
}

__device__ __forceinline__ int wave_sum(int x) {
  return wave_reduced(x, [](int a, int b) { return a + b; });
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

__device__ __forceinline__ int ceil_div(int x, int y) { return (int)(((uint32_t)x + (uint32_t)y - 1) / (uint32_t)y); }

// What a workgroup does: piece `piece` of `pieces` of a segment.
struct Item {
  int request;       // -1: none
  int head, tile, piece, pieces;
  int first;         // the segment's first piece, in an order in which a segment's pieces follow one another
};

// The pages of a piece and the pieces of a call of more than one request.
// P is the smallest of kMinPiecePages or more that makes no more than `target`
// pieces (to a few steps of bisection for up to 64 requests, by the simple
// bound for more); everything stays whole when the scratch is too small.
// Every number fits 31 bits: a call has at most 2^30 rows x query heads.  (Of
// requests that name the same rows again and again the count of segments stops
// at 2^30; item_of turns away what a wrapped total would make.)
struct Cut {
  int page, total;
};
template <typename A>
__device__ __forceinline__ Cut cut_of(const A& a, const AttnLaunch& l, int lane) {
  int segs = 0, my_segs = 0, my_pages = 1;
  float units = 0.0f;
  for (int base = 0; base < a.requests; base += 64) {
    if (base + lane < a.requests) {
      const Req q = request_of(a, l, base + lane);
      my_segs = q.tiles * a.cache.heads;
      my_pages = q.pages;
      segs = min(segs + my_segs, 1 << 24);
      units += (float)my_segs * (float)my_pages;
    }
  }
  segs = wave_sum(segs);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) units += __shfl_xor(units, d);
  const bool one = a.requests <= 64;
  int page = 1 << 30;
  if (segs < l.slots) {
    // (a float's rounding of the bounds is covered by the slack of one part in 10^5)
    int low = max(kMinPiecePages, (int)(units / (float)l.target));
    const float room = (float)(l.target > segs ? l.target - segs : 1);
    page = (int)fminf(fmaxf(units / room * 1.00001f + 1.0f, (float)low), 1e9f);
    for (int i = 0; one && i < 5 && low < page; ++i) {
      const int mid = low + ((page - low) >> 1);
      if (wave_sum(my_segs * ceil_div(my_pages, mid)) <= l.target) page = mid; else low = mid + 1;
    }
  }
  int total = 0;
  if (one) {
    total = my_segs * ceil_div(my_pages, page);
  } else {
    for (int base = 0; base < a.requests; base += 64) {
      if (base + lane < a.requests) {
        const Req q = request_of(a, l, base + lane);
        total += q.tiles * a.cache.heads * ceil_div(q.pages, page);
      }
    }
  }
  return {uniform(page), uniform(wave_sum(total))};
}

// Every wavefront finds its workgroup's item by itself (no barrier): requests,
// then KV heads, pieces, and row tiles, which share their pages.  Consecutive
// items go to one XCD (workgroups are dealt to the 8 XCDs in turn), so
// that tiles of the same pages share its L2.
template <typename A>
__device__ __forceinline__ Item item_of(const A& a, const AttnLaunch& l, int lane, int block, Req& out) {
  const int heads = a.cache.heads;
  Item it{-1, 0, 0, 0, 0, 0};
  int at, before = 0;  // the item among its request's, the items before it
  if (a.requests == 1) {
    out = request_of(a, l, 0);
    const int segs = out.tiles * heads;
    int n = 1;
    if (segs > 0 && segs < l.slots) n = max(1, min(l.target / segs, ceil_div(out.pages, kMinPiecePages)));
    const int total = segs * n, per = (total + 7) / 8;
    at = (block & 7) * per + (block >> 3);
    if ((block >> 3) >= per || at >= total) return it;
    it.request = 0;
    it.pieces = n;
  } else {
    const Cut cut = cut_of(a, l, lane);
    const int per = (cut.total + 7) / 8;
    const int item = (block & 7) * per + (block >> 3);
    if ((block >> 3) >= per || item >= cut.total) return it;
    for (int base = 0;; base += 64) {
      int n = 0;
      if (base + lane < a.requests) {
        const Req q = request_of(a, l, base + lane);
        n = q.tiles * heads * ceil_div(q.pages, cut.page);
      }
      int up = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(up, d);
        if (lane >= d) up += o;
      }
      const uint64_t past = __ballot(before + up > item);
      if (past) {
        const int r = __ffsll((unsigned long long)past) - 1;
        before = uniform(before + __shfl(up - n, r));
        it.request = uniform(base + r);
        break;
      }
      before += __shfl(up, 63);
      if (base + 64 >= a.requests) return it;  // (never: the item is below the total)
    }
    out = request_of(a, l, it.request);
    it.pieces = ceil_div(out.pages, cut.page);
    at = item - before;
  }
  out.row0 = uniform(out.row0), out.rows = uniform(out.rows), out.seq = uniform(out.seq);
  out.first_page = uniform(out.first_page), out.pages = uniform(out.pages), out.tiles = uniform(out.tiles);
  out.bad = uniform(out.bad);
  at = uniform(at);
  const int rest = (int)((uint32_t)at / (uint32_t)out.tiles);
  it.tile = at - rest * out.tiles;
  it.head = (int)((uint32_t)rest / (uint32_t)it.pieces);
  it.piece = rest - it.head * it.pieces;
  it.first = before + (it.head * out.tiles + it.tile) * it.pieces;
  if (out.tiles == 0 || (uint32_t)it.head >= (uint32_t)heads) it.request = -1;
  return it;
}

// Nonzero bytes where a code is NaN (0x7F or 0xFF).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t x) { return ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

__device__ __forceinline__ half8 to_half8(const float4v& a, const float4v& b) {
  half8 h;
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = (_Float16)a[i], h[4 + i] = (_Float16)b[i];
  return h;
}

// The first token that a row sees which sees those below lim.  (lim is negative
// for rows before the first token: no difference is taken below the window.)
__device__ __forceinline__ int low_of(int lim, int window) { return window > 0 && lim > window ? lim - window : 0; }

// What the rows of a wavefront see: tokens [low, lim) of the lane's row of
// each tile, and the extremes over its rows.
template <int RT>
struct View {
  int lim[RT], window;
  int lim_min, lim_max, low_min, low_max;
  __device__ __forceinline__ int low(int rt) const { return low_of(lim[rt], window); }
};

// Bits of the tokens [low, lim) among the 32 from `base` on, from the lane's
// first one (4 g) on: bit 16 t + r is token 16 t + 4 g + r.
__device__ __forceinline__ uint32_t seen_of(int lim, int low, int base, int g) {
  const int to = min(max(lim - base, 0), 32), from = min(max(low - base, 0), 32);
  const uint32_t m = to > from ? (~0u >> (32 - (to - from))) << from : 0u;
  return m >> (4 * g);
}
__device__ __forceinline__ uint32_t all_ones_if(uint32_t seen, int t, int r) {  // ~0 when token (t, r) is seen
  return (uint32_t)__builtin_amdgcn_sbfe((int)seen, 16 * t + r, 1);
}

// -inf for what a row does not see of a page's scores.
template <int RT>
__device__ __forceinline__ void mask_page(float4v (&s)[4][RT], int base, int g, const View<RT>& see) {
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t seen = seen_of(see.lim[rt], see.low(rt), base + 32 * half, g);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t ones = all_ones_if(seen, t, r);
          const float x = s[2 * half + t][rt][r];
          s[2 * half + t][rt][r] =
              __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, x) & ones) | (0xFF800000u & ~ones));
        }
    }
}

// The largest of the lane's 16 scores of a row.  (Of products, which are never
// signalling NaN: one instruction for two of them.)
template <int RT>
__device__ __forceinline__ float page_max(const float4v (&s)[4][RT], int rt) {
  float mx = fmaxf(s[0][rt][0], s[0][rt][1]);
#pragma unroll
  for (int i = 2; i < 16; i += 2) mx = fmaxf(fmaxf(mx, s[i >> 2][rt][i & 3]), s[i >> 2][rt][(i & 3) + 1]);
  return mx;
}

// The rows of a wavefront and their running sums.  ONE: one positive factor makes all
// scores exponents, and values have no page scales.  Then the factor is in the exponentials'
// fused multiply-add, and the matrix unit sums the FP16 weights (32 tokens under one operand
// of ones), where the scales of the 8-bit pages take a multiplication of each score and an
// FP32 sum of what the FP16 weights are rounded from.
template <int DIM, int RT, bool ONE = false>
struct Rows {
  static constexpr int KS = DIM / 32;  // k-steps of the scores
  static constexpr int DT = DIM / 16;  // tiles of output dimensions
  float m[RT];
  std::conditional_t<ONE, float4v, float> sum[RT];  // (of a float4v all four alike, of all lanes' tokens)
  float4v o[DT][RT];
  float vref;  // what the sums are in units of: a power of two

  // The unit for a page scale of kScaleLeast or more.
  static __device__ __forceinline__ float unit_for(float vs) {
    return __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, vs) & 0x7F800000u) - ((uint32_t)kScaleBelow << 23));
  }

  __device__ __forceinline__ void begin(float first_scale) {
    vref = unit_for(fmaxf(first_scale, kScaleLeast));
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      m[t] = kLowest;
      sum[t] = {};
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d][t] = float4v{0, 0, 0, 0};
    }
  }

  // Puts the sums into a unit that a page's V scale (finite, not negative; uniform)
  // is in proportion to.  False when the page's values count as zeros: vs is then
  // a scale in proportion.
  __device__ __forceinline__ bool settle(float& vs) {
    if (vs < kScaleLeast) {
      vs = vref;
      return false;
    }
    const float to = unit_for(vs);
    const int up = (int)(__builtin_bit_cast(uint32_t, vref) >> 23) - (int)(__builtin_bit_cast(uint32_t, to) >> 23);
    vref = to;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[d][rt][r] = __builtin_amdgcn_ldexpf(o[d][rt][r], up);  // (exact)
    return true;
  }

  // The operands of a product are read from LDS this many ahead of their use.
  static constexpr int AHEAD = 2;
  static constexpr int N = 4 * KS;  // operands of a page's keys; as many of its values

  // S^T of a page.  key(i): operand i, of unit 4 (i / 8) + g, half i / 4 % 2, of
  // token 16 (i % 4) + c16.  q[rt][k]: the B operand of k-step k (load_query).
  template <typename Key>
  static __device__ __forceinline__ void scores(const Key& key, const half8 (&q)[RT][KS], float4v (&s)[4][RT]) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) s[t][rt] = float4v{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const half8 kf = key(i);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        s[i & 3][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, q[rt][i >> 2], s[i & 3][rt], 0, 0, 0);
    }
  }

  // Raises the maxima of rows that a page's scores (their largest a lane: high)
  // pass by far.
  __device__ __forceinline__ void raise(const float (&high)[RT]) {
    bool far = false;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) far |= high[rt] > m[rt] + kMaxSlack;
    if (__ballot(far)) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float mx = fmaxf(high[rt], __shfl_xor(high[rt], 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float up = fmaxf(m[rt], mx);
        const float f = __builtin_amdgcn_exp2f(m[rt] - up);
        m[rt] = up;
        sum[rt] *= f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d][rt] *= f;
      }
    }
  }

  // The weights of a page's scores s, as the B operands of the second product
  // (p[h]: tokens of tiles 2 h and 2 h + 1), times vs / vref, 1 to kScaleSlack:
  // exp2(score - m + lift), lift = log2(vs / vref), with their FP32 sum times
  // vref / vs (drop) added to the sums; and the scores of the next page.  (ONE:
  // exp2(score lift - m), and no sums.)  The
  // two in turn, operand by operand, so that the vector and the matrix unit
  // work at the same time: left to itself the compiler puts one behind the other.
  template <typename Key>
  __device__ __forceinline__ void weigh(float4v (&s)[4][RT], float lift, float drop, half8 (&p)[2][RT],
                                        const Key& key, const half8 (&q)[RT][KS], float4v (&next)[4][RT]) {
    half8 kf[AHEAD + 1];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) kf[i] = key(i);
    float off[RT], part[RT][2];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      off[rt] = ONE ? -m[rt] : lift - m[rt];
      part[rt][0] = part[rt][1] = 0.0f;
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) next[t][rt] = float4v{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i + AHEAD < N) kf[(i + AHEAD) % (AHEAD + 1)] = key(i + AHEAD);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        next[i & 3][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[i % (AHEAD + 1)], q[rt][i >> 2], next[i & 3][rt], 0, 0, 0);
#pragma unroll
      for (int v = i * 16 * RT / N; v < (i + 1) * 16 * RT / N; ++v) {
        const int rt = v / 16, t = v / 4 % 4, r = v % 4;
        const float x = __builtin_amdgcn_exp2f(ONE ? __builtin_fmaf(s[t][rt][r], lift, off[rt]) : s[t][rt][r] + off[rt]);
        if constexpr (!ONE) part[rt][r & 1] += x;
        s[t][rt][r] = x;
        if (v % 8 == 7) p[t >> 1][rt] = to_half8(s[t - 1][rt], s[t][rt]);
        if constexpr (!ONE)
          if (v % 16 == 15) sum[rt] = __builtin_fmaf(part[rt][0] + part[rt][1], drop, sum[rt]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // O^T += V^T P^T (ONE: and the sums of the weights); and the next page's scores get
  // their factor kc (ONE: none), and their largest is found.  value(i): the
  // operand of dimension 16 (i / 2) + c16, tokens 16 t + 4 g + r of the tiles
  // t = 2 (i % 2) and one more.
  template <typename Value>
  __device__ __forceinline__ void accumulate(const Value& value, const half8 (&p)[2][RT], float4v (&next)[4][RT], float kc,
                                             float (&high)[RT]) {
    half8 vf[AHEAD + 1];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) vf[i] = value(i);
    if constexpr (ONE) {
      const half8 ones = {1, 1, 1, 1, 1, 1, 1, 1};
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) sum[rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, p[h][rt], sum[rt], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i + AHEAD < N) vf[(i + AHEAD) % (AHEAD + 1)] = value(i + AHEAD);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        o[i >> 1][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[i % (AHEAD + 1)], p[i & 1][rt], o[i >> 1][rt], 0, 0, 0);
#pragma unroll
      for (int v = i * 8 * RT / N; v < (i + 1) * 8 * RT / N; ++v) {  // a pair of scores at a time
        const int rt = v / 8, t = v / 2 % 4, r = v % 2 * 2;
        if constexpr (!ONE) next[t][rt][r] *= kc, next[t][rt][r + 1] *= kc;
        high[rt] = v % 8 ? fmaxf(fmaxf(high[rt], next[t][rt][r]), next[t][rt][r + 1]) : fmaxf(next[t][rt][r], next[t][rt][r + 1]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// NaN into the sums o of the rows that see it; nan: FP16 ones where a value is
// NaN, zeros elsewhere; seen: the tokens of the half page that the row sees.
__device__ __forceinline__ void spread_nan(const half8& nan, uint32_t seen, float4v& o) {
  u32x4 sees;  // FP16 1 where the row sees the token
#pragma unroll
  for (int e = 0; e < 4; ++e)
    sees[e] = (all_ones_if(seen, e >> 1, 2 * (e & 1)) & 0x3C00u) |
              (all_ones_if(seen, e >> 1, 2 * (e & 1) + 1) & 0x3C000000u);
  const float4v hit = __builtin_amdgcn_mfma_f32_16x16x32_f16(nan, __builtin_bit_cast(half8, sees), float4v{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (hit[r] > 0.0f) o[r] = __builtin_nanf("");
  // one product at a time: this is rare, and its registers are the loop's
  asm volatile("" : "+v"(o));
}

// Workgroup barrier that waits for this wavefront's LDS accesses alone: loads
// of pages stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int RT, typename A>
__device__ __forceinline__ View<RT> view_of(const A& a, const AttnLaunch& l, const Req& q, int lane,
                                            int first, int rows) {
  const int c16 = lane & 15, at = q.seq - q.rows + 1;
  View<RT> v;
  v.window = a.window;
#pragma unroll
  for (int t = 0; t < RT; ++t)
    v.lim[t] = t * 16 + c16 < rows ? at + row_of(l, first + t * 16 + c16) : 0;
  v.lim_min = uniform(at + row_of(l, first));
  v.lim_max = uniform(at + row_of(l, first + rows - 1));
  v.low_min = low_of(v.lim_min, a.window);
  v.low_max = low_of(v.lim_max, a.window);
  return v;
}

typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef float float2v __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kDevScope = 16;  // sc1: write-through stores, coherent loads

// A piece's sums in scratch: per row tile `rt` (16 rows) and dimension tile d the
// 64 lanes' four accumulators in lane order, then per row its maximum and its
// weights' sum.  A whole number of 128-byte lines.
template <int DIM, int TILES>
struct Slot {
  static constexpr int DT = DIM / 16;
  static constexpr int kSums = TILES * DT * 1024;     // bytes
  static constexpr int kBytes = kSums + TILES * 128;
  __device__ static int fragment(int rt, int d, int lane) { return (rt * DT + d) * 1024 + lane * 16; }
  __device__ static int row(int rt, int c16) { return kSums + (rt * 16 + c16) * 8; }
};

// Four dimensions of row `rr` of a segment: y.
template <typename A>
__device__ __forceinline__ void write_y(const A& a, const AttnLaunch& l, const Req& q, int head, int rr,
                                        int dim0, int dim, float4v sum, float weight) {
  const int row = row_of(l, rr);
  half4 h;
  float inverse = 1.0f / weight;
  if (weight == 0.0f || q.bad) {
    // nothing seen gives zeros; tokens seen but no weight (every score -inf) has no value, and
    // neither has a row of a request longer than its table (whose rows' places are not known)
    sum = float4v{0, 0, 0, 0};
    inverse = q.bad || q.seq - q.rows + row + 1 > 0 ? __builtin_nanf("") : 0.0f;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = (_Float16)(sum[e] * inverse);
  *reinterpret_cast<half4*>(a.y + (int64_t)(q.row0 + row) * a.y_stride +
                            (int64_t)(head * l.group + rr - row * l.group) * dim + dim0) = h;
}

// Arrivals.  True for the last of n workgroups that count themselves in at
// `counter`, whose stores are then all at the device's point of coherence; the
// counter is left at 0.
__device__ __forceinline__ bool arrive_last(uint32_t* counter, int n, uint32_t* s_arrival) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wavefront's stores are there
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint32_t before = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (before == (uint32_t)(n - 1)) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *s_arrival = before;
  }
  __syncthreads();
  const bool last = *s_arrival == (uint32_t)(n - 1);
  if (last) __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  return last;
}

// Joins the fragments of A row tiles (rt0 on) and B dimension tiles (d0 on) of
// `count` partial sums in order.  slot(i): the i-th one's slot.  The loads of
// CH sums go out together.
template <int DIM, int TILES, int A, int B, int CH, typename SlotOf>
__device__ __forceinline__ void join_fragments(__amdgpu_buffer_rsrc_t res, int lane, int rt0, int d0, int count,
                                               const SlotOf& slot, float4v (&sum)[A][B], float (&top)[A],
                                               float (&weight)[A]) {
  using S = Slot<DIM, TILES>;
  const int c16 = lane & 15;
#pragma unroll
  for (int t = 0; t < A; ++t) {
    top[t] = kLowest, weight[t] = 0.0f;
#pragma unroll
    for (int d = 0; d < B; ++d) sum[t][d] = float4v{0, 0, 0, 0};
  }
#pragma unroll 1
  for (int i0 = 0; i0 < count; i0 += CH) {
    float4v o[CH][A][B];
    float2v ml[CH][A];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (i0 + i < count) {
        const int at = slot(i0 + i) * S::kBytes;
#pragma unroll
        for (int t = 0; t < A; ++t) {
          ml[i][t] = __builtin_bit_cast(float2v, __builtin_amdgcn_raw_buffer_load_b64(res, S::row(rt0 + t, c16), at, kDevScope));
#pragma unroll
          for (int d = 0; d < B; ++d)
            o[i][t][d] = __builtin_bit_cast(
                float4v, __builtin_amdgcn_raw_buffer_load_b128(res, S::fragment(rt0 + t, d0 + d, lane), at, kDevScope));
        }
      } else {
#pragma unroll
        for (int t = 0; t < A; ++t) {
          ml[i][t] = float2v{kLowest, 0.0f};
#pragma unroll
          for (int d = 0; d < B; ++d) o[i][t][d] = float4v{0, 0, 0, 0};
        }
      }
    }
#pragma unroll
    for (int t = 0; t < A; ++t) {
      float up = top[t];
#pragma unroll
      for (int i = 0; i < CH; ++i) up = fmaxf(up, ml[i][t][0]);
      const float old = __builtin_amdgcn_exp2f(top[t] - up);
      top[t] = up;
      weight[t] *= old;
#pragma unroll
      for (int d = 0; d < B; ++d) sum[t][d] *= old;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const float w = __builtin_amdgcn_exp2f(ml[i][t][0] - up);
        weight[t] += ml[i][t][1] * w;
#pragma unroll
        for (int d = 0; d < B; ++d) sum[t][d] += o[i][t][d] * w;
      }
    }
  }
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t partial_of(const AttnLaunch& l) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)l.partial, (short)0, 0x7FFFFFFF, kRsrc);
}

// After the pieces' sums are stored: the last workgroup of a segment (of a
// group of its pieces first, when there are many) joins them in order and
// writes y.  Each wavefront takes dimension tiles of its own, all rows.
template <int DIM, int TILES, int WAVES, typename A>
__device__ __forceinline__ void join_pieces(const A& a, const AttnLaunch& l, const Item& it, const Req& q,
                                            int lane, int wave, int row_first, int rows_here, uint32_t* s_arrival) {
  using S = Slot<DIM, TILES>;
  const int c16 = lane & 15, g = lane >> 4;
  const __amdgpu_buffer_rsrc_t res = partial_of(l);
  uint32_t* const counters = (uint32_t*)a.scratch;
  // groups of pieces: one when all are joined directly, else about the root
  // of their number; group k has pieces k n / groups .. (k + 1) n / groups - 1
  int groups = 1, k = 0;
  if (it.pieces > KindOf<A>::kJoinDirect) {
    while (groups * groups < it.pieces) ++groups;
    k = (int)((uint32_t)(it.piece * groups) / (uint32_t)it.pieces);
    if ((int)((uint32_t)((k + 1) * it.pieces) / (uint32_t)groups) <= it.piece) ++k;
  }
  auto start_of = [&](int j) { return (int)((uint32_t)(j * it.pieces) / (uint32_t)groups); };
  const int p0 = start_of(k), p1 = start_of(k + 1);
  if (!arrive_last(counters + (it.first + p0) * kCounterStep, p1 - p0, s_arrival)) return;
  // slots of groups lie behind those of pieces; a group has two pieces or
  // more, so half its first piece's number is a slot of its own
  int count = p1 - p0;
  const int first = it.first + p0;
  bool inner = groups > 1, outer = false;
  for (;;) {
    auto slot = [&](int i) { return outer ? l.slots + (it.first + start_of(i)) / 2 : first + i; };
#pragma unroll 1
    for (int d = wave; d < S::DT; d += WAVES) {
      float4v sum[TILES][1];
      float top[TILES], weight[TILES];
      join_fragments<DIM, TILES, TILES, 1, KindOf<A>::at_once(TILES)>(res, lane, 0, d, count, slot, sum, top, weight);
      const int at = (l.slots + first / 2) * S::kBytes;
#pragma unroll
      for (int rt = 0; rt < TILES; ++rt) {
        if (inner) {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, sum[rt][0]), res, S::fragment(rt, d, lane), at,
                                                 kDevScope);
          if (d == 0 && g == 0)
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, float2v{top[rt], weight[rt]}), res,
                                                  S::row(rt, c16), at, kDevScope);
        } else if (rt * 16 + c16 < rows_here) {
          write_y(a, l, q, it.head, row_first + rt * 16 + c16, KindOf<A>::template first_dim<DIM>(d, g), DIM, sum[rt][0], weight[rt]);
        }
      }
    }
    if (!inner) return;
    if (!arrive_last(counters + (kMaxPieces + it.first) * kCounterStep, groups, s_arrival)) return;
    inner = false;
    outer = true;
    count = groups;
  }
}

// Joins the pieces of cut segments of many rows: the workgroup of a piece
// takes its share of the segment's fragments.  (A launch of its own: the last
// workgroup alone would need tens of microseconds for a tile of 192 rows.)
template <int DIM, int TILES, typename A>
__global__ __launch_bounds__(kManyWaves * 64) void attention_join_kernel(A a, AttnLaunch l) {
  using S = Slot<DIM, TILES>;
  constexpr int B = 2, SHARES = TILES * S::DT / B;  // a share: two dimension tiles of a row tile
  const int wave = uniform((int)threadIdx.x >> 6), lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
  for (int block = blockIdx.x;; block += gridDim.x) {
    Req q;
    const Item it = item_of(a, l, lane, block, q);
    if (it.request < 0) break;
    if (it.pieces == 1) continue;
    const int row_first = it.tile * 16 * TILES;
    const int rows_here = min(16 * TILES, q.rows * l.group - row_first);
    for (int share = it.piece * kManyWaves + wave; share < SHARES; share += it.pieces * kManyWaves) {
      const int rt = share * B / S::DT, d0 = share * B % S::DT;
      if (rt * 16 >= rows_here) break;
      float4v sum[1][B];
      float top[1], weight[1];
      join_fragments<DIM, TILES, 1, B, KindOf<A>::at_once(B)>(partial_of(l), lane, rt, d0, it.pieces, [&](int i) { return it.first + i; }, sum,
                                       top, weight);
      if (rt * 16 + c16 < rows_here) {
#pragma unroll
        for (int d = 0; d < B; ++d)
          write_y(a, l, q, it.head, row_first + rt * 16 + c16, KindOf<A>::template first_dim<DIM>(d0 + d, g), DIM, sum[0][d], weight[0]);
      }
    }
  }
}

// Segments of a call whose requests all bring max_rows rows.
int64_t most_segments(const Form& f, int requests, int max_rows, int q_heads, int heads) {
  const int64_t rows = (int64_t)max_rows * (q_heads / heads);
  const int64_t tiles = (rows + f.rows() - 1) / f.rows();
  return (int64_t)requests * heads * (tiles < 1 ? 1 : tiles);
}

// Pieces wanted: what the chip holds at once (a workgroup a CU), or two for each
// when there are so many segments that whole ones, or the few that can still be
// cut, would leave it unevenly loaded.  With 256 / 512 pieces, ragged requests of
// up to 8 rows x 5 query heads: 160 segments of up to 4000 tokens 38 / 48 us, 200 of
// up to 9000 108 / 78 us, 272 of up to 9000 129 / 103 us, 320 of up to 2000
// 45 / 48 us; 480 segments of 64 rows 133 / 132 us.
int wanted_pieces(int64_t segments) { return segments <= 192 ? 256 : kMaxPieces; }

size_t slot_bytes(const Form& f, int dim) { return (size_t)f.rows() * dim * 4 + (size_t)f.rows() * 8; }

template <typename Kernel, typename A>
hipError_t launch_kernel(Kernel kernel, int threads, size_t lds, const A& a, const AttnLaunch& l,
                         int64_t grid) {
  if (lds > 0) {
    const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  kernel<<<dim3((uint32_t)grid), dim3(threads), lds, (hipStream_t)a.stream>>>(a, l);
  return hipGetLastError();
}

template <typename A>
size_t scratch_bytes_for(int requests, int max_rows, int q_heads, int heads, int dim, int table_width) {
  const Form f = form_of<A>(requests, max_rows, q_heads, heads, dim, table_width);
  const int64_t segments = most_segments(f, requests, max_rows, q_heads, heads);
  if (table_width <= kMinPiecePages || segments >= kMaxPieces) return kKvZeroedBytes;
  const size_t slots = wanted_pieces(segments);
  return kKvZeroedBytes + (slots + slots / 2) * slot_bytes(f, dim);
}

// The launch of a call: its form, split and grid.
struct AttnPlan {
  Form form;
  AttnLaunch launch;
  int64_t grid;
};
template <typename A>
AttnPlan plan_of(const A& a) {
  const int dim = a.cache.dim, group = a.q_heads / a.cache.heads;
  const Form f = form_of<A>(a.requests, a.max_rows, a.q_heads, a.cache.heads, dim, a.table_width);
  const int64_t segments = most_segments(f, a.requests, a.max_rows, a.q_heads, a.cache.heads);
  AttnLaunch l;
  l.tile_rows = f.rows();
  l.group = group;
  l.inverse = (uint32_t)(((uint64_t(1) << 32) + group - 1) / group);  // (not used for 1)
  l.target = wanted_pieces(segments);
  const size_t room = a.scratch_bytes > kKvZeroedBytes ? (a.scratch_bytes - kKvZeroedBytes) / slot_bytes(f, dim) : 0;
  l.slots = (int)((room > 3 * kMaxPieces ? 3 * kMaxPieces : room) * 2 / 3);
  if (l.slots < l.target) l.target = l.slots;
  if (a.table_width <= kMinPiecePages || segments >= kMaxPieces) l.slots = 0;  // nothing is cut
  l.partial = (float*)((uint8_t*)a.scratch + kKvZeroedBytes);
  // an upper bound of the pieces when the hint of the rows is right, in eights
  int64_t grid = segments;
  if (l.slots > 0) {
    const int64_t most = segments * ((a.table_width + kMinPiecePages - 1) / kMinPiecePages);
    const int64_t cut = most < l.target ? most : l.target;
    grid = cut > grid ? cut : grid;
  }
  grid = (grid + 7) / 8 * 8;
  grid = grid < 8 ? 8 : grid > (1 << 20) ? (1 << 20) : grid;
  return {f, l, grid};
}

}  // namespace

}  // namespace qpn
