// qpn_kv_attn.hip -- attention of a round's rows over the 8-bit paged KV cache
// on gfx950.
//
// y = sum_j w_j v_j / sum_j w_j, w_j = exp(scale q . k_j - m), over the tokens a
// row sees.  K and V codes stay E4M3 until they are in registers, where the
// conversion to FP16 is exact; both products run on the 16x16x32 f16 MFMA with
// FP32 accumulation.  The page scale of K multiplies the scores, that of V the
// weights (as a term of their exponent).
//
// One pass, transposed.  A wavefront holds 16 RT rows (query row, query head of
// the KV head's group) and computes, page by page of 64 tokens, S^T = K Q^T: K is
// the A operand, so a lane's accumulators are 16 tokens of one row, and after
// the exponentials they are, without any exchange between lanes, the B operand of
// O^T = V^T P^T.  The cache layout stores each block in the order these operands
// are read: 16 bytes a lane, over whole lines.  The running maximum of a row is
// only raised when a score exceeds it by more than 2^8 (weights up to 2^8 fit
// FP16 as well as those up to 1), so most pages cost no exchange between lanes
// and no rescaling.  FP16 weights, the second product's input, are off by 2^-11 of
// each (below 2^-14 by 2^-25), as far as the output is by its own rounding.
//
// Two forms, by the rows of a KV head:
//   few rows (up to kFewTiles tiles): each wavefront takes pages of its own,
//     all rows of the segment, straight into registers, the next page's keys on
//     their way while the values of this one are used; the workgroup's
//     wavefronts are joined through LDS.  Reading the cache is the bound.
//   many rows: a workgroup's wavefronts take different rows and share each page
//     through LDS.  The matrix and vector units are the bound.
//
// Work split.  A segment (request, KV head, tile of rows) is cut into pieces of
// about P pages, one workgroup each.  P comes from the lengths on the device, so
// that ragged requests fill the chip evenly with no host read.  The pieces of a
// cut segment leave their sums in scratch, written through to the device's point
// of coherence, and count themselves in; the last to arrive joins them in
// order (of more than kJoinDirect pieces: in groups, then the groups).
#include "qpn_common.h"
#include "qpn_kv_internal.h"

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

// wavefronts of a workgroup, few rows: one per 16 dimensions up to eight
constexpr int few_waves(int dim) { return dim == 64 ? 4 : 8; }
constexpr int kManyWaves = 8;  // and many rows
// Pages of a piece at least: one for each of the eight wavefronts of few rows.
// (8 rows of 40 + 8 heads over 4099 tokens: 20.3 us with 4, 19.0 with 8, 20.8
// with 16; 256 rows over 4096: 46.3, 46.2, 53.2.)
constexpr int kMinPiecePages = 8;
constexpr int kMaxPieces = 512;    // pieces of a call with cut segments
// Pieces joined in one step.  (8 rows over 16384 tokens, 32 pieces a head: 30.6 us
// in one step, 26.0 us in two; over 131001 tokens 78.6 and 75.1 us.)
constexpr int kJoinDirect = 16;
constexpr int kCounterStep = 8;    // 32-bit words between counters
static_assert((size_t)kMaxPieces * 2 * kCounterStep * 4 <= kKvZeroedBytes, "two counters per piece");

// The form and the 16-row tiles of a wavefront (of a workgroup, few rows) for
// `rows` rows of a KV head (query rows x group).  Up to what the registers of
// the few-rows form hold it is the faster one: 40 rows a head over 4099 / 131001
// tokens take 19.0 / 75.1 us there and 23.4 / 104 us with many rows' form, 48
// ragged requests of up to 40 rows 38.8 and 55.5 us.
constexpr int few_tiles(int dim) { return dim == 256 ? 1 : 3; }   // what the registers hold
constexpr int many_tiles(int dim) { return dim == 256 ? 1 : 2; }
struct Form {
  bool many;
  int tiles;
  int rows() const { return 16 * tiles * (many ? kManyWaves : 1); }
};
inline Form form_for(int64_t rows, int dim) {
  const int64_t t = (rows + 15) / 16;
  if (t <= few_tiles(dim)) return {false, t < 1 ? 1 : (int)t};
  return {true, t <= kManyWaves ? 1 : many_tiles(dim)};
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

__device__ __forceinline__ Req request_of(const AttentionArgs& a, const AttnLaunch& l, int r) {
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
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
  return x;
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
__device__ __forceinline__ Cut cut_of(const AttentionArgs& a, const AttnLaunch& l, int lane) {
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
__device__ __forceinline__ Item item_of(const AttentionArgs& a, const AttnLaunch& l, int lane, int block, Req& out) {
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

// The rows of a wavefront and their running sums.
template <int DIM, int RT>
struct Rows {
  static constexpr int KS = DIM / 32;  // k-steps of the scores
  static constexpr int DT = DIM / 16;  // tiles of output dimensions
  float m[RT], sum[RT];
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
      sum[t] = 0.0f;
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
  // vref / vs (drop) added to the sums; and the scores of the next page.  The
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
      off[rt] = lift - m[rt];
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
        const float x = __builtin_amdgcn_exp2f(s[t][rt][r] + off[rt]);
        part[rt][r & 1] += x;
        s[t][rt][r] = x;
        if (v % 8 == 7) p[t >> 1][rt] = to_half8(s[t - 1][rt], s[t][rt]);
        if (v % 16 == 15) sum[rt] = __builtin_fmaf(part[rt][0] + part[rt][1], drop, sum[rt]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // O^T += V^T P^T; and the next page's scores get their factor kc, and their
  // largest is found.  value(i): the
  // operand of dimension 16 (i / 2) + c16, tokens 16 t + 4 g + r of the tiles
  // t = 2 (i % 2) and one more.
  template <typename Value>
  __device__ __forceinline__ void accumulate(const Value& value, const half8 (&p)[2][RT], float4v (&next)[4][RT], float kc,
                                             float (&high)[RT]) {
    half8 vf[AHEAD + 1];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) vf[i] = value(i);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i + AHEAD < N) vf[(i + AHEAD) % (AHEAD + 1)] = value(i + AHEAD);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        o[i >> 1][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[i % (AHEAD + 1)], p[i & 1][rt], o[i >> 1][rt], 0, 0, 0);
#pragma unroll
      for (int v = i * 8 * RT / N; v < (i + 1) * 8 * RT / N; ++v) {  // a pair of scores at a time
        const int rt = v / 8, t = v / 2 % 4, r = v % 2 * 2;
        next[t][rt][r] *= kc, next[t][rt][r + 1] *= kc;
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

// All bits of the bytes of tokens that are seen, a word for each tile t of a
// half page.
__device__ __forceinline__ uint32_t keep_bytes(uint32_t seen, int t) {
  return ((((seen >> (16 * t)) & 15u) * 0x00204081u) & 0x01010101u) * 255u;
}
// Values of a page that some rows see only a part of, codes of the D tiles of a
// wavefront: what no row sees becomes zeros (what is there may be anything); NaN
// that some rows see and others do not is taken out too, and put into the sums
// of the rows that see it.
template <int D, int RT>
__device__ __forceinline__ void clean_values(u32x4 (&v)[D], int base, int g, const View<RT>& see, float4v (&o)[D][RT]) {
  uint32_t any = 0;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const uint32_t keep = keep_bytes(seen_of(see.lim_max, see.low_min, base + 32 * (t >> 1), g), t & 1);
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const uint32_t x = v[d][t] & keep;
      v[d][t] = x;
      any |= nan_bytes(x);
    }
  }
  if (__builtin_expect(__ballot(any != 0) == 0, 1)) return;
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const uint32_t n0 = nan_bytes(v[d][2 * half]) >> 7, n1 = nan_bytes(v[d][2 * half + 1]) >> 7;
      const half8 nan = decode_e4m3x8(n0 * 0x38u, n1 * 0x38u);  // E4M3 ones
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) spread_nan(nan, seen_of(see.lim[rt], see.low(rt), base + 32 * half, g), o[d][rt]);
      v[d][2 * half] &= ~(n0 * 255u);
      v[d][2 * half + 1] &= ~(n1 * 255u);
    }
}

// The numbers and scales of up to 64 pages of a request, one a lane: entries
// first + lane * step below end.
struct Pages {
  int id;  // 0 (with a NaN factor) for one that is not in the cache
  float kc, vs;
  __device__ __forceinline__ void load(const AttentionArgs& a, const int32_t* table, int head, bool bad, int lane,
                                       int first, int step, int end) {
    const int page = first + lane * step;  // (both below 2^25)
    id = 0;
    kc = __builtin_nanf("");
    vs = 1.0f;
    if (page < end && page < a.table_width) {
      const int32_t x = table[page];
      if (x >= 0 && x < a.cache.pages && !bad) {
        const int64_t block = (int64_t)x * a.cache.heads + head;
        id = x;
        kc = a.cache.k_scale[block] * (a.scale * 1.44269504088896340736f);
        vs = a.cache.v_scale[block];
        // A scale that is negative, infinite or NaN: NaN through the scores, which the mask
        // keeps from rows that do not see the page, and not through the values, whose zero
        // weights there it would turn into NaN too.
        if (!(vs >= 0.0f && vs < __builtin_inff())) kc = __builtin_nanf(""), vs = 1.0f;
      }
    }
  }
  // byte offset of the page's block
  template <int DIM>
  __device__ __forceinline__ int64_t offset_at(const AttentionArgs& a, int head, int i) const {
    return ((int64_t)__builtin_amdgcn_readlane(id, i) * a.cache.heads + head) * (kKvPage * DIM);
  }
  static __device__ __forceinline__ float at(float x, int i) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), i));
  }
};

template <int RT>
__device__ __forceinline__ View<RT> view_of(const AttentionArgs& a, const AttnLaunch& l, const Req& q, int lane,
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

// Q: B operand of row tile t: lane (row c16, k 8 g + e) of k-step 2 u + h has
// dimensions 64 u + 16 g + 8 h + e, as the key units' 16 dimensions fall to the
// lanes.  Rows behind `rows` are zeros.
template <int DIM>
__device__ __forceinline__ void load_query(const AttentionArgs& a, const AttnLaunch& l, const Req& r, int head,
                                           int lane, int first, int rows, int t, half8 (&q)[DIM / 32]) {
  const int c16 = lane & 15, g = lane >> 4;
  const bool in = t * 16 + c16 < rows;
  const int rr = in ? first + t * 16 + c16 : 0, row = row_of(l, rr);
  const uint16_t* src = a.q + (int64_t)(r.row0 + row) * a.q_stride +
                        (int64_t)(head * l.group + (rr - row * l.group)) * DIM + 16 * g;
#pragma unroll
  for (int k = 0; k < DIM / 32; ++k)
    q[k] = in ? *reinterpret_cast<const half8*>(src + 64 * (k >> 1) + 8 * (k & 1)) : half8{};
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
__device__ __forceinline__ void write_y(const AttentionArgs& a, const AttnLaunch& l, const Req& q, int head, int rr,
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
template <int DIM, int TILES, int A, int B, typename SlotOf>
__device__ __forceinline__ void join_fragments(__amdgpu_buffer_rsrc_t res, int lane, int rt0, int d0, int count,
                                               const SlotOf& slot, float4v (&sum)[A][B], float (&top)[A],
                                               float (&weight)[A]) {
  using S = Slot<DIM, TILES>;
  constexpr int CH = A * B >= 3 ? 4 : 8;
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
template <int DIM, int TILES, int WAVES>
__device__ __forceinline__ void join_pieces(const AttentionArgs& a, const AttnLaunch& l, const Item& it, const Req& q,
                                            int lane, int wave, int row_first, int rows_here, uint32_t* s_arrival) {
  using S = Slot<DIM, TILES>;
  const int c16 = lane & 15, g = lane >> 4;
  const __amdgpu_buffer_rsrc_t res = partial_of(l);
  uint32_t* const counters = (uint32_t*)a.scratch;
  // groups of pieces: one when all are joined directly, else about the root
  // of their number; group k has pieces k n / groups .. (k + 1) n / groups - 1
  int groups = 1, k = 0;
  if (it.pieces > kJoinDirect) {
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
      join_fragments<DIM, TILES, TILES, 1>(res, lane, 0, d, count, slot, sum, top, weight);
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
          write_y(a, l, q, it.head, row_first + rt * 16 + c16, 16 * d + 4 * g, DIM, sum[rt][0], weight[rt]);
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

// ---------------------------------------------------------------------------
// Few rows: the workgroup takes a page per wavefront at a time.
//
// First product: wavefront w computes the weights of page w of these, all rows,
// against a running maximum of its own (a row's pages need not agree on one),
// and leaves them in LDS as the operands of the second product.  Second product:
// wavefront w takes the 16 dimensions w of all the pages; a page's sums are added
// with the factor exp2(its maximum - the common one) times its V scale.  So every
// code is converted once, no wavefront holds more than its dimensions' sums, and
// nothing is left to join but the weights' sums.  Two buffers: one barrier for W
// pages.  The next keys are on their way once this page's are used, the next
// values of a page once its present ones are.
//
// Bound: over long caches the steps of eight pages, whose weights and values are
// apart by a barrier (8 rows of 40 + 8 heads of 128 over 131001 tokens, 269 MB, not
// in any cache: 81.0 us, 3.3 TB/s, where a large copy reaches 4.9 and a reduction
// reads 5.8; from a graph, with part of it cached, 72.7 us, one row 51.9: the
// bytes alone are not it).  Short calls are bound by their chain of dependent
// steps: launch, table, keys, values, hand-over, join (200 tokens 8.8 us; 4099
// tokens, nine pieces a head, 18.9 us).
// ---------------------------------------------------------------------------
template <int DIM, int RT>
struct FewLds {
  static constexpr int W = few_waves(DIM), KS = DIM / 32, ROWS = 16 * RT;
  half8 p[2][W][2][RT][64];  // operands of the second product: page, k-step, row tile, lane
  half8 q[KS][RT][64];       // operands of the first
  float m[2][ROWS][W];       // the pages' maxima
  float last[ROWS][W], sum[ROWS][W];
};

template <int DIM, int RT>
__global__ __launch_bounds__(few_waves(DIM) * 64) void attention_few_kernel(AttentionArgs a, AttnLaunch l) {
  using S = Slot<DIM, RT>;
  using L = FewLds<DIM, RT>;
  constexpr int W = L::W, KS = L::KS, ROWS = L::ROWS, DW = DIM / 16 / W;  // dimension tiles of a wavefront
  __shared__ uint32_t s_arrival;
  extern __shared__ __attribute__((aligned(16))) uint8_t s_few[];
  L& s = *reinterpret_cast<L*>(s_few);
  const int wave = uniform((int)threadIdx.x >> 6);

  for (int block = blockIdx.x;; block += gridDim.x) {
    // (opaque, so that nothing that follows from it is kept in registers around the loop)
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int c16 = lane & 15, g = lane >> 4;
    Req q;
    const Item it = item_of(a, l, lane, block, q);
    if (it.request < 0) break;  // past the last item: the whole workgroup leaves
    const int row_first = it.tile * ROWS;  // among the segment's rows
    const int rows_here = min(ROWS, q.rows * l.group - row_first);
    const View<RT> see = view_of<RT>(a, l, q, lane, row_first, rows_here);
    // the piece's pages that the tile sees
    const int lo = max(q.first_page + (int)((int64_t)q.pages * it.piece / it.pieces), see.low_min / kKvPage);
    const int hi = min(q.first_page + (int)((int64_t)q.pages * (it.piece + 1) / it.pieces),
                       (see.lim_max + kKvPage - 1) / kKvPage);
    const int count = max(0, hi - lo);
    const int32_t* const table = a.table + it.request * a.table_stride;
    // (the queries first: loads return in order)
    static_assert(RT <= W, "a row tile of queries per wavefront");
    half8 qr[KS];
    if (wave < RT) load_query<DIM>(a, l, q, it.head, lane, row_first, rows_here, wave, qr);
    Pages now;  // of the 64 pages around the present ones
    now.load(a, table, it.head, q.bad, lane, lo, 1, hi);

    u32x4 k[DIM / 64][4], v[W][DW];
    const int k_at = g * (kKvPage * 16) + c16 * 16, v_at = c16 * kKvPage + 16 * g;
    auto load_keys = [&](int64_t offset) {
      const __amdgpu_buffer_rsrc_t res =
          __builtin_amdgcn_make_buffer_rsrc((void*)(a.cache.k + offset), (short)0, kKvPage * DIM, kRsrc);
#pragma unroll
      for (int u = 0; u < DIM / 64; ++u)
#pragma unroll
        for (int t = 0; t < 4; ++t)
          k[u][t] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(res, k_at + t * 256, u * 4 * kKvPage * 16, 0));
    };
    auto load_values = [&](int64_t offset, u32x4(&to)[DW]) {
      const __amdgpu_buffer_rsrc_t res =
          __builtin_amdgcn_make_buffer_rsrc((void*)(a.cache.v + offset), (short)0, kKvPage * DIM, kRsrc);
#pragma unroll
      for (int d = 0; d < DW; ++d)
        to[d] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(res, v_at, (wave * DW + d) * (16 * kKvPage), 0));
    };
    if (count > 0) {
      load_keys(now.template offset_at<DIM>(a, it.head, min(wave, count - 1)));
#pragma unroll
      for (int j = 0; j < W; ++j) load_values(now.template offset_at<DIM>(a, it.head, min(j, count - 1)), v[j]);
    }
    if (wave < RT) {
#pragma unroll
      for (int i = 0; i < KS; ++i) s.q[i][wave][lane] = qr[i];
    }
    lds_barrier();

    float m[RT], sum[RT], top[RT];  // this wavefront's maxima and sums, the common maximum
    float4v o[DW][RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      m[rt] = top[rt] = kLowest;
      sum[rt] = 0.0f;
#pragma unroll
      for (int d = 0; d < DW; ++d) o[d][rt] = float4v{0, 0, 0, 0};
    }

    for (int i0 = 0; i0 < count; i0 += W) {
      const int buffer = (i0 / W) & 1, at = i0 & 63;  // (64 is a multiple of W)
      const int here = min(W, count - i0), left = count - i0 - W;  // pages of this step, behind it
      Pages next = now;  // the next step's pages: lanes (at + W) & 63 on
      if (at + W == 64 && left > 0) next.load(a, table, it.head, q.bad, lane, lo + i0 + W, 1, hi);
      const int next_at = left > 0 ? (at + W) & 63 : at, last = left > 0 ? min(W, left) - 1 : here - 1;
      if (wave < here) {
        // the weights of page i0 + wave
        const float kc = Pages::at(now.kc, at + wave);
        const int base = (lo + i0 + wave) * kKvPage;
        float4v x[4][RT];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) x[t][rt] = float4v{0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < DIM / 64; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            half8 qf[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) qf[rt] = s.q[2 * u + h][rt][lane];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const half8 kf = decode_e4m3x8(k[u][t][2 * h], k[u][t][2 * h + 1]);
#pragma unroll
              for (int rt = 0; rt < RT; ++rt)
                x[t][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[rt], x[t][rt], 0, 0, 0);
            }
          }
        load_keys(next.template offset_at<DIM>(a, it.head, next_at + min(wave, last)));
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) x[t][rt] *= kc;
        if (base + kKvPage > see.lim_min || base < see.low_max) {  // what a row does not see is -inf
          mask_page<RT>(x, base, g, see);
        }
        float high[RT];
        bool raise = false;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          high[rt] = page_max<RT>(x, rt);
          raise |= high[rt] > m[rt] + kMaxSlack;
        }
        if (__ballot(raise)) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            float mx = fmaxf(high[rt], __shfl_xor(high[rt], 16));
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            const float up = fmaxf(m[rt], mx);
            sum[rt] *= __builtin_amdgcn_exp2f(m[rt] - up);
            m[rt] = up;
          }
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float w = __builtin_amdgcn_exp2f(x[t][rt][r] - m[rt]);
              part[t] += w;
              x[t][rt][r] = w;
            }
          sum[rt] += (part[0] + part[1]) + (part[2] + part[3]);
          s.p[buffer][wave][0][rt][lane] = to_half8(x[0][rt], x[1][rt]);
          s.p[buffer][wave][1][rt][lane] = to_half8(x[2][rt], x[3][rt]);
          if (g == 0) s.m[buffer][rt * 16 + c16][wave] = m[rt];
        }
      }
      lds_barrier();

      // the common maximum and the pages' factors
      float f[W][RT];
      bool grown = false;
      float up[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        up[rt] = top[rt];
#pragma unroll
        for (int j = 0; j < W; j += 4) {
          const float4v mj = *reinterpret_cast<const float4v*>(&s.m[buffer][rt * 16 + c16][j]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f[j + e][rt] = mj[e];
            if (j + e < here) up[rt] = fmaxf(up[rt], mj[e]);
          }
        }
        grown |= up[rt] > top[rt];
      }
      if (__ballot(grown)) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const float scale = __builtin_amdgcn_exp2f(top[rt] - up[rt]);
          top[rt] = up[rt];
#pragma unroll
          for (int d = 0; d < DW; ++d) o[d][rt] *= scale;
        }
      }
#pragma unroll
      for (int j = 0; j < W; ++j) {
        if (j < here) {
          const int base = (lo + i0 + j) * kKvPage;
          const float vs = Pages::at(now.vs, at + j);
          half8 pf[2][RT];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) pf[h][rt] = s.p[buffer][j][h][rt][lane];
          if (base + kKvPage > see.lim_min || base < see.low_max)
            clean_values<DW, RT>(v[j], base, g, see, o);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) f[j][rt] = __builtin_amdgcn_exp2f(f[j][rt] - top[rt]) * vs;
#pragma unroll
          for (int d = 0; d < DW; ++d) {
            half8 vf[2];
            decode_fp8_fragment(v[j][d], vf);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              float4v add{0, 0, 0, 0};
#pragma unroll
              for (int h = 0; h < 2; ++h) add = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[h], pf[h][rt], add, 0, 0, 0);
#pragma unroll
              for (int r = 0; r < 4; ++r) o[d][rt][r] = __builtin_fmaf(add[r], f[j][rt], o[d][rt][r]);
            }
          }
          load_values(next.template offset_at<DIM>(a, it.head, next_at + min(j, last)), v[j]);
        }
      }
      now = next;
    }

    // the weights' sums of all pages against the common maximum
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      sum[rt] += __shfl_xor(sum[rt], 16);
      sum[rt] += __shfl_xor(sum[rt], 32);
      if (g == 0) s.last[rt * 16 + c16][wave] = m[rt], s.sum[rt * 16 + c16][wave] = sum[rt];
      sum[rt] = 0.0f;
    }
    lds_barrier();
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int w = 0; w < W; w += 4) {
        const float4v mw = *reinterpret_cast<const float4v*>(&s.last[rt * 16 + c16][w]);
        const float4v sw = *reinterpret_cast<const float4v*>(&s.sum[rt * 16 + c16][w]);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[rt] += sw[e] * __builtin_amdgcn_exp2f(mw[e] - top[rt]);
      }
    const __amdgpu_buffer_rsrc_t res = partial_of(l);
    const int slot = (it.first + it.piece) * S::kBytes;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if (rt * 16 >= rows_here) break;
#pragma unroll
      for (int d = 0; d < DW; ++d) {
        if (it.pieces == 1) {
          if (rt * 16 + c16 < rows_here)
            write_y(a, l, q, it.head, row_first + rt * 16 + c16, 16 * (wave * DW + d) + 4 * g, DIM, o[d][rt], sum[rt]);
        } else {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o[d][rt]), res,
                                                 S::fragment(rt, wave * DW + d, lane), slot, kDevScope);
        }
      }
      if (it.pieces > 1 && wave == 0 && g == 0)
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, float2v{top[rt], sum[rt]}), res, S::row(rt, c16),
                                              slot, kDevScope);
    }
    if (it.pieces > 1) join_pieces<DIM, RT, W>(a, l, it, q, lane, wave, row_first, rows_here, &s_arrival);
    lds_barrier();  // LDS is free for the next item
  }
}

// ---------------------------------------------------------------------------
// Many rows: a workgroup's wavefronts share each page through LDS.
//
// The workgroup converts a page to FP16 once, into the order of the products'
// A operands (a conversion costs as much as two additions, and each wavefront
// on its own would spend half its vector time on them).  The scores of the next
// page are computed beside the weights of this one, so that the matrix and the
// vector units work at the same time; keys are therefore one page ahead of
// values.  Two buffers of each, one barrier a page.  The codes come through a
// ring of kRing pages in LDS (loads straight into it, each wavefront its own
// part), so that a load has three pages' time to arrive; with the pages of
// dimension 256 the ring does not fit, and they come through registers.
//
// Bound: the matrix and vector units of a SIMD, which two wavefronts share (256
// rows of 40 + 8 heads of 128 over 20001 tokens, 104 GFLOP: 133 us with the join's
// 8.9, 782 TFLOP/s, where a large FP16 matrix product reaches 1157).
// ---------------------------------------------------------------------------
constexpr int kRing = 4;

// A load of 16 bytes a lane into LDS: lane i's go to lds + 16 i.
__device__ __forceinline__ void load_to_lds(const uint8_t* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(uniform((int)lds)), "v"(offset), "s"(base)
               : "memory", "m0");
}

// 16 bytes from LDS once no more than N of the loads above are on their way.
template <int N>
__device__ __forceinline__ u32x4 read_arrived(uint32_t lds) {
  u32x4 x;
  asm volatile("s_waitcnt vmcnt(%2)\n\tds_read_b128 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(x) : "v"(lds), "n"(N) : "memory");
  return x;
}

template <int DIM>
struct ManyLds {
  half8 k[2][DIM / 8][64], v[2][DIM / 8][64];  // operands: buffer, operand, lane
  int nan;                                     // values that only some rows of the tile see held NaN
  static constexpr int RING = DIM < 256 ? kRing : 0;
  static constexpr int LOADS = DIM / 8 / kManyWaves;  // 1 KiB of codes each, of a wavefront and page
};

template <int DIM, int RT>
__global__ __launch_bounds__(kManyWaves * 64) void attention_many_kernel(AttentionArgs a, AttnLaunch l) {
  using R = Rows<DIM, RT>;
  using S = Slot<DIM, RT * kManyWaves>;
  constexpr int DT = R::DT, KS = R::KS, ROWS = 16 * RT * kManyWaves;
  using L = ManyLds<DIM>;
  constexpr int LOADS = L::LOADS, RING = L::RING;
  // the ring first, at LDS address 0 (there is no other LDS): 64 KiB, as a load's LDS address has 16 bits
  extern __shared__ __attribute__((aligned(16))) uint8_t s_many[];
  L& lds = *reinterpret_cast<L*>(s_many + RING * DIM * 128);
  const int wave = uniform((int)threadIdx.x >> 6);

  for (int block = blockIdx.x;; block += gridDim.x) {
    int tid = threadIdx.x;  // (opaque, as above)
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, c16 = lane & 15, g = lane >> 4;
    Req q;
    const Item it = item_of(a, l, lane, block, q);
    if (it.request < 0) break;
    const int tile_first = it.tile * ROWS;
    const int tile_rows = min(ROWS, q.rows * l.group - tile_first);
    const int row_first = tile_first + wave * 16 * RT;       // this wavefront's
    const int rows_here = min(16 * RT, tile_rows - wave * 16 * RT);
    const bool some = rows_here > 0;
    const View<1> all = view_of<1>(a, l, q, lane, tile_first, tile_rows);
    const View<RT> see = view_of<RT>(a, l, q, lane, row_first, some ? rows_here : 1);
    const int lo = max(q.first_page + (int)((int64_t)q.pages * it.piece / it.pieces), all.low_min / kKvPage);
    const int hi = min(q.first_page + (int)((int64_t)q.pages * (it.piece + 1) / it.pieces),
                       (all.lim_max + kKvPage - 1) / kKvPage);
    const int32_t* const table = a.table + it.request * a.table_stride;
    Pages now;  // of the 64 pages around the present ones
    now.load(a, table, it.head, q.bad, lane, lo, 1, hi);
    half8 qr[RT][KS];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) load_query<DIM>(a, l, q, it.head, lane, row_first, rows_here, rt, qr[rt]);
    if (threadIdx.x == 0) lds.nan = 0;
    lds_barrier();
    R rows;
    rows.begin(Pages::at(now.vs, 0));

    // The loads of a page, 1 KiB each, in turn to the wavefronts: keys, load n =
    // 4 u + t: unit 4 u + g of token 16 t + c16; values, load n: dimension
    // 16 n + c16, group g.  Keys are a page ahead of values.
    const auto is_key = [&](int j) { return j * kManyWaves + wave < DIM / 16; };
    const auto number = [&](int j) { return (j * kManyWaves + wave) % (DIM / 16); };
    const auto place = [&](int j) {  // within the block
      const int n = number(j);
      return is_key(j) ? (((n >> 2) * 4 + g) * kKvPage + (n & 3) * 16 + c16) * 16 : (n * 16 + c16) * kKvPage + 16 * g;
    };
    const uint32_t ring = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)s_many + wave * (LOADS * 1024);
    u32x4 held[LOADS];  // without a ring
    const auto fetch = [&](int j, int64_t offset, int page) {
      const uint8_t* const base = (is_key(j) ? a.cache.k : a.cache.v) + offset;
      if constexpr (RING > 0)
        load_to_lds(base, place(j), ring + (uint32_t)((page % RING) * (kManyWaves * LOADS) + j) * 1024u);
      else
        held[j] = *reinterpret_cast<const u32x4*>(base + place(j));
    };
    // Codes to operands.  Values of a page that some rows of the tile see only
    // a part of: what none sees becomes zeros (what is there may be anything),
    // and so does NaN, of which a flag is left.
    const auto put = [&](int j, int page) {
      u32x4 x;
      if constexpr (RING > 0)
        x = read_arrived<(RING - 1) * LOADS>(ring + (uint32_t)((page % RING) * (kManyWaves * LOADS) + j) * 1024u + lane * 16u);
      else
        x = held[j];
      const int base = page * kKvPage;
      const bool keys = is_key(j);
      if (!keys && (base + kKvPage > all.lim_min || base < all.low_max)) {
        uint32_t any = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t y = x[t] & keep_bytes(seen_of(all.lim_max, all.low_min, base + 32 * (t >> 1), g), t & 1);
          const uint32_t n = nan_bytes(y) >> 7;
          any |= n;
          x[t] = y & ~(n * 255u);
        }
        const uint64_t some_nan = __ballot(any != 0);
        if (lane == 0 && some_nan) lds.nan = 1;
      }
      half8 f[2];
      decode_fp8_fragment(x, f);
      half8(*const to)[64] = keys ? lds.k[page & 1] : lds.v[page & 1];
#pragma unroll
      for (int h = 0; h < 2; ++h) to[number(j) * 2 + h][lane] = f[h];
    };
    // this wavefront's own pages among the workgroup's
    const int my_lo = some ? max(lo, see.low_min / kKvPage) : hi;
    const int my_hi = some ? min(hi, (see.lim_max + kKvPage - 1) / kKvPage) : hi;
    float4v s[4][RT];  // the scores of page my_lo and on, one page ahead
    float high[RT];    // and the largest of the lane's
    Pages next = now;  // of the 64 pages behind those of `now`
    // step `page`: the weights and values of `page`, the scores of page + 1; keys
    // of page + 2 and values of page + 1 become operands; on their way: RING - 1
    // pages more (without a ring: those two)
    const auto offset_of = [&](int page, int at) {  // of `page` (the last one for any behind it), at most 64 behind lo + at
      const int n = min(page, hi - 1) - lo;
      const int id = (n >> 6) == (at >> 6) ? __builtin_amdgcn_readlane(now.id, n & 63) : __builtin_amdgcn_readlane(next.id, n & 63);
      return ((int64_t)id * a.cache.heads + it.head) * (kKvPage * DIM);
    };
    int64_t values_at = 0;  // the offset of the page whose keys were fetched last
    const auto fetch_all = [&](int page, int at, bool values) {  // keys of `page`, values of the one before
      const int64_t keys_at = offset_of(page, at);
#pragma unroll
      for (int j = 0; j < LOADS; ++j) fetch(j, is_key(j) ? keys_at : values ? values_at : keys_at, is_key(j) ? page : values ? page - 1 : page);
      values_at = keys_at;
    };
    if (lo < hi) {
      constexpr int FIRST = RING > 0 ? RING : 1;
#pragma unroll
      for (int i = 0; i < FIRST; ++i) fetch_all(lo + i, 0, i > 0);
#pragma unroll
      for (int j = 0; j < LOADS; ++j)
        if (is_key(j)) put(j, lo);
    }
    for (int page = lo - 1; page < hi; ++page) {
      const int at = max(page - lo, 0);
      if (at > 0 && (at & 63) == 0) now = next;
      if ((at & 63) == 32 && lo + (at | 63) + 1 < hi) next.load(a, table, it.head, q.bad, lane, lo + (at | 63) + 1, 1, hi);
      lds_barrier();  // values of this page and keys of the next are in LDS, the other buffers have been read
      if (lo < hi) {
        constexpr int MORE = RING > 0 ? RING - 1 : 0;
        fetch_all(page + 2 + MORE, at, true);
      }
      const auto key = [&](int i) { return lds.k[(page + 1) & 1][(i >> 3) * 8 + (i & 3) * 2 + (i >> 2 & 1)][lane]; };
      const int behind = page + 1 - lo;  // the next page's place
      const float next_kc = Pages::at((behind >> 6) == (at >> 6) ? now.kc : next.kc, behind & 63);
      if (page >= my_lo && page < my_hi) {
        float vs = Pages::at(now.vs, at & 63);
        const int base = page * kKvPage;
        bool counts = true;
        if (__builtin_expect(!(vs >= rows.vref && vs <= rows.vref * kScaleSlack), 0)) counts = rows.settle(vs);
        if (base + kKvPage > see.lim_min || base < see.low_max) {
          mask_page<RT>(s, base, g, see);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) high[rt] = page_max<RT>(s, rt);
        }
        rows.raise(high);
        const float drop = rows.vref * __builtin_amdgcn_rcpf(vs), lift = -__builtin_amdgcn_logf(drop);
        half8 p[2][RT];
        float4v ahead[4][RT];  // (of a page that is not there: of what the buffer holds, and not used)
        rows.weigh(s, lift, drop, p, key, qr, ahead);
        if (__builtin_expect(!counts, 0)) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) p[h][rt] = half8{};
        }
        rows.accumulate([&](int i) { return lds.v[page & 1][i][lane]; }, p, ahead, next_kc, high);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) s[t][rt] = ahead[t][rt];
      } else if (page + 1 == my_lo && my_lo < my_hi) {
        R::scores(key, qr, s);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
          for (int t = 0; t < 4; ++t) s[t][rt] *= next_kc;
          high[rt] = page_max<RT>(s, rt);
        }
      }
      if (lo < hi) {
#pragma unroll
        for (int j = 0; j < LOADS; ++j) put(j, is_key(j) ? page + 2 : page + 1);
      }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // nothing more comes into LDS
    lds_barrier();
    if (__builtin_expect(uniform(lds.nan) != 0, 0)) {  // NaN into the rows that see it, from the pages' codes
      for (int page = my_lo; page < my_hi; ++page) {
        const int base = page * kKvPage, id = table[page];
        if ((base + kKvPage <= all.lim_min && base >= all.low_max) || id < 0 || id >= a.cache.pages) continue;
        const uint8_t* const values = a.cache.v + ((int64_t)id * a.cache.heads + it.head) * (kKvPage * DIM);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const u32x4 x = *reinterpret_cast<const u32x4*>(values + (16 * d + c16) * kKvPage + 16 * g);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const half8 n = decode_e4m3x8((nan_bytes(x[2 * half]) >> 7) * 0x38u, (nan_bytes(x[2 * half + 1]) >> 7) * 0x38u);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
              spread_nan(n, seen_of(see.lim[rt], see.low(rt), base + 32 * half, g), rows.o[d][rt]);
          }
        }
      }
    }

    const __amdgpu_buffer_rsrc_t res = partial_of(l);
    const int slot = (it.first + it.piece) * S::kBytes;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if (rt * 16 >= rows_here) break;
      float weight = rows.sum[rt] + __shfl_xor(rows.sum[rt], 16);
      weight += __shfl_xor(weight, 32);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const float4v sum = rows.o[d][rt] * rows.vref;
        if (it.pieces == 1) {
          if (rt * 16 + c16 < rows_here)
            write_y(a, l, q, it.head, row_first + rt * 16 + c16, 16 * d + 4 * g, DIM, sum, weight);
        } else {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, sum), res,
                                                 S::fragment(wave * RT + rt, d, lane), slot, 0);
        }
      }
      if (it.pieces > 1 && g == 0)
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, float2v{rows.m[rt], weight}), res,
                                              S::row(wave * RT + rt, c16), slot, 0);
    }
    lds_barrier();  // LDS is free for the next item
  }
}

// Joins the pieces of cut segments of many rows: the workgroup of a piece
// takes its share of the segment's fragments.  (A launch of its own: the last
// workgroup alone would need tens of microseconds for a tile of 192 rows.)
template <int DIM, int TILES>
__global__ __launch_bounds__(kManyWaves * 64) void attention_join_kernel(AttentionArgs a, AttnLaunch l) {
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
      join_fragments<DIM, TILES, 1, B>(partial_of(l), lane, rt, d0, it.pieces, [&](int i) { return it.first + i; }, sum,
                                       top, weight);
      if (rt * 16 + c16 < rows_here) {
#pragma unroll
        for (int d = 0; d < B; ++d)
          write_y(a, l, q, it.head, row_first + rt * 16 + c16, 16 * (d0 + d) + 4 * g, DIM, sum[0][d], weight[0]);
      }
    }
  }
}

// Segments of a call whose requests all bring max_rows rows.
int64_t most_segments(int requests, int max_rows, int q_heads, int heads, int dim) {
  const int64_t rows = (int64_t)max_rows * (q_heads / heads);
  const Form f = form_for(rows, dim);
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

template <typename Kernel>
hipError_t launch_kernel(Kernel kernel, int threads, size_t lds, const AttentionArgs& a, const AttnLaunch& l,
                         int64_t grid) {
  if (lds > 0) {
    const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  kernel<<<dim3((uint32_t)grid), dim3(threads), lds, (hipStream_t)a.stream>>>(a, l);
  return hipGetLastError();
}

template <int DIM, int RT>
hipError_t launch_many(const AttentionArgs& a, const AttnLaunch& l, int64_t grid) {
  const hipError_t e = launch_kernel(attention_many_kernel<DIM, RT>, kManyWaves * 64,
                                     sizeof(ManyLds<DIM>) + (size_t)ManyLds<DIM>::RING * DIM * 128, a, l, grid);
  if (e != hipSuccess || l.slots == 0) return e;
  return launch_kernel(attention_join_kernel<DIM, RT * kManyWaves>, kManyWaves * 64, 0, a, l, grid);
}

template <int DIM, int RT>
hipError_t launch_few(const AttentionArgs& a, const AttnLaunch& l, int64_t grid) {
  return launch_kernel(attention_few_kernel<DIM, RT>, few_waves(DIM) * 64, sizeof(FewLds<DIM, RT>), a, l, grid);
}

template <int DIM>
hipError_t launch_dim(const Form& f, const AttentionArgs& a, const AttnLaunch& l, int64_t grid) {
  if (f.tiles == 1) return f.many ? launch_many<DIM, 1>(a, l, grid) : launch_few<DIM, 1>(a, l, grid);
  if constexpr (DIM < 256) {
    if (f.tiles == 2) return f.many ? launch_many<DIM, 2>(a, l, grid) : launch_few<DIM, 2>(a, l, grid);
    return launch_few<DIM, 3>(a, l, grid);
  }
  return hipErrorInvalidValue;
}

}  // namespace

size_t attention_scratch_bytes(int requests, int max_rows, int q_heads, int heads, int dim, int table_width) {
  const int64_t segments = most_segments(requests, max_rows, q_heads, heads, dim);
  if (table_width <= kMinPiecePages || segments >= kMaxPieces) return kKvZeroedBytes;
  const Form f = form_for((int64_t)max_rows * (q_heads / heads), dim);
  const size_t slots = wanted_pieces(segments);
  return kKvZeroedBytes + (slots + slots / 2) * slot_bytes(f, dim);
}

hipError_t launch_attention(const AttentionArgs& a) {
  const int dim = a.cache.dim, group = a.q_heads / a.cache.heads;
  const Form f = form_for((int64_t)a.max_rows * group, dim);
  const int64_t segments = most_segments(a.requests, a.max_rows, a.q_heads, a.cache.heads, dim);
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
  return dim == 64 ? launch_dim<64>(f, a, l, grid) : dim == 128 ? launch_dim<128>(f, a, l, grid)
                                                                : launch_dim<256>(f, a, l, grid);
}

}  // namespace qpn
