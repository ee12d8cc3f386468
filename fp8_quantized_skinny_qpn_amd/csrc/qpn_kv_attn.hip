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
// and no rescaling.
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

constexpr float kMaxSlack = 8.0f;     // how far (log2) a score may pass the running maximum
constexpr float kScaleSlack = 64.0f;  // and a page's V scale the running one
constexpr float kLowest = -3e38f;     // the running maximum before any score

// wavefronts of a workgroup, few rows: two a SIMD while their registers allow
// it (a spilled register is a load that waits behind the page's)
constexpr int few_waves(int dim, int tiles) { return dim * tiles <= 384 ? 8 : 4; }
constexpr int kManyWaves = 4;  // and many
constexpr int kMinPiecePages = 8;
constexpr int kMaxPieces = 1024;   // pieces of a call with cut segments
constexpr int kJoinDirect = 8;     // pieces joined in one step
constexpr int kCounterStep = 8;    // 32-bit words between counters
static_assert((size_t)kMaxPieces * 2 * kCounterStep * 4 <= kKvZeroedBytes, "two counters per piece");

// The form and the 16-row tiles of a wavefront for `rows` rows of a KV head
// (query rows x group).
struct Form {
  bool many;
  int tiles;
  int rows() const { return 16 * tiles * (many ? kManyWaves : 1); }
};
inline Form form_for(int64_t rows, int dim) {
  const int few = dim == 256 ? 1 : 3;
  const int64_t t = (rows + 15) / 16;
  if (t <= few) return {false, t < 1 ? 1 : (int)t};
  return {true, t <= kManyWaves ? 1 : 2};
}

struct AttnLaunch {
  int tile_rows;   // rows of a workgroup's segment
  int group;       // query heads of a KV head
  int target;      // pieces the lengths are cut into
  int slots;       // pieces the scratch has room for (0: segments stay whole)
  float* partial;  // 1.5 slots of partial sums (layout at Slot)
};

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
// Every number fits 31 bits: a call has at most 2^30 rows x query heads.
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
      segs += my_segs;
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

// What the rows of a wavefront see: tokens [low, lim) of the lane's row of
// each tile, and the extremes over its rows.
template <int RT>
struct View {
  int lim[RT], low[RT];
  int lim_min, lim_max, low_min, low_max;
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

// The rows of a wavefront and their running sums.
template <int DIM, int RT>
struct Rows {
  static constexpr int KS = DIM / 32;  // k-steps of the scores
  static constexpr int DT = DIM / 16;  // tiles of output dimensions
  float m[RT], sum[RT];
  float4v o[DT][RT];
  float vref;  // what the sums are in units of

  __device__ __forceinline__ void begin(float first_scale) {
    vref = first_scale > 0x1p-100f ? first_scale : 0x1p-100f;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      m[t] = kLowest;
      sum[t] = 0.0f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d][t] = float4v{0, 0, 0, 0};
    }
  }

  // Whether a page is an ordinary one: every row sees all of it, and its
  // scales are positive and in proportion.  (Uniform over the wavefront.)
  __device__ __forceinline__ bool ordinary(float kc, float vs, int base, const View<RT>& see) const {
    return base + kKvPage <= see.lim_min && base >= see.low_max && kc > 0.0f && vs <= vref * kScaleSlack &&
           vs >= vref * 0x1p-20f;
  }

  // One ordinary page (EDGE: any page), in two halves of 32 tokens, so that a
  // half's scores, not a page's, are held in registers beside the sums.
  //   key(u, t): the codes of unit 4 u + g of token 16 t + c16;
  //   query(k, rt): the B operand of k-step k (load_query);
  //   value(d): the codes of dimension 16 d + c16, tokens 16 t + 4 g + r;
  //   kc: the factor of the scores in units of log2 e, vs: the V scale;
  //   fetch(): called when the last key has been used.
  template <bool EDGE, typename Key, typename Query, typename Value, typename Fetch>
  __device__ __forceinline__ void page(const Key& key, const Query& query, const Value& value, const Fetch& fetch,
                                       float kc, float vs, int base, int g, const View<RT>& see) {
    bool plain = true;
    float sign = 1.0f;
    if constexpr (EDGE) {
      // a negative factor moves to the scores; for 0 any does, with zeros
      if (!(kc > 0.0f)) {
        sign = kc == 0.0f ? 0.0f : -1.0f;
        kc = kc == 0.0f ? 1.0f : -kc;
      }
      if (vs > vref * kScaleSlack) {
        const float f = vref / vs;
        vref = vs;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int d = 0; d < DT; ++d) o[d][rt] *= f;
      }
      plain = vs >= vref * 0x1p-20f;
    }
    // weights times vs / vref = exp2(score - m + log2(vs / vref)), and their
    // FP32 sum times vref / vs; where vs is out of proportion (or not
    // positive) the values are multiplied instead
    const float vrel = vs / vref;
    const float lift = plain ? __builtin_amdgcn_logf(vrel) : 0.0f, drop = plain ? vref / vs : 1.0f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float4v s[2][RT];
      scores(key, query, half, s);
      if (half == 1) fetch();
      half8 p[RT];
      if constexpr (EDGE) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const uint32_t seen = seen_of(see.lim[rt], see.low[rt], base + 32 * half, g);
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const uint32_t ones = all_ones_if(seen, t, r);
              const float x = s[t][rt][r] * sign;
              s[t][rt][r] = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, x) & ones) | (0xFF800000u & ~ones));  // -inf
            }
        }
      }
      weigh(s, kc, lift, drop, p);
      if constexpr (EDGE)
        accumulate_edge(value, p, half, plain ? 1.0f : vrel, base + 32 * half, g, see);
      else
        accumulate(value, p, half);
    }
  }

 private:
  // S^T of half a page
  template <typename Key, typename Query>
  __device__ __forceinline__ void scores(const Key& key, const Query& query, int half, float4v (&s)[2][RT]) const {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) s[t][rt] = float4v{0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < DIM / 64; ++u) {
      half8 q[2][RT];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) q[h][rt] = query(2 * u + h, rt);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        half8 kf[2];
        decode_fp8_fragment(key(u, 2 * half + t), kf);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            s[t][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[h], q[h][rt], s[t][rt], 0, 0, 0);
      }
    }
  }

  // The weights of half a page's scores, as the B operands of the second
  // product; the sums and maxima follow.
  __device__ __forceinline__ void weigh(float4v (&s)[2][RT], float kc, float lift, float drop, half8 (&p)[RT]) {
    float top[RT];
    bool raise = false;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float mx = fmaxf(s[0][rt][0], s[0][rt][1]);
#pragma unroll
      for (int i = 2; i < 8; i += 2) mx = fmaxf(fmaxf(mx, s[i >> 2][rt][i & 3]), s[i >> 2][rt][(i & 3) + 1]);
      top[rt] = mx * kc;
      raise |= top[rt] > m[rt] + kMaxSlack;
    }
    if (__ballot(raise)) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float mx = fmaxf(top[rt], __shfl_xor(top[rt], 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float up = fmaxf(m[rt], mx);
        const float f = __builtin_amdgcn_exp2f(m[rt] - up);
        m[rt] = up;
        sum[rt] *= f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d][rt] *= f;
      }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float off = lift - m[rt];
      float part[2] = {0.0f, 0.0f};
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][rt][r], kc, off));
          part[t] += w;
          s[t][rt][r] = w;
        }
      sum[rt] = __builtin_fmaf(part[0] + part[1], drop, sum[rt]);
      p[rt] = to_half8(s[0][rt], s[1][rt]);
    }
  }

  // O^T += V^T P^T over half a page
  template <typename Value>
  __device__ __forceinline__ void accumulate(const Value& value, const half8 (&p)[RT], int half) {
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const u32x4 v = value(d);
      const half8 vf = decode_e4m3x8(v[2 * half], v[2 * half + 1]);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) o[d][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, p[rt], o[d][rt], 0, 0, 0);
    }
  }

  // The same with the values times `factor`, and with codes of tokens that no
  // row of the wavefront sees as zeros (what is there may be anything); a NaN
  // code that some rows see and others do not is taken out too, and put into
  // the rows that see it.
  template <typename Value>
  __device__ __forceinline__ void accumulate_edge(const Value& value, const half8 (&p)[RT], int half, float factor,
                                                  int base, int g, const View<RT>& see) {
    const uint32_t some = seen_of(see.lim_max, see.low_min, base, g);
    uint32_t keep[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) keep[t] = ((((some >> (16 * t)) & 15u) * 0x00204081u) & 0x01010101u) * 255u;
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const u32x4 both = value(d);
      uint32_t v[2], n[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        v[t] = both[2 * half + t] & keep[t];
        n[t] = nan_bytes(v[t]) >> 7;  // 1 in NaN bytes
      }
      if (__ballot((n[0] | n[1]) != 0)) {
        const half8 f = decode_e4m3x8(n[0] * 0x38u, n[1] * 0x38u);  // 1.0 there
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const uint32_t seen = seen_of(see.lim[rt], see.low[rt], base, g);
          u32x4 sees;  // FP16 1 where the row sees the token
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sees[e] = (all_ones_if(seen, e >> 1, 2 * (e & 1)) & 0x3C00u) |
                      (all_ones_if(seen, e >> 1, 2 * (e & 1) + 1) & 0x3C000000u);
          const float4v hit = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, __builtin_bit_cast(half8, sees), float4v{0, 0, 0, 0},
                                                                    0, 0, 0);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (hit[r] > 0.0f) o[d][rt][r] = __builtin_nanf("");
        }
        v[0] &= ~(n[0] * 255u);
        v[1] &= ~(n[1] * 255u);
      }
      const half8 vf = decode_e4m3x8(v[0], v[1]);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const float4v add = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, p[rt], float4v{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) o[d][rt][r] = __builtin_fmaf(add[r], factor, o[d][rt][r]);
        // here, not behind the last tile, where every product would still be held
        asm volatile("" : "+v"(o[d][rt]));
      }
    }
  }
};

// The blocks and scales of up to 64 pages of a request, one a lane: entries
// first + lane * step below end.
struct Pages {
  int64_t block;
  float kc, vs;
  __device__ __forceinline__ void load(const AttentionArgs& a, const int32_t* table, int head, bool bad, int lane,
                                       int first, int step, int end) {
    const int page = first + lane * step;  // (both below 2^25)
    block = head;
    kc = __builtin_nanf("");
    vs = 1.0f;
    if (page < end && page < a.table_width) {
      const int32_t id = table[page];
      if (id >= 0 && id < a.cache.pages && !bad) {
        block = (int64_t)id * a.cache.heads + head;
        kc = a.cache.k_scale[block] * (a.scale * 1.44269504088896340736f);
        vs = a.cache.v_scale[block];
      }
    }
  }
  __device__ __forceinline__ int64_t block_at(int i) const {
    const int lo = __builtin_amdgcn_readlane((int)(block & 0xFFFFFFFF), i);
    const int hi = __builtin_amdgcn_readlane((int)(block >> 32), i);
    return ((int64_t)hi << 32) | (uint32_t)lo;
  }
  static __device__ __forceinline__ float at(float x, int i) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), i));
  }
};

template <int RT>
__device__ __forceinline__ View<RT> view_of(const AttentionArgs& a, int group, const Req& q, int lane, int first,
                                            int rows) {
  const int c16 = lane & 15, at = q.seq - q.rows + 1;
  View<RT> v;
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    v.lim[t] = t * 16 + c16 < rows ? at + (int)((uint32_t)(first + t * 16 + c16) / (uint32_t)group) : 0;
    v.low[t] = a.window > 0 ? max(0, v.lim[t] - a.window) : 0;
  }
  v.lim_min = uniform(at + (int)((uint32_t)first / (uint32_t)group));
  v.lim_max = uniform(at + (int)((uint32_t)(first + rows - 1) / (uint32_t)group));
  v.low_min = a.window > 0 ? max(0, v.lim_min - a.window) : 0;
  v.low_max = a.window > 0 ? max(0, v.lim_max - a.window) : 0;
  return v;
}

// Q: B operand of row tile t: lane (row c16, k 8 g + e) of k-step 2 u + h has
// dimensions 64 u + 16 g + 8 h + e, as the key units' 16 dimensions fall to the
// lanes.  Rows behind `rows` are zeros.
template <int DIM>
__device__ __forceinline__ void load_query(const AttentionArgs& a, int group, const Req& r, int head, int lane,
                                           int first, int rows, int t, half8 (&q)[DIM / 32]) {
  const int c16 = lane & 15, g = lane >> 4;
  const bool in = t * 16 + c16 < rows;
  const uint32_t rr = (uint32_t)(in ? first + t * 16 + c16 : 0), row = rr / (uint32_t)group;
  const uint16_t* src = a.q + (int64_t)(r.row0 + (int)row) * a.q_stride +
                        (int64_t)(head * group + (int)(rr - row * (uint32_t)group)) * DIM + 16 * g;
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

// Four dimensions of a row: y when the piece is the whole segment.
__device__ __forceinline__ void write_y(const AttentionArgs& a, int group, const Req& q, int head, int rr, int dim0,
                                        int dim, float4v sum, float weight) {
  const int row = (int)((uint32_t)rr / (uint32_t)group);
  half4 h;
  if (weight == 0.0f) {
    // nothing seen gives zeros; tokens seen but no weight (every score -inf) has no value
    const int lim = q.seq - q.rows + row + 1;
    const _Float16 x = lim > 0 ? (_Float16)__builtin_nanf("") : (_Float16)0;
    h = half4{x, x, x, x};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = (_Float16)(sum[e] / weight);
  }
  *reinterpret_cast<half4*>(a.y + (int64_t)(q.row0 + row) * a.y_stride +
                            (int64_t)(head * group + rr - row * group) * dim + dim0) = h;
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

// After the pieces' sums are stored: the last workgroup of a segment (of a
// group of its pieces first, when there are many) joins them in order and
// writes y.  Fragments go to the wavefronts in turn.
template <int DIM, int TILES, int WAVES>
__device__ __forceinline__ void join_pieces(const AttentionArgs& a, const AttnLaunch& l, const Item& it, const Req& q,
                                            int lane, int wave, int row_first, int rows_here, uint32_t* s_arrival) {
  using S = Slot<DIM, TILES>;
  const int c16 = lane & 15, g = lane >> 4;
  const __amdgpu_buffer_rsrc_t res = __builtin_amdgcn_make_buffer_rsrc((void*)l.partial, (short)0, 0x7FFFFFFF, kRsrc);
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
  int count = p1 - p0, first = it.first + p0;
  bool inner = groups > 1;
  for (;;) {
    auto slot_of = [&](int i) {
      return inner || groups == 1 ? first + i : l.slots + (it.first + start_of(i)) / 2;
    };
    for (int f = wave; f < TILES * S::DT; f += WAVES) {
      const int rt = f / S::DT, d = f % S::DT;
      if (rt * 16 >= rows_here) break;
      float4v sum{0, 0, 0, 0};
      float top = kLowest, weight = 0.0f;
      for (int i0 = 0; i0 < count; i0 += kJoinDirect) {
        float4v o[kJoinDirect];
        float2v ml[kJoinDirect];
#pragma unroll
        for (int i = 0; i < kJoinDirect; ++i) {
          const int at = slot_of(min(i0 + i, count - 1)) * S::kBytes;
          ml[i] = __builtin_bit_cast(float2v, __builtin_amdgcn_raw_buffer_load_b64(res, at + S::row(rt, c16), 0, kDevScope));
          o[i] = __builtin_bit_cast(float4v, __builtin_amdgcn_raw_buffer_load_b128(res, at + S::fragment(rt, d, lane), 0, kDevScope));
        }
        float up = top;
#pragma unroll
        for (int i = 0; i < kJoinDirect; ++i) up = fmaxf(up, ml[i][0]);
        const float old = __builtin_amdgcn_exp2f(top - up);
        top = up;
        sum *= old;
        weight *= old;
#pragma unroll
        for (int i = 0; i < kJoinDirect; ++i) {
          const float f = i0 + i < count ? __builtin_amdgcn_exp2f(ml[i][0] - top) : 0.0f;
          if (i0 + i < count) {
            sum += o[i] * f;
            weight += ml[i][1] * f;
          }
        }
      }
      if (inner) {
        const int at = (l.slots + first / 2) * S::kBytes;
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, sum), res, at + S::fragment(rt, d, lane), 0, kDevScope);
        if (d == 0 && g == 0)
          __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, float2v{top, weight}), res, at + S::row(rt, c16),
                                                0, kDevScope);
      } else if (rt * 16 + c16 < rows_here) {
        write_y(a, l.group, q, it.head, row_first + rt * 16 + c16, 16 * d + 4 * g, DIM, sum, weight);
      }
    }
    if (!inner) return;
    if (!arrive_last(counters + (kMaxPieces + it.first) * kCounterStep, groups, s_arrival)) return;
    inner = false;
    count = groups;
  }
}

// ---------------------------------------------------------------------------
// Few rows: a wavefront takes whole pages.
// ---------------------------------------------------------------------------
template <int DIM, int RT>
__global__ __launch_bounds__(few_waves(DIM, RT) * 64) void attention_few_kernel(AttentionArgs a, AttnLaunch l) {
  using R = Rows<DIM, RT>;
  using S = Slot<DIM, RT>;
  constexpr int W = few_waves(DIM, RT);
  constexpr int DT = R::DT, KS = R::KS, ROWS = 16 * RT;
  constexpr bool kQueryLds = RT > 1;  // the queries' fragments are read from LDS for each page
  __shared__ float s_m[W][ROWS], s_l[W][ROWS];
  __shared__ __attribute__((aligned(16))) half8 s_q[kQueryLds ? KS * RT * 64 : 1];
  __shared__ uint32_t s_arrival;
  extern __shared__ __attribute__((aligned(16))) float s_o[];  // [W][DT][64][4]
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
    const View<RT> see = view_of<RT>(a, l.group, q, lane, row_first, rows_here);
    // the piece's pages that the tile sees; this wavefront takes every
    // W-th
    const int lo = max(q.first_page + (int)((int64_t)q.pages * it.piece / it.pieces), see.low_min / kKvPage) + wave;
    const int hi = min(q.first_page + (int)((int64_t)q.pages * (it.piece + 1) / it.pieces),
                       (see.lim_max + kKvPage - 1) / kKvPage);
    const int32_t* const table = a.table + it.request * a.table_stride;
    Pages pages;
    pages.load(a, table, it.head, q.bad, lane, lo, W, hi);

    u32x4 k[DIM / 64][4], v[DT];
    const int k_at = g * (kKvPage * 16) + c16 * 16, v_at = c16 * kKvPage + 16 * g;
    auto load_keys = [&](int64_t block) {
      const __amdgpu_buffer_rsrc_t res =
          __builtin_amdgcn_make_buffer_rsrc((void*)(a.cache.k + block * (kKvPage * DIM)), (short)0, kKvPage * DIM, kRsrc);
#pragma unroll
      for (int u = 0; u < DIM / 64; ++u)
#pragma unroll
        for (int t = 0; t < 4; ++t)
          k[u][t] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(res, k_at + t * 256, u * 4 * kKvPage * 16, 0));
    };
    auto load_values = [&](int64_t block) {
      const __amdgpu_buffer_rsrc_t res =
          __builtin_amdgcn_make_buffer_rsrc((void*)(a.cache.v + block * (kKvPage * DIM)), (short)0, kKvPage * DIM, kRsrc);
#pragma unroll
      for (int d = 0; d < DT; ++d)
        v[d] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(res, v_at + d % 4 * (16 * kKvPage), d / 4 * 64 * kKvPage, 0));
    };
    if (lo < hi) {
      const int64_t first = pages.block_at(0);
      load_keys(first);
      load_values(first);
    }
    half8 qr[KS];
    if constexpr (kQueryLds) {
      if (wave < RT) {
        load_query<DIM>(a, l.group, q, it.head, lane, row_first, rows_here, wave, qr);
#pragma unroll
        for (int i = 0; i < KS; ++i) s_q[(i * RT + wave) * 64 + lane] = qr[i];
      }
      __syncthreads();
    } else {
      load_query<DIM>(a, l.group, q, it.head, lane, row_first, rows_here, 0, qr);
    }
    auto query = [&](int i, int rt) { return kQueryLds ? s_q[(i * RT + rt) * 64 + lane] : qr[i]; };
    R rows;
    rows.begin(Pages::at(pages.vs, 0));
    const int count = lo < hi ? (hi - lo + W - 1) / W : 0;
    // Page i with the next page's keys (the last one's again at the end) on
    // their way once its own are used, the next values behind its own.
    const auto key = [&](int u, int t) { return k[u][t]; };
    const auto value = [&](int d) { return v[d]; };
    int i = 0;
    float kc = 0.0f, vs = 0.0f;
    int64_t next = 0;
    const auto turn_to = [&]() {  // page i's factors, the next page's block
      kc = Pages::at(pages.kc, i & 63), vs = Pages::at(pages.vs, i & 63);
      if ((i & 63) == 63 && i + 1 < count)
        pages.load(a, table, it.head, q.bad, lane, lo + (i + 1) * W, W, hi);
      next = pages.block_at(i + 1 < count ? (i + 1) & 63 : i & 63);
    };
    const auto fetch = [&] { load_keys(next); };
    if (count > 0) turn_to();
    while (i < count) {
      // the loop over ordinary pages by itself, which keeps the sums in place
      while (rows.ordinary(kc, vs, (lo + i * W) * kKvPage, see)) {
        rows.template page<false>(key, query, value, fetch, kc, vs, 0, g, see);
        load_values(next);
        if (++i == count) break;
        turn_to();
      }
      if (i < count) {
        rows.template page<true>(key, query, value, fetch, kc, vs, (lo + i * W) * kKvPage, g, see);
        load_values(next);
        if (++i < count) turn_to();
      }
    }

    // join the wavefronts: a common maximum per row, then the sums in order
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      rows.sum[rt] += __shfl_xor(rows.sum[rt], 16);
      rows.sum[rt] += __shfl_xor(rows.sum[rt], 32);
      if (g == 0) s_m[wave][rt * 16 + c16] = rows.m[rt], s_l[wave][rt * 16 + c16] = rows.sum[rt];
    }
    __syncthreads();
    const __amdgpu_buffer_rsrc_t res = __builtin_amdgcn_make_buffer_rsrc((void*)l.partial, (short)0, 0x7FFFFFFF, kRsrc);
    const int slot = (it.first + it.piece) * S::kBytes;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if (rt * 16 >= rows_here) break;
      const int row = rt * 16 + c16;
      float top = s_m[0][row];
#pragma unroll
      for (int w = 1; w < W; ++w) top = fmaxf(top, s_m[w][row]);
      float weight = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) weight += s_l[w][row] * __builtin_amdgcn_exp2f(s_m[w][row] - top);
      const float f = __builtin_amdgcn_exp2f(rows.m[rt] - top) * rows.vref;
      if (rt > 0) __syncthreads();  // the previous tile's sums have been read
#pragma unroll
      for (int d = 0; d < DT; ++d)
        *reinterpret_cast<float4v*>(s_o + ((wave * DT + d) * 64 + lane) * 4) = rows.o[d][rt] * f;
      __syncthreads();
#pragma unroll
      for (int d = wave; d < DT; d += W) {
        float4v sum = *reinterpret_cast<const float4v*>(s_o + (d * 64 + lane) * 4);
#pragma unroll
        for (int w = 1; w < W; ++w) sum += *reinterpret_cast<const float4v*>(s_o + ((w * DT + d) * 64 + lane) * 4);
        if (it.pieces == 1) {
          if (row < rows_here) write_y(a, l.group, q, it.head, row_first + row, 16 * d + 4 * g, DIM, sum, weight);
        } else {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, sum), res, slot + S::fragment(rt, d, lane), 0, kDevScope);
          if (d == 0 && g == 0)
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, float2v{top, weight}), res,
                                                  slot + S::row(rt, c16), 0, kDevScope);
        }
      }
    }
    if (it.pieces > 1) join_pieces<DIM, RT, W>(a, l, it, q, lane, wave, row_first, rows_here, &s_arrival);
    __syncthreads();  // LDS is free for the next item
  }
}

// ---------------------------------------------------------------------------
// Many rows: a workgroup's wavefronts share each page through LDS.
//
// Two buffers of a page: while one is used, the next page is on its way into
// registers, and it goes to the other buffer behind the arithmetic, so there
// is one barrier a page.  16-byte units of values are stored turned by
// (dimension / 4) % 4 within their dimension's four, so that the 16 lanes
// that read one group of 16 dimensions meet all LDS banks.
// ---------------------------------------------------------------------------
template <int DIM, int RT>
__global__ __launch_bounds__(kManyWaves * 64, 2) void attention_many_kernel(AttentionArgs a, AttnLaunch l) {
  using R = Rows<DIM, RT>;
  using S = Slot<DIM, RT * kManyWaves>;
  constexpr int DT = R::DT, KS = R::KS, ROWS = 16 * RT * kManyWaves, THREADS = kManyWaves * 64;
  constexpr int UNITS = kKvPage * DIM / 16;    // 16-byte units of a block
  constexpr int PER = UNITS / THREADS;         // of a thread
  __shared__ __attribute__((aligned(16))) u32x4 s_k[2][UNITS], s_v[2][UNITS];
  __shared__ uint32_t s_arrival;
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
    const View<1> all = view_of<1>(a, l.group, q, lane, tile_first, tile_rows);
    View<RT> see = view_of<RT>(a, l.group, q, lane, row_first, some ? rows_here : 1);
    if (!some) see.lim_min = 0;  // no page is an ordinary one
    const int lo = max(q.first_page + (int)((int64_t)q.pages * it.piece / it.pieces), all.low_min / kKvPage);
    const int hi = min(q.first_page + (int)((int64_t)q.pages * (it.piece + 1) / it.pieces),
                       (all.lim_max + kKvPage - 1) / kKvPage);
    const int32_t* const table = a.table + it.request * a.table_stride;
    Pages pages;
    pages.load(a, table, it.head, q.bad, lane, lo, 1, hi);
    half8 qr[RT][KS];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) load_query<DIM>(a, l.group, q, it.head, lane, row_first, rows_here, rt, qr[rt]);
    R rows;
    rows.begin(Pages::at(pages.vs, 0));

    u32x4 kr[PER], vr[PER];
    auto load = [&](int64_t block) {
      const u32x4* const ks = reinterpret_cast<const u32x4*>(a.cache.k + block * (kKvPage * DIM));
      const u32x4* const vs = reinterpret_cast<const u32x4*>(a.cache.v + block * (kKvPage * DIM));
#pragma unroll
      for (int i = 0; i < PER; ++i) kr[i] = ks[i * THREADS + tid];
#pragma unroll
      for (int i = 0; i < PER; ++i) vr[i] = vs[i * THREADS + tid];
    };
    auto put = [&](int buffer) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int u = i * THREADS + tid;
        s_k[buffer][u] = kr[i];
        s_v[buffer][u ^ ((u >> 4) & 3)] = vr[i];
      }
    };
    if (lo < hi) {
      load(pages.block_at(0));
      put(0);
    }
    int page = lo;
    float kc = 0.0f, vs = 0.0f;
    int buffer = 0;
    // Page `page` and the next one's way into the other buffer; every
    // wavefront of the workgroup goes through the same barriers.
    const auto key = [&](int u, int t) { return s_k[buffer][(4 * u + g) * kKvPage + 16 * t + c16]; };
    const auto query = [&](int i, int rt) { return qr[rt][i]; };
    const auto value = [&](int d) { return s_v[buffer][(16 * d + c16) * 4 + (g ^ (c16 >> 2))]; };
    const auto none = [] {};
    const auto open = [&] {
      const int i = (page - lo) & 63;
      buffer = (page - lo) & 1;
      kc = Pages::at(pages.kc, i), vs = Pages::at(pages.vs, i);
      __syncthreads();  // this page is in LDS, the other buffer has been read
      if (page + 1 < hi) {
        if (i == 63) pages.load(a, table, it.head, q.bad, lane, page + 1, 1, hi);
        load(pages.block_at((i + 1) & 63));
      }
    };
    if (page < hi) open();
    while (page < hi) {
      while (rows.ordinary(kc, vs, page * kKvPage, see)) {
        rows.template page<false>(key, query, value, none, kc, vs, 0, g, see);
        if (page + 1 < hi) put(buffer ^ 1);
        if (++page == hi) break;
        open();
      }
      if (page < hi) {
        const int base = page * kKvPage;
        if (some && base < see.lim_max && base + kKvPage > see.low_min)
          rows.template page<true>(key, query, value, none, kc, vs, base, g, see);
        if (page + 1 < hi) put(buffer ^ 1);
        if (++page < hi) open();
      }
    }

    const __amdgpu_buffer_rsrc_t res = __builtin_amdgcn_make_buffer_rsrc((void*)l.partial, (short)0, 0x7FFFFFFF, kRsrc);
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
            write_y(a, l.group, q, it.head, row_first + rt * 16 + c16, 16 * d + 4 * g, DIM, sum, weight);
        } else {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, sum), res,
                                                 slot + S::fragment(wave * RT + rt, d, lane), 0, kDevScope);
        }
      }
      if (it.pieces > 1 && g == 0)
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, float2v{rows.m[rt], weight}), res,
                                              slot + S::row(wave * RT + rt, c16), 0, kDevScope);
    }
    if (it.pieces > 1) join_pieces<DIM, RT * kManyWaves, kManyWaves>(a, l, it, q, lane, wave, tile_first, tile_rows, &s_arrival);
    __syncthreads();  // LDS is free for the next item
  }
}

// Segments of a call whose requests all bring max_rows rows.
int64_t most_segments(int requests, int max_rows, int q_heads, int heads, int dim) {
  const int64_t rows = (int64_t)max_rows * (q_heads / heads);
  const Form f = form_for(rows, dim);
  const int64_t tiles = (rows + f.rows() - 1) / f.rows();
  return (int64_t)requests * heads * (tiles < 1 ? 1 : tiles);
}

// Pieces wanted: what the chip holds at once (one workgroup a CU of few rows, two
// of many), or four times as many and smaller when there are so many segments
// that whole ones would leave it unevenly loaded.
int wanted_pieces(const Form& f, int64_t segments) {
  const int at_once = f.many ? 512 : 256;
  return segments * 2 <= at_once ? at_once : kMaxPieces;
}

size_t slot_bytes(const Form& f, int dim) { return (size_t)f.rows() * dim * 4 + (size_t)f.rows() * 8; }

template <typename Kernel>
hipError_t launch_kernel(Kernel kernel, int threads, size_t lds, const AttentionArgs& a, const AttnLaunch& l,
                         int64_t grid) {
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  kernel<<<dim3((uint32_t)grid), dim3(threads), lds, (hipStream_t)a.stream>>>(a, l);
  return hipGetLastError();
}

template <int DIM>
hipError_t launch_dim(const Form& f, const AttentionArgs& a, const AttnLaunch& l, int64_t grid) {
  if (f.many) {
    if (f.tiles == 1) return launch_kernel(attention_many_kernel<DIM, 1>, kManyWaves * 64, 0, a, l, grid);
    return launch_kernel(attention_many_kernel<DIM, 2>, kManyWaves * 64, 0, a, l, grid);
  }
  const auto few = [&](auto kernel, int waves) {
    return launch_kernel(kernel, waves * 64, (size_t)waves * DIM / 16 * 1024, a, l, grid);
  };
  if (f.tiles == 1) return few(attention_few_kernel<DIM, 1>, few_waves(DIM, 1));
  if constexpr (DIM < 256) {
    if (f.tiles == 2) return few(attention_few_kernel<DIM, 2>, few_waves(DIM, 2));
    return few(attention_few_kernel<DIM, 3>, few_waves(DIM, 3));
  }
  return hipErrorInvalidValue;
}

}  // namespace

size_t attention_scratch_bytes(int requests, int max_rows, int q_heads, int heads, int dim, int table_width) {
  const int64_t segments = most_segments(requests, max_rows, q_heads, heads, dim);
  if (table_width <= kMinPiecePages || segments >= kMaxPieces) return kKvZeroedBytes;
  const Form f = form_for((int64_t)max_rows * (q_heads / heads), dim);
  const size_t slots = wanted_pieces(f, segments);
  return kKvZeroedBytes + (slots + slots / 2) * slot_bytes(f, dim);
}

hipError_t launch_attention(const AttentionArgs& a) {
  const int dim = a.cache.dim, group = a.q_heads / a.cache.heads;
  const Form f = form_for((int64_t)a.max_rows * group, dim);
  const int64_t segments = most_segments(a.requests, a.max_rows, a.q_heads, a.cache.heads, dim);
  AttnLaunch l;
  l.tile_rows = f.rows();
  l.group = group;
  l.target = wanted_pieces(f, segments);
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
