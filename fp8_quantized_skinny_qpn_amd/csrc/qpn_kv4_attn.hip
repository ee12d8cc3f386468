// qpn_kv4_attn.hip -- attention of a round's rows over the 4-bit paged KV cache
// on gfx950.
//
// y = unit_v sum_j w_j v_j / sum_j w_j, w_j = exp(scale unit_k q . k_j - m), over the
// tokens a row sees; k_j and v_j are E2M1 codes times the E4M3 scale of their 16
// dimensions.  Such a product has at most 6 significant bits and lies in
// [2^-10, 2688] (or is zero), so the FP16 operands that codes and scales are turned
// into in registers are exact; both products run on the 16x16x32 f16 MFMA with FP32
// accumulation.
//
// One pass, transposed, as over the 8-bit cache: S^T = K Q^T leaves a lane 16 tokens
// of one row, which after the exponentials are the B operand of O^T = V^T P^T without
// any exchange between lanes.  The layout (include/qpn_kv4.h) hands each lane whole
// groups of 16 dimensions: a key group is two k-steps of the first product under one
// scale; of values a lane holds, for each of its 16 tokens, the DIM / 16 dimensions
// that it feeds to the dimension tiles of the second, in DIM / 64 groups.  A byte of
// values holds two dimensions of one token (an append then writes whole bytes of its
// own); the operands want two tokens of one dimension, so words of two tokens are
// interleaved first (a quarter of an operation a code).  The running maximum of a row is
// only raised when a score exceeds it by more than 2^8.  FP16 weights are off by 2^-11
// of each (below 2^-14 by 2^-25), as far as the output is by its own rounding.
#include "qpn_kv_attn_core.h"

namespace qpn {

namespace {

constexpr int kFewWaves = 8;

template <>
struct KindOf<Attention4Args> {
  static constexpr int few_tiles(int dim) { return dim == 256 ? 1 : 3; }
  static constexpr int many_tiles(int dim) { return dim == 256 ? 1 : 2; }
  // Several tiles of a KV head in one workgroup decode its codes once, but leave as many times
  // the sums to join: with few segments, up to some length, a workgroup a tile is the faster
  // one.  8 rows of 40 + 8 heads of 128 (three tiles) over 300 / 1000 / 5001 / 32000 / 64000
  // tokens: together 12.7 / 15.5 / 19.3 / 29.0 / 35.7 us, apart 8.8 / 11.4 / 12.7 / 24.2 / 35.4
  // (131001: 56.8 and 68.4); of 64 dimensions together 10.1 / 12.6 / 15.2 / 23.0 / 27.2, apart
  // 8.9 / 9.8 / 10.9 / 18.6 / 25.5; of 256 there is one tile.  3 requests of them over up to 4000
  // 20.7 and 19.9, 4 over up to 8000 27.5 and 28.5.  Where no segment is cut, while a workgroup
  // each finds a CU: 10 requests over up to 500 tokens 14.7 and 9.9, 16 of them 14.5 and 23.2.
  // What the host knows of the lengths is the table's width (the longest request it has room
  // for), and that decides: in a table of more than 24576 pages over tiles x groups (1024 for
  // these heads) short requests take the tiles together, 5001 tokens 19.3 us.
  static constexpr bool apart(int64_t tiles, int64_t groups, int64_t pages) {
    return tiles * groups <= (pages <= kMinPiecePages ? 256 : 80) && tiles * groups * pages <= 24576;
  }
  static constexpr int at_once(int n) { return n >= 3 ? 4 : 8; }
  static constexpr int kJoinDirect = 16;
  // lane group g of the accumulators holds dimensions 16 (G g + i) + 4 j + b, b = 0 .. 3,
  // of the dimension tile d = 4 i + j
  template <int DIM>
  static __device__ __forceinline__ int first_dim(int d, int g) { return (DIM / 4) * g + 4 * d; }
};

// Byte `at` (0 .. 3) of a word of codes: two E2M1 values.
__device__ __forceinline__ half2v e2m1_pair(uint32_t codes, int at) {
  switch (at) {
    case 0: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 0);
    case 1: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 1);
    case 2: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 2);
    default: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 3);
  }
}
// Bytes 2 at, 2 at + 1 of a word of scales.
__device__ __forceinline__ half2v scale_pair(uint32_t scales, int at) {
  return at ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(scales, 1.0f, true)
            : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(scales, 1.0f, false);
}
__device__ __forceinline__ half2v both(half2v s, int which) { return half2v{s[which], s[which]}; }

// A page's keys in a lane: G groups of 16 dimensions of the tokens 16 t + c16.
template <int DIM>
struct Keys {
  static constexpr int G = DIM / 64, LOADS = DIM / 32;
  u32x4 codes[LOADS];
  uint32_t scales[G];  // byte n = t G + i

  __device__ __forceinline__ void load(const KvCache4& c, int64_t block, int lane) {
    const __amdgpu_buffer_rsrc_t res = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(c.k + block * kv4_codes(DIM)), (short)0, kv4_codes(DIM), kRsrc);
#pragma unroll
    for (int j = 0; j < LOADS; ++j)
      codes[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(res, lane * 16, j * 1024, 0));
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(c.k_scale + block * kv4_scales(DIM)), (short)0, kv4_scales(DIM), kRsrc);
    if constexpr (G == 1) {
      scales[0] = __builtin_amdgcn_raw_buffer_load_b32(rs, lane * 4, 0, 0);
    } else if constexpr (G == 2) {
      const u32x2 s = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, lane * 8, 0, 0));
      scales[0] = s[0], scales[1] = s[1];
    } else {
      const u32x4 s = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, lane * 16, 0, 0));
#pragma unroll
      for (int i = 0; i < 4; ++i) scales[i] = s[i];
    }
  }
  // The A operand of tile t, k-step 2 i + h: dimensions 8 h + e of group i.
  __device__ __forceinline__ half8 operand(int t, int i, int h) const {
    const int n = t * G + i;
    return decode_e2m1x8(codes[n / 2][2 * (n % 2) + h], both(scale_pair(scales[n / 4], n / 2 % 2), n % 2));
  }
};

// Half bytes of two words a, b interleaved: byte m holds half byte 2 m (odd: 2 m + 1)
// of a below that of b.
__device__ __forceinline__ uint32_t even_halves(uint32_t a, uint32_t b) {
  return (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
}
__device__ __forceinline__ uint32_t odd_halves(uint32_t a, uint32_t b) {
  return ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
}

// A page's values in a lane: DIM / 16 dimensions d = 4 i + j of the 16 tokens
// 16 t + 4 g + r.
template <int DIM>
struct Values {
  static constexpr int G = DIM / 64, LOADS = DIM / 32, DT = DIM / 16;
  u32x4 codes[LOADS];
  u32x4 scales[G];  // byte r of word t

  __device__ __forceinline__ void load(const KvCache4& c, int64_t block, int lane) {
    const __amdgpu_buffer_rsrc_t res = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(c.v + block * kv4_codes(DIM)), (short)0, kv4_codes(DIM), kRsrc);
#pragma unroll
    for (int j = 0; j < LOADS; ++j)
      codes[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(res, lane * 16, j * 1024, 0));
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(c.v_scale + block * kv4_scales(DIM)), (short)0, kv4_scales(DIM), kRsrc);
#pragma unroll
    for (int i = 0; i < G; ++i)
      scales[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, (lane >> 2) * 16, i * 256, 0));
  }

  // The two tokens 2 rp, 2 rp + 1 of tile t, the eight dimensions 8 w on, interleaved
  // (of 64 dimensions: both pairs of the tile in one word).
  __device__ __forceinline__ uint32_t pairs(int t, int rp, int w, int odd) const {
    uint32_t a, b;
    if constexpr (G == 1) {
      const uint32_t x = codes[t / 2][2 * (t % 2)], y = codes[t / 2][2 * (t % 2) + 1];
      a = __builtin_amdgcn_perm(y, x, 0x05040100u), b = __builtin_amdgcn_perm(y, x, 0x07060302u);
    } else if constexpr (G == 2) {
      a = codes[t][2 * rp], b = codes[t][2 * rp + 1];
    } else {
      a = codes[2 * t + rp][w], b = codes[2 * t + rp][2 + w];
    }
    return odd ? odd_halves(a, b) : even_halves(a, b);
  }
  // The A operand of the dimension tile d, tokens of the tiles 2 h and 2 h + 1.
  __device__ __forceinline__ half8 operand(int d, int h) const {
    half8 f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int t = 2 * h + q / 2, rp = q % 2;
      const half2v x = e2m1_pair(pairs(t, rp, d / 8, d % 2), G == 1 ? 2 * rp + d / 2 : d % 8 / 2) *
                       scale_pair(scales[d / 4][t], rp);
      f[2 * q] = x[0], f[2 * q + 1] = x[1];
    }
    return f;
  }

  // The values of a page that some rows see only a part of: NaN scales are taken out, and
  // put into the sums of the rows that see them.  (What is not seen has no weight, and
  // codes and other scales are numbers, whatever is there.)
  template <int RT>
  __device__ __forceinline__ void clean(int base, int g, const View<RT>& see, float4v (&o)[DT][RT]) {
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
      for (int t = 0; t < 4; ++t) any |= nan_bytes(scales[i][t]);
    if (__builtin_expect(__ballot(any != 0) == 0, 1)) return;
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t n0 = nan_bytes(scales[i][2 * h]) >> 7, n1 = nan_bytes(scales[i][2 * h + 1]) >> 7;
        const half8 nan = decode_e4m3x8(n0 * 0x38u, n1 * 0x38u);  // E4M3 ones
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            spread_nan(nan, seen_of(see.lim[rt], see.low(rt), base + 32 * h, g), o[4 * i + j][rt]);
        scales[i][2 * h] &= ~(n0 * 255u);
        scales[i][2 * h + 1] &= ~(n1 * 255u);
      }
  }
};

// The blocks of up to 64 pages of a request, one a lane: entries first + lane * step
// below end; -1 for one that is not in the cache.
__device__ __forceinline__ int load_ids(const Attention4Args& a, const int32_t* table, bool bad, int lane, int first,
                                        int step, int end) {
  const int page = first + lane * step;  // (below 2^25 + 64 * 8)
  int id = -1;
  if (page < end && page < a.table_width && !bad) {
    const int32_t x = table[page];
    if (x >= 0 && x < a.cache.pages) id = x;
  }
  return id;
}
__device__ __forceinline__ int64_t block_of(const Attention4Args& a, int head, int id) {
  return (int64_t)(id < 0 ? 0 : id) * a.cache.heads + head;
}

// A head's unit; NaN for one that no append takes (zero, negative, infinite, NaN).
__device__ __forceinline__ float unit_of(const float* units, int head) {
  const float u = units[head];
  return u > 0.0f && u < __builtin_inff() ? u : __builtin_nanf("");
}

// Q: B operand of row tile t: lane (row c16, k 8 g + e) of k-step 2 i + h has
// dimensions 16 (G g + i) + 8 h + e.  Rows behind `rows` are zeros.
template <int DIM>
__device__ __forceinline__ void load_query(const Attention4Args& a, const AttnLaunch& l, const Req& r, int head,
                                           int lane, int first, int rows, int t, half8 (&q)[DIM / 32]) {
  const int c16 = lane & 15, g = lane >> 4;
  const bool in = t * 16 + c16 < rows;
  const int rr = in ? first + t * 16 + c16 : 0, row = row_of(l, rr);
  const uint16_t* src = a.q + (int64_t)(r.row0 + row) * a.q_stride +
                        (int64_t)(head * l.group + (rr - row * l.group)) * DIM + (DIM / 4) * g;
#pragma unroll
  for (int k = 0; k < DIM / 32; ++k)
    q[k] = in ? *reinterpret_cast<const half8*>(src + 8 * k) : half8{};
}

// -inf for what a row does not see of half a page's scores; the largest of a lane's eight.
template <int RT>
__device__ __forceinline__ void mask_half(float4v (&x)[2][RT], int base, int g, const View<RT>& see) {
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const uint32_t seen = seen_of(see.lim[rt], see.low(rt), base, g);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t ones = all_ones_if(seen, t, r);
        const float y = x[t][rt][r];  // (a bit cast of an element itself reads the vector's first one)
        x[t][rt][r] = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, y) & ones) | (0xFF800000u & ~ones));
      }
  }
}
template <int RT>
__device__ __forceinline__ float half_max(const float4v (&x)[2][RT], int rt) {
  float mx = fmaxf(x[0][rt][0], x[0][rt][1]);
#pragma unroll
  for (int i = 2; i < 8; i += 2) mx = fmaxf(fmaxf(mx, x[i >> 2][rt][i & 3]), x[i >> 2][rt][(i & 3) + 1]);
  return mx;
}

// ---------------------------------------------------------------------------
// Few rows: each wavefront takes pages of its own, all rows of the segment, straight
// into registers; the workgroup's wavefronts are joined through LDS at the end.
//
// Bound by instructions and the bytes of the cache (4.5 bits a value) alike: of 8 rows of 5 query
// heads a page costs a wavefront 102 matrix instructions, 48 exponentials and the conversion of
// 16384 codes, on a SIMD that two wavefronts share; over 244608 tokens vector instructions are
// issued 66% of the time and the matrix unit is busy 35%, at 3.4 TB/s.  Half a page
// at a time, 32 tokens, a k-step of the second product: scores and weights of a whole page
// leave no registers for the next page's codes, which are loaded as soon as this page's last
// are converted (104 us by whole pages, 87 by halves).  Codes through a ring in LDS, which
// would have more of them on their way, lose (92): what LDS gives back has to be waited for
// again.  Calls one behind another: 8 rows over 244608 tokens, 40 + 8 heads of 128, 282 MB, 82 us;
// 64 requests of up to 12000 tokens (10 + 2 heads, 102 MB) 40; 8 rows over 5001 tokens 12.5; one
// row over 300 8.6.
// ---------------------------------------------------------------------------
template <int DIM, int RT>
struct FewLds {
  static constexpr int W = kFewWaves, KS = DIM / 32, DT = DIM / 16, ROWS = 16 * RT;
  static constexpr int BUFFERS = RT > 1 ? 2 : 1;
  float4v o[BUFFERS][W][DT][64];  // a row tile's sums of each wavefront
  half8 q[KS][RT][64];            // operands of the first product
  float m[ROWS][W], sum[ROWS][W];
};

template <int DIM, int RT>
__global__ __launch_bounds__(kFewWaves * 64) void attention4_few_kernel(Attention4Args a, AttnLaunch l) {
  using S = Slot<DIM, RT>;
  using L = FewLds<DIM, RT>;
  constexpr int W = L::W, KS = L::KS, ROWS = L::ROWS, DT = L::DT;
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
    // The piece's pages that the tile sees.  Of two wavefronts on a SIMD the older one issues
    // first; with much to compute it is 5/3 as fast, and gets as many more pages: the older
    // four the first part, the others the rest, each every fourth page.
    const int first_page = max(q.first_page + (int)((int64_t)q.pages * it.piece / it.pieces), see.low_min / kKvPage);
    const int end_page = min(q.first_page + (int)((int64_t)q.pages * (it.piece + 1) / it.pieces),
                       (see.lim_max + kKvPage - 1) / kKvPage);
    constexpr int STEP = W / 2, SHARE = RT > 1 ? 5 : 4;  // (eighths)
    const int all_pages = max(end_page - first_page, 0);
    const int part = all_pages <= STEP ? all_pages : STEP * ((SHARE * all_pages + 4 * STEP) / (8 * STEP));
    const int lo = first_page + (wave < STEP ? wave : part + wave - STEP), hi = wave < STEP ? first_page + part : end_page;
    const int count = hi > lo ? (hi - lo + STEP - 1) / STEP : 0;
    const int32_t* const table = a.table + it.request * a.table_stride;
    static_assert(RT <= W, "a row tile of queries per wavefront");
    half8 qr[KS];
    if (wave < RT) load_query<DIM>(a, l, q, it.head, lane, row_first, rows_here, wave, qr);
    int ids = load_ids(a, table, q.bad, lane, lo, STEP, hi);
    const float factor = unit_of(a.cache.k_unit, it.head) * (a.scale * 1.44269504088896340736f);
    // (positive and finite, so that -inf stays what it is)
    const float kc = fminf(fmaxf(factor, 0x1p-126f), 0x1p127f);
    const float v_unit = unit_of(a.cache.v_unit, it.head);

    Keys<DIM> k;
    Values<DIM> v;
    int id = __builtin_amdgcn_readfirstlane(ids);
    if (count > 0) {
      k.load(a.cache, block_of(a, it.head, id), lane);
      v.load(a.cache, block_of(a, it.head, id), lane);
    }
    if (wave < RT) {
#pragma unroll
      for (int i = 0; i < KS; ++i) s.q[i][wave][lane] = qr[i];
    }
    lds_barrier();

    float m[RT];
    float4v o[DT][RT], sum[RT];  // (the weights' sums by the matrix unit, too: all four the same)
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      m[rt] = kLowest;
      sum[rt] = float4v{0, 0, 0, 0};
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d][rt] = float4v{0, 0, 0, 0};
    }
    const half8 ones = {1, 1, 1, 1, 1, 1, 1, 1};

#pragma unroll 1
    for (int i0 = 0; i0 < count; ++i0) {
      const int base = (lo + i0 * STEP) * kKvPage;
      const float none_factor = id < 0 || factor != factor ? __builtin_nanf("") : 1.0f;  // no page, or no unit
      // the next page (the last one again behind it)
      if (((i0 + 1) & 63) == 0) ids = load_ids(a, table, q.bad, lane, lo + (i0 + 1) * STEP, STEP, hi);
      const int next = i0 + 1 < count ? __builtin_amdgcn_readlane(ids, (i0 + 1) & 63) : id;
      const int64_t next_block = block_of(a, it.head, next);
      const bool edge = base + kKvPage > see.lim_min || base < see.low_max;
      if (edge) v.template clean<RT>(base, g, see, o);
      const float kp = edge ? kc : kc * none_factor;  // (at the edge NaN only for rows that see the page)

      // by halves of the page, 32 tokens, a k-step of the second product
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float4v x[2][RT];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) x[t][rt] = float4v{0, 0, 0, 0};
#pragma unroll
        for (int k0 = 0; k0 < KS; ++k0) {
          half8 qf[RT];
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) qf[rt] = s.q[k0][rt][lane];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const half8 kf = k.operand(2 * h + t, k0 / 2, k0 % 2);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
              x[t][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[rt], x[t][rt], 0, 0, 0);
          }
        }
        if (h == 1) k.load(a.cache, next_block, lane);
        if (edge) {  // what a row does not see is -inf
          int gg = g;
          asm volatile("; edge" : "+v"(gg));  // (all of this in the branch, not a select of every score)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) x[t][rt] *= none_factor;
          mask_half<RT>(x, base + 32 * h, gg, see);
        }
        float high[RT];
        bool raise = false;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          high[rt] = half_max<RT>(x, rt) * kp;
          raise |= high[rt] > m[rt] + kMaxSlack;
        }
        if (__ballot(raise)) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            float mx = fmaxf(high[rt], __shfl_xor(high[rt], 16));
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            const float up = fmaxf(m[rt], mx);
            const float f = __builtin_amdgcn_exp2f(m[rt] - up);
            sum[rt] *= f;
            m[rt] = up;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d][rt] *= f;
          }
        }
        half8 p[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              x[t][rt][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][rt][r], kp, -m[rt]));
          p[rt] = to_half8(x[0][rt], x[1][rt]);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) sum[rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, p[rt], sum[rt], 0, 0, 0);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const half8 vf = v.operand(d, h);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            o[d][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, p[rt], o[d][rt], 0, 0, 0);
        }
      }
      v.load(a.cache, next_block, lane);
      id = next;
    }

    // the wavefronts' sums against their common maximum
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if (g == 0) s.m[rt * 16 + c16][wave] = m[rt], s.sum[rt * 16 + c16][wave] = sum[rt][0];
    }
    lds_barrier();
    const __amdgpu_buffer_rsrc_t res = partial_of(l);
    const int slot = (it.first + it.piece) * S::kBytes;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if (rt * 16 >= rows_here) break;
      float top = kLowest, weight = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) top = fmaxf(top, s.m[rt * 16 + c16][w]);
#pragma unroll
      for (int w = 0; w < W; ++w) weight += s.sum[rt * 16 + c16][w] * __builtin_amdgcn_exp2f(s.m[rt * 16 + c16][w] - top);
      const float f = __builtin_amdgcn_exp2f(m[rt] - top) * v_unit;
      float4v(*const sums)[DT][64] = s.o[rt % L::BUFFERS];
#pragma unroll
      for (int d = 0; d < DT; ++d) sums[wave][d][lane] = o[d][rt] * f;
      lds_barrier();
#pragma unroll
      for (int d = wave; d < DT; d += W) {
        float4v all = sums[0][d][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) all += sums[w][d][lane];
        if (it.pieces == 1) {
          if (rt * 16 + c16 < rows_here)
            write_y(a, l, q, it.head, row_first + rt * 16 + c16, KindOf<Attention4Args>::template first_dim<DIM>(d, g),
                    DIM, all, weight);
        } else {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, all), res, S::fragment(rt, d, lane), slot,
                                                 kDevScope);
        }
      }
      if (it.pieces > 1 && wave == 0 && g == 0)
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, float2v{top, weight}), res, S::row(rt, c16),
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
// A operands.  The scores of the next page are computed beside the weights of this
// one, so that the matrix and the vector units work at the same time; keys are
// therefore one page ahead of values.  Two buffers of each, one barrier a page.
//
// Bound by the matrix and the vector units, which two wavefronts a SIMD keep from waiting for one
// another only in part: of a page's 5200 cycles the matrix unit is busy 2190 (a SIMD's two
// wavefronts have 64 instructions of 16 cycles each for the products, and the weights' sums) and
// vector instructions are issued in 2470; LDS is busy 1450.  The codes of the next page are loaded
// a step ahead, 1 KiB of them a wavefront (of 128 dimensions: four have keys, four values).  256
// rows over 16500 tokens, 40 + 8 heads of 128: 108 us for both kernels, calls one behind another
// (796 TFLOP/s); under the profiler 102 and 9.6 for the join.
// ---------------------------------------------------------------------------
template <int DIM>
struct ManyLds {
  half8 k[2][DIM / 8][64], v[2][DIM / 8][64];  // operands: buffer, operand, lane
  int nan;                                     // scales of values that only some rows of the tile see held NaN
};

template <int DIM, int RT>
__global__ __launch_bounds__(kManyWaves * 64) void attention4_many_kernel(Attention4Args a, AttnLaunch l) {
  using R = Rows<DIM, RT, true>;
  using S = Slot<DIM, RT * kManyWaves>;
  constexpr int DT = R::DT, KS = R::KS, ROWS = 16 * RT * kManyWaves, G = DIM / 64;
  constexpr int LOADS = DIM / 32;                                    // 1 KiB of codes each, of the keys or the values
  constexpr int MINE = 2 * LOADS / kManyWaves > 0 ? 2 * LOADS / kManyWaves : 1;  // of a wavefront
  using L = ManyLds<DIM>;
  extern __shared__ __attribute__((aligned(16))) uint8_t s_many[];
  L& lds = *reinterpret_cast<L*>(s_many);
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
    int now = load_ids(a, table, q.bad, lane, lo, 1, hi);  // of the 64 pages around the present ones
    half8 qr[RT][KS];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) load_query<DIM>(a, l, q, it.head, lane, row_first, rows_here, rt, qr[rt]);
    const float factor = unit_of(a.cache.k_unit, it.head) * (a.scale * 1.44269504088896340736f);
    const float kc = fminf(fmaxf(factor, 0x1p-126f), 0x1p127f);  // (as above)
    const float v_unit = unit_of(a.cache.v_unit, it.head);
    if (threadIdx.x == 0) lds.nan = 0;
    lds_barrier();
    R rows;
    rows.begin(1.0f);

    // The loads of a page, in turn to the wavefronts: wavefront w has loads w, w + 8, ..
    // of first the keys' LOADS, then the values'.
    const auto has = [&](int j) { return j * kManyWaves + wave < 2 * LOADS; };
    const auto is_key = [&](int j) { return j * kManyWaves + wave < LOADS; };
    const auto number = [&](int j) { return (j * kManyWaves + wave) % LOADS; };
    // The same instructions for both: a branch between them would end in moves of what is loaded,
    // and so in a wait for it.
    constexpr int WORDS = G == 1 ? 2 : G;  // of scales: of keys the first, of values (G > 1) one a group
    u32x4 held[MINE];
    uint32_t scale[MINE][WORDS];
    const auto fetch = [&](int j, int64_t at) {
      if constexpr (2 * LOADS % kManyWaves != 0)
        if (!has(j)) return;
      const int n = number(j), step = is_key(j) ? 0 : G == 1 ? 4 : 256;
      held[j] = *reinterpret_cast<const u32x4*>((is_key(j) ? a.cache.k : a.cache.v) + at * kv4_codes(DIM) + n * 1024 + lane * 16);
      // of keys bytes 2 n, 2 n + 1 of the lane's 4 G; of values the tokens of the load, 16 / LOADS of each group
      const uint8_t* const from = (is_key(j) ? a.cache.k_scale : a.cache.v_scale) + at * kv4_scales(DIM);
      const uint32_t in_lane = is_key(j) ? lane * (4 * G) + (2 * n & ~3) : (lane >> 2) * 16 + (n * (16 / LOADS) & ~3);
#pragma unroll
      for (int i = 0; i < WORDS; ++i) scale[j][i] = *reinterpret_cast<const uint32_t*>(from + step * i + in_lane);
    };
    // Codes to operands.  Values of a page that some rows of the tile see only a part of:
    // NaN scales become zeros, and a flag is left.
    const auto put = [&](int j, int page) {
      if (!has(j)) return;
      const int n = number(j), base = page * kKvPage;
      const u32x4 x = held[j];
      if (is_key(j)) {
        const half2v sc = scale_pair(n % 2 ? scale[j][0] >> 16 : scale[j][0], 0);
#pragma unroll
        for (int u = 0; u < 2; ++u) {  // the group n' = 2 n + u = t G + i
          const int at = 2 * n + u, t = at / G, i = at % G;
#pragma unroll
          for (int h = 0; h < 2; ++h) lds.k[page & 1][(2 * i + h) * 4 + t][lane] = decode_e2m1x8(x[2 * u + h], both(sc, u));
        }
        return;
      }
      if constexpr (G == 4) {  // two of a word's four
#pragma unroll
        for (int i = 0; i < G; ++i) scale[j][i] = n % 2 ? scale[j][i] >> 16 : scale[j][i] & 0xFFFFu;
      }
      if (base + kKvPage > all.lim_min || base < all.low_max) {
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
          const uint32_t bad = nan_bytes(scale[j][i]) >> 7;
          any |= bad;
          scale[j][i] &= ~(bad * 255u);
        }
        const uint64_t some_nan = __ballot(any != 0);
        if (lane == 0 && some_nan) lds.nan = 1;
      }
      half8(*const to)[64] = lds.v[page & 1];
      if constexpr (G == 1) {  // tiles 2 n, 2 n + 1: the whole operands of k-step n
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          half8 f;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t p = __builtin_amdgcn_perm(x[2 * u + 1], x[2 * u], 0x05040100u);
            const uint32_t r = __builtin_amdgcn_perm(x[2 * u + 1], x[2 * u], 0x07060302u);
            const uint32_t w = d % 2 ? odd_halves(p, r) : even_halves(p, r);
#pragma unroll
            for (int rp = 0; rp < 2; ++rp) {
              const half2v y = e2m1_pair(w, 2 * rp + d / 2) * scale_pair(scale[j][u], rp);
              f[4 * u + 2 * rp] = y[0], f[4 * u + 2 * rp + 1] = y[1];
            }
          }
          to[2 * d + n][lane] = f;
        }
      } else if constexpr (G == 2) {  // tile n: half of the operands of k-step n / 2
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          half4 f;
#pragma unroll
          for (int rp = 0; rp < 2; ++rp) {
            const uint32_t w = d % 2 ? odd_halves(x[2 * rp], x[2 * rp + 1]) : even_halves(x[2 * rp], x[2 * rp + 1]);
            const half2v y = e2m1_pair(w, d / 2) * scale_pair(scale[j][d / 4], rp);
            f[2 * rp] = y[0], f[2 * rp + 1] = y[1];
          }
          reinterpret_cast<half4*>(&to[2 * d + n / 2][lane])[n % 2] = f;
        }
      } else {  // two tokens of tile n / 2: a quarter of the operands of k-step n / 4
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const uint32_t w = d % 2 ? odd_halves(x[d / 8], x[2 + d / 8]) : even_halves(x[d / 8], x[2 + d / 8]);
          reinterpret_cast<half2v*>(&to[2 * d + n / 4][lane])[n % 4] = e2m1_pair(w, d % 8 / 2) * scale_pair(scale[j][d / 4], 0);
        }
      }
    };
    // this wavefront's own pages among the workgroup's
    const int my_lo = some ? max(lo, see.low_min / kKvPage) : hi;
    const int my_hi = some ? min(hi, (see.lim_max + kKvPage - 1) / kKvPage) : hi;
    float4v s[4][RT];  // the scores of page my_lo and on, one page ahead
    float high[RT];    // and the largest of the lane's
    int next = now;    // of the 64 pages behind those of `now`
    const auto id_of = [&](int page, int at) {  // of `page` (the last one for any behind it), at most 64 behind lo + at
      const int n = min(page, hi - 1) - lo;
      return (n >> 6) == (at >> 6) ? __builtin_amdgcn_readlane(now, n & 63) : __builtin_amdgcn_readlane(next, n & 63);
    };
    // step `page`: the weights and values of `page`, the scores of page + 1; keys of page + 2
    // and values of page + 1 become operands
    int id = 0, id1 = 0, id2 = 0;  // of `page`, page + 1, page + 2
    int64_t at1 = 0, at2 = 0;      // where the last two are
    if (lo < hi) {
      id2 = id_of(lo, 0), at2 = block_of(a, it.head, id2);
#pragma unroll
      for (int j = 0; j < MINE; ++j) fetch(j, at2);
#pragma unroll
      for (int j = 0; j < MINE; ++j)
        if (is_key(j)) put(j, lo);
    }
#pragma unroll 1
    for (int page = lo - 1; page < hi; ++page) {
      const int at = max(page - lo, 0);
      if (at > 0 && (at & 63) == 0) now = next;
      if ((at & 63) == 32 && lo + (at | 63) + 1 < hi) next = load_ids(a, table, q.bad, lane, lo + (at | 63) + 1, 1, hi);
      lds_barrier();  // values of this page and keys of the next are in LDS, the other buffers have been read
      if (lo < hi) {
        id = id1, id1 = id2, at1 = at2;
        id2 = id_of(page + 2, at), at2 = block_of(a, it.head, id2);
#pragma unroll
        for (int j = 0; j < MINE; ++j) fetch(j, is_key(j) ? at2 : at1);
      }
      const auto key = [&](int i) { return lds.k[(page + 1) & 1][i][lane]; };
      if (page >= my_lo && page < my_hi) {
        const int base = page * kKvPage;
        if (__builtin_expect(id < 0 || factor != factor, 0)) {  // no page, or no unit: NaN to the rows that see it
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) s[t][rt] *= __builtin_nanf("");
        }
        if (base + kKvPage > see.lim_min || base < see.low_max) {
          mask_page<RT>(s, base, g, see);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) high[rt] = page_max<RT>(s, rt);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) high[rt] *= kc;
        rows.raise(high);
        half8 p[2][RT];
        float4v ahead[4][RT];  // (of a page that is not there: of what the buffer holds, and not used)
        rows.weigh(s, kc, 1.0f, p, key, qr, ahead);
        rows.accumulate([&](int i) { return lds.v[page & 1][i][lane]; }, p, ahead, 1.0f, high);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) s[t][rt] = ahead[t][rt];
      } else if (page + 1 == my_lo && my_lo < my_hi) {
        R::scores(key, qr, s);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) high[rt] = page_max<RT>(s, rt);
      }
      if (lo < hi) {
#pragma unroll
        for (int j = 0; j < MINE; ++j) put(j, is_key(j) ? page + 2 : page + 1);
      }
    }
    lds_barrier();
    if (__builtin_expect(uniform(lds.nan) != 0, 0)) {  // NaN into the rows that see it, from the pages' scales
      for (int page = my_lo; page < my_hi; ++page) {
        const int base = page * kKvPage, id = table[page];
        if ((base + kKvPage <= all.lim_min && base >= all.low_max) || id < 0 || id >= a.cache.pages) continue;
        Values<DIM> v;
        v.load(a.cache, block_of(a, it.head, id), lane);
        v.template clean<RT>(base, g, see, rows.o);
      }
    }

    const __amdgpu_buffer_rsrc_t res = partial_of(l);
    const int slot = (it.first + it.piece) * S::kBytes;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if (rt * 16 >= rows_here) break;
      const float weight = rows.sum[rt][0];
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const float4v sum = rows.o[d][rt] * v_unit;
        if (it.pieces == 1) {
          if (rt * 16 + c16 < rows_here)
            write_y(a, l, q, it.head, row_first + rt * 16 + c16, KindOf<Attention4Args>::template first_dim<DIM>(d, g),
                    DIM, sum, weight);
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

template <int DIM, int RT>
hipError_t launch_many(const Attention4Args& a, const AttnPlan& p) {
  const hipError_t e = launch_kernel(attention4_many_kernel<DIM, RT>, kManyWaves * 64, sizeof(ManyLds<DIM>), a, p.launch, p.grid);
  if (e != hipSuccess || p.launch.slots == 0) return e;
  return launch_kernel(attention_join_kernel<DIM, RT * kManyWaves, Attention4Args>, kManyWaves * 64, 0, a, p.launch, p.grid);
}

template <int DIM, int RT>
hipError_t launch_few(const Attention4Args& a, const AttnPlan& p) {
  return launch_kernel(attention4_few_kernel<DIM, RT>, kFewWaves * 64, sizeof(FewLds<DIM, RT>), a, p.launch, p.grid);
}

template <int DIM>
hipError_t launch_dim(const Attention4Args& a, const AttnPlan& p) {
  const Form& f = p.form;
  if (f.tiles == 1) return f.many ? launch_many<DIM, 1>(a, p) : launch_few<DIM, 1>(a, p);
  if constexpr (DIM < 256) {
    if (f.tiles == 2) return f.many ? launch_many<DIM, 2>(a, p) : launch_few<DIM, 2>(a, p);
    return launch_few<DIM, 3>(a, p);
  }
  return hipErrorInvalidValue;
}

}  // namespace

size_t attention4_scratch_bytes(int requests, int max_rows, int q_heads, int heads, int dim, int table_width) {
  return scratch_bytes_for<Attention4Args>(requests, max_rows, q_heads, heads, dim, table_width);
}

hipError_t launch_attention4(const Attention4Args& a) {
  const AttnPlan p = plan_of(a);
  return a.cache.dim == 64 ? launch_dim<64>(a, p) : a.cache.dim == 128 ? launch_dim<128>(a, p) : launch_dim<256>(a, p);
}

}  // namespace qpn
