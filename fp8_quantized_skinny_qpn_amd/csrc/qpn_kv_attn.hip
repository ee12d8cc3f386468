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
#include "qpn_kv_attn_core.h"

namespace qpn {

namespace {

// A load of 16 bytes a lane into LDS: lane i's go to lds + 16 i.
__device__ __forceinline__ void load_to_lds(const uint8_t* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(uniform((int)lds)), "v"(offset), "s"(base)
               : "memory", "m0");
}

// wavefronts of a workgroup, few rows: one per 16 dimensions up to eight
constexpr int few_waves(int dim) { return dim == 64 ? 4 : 8; }

// Up to what the registers of the few-rows form hold it is the faster one: 40 rows a
// head over 4099 / 131001 tokens take 19.0 / 75.1 us there and 23.4 / 104 us with many
// rows' form, 48 ragged requests of up to 40 rows 38.8 and 55.5 us.
template <>
struct KindOf<AttentionArgs> {
  static constexpr int few_tiles(int dim) { return dim == 256 ? 1 : 3; }   // what the registers hold
  static constexpr int many_tiles(int dim) { return dim == 256 ? 1 : 2; }
  static constexpr bool apart(int64_t, int64_t, int64_t) { return false; }
  static constexpr int at_once(int n) { return n >= 3 ? 4 : 8; }
  // 8 rows over 16384 tokens, 32 pieces a head: 30.6 us in one step, 26.0 us in two; over
  // 131001 tokens 78.6 and 75.1 us
  static constexpr int kJoinDirect = 16;
  template <int DIM>
  static __device__ __forceinline__ int first_dim(int d, int g) { return 16 * d + 4 * g; }
};

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

template <int DIM, int RT>
hipError_t launch_many(const AttentionArgs& a, const AttnLaunch& l, int64_t grid) {
  const hipError_t e = launch_kernel(attention_many_kernel<DIM, RT>, kManyWaves * 64,
                                     sizeof(ManyLds<DIM>) + (size_t)ManyLds<DIM>::RING * DIM * 128, a, l, grid);
  if (e != hipSuccess || l.slots == 0) return e;
  return launch_kernel(attention_join_kernel<DIM, RT * kManyWaves, AttentionArgs>, kManyWaves * 64, 0, a, l, grid);
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
  return scratch_bytes_for<AttentionArgs>(requests, max_rows, q_heads, heads, dim, table_width);
}

hipError_t launch_attention(const AttentionArgs& a) {
  const AttnPlan p = plan_of(a);
  const int dim = a.cache.dim;
  return dim == 64 ? launch_dim<64>(p.form, a, p.launch, p.grid) : dim == 128 ? launch_dim<128>(p.form, a, p.launch, p.grid)
                                                                : launch_dim<256>(p.form, a, p.launch, p.grid);
}

}  // namespace qpn
