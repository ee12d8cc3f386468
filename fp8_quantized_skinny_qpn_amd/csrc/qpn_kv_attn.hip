// qpn_kv_attn.hip -- attention of a round's rows over the 8-bit paged KV cache
// on gfx950.
//
// y = sum_j w_j v_j / sum_j w_j, w_j = exp(scale q . k_j - m), over the tokens a
// row sees.  K and V codes stay E4M3 until they are in registers, where the
// conversion to FP16 is exact; both products run on the 16x16x32 f16 MFMA with
// FP32 accumulation.  The page scale of K multiplies the scores, that of V the
// weights.
//
// One pass, transposed.  A wavefront holds 16 RT rows (query row, query head of
// the KV head's group) and takes whole pages of 64 tokens.  It computes
// S^T = K Q^T: K is the A operand, so a lane's accumulators are 16 tokens of one
// row, and after the exponentials they are, without any exchange between lanes,
// the B operand of O^T = V^T P^T.  The cache layout stores each block in the order
// these operands are read, so every load is 16 bytes a lane over whole lines
// straight into registers: no LDS and no barrier in the loop.  The running
// maximum of a row is only raised when a score exceeds it by more than 2^8
// (weights up to 2^8 fit FP16 as well as those up to 1), so most pages cost no
// exchange between lanes and no rescaling.
//
// Work split.  A segment (request, KV head, tile of rows) is cut into pieces of
// P pages, one workgroup each; the wavefronts of a workgroup take its pages in
// turn and are joined through LDS.  P comes from the lengths on the device, so
// that ragged requests fill the chip evenly with no host read.  The pieces of a
// cut segment leave their sums in scratch and a second kernel joins them in order.
#include "qpn_common.h"
#include "qpn_kv_internal.h"

namespace qpn {

namespace {

constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = kAttnThreads / kLanes;
constexpr int kMinPiecePages = kAttnWaves;  // a page for each wavefront
constexpr float kMaxSlack = 8.0f;           // how far (log2) a score may pass the running maximum
constexpr float kScaleSlack = 64.0f;        // and a page's V scale the running one
constexpr float kLowest = -1e30f;           // the running maximum before any score

// 16-row tiles of a wavefront for `rows` rows of a KV head (query rows x group).
constexpr int kMaxTiles = 4;
inline int tiles_for(int64_t rows, int dim) {
  const int most = dim == 256 ? 2 : kMaxTiles;
  const int64_t t = (rows + 15) / 16;
  return t < 1 ? 1 : t > most ? most : (int)t;
}

struct AttnLaunch {
  int tile_rows;     // 16 RT
  int64_t want;      // pieces wanted over all segments
  int64_t slots;     // pieces the scratch has room for (0: segments stay whole)
  float* partial;    // [slots][tile_rows][dim + 2]: sums, maximum, weights' sum
};

// One request as the kernels see it.
struct Req {
  int row0, rows;          // its rows (0: skipped)
  int seq;                 // tokens it sees at its last row, clamped to the table
  bool bad;                // more tokens than the table has pages for
  int first_page, pages;   // pages any of its rows sees (at least 1 when it has rows)
  int tiles;               // row tiles of a KV head
};

__device__ __forceinline__ Req request_of(const AttentionArgs& a, int r, int tile_rows) {
  Req q;
  const int s0 = a.row_start[r], s1 = a.row_start[r + 1];
  q.row0 = s0;
  q.rows = s0 >= 0 && s1 > s0 && s1 <= a.rows ? s1 - s0 : 0;
  const int64_t most = (int64_t)a.table_width * kKvPage;
  const int seq = a.seq_lens[r];
  q.bad = seq > most;
  q.seq = q.bad ? (int)most : seq < 0 ? 0 : seq;
  const int64_t start = a.window > 0 ? (int64_t)q.seq - q.rows + 1 - a.window : 0;
  q.first_page = start > 0 ? (int)(start / kKvPage) : 0;
  const int last = (q.seq + kKvPage - 1) / kKvPage;
  q.pages = last > q.first_page ? last - q.first_page : 1;
  const int group = a.q_heads / a.cache.heads;
  q.tiles = (int)(((int64_t)q.rows * group + tile_rows - 1) / tile_rows);
  return q;
}

// Sum over the workgroup, and the sum up to and including this thread.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* waves, int64_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t o = __shfl_up(x, d);
    if (lane >= d) x += o;
  }
  __syncthreads();
  if (lane == 63) waves[wave] = x;
  __syncthreads();
  int64_t before = 0;
  *total = 0;
#pragma unroll
  for (int w = 0; w < kAttnWaves; ++w) {
    if (w < wave) before += waves[w];
    *total += waves[w];
  }
  return x + before;
}

// The pages of a piece: the same for every segment, so that at most `want` cuts
// and `slots` pieces come out; everything whole when the scratch is too small.
__device__ int64_t piece_pages(const AttentionArgs& a, const AttnLaunch& l, int64_t* s_waves) {
  int64_t units = 0, segments = 0;
  for (int r = threadIdx.x; r < a.requests; r += kAttnThreads) {
    const Req q = request_of(a, r, l.tile_rows);
    if (q.rows) {
      segments += (int64_t)q.tiles * a.cache.heads;
      units += (int64_t)q.tiles * a.cache.heads * q.pages;
    }
  }
  int64_t u = units, s = segments;
  if (a.requests > 1) {
    block_scan(units, s_waves, &u);
    block_scan(segments, s_waves, &s);
  } else {
    __shared__ int64_t s_one[2];
    if (threadIdx.x == 0) s_one[0] = units, s_one[1] = segments;
    __syncthreads();
    u = s_one[0], s = s_one[1];
  }
  const int64_t cuts = l.slots - s < l.want ? l.slots - s : l.want;
  if (cuts < 1) return int64_t(1) << 40;
  const int64_t p = (u + cuts - 1) / cuts;
  return p < kMinPiecePages ? kMinPiecePages : p;
}

struct Item {
  int request;       // -1: none
  int head, tile, piece, pieces;
};

// Piece number `item` of the call: requests, then KV heads, tiles and pieces.
__device__ Item item_of(const AttentionArgs& a, const AttnLaunch& l, int64_t piece, int64_t item,
                        int64_t* s_waves, int64_t* s_found) {
  if (threadIdx.x == 0) s_found[0] = -1;
  int64_t before = 0;
  for (int base = 0; base < a.requests; base += kAttnThreads) {
    const int r = base + threadIdx.x;
    int64_t items = 0;
    if (r < a.requests) {
      const Req q = request_of(a, r, l.tile_rows);
      if (q.rows) items = (int64_t)q.tiles * a.cache.heads * ((q.pages + piece - 1) / piece);
    }
    int64_t total, up;
    if (a.requests > 1) {
      up = before + block_scan(items, s_waves, &total);
    } else {
      __syncthreads();
      up = items;
      total = 0;
    }
    if (items && item < up && item >= up - items) {
      s_found[0] = r;
      s_found[1] = item - (up - items);
    }
    before += total;
    if (before > item) break;  // the whole workgroup agrees
  }
  __syncthreads();
  Item it{(int)s_found[0], 0, 0, 0, 0};
  if (it.request >= 0) {
    const Req q = request_of(a, it.request, l.tile_rows);
    it.pieces = (int)((q.pages + piece - 1) / piece);
    const int64_t at = s_found[1];
    it.piece = (int)(at % it.pieces);
    const int64_t segment = at / it.pieces;
    it.tile = (int)(segment % q.tiles);
    it.head = (int)(segment / q.tiles);
  }
  __syncthreads();  // s_found has been read
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

template <int DIM, int RT>
__global__ __launch_bounds__(kAttnThreads) void attention_kernel(AttentionArgs a, AttnLaunch l) {
  constexpr int KS = DIM / 32;   // k-steps of the scores
  constexpr int DT = DIM / 16;   // tiles of output dimensions
  constexpr int ROWS = 16 * RT;
  constexpr int PAD = DIM + 4;   // row stride of the joined sums in LDS, in floats
  __shared__ int64_t s_waves[kAttnWaves], s_found[2];
  __shared__ float s_m[kAttnWaves][ROWS], s_l[kAttnWaves][ROWS];
  extern __shared__ __attribute__((aligned(16))) float s_o[];  // [kAttnWaves][ROWS][PAD]

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c16 = lane & 15, g = lane >> 4;
  const int group = a.q_heads / a.cache.heads;
  const int64_t piece = piece_pages(a, l, s_waves);

  for (int64_t item = blockIdx.x;; item += gridDim.x) {
    const Item it = item_of(a, l, piece, item, s_waves, s_found);
    if (it.request < 0) break;  // past the last piece: the whole workgroup leaves
    const Req q = request_of(a, it.request, l.tile_rows);
    const int row_first = it.tile * ROWS;                     // among the segment's rows
    const int rows_here = min(ROWS, q.rows * group - row_first);
    // the tokens rows see: [low, lim) per row, and over the tile's rows
    int lim[RT], low[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int rr = row_first + t * 16 + c16;
      const bool in = t * 16 + c16 < rows_here;
      lim[t] = in ? q.seq - q.rows + rr / group + 1 : 0;
      low[t] = a.window > 0 ? max(0, lim[t] - a.window) : 0;
    }
    const int lim_min = q.seq - q.rows + row_first / group + 1;
    const int lim_max = q.seq - q.rows + (row_first + rows_here - 1) / group + 1;
    const int low_min = a.window > 0 ? max(0, lim_min - a.window) : 0;
    const int low_max = a.window > 0 ? max(0, lim_max - a.window) : 0;

    // Q: B operand, lane (row c16, k 8 g + e) of k-step 2 u + h: dimensions
    // 64 u + 16 g + 8 h + e, as the key units' 16 dimensions fall to the lanes
    half8 qf[KS][RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int rr = row_first + t * 16 + c16;
      const uint16_t* src = a.q + (int64_t)(q.row0 + rr / group) * a.q_stride +
                            (int64_t)(it.head * group + rr % group) * DIM + 16 * g;
#pragma unroll
      for (int k = 0; k < KS; ++k)
        qf[k][t] = t * 16 + c16 < rows_here ? *reinterpret_cast<const half8*>(src + 64 * (k >> 1) + 8 * (k & 1))
                                            : half8{};
    }

    float m[RT], lsum[RT];
    float4v o[DT][RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      m[t] = kLowest;
      lsum[t] = 0.0f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d][t] = float4v{0, 0, 0, 0};
    }
    float vref = 0x1p-100f;  // what the sums are in units of

    // this wavefront's pages of the piece: first, first + kAttnWaves, ...
    const int64_t p_first = q.first_page + it.piece * piece + wave;
    const int64_t p_end = min(q.first_page + (it.piece + 1) * piece, (int64_t)q.first_page + q.pages);
    const int32_t* const table = a.table + it.request * a.table_stride;
    const float c_scale = a.scale * 1.44269504088896340736f;  // scores in units of log2 e

    for (int64_t p0 = p_first; p0 < p_end; p0 += 64 * kAttnWaves) {
      // up to 64 pages at a time, one a lane: block numbers and scales
      const int64_t my_page = p0 + (int64_t)lane * kAttnWaves;
      int64_t block_l = it.head;
      float ks_l = 0.0f, vs_l = 0.0f;
      if (my_page < p_end && my_page < a.table_width) {
        const int32_t id = table[my_page];
        const bool known = id >= 0 && id < a.cache.pages && !q.bad;
        if (known) block_l = (int64_t)id * a.cache.heads + it.head;
        ks_l = known ? a.cache.k_scale[block_l] * c_scale : __builtin_nanf("");
        vs_l = known ? a.cache.v_scale[block_l] : 1.0f;
      }
      const int here = (int)min((int64_t)64, (p_end - p0 + kAttnWaves - 1) / kAttnWaves);
      for (int i = 0; i < here; ++i) {
        const int64_t page = p0 + (int64_t)i * kAttnWaves;
        const int base = (int)page * kKvPage;
        if (base >= lim_max || base + kKvPage <= low_min) continue;  // no row of the tile sees it
        const int lo = __builtin_amdgcn_readlane((int)(block_l & 0xFFFFFFFF), i);
        const int hi = __builtin_amdgcn_readlane((int)(block_l >> 32), i);
        const int64_t block = ((int64_t)hi << 32) | (uint32_t)lo;
        const float kc = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ks_l), i));
        const float vs = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, vs_l), i));
        const uint8_t* const kb = a.cache.k + block * (kKvPage * DIM);
        const uint8_t* const vb = a.cache.v + block * (kKvPage * DIM);

        // K: A operand, lane (token c16 of tile t, 16 dimensions of unit 4 u + g)
        u32x4 kc4[DIM / 64][4];
#pragma unroll
        for (int u = 0; u < DIM / 64; ++u)
#pragma unroll
          for (int t = 0; t < 4; ++t)
            kc4[u][t] = *reinterpret_cast<const u32x4*>(kb + (4 * u + g) * (kKvPage * 16) + (16 * t + c16) * 16);
        // V: A operand, lane (dimension c16 of tile d, tokens 16 t + 4 g + r)
        u32x4 vc4[DT];
#pragma unroll
        for (int d = 0; d < DT; ++d)
          vc4[d] = *reinterpret_cast<const u32x4*>(vb + (16 * d + c16) * kKvPage + 16 * g);

        float4v s[4][RT];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) s[t][rt] = float4v{0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < DIM / 64; ++u)
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            half8 kf[2];
            decode_fp8_fragment(kc4[u][t], kf);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int rt = 0; rt < RT; ++rt)
                s[t][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[h], qf[2 * u + h][rt], s[t][rt], 0, 0, 0);
          }

        // scores in log2, masked where this page holds tokens a row does not see
        const bool masked = base + kKvPage > lim_min || base < low_max;
        float top[RT];
        bool raise = false;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          float mx = -__builtin_inff();
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              float z = s[t][rt][r] * kc;
              if (masked) {
                const int j = base + 16 * t + 4 * g + r;
                if (j >= lim[rt] || j < low[rt]) z = -__builtin_inff();
              }
              s[t][rt][r] = z;
              mx = fmaxf(mx, z);
            }
          top[rt] = mx;
          raise |= mx > m[rt] + kMaxSlack;
        }
        if (__ballot(raise)) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            float mx = fmaxf(top[rt], __shfl_xor(top[rt], 16));
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            const float up = fmaxf(m[rt], mx);
            const float f = exp2f(m[rt] - up);
            m[rt] = up;
            lsum[rt] *= f;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d][rt] *= f;
          }
        }
        if (vs > vref * kScaleSlack) {  // uniform over the wavefront
          const float f = vref / vs;
          vref = vs;
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d][rt] *= f;
        }
        const float vrel = vs / vref;

        half8 pf[2][RT];  // B operand of k-step h: tokens of tiles 2 h and 2 h + 1
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float w = exp2f(s[t][rt][r] - m[rt]);
              lsum[rt] += w;
              s[t][rt][r] = w * vrel;
            }
          pf[0][rt] = to_half8(s[0][rt], s[1][rt]);
          pf[1][rt] = to_half8(s[2][rt], s[3][rt]);
        }

        if (masked) {
          // codes of tokens that no row of the tile sees become zeros (what is
          // there may be anything); a NaN code that some rows see and others
          // do not is taken out too, and put into the rows that see it
          uint32_t any_nan = 0;
          uint32_t keep[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            keep[t] = 0;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int j = base + 16 * t + 4 * g + r;
              if (j < lim_max && j >= low_min) keep[t] |= 0xFFu << (8 * r);
            }
          }
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              vc4[d][t] &= keep[t];
              any_nan |= nan_bytes(vc4[d][t]);
            }
          if (__ballot(any_nan != 0)) {
            half8 sees[2][RT];  // 1 where the row sees the token
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const int j = base + 16 * (2 * h + (e >> 2)) + 4 * g + (e & 3);
                  sees[h][rt][e] = j < lim[rt] && j >= low[rt] ? (_Float16)1 : (_Float16)0;
                }
#pragma unroll
            for (int d = 0; d < DT; ++d) {
              u32x4 ones;
#pragma unroll
              for (int t = 0; t < 4; ++t) {
                const uint32_t n = nan_bytes(vc4[d][t]);    // 0x80 in NaN bytes
                vc4[d][t] &= ~((n >> 7) * 255u);
                ones[t] = (n >> 7) * 0x38u;                 // E4M3 1.0 there
              }
              half8 f[2];
              decode_fp8_fragment(ones, f);
#pragma unroll
              for (int rt = 0; rt < RT; ++rt) {
                float4v hit{0, 0, 0, 0};
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  hit = __builtin_amdgcn_mfma_f32_16x16x32_f16(f[h], sees[h][rt], hit, 0, 0, 0);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  if (hit[r] > 0.0f) o[d][rt][r] = __builtin_nanf("");
              }
            }
          }
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          half8 vf[2];
          decode_fp8_fragment(vc4[d], vf);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
              o[d][rt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[h], pf[h][rt], o[d][rt], 0, 0, 0);
        }
      }
    }

    // join the wavefronts: a common maximum per row, then the sums in order
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      lsum[rt] += __shfl_xor(lsum[rt], 16);
      lsum[rt] += __shfl_xor(lsum[rt], 32);
      if (g == 0) s_m[wave][rt * 16 + c16] = m[rt];
    }
    __syncthreads();
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int row = rt * 16 + c16;
      float top = s_m[0][row];
#pragma unroll
      for (int w = 1; w < kAttnWaves; ++w) top = fmaxf(top, s_m[w][row]);
      const float f = exp2f(m[rt] - top);
      if (g == 0) s_l[wave][row] = lsum[rt] * f;
      const float fo = f * vref;
      float* dst = s_o + ((size_t)wave * ROWS + row) * PAD + 4 * g;
#pragma unroll
      for (int d = 0; d < DT; ++d) *reinterpret_cast<float4v*>(dst + 16 * d) = o[d][rt] * fo;
    }
    __syncthreads();
    constexpr int QUADS = DIM / 4;
    for (int u = threadIdx.x; u < rows_here * QUADS; u += kAttnThreads) {
      const int row = u / QUADS, quad = u % QUADS;
      float4v sum = *reinterpret_cast<const float4v*>(s_o + (size_t)row * PAD + 4 * quad);
      float weight = s_l[0][row];
#pragma unroll
      for (int w = 1; w < kAttnWaves; ++w) {
        sum += *reinterpret_cast<const float4v*>(s_o + ((size_t)w * ROWS + row) * PAD + 4 * quad);
        weight += s_l[w][row];
      }
      if (it.pieces == 1) {
        const float inv = weight > 0.0f || weight != weight ? 1.0f / weight : 0.0f;
        const int rr = row_first + row;
        typedef _Float16 half4 __attribute__((ext_vector_type(4)));
        half4 h;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = (_Float16)(weight == 0.0f ? 0.0f : sum[e] * inv);
        *reinterpret_cast<half4*>(a.y + (int64_t)(q.row0 + rr / group) * a.y_stride +
                                  (int64_t)(it.head * group + rr % group) * DIM + 4 * quad) = h;
      } else {
        float* slot = l.partial + ((size_t)item * ROWS + row) * (DIM + 2);
        float top = s_m[0][row];
#pragma unroll
        for (int w = 1; w < kAttnWaves; ++w) top = fmaxf(top, s_m[w][row]);
        typedef float float2v __attribute__((ext_vector_type(2)));
        *reinterpret_cast<float2v*>(slot + 4 * quad) = float2v{sum[0], sum[1]};
        *reinterpret_cast<float2v*>(slot + 4 * quad + 2) = float2v{sum[2], sum[3]};
        if (quad == 0) slot[DIM] = top, slot[DIM + 1] = weight;
      }
    }
    __syncthreads();  // LDS is free for the next piece
  }
}

// Joins the pieces of cut segments: a workgroup per (row, query head) pair
// block, a thread per four dimensions.
template <int DIM>
__global__ __launch_bounds__(kAttnThreads) void attention_join_kernel(AttentionArgs a, AttnLaunch l) {
  constexpr int QUADS = DIM / 4, PAIRS = kAttnThreads / QUADS;
  __shared__ int64_t s_waves[kAttnWaves];
  const int64_t piece = piece_pages(a, l, s_waves);
  const int group = a.q_heads / a.cache.heads;
  const int64_t pair = (int64_t)blockIdx.x * PAIRS + threadIdx.x / QUADS;
  const int row = (int)(pair / a.q_heads), qh = (int)(pair % a.q_heads), quad = threadIdx.x % QUADS;
  if (row >= a.rows) return;
  int64_t before = 0;  // pieces of the requests before the row's
  for (int r = 0; r < a.requests; ++r) {
    const Req q = request_of(a, r, l.tile_rows);
    if (!q.rows) continue;
    const int pieces = (int)((q.pages + piece - 1) / piece);
    if (row >= q.row0 && row < q.row0 + q.rows) {
      if (pieces == 1) return;
      const int head = qh / group, rr = (row - q.row0) * group + qh % group;
      const int tile = rr / l.tile_rows, at = rr % l.tile_rows;
      const int64_t item = before + ((int64_t)head * q.tiles + tile) * pieces;
      const size_t step = (size_t)l.tile_rows * (DIM + 2);
      const float* const slot = l.partial + (size_t)item * step + (size_t)at * (DIM + 2);
      float top = kLowest;
      for (int i = 0; i < pieces; ++i) top = fmaxf(top, slot[i * step + DIM]);
      float4v sum{0, 0, 0, 0};
      float weight = 0.0f;
      for (int i = 0; i < pieces; ++i) {
        const float* p = slot + i * step;
        const float f = exp2f(p[DIM] - top);
        weight += p[DIM + 1] * f;
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += p[4 * quad + e] * f;
      }
      typedef _Float16 half4 __attribute__((ext_vector_type(4)));
      half4 h;
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = (_Float16)(weight == 0.0f ? 0.0f : sum[e] / weight);
      *reinterpret_cast<half4*>(a.y + (int64_t)row * a.y_stride + (int64_t)qh * DIM + 4 * quad) = h;
      return;
    }
    before += (int64_t)q.tiles * a.cache.heads * pieces;
  }
}

// Segments of a call whose requests all bring max_rows rows, and the pieces
// that fill the chip: two workgroups a CU of single-tile rows, one of larger.
int64_t most_segments(int requests, int max_rows, int q_heads, int heads, int dim) {
  const int group = q_heads / heads;
  const int rt = tiles_for((int64_t)max_rows * group, dim);
  return (int64_t)requests * heads * (((int64_t)max_rows * group + 16 * rt - 1) / (16 * rt));
}

int64_t wanted_pieces(int rt) { return rt == 1 ? 512 : 256; }

template <int DIM, int RT>
hipError_t launch_tiles(const AttentionArgs& a, const AttnLaunch& l, int64_t grid) {
  constexpr size_t lds = sizeof(float) * kAttnWaves * 16 * RT * (DIM + 4);
  hipError_t e = hipFuncSetAttribute((const void*)attention_kernel<DIM, RT>,
                                     hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  attention_kernel<DIM, RT><<<dim3((uint32_t)grid), dim3(kAttnThreads), lds, (hipStream_t)a.stream>>>(a, l);
  return hipGetLastError();
}

}  // namespace

size_t attention_scratch_bytes(int requests, int max_rows, int q_heads, int heads, int dim, int table_width) {
  if (table_width <= kMinPiecePages) return kKvZeroedBytes;
  const int rt = tiles_for((int64_t)max_rows * (q_heads / heads), dim);
  const int64_t slots = most_segments(requests, max_rows, q_heads, heads, dim) + wanted_pieces(rt);
  return kKvZeroedBytes + (size_t)slots * 16 * rt * (dim + 2) * sizeof(float);
}

hipError_t launch_attention(const AttentionArgs& a) {
  const int dim = a.cache.dim, group = a.q_heads / a.cache.heads;
  const int rt = tiles_for((int64_t)a.max_rows * group, dim);
  AttnLaunch l;
  l.tile_rows = 16 * rt;
  l.want = wanted_pieces(rt);
  const size_t slot_bytes = (size_t)l.tile_rows * (dim + 2) * sizeof(float);
  l.slots = a.scratch_bytes > kKvZeroedBytes ? (int64_t)((a.scratch_bytes - kKvZeroedBytes) / slot_bytes) : 0;
  if (a.table_width <= kMinPiecePages) l.slots = 0;  // nothing is long enough to be cut
  l.partial = (float*)((uint8_t*)a.scratch + kKvZeroedBytes);
  int64_t grid = most_segments(a.requests, a.max_rows, a.q_heads, a.cache.heads, dim);
  if (l.slots > 0) grid += l.want;
  grid = grid < 1 ? 1 : grid > (1 << 20) ? (1 << 20) : grid;
  hipError_t e = hipErrorInvalidValue;
  switch (dim * 8 + rt) {
    case 64 * 8 + 1: e = launch_tiles<64, 1>(a, l, grid); break;
    case 64 * 8 + 2: e = launch_tiles<64, 2>(a, l, grid); break;
    case 64 * 8 + 3: e = launch_tiles<64, 3>(a, l, grid); break;
    case 64 * 8 + 4: e = launch_tiles<64, 4>(a, l, grid); break;
    case 128 * 8 + 1: e = launch_tiles<128, 1>(a, l, grid); break;
    case 128 * 8 + 2: e = launch_tiles<128, 2>(a, l, grid); break;
    case 128 * 8 + 3: e = launch_tiles<128, 3>(a, l, grid); break;
    case 128 * 8 + 4: e = launch_tiles<128, 4>(a, l, grid); break;
    case 256 * 8 + 1: e = launch_tiles<256, 1>(a, l, grid); break;
    case 256 * 8 + 2: e = launch_tiles<256, 2>(a, l, grid); break;
  }
  if (e != hipSuccess || l.slots == 0) return e;
  const int64_t pairs = (int64_t)a.rows * a.q_heads;
  const int per = kAttnThreads / (dim / 4);
  const dim3 join((uint32_t)((pairs + per - 1) / per));
  const hipStream_t st = (hipStream_t)a.stream;
  if (dim == 64) attention_join_kernel<64><<<join, dim3(kAttnThreads), 0, st>>>(a, l);
  else if (dim == 128) attention_join_kernel<128><<<join, dim3(kAttnThreads), 0, st>>>(a, l);
  else attention_join_kernel<256><<<join, dim3(kAttnThreads), 0, st>>>(a, l);
  return hipGetLastError();
}

}  // namespace qpn
