// qpn_kv_round.hip -- what opens a speculative round and feeds the 8-bit paged
// KV cache on gfx950: page tables and slots from the requests' lengths, and
// the query/key norms with the rotation and the cache append.
#include "qpn_common.h"
#include "qpn_kv_internal.h"

namespace qpn {

namespace {

// ---------------------------------------------------------------------------
// Page tables, slots and positions of a round.
//
// One workgroup: a block scan over the requests (pages and rows asked for, which
// decide admission), a second one only when some are not admitted (then those
// of the admitted ones place them), kept in LDS, after which every new table
// entry and every row finds its request by bisection.  The work is a few KiB at
// most, so the launch and the dependent passes (loads, scan, bisection, stores)
// are all there is to pay: 4.6 us for one request, 6.6 us for 256 (from a graph; an
// empty launch takes 2.4), 31 us for 4096 requests.  (A workgroup of 256 or 512 threads
// is no faster for one request and slower for more: on a stream 7.5 and 7.3 us for
// 256, against 7.0.)
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / kLanes;

struct Pair64 {
  int64_t a, b;
};

// The sums up to and including the thread's, and all of them.  Two calls one
// after the other take different buffers `waves`: then one barrier is enough.
__device__ __forceinline__ Pair64 block_inclusive_scan(Pair64 x, Pair64* waves, Pair64& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t a = __shfl_up(x.a, d), b = __shfl_up(x.b, d);
    if (lane >= d) x.a += a, x.b += b;
  }
  if (lane == 63) waves[wave] = x;
  __syncthreads();
  total = {0, 0};
#pragma unroll
  for (int w = 0; w < kPlanWaves; ++w) {
    const Pair64 o = waves[w];
    if (w < wave) x.a += o.a, x.b += o.b;
    total.a += o.a, total.b += o.b;
  }
  return x;
}

// The last index i in [0, n) with start[i] <= x (start ascending, start[0] <= x).
__device__ __forceinline__ int bisect(const int32_t* start, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ __launch_bounds__(kPlanThreads) void plan_round_kernel(PlanRoundArgs a) {
  __shared__ int32_t s_row[kKvMaxRequests + 1];   // first row of each request
  __shared__ int32_t s_take[kKvMaxRequests + 1];  // pages taken before each request
  __shared__ Pair64 s_waves[2][kPlanWaves];
  const int tid = threadIdx.x;
  const int chunks = (a.requests + kPlanThreads - 1) / kPlanThreads;
  int64_t free_count = *a.free_count;
  free_count = free_count < 0 ? 0 : free_count > a.free_capacity ? a.free_capacity : free_count;

  struct Asked {
    bool fine;
    int64_t before, rows, want;
  };
  auto asked_of = [&](int r) {
    Asked q{false, 0, 0, 0};
    if (r < a.requests) {
      q.before = a.before[r];
      q.rows = a.rows[r];
      const int64_t held = a.held[r], need = (q.before + q.rows + kKvPage - 1) / kKvPage;
      q.fine = q.before >= 0 && q.rows >= 0 && held >= 0 && held <= a.table_width &&
               need <= a.table_width && q.before <= held * kKvPage;
      q.want = q.fine && need > held ? need - held : 0;
      if (!q.fine) q.rows = 0;
    }
    return q;
  };

  Pair64 asked_before{0, 0}, placed_before{0, 0};  // totals of the former chunks
  int buffer = 0;
  for (int c = 0; c < chunks; ++c) {
    const int r = c * kPlanThreads + tid;
    const Asked q = asked_of(r);
    Pair64 mine{q.want, q.rows}, total;
    Pair64 at = block_inclusive_scan(mine, s_waves[buffer], total);
    buffer ^= 1;
    const bool go = q.fine && asked_before.a + at.a <= free_count && asked_before.b + at.b <= a.capacity;
    asked_before.a += total.a, asked_before.b += total.b;
    if (asked_before.a > free_count || asked_before.b > a.capacity) {  // some are not admitted
      if (!go) mine = {0, 0};
      at = block_inclusive_scan(mine, s_waves[buffer], total);
      buffer ^= 1;
    }
    at.a += placed_before.a, at.b += placed_before.b;
    placed_before.a += total.a, placed_before.b += total.b;
    if (r < a.requests) {
      s_row[r] = (int32_t)(at.b - mine.b);
      s_take[r] = (int32_t)(at.a - mine.a);
      a.row_start[r] = (int32_t)(at.b - mine.b);
      a.seq_lens[r] = q.fine ? (int32_t)(q.before + mine.b) : 0;
    }
  }
  const int32_t pages = (int32_t)placed_before.a, rows = (int32_t)placed_before.b;
  if (tid == 0) {
    s_row[a.requests] = rows;
    s_take[a.requests] = pages;
    a.row_start[a.requests] = rows;
  }
  __syncthreads();

  // the entry `index` of request r's table row, new pages from the free list
  auto page_of = [&](int r, int64_t held, int64_t index) {
    return index < held ? a.table[r * a.table_stride + index]
                        : a.free_pages[free_count - 1 - (s_take[r] + (index - held))];
  };
  for (int k = tid; k < pages; k += kPlanThreads) {
    const int r = bisect(s_take, a.requests, k);
    a.table[r * a.table_stride + a.held[r] + (k - s_take[r])] = a.free_pages[free_count - 1 - k];
  }
  for (int t = tid; t < a.capacity; t += kPlanThreads) {
    int32_t slot = -1, position = 0;
    if (t < rows) {
      const int r = bisect(s_row, a.requests, t);
      position = a.before[r] + (t - s_row[r]);
      const int32_t page = page_of(r, a.held[r], position / kKvPage);
      if (page >= 0 && page <= kKvMaxPages) slot = page * kKvPage + position % kKvPage;
    }
    a.slots[t] = slot;
    a.positions[t] = position;
  }
  __syncthreads();  // held has been read (held_out may be held)
  for (int r = tid; r < a.requests; r += kPlanThreads)
    a.held_out[r] = a.held[r] + (s_take[r + 1] - s_take[r]);
  if (tid == 0) *a.free_count_out = (int32_t)(free_count - pages);
}

// ---------------------------------------------------------------------------
// Norms, rotation and cache append.
//
// A head of DIM dimensions lies over LPH = DIM / 8 neighbouring lanes, eight
// elements (one 16-byte load) each, so the norm is a sum over LPH lanes and
// the partner of a half-split rotation sits rot / 16 lanes away.
//
// The grid has two kinds of workgroups.  Query workgroups: a wavefront takes
// one row and steps through its heads, HPW = 64 / LPH at a time, with the
// row's cosines and sines in registers.  Cache workgroups: a few rows (one in
// small calls) and one KV head; a workgroup does the pages that one of its rows
// is the first of in the call, and gathers the other rows of such a page.  A
// page's scale is then one workgroup's business, whatever order the slots come
// in: no atomics, no second launch.  Small calls are bound by the chain of
// dependent loads, so what a page most likely needs (the rows that follow its
// first one, the old codes) is fetched before it is known to be needed.
//
// Bound: one row and 8 rows 8.3 us (40 + 2 x 8 heads of 128; 6.7 from a graph, 3.0
// of them with nothing to append): slots, rows, 64-bit angles, norms and codes one
// after another.  4 x 256 rows of prompt blocks: 19.5 us (27 MB, 1.4 TB/s; 8.5
// with nothing to append): 160 workgroups, of a page and KV head each, on 256 CUs,
// with up to four such steps one after another; every one of them, and every
// wavefront of queries, finds the angles of its rows by itself.
// ---------------------------------------------------------------------------
constexpr int kValuePitch = kKvPage + 4;

// pos * f / (2 pi) less its nearest whole number, in turns.  The product of a
// 31-bit position and a 24-bit frequency is rounded once; 1 / (2 pi) is taken
// in two parts, so the angle's error stays near 1e-16 turns times the product.
__device__ __forceinline__ double turns_of(double position, float freq) {
  constexpr double kInv2Pi = 0.15915494309189535;        // 1 / (2 pi), nearest double
  constexpr double kInv2PiLow = -9.8393383378404447e-18;  // and what is left of it
  const double angle = position * (double)freq;
  const double t = angle * kInv2Pi;
  const double low = fma(angle, kInv2Pi, -t) + angle * kInv2PiLow;
  return (t - rint(t)) + low;
}

// cos and sin of 2 pi t for |t| <= 1/2 (and a little over): quarter turns are
// split off, the rest (at most an eighth of a turn) goes through the Taylor
// series, whose first left-out terms are below 3e-14 there.
__device__ __forceinline__ void cos_sin_turns(double t, double* c, double* s) {
  const double q = rint(4.0 * t);
  const double x = (t - 0.25 * q) * 6.283185307179586;
  const double y = x * x;
  double si = fma(y, 1.0 / 6227020800.0, -1.0 / 39916800.0);
  si = fma(y, si, 1.0 / 362880.0);
  si = fma(y, si, -1.0 / 5040.0);
  si = fma(y, si, 1.0 / 120.0);
  si = fma(y, si, -1.0 / 6.0);
  si = fma(x * y, si, x);
  double co = fma(y, -1.0 / 87178291200.0, 1.0 / 479001600.0);
  co = fma(y, co, -1.0 / 3628800.0);
  co = fma(y, co, 1.0 / 40320.0);
  co = fma(y, co, -1.0 / 720.0);
  co = fma(y, co, 1.0 / 24.0);
  co = fma(y, co, -0.5);
  co = fma(y, co, 1.0);
  const int k = (int)q & 3;
  const double cc = (k & 1) ? si : co, ss = (k & 1) ? co : si;
  *c = (k == 1 || k == 2) ? -cc : cc;
  *s = (k >= 2) ? -ss : ss;
}

// x / scale as an E4M3 code: nearest, ties to even, saturating, NaN to NaN.
// One rounding, from 64 bits: the code is the whole number of steps of the
// value's binade (2^(e-3), e >= -6) plus the binade's first code.
__device__ __forceinline__ uint32_t e4m3_code(double x) {
  const uint64_t bits = (uint64_t)__double_as_longlong(x);
  const uint32_t sign = (uint32_t)(bits >> 63) << 7;
  if (x != x) return sign | 0x7Fu;
  const double a = fmin(fabs(x), 448.0);
  int e = (int)(((uint64_t)__double_as_longlong(a) >> 52)) - 1023;
  e = e < -6 ? -6 : e;
  const double inv_step = __longlong_as_double((long long)(uint64_t)(1023 + 3 - e) << 52);
  return sign | (uint32_t)((e + 7) * 8 + (int)rint(a * inv_step) - 8);
}

// A page's scale, as new codes are divided by it.  By a power of two that is a
// product with its inverse; another one (a caller's, kept by a page) is divided
// by, since a product with a rounded inverse misses values halfway between codes.
struct PageScale {
  double value, inverse;
  bool power_of_two;
  __device__ __forceinline__ explicit PageScale(double s)
      : value(s), inverse(1.0 / s), power_of_two(((uint64_t)__double_as_longlong(s) & 0xFFFFFFFFFFFFFull) == 0) {}
};

// Eight values as E4M3 codes (byte e: element e).  The gfx950
// conversion rounds FP32 correctly; what FP32 holds exactly goes through it.
__device__ __forceinline__ float clamp448(float x) {  // (a NaN stays)
  return x > 448.0f ? 448.0f : x < -448.0f ? -448.0f : x;
}
__device__ __forceinline__ uint2 pack_codes(const float f[8]) {
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(f[0]), clamp448(f[1]), 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(f[2]), clamp448(f[3]), lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(f[4]), clamp448(f[5]), 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(f[6]), clamp448(f[7]), hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}
// FP16 values: a product with a power of two (that FP32 holds with its inverse)
// is exact, another scale goes through 64 bits.
__device__ __forceinline__ uint2 value_codes(const half8& x, const PageScale& s) {
  if (s.power_of_two && s.value <= 0x1p60) {  // (no scale is below 2^-60)
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (float)x[e] * (float)s.inverse;
    return pack_codes(f);
  }
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e >> 2] |= e4m3_code((double)x[e] / s.value) << (8 * (e & 3));
  return make_uint2(w[0], w[1]);
}
// Keys: their FP32 rounding goes the same way unless it lies on a border
// between two codes (or among the subnormal ones, whose borders lie closer).
__device__ __forceinline__ uint2 key_codes(const double x[8], const PageScale& s) {
  double q[8];
  float f[8];
  bool near = false;
  if (s.power_of_two) {  // (one branch for all of them)
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = x[e] * s.inverse;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = x[e] / s.value;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    f[e] = (float)q[e];
    near |= (__builtin_bit_cast(uint32_t, f[e]) & 0xFFFFFu) == 0x80000u || fabsf(f[e]) < 0x1p-6f;
  }
  uint2 w = pack_codes(f);
  if (near) {
    w = make_uint2(0, 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t c = e4m3_code(q[e]) << (8 * (e & 3));
      if (e < 4) w.x |= c; else w.y |= c;
    }
  }
  return w;
}

__device__ __forceinline__ double e4m3_value(uint32_t code) {
  const uint32_t m = code & 7, e = (code >> 3) & 15;
  if ((code & 0x7F) == 0x7F) return __longlong_as_double(0x7FF8000000000000ll);
  const double v = e ? ldexp(8.0 + m, (int)e - 10) : ldexp((double)m, -9);
  return code & 0x80 ? -v : v;
}

// The smallest power of two s with amax <= 448 s, at least 2^-60.
__device__ __forceinline__ double page_scale_for(double amax) {
  if (!(amax > 0.0)) return 0x1p-60;
  const uint64_t bits = (uint64_t)__double_as_longlong(amax);
  const int e = (int)(bits >> 52) - 1023;
  const int up = (bits & 0xFFFFFFFFFFFFFull) > 0xC000000000000ull;  // mantissa above 1.75 = 448 / 256
  const int es = e - 8 + up;
  return es <= -60 ? 0x1p-60 : __longlong_as_double((long long)(uint64_t)(1023 + es) << 52);
}

__device__ __forceinline__ half8 load_half8(const uint16_t* p) {
  return *reinterpret_cast<const half8*>(p);
}

// x of another lane by a data-parallel move: within four lanes (quad_perm 1 0 3 2
// and 2 3 0 1), mirrored within eight, within sixteen.
template <int CTRL>
__device__ __forceinline__ float moved(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ double moved(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)b, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(b >> 32), CTRL, 0xF, 0xF, false);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
// Over LANES (8 to 64) neighbouring lanes, in every one of them.
template <int LANES, typename T>
__device__ __forceinline__ T lanes_sum(T x) {
  x += moved<0xB1>(x);
  x += moved<0x4E>(x);
  x += moved<0x141>(x);
  if constexpr (LANES >= 16) x += moved<0x140>(x);
  if constexpr (LANES >= 32) x += __shfl_xor(x, 16);
  return x;
}
__device__ __forceinline__ double wave_max(double x) {
  x = fmax(x, moved<0xB1>(x));
  x = fmax(x, moved<0x4E>(x));
  x = fmax(x, moved<0x141>(x));
  x = fmax(x, moved<0x140>(x));
  x = fmax(x, __shfl_xor(x, 16));
  return fmax(x, __shfl_xor(x, 32));
}

// T: float for queries, double for keys.  The norm and rotation of eight
// elements of a head; `lane_at` is the lane's place among the head's LPH.
// cs: cosines and sines of the lane's own angles.
// What a lane needs of the weights and frequencies, for all rows.
template <int DIM>
struct Lane {
  half8 weight;
  float freq[8];  // of its own angles (interleaved: entries 0 .. 3)
  bool turned;    // its elements are rotated
  __device__ __forceinline__ void load(const RopeAppendArgs& a, int lane_at, const uint16_t* w) {
    const int d0 = lane_at * 8, half = a.rot / 2;
    weight = half8{};
    if (w) weight = load_half8(w + d0);
    turned = d0 < a.rot;
    const int n = a.interleaved ? 4 : 8;
    const int j0 = a.interleaved ? d0 / 2 : d0 < half ? d0 : d0 - half;
#pragma unroll
    for (int i = 0; i < 8; ++i) freq[i] = turned && i < n ? a.inv_freq[j0 + i] : 0.0f;
  }
};

template <typename T, int DIM>
struct Rotor {
  T c[8], s[8];  // half-split: one per element; interleaved: entries 0 .. 3

  __device__ __forceinline__ void angles(const RopeAppendArgs& a, const Lane<DIM>& f, int lane_at, double position) {
    if (!f.turned) return;
    if constexpr (sizeof(T) == 8) {
      if (!a.interleaved) {
        // the lanes of a pair turn by the same eight angles: each finds four
        // (64-bit arithmetic is what a page's keys cost) and takes the others
        const int step = a.rot / 16, lane = threadIdx.x & 63;
        const bool first = lane_at < step;
        const int from = first ? lane + step : lane - step;
        double cc[4], ss[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) cos_sin_turns(turns_of(position, first ? f.freq[i] : f.freq[i + 4]), &cc[i], &ss[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const double oc = __shfl(cc[i], from), os = __shfl(ss[i], from);
          c[i] = first ? cc[i] : oc;
          s[i] = first ? ss[i] : os;
          c[i + 4] = first ? oc : cc[i];
          s[i + 4] = first ? os : ss[i];
        }
        return;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) cos_sin_turns(turns_of(position, f.freq[i]), &c[i], &s[i]);
    } else {
      const int n = a.interleaved ? 4 : 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i < n) {
          const double t = turns_of(position, f.freq[i]);
          // the hardware's functions take turns; their error (below 2^-20) is
          // far under the FP16 step of the result
          c[i] = __builtin_amdgcn_cosf((float)t);
          s[i] = __builtin_amdgcn_sinf((float)t);
        }
      }
    }
  }

  // x: the raw elements; returns the normed and rotated ones
  __device__ __forceinline__ void turn(const RopeAppendArgs& a, const Lane<DIM>& f, int lane_at, const half8& x,
                                       bool normed, T out[8]) const {
    constexpr int LPH = DIM / 8;
    T r = T(1);
    const bool turned = f.turned;
    if (normed) {
      T sum = T(0);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += (T)x[i] * (T)x[i];
      sum = lanes_sum<LPH>(sum);
      if constexpr (sizeof(T) == 8)
        r = 1.0 / sqrt(sum * (1.0 / DIM) + a.eps);
      else
        r = 1.0f / sqrtf(sum * (1.0f / DIM) + (float)a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) out[i] = (T)x[i] * r * (T)f.weight[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) out[i] = (T)x[i];
    }
    if (a.rot == 0) return;
    if (a.interleaved) {
      if (turned) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const T u = out[2 * i], v = out[2 * i + 1];
          out[2 * i] = u * c[i] - v * s[i];
          out[2 * i + 1] = v * c[i] + u * s[i];
        }
      }
    } else {
      // the other half of each pair: rot / 16 lanes up (first half) or down
      const int step = a.rot / 16, lane = threadIdx.x & 63;
      const bool first = lane_at < step;
      const int from = !turned ? lane : first ? lane + step : lane - step;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const T other = __shfl(out[i], from);
        if (turned) out[i] = first ? out[i] * c[i] - other * s[i] : out[i] * c[i] + other * s[i];
      }
    }
  }
};

template <int DIM, int THREADS>
__device__ __forceinline__ void append_queries(const RopeAppendArgs& a, int wg, int waves_per_row,
                                               int steps) {
  constexpr int LPH = DIM / 8, HPW = kLanes / LPH;
  const int lane = threadIdx.x & 63, lane_at = lane % LPH;
  const int64_t wave = (int64_t)wg * (THREADS / kLanes) + (threadIdx.x >> 6);
  const int64_t row = wave / waves_per_row;
  if (row >= a.rows) return;  // a whole wavefront; no barrier follows
  const int h0 = (int)(wave % waves_per_row) * steps * HPW + lane / LPH;
  const uint16_t* const from = a.qkv + row * a.qkv_stride + lane_at * 8;
  uint16_t* const to = a.q_out + row * a.q_stride + lane_at * 8;
  half8 x = {}, next = {};
  if (h0 < a.q_heads) x = load_half8(from + (int64_t)h0 * DIM);
  Lane<DIM> f;
  f.load(a, lane_at, a.q_weight);
  Rotor<float, DIM> rotor;
  if (a.rot) rotor.angles(a, f, lane_at, (double)a.positions[row]);
  for (int i = 0; i < steps; ++i) {
    const int h = h0 + i * HPW;
    if (i + 1 < steps && h + HPW < a.q_heads) next = load_half8(from + (int64_t)(h + HPW) * DIM);
    float out[8];
    rotor.turn(a, f, lane_at, x, a.q_weight != nullptr, out);
    half8 y;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = (_Float16)out[e];
    if (h < a.q_heads) *reinterpret_cast<half8*>(to + (int64_t)h * DIM) = y;
    x = next;
  }
}

// Sixteen old codes at one place, rounded again to a larger scale.
__device__ __forceinline__ u32x4 recode16(u32x4 c, double ratio) {
  u32x4 o;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint32_t r = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) r |= e4m3_code(e4m3_value((c[w] >> (8 * b)) & 255) * ratio) << (8 * b);
    o[w] = r;
  }
  return o;
}

template <int DIM, int THREADS>
__device__ __forceinline__ void append_page(const RopeAppendArgs& a, int row0, int32_t slot0, int head) {
  constexpr int LPH = DIM / 8;
  constexpr int RPS = THREADS / LPH;  // rows a step of the workgroup takes
  constexpr int STEPS = kKvPage / RPS;
  constexpr int UNITS = (DIM * 4 + THREADS - 1) / THREADS;  // 16-byte units of the values' block, of a thread
  __shared__ int32_t s_row[kKvPage];      // the row at each offset of the page, -1: none
  __shared__ int32_t s_list[kKvPage];     // the offsets that are written, in order
  __shared__ int32_t s_earlier, s_count;
  __shared__ uint64_t s_taken;            // bit o: offset o is written
  __shared__ double s_max[2][THREADS / kLanes];
  // new values' codes; dimensions 68 bytes apart, so that the lanes of a row meet different banks
  __shared__ __attribute__((aligned(16))) uint8_t s_v[DIM * kValuePitch];
  const int tid = threadIdx.x, lane = tid & 63, lane_at = tid % LPH;

  const int32_t page = slot0 / kKvPage;
  const int64_t block = (int64_t)page * a.cache.heads + head;
  uint8_t* const kb = a.cache.k + block * (kKvPage * DIM);
  uint8_t* const vb = a.cache.v + block * (kKvPage * DIM);

  // the rows that follow, the scales and the old values: on their way
  const uint16_t* const k_from = a.qkv + (int64_t)(a.q_heads + head) * DIM + lane_at * 8;
  const uint16_t* const v_from = k_from + (int64_t)a.cache.heads * DIM;
  const int near = min(row0 + tid / LPH, a.rows - 1);
  half8 k_near = load_half8(k_from + near * a.qkv_stride), v_near = load_half8(v_from + near * a.qkv_stride);
  int32_t pos_near = a.positions[near];
  Lane<DIM> f;
  f.load(a, lane_at, a.k_weight);
  const float scale_k = a.cache.k_scale[block], scale_v = a.cache.v_scale[block];
  u32x4 old[UNITS];
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    old[i] = u32x4{0, 0, 0, 0};
    if (tid + i * THREADS < DIM * 4) old[i] = *reinterpret_cast<const u32x4*>(vb + (tid + i * THREADS) * 16);
  }

  if (tid < kKvPage) s_row[tid] = -1;
  if (tid == 0) s_earlier = 0;
  __syncthreads();
  for (int t = tid; t < a.rows; t += THREADS) {
    const int32_t s = a.slots[t];
    if (s >= 0 && s / kKvPage == page) {
      if (t < row0) s_earlier = 1;
      atomicMax(&s_row[s % kKvPage], t);
    }
  }
  __syncthreads();
  if (s_earlier) return;  // an earlier row's workgroup has the page
  if (tid < kKvPage) {
    const uint64_t taken = __ballot(s_row[tid] >= 0);
    if (s_row[tid] >= 0) s_list[__popcll(taken & ((1ull << tid) - 1))] = tid;
    if (tid == 0) s_count = __popcll(taken), s_taken = taken;
  }
  __syncthreads();
  const int count = s_count;
  const bool fresh = s_row[0] >= 0;
  const double old_k = fresh ? 0.0 : (double)scale_k, old_v = fresh ? 0.0 : (double)scale_v;

  // the keys, normed and rotated, and the raw values of the thread's rows (the
  // rows i = RPS st + tid / LPH of the list), and their largest
  double key[STEPS][8], kmax = 0.0, vmax = 0.0;
  half8 val[STEPS];
#pragma unroll
  for (int st = 0; st < STEPS; ++st) {
    if (st * RPS < count) {
      const int i = st * RPS + tid / LPH;
      const int t = s_row[s_list[i < count ? i : 0]];
      half8 x = k_near;
      int32_t position = pos_near;
      val[st] = v_near;
      if (st > 0 || t != near) {
        x = load_half8(k_from + t * a.qkv_stride);
        val[st] = load_half8(v_from + t * a.qkv_stride);
        position = a.positions[t];
      }
      Rotor<double, DIM> rotor;
      if (a.rot) rotor.angles(a, f, lane_at, (double)position);
      rotor.turn(a, f, lane_at, x, a.k_weight != nullptr, key[st]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const double k = fabs(key[st][e]), v = fabs((double)val[st][e]);
        if (k < __builtin_inf()) kmax = fmax(kmax, k);
        if (v < __builtin_inf()) vmax = fmax(vmax, v);
      }
    }
  }
  kmax = wave_max(kmax);
  vmax = wave_max(vmax);
  if (lane == 0) s_max[0][tid >> 6] = kmax, s_max[1][tid >> 6] = vmax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < (THREADS / kLanes); ++w) {
    kmax = fmax(kmax, s_max[0][w]);
    vmax = fmax(vmax, s_max[1][w]);
  }
  const double need_k = page_scale_for(kmax), need_v = page_scale_for(vmax);
  const double new_k = old_k > need_k ? old_k : need_k, new_v = old_v > need_v ? old_v : need_v;
  const bool grow_k = old_k > 0.0 && new_k > old_k, grow_v = old_v > 0.0 && new_v > old_v;
  const PageScale by_k(new_k), by_v(new_v);

  // keys: 8 codes per lane, two lanes make a 16-byte unit of the layout
  if (grow_k) {
    const double ratio = old_k / new_k;
    for (int u = tid; u < (DIM / 16) * kKvPage; u += THREADS) {
      if (s_row[u % kKvPage] >= 0) continue;
      u32x4* p = reinterpret_cast<u32x4*>(kb + u * 16);
      *p = recode16(*p, ratio);
    }
  }
#pragma unroll
  for (int st = 0; st < STEPS; ++st) {
    const int i = st * RPS + tid / LPH;
    if (i < count) {
      const int off = s_list[i], place = ((off >> 2) & 3) * 16 + (off >> 4) * 4 + (off & 3);
      const uint2 pair = key_codes(key[st], by_k), values = value_codes(val[st], by_v);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        s_v[(lane_at * 8 + e) * kValuePitch + place] = (uint8_t)((e < 4 ? values.x : values.y) >> (8 * (e & 3)));
      *reinterpret_cast<uint2*>(kb + (lane_at >> 1) * (kKvPage * 16) + off * 16 + (lane_at & 1) * 8) = pair;
    }
  }
  __syncthreads();

  // values: 16-byte segments (dimension d, group g) of the tokens 16 t + 4 g + r
  const double ratio_v = grow_v ? old_v / new_v : 1.0;
  const uint64_t taken = s_taken;
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    const int u = tid + i * THREADS, g = u & 3;
    if (u >= DIM * 4) break;
    // bit 4 t + r: token 16 t + 4 g + r is new
    const uint64_t mine = taken >> (4 * g);
    const uint32_t fresh_bytes = (uint32_t)(mine & 15) | (uint32_t)(mine >> 12 & 0xF0) | (uint32_t)(mine >> 24 & 0xF00) |
                                 (uint32_t)(mine >> 36 & 0xF000);
    if (!fresh_bytes && !grow_v) continue;
    u32x4 c;
#pragma unroll
    for (int t = 0; t < 4; ++t) c[t] = *reinterpret_cast<const uint32_t*>(s_v + (u >> 2) * kValuePitch + g * 16 + t * 4);
    if (fresh_bytes != 0xFFFFu) {
      u32x4 o = old[i];
      if (grow_v) o = recode16(o, ratio_v);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t bits = (fresh_bytes >> (4 * t)) & 15;
        const uint32_t mask = (bits & 1 ? 0xFFu : 0) | (bits & 2 ? 0xFF00u : 0) |
                              (bits & 4 ? 0xFF0000u : 0) | (bits & 8 ? 0xFF000000u : 0);
        c[t] = (c[t] & mask) | (o[t] & ~mask);
      }
    }
    *reinterpret_cast<u32x4*>(vb + u * 16) = c;
  }
  if (tid == 0) {
    a.cache.k_scale[block] = (float)new_k;
    a.cache.v_scale[block] = (float)new_v;
  }
}

// The pages that rows row0 .. row0 + rows - 1 (at most 64) begin runs of (rows that
// follow one another on one page).
template <int DIM, int THREADS>
__device__ __forceinline__ void append_rows(const RopeAppendArgs& a, int row0, int rows, int head) {
  const int64_t places = a.cache.pages * kKvPage;
  const int lane = threadIdx.x & 63, t = row0 + lane;
  int32_t slot = -1, before = -1;
  if (lane < rows && t < a.rows) {
    slot = a.slots[t];
    if (t > 0) before = a.slots[t - 1];
  }
  const bool starts = slot >= 0 && slot < places && !(before >= 0 && before / kKvPage == slot / kKvPage);
  for (uint64_t left = __ballot(starts); left; left &= left - 1) {  // (every wavefront finds the same)
    const int i = __ffsll((unsigned long long)left) - 1;
    append_page<DIM, THREADS>(a, row0 + i, __builtin_amdgcn_readlane(slot, i), head);
    if (rows > 1) __syncthreads();  // its LDS has been read
  }
}

// Cache workgroup w: KV head w % heads of a block of rows_per_wg rows.  Pages of
// long runs begin in every kKvPage / rows_per_wg'th block; `groups` blocks so far
// apart come one after the other, so that those which have work do not all fall
// to the same few CUs.
template <int DIM, int THREADS>
__global__ __launch_bounds__(THREADS) void rope_append_kernel(RopeAppendArgs a, int cache_wgs, int rows_per_wg,
                                                              int groups, int waves_per_row, int steps) {
  if ((int)blockIdx.x < cache_wgs) {
    const int at = (int)blockIdx.x / a.cache.heads, apart = kKvPage / rows_per_wg;
    const int block = rows_per_wg == 1 ? at : at % groups * apart + at / groups;
    append_rows<DIM, THREADS>(a, block * rows_per_wg, rows_per_wg, (int)blockIdx.x % a.cache.heads);
  } else {
    append_queries<DIM, THREADS>(a, (int)blockIdx.x - cache_wgs, waves_per_row, steps);
  }
}

template <int DIM, int THREADS>
hipError_t launch_append(const RopeAppendArgs& a, int rows_per_wg) {
  constexpr int HPW = kLanes / (DIM / 8), WAVES = THREADS / kLanes;
  // heads per wavefront: one step of HPW while that leaves fewer wavefronts
  // than 8 a CU, else more, so that a row's angles serve more heads (1024 rows of
  // one request: 18.3 us with one step each, 15.7 us so; 257 x 8 rows 58.5 and 49.9)
  const int head_groups = (a.q_heads + HPW - 1) / HPW;
  int64_t steps = (int64_t)a.rows * head_groups / 2048;
  steps = steps < 1 ? 1 : steps > head_groups ? head_groups : steps;
  const int waves_per_row = (int)((head_groups + steps - 1) / steps);
  const int groups = rows_per_wg == 1 ? a.rows : (a.rows + kKvPage - 1) / kKvPage;
  const int64_t cache_wgs = (int64_t)groups * (rows_per_wg == 1 ? 1 : kKvPage / rows_per_wg) * a.cache.heads;
  const int64_t query_wgs = ((int64_t)a.rows * waves_per_row + WAVES - 1) / WAVES;
  rope_append_kernel<DIM, THREADS><<<dim3((uint32_t)(cache_wgs + query_wgs)), dim3(THREADS), 0, (hipStream_t)a.stream>>>(
      a, (int)cache_wgs, rows_per_wg, groups, waves_per_row, (int)steps);
  return hipGetLastError();
}

// Rows of a cache workgroup: one while those of all rows are about what the chip
// holds at once, since each row may have a page of its own (64 requests of one row
// and 8 heads: 10 us; with 16 rows a workgroup 77).  Above that eight: rows of a
// prompt follow others on their pages, and most workgroups of one row would only
// look and leave.  With one, four, eight and 16: 1024 rows of one request 31.6,
// 17.8, 15.7 and 15.6 us; 257 requests of 8 rows 134, 53, 50 and 48; but 300
// requests of one row 36, 43, 51 and 79, and 1000 of them 110, 104, 102 and 102.
// The host does not know how the rows lie on the pages, so the rule serves the
// prompts, and batches of a few hundred single rows pay for it.  Pages of 256
// dimensions take eight wavefronts then (2 x 512 rows of 16 + 2 x 8 heads: 29.6 us
// with four, 21.9 with eight), the others four (1024 rows of 128 dimensions: 15.7
// and 17.8).
template <int DIM>
hipError_t launch_append(const RopeAppendArgs& a) {
  if ((int64_t)a.rows * a.cache.heads <= 2048) return launch_append<DIM, 256>(a, 1);
  return launch_append<DIM, DIM == 256 ? 512 : 256>(a, 8);
}

}  // namespace

hipError_t launch_plan_round(const PlanRoundArgs& a) {
  plan_round_kernel<<<dim3(1), dim3(kPlanThreads), 0, (hipStream_t)a.stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_rope_append(const RopeAppendArgs& a) {
  return a.cache.dim == 64 ? launch_append<64>(a) : a.cache.dim == 128 ? launch_append<128>(a) : launch_append<256>(a);
}

}  // namespace qpn
