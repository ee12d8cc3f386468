// qpn_kv_verify.hip -- verification of drafted tokens against the target's
// probabilities from given random numbers, on gfx950.
//
// With p and q the target's and the drafter's softmax of a row, the draft d is
// accepted when u q(d) < p(d); at the first refusal the next token is drawn
// from max(p - q, 0) by its inverse CDF, after the last draft from p.  Which
// token that is hangs on sums over up to n probabilities compared with a
// random number: a relative error e of the sums moves the answer with
// probability ~ n e, so exponentials and sums are held in 64 bits.
//
// The first kernel reads every logit once and leaves, per row and chunk of
// kVerifyChunk tokens, the chunk's maximum and its sum of exponentials against
// that maximum.  The workgroup of a request that finishes last joins the chunks'
// sums to the rows' normalisers and finds the row where the request stops.  For a
// greedy drafter that is all there is to read but one chunk: what is left of the
// target is p without the draft, whose masses are the chunks' sums, so the same
// workgroup finds the chunk in which the random number falls, and the token in
// it.  For a sampled drafter a second kernel (a workgroup per request and chunk)
// sums max(p - q, 0) of the stopping row, and the last workgroup of the request
// finds the token.  Sums run in an order fixed by the sizes, so results are
// deterministic.
//
// Bound: the 64-bit arithmetic of the exponentials (some 20 operations each) next
// to reading the logits: 32 requests of 8 rows of 151936 tokens, target and
// drafter (156 MB, 78 million exponentials), take 88 to 100 us not in any cache, 70
// of them in the first kernel; at a large copy's rate the bytes alone would take
// 32.  The second one's 22 us are a launch, 32 rows of 38 chunks (19 MB), one a
// workgroup, and their arrivals.  8 rows of a greedy drafter take 16 us: launch, one
// chunk a workgroup, 304 arrivals on one counter, the joins of the last one and its
// search, each waiting for the one before.
//
// What workgroups leave for one another is written through to the device's
// point of coherence, and lies in 128-byte lines of one request alone: a line
// that an XCD's L2 holds is never written again by others before it is read.
#include "qpn_common.h"
#include "qpn_kv_internal.h"

namespace qpn {

namespace {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWaves = kVerifyThreads / kLanes;
constexpr int kVerifyUnits = 2;                            // 8-token units of a thread
constexpr int kVerifyChunk = kVerifyThreads * kVerifyUnits * 8;
constexpr int kArrivalStep = 4;                            // 32-bit words between requests' counters
static_assert((size_t)kKvMaxRequests * kArrivalStep * 4 <= kKvZeroedBytes, "a counter per request");
constexpr int kVerifySpan = 64;       // chunks of a workgroup of the first kernel, at most
constexpr int kVerifyRowsHeld = 16;   // rows of a request whose chunks' masses are held in LDS
// Workgroups of the first kernel aimed at: the six a CU that its registers let
// reside.  (32 x 8 sampled rows of 151936: 97 us with 768, 93 with 1536, 98 with 4096.)
constexpr int kVerifyWgs = 1536;

// Chunks of a row: rows may start anywhere in a 16-byte granule, so a row's
// tokens are counted from the granule's start (up to 7 places before it).
__host__ __device__ constexpr int64_t verify_chunks(int64_t n) { return (n + 7 + kVerifyChunk - 1) / kVerifyChunk; }

constexpr int64_t kMaxVerifyChunks = verify_chunks(kMaxN);

struct ChunkSum {
  double sum;  // of exp(inv_temperature (x - max)); NaN when there is a NaN or +inf
  double max;  // -inf when there is nothing above it
};

// Where the request stops, from the first kernel to the second.
struct alignas(128) Stop {
  double top_p, scale_p, top_q, scale_q;  // maximum and 1 / sum of the row's target and drafter
  int row;
  int drafter;                            // 1: the weights are max(p - q, 0), 0: p
  int valid;                              // 0: the target's row has no distribution
};

struct VerifyLaunch {
  int splits;              // workgroups of a row: split i has chunks i, i + splits, ...
  int64_t chunks, stride;  // of a row: its sums, and in ChunkSums from row to row (whole lines)
  ChunkSum* sums;          // [2 or 1][rows][stride]: target, drafter
  Stop* stops;             // [requests]
  double* masses;          // [requests][mass_stride]
  int64_t mass_stride;
  double scale;            // inv_temperature log2 e, in [1e-30, 1e290]
  double lowest;           // -1000 / scale
};

// 2^(d scale) for d <= 0, as 2^k times 2^r, |r| <= 1/2, by the polynomial of
// degree 8 through the Chebyshev nodes of that interval (1.1e-12 off at most).
// d below `lowest` (2^-1000) counts as that: no sum of larger ones can tell.
__device__ __forceinline__ double exp2_scaled(double d, const VerifyLaunch& l) {
  constexpr double kRound = 6755399441055744.0;  // 1.5 2^52: the sum's low bits are the whole number
  d = fmax(d, l.lowest);
  const double t = fma(d, l.scale, kRound);
  const double r = fma(d, l.scale, kRound - t);
  double p = fma(r, 1.3255224878668817e-06, 1.5310079402249296e-05);
  p = fma(p, r, 0.00015403455852453838);
  p = fma(p, r, 0.0013333450568000645);
  p = fma(p, r, 0.009618129159402558);
  p = fma(p, r, 0.05550410941205933);
  p = fma(p, r, 0.2402265069581299);
  p = fma(p, r, 0.6931471805459335);
  p = fma(p, r, 1.0);
  return ldexp(p, (int)(uint32_t)(uint64_t)__double_as_longlong(t));
}

// The same, 0 from the lowest on.
__device__ __forceinline__ double weight_of(double d, const VerifyLaunch& l) {
  return d > l.lowest ? exp2_scaled(d, l) : 0.0;
}

// x of another lane by a data-parallel move (CTRL: row_shr 1, 2, 4, 8 within 16
// lanes, then the last lane of a row, of two rows, to the next), `none` where
// there is none.
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double x, double none) {
  const uint64_t b = (uint64_t)__double_as_longlong(x), o = (uint64_t)__double_as_longlong(none);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp((int)o, (int)b, CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp((int)(o >> 32), (int)(b >> 32), CTRL, ROWS, 0xF, false);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ double lane_of(double x, int lane) {
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)b, lane), hi = (uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), lane);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
// The sum of x over the lanes up to and including this one.
__device__ __forceinline__ double wave_scan(double x) {
  x += moved<0x111, 0xF>(x, 0.0);
  x += moved<0x112, 0xF>(x, 0.0);
  x += moved<0x114, 0xF>(x, 0.0);
  x += moved<0x118, 0xF>(x, 0.0);
  x += moved<0x142, 0xA>(x, 0.0);
  x += moved<0x143, 0xC>(x, 0.0);
  return x;
}
__device__ __forceinline__ double wave_sum(double x) { return lane_of(wave_scan(x), 63); }
__device__ __forceinline__ double wave_max(double x) {
  constexpr double kNone = -__builtin_inf();
  x = fmax(x, moved<0x111, 0xF>(x, kNone));
  x = fmax(x, moved<0x112, 0xF>(x, kNone));
  x = fmax(x, moved<0x114, 0xF>(x, kNone));
  x = fmax(x, moved<0x118, 0xF>(x, kNone));
  x = fmax(x, moved<0x142, 0xA>(x, kNone));
  x = fmax(x, moved<0x143, 0xC>(x, kNone));
  return lane_of(x, 63);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float moved(float x, float none) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none), __builtin_bit_cast(int, x), CTRL,
                                                               ROWS, 0xF, false));
}
__device__ __forceinline__ float wave_max(float x) {
  constexpr float kNone = -__builtin_inff();
  x = fmaxf(x, moved<0x111, 0xF>(x, kNone));
  x = fmaxf(x, moved<0x112, 0xF>(x, kNone));
  x = fmaxf(x, moved<0x114, 0xF>(x, kNone));
  x = fmaxf(x, moved<0x118, 0xF>(x, kNone));
  x = fmaxf(x, moved<0x142, 0xA>(x, kNone));
  x = fmaxf(x, moved<0x143, 0xC>(x, kNone));
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}

// Eight tokens of a row from place 8 u - shift on; those outside [0, n) are
// -inf.  `base` is the row, `shift` its offset in its 16-byte granule in elements.
__device__ __forceinline__ half8 load_unit(const uint16_t* base, int shift, int64_t n, int64_t u) {
  const int64_t first = u * 8 - shift;
  if (first >= 0 && first + 8 <= n) return *reinterpret_cast<const half8*>(base + first);
  half8 x;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint16_t bits = 0xFC00u;
    if (first + i >= 0 && first + i < n) bits = base[first + i];
    x[i] = __builtin_bit_cast(_Float16, bits);
  }
  return x;
}

__device__ __forceinline__ int shift_of(const uint16_t* row) { return (int)(((uintptr_t)row & 15) >> 1); }

// A double at the device's point of coherence.
__device__ __forceinline__ void put_shared(double* p, double x) {
  __hip_atomic_store(p, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ double get_shared(const double* p) {
  return __hip_atomic_load(const_cast<double*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// True (in the whole workgroup) for the last of n workgroups that count
// themselves in; what they put before is then there.
__device__ __forceinline__ bool arrive_last(uint32_t* counter, uint32_t n, uint32_t* s_arrival) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wavefront's puts are there
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint32_t before = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (before == n - 1) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *s_arrival = before;
  }
  __syncthreads();
  const bool last = *s_arrival == n - 1;
  __syncthreads();  // s_arrival has been read
  if (last) __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  return last;
}

// max and sum of a whole row from its chunks, by one wavefront: valid when the
// maximum is finite and the sum is a number.  mass: the first 64 chunks' sums
// against the row's maximum, one a lane.
struct RowSum {
  double max, sum;
  bool valid;
};
// the first 64 chunks' entries of a row, one a lane (on their way)
struct RowLoad {
  double max, sum;
  __device__ __forceinline__ void load(const ChunkSum* c, const VerifyLaunch& l) {
    const int lane = threadIdx.x & 63;
    const bool in = lane < l.chunks;
    max = in ? get_shared(&c[lane].max) : -__builtin_inf();
    sum = in ? get_shared(&c[lane].sum) : 0.0;
  }
};
__device__ __forceinline__ RowSum join_row(const ChunkSum* c, const RowLoad& first, const VerifyLaunch& l, double* mass) {
  const int lane = threadIdx.x & 63;
  double m = first.max;
  for (int64_t k = 64 + lane; k < l.chunks; k += 64) m = fmax(m, get_shared(&c[k].max));
  m = wave_max(m);
  const bool finite = m > -__builtin_inf() && m < __builtin_inf();
  // (a chunk without any number but NaN has max -inf and a NaN sum)
  auto part = [&](double x, double v) { return v != v ? v : finite ? v * weight_of(x - m, l) : 0.0; };
  double s = part(first.max, first.sum);
  *mass = s;
  for (int64_t k = 64 + lane; k < l.chunks; k += 64) s += part(get_shared(&c[k].max), get_shared(&c[k].sum));
  s = wave_sum(s);
  return {m, s, finite && s == s};
}

// The weight of each token of a request's stopping row.
struct Weigher {
  const uint16_t *p, *q;         // q NULL: the draft alone (or none)
  int shift_p, shift_q;
  double top_p, scale_p, top_q, scale_q;
  int64_t skip;                  // a greedy draft: its weight is 0
  int64_t n;
  // the weights of the 8 tokens of unit u (0 outside the row)
  __device__ __forceinline__ void unit(const VerifyLaunch& l, int64_t u, double w[8]) const {
    const half8 x = load_unit(p, shift_p, n, u);
    const int64_t first = u * 8 - shift_p;
    half8 z;
    if (q) {
      if (shift_q == shift_p) {
        z = load_unit(q, shift_q, n, u);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint16_t bits = 0xFC00u;
          if (first + i >= 0 && first + i < n) bits = q[first + i];
          z[i] = __builtin_bit_cast(_Float16, bits);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      double v = weight_of((double)x[i] - top_p, l) * scale_p;
      if (q) v = fmax(v - weight_of((double)z[i] - top_q, l) * scale_q, 0.0);
      w[i] = first + i == skip ? 0.0 : v;
    }
  }
};

// A chunk's tokens in order: thread t has the units kVerifyUnits t + k.
__device__ __forceinline__ int64_t unit_of(int64_t chunk, int k) {
  return chunk * (kVerifyChunk / 8) + (int64_t)threadIdx.x * kVerifyUnits + k;
}

// LDS of the search for a token.
struct TokenLds {
  double wave[2][kVerifyWaves];
  int first[kVerifyWaves], last[kVerifyWaves];
  int chunk, chunk_last;
  double before;
};

// The mass of a chunk of the weights, in every thread.
__device__ __forceinline__ double chunk_mass(const Weigher& w, const VerifyLaunch& l, int64_t chunk, TokenLds& s) {
  double mass = 0.0;
#pragma unroll
  for (int k = 0; k < kVerifyUnits; ++k) {
    double v[8];
    w.unit(l, unit_of(chunk, k), v);
#pragma unroll
    for (int i = 0; i < 8; ++i) mass += v[i];
  }
  mass = wave_sum(mass);
  __syncthreads();  // what `wave` held has been read
  if ((threadIdx.x & 63) == 0) s.wave[0][threadIdx.x >> 6] = mass;
  __syncthreads();
  mass = 0.0;
#pragma unroll
  for (int k = 0; k < kVerifyWaves; ++k) mass += s.wave[0][k];
  return mass;
}

// Takes the skipped token out of its chunk's mass: by its weight where a good
// part is left (the rounding of the mass is then below 1e-10 of that), else
// the chunk is summed again without it.  The whole workgroup comes here.
__device__ __forceinline__ void skip_token(const Weigher& w, const VerifyLaunch& l, double* mass, TokenLds& s) {
  if (w.skip < 0) return;
  const int64_t c = (w.skip + w.shift_p) / kVerifyChunk;
  const double x = weight_of((double)__builtin_bit_cast(_Float16, w.p[w.skip]) - w.top_p, l) * w.scale_p;
  __syncthreads();  // the masses are there
  const double all = mass[c];
  double left = all - x;
  if (left * 16.0 < all) left = chunk_mass(w, l, c, s);
  __syncthreads();  // and have been read
  if (threadIdx.x == 0) mass[c] = left;
}

// The masses of p alone (less the skipped token) from the chunks' sums of the row.
__device__ __forceinline__ void masses_of_row(const Weigher& w, const VerifyLaunch& l, const ChunkSum* sums,
                                              double* mass, TokenLds& s) {
  for (int64_t c = threadIdx.x; c < l.chunks; c += kVerifyThreads)
    mass[c] = get_shared(&sums[c].sum) * weight_of(get_shared(&sums[c].max) - w.top_p, l) * w.scale_p;
  skip_token(w, l, mass, s);
}

// The token in which u falls, from the masses of the chunks (in LDS).
__device__ __forceinline__ int pick_token(Weigher w, const VerifyLaunch& l, const ChunkSum* sums, float u, double* mass,
                                          TokenLds& s) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  __syncthreads();  // the masses are there
  double total = 0.0, target = 0.0;
  for (int attempt = 0;; ++attempt) {
    // by the first wavefront: 64 chunks at a time, their sum first, then the
    // first chunk that the target falls in and the last that has any mass
    if (wave == 0) {
      double sum = 0.0;
      for (int64_t c = lane; c < l.chunks; c += 64) sum += mass[c];
      total = wave_sum(sum);
      target = (double)u * total;
      double before = 0.0, at = 0.0;
      int chunk = -1, last = -1;
      for (int64_t base = 0; base < l.chunks && chunk < 0; base += 64) {
        const double x = base + lane < l.chunks ? mass[base + lane] : 0.0;
        const double up = before + wave_scan(x);
        const uint64_t some = __ballot(x > 0.0), past = __ballot(x > 0.0 && up > target);
        if (some) last = (int)base + 63 - __builtin_clzll(some);
        const int pick = past ? __ffsll((unsigned long long)past) - 1 : some ? 63 - __builtin_clzll(some) : 0;
        // (not up - x: the sum of what comes before)
        if (past) chunk = (int)base + pick;
        if (some) at = pick ? lane_of(up, pick - 1) : before;
        before = lane_of(up, 63);
      }
      if (lane == 0) s.chunk = chunk >= 0 ? chunk : last, s.before = at, s.wave[1][0] = total, s.wave[1][1] = target;
    }
    __syncthreads();
    total = s.wave[1][0], target = s.wave[1][1];
    if (total > 0.0 || attempt == 1) break;
    w.q = nullptr;  // nowhere above the drafter: the target itself
    w.skip = -1;
    __syncthreads();
    masses_of_row(w, l, sums, mass, s);
    __syncthreads();
  }
  const int64_t pick = s.chunk;
  if (pick < 0) return -1;
  double v[kVerifyUnits][8], mine = 0.0;
#pragma unroll
  for (int k = 0; k < kVerifyUnits; ++k) {
    w.unit(l, unit_of(pick, k), v[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) mine += v[k][i];
  }
  const double scan = wave_scan(mine);
  if (lane == 63) s.wave[0][wave] = scan;
  __syncthreads();
  double up = s.before;  // before this thread's first token
#pragma unroll
  for (int k = 0; k < kVerifyWaves; ++k)
    if (k < wave) up += s.wave[0][k];
  const double left = moved<0x138, 0xF>(scan, 0.0);  // the lane before (the whole wavefront shifted)
  up += left;
  int found = 0x7FFFFFFF, last = -1;
#pragma unroll
  for (int k = 0; k < kVerifyUnits; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int x = (int)(unit_of(pick, k) * 8) - w.shift_p + i;
      up += v[k][i];
      if (v[k][i] > 0.0) {
        last = x;
        if (found == 0x7FFFFFFF && up > target) found = x;
      }
    }
  // tokens rise with the threads: the first thread's, and the last thread's
  const uint64_t hits = __ballot(found != 0x7FFFFFFF), any = __ballot(last >= 0);
  const int f = hits ? __builtin_amdgcn_readlane(found, __ffsll((unsigned long long)hits) - 1) : 0x7FFFFFFF;
  const int e = any ? __builtin_amdgcn_readlane(last, 63 - __builtin_clzll(any)) : -1;
  if (lane == 0) s.first[wave] = f, s.last[wave] = e;
  __syncthreads();
  int token = 0x7FFFFFFF, end = -1;
#pragma unroll
  for (int k = 0; k < kVerifyWaves; ++k) {
    token = s.first[k] < token ? s.first[k] : token;
    end = s.last[k] > end ? s.last[k] : end;
  }
  return token != 0x7FFFFFFF ? token : end;
}

// LDS of a request's rows, by its last workgroup of the first kernel.
struct StopLds {
  int stop;
  Stop state;
  RowSum p[kVerifyRowsHeld], q[kVerifyRowsHeld];
  double mass[kVerifyRowsHeld][64];  // of the target: the first 64 chunks
};

// Where request r stops; accepted and accept_prob are written.
__device__ __forceinline__ Stop stop_of(const VerifyArgs& a, const VerifyLaunch& l, int r, int r0, int r1, StopLds& s) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid == 0) s.stop = r1 - 1;
  __syncthreads();
  for (int t = r0 + wave; t < r1; t += kVerifyWaves) {
    const bool drafted = t < r1 - 1;
    const int64_t d = drafted ? a.tokens[t + 1] : -1;
    const ChunkSum* const rows[2] = {l.sums + t * l.stride, l.sums + ((int64_t)a.rows + t) * l.stride};
    RowLoad first[2];  // all on their way at once
    first[0].load(rows[0], l);
    if (a.draft_logits) first[1].load(rows[1], l);
    const bool known = d >= 0 && d < a.n;
    double xp = 0.0, xq = 0.0;
    if (known) {
      xp = (double)__builtin_bit_cast(_Float16, a.logits[t * a.logits_stride + d]);
      if (a.draft_logits) xq = (double)__builtin_bit_cast(_Float16, a.draft_logits[t * a.draft_stride + d]);
    }
    const float u = drafted ? a.accept_u[t] : 0.0f;
    double mass, other;
    const RowSum p = join_row(rows[0], first[0], l, &mass);
    RowSum q{0.0, 1.0, false};
    if (a.draft_logits && drafted) q = join_row(rows[1], first[1], l, &other);
    if (t - r0 < kVerifyRowsHeld) {
      s.mass[t - r0][lane] = mass;
      if (lane == 0) s.p[t - r0] = p, s.q[t - r0] = q;
    }
    if (!drafted) {
      if (lane == 0) a.accept_prob[t] = 0.0f;
      break;
    }
    double pd = 0.0, qd = 1.0;
    if (known) pd = weight_of(xp - p.max, l) / p.sum;
    if (a.draft_logits) qd = !known ? 0.0 : q.valid ? weight_of(xq - q.max, l) / q.sum : __builtin_nan("");
    if (!p.valid) pd = __builtin_nan("");
    const bool accept = known && (double)u * qd < pd;
    if (lane == 0) {
      if (!accept) atomicMin(&s.stop, t);
      a.accept_prob[t] = !known ? 0.0f : pd != pd || qd != qd ? __builtin_nanf("")
                         : (float)(pd >= qd ? (pd > 0.0 ? 1.0 : 0.0) : pd / qd);
    }
  }
  __syncthreads();
  const int stop = s.stop, at = stop - r0;
  RowSum p, q{0.0, 1.0, false};
  if (at < kVerifyRowsHeld) {
    p = s.p[at], q = s.q[at];
  } else {  // (every wavefront by itself)
    RowLoad first;
    double mass;
    first.load(l.sums + stop * l.stride, l);
    p = join_row(l.sums + stop * l.stride, first, l, &mass);
    if (a.draft_logits && stop < r1 - 1) {
      first.load(l.sums + ((int64_t)a.rows + stop) * l.stride, l);
      q = join_row(l.sums + ((int64_t)a.rows + stop) * l.stride, first, l, &mass);
    }
  }
  if (tid == 0) a.accepted[r] = at;
  return {p.max, 1.0 / p.sum, q.max, 1.0 / q.sum, stop, q.valid, p.valid};
}

__device__ __forceinline__ Weigher weigher_of(const VerifyArgs& a, const Stop& s) {
  const uint16_t* const row = a.logits + s.row * a.logits_stride;
  const uint16_t* const drafter = s.drafter ? a.draft_logits + s.row * a.draft_stride : nullptr;
  return {row, drafter, shift_of(row), shift_of(drafter), s.top_p, s.scale_p, s.top_q, s.scale_q, -1, a.n};
}

// Request r's rows when it has any (false: it gets accepted 0, next -1).
__device__ __forceinline__ bool rows_of(const VerifyArgs& a, int r, int* r0, int* r1) {
  *r0 = a.row_start[r], *r1 = a.row_start[r + 1];
  return *r0 >= 0 && *r1 > *r0 && *r1 <= a.rows;
}

template <bool SAMPLED>
__global__ __launch_bounds__(kVerifyThreads) void verify_sums_kernel(VerifyArgs a, VerifyLaunch l) {
  __shared__ float s_max[kVerifySpan][kVerifyWaves];
  __shared__ double s_sum[kVerifySpan][kVerifyWaves];
  __shared__ uint64_t s_mine[kVerifyWaves];
  __shared__ uint32_t s_arrival;
  __shared__ StopLds s_stop;
  __shared__ TokenLds s_token;
  extern __shared__ double s_mass[];  // [chunks], greedy
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int split = blockIdx.x;
  const int64_t row = blockIdx.y;
  const bool draft = SAMPLED && blockIdx.z != 0;
  if (row < a.rows) {
    const uint16_t* const x = draft ? a.draft_logits + row * a.draft_stride : a.logits + row * a.logits_stride;
    const int shift = shift_of(x);
    auto load = [&](half8 (&v)[kVerifyUnits], int64_t chunk) {
#pragma unroll
      for (int k = 0; k < kVerifyUnits; ++k)
        v[k] = load_unit(x, shift, a.n, chunk * (kVerifyChunk / 8) + k * kVerifyThreads + tid);
    };
    half8 v[kVerifyUnits], next[kVerifyUnits];
    load(v, split);
    int spans = 0;
    for (int64_t chunk = split; chunk < l.chunks; chunk += l.splits, ++spans) {
      // (the last chunk again behind it)
      load(next, chunk + l.splits < l.chunks ? chunk + l.splits : chunk);
      // the wavefront's maximum, and whether it has a NaN or +inf
      float m = -__builtin_inff();
      bool bad = false;
#pragma unroll
      for (int k = 0; k < kVerifyUnits; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          m = fmaxf(m, (float)v[k][i]);
          bad |= !((float)v[k][i] < __builtin_inff());
        }
      m = wave_max(m);
      const bool none = m == -__builtin_inff();
      const double top = none || m == __builtin_inff() ? 0.0 : (double)m;
      double sum[2] = {0.0, 0.0};
#pragma unroll
      for (int k = 0; k < kVerifyUnits; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i & 1] += exp2_scaled((double)v[k][i] - top, l);
      double all = wave_sum(sum[0] + sum[1]);
      if (__ballot(bad)) all = __builtin_nan("");
      else if (none) all = 0.0;
      if (lane == 0) s_max[spans][wave] = m, s_sum[spans][wave] = all;
#pragma unroll
      for (int k = 0; k < kVerifyUnits; ++k) v[k] = next[k];
    }
    __syncthreads();
    if (tid < spans) {
      float high = s_max[tid][0];
#pragma unroll
      for (int w = 1; w < kVerifyWaves; ++w) high = fmaxf(high, s_max[tid][w]);
      double all = 0.0;
#pragma unroll
      for (int w = 0; w < kVerifyWaves; ++w) {
        const double x = s_sum[tid][w];
        all += x != x ? x : s_max[tid][w] > -__builtin_inff() ? x * weight_of((double)s_max[tid][w] - (double)high, l) : 0.0;
      }
      ChunkSum* const to = l.sums + ((draft ? a.rows : 0) + row) * l.stride + split + (int64_t)tid * l.splits;
      put_shared(&to->sum, all);
      put_shared(&to->max, (double)high);
    }
  }

  // the requests that hold this row (one, when row_start is in order); the
  // first workgroup answers for those without rows
  const bool first = split == 0 && row == 0 && !draft;
  for (int base = 0; base < a.requests; base += kVerifyThreads) {
    int r0, r1;
    bool mine = false;
    if (base + tid < a.requests) {
      const bool some = rows_of(a, base + tid, &r0, &r1);
      mine = some && row >= r0 && row < r1;
      if (!some && first) a.accepted[base + tid] = 0, a.next[base + tid] = -1;
    }
    const uint64_t bits = __ballot(mine);
    if (lane == 0) s_mine[wave] = bits;
    __syncthreads();
    for (int w = 0; w < kVerifyWaves; ++w) {
      uint64_t left = s_mine[w];
      while (left) {  // (the whole workgroup agrees)
        const int r = base + w * 64 + (__ffsll((unsigned long long)left) - 1);
        left &= left - 1;
        rows_of(a, r, &r0, &r1);
        const uint32_t count = (uint32_t)(r1 - r0) * (uint32_t)l.splits * (SAMPLED ? 2u : 1u);
        if (!arrive_last((uint32_t*)a.scratch + r * kArrivalStep, count, &s_arrival)) continue;
        const Stop s = stop_of(a, l, r, r0, r1, s_stop);
        if constexpr (SAMPLED) {
          if (tid == 0) l.stops[r] = s;
        } else {
          int token = -1;
          if (s.valid) {
            Weigher weigher = weigher_of(a, s);
            if (s.row < r1 - 1) weigher.skip = a.tokens[s.row + 1];
            if (weigher.skip >= a.n) weigher.skip = -1;
            const ChunkSum* const sums = l.sums + s.row * l.stride;
            if (s.row - r0 < kVerifyRowsHeld && l.chunks <= 64) {
              if (tid < l.chunks) s_mass[tid] = s_stop.mass[s.row - r0][tid] * s.scale_p;
              skip_token(weigher, l, s_mass, s_token);
            } else {
              masses_of_row(weigher, l, sums, s_mass, s_token);
            }
            token = pick_token(weigher, l, sums, a.sample_u[r], s_mass, s_token);
          }
          if (tid == 0) a.next[r] = token;
        }
        __syncthreads();
      }
    }
    __syncthreads();  // s_mine has been read
  }
}

__global__ __launch_bounds__(kVerifyThreads) void verify_token_kernel(VerifyArgs a, VerifyLaunch l) {
  __shared__ uint32_t s_arrival;
  __shared__ TokenLds s_token;
  extern __shared__ double s_mass[];  // [chunks]
  const int64_t chunk = blockIdx.x;
  const int r = blockIdx.y, tid = threadIdx.x;
  int r0, r1;
  if (!rows_of(a, r, &r0, &r1)) return;
  const Stop s = l.stops[r];
  if (!s.valid) {
    if (chunk == 0 && tid == 0) a.next[r] = -1;
    return;
  }
  const Weigher w = weigher_of(a, s);
  const ChunkSum* const sums = l.sums + s.row * l.stride;
  if (!s.drafter) {  // from p: the masses are there
    if (chunk != 0) return;
    masses_of_row(w, l, sums, s_mass, s_token);
  } else {
    double* const masses = l.masses + r * l.mass_stride;
    const double mass = chunk_mass(w, l, chunk, s_token);
    if (tid == 0) put_shared(masses + chunk, mass);
    if (!arrive_last((uint32_t*)a.scratch + r * kArrivalStep, (uint32_t)l.chunks, &s_arrival)) return;
    for (int64_t c = tid; c < l.chunks; c += kVerifyThreads) s_mass[c] = get_shared(masses + c);
  }
  const int token = pick_token(w, l, sums, a.sample_u[r], s_mass, s_token);
  if (tid == 0) a.next[r] = token;
}

constexpr size_t round_128(size_t x) { return (x + 127) / 128 * 128; }

}  // namespace

size_t verify_scratch_bytes(int rows, int requests, int64_t n) {
  const size_t chunks = (size_t)verify_chunks(n);
  return kKvZeroedBytes + 128 + 2 * (size_t)rows * round_128(chunks * sizeof(ChunkSum)) +
         (size_t)requests * (sizeof(Stop) + round_128(chunks * sizeof(double)));
}

hipError_t launch_verify(const VerifyArgs& a) {
  VerifyLaunch l;
  l.chunks = verify_chunks(a.n);
  l.stride = (int64_t)(round_128(l.chunks * sizeof(ChunkSum)) / sizeof(ChunkSum));
  l.mass_stride = (int64_t)(round_128(l.chunks * sizeof(double)) / sizeof(double));
  // (the scratch's address is a multiple of 16, lines are counted from 128)
  uint8_t* const base = (uint8_t*)round_128((uintptr_t)a.scratch + kKvZeroedBytes);
  l.sums = (ChunkSum*)base;
  l.stops = (Stop*)(l.sums + 2 * (int64_t)a.rows * l.stride);
  l.masses = (double*)(l.stops + a.requests);
  const double scale = a.inv_temperature * 1.4426950408889634;
  l.scale = scale < 1e-30 ? 1e-30 : scale > 1e290 ? 1e290 : scale;
  l.lowest = -1000.0 / l.scale;
  const hipStream_t st = (hipStream_t)a.stream;
  const size_t lds = (size_t)l.chunks * sizeof(double);
  const uint32_t rows = a.rows > 0 ? (uint32_t)a.rows : 1;  // (one workgroup answers for requests without rows)
  // as many workgroups a row as fill the chip, with no more chunks each than their LDS has room for
  const int64_t each = (kVerifyWgs + rows * (a.draft_logits ? 2 : 1) - 1) / (rows * (a.draft_logits ? 2 : 1));
  const int64_t least = (l.chunks + kVerifySpan - 1) / kVerifySpan;
  l.splits = (int)(each > l.chunks ? l.chunks : each < least ? least : each);
  if (!a.draft_logits) {
    verify_sums_kernel<false><<<dim3((uint32_t)l.splits, rows), dim3(kVerifyThreads), lds, st>>>(a, l);
    return hipGetLastError();
  }
  verify_sums_kernel<true><<<dim3((uint32_t)l.splits, rows, 2), dim3(kVerifyThreads), 0, st>>>(a, l);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  verify_token_kernel<<<dim3((uint32_t)l.chunks, (uint32_t)a.requests), dim3(kVerifyThreads), lds, st>>>(a, l);
  return hipGetLastError();
}

}  // namespace qpn
