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
// Two kernels.  The first reads every logit once and leaves, per row and chunk
// of kVerifyChunk tokens, the chunk's maximum and its sum of exponentials
// against that maximum.  The second (a workgroup per request and chunk) joins
// the chunks' sums to the rows' normalisers, finds the row L where the request
// stops, sums its chunk of max(p - q, 0) there and leaves the mass; the
// workgroup of a request that finishes last takes the masses' prefix sums,
// finds the chunk in which the random number falls, and the token in it.
// Sums run in an order fixed by the sizes, so results are deterministic.
#include "qpn_common.h"
#include "qpn_kv_internal.h"

namespace qpn {

namespace {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWaves = kVerifyThreads / kLanes;
constexpr int kVerifyUnits = 2;                            // 8-token units of a thread
constexpr int kVerifyChunk = kVerifyThreads * kVerifyUnits * 8;

// Chunks of a row: rows may start anywhere in a 16-byte granule, so a row's
// tokens are counted from the granule's start (up to 7 places before it).
__host__ __device__ constexpr int64_t verify_chunks(int64_t n) { return (n + 7 + kVerifyChunk - 1) / kVerifyChunk; }

constexpr int64_t kMaxVerifyChunks = verify_chunks(kMaxN);

struct ChunkSum {
  double sum;  // of exp(inv_temperature (x - max))
  double max;
};

// exp(x) for x <= 0 (or NaN): 2^k times the Taylor series of the rest, at most
// 0.347, whose first left-out term is below 7e-12 of it.
__device__ __forceinline__ double exp_of(double x) {
  x = fmax(x, -800.0);  // exp(-800) is 0 in 64 bits below; -inf needs no case of its own
  const double k = rint(x * 1.4426950408889634);
  // ln 2 as the nearest double and what is left of it
  const double r = fma(k, -2.3190468138462996e-17, fma(k, -0.6931471805599453, x));
  double p = fma(r, 1.0 / 362880.0, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return ldexp(p, (int)k);
}

// Eight tokens of a row from place 8 u - shift on; `in`: bit i set when token
// i of them is in [0, n).  `base` is the row, `shift` its offset in its
// 16-byte granule in elements.
__device__ __forceinline__ half8 load_unit(const uint16_t* base, int shift, int64_t n, int64_t u, uint32_t* in) {
  const int64_t first = u * 8 - shift;
  half8 x = {};
  if (first >= 0 && first + 8 <= n) {
    *in = 0xFF;
    x = *reinterpret_cast<const half8*>(base + first);
  } else {
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (first + i >= 0 && first + i < n) {
        bits |= 1u << i;
        x[i] = __builtin_bit_cast(_Float16, base[first + i]);
      }
    }
    *in = bits;
  }
  return x;
}

__device__ __forceinline__ int shift_of(const uint16_t* row) { return (int)(((uintptr_t)row & 15) >> 1); }

__global__ __launch_bounds__(kVerifyThreads) void verify_sums_kernel(VerifyArgs a, ChunkSum* sums) {
  __shared__ float s_max[kVerifyWaves];
  __shared__ double s_sum[kVerifyWaves];
  const int64_t chunk = blockIdx.x, row = blockIdx.y, chunks = gridDim.x;
  const bool draft = blockIdx.z != 0;
  const uint16_t* const x = draft ? a.draft_logits + row * a.draft_stride : a.logits + row * a.logits_stride;
  const int shift = shift_of(x), wave = threadIdx.x >> 6;
  half8 v[kVerifyUnits];
  uint32_t in[kVerifyUnits];
  float m = -__builtin_inff();
#pragma unroll
  for (int k = 0; k < kVerifyUnits; ++k) {
    v[k] = load_unit(x, shift, a.n, chunk * (kVerifyChunk / 8) + k * kVerifyThreads + threadIdx.x, &in[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (in[k] >> i & 1) m = fmaxf(m, (float)v[k][i]);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
  if ((threadIdx.x & 63) == 0) s_max[wave] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kVerifyWaves; ++w) m = fmaxf(m, s_max[w]);
  // a chunk of -inf alone sums nothing; NaN and +inf make the sum NaN
  double sum = 0.0;
  const double top = m;
#pragma unroll
  for (int k = 0; k < kVerifyUnits; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = (float)v[k][i];
      const bool some = (in[k] >> i & 1) && !(f == -__builtin_inff());
      const double e = f < __builtin_inff() ? exp_of(((double)f - top) * a.inv_temperature) : __builtin_nan("");
      sum += some ? e : 0.0;
    }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
  if ((threadIdx.x & 63) == 0) s_sum[wave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.0;
    for (int w = 0; w < kVerifyWaves; ++w) sum += s_sum[w];
    sums[((draft ? a.rows : 0) + row) * chunks + chunk] = ChunkSum{sum, top};
  }
}

// max and sum of a whole row from its chunks, by one wavefront: valid when the
// maximum is finite and the sum is a number.
struct RowSum {
  double max, sum;
  bool valid;
};
__device__ __forceinline__ RowSum join_row(const ChunkSum* c, int64_t chunks, double inv_temperature) {
  const int lane = threadIdx.x & 63;
  double m = -__builtin_inf(), s = 0.0;
  for (int64_t k = lane; k < chunks; k += 64) m = fmax(m, c[k].max);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = fmax(m, __shfl_xor(m, d));
  const bool finite = m > -__builtin_inf() && m < __builtin_inf();
  for (int64_t k = lane; k < chunks; k += 64) {
    const ChunkSum v = c[k];
    // (a chunk without any number but NaN has max -inf and a NaN sum)
    s += v.sum != v.sum ? v.sum : v.max > -__builtin_inf() && finite ? v.sum * exp_of((v.max - m) * inv_temperature) : 0.0;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
  return {m, s, finite && s == s};
}

// The weight of each token of a request's stopping row.
struct Weigher {
  const uint16_t *p, *q;         // q NULL: the draft alone (or none)
  int shift_p, shift_q;
  double top_p, scale_p, top_q, scale_q, inv_temperature;
  int64_t skip;                  // a greedy draft: its weight is 0
  int64_t n;
  // the weights of the 8 tokens of unit u (0 outside the row)
  __device__ __forceinline__ void unit(int64_t u, double w[8]) const {
    uint32_t in;
    const half8 x = load_unit(p, shift_p, n, u, &in);
    const int64_t first = u * 8 - shift_p;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      double v = 0.0;
      if (in >> i & 1) {
        v = exp_of(((double)x[i] - top_p) * inv_temperature) * scale_p;
        if (q) {
          const double z = (double)__builtin_bit_cast(_Float16, q[first + i]);
          v = fmax(v - exp_of((z - top_q) * inv_temperature) * scale_q, 0.0);
        }
        if (first + i == skip) v = 0.0;
      }
      w[i] = v;
    }
  }
};

// A chunk's tokens in order: thread t has the units kVerifyUnits t + k.
__device__ __forceinline__ int64_t unit_of(int64_t chunk, int k) {
  return chunk * (kVerifyChunk / 8) + (int64_t)threadIdx.x * kVerifyUnits + k;
}

// The sum of x over the threads before this one, and over all of them.
__device__ __forceinline__ double block_exclusive_scan(double x, double* waves, double* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double up = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double o = __shfl_up(up, d);
    if (lane >= d) up += o;
  }
  __syncthreads();  // what `waves` held has been read
  if (lane == 63) waves[wave] = up;
  __syncthreads();
  double before = 0.0;
  *total = 0.0;
#pragma unroll
  for (int w = 0; w < kVerifyWaves; ++w) {
    if (w < wave) before += waves[w];
    *total += waves[w];
  }
  // (not up - x: the exact sum of what comes before)
  const double left = __shfl_up(up, 1);
  return before + (lane ? left : 0.0);
}

__global__ __launch_bounds__(kVerifyThreads) void verify_token_kernel(VerifyArgs a, const ChunkSum* sums,
                                                                      double* masses, uint32_t* arrivals) {
  __shared__ int s_stop;
  __shared__ RowSum s_p, s_q;
  __shared__ double s_wave[kVerifyWaves];
  __shared__ uint32_t s_arrival;
  __shared__ double s_mass[kMaxVerifyChunks];
  __shared__ unsigned long long s_chunk, s_token;
  __shared__ long long s_last_chunk, s_last;
  __shared__ double s_before;
  const int64_t chunk = blockIdx.x, chunks = gridDim.x;
  const int r = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r0 = a.row_start[r], r1 = a.row_start[r + 1];
  const bool some = r0 >= 0 && r1 > r0 && r1 <= a.rows;  // the whole grid row agrees
  if (!some) {
    if (chunk == 0 && tid == 0) a.accepted[r] = 0, a.next[r] = -1;
    return;
  }
  const double it = a.inv_temperature;
  auto row_p = [&](int t) { return a.logits + t * a.logits_stride; };
  auto row_q = [&](int t) { return a.draft_logits + t * a.draft_stride; };

  // where the request stops: the first row whose draft is refused
  if (tid == 0) s_stop = r1 - 1;
  __syncthreads();
  for (int t = r0 + wave; t < r1; t += kVerifyWaves) {
    if (t == r1 - 1) {
      if (chunk == 0 && lane == 0) a.accept_prob[t] = 0.0f;
      break;
    }
    const int64_t d = a.tokens[t + 1];
    const RowSum p = join_row(sums + t * chunks, chunks, it);
    double pd = 0.0, qd = 1.0;
    const bool known = d >= 0 && d < a.n;
    if (known) pd = exp_of(((double)__builtin_bit_cast(_Float16, row_p(t)[d]) - p.max) * it) / p.sum;
    if (a.draft_logits) {
      const RowSum q = join_row(sums + ((int64_t)a.rows + t) * chunks, chunks, it);
      qd = !known ? 0.0 : q.valid ? exp_of(((double)__builtin_bit_cast(_Float16, row_q(t)[d]) - q.max) * it) / q.sum
                                  : __builtin_nan("");
    }
    if (!p.valid) pd = __builtin_nan("");
    const bool accept = known && (double)a.accept_u[t] * qd < pd;
    if (lane == 0) {
      if (!accept) atomicMin(&s_stop, t);
      if (chunk == 0)
        a.accept_prob[t] = !known ? 0.0f : pd != pd || qd != qd ? __builtin_nanf("")
                           : (float)(pd >= qd ? (pd > 0.0 ? 1.0 : 0.0) : pd / qd);
    }
  }
  __syncthreads();
  const int stop = s_stop;
  const bool last_row = stop == r1 - 1;
  if (wave == 0) {
    const RowSum p = join_row(sums + stop * chunks, chunks, it);
    if (lane == 0) s_p = p;
  } else if (wave == 1 && a.draft_logits && !last_row) {
    const RowSum q = join_row(sums + ((int64_t)a.rows + stop) * chunks, chunks, it);
    if (lane == 0) s_q = q;
  }
  __syncthreads();
  Weigher w{row_p(stop), nullptr, shift_of(row_p(stop)), 0, s_p.max, 1.0 / s_p.sum, 0.0, 0.0, it, -1, a.n};
  if (!last_row) {
    if (!a.draft_logits) {
      w.skip = a.tokens[stop + 1];
    } else if (s_q.valid) {
      w.q = row_q(stop);
      w.top_q = s_q.max;
      w.scale_q = 1.0 / s_q.sum;
    }
  }

  // this chunk's mass of the weights
  double mass = 0.0;
  {
#pragma unroll
    for (int k = 0; k < kVerifyUnits; ++k) {
      double v[8];
      w.unit(unit_of(chunk, k), v);
#pragma unroll
      for (int i = 0; i < 8; ++i) mass += v[i];
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) mass += __shfl_xor(mass, d);
  if (lane == 0) s_wave[wave] = mass;
  __syncthreads();
  if (tid == 0) {
    mass = 0.0;
    for (int k = 0; k < kVerifyWaves; ++k) mass += s_wave[k];
    // at the device's point of coherence before the arrival is counted
    __hip_atomic_store(masses + r * chunks + chunk, mass, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    s_arrival = __hip_atomic_fetch_add(arrivals + r, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (s_arrival != (uint32_t)(chunks - 1)) return;

  // the last workgroup of the request: the chunk in which the random number
  // falls.  Thread t has the chunks per t .. per t + per - 1.
  if (tid == 0) {
    __hip_atomic_store(arrivals + r, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    a.accepted[r] = stop - r0;
    s_chunk = s_token = ~0ull;
    s_last_chunk = s_last = -1;
  }
  const int64_t per = (chunks + kVerifyThreads - 1) / kVerifyThreads;
  const int64_t c0 = per * tid, c1 = c0 + per < chunks ? c0 + per : chunks;
  for (int64_t c = tid; c < chunks; c += kVerifyThreads)
    s_mass[c] = __hip_atomic_load(masses + r * chunks + c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  double up, total;
  auto scan_masses = [&]() {  // up: the masses before thread t's chunks
    __syncthreads();
    double own = 0.0;
    for (int64_t c = c0; c < c1; ++c) own += s_mass[c];
    up = block_exclusive_scan(own, s_wave, &total);
  };
  scan_masses();
  if (!(total > 0.0)) {  // nowhere above the drafter: the target itself
    w.q = nullptr;
    w.skip = -1;
    __syncthreads();
    for (int64_t c = tid; c < chunks; c += kVerifyThreads) {
      const ChunkSum v = sums[stop * chunks + c];
      s_mass[c] = v.max > -__builtin_inf() ? v.sum * exp_of((v.max - w.top_p) * it) * w.scale_p : 0.0;
    }
    scan_masses();
  }
  const double target = (double)a.sample_u[r] * total;
  {
    double at = up;
    for (int64_t c = c0; c < c1; ++c) {
      if (s_mass[c] > 0.0) {
        atomicMax(&s_last_chunk, (long long)c);
        if (at + s_mass[c] > target) atomicMin(&s_chunk, (unsigned long long)c);
      }
      at += s_mass[c];
    }
  }
  __syncthreads();
  const int64_t pick = s_chunk != ~0ull ? (int64_t)s_chunk : s_last_chunk;
  if (!s_p.valid || pick < 0) {
    if (tid == 0) a.next[r] = -1;
    return;
  }
  if (pick >= c0 && pick < c1) {
    double at = up;
    for (int64_t c = c0; c < pick; ++c) at += s_mass[c];
    s_before = at;
  }
  __syncthreads();
  double v[kVerifyUnits][8], mine = 0.0;
#pragma unroll
  for (int k = 0; k < kVerifyUnits; ++k) {
    w.unit(unit_of(pick, k), v[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) mine += v[k][i];
  }
  up = s_before + block_exclusive_scan(mine, s_wave, &total);  // before this thread's first token
  bool found = false;
  long long last = -1;
#pragma unroll
  for (int k = 0; k < kVerifyUnits; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const long long x = unit_of(pick, k) * 8 - w.shift_p + i;
      up += v[k][i];
      if (v[k][i] > 0.0) {
        last = x;
        if (!found && up > target) {
          found = true;
          atomicMin(&s_token, (unsigned long long)x);
        }
      }
    }
  if (last >= 0) atomicMax(&s_last, last);
  __syncthreads();
  if (tid == 0) a.next[r] = (int32_t)(s_token != ~0ull ? (long long)s_token : s_last);
}

}  // namespace

size_t verify_scratch_bytes(int rows, int requests, int64_t n) {
  const int64_t chunks = verify_chunks(n);
  return kKvZeroedBytes + (size_t)chunks * (2 * (size_t)rows * sizeof(ChunkSum) + (size_t)requests * sizeof(double));
}

hipError_t launch_verify(const VerifyArgs& a) {
  const int64_t chunks = verify_chunks(a.n);
  uint32_t* const arrivals = (uint32_t*)a.scratch;
  ChunkSum* const sums = (ChunkSum*)((uint8_t*)a.scratch + kKvZeroedBytes);
  double* const masses = (double*)(sums + 2 * (int64_t)a.rows * chunks);
  const hipStream_t st = (hipStream_t)a.stream;
  if (a.rows > 0) {
    verify_sums_kernel<<<dim3((uint32_t)chunks, (uint32_t)a.rows, a.draft_logits ? 2 : 1), dim3(kVerifyThreads), 0,
                         st>>>(a, sums);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  verify_token_kernel<<<dim3((uint32_t)chunks, (uint32_t)a.requests), dim3(kVerifyThreads), 0, st>>>(a, sums, masses,
                                                                                                  arrivals);
  return hipGetLastError();
}

}  // namespace qpn
