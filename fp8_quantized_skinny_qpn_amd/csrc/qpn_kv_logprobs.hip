// qpn_kv_logprobs.hip -- log probabilities of given tokens, the entropy and the
// likeliest tokens of each row of logits on gfx950.
//
// With x_i = (z_i - m) / T, m the row's largest logit: S = sum exp(x_i), and
//   log p_i = x_i - log S,   entropy = log S - sum x_i exp(x_i) / S.
//
// One pass.  A row is cut into pieces, one workgroup each, a piece into tiles of 1024
// tokens that the workgroup's wavefronts take in turn, 16 tokens a lane.  Each lane
// keeps its own running maximum, S (in 64 bits: the largest token's 1 must not swallow
// the rest, which is what the log of a likely token is made of) and sum of x exp(x).
//
// The likeliest tokens.  Keys, unique and in the order wanted: the logit's bits made
// ascending, then the index descending.  A wavefront holds a list of at most `top` keys in
// LDS and its smallest one as a bound.  Of a tile, only lanes whose largest logit is among
// the `top` largest of all lanes' (found by bisection with ballots: the scalar unit's
// work) or above the bound can hold one that counts; these are put behind the list, which
// is then cut to its `top` largest by a bisection over the keys.  Wavefronts of a
// workgroup and then the pieces of a row are joined in the same way, by the last one of a row
// to arrive, which also sorts.
#include "qpn_common.h"
#include "qpn_kv_internal.h"

namespace qpn {

namespace {

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kLanes;
constexpr int kVecs = 2;                          // loads of eight logits a lane, of a tile
constexpr int kTile = kVecs * 8 * kLanes;         // tokens of a wavefront's tile
constexpr int kMaxTop = kLogprobsMaxTop;
constexpr int kMaxPieces = 64;                    // of a row
constexpr int kWanted = 1024;                     // workgroups wanted
constexpr int kCounterStep = 16;                  // 32-bit words between the rows' counters
static_assert((size_t)kWanted * kCounterStep * 4 <= kKvZeroedBytes, "a counter per row of a call with cut rows");
constexpr float kLowest = -65504.0f;

struct Sums {
  float m;      // the largest logit (at least kLowest)
  double s, u;  // sum exp(x), sum of x exp(x), x in units of log 2, against m
};

// What a piece leaves in scratch, and behind it its kMaxTop keys.
struct Piece {
  double s, u;
  float m, pad;
  uint64_t keys[kMaxTop];
};

// Ascending in the value: the bits of an FP16 number (no NaN; -0 as 0).
__device__ __forceinline__ uint32_t ordered(float z) {
  const uint32_t b = __builtin_bit_cast(uint16_t, (_Float16)(z + 0.0f));
  return b & 0x8000u ? b ^ 0xFFFFu : b | 0x8000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)(o & 0x8000u ? o ^ 0x8000u : o ^ 0xFFFFu));
}
__device__ __forceinline__ uint64_t key_of(float z, int64_t index) {
  return (uint64_t)ordered(z) << 32 | (uint32_t)(0xFFFFFFFFu - (uint32_t)index);
}
__device__ __forceinline__ int index_of(uint64_t key) { return (int)(0xFFFFFFFFu - (uint32_t)key); }

// The largest t for which at least `top` of the wavefront's values are t or more (0 when
// there are fewer values).
__device__ __forceinline__ uint32_t bound_of(uint32_t x, int top) {
  uint32_t t = 0;
#pragma unroll 1
  for (int bit = 15; bit >= 0; --bit) {
    const uint32_t up = t | 1u << bit;
    const int n = __popcll(__ballot(x >= up));
    if (n >= top) t = up;
    if (n == top) break;
  }
  return t;
}
// The same of up to N keys a lane (0: none).
template <int N>
__device__ __forceinline__ uint64_t bound_of(const uint64_t (&key)[N], int top) {
  uint64_t t = 0;
#pragma unroll 1
  for (int bit = 47; bit >= 0; --bit) {
    const uint64_t up = t | 1ull << bit;
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n += __popcll(__ballot(key[i] >= up));
    if (n >= top) t = up;
    if (n == top) break;
  }
  return t;
}

// A wavefront's list.
struct List {
  uint64_t* keys;  // LDS, room for kMaxTop + kTile
  int count;       // uniform
  uint64_t bound;  // the smallest key when there are `top`, else 0

  // Puts the keys of the lanes in `mask` behind the list.
  __device__ __forceinline__ void add(uint64_t mask, uint64_t key) {
    if (mask >> (threadIdx.x & 63) & 1)
      keys[count + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0))] = key;
    count += __popcll(mask);
  }

  // Cuts the list to its `top` largest keys.  N keys a lane at a time: what is above
  // the bound of those and of the ones before.
  __device__ __forceinline__ void cut(int top) {
    constexpr int N = 4;
    const int lane = threadIdx.x & 63;
    if (count <= top) return;
    int kept = 0;
#pragma unroll 1
    for (int from = 0; from < count; from += (N - 1) * kLanes) {
      uint64_t key[N];
      key[0] = lane < kept ? keys[lane] : 0;  // (top is at most 64)
#pragma unroll
      for (int i = 1; i < N; ++i) {
        const int at = from + (i - 1) * kLanes + lane;
        key[i] = at >= kept && at < count ? keys[at] : 0;
      }
      bound = bound_of(key, top);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before they are written over
      const int all = count;
      count = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) add(__ballot(key[i] >= bound && key[i] != 0), key[i]);
      kept = count;
      count = all;
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    count = kept;
  }
};

// The sums of the wavefront's lanes, in every lane.  (A logit of +inf leaves NaN in s.)
__device__ __forceinline__ Sums wave_joined(const Sums& x, double c) {
  Sums r;
  r.m = x.m;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) r.m = fmaxf(r.m, __shfl_xor(r.m, d));
  const double d0 = ((double)x.m - (double)r.m) * c, f = exp2(d0);
  r.s = x.s * f;
  r.u = (x.u + x.s * d0) * f;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) r.s += __shfl_xor(r.s, d), r.u += __shfl_xor(r.u, d);
  return r;
}

template <bool TOP>
__global__ __launch_bounds__(kThreads) void logprobs_kernel(LogprobsArgs a, int pieces) {
  __shared__ uint64_t s_keys[TOP ? kWaves : 1][TOP ? kMaxTop + kTile : 1];
  __shared__ Sums s_sums[kWaves];
  __shared__ int s_count[kWaves];
  __shared__ uint32_t s_arrival;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int row = (int)(blockIdx.x / (uint32_t)pieces), piece = (int)(blockIdx.x % (uint32_t)pieces);
  const uint16_t* const z = a.logits + row * a.logits_stride;
  // (as good as any larger one: two logits differ by 2^-24 at least)
  const double cd = fmin(a.inv_temperature, 1e30) * 1.4426950408889634074;
  const float c = (float)cd;

  // tiles start at multiples of 16 bytes: the first one up to seven tokens before the row
  const int before = (int)(((uintptr_t)z >> 1) & 7);
  const int64_t tiles = (a.n + before + kTile - 1) / kTile;
  const int64_t first = tiles * piece / pieces, end = tiles * (piece + 1) / pieces;
  auto load = [&](int64_t tile, half8 (&x)[kVecs]) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int64_t at = tile * kTile - before + v * (8 * kLanes) + lane * 8;
      if (at >= 0 && at + 8 <= a.n) {
        x[v] = *reinterpret_cast<const half8*>(z + at);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[v][e] = at + e >= 0 && at + e < a.n ? __builtin_bit_cast(_Float16, z[at + e]) : (_Float16)-__builtin_inff();
      }
    }
  };

  Sums mine{kLowest, 0.0, 0.0};
  List list{s_keys[TOP ? wave : 0], 0, 0};
  half8 next[kVecs];
  if (first + wave < end) load(first + wave, next);
#pragma unroll 1
  for (int64_t tile = first + wave; tile < end; tile += kWaves) {
    half8 x[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) x[v] = next[v];
    if (tile + kWaves < end) load(tile + kWaves, next);
    float zf[kVecs * 8], high = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < kVecs * 8; ++i) {
      zf[i] = (float)x[i >> 3][i & 7];
      high = fmaxf(high, zf[i]);
    }
    const float m = fmaxf(mine.m, high), up = (mine.m - m) * c;
    const double f = (double)__builtin_amdgcn_exp2f(up);
    double s = mine.s * f;
    float u = 0.0f;
#pragma unroll
    for (int i = 0; i < kVecs * 8; ++i) {
      const float t = (zf[i] - m) * c, e = __builtin_amdgcn_exp2f(t);
      s += (double)e;
      u = __builtin_fmaf(e, fmaxf(t, -1e4f), u);  // (0 where the logit is -inf)
    }
    mine.u = (mine.u + mine.s * (double)up) * f + (double)u;
    mine.s = s;
    mine.m = m;
    if constexpr (TOP) {
      const uint32_t o = ordered(high), floor = (uint32_t)(list.bound >> 32);
      if (__ballot(o >= floor)) {
        const float least = value_of(max(bound_of(o, a.top), max(floor, 0x03FFu)));
#pragma unroll
        for (int i = 0; i < kVecs * 8; ++i) {
          uint64_t mask = __ballot(zf[i] >= least);
          if (mask) {
            const int64_t at = tile * kTile - before + (i >> 3) * (8 * kLanes) + lane * 8 + (i & 7);
            const uint64_t key = key_of(zf[i], at);
            mask = __ballot(zf[i] >= least && at >= 0 && at < a.n && key > list.bound);
            list.add(mask, key);
          }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        list.cut(a.top);
      }
    }
  }

  // the workgroup's wavefronts, by the first one
  mine = wave_joined(mine, cd);
  if (lane == 0) s_sums[wave] = mine, s_count[wave] = list.count;
  __syncthreads();
  Piece* const out = reinterpret_cast<Piece*>((uint8_t*)a.scratch + kKvZeroedBytes) + (int64_t)row * pieces;
  if (wave == 0) {
    mine = wave_joined(lane < kWaves ? s_sums[lane] : Sums{kLowest, 0.0, 0.0}, cd);
    if constexpr (TOP) {
#pragma unroll 1
      for (int w = 1; w < kWaves; ++w) {
        const int n = s_count[w];  // (at most top <= 64)
        list.add(n >= 64 ? ~0ull : (1ull << n) - 1, s_keys[w][lane < n ? lane : 0]);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      list.cut(a.top);
    }
    if (pieces > 1) {
      if (lane == 0) {
        __hip_atomic_store(&out[piece].s, mine.s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(&out[piece].u, mine.u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(&out[piece].m, mine.m, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      if (TOP && lane < a.top)
        __hip_atomic_store(&out[piece].keys[lane], lane < list.count ? list.keys[lane] : 0ull, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  if (pieces > 1) {
    uint32_t* const counter = (uint32_t*)a.scratch + row * kCounterStep;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wavefront's stores are there
    __syncthreads();
    if (threadIdx.x == 0) {
      const uint32_t arrived = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (arrived == (uint32_t)(pieces - 1))
        __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      s_arrival = arrived;
    }
    __syncthreads();
    if (s_arrival != (uint32_t)(pieces - 1)) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  }
  if (wave != 0) return;
  if (pieces > 1) {
    Sums of{kLowest, 0.0, 0.0};
    if (lane < pieces) {
      of.s = __hip_atomic_load(&out[lane].s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      of.u = __hip_atomic_load(&out[lane].u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      of.m = __hip_atomic_load(&out[lane].m, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    mine = wave_joined(of, cd);
    if constexpr (TOP) {
      // all pieces' keys through the list, as many as it has room for at a time
      list.count = 0;
      list.bound = 0;
      const int total = pieces * a.top;
#pragma unroll 1
      for (int from = 0; from < total; from += kTile) {
#pragma unroll 1
        for (int i = from; i < total && i < from + kTile; i += kLanes) {
          const int at = i + lane;
          uint64_t key = 0;
          if (at < total && at < from + kTile)
            key = __hip_atomic_load(&out[at / a.top].keys[at % a.top], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          list.add(__ballot(key > list.bound), key);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        list.cut(a.top);
      }
    }
  }

  const double log2e = 1.4426950408889634074;
  const bool bad = !(mine.s > 0.0) || !(mine.s < __builtin_inf()) || !(mine.m < __builtin_inff());
  const double rest = mine.s - 1.0;                       // what is not the largest token
  const double log_s = bad ? __builtin_nan("") : log1p(rest);
  if (lane == 0) {
    const int32_t token = a.tokens[row];
    double lp = __builtin_nan("");
    if (token >= 0 && token < a.n && !bad)
      lp = ((double)(float)__builtin_bit_cast(_Float16, z[token]) - (double)mine.m) * a.inv_temperature - log_s;
    a.logprob[row] = (float)lp;
    a.entropy[row] = (float)(log_s - mine.u / mine.s / log2e);
  }
  if constexpr (TOP) {
    // by rank: the keys are all different
    const uint64_t key = lane < list.count ? list.keys[lane] : 0;
    int rank = 0;
#pragma unroll 1
    for (int i = 0; i < list.count; ++i) rank += list.keys[i] > key;
    if (lane >= list.count) rank = lane;  // (never: there are top tokens, unless some are NaN)
    if (lane < a.top) {
      const bool none = bad || lane >= list.count;
      const double zi = value_of((uint32_t)(key >> 32));
      a.top_ids[(int64_t)row * a.top + rank] = none ? -1 : index_of(key);
      a.top_logprobs[(int64_t)row * a.top + rank] =
          none ? __builtin_nanf("") : (float)((zi - (double)mine.m) * a.inv_temperature - log_s);
    }
  }
}

// Pieces of a row: about kWanted workgroups in all, a tile a wavefront at least.
int pieces_of(int rows, int64_t n) {
  const int64_t most = (n + 7 + kWaves * kTile - 1) / (kWaves * kTile);
  int64_t p = kWanted / (rows < 1 ? 1 : rows);
  p = p > most ? most : p;
  p = p > kMaxPieces ? kMaxPieces : p;
  return p < 1 ? 1 : (int)p;
}

}  // namespace

size_t logprobs_scratch_bytes(int rows, int64_t n) {
  const int p = pieces_of(rows, n);
  return kKvZeroedBytes + (p > 1 ? (size_t)rows * p * sizeof(Piece) : 0);
}

hipError_t launch_logprobs(const LogprobsArgs& a) {
  const int pieces = pieces_of(a.rows, a.n);
  const dim3 grid((uint32_t)a.rows * (uint32_t)pieces);
  if (a.top > 0)
    logprobs_kernel<true><<<grid, dim3(kThreads), 0, (hipStream_t)a.stream>>>(a, pieces);
  else
    logprobs_kernel<false><<<grid, dim3(kThreads), 0, (hipStream_t)a.stream>>>(a, pieces);
  return hipGetLastError();
}

}  // namespace qpn
