// qpn_kv_logprobs.hip -- log probabilities of given tokens, the entropy and the
// likeliest tokens of each row of logits on gfx950.
//
// With x_i = (z_i - m) / T, m the row's largest logit: S = sum exp(x_i), and
//   log p_i = x_i - log S,   entropy = log S - sum x_i exp(x_i) / S.
//
// One pass.  A row is cut into pieces, one workgroup each, a piece into tiles of 1024
// tokens that the workgroup's wavefronts take in turn, 16 tokens a lane.  A wavefront
// has a running maximum (at first the largest of all the workgroup's first tiles), each lane
// its part of S (in 64 bits: the largest token's 1 must not swallow the rest, which is what
// the log of a likely token is made of) and of the sum of x exp(x).
//
// The likeliest tokens.  Keys, unique and in the order wanted: the logit's bits made
// ascending, then the index descending.  A wavefront holds a list of keys in LDS and the
// least value that can still count.  Of a tile, only lanes whose largest logit reaches it
// can hold one; when more than `top` lanes do, the value that `top` of them reach is the
// new least one (found by bisection with ballots: the scalar unit's work).  What
// reaches it goes behind the list, which is cut to its `top` largest keys, by
// bisections of the values and then of the indices of the last one's equals, when it is
// long and at the end.  Wavefronts of a workgroup and then the pieces of a row are
// joined in the same way, by the last one of a row to arrive, which also sorts.
//
// Rows of 151936 tokens, calls one behind another: one, top 20, in 13.5 us, eight, top 5, in 11.1
// (both 8.6 without alternatives): a chain of the launch, a tile, the joins within a workgroup and
// between ten of them, each step of which waits for the one before (an instruction of the joins is
// run once and by few wavefronts).  256 rows, top 20, in 27.9 (16.6 without), 78 MB at 2.8 TB/s: a
// workgroup a CU; vector instructions are issued 82% of the time.  257 rows take a second turn of
// the chip: 47.  Of the value's bits only those are bisected in which the least and the largest
// differ (with all 16, and wavefronts reduced through LDS: 16.9, 14.6 and 30.8).
//
// That is of logits that spread.  A list is only cut, and `least` not raised, when tokens equal to
// the last one that counts keep coming, so that they all go through the lists: a row with all but
// ten tokens at -inf takes 42 us (256 rows 217), of equal logits 28 (148), of whole numbers 20 (35).
#include <type_traits>

#include "qpn_common.h"
#include "qpn_kv_internal.h"
#include "qpn_kv_lanes.h"
#include "qpn_kv_order.h"

namespace qpn {

namespace {

constexpr int kWaves = 16;
constexpr int kThreads = kWaves * kLanes;
constexpr int kVecs = 2;                          // loads of eight logits a lane, of a tile
constexpr int kTile = kVecs * 8 * kLanes;         // tokens of a wavefront's tile
constexpr int kMaxTop = kLogprobsMaxTop;
constexpr int kListMax = 192;                     // keys that a list is cut behind
constexpr int kListRoom = kListMax + kLanes;
constexpr int kMaxPieces = 64;                    // of a row
constexpr int kWanted = 256;                      // workgroups wanted: one a CU
constexpr int kCounterStep = 16;                  // 32-bit words between the rows' counters
static_assert((size_t)kWanted * kCounterStep * 4 <= kKvZeroedBytes, "a counter per row of a call with cut rows");
constexpr float kLowest = -65504.0f;
constexpr uint32_t kOrderedLowest = ordered_bits(0xFC00u);  // -inf's

struct Sums {
  float m;      // the largest logit (at least kLowest)
  double s, u;  // sum exp(x), sum of x exp(x), x in units of log 2, against m
};

// What a piece leaves in scratch; its keys, `top` of them, lie behind those of all rows.
struct Piece {
  double s, u;
  float m, pad;
};

__device__ __forceinline__ uint32_t ordered(float z) {
  return ordered_bits(__builtin_bit_cast(uint16_t, (_Float16)z));
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)bits_of_ordered(o));
}

__device__ __forceinline__ float wave_max(float x) {
  return wave_reduced(x, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  return wave_reduced(x, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ __forceinline__ uint32_t wave_min(uint32_t x) {
  return wave_reduced(x, [](uint32_t a, uint32_t b) { return min(a, b); });
}
__device__ __forceinline__ double wave_sum(double x) {
  return wave_reduced(x, [](double a, double b) { return a + b; });
}

// The largest t for which at least `top` of the wavefront's values (N a lane, from 1 on; those of
// lanes without one: 0) are t or more, and how many are; 0 and their number when there are fewer.
// Bisected between the least and the largest of them.
template <int N>
__device__ __forceinline__ uint32_t bound_of(const uint32_t (&x)[N], int top, int& reach) {
  uint32_t low = 0xFFFFFFFFu, high = 0;
  reach = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    reach += __popcll(__ballot(x[i] != 0));
    high = max(high, x[i]);
    low = min(low, x[i] - 1u);  // (0: the largest)
  }
  if (reach < top) return 0;
  uint32_t t = wave_min(low) + 1;
  const uint32_t most = wave_max(high);
#pragma unroll 1
  for (int bit = 31 - __clz((int)(most - t)); bit >= 0 && reach != top; --bit) {
    const uint32_t up = t + (1u << bit);
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n += __popcll(__ballot(x[i] >= up));
    if (n >= top) t = up, reach = n;
  }
  return t;
}

// The `top` largest of the wavefront's keys (N a lane; 0: none, and there are more than `top`):
// true at those.
template <int N>
__device__ __forceinline__ void choose(const uint64_t (&key)[N], int top, bool (&in)[N]) {
  uint32_t value[N];
  int reach;
#pragma unroll
  for (int i = 0; i < N; ++i) value[i] = (uint32_t)(key[i] >> 32);
  const uint32_t t = bound_of(value, top, reach);
#pragma unroll
  for (int i = 0; i < N; ++i) in[i] = key[i] != 0 && value[i] >= t;
  if (reach <= top) return;
  // of those equal to the last value the lowest indices (the others' keys count as their largest)
  int above = 0;
  uint32_t equal[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    above += __popcll(__ballot(value[i] > t));
    equal[i] = key[i] != 0 && value[i] == t ? ((uint32_t)key[i] & 0xFFFFFFu) + 1 : 0u;
  }
  const uint32_t least = bound_of(equal, top - above, reach);
#pragma unroll
  for (int i = 0; i < N; ++i) in[i] = key[i] != 0 && (value[i] > t || (value[i] == t && equal[i] >= least));
}

// A wavefront's list.
struct List {
  uint64_t* keys;  // LDS, kListRoom of them
  int count;       // uniform

  // Puts the keys of the lanes in `mask` behind the list.
  __device__ __forceinline__ void add(uint64_t mask, uint64_t key) {
    if (mask >> (threadIdx.x & 63) & 1)
      keys[count + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0))] = key;
    count += __popcll(mask);
  }

  // Cuts the list, of more than `top` keys, to its `top` largest.  (Just as many, whatever the logits
  // were: every key counts in bound_of, as ordered_bits is never 0, and no two are equal.  The room
  // behind kListMax is for what one add() may bring after it.)
  __device__ __forceinline__ void cut(int top) {
    constexpr int N = kListRoom / kLanes;
    const int lane = threadIdx.x & 63;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // what was added is there
    uint64_t key[N];
    bool in[N];
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] = i * kLanes + lane < count ? keys[i * kLanes + lane] : 0;
    choose(key, top, in);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before they are written over
    count = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) add(__ballot(in[i]), key[i]);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
};

// Of the wavefront's keys (N a lane; 0: none) a key a lane, the `top` largest among them.
// room: LDS for kLanes keys.
template <int N>
__device__ __forceinline__ uint64_t gathered(const uint64_t (&key)[N], int top, uint64_t* room) {
  uint32_t value[N];
  bool in[N];
  int reach;
#pragma unroll
  for (int i = 0; i < N; ++i) value[i] = (uint32_t)(key[i] >> 32);
  const uint32_t t = bound_of(value, top, reach);
#pragma unroll
  for (int i = 0; i < N; ++i) in[i] = key[i] != 0 && value[i] >= t;
  if (reach > kLanes) choose(key, top, in);  // (many equal ones)
  List list{room, 0};
#pragma unroll
  for (int i = 0; i < N; ++i) list.add(__ballot(in[i]), key[i]);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  const int lane = threadIdx.x & 63;
  return lane < list.count ? room[lane] : 0;
}

// A key's place among the wavefront's, the largest first (they are all different, in the first
// lanes; 0: none).  room: LDS for kLanes keys.
__device__ __forceinline__ int rank_of(uint64_t key, uint64_t* room) {
  room[threadIdx.x & 63] = key;
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  const int count = __popcll(__ballot(key != 0));
  int rank = 0;
#pragma unroll 1
  for (int i = 0; i < count; i += 8) {
    uint64_t other[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) other[j] = room[i + j];
#pragma unroll
    for (int j = 0; j < 8; ++j) rank += other[j] > key;
  }
  return rank;
}

__device__ __forceinline__ float lane_max(const half8 (&x)[kVecs]) {
  float high = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < kVecs * 8; ++i) high = fmaxf(high, (float)x[i >> 3][i & 7]);
  return high;
}

// The sums of the wavefront's lanes, in every lane.  (A logit of +inf leaves NaN in s.)
__device__ __forceinline__ Sums wave_joined(const Sums& x, float c) {
  Sums r;
  r.m = wave_max(x.m);
  const float d = (x.m - r.m) * c;
  const double f = (double)__builtin_amdgcn_exp2f(d);
  r.s = wave_sum(x.s * f);
  r.u = wave_sum((x.u + x.s * (double)fmaxf(d, -1e4f)) * f);
  return r;
}

template <bool TOP>
__global__ __launch_bounds__(kThreads) void logprobs_kernel(LogprobsArgs a, int pieces) {
  __shared__ uint64_t s_keys[TOP ? kWaves : 1][TOP ? kListRoom : 1];
  __shared__ Sums s_sums[kWaves];
  __shared__ uint64_t s_all[TOP ? kWaves * kMaxTop : 1];
  __shared__ int s_total;
  __shared__ uint32_t s_least, s_first_value[kWaves];
  __shared__ float s_first_max[kWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int row = (int)(blockIdx.x / (uint32_t)pieces), piece = (int)(blockIdx.x % (uint32_t)pieces);
  const uint16_t* const z = a.logits + row * a.logits_stride;
  // (as good as any larger or smaller one: two logits differ by 2^-24 at least and, but for -inf, by
  // 2^17 at most; not zero, so that -inf stays what it is)
  const float c = (float)(fmin(fmax(a.inv_temperature, 1e-30), 1e30) * 1.4426950408889634074);

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

  half8 next[kVecs];
#pragma unroll
  for (int v = 0; v < kVecs; ++v) next[v] = half8{} - (_Float16)__builtin_inff();
  if (first + wave < end) load(first + wave, next);
  const int32_t token = a.tokens[row];
  const bool good_token = token >= 0 && token < a.n;
  const uint16_t token_logit = z[good_token ? token : 0];

  // what the wavefronts' first tiles tell: the largest logit, and a value that `top` tokens
  // reach, since each wavefront has its share of them
  {
    const float high = lane_max(next), m = wave_max(high);
    if (lane == 0) s_first_max[wave] = m;
    if constexpr (TOP) {
      static_assert(kMaxTop <= 2 * kWaves, "its share is a token or two");
      float v = m;
      if (a.top > kWaves && __popcll(__ballot(high == m)) == 1) v = wave_max(high == m ? -__builtin_inff() : high);
      if (lane == 0) s_first_value[wave] = ordered(v);
      if (threadIdx.x == 0) s_least = kOrderedLowest, s_total = 0;
    }
    __syncthreads();
  }
  Sums mine{fmaxf(wave_max(lane < kWaves ? s_first_max[lane] : kLowest), kLowest), 0.0, 0.0};
  List list{s_keys[TOP ? wave : 0], 0};
  // the least value that counts (ordered): that `top` tokens reach, whichever wavefront saw them
  uint32_t least = kOrderedLowest;
  if constexpr (TOP) {
    least = max(least, wave_min(lane < kWaves ? s_first_value[lane] : 0xFFFFu));
  }
#pragma unroll 1
  for (int64_t tile = first + wave; tile < end; tile += kWaves) {
    half8 x[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) x[v] = next[v];
    if (tile + kWaves < end) load(tile + kWaves, next);
    const float high = lane_max(x);
    if (__ballot(high > mine.m)) {
      const float m = wave_max(fmaxf(high, mine.m)), d = (mine.m - m) * c;
      const double f = (double)__builtin_amdgcn_exp2f(d);
      mine.u = (mine.u + mine.s * (double)fmaxf(d, -1e4f)) * f;
      mine.s *= f;
      mine.m = m;
    }
    float u = 0.0f;
    if (__ballot(high == mine.m)) {  // the largest one's 1 is not added to small numbers in 32 bits
#pragma unroll
      for (int i = 0; i < kVecs * 8; ++i) {
        const float t = ((float)x[i >> 3][i & 7] - mine.m) * c, e = __builtin_amdgcn_exp2f(t);
        mine.s += (double)e;
        u = __builtin_fmaf(e, fmaxf(t, -1e4f), u);  // (0 where the logit is -inf)
      }
    } else {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < kVecs * 8; ++i) {
        const float t = ((float)x[i >> 3][i & 7] - mine.m) * c, e = __builtin_amdgcn_exp2f(t);
        s += e;
        u = __builtin_fmaf(e, fmaxf(t, -1e4f), u);
      }
      mine.s += (double)s;
    }
    mine.u += (double)u;
    if constexpr (TOP) {
      least = max(least, (uint32_t)__builtin_amdgcn_readfirstlane((int)*(volatile uint32_t*)&s_least));
      float at_least = value_of(least);
      const int lanes = __popcll(__ballot(high >= at_least));
      if (lanes > 0) {
        if (lanes > a.top) {
          int reach;
          const uint32_t o[1] = {ordered(high)};
          const uint32_t t = bound_of(o, a.top, reach);
          if (t > least) {
            least = t;
            at_least = value_of(least);
            if (lane == 0) atomicMax(&s_least, least);
          }
        }
        // the tokens that count: bit 8 + d for the lower half of the lane's word d, 24 + d for
        // the upper one, the signs of their differences from the least value
        uint32_t bits = 0;
        uint32_t less = __builtin_bit_cast(uint16_t, (_Float16)at_least) ^ 0x8000u;
        less = less == 0x8000u ? 0u : less;  // (+0 for 0, so that -0 is no less)
        const half2v from2 = __builtin_bit_cast(half2v, less * 0x10001u);
#pragma unroll
        for (int d = 0; d < kVecs * 4; ++d) {
          const u32x4 w = __builtin_bit_cast(u32x4, x[d >> 2]);
          const uint32_t y = w[d & 3];
          const half2v diff = __builtin_bit_cast(half2v, y) + from2;
          bits = bits >> 1 | (~__builtin_bit_cast(uint32_t, diff) & 0x80008000u);
        }
        if (least == kOrderedLowest) bits = 0xFF00FF00u;  // (-inf less -inf has no sign)
        // but for those that are not there, before the row or behind it
        const int64_t tile_at = tile * kTile - before;
        if (tile_at < 0 || tile_at + kTile > a.n) {
          int l = lane * 8;
          asm volatile("; ends" : "+v"(l));
#pragma unroll
          for (int i = 0; i < kVecs * 8; ++i) {
            const int64_t at = tile_at + l + (i >> 3) * (8 * kLanes) + (i & 7);
            if (at < 0 || at >= a.n) bits &= ~(1u << (8 + (i >> 1) + 16 * (i & 1)));
          }
        }
        while (__ballot(bits != 0)) {  // one of each lane
          const bool some = bits != 0;
          const int b = some ? __ffs((int)bits) - 1 : 8, d = b & 7;
          bits &= bits - 1;
          uint32_t w = 0;
#pragma unroll
          for (int k = 0; k < kVecs * 4; ++k) {
            const u32x4 y = __builtin_bit_cast(u32x4, x[k >> 2]);
            w = k == d ? y[k & 3] : w;
          }
          const uint32_t o = ordered_bits(b & 16 ? w >> 16 : w & 0xFFFFu);
          list.add(__ballot(some), key_of(o, (uint32_t)tile_at + lane * 8 + (d >> 2) * (8 * kLanes) + 2 * (d & 3) + (b >> 4)));
          if (list.count > kListMax) list.cut(a.top);
        }
      }
    }
  }

  // the workgroup's wavefronts, by the first one
  mine.s = wave_sum(mine.s), mine.u = wave_sum(mine.u);  // (a wavefront has one maximum)
  if (lane == 0) s_sums[wave] = mine;
  if constexpr (TOP) {  // (in any order: the keys are all different)
    if (list.count > kMaxTop) list.cut(a.top);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    int at = 0;
    if (lane == 0) at = atomicAdd(&s_total, list.count);
    at = __builtin_amdgcn_readfirstlane(at);
    if (lane < list.count) s_all[at + lane] = list.keys[lane];
  }
  __syncthreads();
  if (wave != 0) return;  // (no barrier follows)
  mine = wave_joined(lane < kWaves ? s_sums[lane] : Sums{kLowest, 0.0, 0.0}, c);
  uint64_t key = 0;  // the likeliest tokens', a lane each
  if constexpr (TOP) {
    const int total = s_total;
    if (total <= kLanes) {
      key = lane < total ? s_all[lane] : 0;
    } else {
      const auto gather = [&](auto n) {
        constexpr int N = decltype(n)::value;
        uint64_t some[N];
#pragma unroll
        for (int i = 0; i < N; ++i) some[i] = i * kLanes + lane < total ? s_all[i * kLanes + lane] : 0;
        key = gathered(some, a.top, list.keys);
      };
      if (total <= 2 * kLanes)
        gather(std::integral_constant<int, 2>{});
      else
        gather(std::integral_constant<int, kWaves * kMaxTop / kLanes>{});
    }
  }
  if (pieces > 1) {
    Piece* const out = reinterpret_cast<Piece*>((uint8_t*)a.scratch + kKvZeroedBytes) + (int64_t)row * pieces;
    uint64_t* const out_keys = reinterpret_cast<uint64_t*>((uint8_t*)a.scratch + kKvZeroedBytes +
                                                           (int64_t)a.rows * pieces * sizeof(Piece)) + (int64_t)row * pieces * a.top;
    if (lane == 0) {
      __hip_atomic_store(&out[piece].s, mine.s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(&out[piece].u, mine.u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(&out[piece].m, mine.m, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if constexpr (TOP) {  // `top` of them in any order, and zeros where there are fewer
      const uint64_t one[1] = {key};
      bool in[1] = {key != 0};
      if (__popcll(__ballot(in[0])) > a.top) choose(one, a.top, in);
      const uint64_t mask = __ballot(in[0]), other = ~mask;
      const uint64_t mine_of = in[0] ? mask : other;
      const int at = (in[0] ? 0 : __popcll(mask)) +
                     __builtin_amdgcn_mbcnt_hi((uint32_t)(mine_of >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mine_of, 0));
      if (at < a.top)
        __hip_atomic_store(&out_keys[piece * a.top + at], in[0] ? key : 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    uint32_t* const counter = (uint32_t*)a.scratch + row * kCounterStep;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wavefront's stores are there
    uint32_t arrived = 0;
    if (lane == 0) {
      arrived = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (arrived == (uint32_t)(pieces - 1))
        __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (__builtin_amdgcn_readfirstlane((int)arrived) != pieces - 1) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    Sums of{kLowest, 0.0, 0.0};
    constexpr int N = 4;  // keys a lane, of a step
    const int total = TOP ? pieces * a.top : 0;
    uint64_t some[N + 1];
    const auto load_keys = [&](int from) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int at = from + i * kLanes + lane;
        some[i] = at < total ? __hip_atomic_load(&out_keys[at], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0;
      }
    };
    if constexpr (TOP) load_keys(0);
    if (lane < pieces) {
      of.s = __hip_atomic_load(&out[lane].s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      of.u = __hip_atomic_load(&out[lane].u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      of.m = __hip_atomic_load(&out[lane].m, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    mine = wave_joined(of, c);
    if constexpr (TOP) {
      key = 0;
      for (int from = 0;;) {
        some[N] = key;
        key = gathered(some, a.top, list.keys);
        from += N * kLanes;
        if (from >= total) break;
        load_keys(from);
      }
    }
  }

  const bool bad = !(mine.s > 0.0) || !(mine.s < __builtin_inf()) || !(mine.m < __builtin_inff());
  const double log_s = bad ? __builtin_nan("") : log1p(mine.s - 1.0);  // (what is not the largest token)
  if (lane == 0) {
    double lp = __builtin_nan("");
    if (good_token && !bad)
      lp = ((double)(float)__builtin_bit_cast(_Float16, token_logit) - (double)mine.m) * a.inv_temperature - log_s;
    a.logprob[row] = (float)lp;
    a.entropy[row] = (float)(log_s - mine.u / mine.s * 0.69314718055994530942);
  }
  if constexpr (TOP) {
    const int found = __popcll(__ballot(key != 0));
    // (there are `top` of them, unless some logits are NaN; then the lanes behind fill the row)
    const int place = rank_of(key, list.keys), rank = key ? place : lane;
    if (rank < a.top && (key || lane >= found)) {
      const bool none = bad || !key;
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
  return kKvZeroedBytes + (p > 1 ? (size_t)rows * p * (sizeof(Piece) + kMaxTop * sizeof(uint64_t)) : 0);
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
