// qpn_kv_rope_core.h -- what the cache appends share whatever their codes are:
// norms and rotation of queries and keys.
//
// A head of DIM dimensions lies over LPH = DIM / 8 neighbouring lanes, eight
// elements (one 16-byte load) each, so the norm is a sum over LPH lanes and
// the partner of a half-split rotation sits rot / 16 lanes away.
#pragma once

#include "qpn_common.h"
#include "qpn_kv_internal.h"
#include "qpn_kv_lanes.h"

namespace qpn {

namespace {

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

__device__ __forceinline__ double e4m3_value(uint32_t code) {
  const uint32_t m = code & 7, e = (code >> 3) & 15;
  if ((code & 0x7F) == 0x7F) return __longlong_as_double(0x7FF8000000000000ll);
  const double v = e ? ldexp(8.0 + m, (int)e - 10) : ldexp((double)m, -9);
  return code & 0x80 ? -v : v;
}

__device__ __forceinline__ half8 load_half8(const uint16_t* p) {
  return *reinterpret_cast<const half8*>(p);
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
// T: float for queries, double for keys.  The norm and rotation of eight
// elements of a head; `lane_at` is the lane's place among the head's LPH.
// cs: cosines and sines of the lane's own angles.
// What a lane needs of the weights and frequencies, for all rows.
template <int DIM>
struct Lane {
  half8 weight;
  float freq[8];  // of its own angles (interleaved: entries 0 .. 3)
  bool turned;    // its elements are rotated
  template <typename A>
  __device__ __forceinline__ void load(const A& a, int lane_at, const uint16_t* w) {
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

  template <typename A>
  __device__ __forceinline__ void angles(const A& a, const Lane<DIM>& f, int lane_at, double position) {
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
  template <typename A>
  __device__ __forceinline__ void turn(const A& a, const Lane<DIM>& f, int lane_at, const half8& x,
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

template <int DIM, int THREADS, typename A>
__device__ __forceinline__ void append_queries(const A& a, int wg, int waves_per_row,
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

}  // namespace

}  // namespace qpn
