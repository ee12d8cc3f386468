// qpn_kv4_cache.hip -- the 4-bit paged KV cache is written and read back on
// gfx950: query/key norms with the rotation and the append, and tokens of the
// cache as FP16 rows.
#include "qpn_kv_rope_core.h"

namespace qpn {

namespace {

constexpr int kThreads = 256;

// The place of eight dimensions (the half `half` of the group `group` of 16) of token
// `off` of a page, in a block of the layout of include/qpn_kv4.h.
template <int DIM>
struct Place {
  static constexpr int G = DIM / 64;
  int k_code;   // byte offset of their four bytes of key codes
  int k_scale;  // byte offset of the key group's scale
  int v_code;   // byte offset of their byte of value codes for b = 0 (b: 16 bytes on each)
  int v_scale;
  __device__ __forceinline__ Place(int off, int group, int half) {
    const int t = off >> 4, c = off & 15, outer = group / G, i = group % G, n = t * G + i;
    k_code = (n / 2) * 1024 + (outer * 16 + c) * 16 + (n % 2) * 8 + 4 * half;
    k_scale = (outer * 16 + c) * (4 * G) + n;
    const int g = (off >> 2) & 3, r = off & 3, byte = (4 * t + r) * (2 * G) + 2 * i + half;
    v_code = (byte / 16) * 1024 + (16 * g + 4 * outer) * 16 + byte % 16;
    v_scale = i * 256 + (4 * g + outer) * 16 + 4 * t + r;
  }
};

// ---------------------------------------------------------------------------
// Norms, rotation and cache append.
//
// A group's scale is its token's own, so rows do not depend on one another (but for
// the rule that the later of two rows with one slot counts: a wavefront looks through
// the slots behind its row's), and every code goes to a byte that no other row writes.
// A wavefront takes a row and HPW = 64 / LPH KV heads, eight dimensions a lane; two
// neighbouring lanes are a group.
//
// One row is bound by a chain (slot, row, 64-bit angles, norms and codes, stores) behind a
// launch: 4.8 us with 40 + 8 heads of 128.  1024 rows, 30 MB, take 13.4 where a copy of the bytes
// takes 6.2: 9.0 with the queries alone, 8.8 with keys and values alone, of which the vector
// units' work adds up.  (A row's angles are found by each of its wavefronts: five of queries
// instead of two 13.9, ten 16.1.)
// ---------------------------------------------------------------------------

// Eight values of a group as E2M1 codes, element e at bits 4 e, and the group's scale
// (E4M3 code).  From 64 bits: bounds between codes are products of at most 31 bits with
// the group's step, so a value's code is exact, and a key's unless its FP64 error
// crosses a bound.
struct Codes {
  uint32_t codes, scale;
};
__device__ __forceinline__ Codes quantise(const double x[8], double unit) {
  double amax = 0.0;
  bool finite = unit > 0.0 && unit < __builtin_inf();
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const double a = fabs(x[e]);
    finite &= a < __builtin_inf();  // (not NaN either)
    amax = fmax(amax, a);
  }
  amax = fmax(amax, moved<0xB1>(amax));
  finite &= moved<0xB1>((int)finite) != 0;
  if (!finite) return {0u, 0x7Fu};
  const uint32_t scale = e4m3_code(amax / (6.0 * unit));
  const double step = e4m3_value(scale) * unit;
  uint32_t codes = 0;
  if (scale != 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double a = fabs(x[e]);
      // ties go to the even code: up to 2, 4, 6 at 0.75, 1.75, 3.5
      const uint32_t c = (uint32_t)(a > 0.25 * step) + (uint32_t)(a >= 0.75 * step) + (uint32_t)(a > 1.25 * step) +
                         (uint32_t)(a >= 1.75 * step) + (uint32_t)(a > 2.5 * step) + (uint32_t)(a >= 3.5 * step) +
                         (uint32_t)(a > 5.0 * step);
      const uint32_t sign = (uint32_t)((uint64_t)__double_as_longlong(x[e]) >> 63) << 3;
      codes |= (c | sign) << (4 * e);
    }
  }
  return {codes, scale};
}

// Whether a row behind `row` has its slot: 16 slots a lane at a time, in loads that do not wait
// for one another.
__device__ __forceinline__ bool taken_later(const int32_t* slots, int rows, int row, int32_t slot, int lane) {
  constexpr int STEP = 4 * kLanes;
  int from = row + 1;
  bool later = false;
  for (; rows - from >= 4 * STEP; from += 4 * STEP) {
    int32_t s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) __builtin_memcpy(s[i], slots + from + i * STEP + lane * 4, 16);
#pragma unroll
    for (int i = 0; i < 16; ++i) later |= s[i >> 2][i & 3] == slot;
    if (__ballot(later)) return true;
  }
  if (from >= rows) return false;
  int32_t s[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = slots[min(from + i * kLanes + lane, rows - 1)];
#pragma unroll
  for (int i = 0; i < 16; ++i) later |= s[i] == slot && from + i * kLanes + lane < rows;
  return __ballot(later) != 0;
}

template <int DIM>
__device__ __forceinline__ void append_tokens(const RopeAppend4Args& a, int wg, int waves_per_row) {
  constexpr int LPH = DIM / 8, HPW = kLanes / LPH;
  const int lane = threadIdx.x & 63, lane_at = lane % LPH;
  const int64_t wave = (int64_t)wg * (kThreads / kLanes) + (threadIdx.x >> 6);
  const int row = (int)(wave / waves_per_row);
  if (row >= a.rows) return;  // a whole wavefront; no barrier follows
  const int32_t slot = a.slots[row];
  if (slot < 0 || slot >= a.cache.pages * kKvPage) return;
  const int head = (int)(wave % waves_per_row) * HPW + lane / LPH;
  const bool there = head < a.cache.heads;
  const uint16_t* const from = a.qkv + row * a.qkv_stride + (int64_t)(a.q_heads + (there ? head : 0)) * DIM + lane_at * 8;
  const half8 kx = load_half8(from), vx = load_half8(from + (int64_t)a.cache.heads * DIM);
  Lane<DIM> f;
  f.load(a, lane_at, a.k_weight);
  const double k_unit = a.cache.k_unit[there ? head : 0], v_unit = a.cache.v_unit[there ? head : 0];
  if (taken_later(a.slots, a.rows, row, slot, lane)) return;

  double x[8];
  Rotor<double, DIM> rotor;
  if (a.rot) rotor.angles(a, f, lane_at, (double)a.positions[row]);
  rotor.turn(a, f, lane_at, kx, a.k_weight != nullptr, x);
  const Codes k = quantise(x, k_unit);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = (double)vx[e];
  const Codes v = quantise(x, v_unit);
  if (!there) return;
  const int64_t block = (int64_t)(slot / kKvPage) * a.cache.heads + head;
  const Place<DIM> at(slot % kKvPage, lane_at >> 1, lane_at & 1);
  *reinterpret_cast<uint32_t*>(a.cache.k + block * kv4_codes(DIM) + at.k_code) = k.codes;
  uint8_t* const vb = a.cache.v + block * kv4_codes(DIM) + at.v_code;
#pragma unroll
  for (int b = 0; b < 4; ++b)  // dimensions b and 4 + b of the eight: j even and odd
    vb[16 * b] = (uint8_t)((v.codes >> (4 * b) & 15u) | (v.codes >> (16 + 4 * b) & 15u) << 4);
  if ((lane_at & 1) == 0) {
    a.cache.k_scale[block * kv4_scales(DIM) + at.k_scale] = (uint8_t)k.scale;
    a.cache.v_scale[block * kv4_scales(DIM) + at.v_scale] = (uint8_t)v.scale;
  }
}

template <int DIM>
__global__ __launch_bounds__(kThreads) void rope_append4_kernel(RopeAppend4Args a, int cache_wgs, int cache_waves_per_row,
                                                                int waves_per_row, int steps) {
  if ((int)blockIdx.x < cache_wgs)
    append_tokens<DIM>(a, (int)blockIdx.x, cache_waves_per_row);
  else
    append_queries<DIM, kThreads>(a, (int)blockIdx.x - cache_wgs, waves_per_row, steps);
}

template <int DIM>
hipError_t launch_append4(const RopeAppend4Args& a) {
  constexpr int HPW = kLanes / (DIM / 8), WAVES = kThreads / kLanes;
  // heads per wavefront of queries: one step of HPW while that leaves fewer wavefronts than
  // 8 a CU, else more, so that a row's angles serve more heads
  const int head_groups = (a.q_heads + HPW - 1) / HPW;
  int64_t steps = (int64_t)a.rows * head_groups / 2048;
  steps = steps < 1 ? 1 : steps > head_groups ? head_groups : steps;
  const int waves_per_row = (int)((head_groups + steps - 1) / steps);
  const int cache_waves_per_row = (a.cache.heads + HPW - 1) / HPW;
  const int64_t cache_wgs = ((int64_t)a.rows * cache_waves_per_row + WAVES - 1) / WAVES;
  const int64_t query_wgs = ((int64_t)a.rows * waves_per_row + WAVES - 1) / WAVES;
  rope_append4_kernel<DIM><<<dim3((uint32_t)(cache_wgs + query_wgs)), dim3(kThreads), 0, (hipStream_t)a.stream>>>(
      a, (int)cache_wgs, cache_waves_per_row, waves_per_row, (int)steps);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Reading back: a lane takes eight dimensions of a token and head, a workgroup
// neighbouring rows of one head, so that the lines of a page that neighbouring tokens
// share are read together and rows are written in whole lines.  Bound by what it writes:
// 32768 tokens of 8 heads of 128, 172 MB, in 40 us, 4.3 TB/s (a large copy: 4.9).
// ---------------------------------------------------------------------------
__device__ __forceinline__ half8 scaled(const float x[8], float unit) {
  half8 y;
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = (_Float16)(x[e] * unit);
  return y;
}
__device__ __forceinline__ float read_unit(float u) { return u > 0.0f && u < __builtin_inff() ? u : __builtin_nanf(""); }

template <int DIM>
__global__ __launch_bounds__(kThreads) void read4_kernel(Read4Args a) {
  constexpr int LPH = DIM / 8, ROWS = kThreads / LPH;
  const int lane_at = threadIdx.x % LPH, head = (int)(blockIdx.x % (uint32_t)a.cache.heads);
  const int64_t row = (int64_t)(blockIdx.x / (uint32_t)a.cache.heads) * ROWS + threadIdx.x / LPH;
  if (row >= a.rows) return;
  const int32_t slot = a.slots[row];
  const bool there = slot >= 0 && slot < a.cache.pages * kKvPage;
  half8 k = {}, v = {};
  if (there) {
    const int64_t block = (int64_t)(slot / kKvPage) * a.cache.heads + head;
    const Place<DIM> at(slot % kKvPage, lane_at >> 1, lane_at & 1);
    const uint32_t kc = *reinterpret_cast<const uint32_t*>(a.cache.k + block * kv4_codes(DIM) + at.k_code);
    const uint8_t* const vb = a.cache.v + block * kv4_codes(DIM) + at.v_code;
    uint32_t vc = 0;  // byte b: dimensions b (low) and 4 + b
#pragma unroll
    for (int b = 0; b < 4; ++b) vc |= (uint32_t)vb[16 * b] << (8 * b);
    const uint32_t ks = a.cache.k_scale[block * kv4_scales(DIM) + at.k_scale];
    const uint32_t vs = a.cache.v_scale[block * kv4_scales(DIM) + at.v_scale];
    const half2v s = ue4m3_pair_to_f16(ks | vs << 8);
    const half8 kd = decode_e2m1x8(kc, half2v{s[0], s[0]}), vd = decode_e2m1x8(vc, half2v{s[1], s[1]});
    float kf[8], vf[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      kf[e] = (float)kd[e];
      vf[e] = (float)vd[2 * (e % 4) + e / 4];
    }
    k = scaled(kf, read_unit(a.cache.k_unit[head]));
    v = scaled(vf, read_unit(a.cache.v_unit[head]));
  }
  const int64_t column = (int64_t)head * DIM + lane_at * 8;
  *reinterpret_cast<half8*>(a.k_out + row * a.k_stride + column) = k;
  *reinterpret_cast<half8*>(a.v_out + row * a.v_stride + column) = v;
}

template <int DIM>
hipError_t launch_read4(const Read4Args& a) {
  constexpr int ROWS = kThreads / (DIM / 8);
  const int64_t grid = (int64_t)((a.rows + ROWS - 1) / ROWS) * a.cache.heads;
  read4_kernel<DIM><<<dim3((uint32_t)grid), dim3(kThreads), 0, (hipStream_t)a.stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope_append4(const RopeAppend4Args& a) {
  return a.cache.dim == 64 ? launch_append4<64>(a) : a.cache.dim == 128 ? launch_append4<128>(a) : launch_append4<256>(a);
}

hipError_t launch_read4(const Read4Args& a) {
  return a.cache.dim == 64 ? launch_read4<64>(a) : a.cache.dim == 128 ? launch_read4<128>(a) : launch_read4<256>(a);
}

}  // namespace qpn
