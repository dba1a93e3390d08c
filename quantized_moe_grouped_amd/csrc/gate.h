// The gate of a gated feed-forward block, forward and backward, on the 32 x 32
// blocks of sums that a product leaves in registers, and how such a block's
// values go to memory and come back.
//
//   h = a(u) v,  a(u) = u s(z),  s(z) = 1 / (1 + exp(-z)),  s'(z) = s (1 - s)
//   silu: z = u;  gelu (its tanh form: 1 + tanh(y) = 2 s(2 y)): z = sqrt(8/pi) (u + 0.044715 u^3)
//   du = dh v a'(u),  a'(u) = s (1 + u z'(u) (1 - s));  dv = dh a(u)
//
// A lane holds 16 values of one row of a block: of row l % 32 the columns
// 8 q + 4 h + r, q, r = 0..3, h = l / 32.  A register swap between the wave's
// halves gives it neighbouring columns to store, and is its own inverse.
//
// The gate is two of the quarter-rate instructions (2^x, 1/x) and about six
// others a value forward, ten backward; what its products leave of a tile's time
// is the memory's (see gated_matmul.hip).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "mx_codes.h"

namespace gmmgm {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// u / (1 + exp(-u)) * v with the hardware's 2^x and 1/x, each within 1 ulp; the
// rounded exponent adds 0.6 |u| 2^-23.  Both flush results below the normal
// range, 1/x from u = -87 on.
__device__ __forceinline__ float swiglu(float u, float v) {
  return u * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u * -1.44269504f)) * v;
}
// The same below that, with h = exp(u / 2): u h * v * h (1 + h h is 1).  h stays
// normal down to u = -174, past which less than 2^-115 is left of any v.
__device__ __forceinline__ float swiglu_far(float u, float v) {
  const float h = __builtin_amdgcn_exp2f(u * 0.72134752f);
  return u * h * v * h;
}
// For a lane's values.  Gates below -87 are rare: both forms, and a choice for
// each value by its own gate alone, only where a lane of the wave has one (a form
// right for all gates, taken for all: 1.3%, FP4, 131072 x 7168 x 4096 over 32
// experts, 2034 -> 2060 us; the test of the gates 0.5%).
template <int N>
__device__ __forceinline__ void swiglus(const float (&u)[N], const float (&v)[N], float (&o)[N]) {
  uint32_t least = 0;  // the most negative gate has the largest bits
#pragma unroll
  for (int r = 0; r < N; ++r) least = max(least, __float_as_uint(u[r]));
  if (__any(least > __float_as_uint(-87.0f))) {
#pragma unroll
    for (int r = 0; r < N; ++r) o[r] = u[r] < -87.0f ? swiglu_far(u[r], v[r]) : swiglu(u[r], v[r]);
  } else {
#pragma unroll
    for (int r = 0; r < N; ++r) o[r] = swiglu(u[r], v[r]);
  }
}


// ---------------------------------------------------------------- gelu

constexpr float kGelu = 1.59576912f;           // sqrt(8 / pi)
constexpr float kGeluLog2 = 2.30220820f;       // times log2(e)
constexpr float kGeluCube = 0.044715f;
// z passes 300 at |u| = 16, far past where s is 0 or 1: u^2 goes no further,
// so that no square overflows (infinity times a factor that is 0 by then).
__device__ __forceinline__ float gelu_square(float u) { return fminf(u * u, 256.0f); }
__device__ __forceinline__ float gelu_exponent(float u, float square) {  // -z log2(e)
  return u * __builtin_fmaf(square, -kGeluLog2 * kGeluCube, -kGeluLog2);
}
// z'(u), up to 56.  u z' meets s (1 - s), which is 0 past |u| = 16, so that u
// goes no further than 16 there: beyond 6e36 the product would be infinite, and
// with that 0 no number.  (An infinite gate's du is the limit, dh v or 0.)
__device__ __forceinline__ float gelu_slope(float u) {
  return __builtin_fmaf(gelu_square(u), 3.0f * kGelu * kGeluCube, kGelu);
}
// As swiglus, with gelu: past z = -87 with exp(z / 2) twice.
template <int N>
__device__ __forceinline__ void geglus(const float (&u)[N], const float (&v)[N], float (&o)[N]) {
  float t[N], most = 0.0f;
#pragma unroll
  for (int r = 0; r < N; ++r) {
    t[r] = gelu_exponent(u[r], gelu_square(u[r]));
    most = fmaxf(most, t[r]);
  }
  if (__any(most > 125.0f)) {
#pragma unroll
    for (int r = 0; r < N; ++r) {
      const float h = __builtin_amdgcn_exp2f(t[r] * -0.5f);
      o[r] = t[r] > 125.0f ? u[r] * h * v[r] * h : u[r] * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t[r])) * v[r];
    }
  } else {
#pragma unroll
    for (int r = 0; r < N; ++r) o[r] = u[r] * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t[r])) * v[r];
  }
}

// ---------------------------------------------------------------- the way back

// One value, gates down to z = -87: with e = exp(-z), s = 1 / (1 + e) and 1 - s = e s.
// u and v become their gradients.
template <bool GELU>
__device__ __forceinline__ void gate_back(float t, float dh, float& u, float& v, float& h) {
  const float e = __builtin_amdgcn_exp2f(t), s = __builtin_amdgcn_rcpf(1.0f + e), a = u * s;
  float b = a;
  if constexpr (GELU) b = fminf(a, 16.0f) * gelu_slope(u);
  const float d = dh * v * __builtin_fmaf(b, e * s, s);
  h = a * v;
  v = dh * a;
  u = d;
}
// The same below that: s is p p with p = exp(z / 2), and 1 - s is 1.
template <bool GELU>
__device__ __forceinline__ void gate_back_far(float t, float dh, float& u, float& v, float& h) {
  const float p = __builtin_amdgcn_exp2f(t * -0.5f), a = u * p;
  float b = u;
  if constexpr (GELU) b = fmaxf(u, -16.0f) * gelu_slope(u);
  const float d = dh * v * p * (1.0f + b) * p;
  h = a * v * p;
  v = a * dh * p;
  u = d;
}
// For eight of a lane's values; as in swiglus the far form only where a lane of
// the wave needs it, and each value by its own gate.
template <bool GELU>
__device__ __forceinline__ void gate_back8(const float (&dh)[8], float (&u)[8], float (&v)[8], float (&h)[8]) {
  float t[8], most = 0.0f;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    t[r] = GELU ? gelu_exponent(u[r], gelu_square(u[r])) : u[r] * -1.44269504f;
    most = fmaxf(most, t[r]);
  }
  if (__any(most > 125.0f)) {
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      float fu = u[r], fv = v[r], fh;
      gate_back_far<GELU>(t[r], dh[r], fu, fv, fh);
      gate_back<GELU>(t[r], dh[r], u[r], v[r], h[r]);
      if (t[r] > 125.0f) u[r] = fu, v[r] = fv, h[r] = fh;
    }
  } else {
#pragma unroll
    for (int r = 0; r < 8; ++r) gate_back<GELU>(t[r], dh[r], u[r], v[r], h[r]);
  }
}

// ---------------------------------------------------------------- blocks in memory

enum Keep { kKeepNone = 0, kKeepFull = 1, kKeepFp8 = 2 };

// In 16 bits: two pieces of eight neighbouring columns a lane, piece q of the
// values 8 q .. 8 q + 7.  `row`: the block's row of the lane, n: the block's
// first column, of `width` (a multiple of 8).
template <bool HALF>
__device__ __forceinline__ void store_piece(uint16_t* row, int n, int width, int lane, int q, const float* v) {
  uint32_t d[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (HALF) {
      typedef _Float16 v2h __attribute__((ext_vector_type(2)));
      d[i] = __builtin_bit_cast(uint32_t, v2h{(_Float16)v[2 * i], (_Float16)v[2 * i + 1]});
    } else {
      typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
      d[i] = __builtin_bit_cast(uint32_t, v2bf{(__bf16)v[2 * i], (__bf16)v[2 * i + 1]});
    }
  }
  const auto a = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
  const int at = n + 16 * q + 8 * (lane >> 5);
  if (at < width) *(v4u*)(row + at) = v4u{a[0], b[0], a[1], b[1]};
}
template <bool HALF>
__device__ __forceinline__ void store_16(uint16_t* row, int n, int width, int lane, const float (&v)[16]) {
  store_piece<HALF>(row, n, width, lane, 0, v);
  store_piece<HALF>(row, n, width, lane, 1, v + 8);
}
__device__ __forceinline__ void load_16(const uint16_t* row, int n, int width, int lane, v4u (&d)[2]) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int at = n + 16 * q + 8 * (lane >> 5);
    d[q] = at < width ? *(const v4u*)(row + at) : v4u{0, 0, 0, 0};
  }
}
template <bool HALF>
__device__ __forceinline__ void values_16(const v4u& d, float (&v)[8]) {
  const auto a = __builtin_amdgcn_permlane32_swap(d.x, d.z, false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(d.y, d.w, false, false);
  const uint32_t two[4] = {a[0], b[0], a[1], b[1]};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (HALF) {
      v[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(two[i] & 0xFFFFu));
      v[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(two[i] >> 16));
    } else {
      v[2 * i] = __uint_as_float(two[i] << 16);
      v[2 * i + 1] = __uint_as_float(two[i] & 0xFFFF0000u);
    }
  }
}

// In FP8 with a scale for the block's 32 columns (all of which exist): 16
// neighbouring codes a lane.  The rules are quant_rows_kernel's.
__device__ __forceinline__ void store_fp8(uint8_t* row, uint8_t* scales, int n, int lane, const float (&v)[16]) {
  uint32_t mag = 0;
#pragma unroll
  for (int r = 0; r < 16; ++r) mag = max(mag, __float_as_uint(v[r]) & 0x7FFFFFFFu);
  const auto both = __builtin_amdgcn_permlane32_swap(mag, mag, false, false);
  const uint32_t code = gmmmq::scale_code<true>(max((uint32_t)both[0], (uint32_t)both[1]));
  const float scale = code == 255 ? 1.0f : gmmmq::scale_value(code), top = 448.0f * scale;
  uint32_t d[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float x[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = __builtin_amdgcn_fmed3f(v[4 * q + r], -top, top);
    typedef short v2s __attribute__((ext_vector_type(2)));
    v2s two = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v2s{0, 0}, x[0], x[1], scale, false);
    two = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(two, x[2], x[3], scale, true);
    d[q] = code == 255 ? 0u : __builtin_bit_cast(uint32_t, two);
  }
  const auto a = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
  *(v4u*)(row + n + 16 * (lane >> 5)) = v4u{a[0], a[1], b[0], b[1]};
  if (lane < 32) scales[n / 32] = (uint8_t)code;
}
__device__ __forceinline__ v4u load_fp8(const uint8_t* row, int n, int lane) { return *(const v4u*)(row + n + 16 * (lane >> 5)); }
// Brings the codes back to the lanes that compute: dwords 2 q and 2 q + 1 hold
// piece q's eight.
__device__ __forceinline__ void spread_fp8(v4u& d) {
  const auto a = __builtin_amdgcn_permlane32_swap(d.x, d.y, false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(d.z, d.w, false, false);
  d = v4u{a[0], b[0], a[1], b[1]};
}
__device__ __forceinline__ void values_fp8(uint32_t d0, uint32_t d1, uint32_t scale, float (&v)[8]) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  const float s = __uint_as_float(scale << 23);  // the conversion takes the exponent, 0 as 2^-127 and 255 as NaN
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t four = q ? d1 : d0;
    const v2f lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(four, s, false), hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(four, s, true);
    v[4 * q] = lo.x, v[4 * q + 1] = lo.y, v[4 * q + 2] = hi.x, v[4 * q + 3] = hi.y;
  }
}

// What was kept of a block's two halves, as it lies in memory.
template <bool FP8>
struct Kept {
  v4u gate[FP8 ? 1 : 2], up[FP8 ? 1 : 2];
  uint32_t gate_scale, up_scale;
};

}  // namespace gmmgm
