// Microscaled quantisation of 16- and 32-bit values and its inverse.
//
// Blocks of 32 values along k share the power of two 2^s with
//   s = floor(log2(amax)) - emax   (emax = 2 for FP4 E2M1, 8 for FP8 E4M3),
// clamped to [-127, 127] and -127 for a block of zeros; codes are the element
// format's nearest value to x * 2^-s, ties to even, saturated.  The exponent
// is read off amax's bits (fp16 values are widened first, so that subnormal
// ones have a normal exponent); scaling by a power of two is exact, so each
// code is rounded once.  A block with a NaN or an infinity gets the NaN scale
// 255 and zero codes.
//
// quant_rows_kernel  k is the fast axis of x: blocks lie flat in memory, and
//                    rows play no part.  8 values a lane, 4 lanes a block.
// quant_cols_kernel  x (e,k,n), blocks run down the rows: a lane holds 32 rows
//                    of two neighbouring columns, and a workgroup's codes go
//                    through LDS to leave as whole rows of (e,n,k).
// dequant_kernel     8 values a lane.
// All are bound by HBM.  x is read and the values are written past the caches
// (nontemporal: each is touched once here; codes and scales, which the next
// product or the inverse reads, go through them), two chunks to a thread:
// quantising 16384 x 7168 bf16 to FP8 and back 147 -> 118 us (6.1 TB/s), 32 x
// 2048 x 7168 bf16 weights turned to FP4 and back 500 -> 409 us (5.8 TB/s);
// four and eight chunks to a thread took 120 and 127 us.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/gmmfr.h"
#include "mx_codes.h"

namespace gmmmq {

typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef short v2s __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));

enum In { kBf16 = 0, kF16 = 1, kF32 = 2 };

struct Params {
  const void* x;
  uint8_t* codes;
  uint8_t* scales;
  void* values;     // dequantisation's output
  int64_t chunks;   // 8-value chunks in all (rows), or 0
  int64_t k, n;     // columns kernel
  int64_t tiles_k, tiles_n;
  int64_t first;    // workgroups of the launches before this one
};

template <int IN>
__device__ __forceinline__ float value(uint32_t two, int i) {
  if constexpr (IN == kBf16) return __uint_as_float(i ? two & 0xFFFF0000u : two << 16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)(i ? two >> 16 : two & 0xFFFFu));
}

// Codes of two values over the block's scale.  The FP4 conversion saturates by
// itself; FP8's gives NaN past 464, so values are first held to +-448 scale.
template <bool FP8>
__device__ __forceinline__ uint32_t codes2(float a, float b, uint32_t code, float scale) {
  if (code == 255) a = b = 0.0f, scale = 1.0f;
  if constexpr (FP8) {
    const float top = 448.0f * scale;
    a = fminf(fmaxf(a, -top), top);
    b = fminf(fmaxf(b, -top), top);
    const v2s r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v2s{0, 0}, a, b, scale, false);
    return (uint16_t)r.x;
  } else {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, a, b, scale, 0) & 0xFFu;
  }
}

template <int IN>
__device__ __forceinline__ void load8(const void* x, int64_t chunk, float (&v)[8]) {
  if constexpr (IN == kF32) {
    const v4f a = __builtin_nontemporal_load((const v4f*)x + 2 * chunk);
    const v4f b = __builtin_nontemporal_load((const v4f*)x + 2 * chunk + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
  } else {
    const v4u a = __builtin_nontemporal_load((const v4u*)x + chunk);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = value<IN>(a[i / 2], i & 1);
  }
}

constexpr int kThreads = 256, kPer = 2;  // chunks of a thread, kThreads apart

template <int IN, bool FP8>
__global__ __launch_bounds__(kThreads) void quant_rows_kernel(Params p) {
  const int64_t first = (p.first + blockIdx.x) * (kThreads * kPer) + threadIdx.x;
  float v[kPer][8];
#pragma unroll
  for (int u = 0; u < kPer; ++u)
    if (first + u * kThreads < p.chunks) load8<IN>(p.x, first + u * kThreads, v[u]);
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int64_t c = first + u * kThreads;
    if (c >= p.chunks) break;  // the four lanes of a block end together: chunks % 8 == 0
    uint32_t mag = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) mag = max(mag, __float_as_uint(v[u][i]) & 0x7FFFFFFFu);
    mag = max(mag, (uint32_t)__shfl_xor((int)mag, 1));
    mag = max(mag, (uint32_t)__shfl_xor((int)mag, 2));
    const uint32_t code = scale_code<FP8>(mag);
    const float scale = scale_value(code);
    uint32_t d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = codes2<FP8>(v[u][2 * i], v[u][2 * i + 1], code, scale);
    if constexpr (FP8) ((v2u*)p.codes)[c] = v2u{d[0] | d[1] << 16, d[2] | d[3] << 16};
    else ((uint32_t*)p.codes)[c] = d[0] | d[1] << 8 | d[2] << 16 | d[3] << 24;
    if ((c & 3) == 0) p.scales[c >> 2] = (uint8_t)code;
  }
}

// A workgroup: 128 columns, 256 rows (8 blocks); its four waves take two
// blocks each, a lane two neighbouring columns.
constexpr int kColN = 128, kColK = 256;

template <int IN, bool FP8>
__global__ __launch_bounds__(kThreads) void quant_cols_kernel(Params p) {
  constexpr int kBytes = FP8 ? 32 : 16;         // codes of a block
  constexpr int kRow = 8 * kBytes + 16;         // of a column, padded apart in the banks
  __shared__ __attribute__((aligned(16))) uint8_t s_codes[kColN * kRow];
  __shared__ __attribute__((aligned(16))) uint8_t s_scales[kColN * 8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t per = p.tiles_k * p.tiles_n, at_tile = p.first + blockIdx.x, g = at_tile / per, t = at_tile % per;
  const int64_t k0 = (t % p.tiles_k) * kColK, n0 = (t / p.tiles_k) * kColN;
  const int64_t col = n0 + 2 * lane;
  const int blocks = (int)min((int64_t)8, (p.k - k0) / 32);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int b = wave * 2 + half;
    if (b >= blocks || col >= p.n) continue;
    const int64_t at = (g * p.k + k0 + b * 32) * p.n + col;
    float v[2][32];
    if constexpr (IN == kF32) {
#pragma unroll
      for (int r = 0; r < 32; ++r) {
        const v2f two = __builtin_nontemporal_load((const v2f*)((const float*)p.x + at + r * p.n));
        v[0][r] = two.x, v[1][r] = two.y;
      }
    } else {
      uint32_t two[32];
#pragma unroll
      for (int r = 0; r < 32; ++r)
        two[r] = __builtin_nontemporal_load((const uint32_t*)((const uint16_t*)p.x + at + r * p.n));
#pragma unroll
      for (int r = 0; r < 32; ++r) v[0][r] = value<IN>(two[r], 0), v[1][r] = value<IN>(two[r], 1);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t mag = 0;
#pragma unroll
      for (int r = 0; r < 32; ++r) mag = max(mag, __float_as_uint(v[c][r]) & 0x7FFFFFFFu);
      const uint32_t code = scale_code<FP8>(mag);
      const float scale = scale_value(code);
      uint32_t d[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) d[i] = codes2<FP8>(v[c][2 * i], v[c][2 * i + 1], code, scale);
      v4u* to = (v4u*)&s_codes[(2 * lane + c) * kRow + b * kBytes];
      if constexpr (FP8) {
        to[0] = v4u{d[0] | d[1] << 16, d[2] | d[3] << 16, d[4] | d[5] << 16, d[6] | d[7] << 16};
        to[1] = v4u{d[8] | d[9] << 16, d[10] | d[11] << 16, d[12] | d[13] << 16, d[14] | d[15] << 16};
      } else {
        v4u o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = d[4 * i] | d[4 * i + 1] << 8 | d[4 * i + 2] << 16 | d[4 * i + 3] << 24;
        to[0] = o;
      }
      s_scales[(2 * lane + c) * 8 + b] = (uint8_t)code;
    }
  }
  __syncthreads();
  // out: a column's codes of this tile in 16-byte pieces
  constexpr int kPieces = 8 * kBytes / 16;
  const int64_t row = FP8 ? p.k : p.k / 2;
#pragma unroll
  for (int q = threadIdx.x; q < kColN * kPieces; q += kThreads) {
    const int c = q / kPieces, piece = q % kPieces;
    if (n0 + c < p.n && piece * 16 < blocks * kBytes)
      *(v4u*)(p.codes + (g * p.n + n0 + c) * row + k0 * kBytes / 32 + piece * 16) =
          *(const v4u*)&s_codes[c * kRow + piece * 16];
  }
  // scales in pairs (k / 64 of them a column)
  for (int q = threadIdx.x; q < kColN * 4; q += kThreads) {
    const int c = q / 4, pair = q % 4;
    if (n0 + c < p.n && pair * 2 < blocks)
      *(uint16_t*)(p.scales + (g * p.n + n0 + c) * (p.k / 32) + k0 / 32 + pair * 2) =
          *(const uint16_t*)&s_scales[c * 8 + pair * 2];
  }
}

template <int OUT, bool FP8>
__global__ __launch_bounds__(kThreads) void dequant_kernel(Params p) {
  const int64_t first = (p.first + blockIdx.x) * (kThreads * kPer) + threadIdx.x;
  v2u d[kPer];
  uint32_t s[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int64_t c = first + u * kThreads;
    if (c < p.chunks) {
      if constexpr (FP8) d[u] = ((const v2u*)p.codes)[c];
      else d[u] = v2u{((const uint32_t*)p.codes)[c], 0};
      s[u] = p.scales[c >> 2];
    }
  }
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int64_t c = first + u * kThreads;
    if (c >= p.chunks) break;
    const float scale = scale_value(s[u]);
    float v[8];
    if constexpr (FP8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const v2f two = (i & 1) ? __builtin_amdgcn_cvt_pk_f32_fp8((int)d[u][i / 2], true)
                                : __builtin_amdgcn_cvt_pk_f32_fp8((int)d[u][i / 2], false);
        v[2 * i] = two.x * scale, v[2 * i + 1] = two.y * scale;
      }
    } else {
      static_assert(FP8 || sizeof(v) == 32, "eight values");
      const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d[u].x, 1.0f, 0);
      const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d[u].x, 1.0f, 1);
      const v2f e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d[u].x, 1.0f, 2);
      const v2f f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d[u].x, 1.0f, 3);
      v[0] = a.x * scale, v[1] = a.y * scale, v[2] = b.x * scale, v[3] = b.y * scale;
      v[4] = e.x * scale, v[5] = e.y * scale, v[6] = f.x * scale, v[7] = f.y * scale;
    }
    if constexpr (OUT == kF32) {
      __builtin_nontemporal_store(v4f{v[0], v[1], v[2], v[3]}, (v4f*)p.values + 2 * c);
      __builtin_nontemporal_store(v4f{v[4], v[5], v[6], v[7]}, (v4f*)p.values + 2 * c + 1);
    } else {
      v4u o;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (OUT == kBf16) {
          typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
          o[i] = __builtin_bit_cast(uint32_t, v2bf{(__bf16)v[2 * i], (__bf16)v[2 * i + 1]});
        } else {
          typedef _Float16 v2h __attribute__((ext_vector_type(2)));
          o[i] = __builtin_bit_cast(uint32_t, v2h{(_Float16)v[2 * i], (_Float16)v[2 * i + 1]});
        }
      }
      __builtin_nontemporal_store(o, (v4u*)p.values + c);
    }
  }
}

// ---------------------------------------------------------------- host side

bool given(const gmmfr_tensor& t) {
  if (t.data != nullptr) return true;
  for (int i = 0; i < t.ndim && i < 4; ++i)
    if (t.dims[i] == 0) return true;
  return false;
}

int validate(const gmmmq_args* a, bool back, Params* p, int* in, bool* fp8, int64_t* e) {
  if (!a) return GMMFR_ERR_NULLPTR;
  if (!given(a->x) || !given(a->codes) || !given(a->scales)) return GMMFR_ERR_NULLPTR;
  if (a->x.dtype == GMMFR_DT_BFLOAT16) *in = kBf16;
  else if (a->x.dtype == GMMFR_DT_FLOAT16) *in = kF16;
  else if (a->x.dtype == GMMFR_DT_FLOAT32) *in = kF32;
  else return GMMFR_ERR_DTYPE;
  if (a->codes.dtype != GMMFR_DT_FLOAT4_E2M1X2 && a->codes.dtype != GMMFR_DT_FLOAT8_E4M3FN) return GMMFR_ERR_DTYPE;
  *fp8 = a->codes.dtype == GMMFR_DT_FLOAT8_E4M3FN;
  if (a->scales.dtype != GMMFR_DT_FLOAT8_E8M0) return GMMFR_ERR_DTYPE;
  if (a->transpose != 0 && (a->transpose != 1 || back)) return GMMFR_ERR_ATTR;
  const int nd = a->x.ndim;
  if ((nd != 2 && nd != 3) || (a->transpose && nd != 3)) return GMMFR_ERR_SHAPE;
  const int64_t lead = nd == 3 ? a->x.dims[0] : 1;
  const int64_t k = a->transpose ? a->x.dims[1] : a->x.dims[nd - 1];
  const int64_t n = a->transpose ? a->x.dims[2] : a->x.dims[nd - 2];
  if (lead < 0 || n < 0 || lead >= (int64_t(1) << 31) || n >= (int64_t(1) << 31) || lead * n >= (int64_t(1) << 31))
    return GMMFR_ERR_SHAPE;
  if (k < 64 || k > 65536 || k % 64 != 0 || (a->transpose && n % 8 != 0)) return GMMFR_ERR_SHAPE;
  if (a->codes.ndim != nd || a->scales.ndim != nd + 1) return GMMFR_ERR_SHAPE;
  if (nd == 3 && (a->codes.dims[0] != lead || a->scales.dims[0] != lead)) return GMMFR_ERR_SHAPE;
  if (a->codes.dims[nd - 2] != n || a->codes.dims[nd - 1] != (*fp8 ? k : k / 2)) return GMMFR_ERR_SHAPE;
  if (a->scales.dims[nd - 2] != n || a->scales.dims[nd - 1] != k / 64 || a->scales.dims[nd] != 2) return GMMFR_ERR_SHAPE;
  for (const gmmfr_tensor* t : {&a->x, &a->codes, &a->scales})
    if (((uintptr_t)t->data & 15u) != 0) return GMMFR_ERR_ALIGN;
  p->x = p->values = a->x.data;
  p->codes = (uint8_t*)a->codes.data;
  p->scales = (uint8_t*)a->scales.data;
  p->k = k;
  p->n = n;
  p->chunks = lead * n * (k / 8);
  p->tiles_k = (k + kColK - 1) / kColK;
  p->tiles_n = (n + kColN - 1) / kColN;
  *e = lead;
  return GMMFR_OK;
}

template <typename F>
void with(int in, bool fp8, F&& f) {
  auto go = [&](auto i_) {
    if (fp8) f(i_, std::true_type{});
    else f(i_, std::false_type{});
  };
  if (in == kBf16) go(std::integral_constant<int, kBf16>{});
  else if (in == kF16) go(std::integral_constant<int, kF16>{});
  else go(std::integral_constant<int, kF32>{});
}

// A launch holds fewer than 2^32 threads (more are dropped without an error):
// `groups` workgroups in launches of at most 2^23.  hipLaunchKernel gives each
// launch's own status, where the runtime's last error may be an earlier one of
// the program's.
int in_launches(const void* kernel, int64_t groups, Params p, void* stream) {
  constexpr int64_t kMost = int64_t(1) << 23;
  static_assert(kMost * kThreads < (int64_t(1) << 32), "threads of a launch");
  void* args[] = {&p};
  for (p.first = 0; p.first < groups; p.first += kMost) {
    const int64_t left = groups - p.first;
    const dim3 grid((uint32_t)(left < kMost ? left : kMost));
    if (hipLaunchKernel(kernel, grid, dim3(kThreads), args, 0, (hipStream_t)stream) != hipSuccess) return GMMFR_ERR_HIP;
  }
  return GMMFR_OK;
}

int quantize(const gmmmq_args* a, void* stream) {
  Params p;
  int in;
  bool fp8;
  int64_t e;
  const int st = validate(a, false, &p, &in, &fp8, &e);
  if (st != GMMFR_OK) return st;
  const void* kernel = nullptr;
  with(in, fp8, [&](auto in_, auto fp8_) {
    kernel = a->transpose ? (const void*)quant_cols_kernel<decltype(in_)::value, decltype(fp8_)::value>
                          : (const void*)quant_rows_kernel<decltype(in_)::value, decltype(fp8_)::value>;
  });
  const int64_t groups = a->transpose ? e * p.tiles_k * p.tiles_n : (p.chunks + kThreads * kPer - 1) / (kThreads * kPer);
  return in_launches(kernel, groups, p, stream);
}

int dequantize(const gmmmq_args* a, void* stream) {
  Params p;
  int out;
  bool fp8;
  int64_t e;
  const int st = validate(a, true, &p, &out, &fp8, &e);
  if (st != GMMFR_OK) return st;
  const void* kernel = nullptr;
  with(out, fp8, [&](auto out_, auto fp8_) {
    kernel = (const void*)dequant_kernel<decltype(out_)::value, decltype(fp8_)::value>;
  });
  return in_launches(kernel, (p.chunks + kThreads * kPer - 1) / (kThreads * kPer), p, stream);
}

}  // namespace gmmmq

extern "C" {

int gmm_mx_quantize(const gmmmq_args* args, void* stream) { return gmmmq::quantize(args, stream); }
int gmm_mx_dequantize(const gmmmq_args* args, void* stream) { return gmmmq::dequantize(args, stream); }

}  // extern "C"
