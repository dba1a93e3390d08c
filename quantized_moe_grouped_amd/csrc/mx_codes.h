// E8M0 block scales of the MX formats: a byte e stands for 2^(e - 127), 255 for NaN.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace gmmmq {

// E8M0 code of a block whose largest magnitude has the fp32 bits `mag`: the
// exponent field minus emax, at least 0; 255 when the block is not finite.
template <bool FP8>
__device__ __forceinline__ uint32_t scale_code(uint32_t mag) {
  const uint32_t e = mag >> 23, emax = FP8 ? 8 : 2;
  return e == 255 ? 255u : (e > emax ? e - emax : 0u);
}
// The power of two of an E8M0 code (0: 2^-127, a subnormal); NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t code) {
  return __uint_as_float(code == 255 ? 0x7FC00000u : (code ? code << 23 : 0x00400000u));
}

}  // namespace gmmmq
