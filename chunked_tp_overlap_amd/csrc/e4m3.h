// fp32 -> OCP E4M3 with saturation, as quantize_fp8.hip uses it.  kv_append.hip gives the same codes
// by the hardware's conversion, which the tests compare with this one for every bf16 value.
//
//   e4m3(y) = sat(RNE_e4m3(y)): the nearest OCP E4M3 value (bias 7, 3 significand bits,
//   subnormal spacing 2^-9), ties to even; magnitudes beyond 448 (and infinities) saturate
//   to 448; NaN stays NaN (0x7F with its sign); zeros keep their sign.
//
// The rounding is done on the fp32 bits with integer operations, so it is exactly that
// definition for every input.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ubx {
namespace {

__device__ inline uint32_t e4m3(float y) {
  const uint32_t u = __float_as_uint(y);
  const uint32_t sign = (u >> 24) & 0x80u;
  const uint32_t a = u & 0x7FFFFFFFu;
  if (a > 0x7F800000u) return sign | 0x7Fu;                 // NaN
  if (a >= 0x43E00000u) return sign | 0x7Eu;                // >= 448 (and inf): saturate
  if (a >= 0x3C800000u) {                                   // >= 2^-6: normal E4M3
    // round the 23-bit fp32 significand to 3 bits, ties to even (a carry moves the
    // exponent up), then rebias the exponent from 127 to 7
    const uint32_t r = (a + 0x7FFFFu + ((a >> 20) & 1u)) >> 20;
    return sign | (r - (120u << 3));
  }
  // subnormal range: multiples of 2^-9 (8 * 2^-9 = 2^-6 is code 0x08, the smallest normal)
  return sign | (uint32_t)__builtin_rintf(__uint_as_float(a) * 512.0f);
}

}  // namespace
}  // namespace ubx
