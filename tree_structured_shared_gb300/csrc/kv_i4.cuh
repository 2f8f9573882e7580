// The 4-bit pool's format: 16-token blocks of signed 4-bit codes with one
// scale per group of 16 head dims.
//
// One (block, kv head) is kI4Unit = 1152 contiguous bytes: 1024 of codes, 128
// of scales.  A 32-bit word holds eight consecutive dims, nibble j the dim 2j
// and nibble 4 + j the dim 2j + 1, so a masked shift leaves a natural pair of
// dims in the two halves of a register.  A code is n + 8 with n in [-7, 7]; a
// value is n * s.  K and V order their words differently, each so that the
// warp-level matrix instruction's fragments come from 16-byte loads that cover
// whole sectors:
//   K codes [4 chunks of 32 dims][16 slots][16 bytes]  scales [16 slots][8 groups]
//   V codes [8 groups of 16 dims][16 slots][8 bytes]   scales [8 groups][16 slots]
//
// A scale is one byte, bits 14..7 of an fp16 number (5 exponent and 3 mantissa
// bits, no sign): n has 3 significant bits and s has 4, so every value n * s
// is exact in fp16 (and bf16), and no second-level scale is needed for
// magnitudes from 2^-17 to 7 * 896.  Scales stop at 896 so that 72 * s, the
// offset of the decode below, stays finite in fp16.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>

#include "padoc_internal.h"

namespace padoc {

constexpr int kI4Unit = kI4UnitBytes;
constexpr int kI4Scales = 1024;   // offset of its scales
constexpr float kI4MaxScale = 896.f;
constexpr uint32_t kI4Nan = 0xFFu;  // scale byte of a poisoned group (an fp16 NaN)

// Scale byte of a group whose largest magnitude is 7 * a (a >= 0, finite): a rounded to
// three mantissa bits, ties to even; below 2^-14 in steps of 2^-17.
__device__ __forceinline__ uint32_t i4_scale_byte(float a) {
  a = fminf(a, kI4MaxScale);
  if (a < 6.103515625e-5f) return static_cast<uint32_t>(__float2int_rn(a * 131072.f));  // 8 is the smallest normal
  uint32_t b = __float_as_uint(a);
  b += 0x7FFFFu + ((b >> 20) & 1u);
  return (b >> 20) - (112u << 3);  // exponent bias 127 -> 15
}
__device__ __forceinline__ float i4_scale_value(uint32_t byte) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
}

// Two scale bytes as an fp16 pair: lo's in the low half.
__device__ __forceinline__ uint32_t i4_scale_pair(uint32_t lo, uint32_t hi) { return (lo << 7) | (hi << 23); }

__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// -72 s, the offset that i4_pair wants next to s.
__device__ __forceinline__ uint32_t i4_offset(uint32_t s2) { return h2_mul(s2, 0xD480D480u); }

// The pair of values in nibbles j and 4 + j of w.  The nibble in mantissa bits
// 7..4 of 64.0 makes 64 + n + 8; one fma takes (72 + n) s - 72 s = n s, exact
// (72 s has 7 significant bits, n s has 7).
template <int J>
__device__ __forceinline__ uint32_t i4_pair(uint32_t w, uint32_t s2, uint32_t off2) {
  const uint32_t x = J == 0 ? w << 4 : J == 1 ? w : J == 2 ? w >> 4 : w >> 8;
  return h2_fma((x & 0x00F000F0u) | 0x54005400u, s2, off2);
}

}  // namespace padoc
