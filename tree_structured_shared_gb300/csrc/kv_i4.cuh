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
// magnitudes from 2^-17 to 7 * 896.  Scales stop at 896 so that the decode's
// offsets below stay finite in fp16.
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
// Whether a is in [2^-14, 896): a normal scale, and not held at the limit; and
// such a scale itself, its byte in *byte.
__device__ __forceinline__ bool i4_plain(float a) { return __float_as_uint(a) - 0x38800000u < 0x44600000u - 0x38800000u; }
__device__ __forceinline__ float i4_plain_scale(float a, uint32_t* byte) {
  uint32_t b = __float_as_uint(a);
  b += 0x7FFFFu + ((b >> 20) & 1u);
  *byte = (b >> 20) - (112u << 3);
  return __uint_as_float(b & 0xFFF00000u);
}
__device__ __forceinline__ float i4_scale_value(uint32_t byte) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
}

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

// Decoding.  A nibble or-ed into the mantissa of a power of two makes that power
// plus n + 8 without a conversion: bits 3..0 of a half under 1024, bits 7..4
// under 64.  One fma then takes the bias off and the scale on,
//   (1032 + n) s' - 1032 s' = n s',   (72 + n) s' - 72 s' = n s',
// exact with s' = s / 16: 1032 s' has at most 11 significant bits (129 times a
// 4-bit mantissa) and stays below 65504 for every s up to 896, n s' has 7, and
// s' of the smallest s is still a multiple of 2^-21.  The factor 16 joins the
// softmax's scale (K) or the output's (V).  A word so costs one shift, four
// masks and four fmas; the integer pipe, half as wide as the others, is what the
// decode kernels fill first (three shifts a word: 60 % of its cycles in the own
// pass at 58 % issue).
constexpr float kI4Unscale = 16.f;
struct I4Scale {
  uint32_t s, lo, hi;  // s', -1032 s', -72 s', for the two halves of a register
};
// pair: two scale bytes in bits 7..0 and 23..16.
__device__ __forceinline__ I4Scale i4_scale(uint32_t pair) {
  const uint32_t h = pair * 128u;  // bits 14..7 of each half; a multiply, off the integer pipe
  return I4Scale{h2_mul(h, 0x2C002C00u), h2_mul(h, 0xD408D408u), h2_mul(h, 0xC480C480u)};
}
// Byte B of x for both halves of a register, or bytes B and B + 1 for one each.
template <int B>
__device__ __forceinline__ I4Scale i4_scale_both(uint32_t x) {
  return i4_scale(__byte_perm(x, 0u, 0x4040u | B | (B << 8)));
}
template <int B>
__device__ __forceinline__ I4Scale i4_scale_two(uint32_t x) {
  return i4_scale(__byte_perm(x, 0u, 0x4040u | B | ((B + 1) << 8)));
}
// (x & mask) | bits in one instruction.
__device__ __forceinline__ uint32_t mask_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(x), "r"(mask), "r"(bits));
  return d;
}
// n s' of nibbles J and 4 + J of w in the halves of a register, v = w >> 8.
template <int J>
__device__ __forceinline__ uint32_t i4_pair(uint32_t w, uint32_t v, const I4Scale& s) {
  const uint32_t x = J < 2 ? w : v;
  return (J & 1) ? h2_fma(mask_or(x, 0x00F000F0u, 0x54005400u), s.s, s.hi)
                 : h2_fma(mask_or(x, 0x000F000Fu, 0x64006400u), s.s, s.lo);
}

// x / G for x below 2^29 (g_inv = 2^32 / G rounded up; 0 for G = 1).
__device__ __forceinline__ int div_g(int x, uint32_t g_inv) {
  return g_inv ? static_cast<int>(__umulhi(static_cast<uint32_t>(x), g_inv)) : x;
}

}  // namespace padoc
