// Rows of a cache held in 4 bits: codes of all the row's elements, two a byte, then a scale byte for every
// 32 of them, rounded up to 16 bytes.
//
//   value = sign * {0, 0.5, 1, 1.5, 2, 3, 4, 6}[code] * 2^(scale - 127)
//
// The conversions are the hardware's: eight codes of a dword become eight 16-bit elements in four
// instructions, exactly where the type holds the value (all scales and codes compared on the device:
// bf16 and fp16, subnormals included, infinite past the type's range, NaN for scale 255), and fp32 values become codes
// rounded to nearest, halves to even, above 6 to 6.
#pragma once

#include <stdint.h>

namespace hc {

constexpr int kMxBlock = 32;  // elements of a scale

// Bytes of a row's codes, where its scales begin, and of the whole row.
constexpr int64_t mxfp4_codes(int64_t elems) { return elems / 2; }
constexpr int64_t mxfp4_row(int64_t elems) { return (elems / 2 + elems / kMxBlock + 15) / 16 * 16; }

#if defined(__HIP_DEVICE_COMPILE__) || defined(__HIPCC__)
typedef unsigned int mx_v4u __attribute__((ext_vector_type(4)));
typedef __bf16 mx_bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 mx_f16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float mx_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight codes as elements, in 16 bytes.
template <bool BF16>
__device__ __forceinline__ mx_v4u mx_decode(uint32_t codes, float scale) {
  mx_v4u y;
#define HC_MX_PAIR(i)                                                                                           \
  if constexpr (BF16)                                                                                           \
    y[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, i));             \
  else                                                                                                          \
    y[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, i));
  HC_MX_PAIR(0) HC_MX_PAIR(1) HC_MX_PAIR(2) HC_MX_PAIR(3)
#undef HC_MX_PAIR
  return y;
}

// The scale byte of a block whose largest magnitude has these bits: 2^e with largest <= 7 * 2^e = 1.75 * 2^(e + 2).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
  if (top >= 0x7f800000u) return 255;                      // infinity or NaN
  const int e = (int)((top + 0x1fffffu) >> 23) - 2;         // the carry: a mantissa above 1.75
  return e < 0 ? 0 : (uint32_t)e;
}

// A double as an fp32 value between the same two 4-bit borders.  Borders (between codes, and of a block's scale) have
// three bits; rounded to 24, a value can come to lie on one that it was next to, and is then put back.  (Below 2^-126, where
// the least scale has its borders, fp32's step is 2^-149 and the lowest border 2^-129, bit 20.  What has only bits from there on
// and is no border may be put back as well: it stays between the same two.)
__device__ __forceinline__ float mx_beside(double x) {
  const float y = (float)x;
  uint32_t u = __float_as_uint(y);
  if ((u & 0xfffffu) == 0 && (double)y != x && u << 1 < 0xff000000u) u += fabs((double)y) > fabs(x) ? -1 : 1;
  return __uint_as_float(u);
}

// Elements before their rounding by a scale so large that its codes go past the element type: 4 * 2^14 is 2^16, which fp16 does not
// hold, though it holds elements up to 65504 that round to it.  An element below the power of two behind the type's
// largest value (2^16, and of bf16 any that is finite) is held down to the largest code that the type holds:
// 3 * 2^14, 1.5 * 2^15, 0.5 * 2^16 and none from 2^17 on, of bf16 3 * 2^126.  Scales above 2^14 and elements from 2^16
// on are rotated keys', which fp16 has no number for.  (Holding elements down where rows are read would be nearer,
// 65504 for 65536, at the price of more instructions on every element of every attention.)
template <bool BF16>
__device__ __forceinline__ void mx_hold(float* x, uint32_t scale_byte) {
  if (scale_byte <= (BF16 ? 252u : 140u)) return;
  const float behind = BF16 ? INFINITY : 0x1p16f;
  const float most = BF16 ? 0x1.8p127f : scale_byte <= 142 ? 0x1.8p15f : scale_byte == 143 ? 0x1p15f : 0.f;
  for (int j = 0; j < 8; j++)
    if (fabsf(x[j]) < behind) x[j] = copysignf(fminf(fabsf(x[j]), most), x[j]);
}

__device__ __forceinline__ uint32_t mx_encode(const float* x, float scale) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], scale, 3);
}
#endif

}  // namespace hc
