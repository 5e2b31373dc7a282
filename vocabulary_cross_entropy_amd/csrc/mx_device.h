// Microscaled (MX) number formats of libvce: blocks of 32 values share one
// power-of-two scale, stored as a biased exponent byte (E8M0: byte b stands
// for 2^(b - 127), 255 for NaN).
//   E4M3: sign, 4 exponent bits (bias 7), 3 mantissa bits; largest value 448
//   E2M1: sign, 2 exponent bits (bias 1), 1 mantissa bit; 0 .5 1 1.5 2 3 4 6
// The scale of a block is the least power of two s with amax <= Vmax s, so no
// element is clipped and each is rounded (to nearest even) by at most half a
// step of its grid.
#pragma once

#include "vce_device.h"

namespace vce {

constexpr int kMxE4M3 = 0;
constexpr int kMxE2M1 = 1;
constexpr int kMxBlock = 32;

typedef int16_t i16x2_t __attribute__((ext_vector_type(2)));

// |x| as ordered bits: compares like the magnitude, infinities and NaN last.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Scale byte of a block from the largest magnitude's bits.  With amax =
// 1.f * 2^E the least s is 2^(E - 8) while 1.f <= 1.75 (448 = 1.75 * 2^8), or
// 2^(E - 2) while 1.f <= 1.5 (6 = 1.5 * 2^2), else twice that.  Zero and FP32
// denormals land on the least scale, 2^-127; a block holding an infinity or a
// NaN has no scale and is marked NaN.
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255u;
  const int e = (int)(amax_bits >> 23);
  const uint32_t f = amax_bits & 0x7fffffu;
  const int b = FMT == kMxE4M3 ? e - 8 + (f > 0x600000u ? 1 : 0) : e - 2 + (f > 0x400000u ? 1 : 0);
  return (uint32_t)(b < 0 ? 0 : b);
}

// The scale as FP32 (2^-127 is a denormal: bits 0x00400000).  Not for 255.
__device__ __forceinline__ float mx_scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
}

// Four values over the scale, rounded to nearest even, as four E4M3 bytes;
// eight as eight E2M1 nibbles (first value in the low nibble).  The block's
// scale keeps every quotient within the format's range.
__device__ __forceinline__ uint32_t mx_pack4_e4m3(const float* v, float s) {
  i16x2_t r = {0, 0};
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, v[0], v[1], s, false);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, v[2], v[3], s, true);
  return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ uint32_t mx_pack8_e2m1(const float* v, float s) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], s, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], s, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], s, 3);
  return r;
}
__device__ __forceinline__ uint32_t mx_pack4_e2m1(const float* v, float s) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], s, 1);
  return r & 0xffffu;
}

// Quantises one block spread over the wavefront: lane holds VE consecutive
// values of it (VE = 8: 4 lanes per block, 4: 8 lanes, 1: 32 lanes) and
// writes its bytes to q and, from the block's first lane, the scale byte.
// `e` is the lane's first element in the row, a row's bytes start at q and
// s.  Every lane of a block must be active; `ok` false only skips the stores.
template <int FMT, int VE>
__device__ __forceinline__ void mx_store_block(const float* v, int64_t e, uint8_t* q, uint8_t* s,
                                               bool ok) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < VE; ++i) {
    const uint32_t b = abs_bits(v[i]);
    a = a > b ? a : b;
  }
#pragma unroll
  for (int off = 1; off < kMxBlock / VE; off <<= 1) {
    const uint32_t b = (uint32_t)__shfl_xor((int)a, off, 64);
    a = a > b ? a : b;
  }
  const uint32_t byte = mx_scale_byte<FMT>(a);
  const bool bad = byte == 255u;
  const float sc = mx_scale_value(bad ? 127u : byte);
  if (ok && e % kMxBlock == 0) s[e / kMxBlock] = (uint8_t)byte;
  if constexpr (FMT == kMxE4M3) {
    if constexpr (VE == 8) {
      const u32x2_t w = {mx_pack4_e4m3(v, sc), mx_pack4_e4m3(v + 4, sc)};
      if (ok) *reinterpret_cast<u32x2_t*>(q + e) = bad ? u32x2_t{0, 0} : w;
    } else if constexpr (VE == 4) {
      const uint32_t w = mx_pack4_e4m3(v, sc);
      if (ok) *reinterpret_cast<uint32_t*>(q + e) = bad ? 0u : w;
    } else {
      const float t[4] = {v[0], 0.0f, 0.0f, 0.0f};
      const uint32_t w = mx_pack4_e4m3(t, sc);
      if (ok) q[e] = bad ? (uint8_t)0 : (uint8_t)w;
    }
  } else {
    if constexpr (VE == 8) {
      const uint32_t w = mx_pack8_e2m1(v, sc);
      if (ok) *reinterpret_cast<uint32_t*>(q + e / 2) = bad ? 0u : w;
    } else if constexpr (VE == 4) {
      const uint32_t w = mx_pack4_e2m1(v, sc);
      if (ok) *reinterpret_cast<uint16_t*>(q + e / 2) = bad ? (uint16_t)0 : (uint16_t)w;
    } else {
      const float hi = __shfl_xor(v[0], 1, 64);  // the odd element of an even lane's pair
      const float t[4] = {v[0], hi, 0.0f, 0.0f};
      const uint32_t w = mx_pack4_e2m1(t, sc);
      if (ok && e % 2 == 0) q[e / 2] = bad ? (uint8_t)0 : (uint8_t)w;
    }
  }
}

}  // namespace vce
