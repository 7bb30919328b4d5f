// dequant_pairs.cuh -- decoding of packed fields on the FMA and integer pipes,
// two values per instruction.
#pragma once
#include "dequant.cuh"
#include "tc.cuh"

namespace qwm {

using tc::f2pack;

// Residual decode without an int-to-float conversion: for the code c of
// position i (0..3) of a code byte shifted to bits 15..22, OR-ing the masked
// bits into 1.0f gives exactly 1 + c 2^(2i-8); with S_i = sc 2^(8-2i) and
// M_i = mn - S_i one fma then yields mn + c sc (S_i is exact, and M_i is exact
// whenever mn and S_i lie within 2^13 of each other).  Pairs of positions share
// one f32x2 fma; the centroid is added with one f32x2 add.
struct GroupConst {
  uint64_t s01, s23, m01, m23;  // {S_0, S_1}, {S_2, S_3}, {M_0, M_1}, {M_2, M_3}
};

// binary16 -> fp32 on the FMA and integer pipes (the conversion unit is left to
// the softmax's exponentials): the 15 magnitude bits moved to the fp32
// exponent/mantissa position give 2^-112 times the value, normals and
// subnormals alike, so one exact multiply by 2^112 restores it.
__device__ __forceinline__ float half_bits_to_f32(uint32_t h) {
  const float m = __uint_as_float((h & 0x7fffu) << 13) * 0x1p112f;
  return __uint_as_float(__float_as_uint(m) | ((h & 0x8000u) << 16));
}

// int8 -> fp32 without a conversion instruction: adding c to the bit pattern of
// 1.5 * 2^23 gives 1.5 * 2^23 + c exactly (|c| < 2^22).
__device__ __forceinline__ float i8_to_f32(int c) {
  return __uint_as_float(0x4B400000u + (uint32_t)c) - 12582912.0f;
}

__device__ __forceinline__ GroupConst group_const(uint32_t par) {
  const float mn = half_bits_to_f32(par & 0xffffu), sc = half_bits_to_f32(par >> 16);
  const float s0 = sc * 256.0f, s1 = sc * 64.0f, s2 = sc * 16.0f, s3 = sc * 4.0f;
  GroupConst g;
  g.s01 = f2pack(s0, s1);
  g.s23 = f2pack(s2, s3);
  g.m01 = f2pack(__fsub_rn(mn, s0), __fsub_rn(mn, s1));
  g.m23 = f2pack(__fsub_rn(mn, s2), __fsub_rn(mn, s3));
  return g;
}

__device__ __forceinline__ float magic_code(uint32_t x, int i) {
  return __uint_as_float((x & (3u << (15 + 2 * i))) | 0x3F800000u);
}

}  // namespace qwm
