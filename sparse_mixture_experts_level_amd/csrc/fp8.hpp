// 8-bit floating point with a scale for each block of 128 values (gfx950): codes, scales and layouts.
//
// Codes are e4m3 (sign, 4 exponent, 3 mantissa bits; largest 448, one NaN, no infinity).  Scales are
// powers of two held as a byte, exponent + 127: the matrix instructions multiply their operands
// by such bytes themselves, so that a block's scale costs no instruction of its own.  A float
// scale would cost an fma per accumulator and 128 of K, about half of the matrix
// instructions' own time.
//
// Rows: codes [rows, fp8_row_bytes(K)] with zeros behind K, scales [rows, fp8_scale_bytes(K)], one byte
// per 128 columns; the bytes behind the last block are padding (to a multiple of four, so that four
// blocks' scales are one aligned load) and are not looked at.
// Weights of a group, [N, K]: blocks of 16 rows x 128 of K, 2 KB each, in the order [N / 16][K / 128];
// within a block the 16 bytes k = 64 p + 16 c .. + 15 of row r stand at 1024 p + 256 c + 16 r, which
// is the matrix instructions' operand layout: a wave's load of half a block is 1 KB of consecutive
// bytes.  gate_up matrices alternate blocks of gate rows and of the matching up rows.  Scales
// [N / 128][fp8_scale_bytes(K)] (gate_up: [f / 128][2][...], gate then up).
#pragma once

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

constexpr int kFp8Tile = 2048;  // bytes of a 16 x 128 block of weights

// |v| where it is finite, else 0: values that are not finite have no part in a block's scale.
__device__ __forceinline__ float fp8_magnitude(float v) {
  const float a = fabsf(v);
  return a < __builtin_inff() ? a : 0.0f;
}

// The scale's byte for the largest finite magnitude: the least exponent e >= -126 with amax <= 448 2^e
// (448 = 1.75 * 2^8); 127 (one) for a block of zeros.
__device__ __forceinline__ uint32_t fp8_scale_byte(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return b == 0u ? 127u : (uint32_t)max(e, 1);
}
// 2^-(exponent) of a byte that fp8_scale_byte() gave (1 .. 247): exact, a normal float.
__device__ __forceinline__ float fp8_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Codes of four values, lowest byte first: the nearest, ties to even; values that are not finite
// have the NaN code.
__device__ __forceinline__ uint32_t fp8_codes(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

typedef int i32x8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ i32x8 fp8_operand(u32x4 lo, u32x4 hi) {
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}
// c + (A 2^sa) (B 2^sb), 16 x 16 over 128 of K, the scales byte J of sa and sb.  Lane l holds row l % 16
// of each operand, k = 16 (l / 16) .. + 15 and 64 + 16 (l / 16) .. + 15 (any order shared by the two
// operands gives the same sum); c: columns (of B) l % 16, rows (of A) 4 (l / 16) .. + 3.
// Within a lane's 16 products the instruction drops what lies about 2^-14 below the largest
// of them; the accumulator is a full float.  Against 64 bits the sums of Gaussian rows are off by 1.2e-5 to
// 1.6e-5 of their size, over any length: a hundredth of the bf16 rounding that follows.
template <int J>
__device__ __forceinline__ f32x4 mfma_fp8_16(i32x8 a, i32x8 b, f32x4 c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, J, (int)sa, J, (int)sb);
}

}  // namespace moe
