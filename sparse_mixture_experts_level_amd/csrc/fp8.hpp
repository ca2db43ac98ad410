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
// Weights of a group, [N, K]: blocks of 16 rows (gate_up matrices alternate blocks of gate rows and of the
// matching up rows), tiles of 16 blocks (the last has what is left, b <= 16), and in a tile the pieces
// [K / 128][2][b] of 1 KB: 16 rows x 64 of K as [4 chunks of 16 codes][16 rows], the matrix instructions' operand layout.
// So a wave's load is 1 KB of consecutive bytes, and a workgroup of 256 rows walks one region of memory, 32 KB a step,
// whatever K is: with each block's K on its own, workgroups in step read addresses a power of two
// apart for such K, on few memory channels.  Scales [N / 128][fp8_scale_bytes(K)] (gate_up: [f / 128][2][...],
// gate then up).
#pragma once

#include "common.hpp"
#include "kernels.hpp"
#include "lanes.hpp"

namespace moe {

constexpr int kFp8Tile = 2048;  // bytes of 16 x 128 codes

// Eight consecutive values of a row of d as they are held, loaded and stored as 16-byte pieces at any alignment of the
// element's own size (the vector memory path takes unaligned addresses).  `n` of them exist (n <= 0: none; the
// rest count as zeros and are not stored); WHOLE: rows are whole vectors, n is at least eight or
// at most zero.  A row's last n < 8 are loaded one by one, each behind a branch and its own wait, or (BACK) as the
// row's last eight, which front() moves to their places once all loads are under way.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
template <typename T>
struct Raw8 {
  u32x4 v[sizeof(T) / 2];
  __device__ __forceinline__ void to(float *f) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 2)
        f[i] = __uint_as_float(i % 2 ? v[0][i / 2] & 0xffff0000u : v[0][i / 2] << 16);
      else
        f[i] = __uint_as_float(v[i / 4][i % 4]);
    }
  }
  __device__ __forceinline__ void front(int n) {
    static_assert(sizeof(T) == 2, "of bf16");
    if (n <= 0 || n >= 8) return;
    const int by = 8 - n;
#pragma unroll
    for (int o = 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (by / 2 & o) v[0][i] = i + o < 4 ? v[0][(i + o) % 4] : 0u;
    if (by % 2)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[0][i] = v[0][i] >> 16 | (i < 3 ? v[0][(i + 1) % 4] << 16 : 0u);
  }
};
template <typename T, bool WHOLE, bool BACK = false>
__device__ __forceinline__ Raw8<T> load8(const T *p, int n, int d) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = u32x4{0u, 0u, 0u, 0u};
  if (n >= 8 || (BACK && n > 0 && d >= 8)) {
    const T *q = BACK ? p + min(n - 8, 0) : p;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = reinterpret_cast<const u32x4_any *>(q)[i];
  } else if (!WHOLE && n > 0) {
    const int by = BACK ? 8 - n : 0;
    T t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = i >= by && i - by < n ? p[i - by] : T(0);
    __builtin_memcpy(r.v, t, sizeof t);
  }
  return r;
}
template <typename T, bool WHOLE>
__device__ __forceinline__ void store8(T *p, int n, const float *f) {
  if (n >= 8) {
    u32x4 v[sizeof(T) / 2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) {
        v[0][i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
      } else {
        v[0][i] = __float_as_uint(f[i]);
        v[1][i] = __float_as_uint(f[4 + i]);
      }
    }
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<u32x4_any *>(p)[i] = v[i];
  } else if (!WHOLE && n > 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) store_out(p + i, f[i]);
  }
}

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

// 4 bytes per lane from a buffer straight into LDS, as buf_ld16_lds.
__device__ __forceinline__ void buf_ld4_lds(rsrc_t r, uint32_t off, void *lds_wave_base) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)lds_wave_base, 4, off, 0, 0, 0);
}

// A word at an address that is the same in every lane, by the scalar unit (the compiler takes the vector path for memory
// that it cannot prove unwritten).
__device__ __forceinline__ uint32_t scalar_load(const uint8_t *p) {
  return *reinterpret_cast<const __attribute__((address_space(4))) uint32_t *>(reinterpret_cast<uintptr_t>(p));
}

// What a group has of the rows, clamped to the buffers.
__device__ __forceinline__ void fp8_group_rows(const Fp8GemmArgs &a, int g, int &begin, int &end) {
  begin = min(max(a.offsets[g], 0), a.rows_max);
  end = min(max(a.offsets[g + 1], begin), a.rows_max);
}
// The same for a group that is the same in every lane, in scalar registers, with all that derives from it (the compiler does
// not see that the offsets stay as they are, and runs a loop over the lanes around every buffer load).
__device__ __forceinline__ void fp8_group_rows_uniform(const Fp8GemmArgs &a, int g, int &begin, int &end) {
  fp8_group_rows(a, g, begin, end);
  begin = __builtin_amdgcn_readfirstlane(begin);
  end = __builtin_amdgcn_readfirstlane(end);
}
// The n-th group (from 0) of more than 0 and at most `most` rows and its rows, in scalar registers; -1: there are not that
// many.  A launch has as many workgroups as groups can have rows, not as there are groups: one of an empty group holds its
// CU until it has read the offsets.
__device__ __forceinline__ int fp8_nth_group(const Fp8GemmArgs &a, int n, int most, int &begin, int &end) {
  const int lane = threadIdx.x & 63;
  int seen = 0;
#pragma unroll 1
  for (int g0 = 0; g0 < a.num_groups; g0 += 64) {
    int b = 0, e = 0;
    if (g0 + lane < a.num_groups) fp8_group_rows(a, g0 + lane, b, e);
    const uint64_t some = __ballot(e > b && e - b <= most);
    const int count = __popcll(some);
    if (n < seen + count) {
      const bool mine = (some >> lane & 1) && __popcll(some & ((1ull << lane) - 1)) == n - seen;
      const int l = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)__ballot(mine)) - 1);
      begin = __builtin_amdgcn_readlane(b, l);
      end = __builtin_amdgcn_readlane(e, l);
      return g0 + l;
    }
    seen += count;
  }
  return -1;
}
// Where a block's piece (k step 0, first half) stands in its group, and the distance from half a step to the next.
__device__ __forceinline__ uint32_t fp8_block_offset(int block, int blocks, int kt, uint32_t &half) {
  const int tile = block / 16;
  half = (uint32_t)min(16, blocks - tile * 16) * 1024u;
  return (uint32_t)(tile * 16 * kt) * 2048u + (uint32_t)(block % 16) * 1024u;
}
// Bytes of one group's codes.
__host__ __device__ __forceinline__ int64_t fp8_group_bytes(int n_out, int k, bool swiglu) {
  return (int64_t)((n_out + 15) / 16) * (swiglu ? 2 : 1) * fp8_blocks(k) * kFp8Tile;
}

// c + (A 2^sa) (B 2^sb), 16 x 16 over 128 of K, the scales byte J of sa and sb.  Lane l holds row l % 16
// of each operand, k = 16 (l / 16) .. + 15 and 64 + 16 (l / 16) .. + 15 (any order shared by the two
// operands gives the same sum); c: columns (of B) l % 16, rows (of A) 4 (l / 16) .. + 3.
// Within a lane's 16 products the instruction drops what lies about 2^-14 below the largest
// of them; the accumulator is a full float.  Against 64 bits the sums of Gaussian rows are off by 1.2e-5 to
// 1.6e-5 of their size, over any length: a hundredth of a bf16 rounding, but codes of H, formed from such sums, move over
// a border one in two thousand (2 x 80 rows, 7168 x 2048: the FFN's error 1.92e-3 of its norm for 1.66e-3).  The bf16
// instruction has no such loss, at half the rate: the choice for many rows is speed.
template <int J>
__device__ __forceinline__ f32x4 mfma_fp8_16(i32x8 a, i32x8 b, f32x4 c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, J, (int)sa, J, (int)sb);
}

// Eight codes as bf16, times 2^e for a scale given as a float, of which the instruction takes the exponent field f alone: e is
// f - 127, 0 (e = -127) and 254 too, and 255 makes every value NaN.  Exact for f from 3 to 246: below, codes of 2^-9 and up fall
// under bf16's least step of 2^-133; above, those up to 448 pass its range and become infinite.
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u32x4 fp8_to_bf16(uint32_t lo, uint32_t hi, float scale) {
  return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true))};
}
// Such fields, as floats, for products of a row's block and of one or two weight blocks (`w0`, `w1`) whose scale bytes are
// byte J of those given: the weights' exponents less `shift`, the row's that much more.  The row's byte may be any, and
// no shift of its own is possible (a weight meets all rows), so that up to 8 of the weights' exponent, towards zero, goes to
// the rows: with it both factors are in the conversion's exact range wherever row's and weights' exponents together are from -121
// to 119 (checked for all bytes).  Past 119 a field of 255 gives NaN; below, products of less than 2^-103 lose bits.
template <int J>
__device__ __forceinline__ int fp8_shift(uint32_t w0, uint32_t w1) {
  const int a = (int)(w0 >> (8 * J) & 0xffu) - 127, b = (int)(w1 >> (8 * J) & 0xffu) - 127;
  return min(min(max(max(a, b), -8), 8), min(a, b) + 121);
}
template <int J>
__device__ __forceinline__ float fp8_shifted(uint32_t four, int by) {
  const int byte = (int)(four >> (8 * J) & 0xffu);
  return __uint_as_float((uint32_t)(byte == 255 ? 255 : min(max(byte + by, 0), 255)) << 23);
}

}  // namespace moe
