// Rows and weights between bf16 or float and 8 bits with scales (layouts in fp8.hpp).
//
// Memory bound, and off the path of a forward pass but for the rows: x is quantised once for all experts.  16384 x 7168 of bf16
// 60 us (5.9 TB/s), weights of 32 x 5760 x 2880 from bf16 288 us (5.5).
#include "fp8.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  if constexpr (sizeof(T) == 2)
    return bf16_to_f32(v);
  else
    return v;
}

// One block of 128 columns by 16 lanes of eight columns each; four blocks of a row a wave, one after the
// other over the row and the rows.
template <typename T>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const T *__restrict__ x, int64_t rows, int K,
                                                            uint8_t *__restrict__ codes, uint8_t *__restrict__ scale) {
  const int blocks = fp8_blocks(K), row_bytes = fp8_row_bytes(K), scale_bytes = fp8_scale_bytes(K);
  const int l = threadIdx.x & 15;
  const int64_t n = rows * scale_bytes;  // padding scales are written too, as ones
  for (int64_t q = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 4; q < n; q += (int64_t)gridDim.x * 16) {
    const int64_t row = q / scale_bytes;
    const int b = (int)(q - row * scale_bytes), c0 = b * kFp8Block + l * 8;
    float v[8], top = 0.0f;
    load8<T, false>(x + row * K + c0, K - c0, K).to(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fp8_magnitude(v[i]));
    top = group_reduce<16>(top, [](float a, float b) { return fmaxf(a, b); });
    const uint32_t byte = fp8_scale_byte(top);
    const float inv = fp8_inverse(byte);
    if (b < blocks) {
      uint2 w;
      w.x = fp8_codes(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
      w.y = fp8_codes(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
      *reinterpret_cast<uint2 *>(codes + row * row_bytes + c0) = w;
    }
    if (l == 0) scale[q] = (uint8_t)byte;
  }
}

// The values that codes stand for.
template <typename T>
__global__ __launch_bounds__(256) void dequantize_rows_kernel(const uint8_t *__restrict__ codes,
                                                              const uint8_t *__restrict__ scale, int64_t rows, int K,
                                                              T *__restrict__ out) {
  const int row_bytes = fp8_row_bytes(K), scale_bytes = fp8_scale_bytes(K), pieces = row_bytes / 8;
  const int64_t n = rows * pieces;
  for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < n; q += (int64_t)gridDim.x * 256) {
    const int64_t row = q / pieces;
    const int c0 = (int)(q - row * pieces) * 8;
    const uint2 w = *reinterpret_cast<const uint2 *>(codes + row * row_bytes + c0);
    const int e = (int)scale[row * scale_bytes + c0 / kFp8Block] - 127;
    const float v[8] = {__builtin_amdgcn_cvt_f32_fp8((int)w.x, 0), __builtin_amdgcn_cvt_f32_fp8((int)w.x, 1),
                        __builtin_amdgcn_cvt_f32_fp8((int)w.x, 2), __builtin_amdgcn_cvt_f32_fp8((int)w.x, 3),
                        __builtin_amdgcn_cvt_f32_fp8((int)w.y, 0), __builtin_amdgcn_cvt_f32_fp8((int)w.y, 1),
                        __builtin_amdgcn_cvt_f32_fp8((int)w.y, 2), __builtin_amdgcn_cvt_f32_fp8((int)w.y, 3)};
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = e == 128 ? __builtin_nanf("") : ldexpf(v[i], e);
    store8<T, false>(out + row * K + c0, K - c0, o);
  }
}

// One 128 x 128 block of one group's matrix a workgroup.  With swiglu the matrix is [2 n_out, K], gate rows
// then up rows, and blocks alternate gate and up (each of its own n_out rows).
template <typename T>
__global__ __launch_bounds__(256) void quantize_weights_kernel(const T *__restrict__ w, int n_out, int K, int swiglu,
                                                               uint8_t *__restrict__ codes,
                                                               uint8_t *__restrict__ scale) {
  __shared__ float part[4];
  __shared__ __attribute__((aligned(16))) uint8_t tile[128 * 128];
  const int kt = fp8_blocks(K), nt = (n_out + 15) / 16, halves = swiglu ? 2 : 1;
  const int block = __builtin_amdgcn_readfirstlane((int)blockIdx.x / kt), kb = (int)blockIdx.x - block * kt;
  const int nb = __builtin_amdgcn_readfirstlane(block / halves), half = block - nb * halves;
  const int64_t g = blockIdx.y;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const T *m = w + (g * halves + half) * (int64_t)n_out * K;
  // this wave's 32 rows; past the matrix zeros (range-checked loads: behind a branch each they would go one at a time)
  const int first = nb * 128 + wave * 32, rows = __builtin_amdgcn_readfirstlane(max(0, min(32, n_out - first)));
  const rsrc_t from = make_rsrc(m + (int64_t)first * K, (uint32_t)rows * (uint32_t)K * (uint32_t)sizeof(T));
  float v[32][2], top = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = kb * 128 + h * 64 + lane;
      const uint32_t at = c < K ? ((uint32_t)(i * K + c)) * (uint32_t)sizeof(T) : kOob;
      if constexpr (sizeof(T) == 4)
        v[i][h] = __builtin_bit_cast(float, (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(from, at, 0, 0));
      else
        v[i][h] = to_f32((T)__builtin_amdgcn_raw_buffer_load_b16(from, at, 0, 0));
    }
  }
#pragma unroll
  for (int i = 0; i < 32; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) top = fmaxf(top, fp8_magnitude(v[i][h]));
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  if (lane == 0) part[wave] = top;
  __syncthreads();
  top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  const uint32_t byte = fp8_scale_byte(top);
  const float inv = fp8_inverse(byte);
#pragma unroll
  for (int i = 0; i < 32; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      tile[(wave * 32 + i) * 128 + h * 64 + lane] =
          (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[i][h] * inv, 0.0f, 0, false);
  __syncthreads();
  // 16-byte pieces of the eight blocks of 16 rows: piece q holds row q % 16 of block q / 128
  for (int q = threadIdx.x; q < 1024; q += 256) {
    const int blk = q >> 7, pc = (q >> 4) & 7, r = q & 15, t = nb * 8 + blk;
    if (t >= nt) continue;
    uint32_t step;
    const uint32_t at = fp8_block_offset(t * halves + half, nt * halves, kt, step);
    uint8_t *o = codes + g * fp8_group_bytes(n_out, K, swiglu != 0) + at + (int64_t)(kb * 2 + (pc >> 2)) * step;
    *reinterpret_cast<u32x4 *>(o + (pc & 3) * 256 + r * 16) =
        *reinterpret_cast<const u32x4 *>(tile + (blk * 16 + r) * 128 + pc * 16);
  }
  uint8_t *so = scale + ((g * fp8_blocks(n_out) + nb) * halves + half) * (int64_t)fp8_scale_bytes(K);
  if (threadIdx.x == 0) so[kb] = (uint8_t)byte;
  // the padding bytes, by the last block's workgroup
  if (kb == kt - 1 && (int)threadIdx.x < fp8_scale_bytes(K) - kt) so[kt + threadIdx.x] = 127;
}

}  // namespace

hipError_t launch_quantize_rows(const void *x, bool f32, int64_t rows, int K, uint8_t *codes, uint8_t *scale,
                                hipStream_t s) {
  const int64_t n = rows * fp8_scale_bytes(K);
  if (n == 0) return hipSuccess;
  const unsigned grid = (unsigned)((n + 15) / 16 < 16384 ? (n + 15) / 16 : 16384);
  if (f32)
    hipLaunchKernelGGL(quantize_rows_kernel<float>, dim3(grid), dim3(256), 0, s, static_cast<const float *>(x), rows, K,
                       codes, scale);
  else
    hipLaunchKernelGGL(quantize_rows_kernel<bf16_t>, dim3(grid), dim3(256), 0, s, static_cast<const bf16_t *>(x), rows,
                       K, codes, scale);
  return hipGetLastError();
}

hipError_t launch_dequantize_rows(const uint8_t *codes, const uint8_t *scale, int64_t rows, int K, void *out, bool f32,
                                  hipStream_t s) {
  const int64_t n = (rows * (fp8_row_bytes(K) / 8) + 255) / 256;
  if (n == 0) return hipSuccess;
  const unsigned grid = (unsigned)(n < 16384 ? n : 16384);
  if (f32)
    hipLaunchKernelGGL(dequantize_rows_kernel<float>, dim3(grid), dim3(256), 0, s, codes, scale, rows, K,
                       static_cast<float *>(out));
  else
    hipLaunchKernelGGL(dequantize_rows_kernel<bf16_t>, dim3(grid), dim3(256), 0, s, codes, scale, rows, K,
                       static_cast<bf16_t *>(out));
  return hipGetLastError();
}

int64_t fp8_weights_bytes(int n_out, int K, bool swiglu) { return fp8_group_bytes(n_out, K, swiglu); }
int64_t fp8_weight_scales_bytes(int n_out, int K, bool swiglu) {
  return (int64_t)fp8_blocks(n_out) * (swiglu ? 2 : 1) * fp8_scale_bytes(K);
}

hipError_t launch_quantize_weights(const void *w, bool f32, int G, int n_out, int K, bool swiglu, uint8_t *codes,
                                   uint8_t *scale, hipStream_t s) {
  // (a group's blocks of 16 KB are below 2^17, as its codes are below 2 GiB)
  const dim3 grid((unsigned)(fp8_blocks(n_out) * (swiglu ? 2 : 1)) * (unsigned)fp8_blocks(K), (unsigned)G);
  if (f32)
    hipLaunchKernelGGL(quantize_weights_kernel<float>, grid, dim3(256), 0, s, static_cast<const float *>(w), n_out, K,
                       swiglu ? 1 : 0, codes, scale);
  else
    hipLaunchKernelGGL(quantize_weights_kernel<bf16_t>, grid, dim3(256), 0, s, static_cast<const bf16_t *>(w), n_out, K,
                       swiglu ? 1 : 0, codes, scale);
  return hipGetLastError();
}

}  // namespace moe
