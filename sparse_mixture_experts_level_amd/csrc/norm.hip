// Root-mean-square norm with the residual's addition and an 8-bit output, and its backward pass.
//
//   h = x + residual (rounded to the layer's type: it is what the residual stream carries on and what the
//   backward pass reads), rstd = 1 / sqrt(mean h^2 + eps), y = (h rstd) w
//   dx = dh + rstd (g - xhat mean(g xhat)),  g = dy w, xhat = h rstd;  dw = sum_t dy xhat
//
// Memory bound: a row is read once into registers, as vectors of eight values a thread, and
// written once.
#include <algorithm>

#include "fp8.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

// Eight consecutive values at any alignment of the element's own size (the vector memory path takes
// unaligned addresses); `n` of them exist, the rest read as zeros.
template <typename T>
__device__ __forceinline__ void load8(const T *p, int n, float *v) {
  T t[8];
  if (n >= 8) {
    __builtin_memcpy(t, p, sizeof t);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = i < n ? p[i] : T(0);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 2)
      v[i] = bf16_to_f32(t[i]);
    else
      v[i] = t[i];
  }
}

template <typename T>
__device__ __forceinline__ void store8(T *p, int n, const float *v) {
  T t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) store_out(&t[i], v[i]);
  if (n >= 8) {
    __builtin_memcpy(p, t, sizeof t);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = t[i];
  }
}

// The sum over the TPR threads that share a row, in every one of them; `part` has room for
// the waves of the workgroup.  TPR is 64 (one wave) or the whole workgroup.
template <typename V, int TPR>
__device__ __forceinline__ V row_sum(V v, V *part) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if constexpr (TPR > 64) {
    __syncthreads();  // the sums of the row before are read
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w) v += part[w];
  }
  return v;
}

// TPR threads a row, NV vectors of eight a thread: vector i of thread t at column 8 (t + i TPR).  The mean of
// squares is formed in 64 bits, and h rstd and its product with w are each rounded to float, so
// that the codes, which jump next to a border, are the same in any order of the sum.
template <typename T, int TPR, int NV>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void rms_norm_kernel(const NormCall c) {
  constexpr int RPB = TPR >= 256 ? 1 : 256 / TPR;
  __shared__ double part[TPR > 64 ? TPR / 64 : 1];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if (row >= c.T) return;  // whole waves, and whole workgroups where a barrier follows
  const int d = c.d;
  const T *x = static_cast<const T *>(c.x) + row * d;
  const T *res = c.residual ? static_cast<const T *>(c.residual) + row * d : nullptr;
  float h[NV][8];
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = 8 * (t + i * TPR), n = d - col;
    if (n <= 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = 0.0f;
      continue;
    }
    load8(x + col, n, h[i]);
    if (res) {
      float r[8];
      load8(res + col, n, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[i][j] += r[j];
        if constexpr (sizeof(T) == 2) h[i][j] = bf16_to_f32(f32_to_bf16(h[i][j]));
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += (double)h[i][j] * (double)h[i][j];
  }
  sum = row_sum<double, TPR>(sum, part);
  const float rstd = (float)(1.0 / sqrt(sum / (double)d + (double)c.eps));
  if (c.rstd && t == 0) c.rstd[row] = rstd;
  const int row_bytes = fp8_row_bytes(d), scale_bytes = fp8_scale_bytes(d);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = 8 * (t + i * TPR), n = d - col;
    float y[8];
    if (n > 0) {
      load8(static_cast<const T *>(c.weight) + col, n, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] *= h[i][j] * rstd;
      if (c.h) store8(static_cast<T *>(c.h) + row * d + col, n, h[i]);
      if (c.y) store8(static_cast<T *>(c.y) + row * d + col, n, y);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = 0.0f;
    }
    if (c.y8) {
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, fp8_magnitude(y[j]));
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
      const uint32_t byte = fp8_scale_byte(top);
      const float inv = fp8_inverse(byte);
      if (col < row_bytes) {
        uint2 w;
        w.x = fp8_codes(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
        w.y = fp8_codes(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
        *reinterpret_cast<uint2 *>(c.y8 + row * row_bytes + col) = w;
      }
      // padding scales, of blocks of zeros, are ones
      if ((t & 15) == 0 && col / kFp8Block < scale_bytes) c.y_scale[row * scale_bytes + col / kFp8Block] = (uint8_t)byte;
    }
  }
}

// Each workgroup takes rows b, b + blocks, ...; a thread keeps its columns' part of dw over them, and the
// finish kernel adds the workgroups' parts in order.
template <typename T, int TPR, int NV>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void rms_norm_backward_kernel(const NormBwdCall c,
                                                                                  float *__restrict__ parts) {
  constexpr int RPB = TPR >= 256 ? 1 : 256 / TPR;
  __shared__ float part[TPR > 64 ? TPR / 64 : 1];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int d = c.d;
  float dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  for (int64_t row = (int64_t)blockIdx.x * RPB + sub; row < c.T; row += (int64_t)gridDim.x * RPB) {
    const float rstd = c.rstd[row];
    float g[NV][8], xh[NV][8], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = 8 * (t + i * TPR), n = d - col;
      if (n <= 0) continue;
      float w[8];
      load8(static_cast<const T *>(c.dy) + row * d + col, n, g[i]);
      load8(static_cast<const T *>(c.h) + row * d + col, n, xh[i]);
      load8(static_cast<const T *>(c.weight) + col, n, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[i][j] *= rstd;
        dw[i][j] += g[i][j] * xh[i][j];
        g[i][j] *= w[j];
        sum += g[i][j] * xh[i][j];
      }
    }
    const float mean = row_sum<float, TPR>(sum, part) / (float)d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = 8 * (t + i * TPR), n = d - col;
      if (n <= 0) continue;
      float o[8];
      if (c.dh)
        load8(static_cast<const T *>(c.dh) + row * d + col, n, o);
      else
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] += rstd * (g[i][j] - xh[i][j] * mean);
      store8(static_cast<T *>(c.dx) + row * d + col, n, o);
    }
  }
  float *p = parts + ((int64_t)blockIdx.x * RPB + sub) * d;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = 8 * (t + i * TPR), n = d - col;
    if (n > 0) store8(p + col, n, dw[i]);
  }
}

__global__ __launch_bounds__(256) void rms_norm_dweight_kernel(const float *__restrict__ parts, int n, int d,
                                                               float *__restrict__ dweight) {
  __shared__ float s[4][64];
  const int col = blockIdx.x * 64 + (threadIdx.x & 63), q = threadIdx.x >> 6;
  float sum = 0.0f;
  if (col < d)
    for (int r = q; r < n; r += 4) sum += parts[(int64_t)r * d + col];
  s[q][threadIdx.x & 63] = sum;
  __syncthreads();
  if (q == 0 && col < d) dweight[col] = (s[0][threadIdx.x] + s[1][threadIdx.x]) + (s[2][threadIdx.x] + s[3][threadIdx.x]);
}

// Threads a row and vectors a thread for rows of d values (whole blocks of 128, the 8-bit output's padding).
template <typename F>
auto by_width(int d, F f) {
  const int vecs = fp8_row_bytes(d) / 8;
#define MOE_WIDTH(TPR, NV) \
  if (vecs <= TPR * NV) return f(std::integral_constant<int, TPR>{}, std::integral_constant<int, NV>{})
  MOE_WIDTH(64, 1);
  MOE_WIDTH(64, 2);
  MOE_WIDTH(64, 4);
  MOE_WIDTH(256, 2);
  MOE_WIDTH(256, 4);
  MOE_WIDTH(256, 8);
#undef MOE_WIDTH
  return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
}

int backward_blocks(int T, int d) {
  const int rpb = by_width(d, [](auto tpr, auto) { return tpr.value >= 256 ? 1 : 256 / tpr.value; });
  return std::min((T + rpb - 1) / rpb, 512);
}

}  // namespace

hipError_t launch_rms_norm(const NormCall &c, hipStream_t s) {
  by_width(c.d, [&](auto tpr, auto nv) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    constexpr int RPB = TPR >= 256 ? 1 : 256 / TPR;
    const dim3 grid((unsigned)((c.T + RPB - 1) / RPB)), block(TPR > 256 ? TPR : 256);
    if (c.f32)
      hipLaunchKernelGGL((rms_norm_kernel<float, TPR, NV>), grid, block, 0, s, c);
    else
      hipLaunchKernelGGL((rms_norm_kernel<bf16_t, TPR, NV>), grid, block, 0, s, c);
  });
  return hipGetLastError();
}

size_t rms_norm_backward_workspace_bytes(int T, int d) {
  const int rpb = by_width(d, [](auto tpr, auto) { return tpr.value >= 256 ? 1 : 256 / tpr.value; });
  return (size_t)backward_blocks(T, d) * rpb * d * 4;
}

hipError_t launch_rms_norm_backward(const NormBwdCall &c, void *ws, hipStream_t s) {
  const int blocks = backward_blocks(c.T, c.d);
  int parts = blocks;
  by_width(c.d, [&](auto tpr, auto nv) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    parts = blocks * (TPR >= 256 ? 1 : 256 / TPR);
    const dim3 grid((unsigned)blocks), block(TPR > 256 ? TPR : 256);
    if (c.f32)
      hipLaunchKernelGGL((rms_norm_backward_kernel<float, TPR, NV>), grid, block, 0, s, c, static_cast<float *>(ws));
    else
      hipLaunchKernelGGL((rms_norm_backward_kernel<bf16_t, TPR, NV>), grid, block, 0, s, c, static_cast<float *>(ws));
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(rms_norm_dweight_kernel, dim3((unsigned)((c.d + 63) / 64)), dim3(256), 0, s,
                     static_cast<const float *>(ws), parts, c.d, c.dweight);
  return hipGetLastError();
}

}  // namespace moe
