// Root-mean-square norm with the residual's addition and an 8-bit output, and its backward pass.
//
//   h = x + residual (rounded to the layer's type: it is what the residual stream carries on and what the
//   backward pass reads), rstd = 1 / sqrt(mean h^2 + eps), y = (h rstd) w
//   dx = dh + rstd (g - xhat mean(g xhat)),  g = dy w, xhat = h rstd;  dw = sum_t dy xhat
//
// Memory bound: a row is read once into registers, as vectors of eight values a thread, and
// written once.  16384 x 7168 of bf16 with residual, y and codes 189 us (5.6 TB/s beyond L2, a copy's rate 4.9 over more
// bytes), backward of 4096 x 4096 28 us (5.2) and 5 for dweight.
#include <algorithm>

#include "fp8.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

// Sum over the wavefront in every lane, by lane moves (two 32-bit halves of a double).
__device__ __forceinline__ float wave_sum(float v) {
  return group_reduce<64>(v, [](float a, float b) { return a + b; });
}
template <int CTRL>
__device__ __forceinline__ double double_move(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint64_t lo = lane_move<CTRL>((uint32_t)u), hi = lane_move<CTRL>((uint32_t)(u >> 32));
  return __builtin_bit_cast(double, lo | hi << 32);
}
__device__ __forceinline__ double wave_sum(double v) {
  v += double_move<0xb1>(v);
  v += double_move<0x4e>(v);
  v += double_move<0x141>(v);
  v += double_move<0x140>(v);
  auto pair = [](auto lo, auto hi) {
    return __builtin_bit_cast(double, (uint64_t)lo[0] | (uint64_t)hi[0] << 32) +
           __builtin_bit_cast(double, (uint64_t)lo[1] | (uint64_t)hi[1] << 32);
  };
  uint64_t u = __builtin_bit_cast(uint64_t, v);
  uint32_t lo = (uint32_t)u, hi = (uint32_t)(u >> 32);
  v = pair(__builtin_amdgcn_permlane16_swap(lo, lo, false, false), __builtin_amdgcn_permlane16_swap(hi, hi, false, false));
  u = __builtin_bit_cast(uint64_t, v);
  lo = (uint32_t)u;
  hi = (uint32_t)(u >> 32);
  return pair(__builtin_amdgcn_permlane32_swap(lo, lo, false, false), __builtin_amdgcn_permlane32_swap(hi, hi, false, false));
}

// The sum over the TPR threads that share a row, in every one of them; TPR is 64 (one wave) or the
// whole workgroup, whose waves leave their sums in `part` (the caller's next use is of another array).
template <typename V, int TPR>
__device__ __forceinline__ V row_sum(V v, V *part) {
  v = wave_sum(v);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w) v += part[w];
  }
  return v;
}

// TPR threads a row, NV vectors of eight a thread: vector i of thread t at column 8 (t + i TPR).  Everything is
// loaded before the sum, the weight too, so that its latency is waited for once.  The mean of
// squares is formed in 64 bits, and h rstd and its product with w are each rounded to float, so
// that the codes, which jump next to a border, are the same in any order of the sum.
template <typename T, int TPR, int NV, bool WHOLE>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void rms_norm_kernel(const NormCall c) {
  constexpr int RPB = TPR >= 256 ? 1 : 256 / TPR;
  __shared__ double part[TPR > 64 ? TPR / 64 : 1];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if (row >= c.T) return;  // whole waves, and whole workgroups where a barrier follows
  const int d = c.d;
  // TB/s one by one and back: 45829 x 1091 of bf16 4.64 and 5.41, 17355 x 2881 4.22 and 4.84; of floats 5.07 and 4.24
  constexpr bool BACK = !WHOLE && sizeof(T) == 2;
  const T *x = static_cast<const T *>(c.x) + row * d;
  const T *res = c.residual ? static_cast<const T *>(c.residual) + row * d : nullptr;
  Raw8<T> xr[NV], rr[NV], wr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = 8 * (t + i * TPR);
    xr[i] = load8<T, WHOLE, BACK>(x + col, d - col, d);
    if (res) rr[i] = load8<T, WHOLE, BACK>(res + col, d - col, d);
    wr[i] = load8<T, WHOLE, BACK>(static_cast<const T *>(c.weight) + col, d - col, d);
  }
  float h[NV][8];
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (BACK) {
      const int n = d - 8 * (t + i * TPR);
      xr[i].front(n);
      if (res) rr[i].front(n);
      wr[i].front(n);
    }
    xr[i].to(h[i]);
    if (res) {
      float r[8];
      rr[i].to(r);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[i][j] += r[j];
        if constexpr (sizeof(T) == 2) h[i][j] = bf16_to_f32(f32_to_bf16(h[i][j]));
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += (double)h[i][j] * (double)h[i][j];
    const int col = 8 * (t + i * TPR);
    if (c.h) store8<T, WHOLE>(static_cast<T *>(c.h) + row * d + col, d - col, h[i]);
  }
  sum = row_sum<double, TPR>(sum, part);
  const float rstd = (float)(1.0 / sqrt(sum / (double)d + (double)c.eps));
  if (c.rstd && t == 0) c.rstd[row] = rstd;
  const int row_bytes = fp8_row_bytes(d), scale_bytes = fp8_scale_bytes(d);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = 8 * (t + i * TPR);
    float y[8];
    wr[i].to(y);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] *= h[i][j] * rstd;
    if (c.y) store8<T, WHOLE>(static_cast<T *>(c.y) + row * d + col, d - col, y);
    if (c.y8) {
      if (d - col < 8) {  // behind the row: zeros, whatever rstd is
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = col + j < d ? y[j] : 0.0f;
      }
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, fp8_magnitude(y[j]));
      top = group_reduce<16>(top, [](float a, float b) { return fmaxf(a, b); });
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

// Each workgroup takes rows b, b + blocks, ...; a thread keeps its columns' part of dw over them. Waves with rows
// of their own add theirs up in LDS at the end, and the finish kernel adds the workgroups' parts, all in order.
template <typename T, int TPR, int NV, bool WHOLE>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void rms_norm_backward_kernel(const NormBwdCall c,
                                                                                  float *__restrict__ parts) {
  constexpr int RPB = TPR >= 256 ? 1 : 256 / TPR;
  __shared__ float part[2][TPR > 64 ? TPR / 64 : 1];
  __shared__ float rows_dw[RPB > 1 ? RPB - 1 : 1][RPB > 1 ? TPR * NV * 8 : 1];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int d = c.d;
  // From 64 sums a thread on the weight and dh are loaded where they are used, the weight from the caches: held over the
  // rows they did not fit.
  constexpr bool LEAN = NV >= 8;
  float dw[NV][8];
  Raw8<T> wr[LEAN ? 1 : NV];
  auto weight = [&](int i) -> Raw8<T> {
    const int col = 8 * (t + i * TPR);
    return load8<T, WHOLE>(static_cast<const T *>(c.weight) + col, d - col, d);
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (!LEAN) wr[i] = weight(i);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  }
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPB + sub; row < c.T; row += (int64_t)gridDim.x * RPB, turn ^= 1) {
    const float rstd = c.rstd[row];
    Raw8<T> gr[NV], hr[NV], ar[LEAN ? 1 : NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = 8 * (t + i * TPR);
      gr[i] = load8<T, WHOLE>(static_cast<const T *>(c.dy) + row * d + col, d - col, d);
      hr[i] = load8<T, WHOLE>(static_cast<const T *>(c.h) + row * d + col, d - col, d);
      if constexpr (!LEAN)
        if (c.dh) ar[i] = load8<T, WHOLE>(static_cast<const T *>(c.dh) + row * d + col, d - col, d);
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float g[8], xh[8], w[8];
      gr[i].to(g);
      hr[i].to(xh);
      if constexpr (LEAN)
        weight(i).to(w);
      else
        wr[i].to(w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[j] *= rstd;
        dw[i][j] += g[j] * xh[j];
        sum += g[j] * w[j] * xh[j];
      }
    }
    const float mean = row_sum<float, TPR>(sum, part[turn]) / (float)d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float g[8], xh[8], w[8], o[8];
      gr[i].to(g);
      hr[i].to(xh);
      if constexpr (LEAN)
        weight(i).to(w);
      else
        wr[i].to(w);
      const int col = 8 * (t + i * TPR);
      if (c.dh) {
        Raw8<T> r;
        if constexpr (LEAN)
          r = load8<T, WHOLE>(static_cast<const T *>(c.dh) + row * d + col, d - col, d);
        else
          r = ar[i];
        r.to(o);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] += rstd * (g[j] * w[j] - xh[j] * rstd * mean);
      store8<T, WHOLE>(static_cast<T *>(c.dx) + row * d + col, d - col, o);
    }
  }
  if constexpr (RPB > 1) {
    if (sub > 0)
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) rows_dw[sub - 1][(i * 8 + j) * TPR + t] = dw[i][j];
    __syncthreads();
    if (sub > 0) return;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int q = 0; q < RPB - 1; ++q) dw[i][j] += rows_dw[q][(i * 8 + j) * TPR + t];
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = 8 * (t + i * TPR);
    store8<float, WHOLE>(parts + (int64_t)blockIdx.x * d + col, d - col, dw[i]);
  }
}

// 16 columns a workgroup, sixteen rows of parts at a time, all loads of 512 rows in flight
// (range-checked: behind a branch each, one at a time, 12 us for 4); sums in 64 bits: added in floats the parts lost 1.5e-7 of
// dweight's norm at 5003 x 1091, for 6e-8 now, half a step of the result.  The parts themselves are floats, as 64 bits would
// double the registers that they take; they lose more with more rows a thread: 1.1e-7 at 10^5 rows of 64, 3.3e-7 at 10^6,
// 1.4e-6 at 1.6 10^7 (torch's sums in floats: 1.6e-7, 2.8e-7, 8.0e-7).
__global__ __launch_bounds__(256) void rms_norm_dweight_kernel(const float *__restrict__ parts, int n, int d,
                                                               float *__restrict__ dweight) {
  __shared__ double s[16][17];
  const int q = threadIdx.x >> 4, l = threadIdx.x & 15, col = blockIdx.x * 16 + l;
  double sum = 0.0;
  const rsrc_t from = make_rsrc(parts, (uint32_t)n * (uint32_t)d * 4u);  // zeros past the last row
  for (int r0 = q; r0 < n; r0 += 16 * 32) {
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j)
      v[j] = __builtin_bit_cast(float, (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(
                                           from, col < d ? (uint32_t)((r0 + 16 * j) * d + col) * 4u : kOob, 0, 0));
#pragma unroll
    for (int j = 0; j < 32; ++j) sum += v[j];
  }
  s[q][l] = sum;
  __syncthreads();
  if (q == 0 && col < d) {
    for (int r = 1; r < 16; ++r) sum += s[r][l];
    dweight[col] = (float)sum;
  }
}

// Threads a row and vectors a thread for rows of d values (whole blocks of 128, the 8-bit output's padding), and
// whether rows are whole vectors.
template <bool BACKWARD, typename F>
void by_width(int d, F f) {
  const int vecs = fp8_row_bytes(d) / 8;
  const auto whole = [&](auto tpr, auto nv) {
    if (d % 8 == 0)
      f(tpr, nv, std::true_type{});
    else
      f(tpr, nv, std::false_type{});
  };
#define MOE_WIDTH(TPR, NV) \
  if (vecs <= TPR * NV) return whole(std::integral_constant<int, TPR>{}, std::integral_constant<int, NV>{})
  MOE_WIDTH(64, 1);
  MOE_WIDTH(64, 2);
  MOE_WIDTH(64, 4);
  MOE_WIDTH(256, 2);
  MOE_WIDTH(256, 4);
  MOE_WIDTH(256, 8);
#undef MOE_WIDTH
  if constexpr (BACKWARD)  // (1024 x 4 have 128 registers each and spilled: 3050 x 16391 of bf16 at 0.9 TB/s for 2.3. 512 x 8
                           // still spill 14 to 24 registers of bf16 and 106 to 205 of float rows: 2.0 TB/s)
    whole(std::integral_constant<int, 512>{}, std::integral_constant<int, 8>{});
  else
    whole(std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
}

// Workgroups of the backward: eight rows or more for each thread's part of dw, whose
// writing and reading again is then at most an eighth of the rows' own bytes, but enough to fill the GPU.
int backward_blocks(int T, int d) {
  const int rpb = fp8_row_bytes(d) / 8 <= 256 ? 4 : 1;  // rows a workgroup has at once (by_width)
  const int all = T / rpb + (T % rpb != 0);
  return std::min(all, std::min(1024, std::max(512, all / 8)));
}

}  // namespace

hipError_t launch_rms_norm(const NormCall &call, hipStream_t s) {
  const int64_t size = call.f32 ? 4 : 2, row_bytes = fp8_row_bytes(call.d), scale_bytes = fp8_scale_bytes(call.d);
  by_width<false>(call.d, [&](auto tpr, auto nv, auto whole) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    constexpr bool WHOLE = decltype(whole)::value;
    constexpr int RPB = TPR >= 256 ? 1 : 256 / TPR, THREADS = TPR > 256 ? TPR : 256;
    constexpr int64_t kRows = TPR > 512 ? 1 << 21 : 1 << 22;  // a launch: the threads of one are counted in 32 bits
    static_assert(kRows / RPB * THREADS <= UINT32_MAX, "threads of a launch");
    for (int64_t first = 0; first < call.T; first += kRows) {
      NormCall c = call;
      auto from = [&](auto p, int64_t bytes) { return p ? (decltype(p))((uintptr_t)p + (size_t)(first * bytes)) : p; };
      c.x = from(call.x, call.d * size);
      c.residual = from(call.residual, call.d * size);
      c.h = from(call.h, call.d * size);
      c.y = from(call.y, call.d * size);
      c.y8 = from(call.y8, row_bytes);
      c.y_scale = from(call.y_scale, scale_bytes);
      c.rstd = from(call.rstd, 4);
      c.T = (int)std::min<int64_t>(kRows, call.T - first);
      const dim3 grid((unsigned)((c.T + RPB - 1) / RPB)), block(THREADS);
      if (c.f32)
        hipLaunchKernelGGL((rms_norm_kernel<float, TPR, NV, WHOLE>), grid, block, 0, s, c);
      else
        hipLaunchKernelGGL((rms_norm_kernel<bf16_t, TPR, NV, WHOLE>), grid, block, 0, s, c);
    }
  });
  return hipGetLastError();
}

size_t rms_norm_backward_workspace_bytes(int T, int d) { return (size_t)backward_blocks(T, d) * d * 4; }

hipError_t launch_rms_norm_backward(const NormBwdCall &c, void *ws, hipStream_t s) {
  const int blocks = backward_blocks(c.T, c.d);
  if (blocks > 0)
    by_width<true>(c.d, [&](auto tpr, auto nv, auto whole) {
      constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
      constexpr bool WHOLE = decltype(whole)::value;
      const dim3 grid((unsigned)blocks), block(TPR > 256 ? TPR : 256);
      if (c.f32)
        hipLaunchKernelGGL((rms_norm_backward_kernel<float, TPR, NV, WHOLE>), grid, block, 0, s, c,
                           static_cast<float *>(ws));
      else
        hipLaunchKernelGGL((rms_norm_backward_kernel<bf16_t, TPR, NV, WHOLE>), grid, block, 0, s, c,
                           static_cast<float *>(ws));
    });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(rms_norm_dweight_kernel, dim3((unsigned)((c.d + 15) / 16)), dim3(256), 0, s,
                     static_cast<const float *>(ws), blocks, c.d, c.dweight);
  return hipGetLastError();
}

}  // namespace moe
