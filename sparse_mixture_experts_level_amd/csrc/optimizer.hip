// Gradient norm and AdamW step over many tensors at once.
//   norm = sqrt(sum g^2 over every tensor), scale = min(1, max_norm / (norm + 1e-6));
//   g' = scale g,  m' = b1 m + (1 - b1) g',  v' = b2 v + (1 - b2) g'^2,
//   w' = w (1 - lr wd) - lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps).
// Everything here touches each value once and is bound by memory.  A launch takes up to
// some tens of tensors as its kernel argument, so that a layer's few tensors (or a model's
// many small ones) cost one launch, no table in device memory and no copy; each block
// finds its tensor from the blocks' prefix sums.
//
// States in 8 bits: 256 values share a float scale, the block's largest magnitude.  m is a
// signed code c that stands for scale c |c| / 127^2, v an unsigned one for scale (c/255)^4,
// so that v's root, which the update divides by, has the same square law as m: fine steps
// near zero, 1.6% (m) and 0.8% (root of v) apart near the largest.  The nearest code to
// u = 127^2 |m'| / scale is the c with c (c - 1) + 1/2 <= u < c (c + 1) + 1/2; for v the
// same holds with u = 255^2 sqrt(v' / scale), or with both sides squared.  m' and v' are
// formed and compared in 64 bits: a float's rounding would move values next to a border
// by one code.  Each 64-bit operation is rounded by itself (no fused multiply-add), so that
// any program that follows the formulas holds the same codes and scales: with b1 = 0.9 a
// block's largest, 0.9 scale + 0.1 g, lies halfway between two floats in some percent of
// the blocks, and the last place then decides the scale.  A v' above zero takes one code at
// least: held as zero, it would let the next step divide by eps alone.
#include <algorithm>
#include <cmath>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = 1 << 23;  // blocks a launch: below 2^32 threads

// ------------------------------------------------------------------------ gradient norm

constexpr int kNormTensors = 64;
struct NormArgs {
  NormTensor t[kNormTensors];
  int32_t first[kNormTensors];  // first block of each tensor
  int32_t count;
  int32_t chunk;  // values a block
  double *part;
};

__device__ __forceinline__ int find_tensor(const int32_t *first, int count) {
  const int lane = threadIdx.x & 63;
  const bool at = lane < count && first[lane] <= (int)blockIdx.x;
  return __builtin_amdgcn_readfirstlane(__popcll(__ballot(at)) - 1);
}

// Sum of squares of one chunk, in 64 bits.
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(NormArgs a) {
  __shared__ double s_sum[kThreads / 64];
  const int ti = find_tensor(a.first, a.count);
  const NormTensor t = a.t[ti];
  const int64_t i0 = (int64_t)(blockIdx.x - a.first[ti]) * a.chunk;
  const int64_t i1 = min(t.n, i0 + a.chunk);
  double sum = 0;
  if (t.f32) {
    const float *g = static_cast<const float *>(t.grad);
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) sum += (double)g[i] * (double)g[i];
  } else {
    const bf16_t *g = static_cast<const bf16_t *>(t.grad);
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) {
      const double x = bf16_to_f32(g[i]);
      sum += x * x;
    }
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
  if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) a.part[blockIdx.x] = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
}

__global__ __launch_bounds__(1024) void grad_norm_finish_kernel(const double *__restrict__ part, int64_t n,
                                                                float max_norm, float *__restrict__ out) {
  __shared__ double s_sum[16];
  double sum = 0;
  for (int64_t i = threadIdx.x; i < n; i += 1024) sum += part[i];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
  if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double all = 0;
    for (int w = 0; w < 16; ++w) all += s_sum[w];
    const double norm = sqrt(all);
    out[0] = (float)norm;
    const double scale = (double)max_norm / (norm + 1e-6);
    // a norm that is not finite has no scale; AdamW then leaves everything as it was
    out[1] = norm < INFINITY ? (float)(scale < 1.0 ? scale : 1.0) : NAN;
  }
}

int64_t norm_chunk(const NormTensor *t, int count) {
  int64_t total = 0;
  for (int i = 0; i < count; ++i) total += t[i].n;
  const int64_t c = (total / 2048 + 2047) / 2048 * 2048;
  return std::min<int64_t>(std::max<int64_t>(c, 2048), 65536);
}

// ---------------------------------------------------------------------------- AdamW step

constexpr int kAdamTensors = 40;
struct AdamArgs {
  AdamTensor t[kAdamTensors];
  int32_t first[kAdamTensors];
  int32_t count;
  int32_t pad;
  AdamScalars h;
  double log_beta1, log_beta2;
};

struct Rates {
  float step;      // lr / (1 - b1^t)
  float inv_bc2;   // 1 / sqrt(1 - b2^t)
  float keep;      // 1 - lr wd
  float gscale;
};

// False: a gradient scale that is not a number (the norm was not finite) leaves everything.
__device__ __forceinline__ bool rates(const AdamArgs &a, float decay, Rates &r) {
  double lr = a.h.lr;
  int64_t t = a.h.step;
  if (a.h.lr_dev) lr = (double)*a.h.lr_dev;
  if (a.h.step_dev) t = max(*a.h.step_dev, (int64_t)1);
  r.step = (float)(lr / -expm1((double)t * a.log_beta1));
  r.inv_bc2 = (float)(1.0 / sqrt(-expm1((double)t * a.log_beta2)));
  r.keep = (float)(1.0 - lr * (double)decay);
  r.gscale = a.h.grad_scale ? *a.h.grad_scale : 1.f;
  return r.gscale == r.gscale;
}

__device__ __forceinline__ float load_grad(const AdamTensor &t, int64_t i) {
  return t.grad_f32 ? static_cast<const float *>(t.grad)[i] : bf16_to_f32(static_cast<const bf16_t *>(t.grad)[i]);
}
__device__ __forceinline__ float load_weight(const AdamTensor &t, int64_t i) {
  if (t.master) return t.master[i];
  return t.param_f32 ? static_cast<const float *>(t.param)[i] : bf16_to_f32(static_cast<const bf16_t *>(t.param)[i]);
}
__device__ __forceinline__ void store_weight(const AdamTensor &t, int64_t i, float w) {
  if (t.master) t.master[i] = w;
  if (t.param_f32)
    static_cast<float *>(t.param)[i] = w;
  else
    static_cast<bf16_t *>(t.param)[i] = f32_to_bf16(w);
}

constexpr int kAdamChunk = 2048;  // values a block

__global__ __launch_bounds__(kThreads) void adamw32_kernel(AdamArgs a) {
  const int ti = find_tensor(a.first, a.count);
  const AdamTensor t = a.t[ti];
  Rates r;
  if (!rates(a, t.decay, r)) return;
  const float b1 = (float)a.h.beta1, b2 = (float)a.h.beta2, c1 = (float)(1.0 - a.h.beta1),
              c2 = (float)(1.0 - a.h.beta2), eps = (float)a.h.eps;
  const int64_t i0 = (int64_t)(blockIdx.x - a.first[ti]) * kAdamChunk;
  const int64_t i1 = min(t.n, i0 + kAdamChunk);
  float *pm = static_cast<float *>(t.m), *pv = static_cast<float *>(t.v);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) {
    const float g = load_grad(t, i) * r.gscale;
    const float m = b1 * pm[i] + c1 * g;
    const float v = b2 * pv[i] + c2 * (g * g);
    pm[i] = m;
    pv[i] = v;
    const float u = m / (sqrtf(v) * r.inv_bc2 + eps);
    store_weight(t, i, load_weight(t, i) * r.keep - r.step * u);
  }
}

constexpr double kPerM = 1.0 / 16129.0, kPerV = 1.0 / 4228250625.0;  // 1 / 127^2, 1 / 255^4

// m' and v' in 64 bits from the values held, every operation rounded by itself.
__device__ __forceinline__ double next_m(int code, double scale, double g, double b1, double c1) {
#pragma clang fp contract(off)
  const double old = (double)(code * abs(code)) * scale;
  const double a = b1 * old, b = c1 * g;
  return a + b;
}
__device__ __forceinline__ double next_v(uint32_t code, double scale, double g, double b2, double c2) {
#pragma clang fp contract(off)
  const double old = (double)(code * code * (code * code)) * scale;
  const double gg = g * g;
  const double a = b2 * old, b = c2 * gg;
  return a + b;
}

// The code whose square is nearest to u (u >= 0, at most top^2 and a little).
__device__ __forceinline__ int nearest_root(double u, int top) {
  int c = (int)(__builtin_amdgcn_sqrtf(fmaxf((float)u - 0.25f, 0.f)) + 0.5f);
  c = min(c, top);
  // the float's error can put c one off at a border; the border itself is exact in 64 bits
  if (c > 0 && u < (double)(c * (c - 1)) + 0.5) --c;
  if (c < top && u >= (double)(c * (c + 1)) + 0.5) ++c;
  return c;
}
// The same with u given squared.
__device__ __forceinline__ int nearest_fourth_root(double uu, int top) {
  int c = (int)(__builtin_amdgcn_sqrtf(fmaxf(__builtin_amdgcn_sqrtf((float)uu) - 0.25f, 0.f)) + 0.5f);
  c = min(c, top);
  const double lo = (double)(c * (c - 1)) + 0.5, hi = (double)(c * (c + 1)) + 0.5;
  if (c > 0 && uu < lo * lo) --c;
  else if (c < top && uu >= hi * hi) ++c;
  return c;
}

__device__ __forceinline__ uint32_t max32(uint32_t v) {  // over the 32 lanes of a half wavefront
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
  return v;
}

// The scale held for a block whose largest magnitude has these bits: zero below the smallest
// normal float, NaN for a block with a value that is not finite.
__device__ __forceinline__ float held_scale(uint32_t bits) {
  if (bits >= 0x7f800000u) return NAN;
  return bits < 0x00800000u ? 0.f : __uint_as_float(bits);
}

// Eight values a thread, 32 threads a block of 256 values.
__global__ __launch_bounds__(kThreads) void adamw8_kernel(AdamArgs a) {
  const int ti = find_tensor(a.first, a.count);
  const AdamTensor t = a.t[ti];
  Rates r;
  if (!rates(a, t.decay, r)) return;
  const double b1 = a.h.beta1, b2 = a.h.beta2, c1 = 1.0 - b1, c2 = 1.0 - b2;
  const float eps = (float)a.h.eps;
  const int64_t i = (int64_t)(blockIdx.x - a.first[ti]) * kAdamChunk + threadIdx.x * 8;
  const int64_t q = i / kAdamBlock;
  const bool any = i < t.n;
  int8_t *pm = static_cast<int8_t *>(t.m);
  uint8_t *pv = static_cast<uint8_t *>(t.v);
  const bool blk = q * kAdamBlock < t.n;
  const double sm = blk ? (double)t.m_scale[q] * kPerM : 0.0, sv = blk ? (double)t.v_scale[q] * kPerV : 0.0;
  double m[8], v[8];
  uint32_t bm = 0, bv = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    m[j] = v[j] = 0;
    if (any && i + j < t.n) {
      const double g = (double)load_grad(t, i + j) * (double)r.gscale;
      const int cm = pm[i + j];
      const uint32_t cv = pv[i + j];
      m[j] = next_m(cm, sm, g, b1, c1);
      v[j] = next_v(cv, sv, g, b2, c2);
      bm = max(bm, __float_as_uint((float)m[j]) & 0x7fffffffu);
      bv = max(bv, __float_as_uint((float)v[j]) & 0x7fffffffu);
    }
  }
  const float hm = held_scale(max32(bm)), hv = held_scale(max32(bv));
  if (!any) return;
  if ((threadIdx.x & 31) == 0) {
    t.m_scale[q] = hm;
    t.v_scale[q] = hv;
  }
  const double im = hm > 0.f ? 16129.0 / (double)hm : 0.0, iv = hv > 0.f ? 4228250625.0 / (double)hv : 0.0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (i + j >= t.n) break;
    const float mf = (float)m[j], vf = (float)v[j];
    const float u = mf / (sqrtf(vf) * r.inv_bc2 + eps);
    store_weight(t, i + j, load_weight(t, i + j) * r.keep - r.step * u);
    const int cm = hm > 0.f ? nearest_root(fabs(m[j]) * im, 127) : 0;
    pm[i + j] = (int8_t)(m[j] < 0 ? -cm : cm);
    int cv = hv > 0.f ? nearest_fourth_root(v[j] * iv, 255) : 0;
    if (hv > 0.f && v[j] > 0) cv = max(cv, 1);
    pv[i + j] = (uint8_t)cv;
  }
}

// ------------------------------------------------------------- 8-bit states read as floats

struct ReadTensor {
  const int8_t *m;
  const uint8_t *v;
  const float *m_scale, *v_scale;
  float *m_out, *v_out;
  int64_t n;
};
struct ReadArgs {
  ReadTensor t[kAdamTensors];
  int32_t first[kAdamTensors];
  int32_t count;
};

__global__ __launch_bounds__(kThreads) void adamw_read_kernel(ReadArgs a) {
  const int ti = find_tensor(a.first, a.count);
  const ReadTensor t = a.t[ti];
  const int64_t i0 = (int64_t)(blockIdx.x - a.first[ti]) * kAdamChunk;
  const int64_t i1 = min(t.n, i0 + kAdamChunk);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) {
    const int64_t q = i / kAdamBlock;
    if (t.m_out) {
      const int c = t.m[i];
      t.m_out[i] = (float)((double)(c * abs(c)) * ((double)t.m_scale[q] * kPerM));
    }
    if (t.v_out) {
      const uint32_t c = t.v[i];
      t.v_out[i] = (float)((double)(c * c * (c * c)) * ((double)t.v_scale[q] * kPerV));
    }
  }
}

}  // namespace

size_t grad_norm_workspace_bytes(const NormTensor *t, int count) {
  const int64_t chunk = norm_chunk(t, count);
  int64_t blocks = 1;
  for (int i = 0; i < count; ++i) blocks += (t[i].n + chunk - 1) / chunk;
  return (size_t)blocks * 8;
}

hipError_t launch_grad_norm(const NormTensor *t, int count, float max_norm, float *out, void *ws, hipStream_t s) {
  NormArgs a{};
  a.chunk = (int32_t)norm_chunk(t, count);
  double *part = static_cast<double *>(ws);
  int64_t done = 0, blocks = 0;
  auto flush = [&]() -> hipError_t {
    if (a.count == 0) return hipSuccess;
    a.part = part + done;
    hipLaunchKernelGGL(grad_norm_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
    done += blocks;
    blocks = 0;
    a.count = 0;
    return hipGetLastError();
  };
  for (int i = 0; i < count; ++i) {
    const int64_t nb = (t[i].n + a.chunk - 1) / a.chunk;
    if (nb == 0) continue;
    if (a.count == kNormTensors || blocks + nb > kMaxBlocks) {
      const hipError_t e = flush();
      if (e != hipSuccess) return e;
    }
    a.t[a.count] = t[i];
    a.first[a.count++] = (int32_t)blocks;
    blocks += nb;
  }
  hipError_t e = flush();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(grad_norm_finish_kernel, dim3(1), dim3(1024), 0, s, part, done, max_norm, out);
  return hipGetLastError();
}

hipError_t launch_adamw(const AdamTensor *t, int count, const AdamScalars &h, hipStream_t s) {
  AdamArgs a{};
  a.h = h;
  a.log_beta1 = std::log(h.beta1);
  a.log_beta2 = std::log(h.beta2);
  for (int eight = 0; eight < 2; ++eight) {
    int64_t blocks = 0;
    a.count = 0;
    auto flush = [&]() -> hipError_t {
      if (a.count == 0) return hipSuccess;
      if (eight)
        hipLaunchKernelGGL(adamw8_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
      else
        hipLaunchKernelGGL(adamw32_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
      blocks = 0;
      a.count = 0;
      return hipGetLastError();
    };
    for (int i = 0; i < count; ++i) {
      if (t[i].eight != eight || t[i].n == 0) continue;
      const int64_t nb = (t[i].n + kAdamChunk - 1) / kAdamChunk;
      if (a.count == kAdamTensors || blocks + nb > kMaxBlocks) {
        const hipError_t e = flush();
        if (e != hipSuccess) return e;
      }
      a.t[a.count] = t[i];
      a.first[a.count++] = (int32_t)blocks;
      blocks += nb;
    }
    const hipError_t e = flush();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_adamw_read(const AdamTensor *t, int count, float *const *m_out, float *const *v_out, hipStream_t s) {
  ReadArgs a{};
  int64_t blocks = 0;
  auto flush = [&]() -> hipError_t {
    if (a.count == 0) return hipSuccess;
    hipLaunchKernelGGL(adamw_read_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
    blocks = 0;
    a.count = 0;
    return hipGetLastError();
  };
  for (int i = 0; i < count; ++i) {
    float *mo = m_out ? m_out[i] : nullptr, *vo = v_out ? v_out[i] : nullptr;
    if (t[i].n == 0 || (!mo && !vo)) continue;
    const int64_t nb = (t[i].n + kAdamChunk - 1) / kAdamChunk;
    if (a.count == kAdamTensors || blocks + nb > kMaxBlocks) {
      const hipError_t e = flush();
      if (e != hipSuccess) return e;
    }
    a.t[a.count] = ReadTensor{static_cast<const int8_t *>(t[i].m), static_cast<const uint8_t *>(t[i].v),
                              t[i].m_scale, t[i].v_scale, mo, vo, t[i].n};
    a.first[a.count++] = (int32_t)blocks;
    blocks += nb;
  }
  return flush();
}

}  // namespace moe
