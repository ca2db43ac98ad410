// Gradient norm and AdamW step over many tensors at once.
//   norm = sqrt(sum g^2 over every tensor), scale = min(1, max_norm / (norm + 1e-6));
//   g' = scale g,  m' = b1 m + (1 - b1) g',  v' = b2 v + (1 - b2) g'^2,
//   w' = w (1 - lr wd) - lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps).
// Everything here touches each value once and is bound by memory.  A launch takes up to
// some tens of tensors as its kernel argument, so that a layer's few tensors (or a model's
// many small ones) cost one launch, no table in device memory and no copy; each block
// finds its tensor from the blocks' prefix sums.  Measured, where a copy of 4 GiB reaches
// 5.9 TB/s read and written and a plain read 7.0: the norm of 176 M bf16 gradients 57 us (6.2
// TB/s); AdamW with 32-bit states and a float copy on as many bf16 weights 880 us (5.6 TB/s);
// with 8-bit states on 201 M and a float copy 564 us (5.9 TB/s beyond L2, its arithmetic of some 80
// instructions a value nearly as long), 1008 us with the norm before it and both states read back
// after it.  Without a float copy the arithmetic is what bounds it (13 M values: 40 us, 3.3 TB/s).
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
// What rounding to nearest costs: a v without gradients leaves its code only if beta2 < (1 - 1 / c
// + 1 / (2 c^2))^2, never from 0.9922 on: beta2 = 0.999 is for states in 32 bits.
#include <algorithm>
#include <cmath>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = 1 << 23;  // blocks a launch: below 2^32 threads

// Index of the block's tensor: the last of `count` whose first block is not past this one.
__device__ __forceinline__ int find_tensor(const int32_t *first, int count) {
  const int lane = threadIdx.x & 63;
  int found = -1;
  for (int c = 0; c < count; c += 64) {
    const bool at = c + lane < count && first[c + lane] <= (int)blockIdx.x;
    found += __popcll(__ballot(at));
  }
  return __builtin_amdgcn_readfirstlane(found);
}

// --------------------------------------------------------------------- groups of values

// Four or eight neighbouring values of a tensor as floats; `p` points at them, 16-byte
// aligned for floats and for eight bf16, 8-byte for four bf16.
// Accesses past the caches, since a step comes round to a value only once: 880 against 931 us on
// 176 M values with plain ones (loads or stores alone: 926, 920).
template <int N>
struct Vals {
  float v[N];
};
__device__ __forceinline__ f32x4 ld_f32x4(const float *p) {
  return __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p));
}
__device__ __forceinline__ void st_f32x4(float *p, f32x4 v) {
  __builtin_nontemporal_store(v, reinterpret_cast<f32x4 *>(p));
}
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <int N>
__device__ __forceinline__ Vals<N> load_vals(const float *p) {
  Vals<N> r;
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const f32x4 q = ld_f32x4(p + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) r.v[i + j] = q[j];
  }
  return r;
}
template <int N>
__device__ __forceinline__ Vals<N> load_vals(const bf16_t *p) {
  Vals<N> r;
  uint32_t w[N / 2];
  if constexpr (N == 8) {
    const u32x4 q = ldg16_nt(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = q[i];
  } else {
    const u32x2 q = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(p));
    w[0] = q[0];
    w[1] = q[1];
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    r.v[2 * i] = __uint_as_float(w[i] << 16);
    r.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return r;
}
template <int N>
__device__ __forceinline__ void store_vals(float *p, const Vals<N> &x) {
#pragma unroll
  for (int i = 0; i < N; i += 4) st_f32x4(p + i, f32x4{x.v[i], x.v[i + 1], x.v[i + 2], x.v[i + 3]});
}
template <int N>
__device__ __forceinline__ void store_vals(bf16_t *p, const Vals<N> &x) {
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) w[i] = pack_bf16x2(x.v[2 * i], x.v[2 * i + 1]);
  if constexpr (N == 8)
    stg16_nt(p, u32x4{w[0], w[1], w[2], w[3]});
  else
    __builtin_nontemporal_store(u32x2{w[0], w[1]}, reinterpret_cast<u32x2 *>(p));
}
// The first `n` of them (n < N).
template <int N, typename T>
__device__ __forceinline__ Vals<N> load_some(const T *p, int n) {
  Vals<N> r;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    r.v[i] = 0.f;
    if (i < n) {
      if constexpr (sizeof(T) == 4)
        r.v[i] = p[i];
      else
        r.v[i] = bf16_to_f32(p[i]);
    }
  }
  return r;
}
template <int N, typename T>
__device__ __forceinline__ void store_some(T *p, const Vals<N> &x, int n) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < n) store_out(p + i, x.v[i]);
}
template <int N, typename T>
__device__ __forceinline__ Vals<N> load_n(const T *p, int n) {
  return n >= N ? load_vals<N>(p) : load_some<N>(p, n);
}
template <int N, typename T>
__device__ __forceinline__ void store_n(T *p, const Vals<N> &x, int n) {
  if (n >= N)
    store_vals<N>(p, x);
  else
    store_some<N>(p, x, n);
}

// ------------------------------------------------------------------------ gradient norm

constexpr int kNormTensors = 192;
struct NormArgs {
  const void *grad[kNormTensors];
  int64_t n[kNormTensors];         // values, negative (~n): floats
  int32_t first[kNormTensors];     // first block of each tensor
  int32_t count;
  int32_t chunk;  // values a block, a multiple of 2048
  double *part;
};

template <typename T>
__device__ __forceinline__ double chunk_squares(const T *g, int64_t i0, int64_t i1) {
  double sum = 0;
  int64_t i = i0 + threadIdx.x * 8;
#pragma unroll 2
  for (; i + 8 <= i1; i += kThreads * 8) {
    const Vals<8> x = load_vals<8>(g + i);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += (double)x.v[j] * (double)x.v[j];
  }
  if (i < i1) {
    const Vals<8> x = load_some<8>(g + i, (int)(i1 - i));
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += (double)x.v[j] * (double)x.v[j];
  }
  return sum;
}

// Sum of squares of one chunk, in 64 bits.
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(NormArgs a) {
  __shared__ double s_sum[kThreads / 64];
  const int ti = find_tensor(a.first, a.count);
  const int64_t code = a.n[ti], n = code < 0 ? ~code : code;
  const int64_t i0 = (int64_t)(blockIdx.x - a.first[ti]) * a.chunk;
  const int64_t i1 = min(n, i0 + a.chunk);
  double sum = code < 0 ? chunk_squares(static_cast<const float *>(a.grad[ti]), i0, i1)
                        : chunk_squares(static_cast<const bf16_t *>(a.grad[ti]), i0, i1);
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
#pragma unroll 4
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
    // a gradient that is not finite leaves no scale, and AdamW everything as it was; a norm that is
    // finite here but past the floats has its scale
    out[1] = norm < INFINITY ? (float)(scale < 1.0 ? scale : 1.0) : NAN;
  }
}

// About 2048 blocks (eight a compute unit) where there is enough, of at most 32768 values: larger
// ones leave compute units idle at the end (176 M values: 57 us, 65536 a block 65 us, 8192 a
// block 61), more blocks lengthen the sum of their results.
int64_t norm_chunk(const NormTensor *t, int count) {
  int64_t total = 0;
  for (int i = 0; i < count; ++i) total += t[i].n;
  const int64_t c = (total / 2048 + 2047) / 2048 * 2048;
  return std::min<int64_t>(std::max<int64_t>(c, 2048), 32768);
}

// ---------------------------------------------------------------------------- AdamW step

// A tensor as a kernel argument: with states in 32 bits it has no scales.
struct Adam32 {
  void *param;
  const void *grad;
  float *master;
  void *m, *v;
  int64_t n;
  float decay;
  uint8_t param_f32, grad_f32, pad[2];
};
struct Adam8 : Adam32 {
  float *m_scale, *v_scale;
};
template <typename Tensor, int N>
struct AdamArgs {
  Tensor t[N];
  int32_t first[N];
  int32_t count;
  int32_t last;         // the step's last launch
  float step, inv_bc2;  // from the host's lr and t
  AdamScalars h;
  double log_beta1, log_beta2;
};
// As many as go into 4 KB of arguments (120 tensors of 12 M values with 32-bit states,
// clipped: 48 a launch 76.9 us, 64 72.9).
using Adam32Args = AdamArgs<Adam32, 64>;
using Adam8Args = AdamArgs<Adam8, 48>;
static_assert(sizeof(Adam32Args) <= 4096 && sizeof(Adam8Args) <= 4096 && sizeof(NormArgs) <= 4096, "kernel arguments");

struct Rates {
  float step;      // lr / (1 - b1^t)
  float inv_bc2;   // 1 / sqrt(1 - b2^t)
  float keep;      // 1 - lr wd
  float gscale;
};

__device__ float d_no_scale = 1.f;
__device__ int64_t d_none_skipped = 0;

// False: a gradient scale that is not a number (the norm was not finite) leaves everything, and
// the step's last launch, of which then no block looks at the count, counts it.
template <typename Args>
__device__ __forceinline__ bool rates(const Args &a, float decay, Rates &r) {
  double lr = a.h.lr;
  r.step = a.step;
  r.inv_bc2 = a.inv_bc2;
  // both in flight together, from what stands for them where they are not given: one after the other
  // 201 M values with 8-bit states, clipped and read back, took 1024 us, so 1008
  const float *gscale = a.h.grad_scale ? a.h.grad_scale : &d_no_scale;
  const int64_t *count = a.h.skipped ? a.h.skipped : &d_none_skipped;
  r.gscale = *gscale;
  const int64_t skipped = *count;
  if (r.gscale != r.gscale) {  // (what block 0 writes is not looked at here)
    if (a.last && a.h.skipped && blockIdx.x == 0 && threadIdx.x == 0) *a.h.skipped = skipped + 1;
    return false;
  }
  if (a.h.lr_dev || a.h.step_dev || skipped) {  // equal for the whole launch
    __shared__ float s_rates[2];
    if (a.h.lr_dev) lr = (double)*a.h.lr_dev;
    if (threadIdx.x < 64) {  // some hundred instructions: for one wavefront
      const int64_t t = max((a.h.step_dev ? *a.h.step_dev : a.h.step) - skipped, (int64_t)1);
      s_rates[0] = (float)(lr / -expm1((double)t * a.log_beta1));
      s_rates[1] = (float)(1.0 / sqrt(-expm1((double)t * a.log_beta2)));
    }
    __syncthreads();
    r.step = s_rates[0];
    r.inv_bc2 = s_rates[1];
  }
  r.keep = (float)(1.0 - lr * (double)decay);
  return true;
}

// The weight after a step, from m' and the root of v' (hardware reciprocal: one in the last
// place, as the root; the step is some percent of a weight at most).
__device__ __forceinline__ float next_weight(float w, float m, float root, const Rates &r, float eps) {
  const float u = m * __builtin_amdgcn_rcpf(root * r.inv_bc2 + eps);
  return w * r.keep - r.step * u;
}

// Values a block, by the states' bits.  32: one group of four a thread; 2048 a block measured 81
// against 77 us on 120 tensors of 12 M values, the same on 176 M.  8: eight a thread.
constexpr int kAdam32Chunk = 1024, kAdamChunk = 2048;

// States in 32 bits: four values a thread.  G: gradients' type; P: parameters'; MASTER:
// the float copy is read instead of the parameter.
template <typename G, typename P, bool MASTER>
__device__ __forceinline__ void adamw32(const Adam32Args &a, const Adam32 &t, const Rates &r, int64_t i0) {
  constexpr int U = kAdam32Chunk / (4 * kThreads);
  const float b1 = (float)a.h.beta1, b2 = (float)a.h.beta2, c1 = (float)(1.0 - a.h.beta1),
              c2 = (float)(1.0 - a.h.beta2), eps = (float)a.h.eps;
  const G *pg = static_cast<const G *>(t.grad);
  P *pp = static_cast<P *>(t.param);
  float *pm = static_cast<float *>(t.m), *pv = static_cast<float *>(t.v);
  auto run = [&](auto whole) {
    Vals<4> g[U], m[U], v[U], w[U];
    int n[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t i = i0 + (k * kThreads + (int)threadIdx.x) * 4;
      n[k] = whole ? 4 : (int)min(max(t.n - i, (int64_t)0), (int64_t)4);
      if (n[k] == 0) continue;
      g[k] = load_n<4>(pg + i, n[k]);
      m[k] = load_n<4>(pm + i, n[k]);
      v[k] = load_n<4>(pv + i, n[k]);
      if constexpr (MASTER)
        w[k] = load_n<4>(t.master + i, n[k]);
      else
        w[k] = load_n<4>(pp + i, n[k]);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t i = i0 + (k * kThreads + (int)threadIdx.x) * 4;
      if (n[k] == 0) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float gs = g[k].v[j] * r.gscale;
        m[k].v[j] = b1 * m[k].v[j] + c1 * gs;
        v[k].v[j] = b2 * v[k].v[j] + c2 * (gs * gs);
        w[k].v[j] = next_weight(w[k].v[j], m[k].v[j], sqrtf(v[k].v[j]), r, eps);
      }
      store_n<4>(pm + i, m[k], n[k]);
      store_n<4>(pv + i, v[k], n[k]);
      if constexpr (MASTER) store_n<4>(t.master + i, w[k], n[k]);
      store_n<4>(pp + i, w[k], n[k]);
    }
  };
  struct Yes { constexpr operator bool() const { return true; } };
  struct No { constexpr operator bool() const { return false; } };
  if (i0 + kAdam32Chunk <= t.n)
    run(Yes{});
  else
    run(No{});
}

// The types are equal for a whole block, so one launch takes tensors of every kind.
#define ADAM_BY_TYPE(F, ...)                                  \
  do {                                                        \
    if (t.master) {                                           \
      if (t.grad_f32)                                         \
        F<float, bf16_t, true>(__VA_ARGS__);                  \
      else                                                    \
        F<bf16_t, bf16_t, true>(__VA_ARGS__);                 \
    } else if (t.param_f32) {                                 \
      if (t.grad_f32)                                         \
        F<float, float, false>(__VA_ARGS__);                  \
      else                                                    \
        F<bf16_t, float, false>(__VA_ARGS__);                 \
    } else {                                                  \
      if (t.grad_f32)                                         \
        F<float, bf16_t, false>(__VA_ARGS__);                 \
      else                                                    \
        F<bf16_t, bf16_t, false>(__VA_ARGS__);                \
    }                                                         \
  } while (0)

__global__ __launch_bounds__(kThreads) void adamw32_kernel(Adam32Args a) {
  const int ti = find_tensor(a.first, a.count);
  const Adam32 t = a.t[ti];
  Rates r;
  if (!rates(a, t.decay, r)) return;
  const int64_t i0 = (int64_t)(blockIdx.x - a.first[ti]) * kAdam32Chunk;
  ADAM_BY_TYPE(adamw32, a, t, r, i0);
}

constexpr double kPerM = 1.0 / 16129.0, kPerV = 1.0 / 4228250625.0;  // 1 / 127^2, 1 / 255^4

// m' and v' in 64 bits from the values held, every operation rounded by itself.
__device__ __forceinline__ double next_m(int code, double scale, double g, double b1, double c1) {
#pragma clang fp contract(off)
  const float c = (float)code;
  const double old = (double)(c * fabsf(c)) * scale;  // the square is exact in a float
  const double a = b1 * old, b = c1 * g;
  return a + b;
}
__device__ __forceinline__ double next_v(uint32_t code, double scale, double g, double b2, double c2) {
#pragma clang fp contract(off)
  const float c = (float)code;
  const double square = (double)(c * c);  // exact, and its own square in 64 bits too
  const double old = (square * square) * scale;
  const double gg = g * g;
  const double a = b2 * old, b = c2 * gg;
  return a + b;
}

// The code whose square is nearest to u, from u as a float within `off` of it, relative: the
// c with c (c - 1) + 1/2 <= u < c (c + 1) + 1/2.  `sure` is cleared where a border is that
// near, and 64 bits have to decide.
__device__ __forceinline__ float nearest_root(float u, float off, bool &sure) {
  const float c = rintf(__builtin_amdgcn_sqrtf(fabsf(u - 0.25f)));
  // distance from the nearer border; code 0 has none below it
  const float inside = fmaxf(c - fabsf((u - c * c) - 0.5f), 0.4f - u);
  sure = sure && inside > off * u;
  return c;
}
// The same from u in 64 bits, `at(x)` saying whether it is at or past the border x (u itself
// may be held squared there).
template <typename At>
__device__ __forceinline__ int nearest_root_64(float u, int top, At at) {
  int c = min((int)rintf(__builtin_amdgcn_sqrtf(fabsf(u - 0.25f))), top);
  if (c > 0 && !at((double)(c * (c - 1)) + 0.5))
    --c;
  else if (c < top && at((double)(c * (c + 1)) + 0.5))
    ++c;
  return c;
}

// Largest of 32 neighbouring lanes' values, in every lane.
template <int CTRL>
__device__ __forceinline__ uint32_t lane_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ uint32_t max32(uint32_t v) {
  v = lane_max<0xb1>(v);   // lane ^ 1
  v = lane_max<0x4e>(v);   // lane ^ 2
  v = lane_max<0x141>(v);  // the halves of 8
  v = lane_max<0x140>(v);  // the halves of 16
  const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return max((uint32_t)r[0], (uint32_t)r[1]);
}

// The scale held for a block whose largest magnitude has these bits: zero below the smallest
// normal float, NaN for a block with a value that is not finite.
__device__ __forceinline__ float held_scale(uint32_t bits) {
  if (bits >= 0x7f800000u) return NAN;
  return bits < 0x00800000u ? 0.f : __uint_as_float(bits);
}

// Codes of eight neighbouring values.  They are a small part of the traffic, and cached: what
// reads the states next finds them there (13 M values, step and states read back: 60 against 69
// us past the caches).  A step alone does not care: 13 M values 39.9 against 38.5 us, with a float
// copy 42.9 against 43.3; 201 M 497 against 497, with a copy 595 against 587.
struct Codes {
  uint32_t w[2];
  __device__ __forceinline__ uint32_t u(int j) const { return (w[j >> 2] >> (8 * (j & 3))) & 0xffu; }
  __device__ __forceinline__ void put(int j, int c) { w[j >> 2] |= ((uint32_t)c & 0xffu) << (8 * (j & 3)); }
  __device__ __forceinline__ int s(int j) const { return (int)(w[j >> 2] << (24 - 8 * (j & 3))) >> 24; }
};
__device__ __forceinline__ Codes load_codes(const uint8_t *p, int n) {
  Codes c{{0u, 0u}};
  if (n >= 8) {
    const u32x2 q = *reinterpret_cast<const u32x2 *>(p);
    c.w[0] = q[0];
    c.w[1] = q[1];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) c.w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
  }
  return c;
}
__device__ __forceinline__ void store_codes(uint8_t *p, const Codes &c, int n) {
  if (n >= 8) {
    *reinterpret_cast<u32x2 *>(p) = u32x2{c.w[0], c.w[1]};
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = (uint8_t)c.u(j);
  }
}

// States in 8 bits: eight values a thread, 32 threads a block of 256 values.
template <typename G, typename P, bool MASTER>
__device__ __forceinline__ void adamw8(const Adam8Args &a, const Adam8 &t, const Rates &r, int64_t i0) {
  const double b1 = a.h.beta1, b2 = a.h.beta2, c1 = 1.0 - b1, c2 = 1.0 - b2;
  const float eps = (float)a.h.eps;
  const int64_t i = i0 + threadIdx.x * 8, q = i / kAdamBlock;
  const int n = (int)min(max(t.n - i, (int64_t)0), (int64_t)8);
  uint8_t *pm = static_cast<uint8_t *>(t.m) + i, *pv = static_cast<uint8_t *>(t.v) + i;
  P *pp = static_cast<P *>(t.param) + i;
  Vals<8> g{}, w{};
  Codes cm{{0u, 0u}}, cv{{0u, 0u}};
  double sm = 0, sv = 0;
  if (n > 0) {
    g = load_n<8>(static_cast<const G *>(t.grad) + i, n);
    cm = load_codes(pm, n);
    cv = load_codes(pv, n);
    if constexpr (MASTER)
      w = load_n<8>(t.master + i, n);
    else
      w = load_n<8>(pp, n);
    sm = (double)t.m_scale[q] * kPerM;
    sv = (double)t.v_scale[q] * kPerV;
  }
  // (values past the tensor's end stay zero here)
  double m[8], v[8];
  uint32_t bm = 0, bv = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const double gs = (double)g.v[j] * (double)r.gscale;
    m[j] = next_m(cm.s(j), sm, gs, b1, c1);
    v[j] = next_v(cv.u(j), sv, gs, b2, c2);
    bm = max(bm, __float_as_uint((float)m[j]) & 0x7fffffffu);
    bv = max(bv, __float_as_uint((float)v[j]) & 0x7fffffffu);
  }
  const float hm = held_scale(max32(bm)), hv = held_scale(max32(bv));
  if (n <= 0) return;
  if ((threadIdx.x & 31) == 0) {
    t.m_scale[q] = hm;
    t.v_scale[q] = hv;
  }
  // Roots are taken of v' times 2^64 unless the block's largest would leave the floats, so that the
  // smallest floats, which the instruction takes for zeros, do not come up (they would beside an
  // eps below 1e-12).  Powers of two: the same roots otherwise.
  const bool small = hv < 0x1p60f;
  const double up = small ? 0x1p64 : 1.0;
  Rates rr = r;
  rr.inv_bc2 = small ? r.inv_bc2 * 0x1p-32f : r.inv_bc2;
  // u as floats.  |m'| 127^2 / scale: the reciprocal (one in the last place), two products and
  // m' rounded, at most 3e-7; for v' the root of v' times 255^2 over the root of scale: two
  // instructions of one in the last place, two products and half of v's rounding, at most
  // 4e-7.  A scale of m so small or large that its reciprocal leaves the normal floats is for 64
  // bits (a reciprocal below them is taken for zero).
  const bool none_m = !(hm > 0.f), none_v = !(hv > 0.f);  // zero or NaN: codes of zero
  const float imf = none_m ? 0.f : 16129.f * __builtin_amdgcn_rcpf(hm);
  const float ivf = none_v ? 0.f : 65025.f * __builtin_amdgcn_rsqf(hv) * (small ? 0x1p-32f : 1.f);
  bool sure_m = none_m || (hm > 0x1p-90f && hm < 0x1p120f), sure_v = true;
  Codes nm{{0u, 0u}}, nv{{0u, 0u}};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float mf = (float)m[j], root = __builtin_amdgcn_sqrtf((float)(v[j] * up));
    w.v[j] = next_weight(w.v[j], mf, root, rr, eps);
    nm.put(j, (int)copysignf(nearest_root(fabsf(mf) * imf, 4e-7f, sure_m), mf));
    const float c = nearest_root(root * ivf, 6e-7f, sure_v);
    nv.put(j, (int)fmaxf(c, v[j] > 0 ? 1.f : 0.f));
  }
  if (none_m) nm = Codes{{0u, 0u}};
  if (none_v) nv = Codes{{0u, 0u}};
  if (!sure_m && !none_m) {
    const double im = 16129.0 / (double)hm;
    nm = Codes{{0u, 0u}};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double u = fabs(m[j]) * im;
      const int c = nearest_root_64((float)u, 127, [&](double x) { return u >= x; });
      nm.put(j, m[j] < 0 ? -c : c);
    }
  }
  if (!sure_v && !none_v) {
    const double iv = 4228250625.0 / (double)hv;
    nv = Codes{{0u, 0u}};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double uu = v[j] * iv;
      const int c = nearest_root_64(__builtin_amdgcn_sqrtf((float)uu), 255, [&](double x) { return uu >= x * x; });
      nv.put(j, max(c, v[j] > 0 ? 1 : 0));
    }
  }
  if constexpr (MASTER) store_n<8>(t.master + i, w, n);
  store_n<8>(pp, w, n);
  store_codes(pm, nm, n);
  store_codes(pv, nv, n);
}

__global__ __launch_bounds__(kThreads) void adamw8_kernel(Adam8Args a) {
  const int ti = find_tensor(a.first, a.count);
  const Adam8 t = a.t[ti];
  Rates r;
  if (!rates(a, t.decay, r)) return;
  const int64_t i0 = (int64_t)(blockIdx.x - a.first[ti]) * kAdamChunk;
  ADAM_BY_TYPE(adamw8, a, t, r, i0);
}
#undef ADAM_BY_TYPE

// ------------------------------------------------------------- 8-bit states read as floats

struct ReadTensor {
  const uint8_t *m, *v;
  const float *m_scale, *v_scale;
  float *m_out, *v_out;
  int64_t n;
};
constexpr int kReadTensors = 64;
struct ReadArgs {
  ReadTensor t[kReadTensors];
  int32_t first[kReadTensors];
  int32_t count;
};
static_assert(sizeof(ReadArgs) <= 4096, "kernel arguments");

// Four values a thread, twice.
__global__ __launch_bounds__(kThreads) void adamw_read_kernel(ReadArgs a) {
  const int ti = find_tensor(a.first, a.count);
  const ReadTensor t = a.t[ti];
  const int64_t i0 = (int64_t)(blockIdx.x - a.first[ti]) * kAdamChunk;
#pragma unroll
  for (int k = 0; k < kAdamChunk / (4 * kThreads); ++k) {
    const int64_t i = i0 + (k * kThreads + (int)threadIdx.x) * 4, q = i / kAdamBlock;
    const int n = (int)min(max(t.n - i, (int64_t)0), (int64_t)4);
    if (n == 0) continue;
    auto codes = [&](const uint8_t *p) {
      uint32_t w = 0;
      if (n == 4) return *reinterpret_cast<const uint32_t *>(p + i);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n) w |= (uint32_t)p[i + j] << (8 * j);
      return w;
    };
    if (t.m_out) {
      const uint32_t w = codes(t.m);
      const double scale = (double)t.m_scale[q] * kPerM;
      Vals<4> x;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float c = (float)((int)(w << (24 - 8 * j)) >> 24);
        x.v[j] = (float)((double)(c * fabsf(c)) * scale);
      }
      store_n<4>(t.m_out + i, x, n);
    }
    if (t.v_out) {
      const uint32_t w = codes(t.v);
      const double scale = (double)t.v_scale[q] * kPerV;
      Vals<4> x;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float c = (float)((w >> (8 * j)) & 0xffu);
        const double square = (double)(c * c);
        x.v[j] = (float)((square * square) * scale);
      }
      store_n<4>(t.v_out + i, x, n);
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
    a.grad[a.count] = t[i].grad;
    a.n[a.count] = t[i].f32 ? ~t[i].n : t[i].n;
    a.first[a.count++] = (int32_t)blocks;
    blocks += nb;
  }
  hipError_t e = flush();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(grad_norm_finish_kernel, dim3(1), dim3(1024), 0, s, part, done, max_norm, out);
  return hipGetLastError();
}

namespace {

Adam32 as_argument(const AdamTensor &t, Adam32 *) {
  return Adam32{t.param, t.grad, t.master, t.m, t.v, t.n, t.decay, t.param_f32, t.grad_f32, {0, 0}};
}
Adam8 as_argument(const AdamTensor &t, Adam8 *) {
  return Adam8{as_argument(t, static_cast<Adam32 *>(nullptr)), t.m_scale, t.v_scale};
}

// Whether any value of the tensors has its states in 8 (or in 32) bits.
bool any_of_kind(bool eight, const AdamTensor *t, int count) {
  return std::any_of(t, t + count, [&](const AdamTensor &x) { return x.eight == eight && x.n > 0; });
}

// Launches for the tensors with 32-bit or with 8-bit states.  last: no launch of the step follows.
template <typename Tensor, int N>
hipError_t launch_adamw_of(void (*kernel)(AdamArgs<Tensor, N>), bool eight, int64_t chunk, const AdamTensor *t,
                           int count, const AdamScalars &h, bool last, hipStream_t s) {
  if (!any_of_kind(eight, t, count)) return hipSuccess;
  AdamArgs<Tensor, N> a{};
  a.h = h;
  a.log_beta1 = std::log(h.beta1);
  a.log_beta2 = std::log(h.beta2);
  a.step = (float)(h.lr / (1.0 - std::pow(h.beta1, (double)h.step)));
  a.inv_bc2 = (float)(1.0 / std::sqrt(1.0 - std::pow(h.beta2, (double)h.step)));
  int64_t blocks = 0;
  auto flush = [&]() -> hipError_t {
    if (a.count == 0) return hipSuccess;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
    blocks = 0;
    a.count = 0;
    return hipGetLastError();
  };
  for (int i = 0; i < count; ++i) {
    if (t[i].eight != eight || t[i].n == 0) continue;
    const int64_t nb = (t[i].n + chunk - 1) / chunk;
    if (a.count == N || blocks + nb > kMaxBlocks) {
      const hipError_t e = flush();
      if (e != hipSuccess) return e;
    }
    a.t[a.count] = as_argument(t[i], static_cast<Tensor *>(nullptr));
    a.first[a.count++] = (int32_t)blocks;
    blocks += nb;
  }
  a.last = last;
  return flush();
}

}  // namespace

hipError_t launch_adamw(const AdamTensor *t, int count, const AdamScalars &h, hipStream_t s) {
  const hipError_t e =
      launch_adamw_of(adamw32_kernel, false, kAdam32Chunk, t, count, h, !any_of_kind(true, t, count), s);
  if (e != hipSuccess) return e;
  return launch_adamw_of(adamw8_kernel, true, kAdamChunk, t, count, h, true, s);
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
    if (a.count == kReadTensors || blocks + nb > kMaxBlocks) {
      const hipError_t e = flush();
      if (e != hipSuccess) return e;
    }
    a.t[a.count] = ReadTensor{static_cast<const uint8_t *>(t[i].m), static_cast<const uint8_t *>(t[i].v),
                              t[i].m_scale, t[i].v_scale, mo, vo, t[i].n};
    a.first[a.count++] = (int32_t)blocks;
    blocks += nb;
  }
  return flush();
}

}  // namespace moe
