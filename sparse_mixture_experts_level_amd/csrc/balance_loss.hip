// Load-balancing loss with its gradient, the router's z loss and per-expert counts
// ("Sparse Mixture-of-Experts", bigdataschool.ru wiki, section "Маршрутизация токена и
// auxiliary loss": alpha times the number of experts times the sum over experts of
// f_i * P_i), per sequence of a ragged batch.  For sequence s with its N_s counted tokens:
//   p_t = softmax(l_t),  z_t = log sum_i exp(l_ti),
//   f_si = c_si / (k N_s),  P_si = 1/N_s sum_t p_ti,
//   balance = alpha E / S' sum_s sum_i f_si P_si,   z loss = beta / N sum_t z_t^2,
//   d/dl_ti = p_ti (alpha E / (S' N_s) (f_si - sum_j f_sj p_tj) + 2 beta / N z_t)
// (f is piecewise constant in the logits; S' sequences count a token, N tokens in all).
// The gradient needs the counts but not the probabilities' means, so one pass over the
// logits gives both: it is bound by reading the logits and writing the gradient once.
// Every sum has a fixed order (bit-reproducible); counts are whole numbers.
#include <algorithm>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr int BL_COUNT_THREADS = 1024;

struct Span {
  int seq;    // -1: none
  int first;  // index of the sequence's first chunk
  int begin, end;
};

__device__ __forceinline__ void seq_range(const int32_t *off, int T, int s, int &b, int &e) {
  if (!off) {
    b = 0;
    e = T;
    return;
  }
  // offsets outside [0, T] or running backwards (a caller's mistake) stay inside the tables
  b = min(max(off[s], 0), T);
  e = min(max(off[s + 1], b), T);
}

// Chunk `lin` when every sequence is cut into pieces of `chunk` tokens, numbered sequence
// after sequence; total chunks in `total` when the chunk is past the last.  One wavefront
// scans the offsets; equal in every lane.
__device__ __forceinline__ Span find_span(const int32_t *off, int S, int T, int chunk, int lin, int &total) {
  Span r{-1, 0, 0, 0};
  if (S == 1) {
    int b, e;
    seq_range(off, T, 0, b, e);
    total = (e - b + chunk - 1) / chunk;
    if (lin < total) r = Span{0, 0, b + lin * chunk, min(e, b + (lin + 1) * chunk)};
    return r;
  }
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int s0 = 0; s0 < S; s0 += 64) {
    const int s = s0 + lane;
    int b = 0, e = 0;
    if (s < S) seq_range(off, T, s, b, e);
    const int n = (e - b + chunk - 1) / chunk;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o, 64);
      if (lane >= o) incl += v;
    }
    const uint64_t hit = __ballot(base + incl > lin);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      r.seq = s0 + l;
      r.first = base + __shfl(incl - n, l, 64);
      const int sb = __shfl(b, l, 64), se = __shfl(e, l, 64);
      r.begin = sb + (lin - r.first) * chunk;
      r.end = min(se, r.begin + chunk);
      return r;
    }
    base += __shfl(incl, 63, 64);
  }
  total = base;
  return r;
}

// Counts of one chunk: part[block][0..E-1] choices, part[block][E] counted tokens.  Each
// expert has `copies` bins, taken by lane, so that a wavefront whose tokens all chose one
// expert does not add 64 times to one address.
__global__ __launch_bounds__(BL_COUNT_THREADS) void balance_count_kernel(const int32_t *__restrict__ ids,
                                                                         const uint8_t *__restrict__ mask,
                                                                         const int32_t *__restrict__ off, int T, int E,
                                                                         int k, int S, int chunk, int copies,
                                                                         int32_t *__restrict__ part) {
  extern __shared__ int32_t s_bins[];  // [copies][E], then 1
  int total = 0;
  const Span sp = find_span(off, S, T, chunk, blockIdx.x, total);
  if (sp.seq < 0) return;  // equal in every thread
  for (int i = threadIdx.x; i < copies * E + 1; i += BL_COUNT_THREADS) s_bins[i] = 0;
  __syncthreads();
  int32_t *bins = s_bins + (threadIdx.x & (copies - 1)) * E;
  const int64_t i0 = (int64_t)sp.begin * k, i1 = (int64_t)sp.end * k;
  for (int64_t i = i0 + threadIdx.x; i < i1; i += BL_COUNT_THREADS) {
    const int t = (int)(i / k);
    const int e = ids[i];
    if (mask && mask[t] == 0) continue;
    if (e >= 0 && e < E) atomicAdd(&bins[e], 1);
  }
  int mine = 0;
  for (int t = sp.begin + (int)threadIdx.x; t < sp.end; t += BL_COUNT_THREADS) mine += !mask || mask[t] != 0;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) mine += __shfl_xor(mine, o, 64);
  if ((threadIdx.x & 63) == 0 && mine) atomicAdd(&s_bins[copies * E], mine);
  __syncthreads();
  int32_t *out = part + (size_t)blockIdx.x * (E + 1);
  for (int e = threadIdx.x; e < E; e += BL_COUNT_THREADS) {
    int c = 0;
    for (int q = 0; q < copies; ++q) c += s_bins[q * E + e];
    out[e] = c;
  }
  if (threadIdx.x == 0) out[E] = s_bins[copies * E];
}

// One block a sequence: its counts and counted tokens from the chunks', and the index of its
// first block of the main pass.
__global__ __launch_bounds__(256) void balance_tables_kernel(const int32_t *__restrict__ off, int T, int E, int S,
                                                             int chunk, int main_chunk, int blocks, int main_blocks,
                                                             const int32_t *__restrict__ part,
                                                             int32_t *__restrict__ counts,
                                                             int32_t *__restrict__ seq_tokens,
                                                             int32_t *__restrict__ first_main) {
  const int s = blockIdx.x;
  const int lane = threadIdx.x & 63;
  int first = 0, fm = 0;
  for (int q = lane; q < s; q += 64) {
    int b, e;
    seq_range(off, T, q, b, e);
    first += (e - b + chunk - 1) / chunk;
    fm += (e - b + main_chunk - 1) / main_chunk;
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    first += __shfl_xor(first, o, 64);
    fm += __shfl_xor(fm, o, 64);
  }
  int b, e;
  seq_range(off, T, s, b, e);
  const int n = (e - b + chunk - 1) / chunk;
  for (int i = threadIdx.x; i <= E; i += 256) {
    int c = 0;
    // (offsets that run backwards could name more chunks than there are)
    for (int q = 0; q < n && first + q < blocks; ++q) c += part[(size_t)(first + q) * (E + 1) + i];
    if (i < E)
      counts[(size_t)s * E + i] = c;
    else
      seq_tokens[s] = c;
  }
  if (threadIdx.x == 0) {
    first_main[s] = min(fm, main_blocks);
    if (s == S - 1) first_main[S] = min(fm + (e - b + main_chunk - 1) / main_chunk, main_blocks);
  }
}

struct BalanceArgs {
  const float *logits;
  const uint8_t *mask;
  const int32_t *off;
  const int32_t *counts;
  const int32_t *seq_tokens;
  const float *dloss;  // upstream gradients of the two losses, or NULL (ones)
  float *dlogits;      // or NULL
  float *part;         // [blocks][E]: column sums of p
  double *zpart;       // [blocks]: sums of z^2 (a finite z's square can pass the largest float)
  int T, E, k, S, chunk;
  float alpha, beta;
};

// A token's row in LPT lanes of NV groups of four values each; 64 / LPT tokens a wavefront.
// With VEC (E a multiple of 4) a group is one 16-byte load; otherwise its values lie LPT
// apart, so that each load of a group still covers neighbouring words.
template <int LPT, int NV, bool VEC, bool LOSS>
__global__ __launch_bounds__(256) void balance_main_kernel(BalanceArgs a) {
  constexpr int TPW = 64 / LPT;
  __shared__ float s_acc[LOSS ? 4 : 1][LOSS ? LPT * NV * 4 : 1];
  __shared__ double s_z[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int li = lane & (LPT - 1), sub = lane / LPT;
  const int E = a.E;
  auto expert = [&](int v, int i) { return VEC ? 4 * (li + LPT * v) + i : li + LPT * (4 * v + i); };
  int total = 0;
  const Span sp = find_span(a.off, a.S, a.T, a.chunk, blockIdx.x, total);
  if (sp.seq < 0) {
    // blocks past the last chunk: rows outside every sequence get a zero gradient
    if (a.dlogits && a.off) {
      int b0, e0, b1, e1;
      seq_range(a.off, a.T, 0, b0, e0);
      seq_range(a.off, a.T, a.S - 1, b1, e1);
      const int64_t lead = (int64_t)b0 * E, tail = (int64_t)(a.T - e1) * E;
      const int64_t step = (int64_t)(gridDim.x - total) * 256;
      for (int64_t i = (int64_t)(blockIdx.x - total) * 256 + threadIdx.x; i < lead + tail; i += step)
        a.dlogits[i < lead ? i : i - lead + (int64_t)e1 * E] = 0.f;
    }
    return;
  }
  // sequences that count a token, tokens in all
  int live = 0, all = 0;
  for (int s = lane; s < a.S; s += 64) {
    const int n = a.seq_tokens[s];
    live += n > 0;
    all += n;
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    live += __shfl_xor(live, o, 64);
    all += __shfl_xor(all, o, 64);
  }
  const int ns = a.seq_tokens[sp.seq];
  const float up0 = a.dloss ? a.dloss[0] : 1.f, up1 = a.dloss ? a.dloss[1] : 1.f;
  const float ca = up0 * (a.alpha * (float)E / ((float)max(live, 1) * (float)max(ns, 1)));
  const float cb = up1 * (2.f * a.beta / (float)max(all, 1));
  const float fden = (float)max(ns, 1) * (float)a.k;
  float f[NV][4], acc[NV][4];
  double zacc = 0.;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = expert(v, i);
      f[v][i] = e < E ? (float)a.counts[(size_t)sp.seq * E + e] / fden : 0.f;
      acc[v][i] = 0.f;
    }
  for (int t0 = sp.begin + wave * TPW; t0 < sp.end; t0 += 4 * TPW) {
    const int t = t0 + sub;
    const bool in = t < sp.end;
    const bool counted = in && (!a.mask || a.mask[t] != 0);
    const float *row = a.logits + (size_t)t * E;
    float l[NV][4];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if constexpr (VEC) {
        f32x4 q = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (counted && expert(v, 0) < E) q = *reinterpret_cast<const f32x4 *>(row + expert(v, 0));
#pragma unroll
        for (int i = 0; i < 4; ++i) l[v][i] = q[i];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) l[v][i] = counted && expert(v, i) < E ? row[expert(v, i)] : -INFINITY;
      }
    }
    float m = -INFINITY;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) m = fmaxf(m, l[v][i]);
#pragma unroll
    for (int o = LPT / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
    // a row without any finite logit (or an uncounted one) has sum 0: no probabilities
    const float base = m == -INFINITY ? 0.f : m;
    float sum = 0.f, dot = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        l[v][i] = __expf(l[v][i] - base);
        sum += l[v][i];
        dot += l[v][i] * f[v][i];
      }
#pragma unroll
    for (int o = LPT / 2; o >= 1; o >>= 1) {
      sum += __shfl_xor(sum, o, 64);
      dot += __shfl_xor(dot, o, 64);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const float z = sum == 0.f ? 0.f : base + __logf(sum);
    dot *= inv;
    if constexpr (LOSS) zacc += li == 0 ? (double)z * (double)z : 0.;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        l[v][i] *= inv;
        if constexpr (LOSS) acc[v][i] += l[v][i];
      }
    if (a.dlogits && in) {
      float *drow = a.dlogits + (size_t)t * E;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        f32x4 q;
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = l[v][i] * (ca * (f[v][i] - dot) + cb * z);
        if constexpr (VEC) {
          if (expert(v, 0) < E) *reinterpret_cast<f32x4 *>(drow + expert(v, 0)) = q;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (expert(v, i) < E) drow[expert(v, i)] = q[i];
        }
      }
    }
  }
  if constexpr (LOSS) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int o = LPT; o < 64; o <<= 1) acc[v][i] += __shfl_xor(acc[v][i], o, 64);
        if (sub == 0 && expert(v, i) < E) s_acc[wave][expert(v, i)] = acc[v][i];
      }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) zacc += __shfl_xor(zacc, o, 64);
    if (lane == 0) s_z[wave] = zacc;
    __syncthreads();
    if (threadIdx.x == 0) a.zpart[blockIdx.x] = (s_z[0] + s_z[1]) + (s_z[2] + s_z[3]);
    float *out = a.part + (size_t)blockIdx.x * E;
    for (int e = threadIdx.x; e < E; e += 256) out[e] = (s_acc[0][e] + s_acc[1][e]) + (s_acc[2][e] + s_acc[3][e]);
  }
}

// One block: the mean probabilities and the two losses from the main pass's partial sums, in
// 64 bits.
__global__ __launch_bounds__(1024) void balance_finish_kernel(const float *__restrict__ part,
                                                              const double *__restrict__ zpart,
                                                              const int32_t *__restrict__ first_main,
                                                              const int32_t *__restrict__ counts,
                                                              const int32_t *__restrict__ seq_tokens, int E, int k,
                                                              int S, float alpha, float beta,
                                                              float *__restrict__ mean_probs,
                                                              float *__restrict__ losses) {
  __shared__ double s_bal[1024], s_z[1024];
  __shared__ int s_live, s_all;
  if (threadIdx.x == 0) s_live = s_all = 0;
  __syncthreads();
  int live = 0, all = 0;
  for (int s = threadIdx.x; s < S; s += 1024) {
    live += seq_tokens[s] > 0;
    all += seq_tokens[s];
  }
  if (live) atomicAdd(&s_live, live);
  if (all) atomicAdd(&s_all, all);
  double bal = 0, z = 0;
  for (int64_t i = threadIdx.x; i < (int64_t)S * E; i += 1024) {
    const int s = (int)(i / E), e = (int)(i - (int64_t)s * E);
    double p = 0;
    for (int b = first_main[s]; b < first_main[s + 1]; ++b) p += part[(size_t)b * E + e];
    const int n = seq_tokens[s];
    const double P = n > 0 ? p / n : 0.0;
    mean_probs[i] = (float)P;
    if (n > 0) bal += P * ((double)counts[i] / ((double)n * k));
  }
  for (int b = threadIdx.x; b < first_main[S]; b += 1024) z += zpart[b];
  s_bal[threadIdx.x] = bal;
  s_z[threadIdx.x] = z;
  __syncthreads();
  for (int o = 512; o >= 1; o >>= 1) {
    if (threadIdx.x < o) {
      s_bal[threadIdx.x] += s_bal[threadIdx.x + o];
      s_z[threadIdx.x] += s_z[threadIdx.x + o];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    losses[0] = (float)((double)alpha * E * s_bal[0] / max(s_live, 1));
    losses[1] = (float)((double)beta * s_z[0] / max(s_all, 1));
  }
}

int count_chunk(int T) { return std::max(1024, (T + 63) / 64); }
int main_chunk(int T) { return std::max(32, (T + 511) / 512); }

// Chunks of the two passes: sequences cut into whole chunks, at most one partial chunk each,
// and in the main pass one block more for the rows outside every sequence.
int count_blocks(int T, int S, bool off) { return (T + count_chunk(T) - 1) / count_chunk(T) + (off ? S : 0); }
int main_blocks(int T, int S, bool off) { return (T + main_chunk(T) - 1) / main_chunk(T) + (off ? S + 1 : 0); }

template <bool LOSS>
hipError_t launch_main(const BalanceArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)main_blocks(a.T, a.S, a.off != nullptr));
  const int E = a.E;
#define BL_CASE(L, N)                                                                             \
  do {                                                                                            \
    if (E % 4 == 0)                                                                               \
      hipLaunchKernelGGL((balance_main_kernel<L, N, true, LOSS>), grid, dim3(256), 0, s, a);      \
    else                                                                                          \
      hipLaunchKernelGGL((balance_main_kernel<L, N, false, LOSS>), grid, dim3(256), 0, s, a);     \
    return hipGetLastError();                                                                     \
  } while (0)
  if (E <= 4) BL_CASE(1, 1);
  if (E <= 8) BL_CASE(2, 1);
  if (E <= 16) BL_CASE(4, 1);
  if (E <= 32) BL_CASE(8, 1);
  if (E <= 64) BL_CASE(16, 1);
  if (E <= 128) BL_CASE(32, 1);
  if (E <= 256) BL_CASE(64, 1);
  if (E <= 512) BL_CASE(64, 2);
  BL_CASE(64, 4);
#undef BL_CASE
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

struct BalanceWs {
  size_t count_part, main_part, z_part, first_main, total;
};
BalanceWs balance_ws(int T, int E, int S) {
  BalanceWs w;
  const size_t cb = count_blocks(T, S, true), mb = main_blocks(T, S, true);
  w.count_part = 0;
  w.main_part = align256(cb * (E + 1) * 4);
  w.z_part = w.main_part + align256(mb * E * 4);
  w.first_main = w.z_part + align256(mb * 8);
  w.total = w.first_main + align256(((size_t)S + 1) * 4);
  return w;
}

}  // namespace

size_t balance_workspace_bytes(int T, int E, int S) { return balance_ws(T, E, S).total; }

hipError_t launch_balance_loss(const BalanceCall &c, int32_t *counts, int32_t *seq_tokens, float *mean_probs,
                               float *losses, void *ws, hipStream_t s) {
  const BalanceWs w = balance_ws(c.T, c.E, c.S);
  uint8_t *base = static_cast<uint8_t *>(ws);
  int32_t *cpart = reinterpret_cast<int32_t *>(base + w.count_part);
  float *mpart = reinterpret_cast<float *>(base + w.main_part);
  double *zpart = reinterpret_cast<double *>(base + w.z_part);
  int32_t *first_main = reinterpret_cast<int32_t *>(base + w.first_main);
  const int cc = count_chunk(c.T), mc = main_chunk(c.T);
  const int cb = count_blocks(c.T, c.S, c.off != nullptr), mb = main_blocks(c.T, c.S, c.off != nullptr);
  int copies = 1;
  while (copies < 64 && copies * 2 * c.E <= 4096) copies *= 2;
  hipLaunchKernelGGL(balance_count_kernel, dim3((unsigned)cb), dim3(BL_COUNT_THREADS),
                     (copies * c.E + 1) * 4, s, c.ids, c.mask, c.off, c.T, c.E, c.k, c.S, cc, copies, cpart);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(balance_tables_kernel, dim3((unsigned)c.S), dim3(256), 0, s, c.off, c.T, c.E, c.S, cc, mc, cb, mb, cpart,
                     counts, seq_tokens, first_main);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  BalanceArgs a{c.logits, c.mask, c.off, counts, seq_tokens, c.dloss, c.dlogits, mpart, zpart, c.T, c.E, c.k, c.S, mc,
                c.alpha,  c.beta};
  e = launch_main<true>(a, s);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(balance_finish_kernel, dim3(1), dim3(1024), 0, s, mpart, zpart, first_main, counts, seq_tokens, c.E, c.k,
                     c.S, c.alpha, c.beta, mean_probs, losses);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceCall &c, const int32_t *counts, const int32_t *seq_tokens,
                                   hipStream_t s) {
  BalanceArgs a{c.logits, c.mask, c.off, counts, seq_tokens, c.dloss, c.dlogits, nullptr, nullptr, c.T, c.E, c.k, c.S,
                main_chunk(c.T), c.alpha, c.beta};
  return launch_main<false>(a, s);
}

}  // namespace moe
