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
constexpr int BL_WAVES = 4, BL_THREADS = 64 * BL_WAVES;  // main pass
constexpr int BL_BINS = 4096;                            // LDS bins of a block that counts

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

// Reductions over groups of LPT neighbouring lanes, the result in every lane: lane moves
// within a row of 16 (lane ^ 1, lane ^ 2, then half-row and row mirrors, which pair equal
// values), then rows and halves of the wavefront exchanged.  T: a 32-bit type.
template <int CTRL, typename T>
__device__ __forceinline__ T lane_move(T v) {
  return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
template <int LPT, typename T, typename Op>
__device__ __forceinline__ T group_reduce(T v, Op op) {
  if constexpr (LPT >= 2) v = op(v, lane_move<0xb1>(v));
  if constexpr (LPT >= 4) v = op(v, lane_move<0x4e>(v));
  if constexpr (LPT >= 8) v = op(v, lane_move<0x141>(v));
  if constexpr (LPT >= 16) v = op(v, lane_move<0x140>(v));
  if constexpr (LPT >= 32) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = op(__builtin_bit_cast(T, (uint32_t)r[0]), __builtin_bit_cast(T, (uint32_t)r[1]));
  }
  if constexpr (LPT >= 64) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    v = op(__builtin_bit_cast(T, (uint32_t)r[0]), __builtin_bit_cast(T, (uint32_t)r[1]));
  }
  return v;
}
constexpr auto add = [](auto x, auto y) { return x + y; };

// Sum of each value over the block's threads, returned to thread 0 (s_red: two doubles a wave).
// STEP: only lanes that are multiples of it hold anything.
template <int WAVES, int STEP = 1>
__device__ __forceinline__ void block_sum2(double &x, double &y, double (*s_red)[2]) {
#pragma unroll
  for (int o = 32; o >= STEP; o >>= 1) {
    x += __shfl_xor(x, o, 64);
    y += __shfl_xor(y, o, 64);
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) {
    s_red[threadIdx.x >> 6][0] = x;
    s_red[threadIdx.x >> 6][1] = y;
  }
  __syncthreads();
  x = y = 0;
  if (threadIdx.x == 0)
    for (int w = 0; w < WAVES; ++w) {
      x += s_red[w][0];
      y += s_red[w][1];
    }
}

// ---------------------------------------------------------------------------------- counts

// Choices and counted tokens of tokens [begin, end) into bins in LDS: bins[copies][E], then
// one for the tokens.  Each expert has `copies` bins, taken by lane, so that a wavefront whose
// tokens all chose one expert does not add 64 times to one address.  Ends synchronised, with
// the experts' sums in bins[0 .. E - 1] and the tokens in bins[copies * E].
template <int THREADS>
__device__ __forceinline__ void count_chunk_lds(int32_t *bins, int copies, const int32_t *ids, const uint8_t *mask,
                                                int begin, int end, int E, int k) {
  for (int i = threadIdx.x; i < copies * E + 1; i += THREADS) bins[i] = 0;
  __syncthreads();
  int32_t *mine = bins + (threadIdx.x & (copies - 1)) * E;
  const int32_t *src = ids + (size_t)begin * k;
  const uint32_t n = (uint32_t)(end - begin) * (uint32_t)k;
  int tokens = 0;
  constexpr int B = 8;  // loads in flight
  for (uint32_t i0 = threadIdx.x; i0 < n; i0 += B * THREADS) {
    int e[B];
#pragma unroll
    for (int j = 0; j < B; ++j) e[j] = i0 + j * THREADS < n ? src[i0 + j * THREADS] : -1;
    if (mask) {
      uint8_t in[B];
#pragma unroll
      for (int j = 0; j < B; ++j)
        in[j] = i0 + j * THREADS < n ? mask[begin + (i0 + j * THREADS) / (uint32_t)k] : 0;
#pragma unroll
      for (int j = 0; j < B; ++j) e[j] = in[j] ? e[j] : -1;
    }
#pragma unroll
    for (int j = 0; j < B; ++j)
      if (e[j] >= 0 && e[j] < E) atomicAdd(&mine[e[j]], 1);
  }
  if (mask) {
    for (int t = begin + (int)threadIdx.x; t < end; t += THREADS) tokens += mask[t] != 0;
  } else if (threadIdx.x == 0) {
    tokens = end - begin;
  }
  tokens = group_reduce<64>(tokens, add);
  if ((threadIdx.x & 63) == 0 && tokens) atomicAdd(&bins[copies * E], tokens);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += THREADS) {
    int c = 0;
    for (int q = 0; q < copies; ++q) c += bins[q * E + e];
    bins[e] = c;  // column e belongs to this thread
  }
  __syncthreads();
}

// What a counting block wrote: its sequence (-1: none) and the tokens it counted there.
struct ChunkTokens {
  int32_t seq, tokens;
};

// Counts of one chunk: choices in part[block][0..E-1], tokens in chunks[block].
__global__ __launch_bounds__(BL_COUNT_THREADS) void balance_count_kernel(const int32_t *__restrict__ ids,
                                                                         const uint8_t *__restrict__ mask,
                                                                         const int32_t *__restrict__ off, int T, int E,
                                                                         int k, int S, int chunk, int copies,
                                                                         int32_t *__restrict__ part,
                                                                         ChunkTokens *__restrict__ chunks) {
  extern __shared__ int32_t s_mem[];
  int total = 0;
  const Span sp = find_span(off, S, T, chunk, blockIdx.x, total);
  if (sp.seq < 0) {  // equal in every thread
    if (threadIdx.x == 0) chunks[blockIdx.x] = ChunkTokens{-1, 0};
    return;
  }
  count_chunk_lds<BL_COUNT_THREADS>(s_mem, copies, ids, mask, sp.begin, sp.end, E, k);
  int32_t *out = part + (size_t)blockIdx.x * E;
  for (int e = threadIdx.x; e < E; e += BL_COUNT_THREADS) out[e] = s_mem[e];
  if (threadIdx.x == 0) chunks[blockIdx.x] = ChunkTokens{sp.seq, s_mem[copies * E]};
}

// One block a sequence: its counts and counted tokens from the chunks', and the index of its
// first block of the main pass.
__global__ __launch_bounds__(256) void balance_tables_kernel(const int32_t *__restrict__ off, int T, int E, int S,
                                                             int chunk, int main_chunk, int blocks, int main_blocks,
                                                             const int32_t *__restrict__ part,
                                                             const ChunkTokens *__restrict__ chunks,
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
  // (offsets that run backwards could name more chunks than there are)
  const int n = min((e - b + chunk - 1) / chunk, max(blocks - first, 0));
  for (int i = threadIdx.x; i < E; i += 256) {
    int c = 0;
#pragma unroll 8
    for (int q = 0; q < n; ++q) c += part[(size_t)(first + q) * E + i];
    counts[(size_t)s * E + i] = c;
  }
  if (threadIdx.x < 64) {
    int c = 0;
    for (int q = lane; q < n; q += 64) c += chunks[first + q].tokens;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) c += __shfl_xor(c, o, 64);
    if (lane == 0) seq_tokens[s] = c;
  }
  if (threadIdx.x == 0) {
    first_main[s] = min(fm, main_blocks);
    if (s == S - 1) first_main[S] = min(fm + (e - b + main_chunk - 1) / main_chunk, main_blocks);
  }
}

// ------------------------------------------------------------------------------- main pass

// Chunks of sequence `seq` among the counting blocks' (they are neighbours), its tokens, the
// tokens and the sequences that count any of all of them (up to 64).
struct SeqCounts {
  int first, n, tokens, all, live;
};
__device__ __forceinline__ SeqCounts seq_counts(const ChunkTokens *chunks, int blocks, int seq) {
  const int lane = threadIdx.x & 63;
  SeqCounts r{0, 0, 0, 0, 0};
  uint64_t seen = 0;
  for (int c0 = 0; c0 < blocks; c0 += 64) {
    const ChunkTokens c = c0 + lane < blocks ? chunks[c0 + lane] : ChunkTokens{-1, 0};
    const uint64_t mine = __ballot(c.seq == seq);
    if (mine && r.n == 0) r.first = c0 + __ffsll((unsigned long long)mine) - 1;
    r.n += __popcll(mine);
    if (c.seq == seq) r.tokens += c.tokens;
    r.all += c.tokens;
    if (c.tokens > 0) seen |= 1ull << c.seq;
  }
  r.tokens = group_reduce<64>(r.tokens, add);
  r.all = group_reduce<64>(r.all, add);
  const auto either = [](uint32_t x, uint32_t y) { return x | y; };
  r.live = __popc(group_reduce<64>((uint32_t)seen, either)) + __popc(group_reduce<64>((uint32_t)(seen >> 32), either));
  return r;
}

struct BalanceArgs {
  const float *logits;
  const int32_t *ids;  // the block counts for itself (one sequence of few choices), or NULL
  const uint8_t *mask;
  const int32_t *off;
  int32_t *counts;
  int32_t *seq_tokens;
  const float *dloss;  // upstream gradients of the two losses, or NULL (ones)
  float *dlogits;      // or NULL
  float *part;         // [blocks][E]: column sums of p
  double *sums;        // [blocks][2]: sum of sum_i f_i p_ti / N_s, sum of z^2 (a finite z's square can pass
                       // the largest float)
  const int32_t *cpart;       // the counting blocks' results, added up by each block for itself,
  const ChunkTokens *chunks;  // or NULL: counts and seq_tokens hold them
  int cblocks;
  float *mean_probs, *losses;
  int T, E, k, S, chunk, copies, cols;
  int one;  // the only block: it finishes too
  float alpha, beta;
};

constexpr int at_once(int values) { return values <= 4 ? 4 : values <= 8 ? 2 : 1; }

// A token's row in LPT lanes of up to 16 values each, 64 / LPT tokens a wavefront: few lanes a
// row, so that the three reductions over a row and the row's own factors cost little beside
// its values (64 lanes of four values: ...).  With VEC (E a multiple of 4) a lane's values are
// 16-byte groups; otherwise they lie LPT apart, so that each load still covers neighbouring
// words.
template <int LPT, int VPL, bool VEC, bool LOSS>
__global__ __launch_bounds__(BL_THREADS) void balance_main_kernel(BalanceArgs a) {
  // fused multiply-adds where they are written: with and without the losses the gradient is
  // the same bit for bit
#pragma clang fp contract(off)
  constexpr int TPW = 64 / LPT;
  constexpr int NT = at_once(VPL);  // tokens a lane at a time
  extern __shared__ int32_t s_mem[];  // counting bins, then the waves' column sums [BL_WAVES][E]
  __shared__ double s_red[BL_WAVES][2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int li = lane & (LPT - 1), sub = lane / LPT;
  const int E = a.E;
  auto expert = [&](int v) { return VEC ? 4 * (li + LPT * (v / 4)) + v % 4 : li + LPT * v; };
  int total = 0;
  const Span sp = find_span(a.off, a.S, a.T, a.chunk, blockIdx.x, total);
  if (sp.seq < 0) {
    // blocks past the last chunk: rows outside every sequence get a zero gradient
    if (a.dlogits && a.off) {
      int b0, e0, b1, e1;
      seq_range(a.off, a.T, 0, b0, e0);
      seq_range(a.off, a.T, a.S - 1, b1, e1);
      const int64_t lead = (int64_t)b0 * E, tail = (int64_t)(a.T - e1) * E;
      const int64_t step = (int64_t)(gridDim.x - total) * BL_THREADS;
      for (int64_t i = (int64_t)(blockIdx.x - total) * BL_THREADS + threadIdx.x; i < lead + tail; i += step)
        a.dlogits[i < lead ? i : i - lead + (int64_t)e1 * E] = 0.f;
    }
    if (!(LOSS && a.ids && blockIdx.x == 0)) return;  // block 0 counts also where there are no rows
  }
  float l[NT][VPL];
  bool counted[NT];
  // rows of uncounted tokens are read and not looked at: the loads do not wait for the mask
  auto load = [&](int t0) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int t = t0 + n * TPW + sub;
      const bool in = t < sp.end;
      const float *row = a.logits + (size_t)t * E;
      counted[n] = in && (!a.mask || a.mask[t] != 0);
      if constexpr (VEC) {
#pragma unroll
        for (int v = 0; v < VPL; v += 4) {
          f32x4 q = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          if (in && expert(v) < E) q = *reinterpret_cast<const f32x4 *>(row + expert(v));
#pragma unroll
          for (int i = 0; i < 4; ++i) l[n][v + i] = q[i];
        }
      } else {
#pragma unroll
        for (int v = 0; v < VPL; ++v) l[n][v] = in && expert(v) < E ? row[expert(v)] : -INFINITY;
      }
    }
  };
  const int t_first = sp.begin + wave * (NT * TPW);
  load(t_first);  // in flight while the tables are read
  // sequences that count a token, tokens in all, this sequence's
  int live = 0, all = 0, ns = 0;
  float f[VPL];
  if (LOSS && a.ids) {
    int b, e;
    seq_range(a.off, a.T, 0, b, e);
    count_chunk_lds<BL_THREADS>(s_mem, a.copies, a.ids, a.mask, b, e, E, a.k);
    ns = all = s_mem[a.copies * E];
    live = ns > 0;
    if (blockIdx.x == 0) {
      for (int i = threadIdx.x; i < E; i += BL_THREADS) a.counts[i] = s_mem[i];
      if (threadIdx.x == 0) {
        a.seq_tokens[0] = ns;
      }
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v) f[v] = expert(v) < E ? (float)s_mem[expert(v)] : 0.f;
    __syncthreads();
  } else if (LOSS && a.chunks) {
    for (int e = threadIdx.x; e < E; e += BL_THREADS) s_mem[e] = 0;
    const SeqCounts sc = seq_counts(a.chunks, a.cblocks, sp.seq);
    live = sc.live;
    all = sc.all;
    ns = sc.tokens;
    __syncthreads();
    // threads on neighbouring experts (cols: a power of two), the others on further chunks
    const int col = threadIdx.x & (a.cols - 1), row = threadIdx.x / a.cols, rows = BL_THREADS / a.cols;
    for (int e = col; e < E; e += a.cols) {
      int c = 0;
#pragma unroll 8
      for (int q = row; q < sc.n; q += rows) c += a.cpart[(size_t)(sc.first + q) * E + e];
      atomicAdd(&s_mem[e], c);
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < VPL; ++v) f[v] = expert(v) < E ? (float)s_mem[expert(v)] : 0.f;
    __syncthreads();
  } else {
    for (int s = lane; s < a.S; s += 64) {
      const int n = a.seq_tokens[s];
      live += n > 0;
      all += n;
    }
    live = group_reduce<64>(live, add);
    all = group_reduce<64>(all, add);
    ns = a.seq_tokens[sp.seq];
#pragma unroll
    for (int v = 0; v < VPL; ++v) f[v] = expert(v) < E ? (float)a.counts[(size_t)sp.seq * E + expert(v)] : 0.f;
  }
  const float up0 = a.dloss ? a.dloss[0] : 1.f, up1 = a.dloss ? a.dloss[1] : 1.f;
  const float ca = up0 * (a.alpha * (float)E / ((float)max(live, 1) * (float)max(ns, 1)));
  const float cb = up1 * (2.f * a.beta / (float)max(all, 1));
  const float fden = (float)max(ns, 1) * (float)a.k;
  float acc[VPL];
  double bacc = 0., zacc = 0.;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    f[v] /= fden;
    acc[v] = 0.f;
  }
  for (int t0 = t_first; t0 < sp.end; t0 += BL_WAVES * NT * TPW) {
    if (t0 != t_first) load(t0);
    float base[NT], sum[NT], dot[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float m = -INFINITY;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        l[n][v] = counted[n] ? l[n][v] : -INFINITY;
        m = fmaxf(m, l[n][v]);
      }
      m = group_reduce<LPT>(m, [](float x, float y) { return fmaxf(x, y); });
      // a row without any finite logit (or an uncounted one) has sum 0: no probabilities
      base[n] = m == -INFINITY ? 0.f : m;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      sum[n] = dot[n] = 0.f;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        l[n][v] = __expf(l[n][v] - base[n]);
        sum[n] += l[n][v];
        dot[n] = __builtin_fmaf(l[n][v], f[v], dot[n]);
      }
      sum[n] = group_reduce<LPT>(sum[n], add);
      dot[n] = group_reduce<LPT>(dot[n], add);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int t = t0 + n * TPW + sub;
      const float inv = sum[n] == 0.f ? 0.f : __builtin_amdgcn_rcpf(sum[n]);  // sum is in [1, E]
      const float z = sum[n] == 0.f ? 0.f : base[n] + __logf(sum[n]);
      const float mean_f = dot[n] * inv;  // sum_i f_i p_i
      const float shift = __builtin_fmaf(ca, mean_f, -(cb * z));
      if constexpr (LOSS) {
        if (li == 0) {
          bacc += (double)mean_f;
          zacc += (double)z * (double)z;
        }
      }
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        l[n][v] *= inv;
        if constexpr (LOSS) acc[v] += l[n][v];
      }
      if (a.dlogits && t < sp.end) {
        float *drow = a.dlogits + (size_t)t * E;
        if constexpr (VEC) {
#pragma unroll
          for (int v = 0; v < VPL; v += 4) {
            f32x4 q;
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = l[n][v + i] * __builtin_fmaf(ca, f[v + i], -shift);
            if (expert(v) < E) __builtin_nontemporal_store(q, reinterpret_cast<f32x4 *>(drow + expert(v)));
          }
        } else {
#pragma unroll
          for (int v = 0; v < VPL; ++v)
            if (expert(v) < E) __builtin_nontemporal_store(l[n][v] * __builtin_fmaf(ca, f[v], -shift), drow + expert(v));
        }
      }
    }
  }
  if constexpr (LOSS) {
    float *s_acc = reinterpret_cast<float *>(s_mem);
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
#pragma unroll
      for (int o = LPT; o < 64; o <<= 1) acc[v] += __shfl_xor(acc[v], o, 64);
      if (sub == 0 && expert(v) < E) s_acc[wave * E + expert(v)] = acc[v];
    }
    block_sum2<BL_WAVES, LPT>(bacc, zacc, s_red);  // synchronises: the column sums are visible after it
    const float per = a.one ? 1.f / (float)max(ns, 1) : 1.f;
    float *out = a.one ? a.mean_probs : a.part + (size_t)blockIdx.x * E;
    for (int e = threadIdx.x; e < E; e += BL_THREADS) {
      float p = 0;
#pragma unroll
      for (int w = 0; w < BL_WAVES; ++w) p += s_acc[w * E + e];
      out[e] = p * per;
    }
    if (threadIdx.x == 0) {
      bacc /= max(ns, 1);
      if (a.one) {
        a.losses[0] = (float)((double)a.alpha * E * bacc);
        a.losses[1] = (float)((double)a.beta * zacc / max(ns, 1));
      } else {
        a.sums[2 * (size_t)blockIdx.x] = bacc;
        a.sums[2 * (size_t)blockIdx.x + 1] = zacc;
      }
    }
  }
}

// ---------------------------------------------------------------------------------- finish

constexpr int BL_FIN_THREADS = 512, BL_FIN_WAVES = BL_FIN_THREADS / 64;

struct FinishArgs {
  const float *part;
  const double *sums;
  const int32_t *off;
  const int32_t *first_main;  // with the tables, or NULL
  const int32_t *cpart;       // without them: the counting blocks' results (chunks), or NULL
  const ChunkTokens *chunks;
  int32_t *counts, *seq_tokens;
  float *mean_probs, *losses;
  int T, E, S, chunk, blocks, cblocks, cols, parts;
  float alpha, beta;
};

// Block s < S * parts: `cols` (a power of two) of a sequence's mean probabilities, threads on
// neighbouring experts and on further blocks of the main pass.  The last block: the two
// losses, since sum_i f_si P_si is the mean over the sequence's tokens of sum_i f_si p_ti.
__global__ __launch_bounds__(BL_FIN_THREADS) void balance_finish_kernel(FinishArgs a) {
  __shared__ double s_p[BL_FIN_WAVES][32];
  __shared__ int s_c[BL_FIN_WAVES][32];
  __shared__ double s_red[BL_FIN_WAVES][2];
  const int S = a.S, E = a.E;
  const bool losses = blockIdx.x == (unsigned)(S * a.parts);
  const int s = losses ? S - 1 : blockIdx.x / a.parts;
  // blocks of the main pass: of sequence s, and in all
  int b0, b1, nb;
  if (a.first_main) {
    b0 = a.first_main[s];
    b1 = a.first_main[s + 1];
    nb = a.first_main[S];
  } else {
    const int lane = threadIdx.x & 63;  // of sequence: S <= 64
    int b = 0, e = 0;
    if (lane < S) seq_range(a.off, a.T, lane, b, e);
    const int n = (e - b + a.chunk - 1) / a.chunk;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o, 64);
      if (lane >= o) incl += v;
    }
    // (offsets that run backwards could name more blocks than there are)
    b0 = min(__shfl(incl - n, s, 64), a.blocks);
    b1 = min(__shfl(incl, s, 64), a.blocks);
    nb = min(__shfl(incl, S - 1, 64), a.blocks);
  }
  if (losses) {
    double bal = 0, z = 0, live = 0, all = 0;
    for (int b = threadIdx.x; b < nb; b += BL_FIN_THREADS) {
      bal += a.sums[2 * (size_t)b];
      z += a.sums[2 * (size_t)b + 1];
    }
    if (a.chunks) {
      const SeqCounts sc = seq_counts(a.chunks, a.cblocks, s);
      if (threadIdx.x == 0) {
        live = sc.live;
        all = sc.all;
      }
    } else {
      for (int q = threadIdx.x; q < S; q += BL_FIN_THREADS) {
        live += a.seq_tokens[q] > 0;
        all += a.seq_tokens[q];
      }
    }
    block_sum2<BL_FIN_WAVES>(bal, z, s_red);
    block_sum2<BL_FIN_WAVES>(live, all, s_red);
    if (threadIdx.x == 0) {
      a.losses[0] = (float)((double)a.alpha * E * bal / max(live, 1.0));
      a.losses[1] = (float)((double)a.beta * z / max(all, 1.0));
    }
    return;
  }
  const int col = threadIdx.x & (a.cols - 1), row = threadIdx.x / a.cols, rows = BL_FIN_THREADS / a.cols;
  const int part = blockIdx.x - s * a.parts, e = part * a.cols + col;
  SeqCounts sc{0, 0, 0, 0, 0};
  int n, c = 0;
  if (a.chunks) {
    sc = seq_counts(a.chunks, a.cblocks, s);
    n = sc.tokens;
    if (part == 0 && threadIdx.x == 0) a.seq_tokens[s] = n;
  } else {
    n = a.seq_tokens[s];
  }
  double p = 0;
  if (e < E) {
#pragma unroll 8
    for (int b = b0 + row; b < b1; b += rows) p += a.part[(size_t)b * E + e];
    for (int q = row; q < sc.n; q += rows) c += a.cpart[(size_t)(sc.first + q) * E + e];
  }
  // rows of one wavefront (cols <= 32), then one row of each
  for (int o = 32; o >= a.cols; o >>= 1) {
    p += __shfl_xor(p, o, 64);
    c += __shfl_xor(c, o, 64);
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (lane < a.cols) {
    s_p[wave][lane] = p;
    s_c[wave][lane] = c;
  }
  __syncthreads();
  if (row == 0 && e < E) {
    p = 0;
    c = 0;
#pragma unroll
    for (int w = 0; w < BL_FIN_WAVES; ++w) {
      p += s_p[w][col];
      c += s_c[w][col];
    }
    a.mean_probs[(size_t)s * E + e] = (float)(p / max(n, 1));
    if (a.chunks) a.counts[(size_t)s * E + e] = c;
  }
}

constexpr int kVecValues = 4, kOddValues = 6;  // values a lane takes at most (16 past 64 lanes)
// Lanes a token takes: a power of two.
int lanes_per_token(int E) {
  int l = 1;
  while (l < 64 && (E % 4 == 0 ? kVecValues : kOddValues) * l < E) l *= 2;
  return l;
}
// Values of a lane, as the kernel is built for.
int values_per_lane(int E) {
  const int l = lanes_per_token(E), v = (E + l - 1) / l;
  if (E % 4 == 0) return v <= 4 ? 4 : v <= 8 ? 8 : v <= 12 ? 12 : 16;
  return v <= 4 ? 4 : v <= 6 ? 6 : v <= 8 ? 8 : v <= 10 ? 10 : v <= 12 ? 12 : 16;
}
int tokens_at_once(int E) { return 64 / lanes_per_token(E) * at_once(values_per_lane(E)); }  // of a wavefront

int count_chunk(int T) { return std::max(512, (T + 127) / 128); }
// Tokens of a block of the main pass: one round of its wavefronts at least.
int main_chunk(int T, int E, bool loss) {
  const int blocks = loss ? 512 : 2048;
  return std::max(BL_WAVES * tokens_at_once(E), (T + blocks - 1) / blocks);
}

// Chunks of the two passes: sequences cut into whole chunks, at most one partial chunk each,
// and in the main pass one block more for the rows outside every sequence.
int count_blocks(int T, int S, bool off) { return (T + count_chunk(T) - 1) / count_chunk(T) + (off ? S : 0); }
int main_blocks(int T, int E, int S, bool off, bool loss) {
  return (T + main_chunk(T, E, loss) - 1) / main_chunk(T, E, loss) + (off ? S + 1 : 0);
}

int bin_copies(int E) {
  int copies = 1;
  while (copies < 8 && copies * 2 * E <= BL_BINS) copies *= 2;
  return copies;
}

template <bool LOSS>
hipError_t launch_main(const BalanceArgs &a, int blocks, hipStream_t s) {
  const int E = a.E;
  const size_t lds = LOSS ? std::max((size_t)BL_WAVES * E * 4, a.ids ? ((size_t)a.copies * E + 1) * 4 : (size_t)0) : 0;
#define BL_LAUNCH(L, V, VEC)                                                                                        \
  do {                                                                                                              \
    hipLaunchKernelGGL((balance_main_kernel<L, V, VEC, LOSS>), dim3((unsigned)blocks), dim3(BL_THREADS), lds, s, a); \
    return hipGetLastError();                                                                                       \
  } while (0)
  const int v = values_per_lane(E);
#define BL_CASE(L)                                  \
  case L:                                           \
    if (E % 4 == 0) {                               \
      if (v == 4) BL_LAUNCH(L, 4, true);            \
      if (v == 8) BL_LAUNCH(L, 8, true);            \
      if (L < 64) return hipErrorInvalidValue;      \
      if (v == 12) BL_LAUNCH(64, 12, true);         \
      BL_LAUNCH(64, 16, true);                      \
    }                                               \
    if (v == 4) BL_LAUNCH(L, 4, false);             \
    if (v == 6) BL_LAUNCH(L, 6, false);             \
    if (v == 8) BL_LAUNCH(L, 8, false);             \
    if (v == 10) BL_LAUNCH(L, 10, false);           \
    if (v == 12) BL_LAUNCH(L, 12, false);           \
    if (L < 64) return hipErrorInvalidValue;        \
    BL_LAUNCH(64, 16, false);
  switch (lanes_per_token(E)) {
    BL_CASE(1)
    BL_CASE(2)
    BL_CASE(4)
    BL_CASE(8)
    BL_CASE(16)
    BL_CASE(32)
    BL_CASE(64)
  }
  return hipErrorInvalidValue;
#undef BL_CASE
#undef BL_LAUNCH
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

struct BalanceWs {
  size_t count_part, chunks, main_part, sums, first_main, total;
};
BalanceWs balance_ws(int T, int E, int S) {
  BalanceWs w;
  const size_t cb = count_blocks(T, S, true), mb = main_blocks(T, E, S, true, true);
  w.count_part = 0;
  w.chunks = align256(cb * E * 4);
  w.main_part = w.chunks + align256(cb * sizeof(ChunkTokens));
  w.sums = w.main_part + align256(mb * E * 4);
  w.first_main = w.sums + align256(mb * 16);
  w.total = w.first_main + align256(((size_t)S + 1) * 4);
  return w;
}

// One sequence with at most this many choices is counted by every block of the main pass for
// itself.
constexpr int64_t kSelfCount = 16384;
// Up to 64 sequences, and at most this many partial counts: every block of the main pass adds
// up its sequence's for itself, and no launch for the tables is made.
constexpr int64_t kSelfTables = 32768;

}  // namespace

size_t balance_workspace_bytes(int T, int E, int S) { return balance_ws(T, E, S).total; }

hipError_t launch_balance_loss(const BalanceCall &c, int32_t *counts, int32_t *seq_tokens, float *mean_probs,
                               float *losses, void *ws, hipStream_t s) {
  const BalanceWs w = balance_ws(c.T, c.E, c.S);
  uint8_t *base = static_cast<uint8_t *>(ws);
  int32_t *cpart = reinterpret_cast<int32_t *>(base + w.count_part);
  ChunkTokens *chunks = reinterpret_cast<ChunkTokens *>(base + w.chunks);
  const bool off = c.off != nullptr;
  const int cc = count_chunk(c.T), mc = main_chunk(c.T, c.E, true);
  const int cb = count_blocks(c.T, c.S, off), mb = main_blocks(c.T, c.E, c.S, off, true);
  const int copies = bin_copies(c.E);
  BalanceArgs a{};
  a.logits = c.logits;
  a.mask = c.mask;
  a.off = c.off;
  a.counts = counts;
  a.seq_tokens = seq_tokens;
  a.dloss = c.dloss;
  a.dlogits = c.dlogits;
  a.part = reinterpret_cast<float *>(base + w.main_part);
  a.sums = reinterpret_cast<double *>(base + w.sums);
  int32_t *first_main = reinterpret_cast<int32_t *>(base + w.first_main);
  a.mean_probs = mean_probs;
  a.losses = losses;
  a.T = c.T;
  a.E = c.E;
  a.k = c.k;
  a.S = c.S;
  a.chunk = mc;
  a.copies = copies;
  a.alpha = c.alpha;
  a.beta = c.beta;
  hipError_t e;
  bool tables = false;
  if (c.S == 1 && (int64_t)c.T * c.k <= kSelfCount) {
    a.ids = c.ids;
    a.one = mb == 1;
  } else {
    hipLaunchKernelGGL(balance_count_kernel, dim3((unsigned)cb), dim3(BL_COUNT_THREADS), (copies * c.E + 1) * 4, s,
                       c.ids, c.mask, c.off, c.T, c.E, c.k, c.S, cc, copies, cpart, chunks);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (c.S <= 64 && (int64_t)cb * c.E <= kSelfTables) {
      a.cpart = cpart;
      a.chunks = chunks;
      a.cblocks = cb;
      a.cols = 1;
      while (a.cols < BL_THREADS && a.cols < c.E) a.cols *= 2;
    } else {
      hipLaunchKernelGGL(balance_tables_kernel, dim3((unsigned)c.S), dim3(256), 0, s, c.off, c.T, c.E, c.S, cc, mc, cb,
                         mb, cpart, chunks, counts, seq_tokens, first_main);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      tables = true;
    }
  }
  if ((e = launch_main<true>(a, mb, s)) != hipSuccess || a.one) return e;
  FinishArgs f{};
  f.part = a.part;
  f.sums = a.sums;
  f.off = c.off;
  f.first_main = tables ? first_main : nullptr;
  f.cpart = a.cpart;
  f.chunks = a.chunks;
  f.cblocks = a.cblocks;
  f.counts = counts;
  f.seq_tokens = seq_tokens;
  f.mean_probs = mean_probs;
  f.losses = losses;
  f.T = c.T;
  f.E = c.E;
  f.S = c.S;
  f.chunk = mc;
  f.blocks = mb;
  f.cols = 1;
  while (f.cols < 32 && f.cols < c.E) f.cols *= 2;
  f.parts = (c.E + f.cols - 1) / f.cols;
  f.alpha = c.alpha;
  f.beta = c.beta;
  hipLaunchKernelGGL(balance_finish_kernel, dim3((unsigned)(c.S * f.parts + 1)), dim3(BL_FIN_THREADS), 0, s, f);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceCall &c, const int32_t *counts, const int32_t *seq_tokens,
                                   hipStream_t s) {
  BalanceArgs a{};
  a.logits = c.logits;
  a.mask = c.mask;
  a.off = c.off;
  a.counts = const_cast<int32_t *>(counts);  // read only without the loss
  a.seq_tokens = const_cast<int32_t *>(seq_tokens);
  a.dloss = c.dloss;
  a.dlogits = c.dlogits;
  a.T = c.T;
  a.E = c.E;
  a.k = c.k;
  a.S = c.S;
  a.chunk = main_chunk(c.T, c.E, false);
  a.alpha = c.alpha;
  a.beta = c.beta;
  return launch_main<false>(a, main_blocks(c.T, c.E, c.S, c.off != nullptr, false), s);
}

}  // namespace moe
