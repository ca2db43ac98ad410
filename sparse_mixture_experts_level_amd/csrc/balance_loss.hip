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
// logits gives both.  Counts come first (their own launch, or inside the main pass), the
// column sums' ends last.  Large batches are bound by reading the logits and writing the
// gradient once (gradient of 60001 x 161 alone 18.0 us, 4.3 TB/s; 65536 x 128 14.3 us, 4.7
// TB/s), smaller ones by the launches and the chains of loads in them (16384 x 256 in nine
// sequences with the losses 21 us in three launches; 8192 x 64 9.8 us in two; 16 x 32 5.0 us
// in one).  Without the gradient: 4.8, 9.3 and 19 us.  Many sequences cost blocks: a piece is one
// however short, and with more than 64 sequences each block of the gradient alone adds up every
// sequence's tokens (65536 x 64 in 512, 4096, 16384 and 65536 sequences: 29, 99, 340 and 1240 us
// with the losses; 11, 25, 111 and 820 alone).  Every sum has a fixed order (bit-reproducible);
// counts are whole numbers.
#include <algorithm>

#include "common.hpp"
#include "kernels.hpp"
#include "lanes.hpp"

namespace moe {

namespace {

constexpr int BL_COUNT_THREADS = 1024;
// Main pass.  8 wavefronts a block: 60001 x 161 20.7 against 17.5 us, 8192 x 64 12.7 against 11.7.
constexpr int BL_WAVES = 4, BL_THREADS = 64 * BL_WAVES;
constexpr int BL_BINS = 4096;                            // LDS bins of a block that counts

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

// Every pass cuts the batch into chunks of tokens whatever the sequences; the tokens of one
// sequence in one chunk are a piece, and a block's work.  With offsets the rows before the
// first sequence count as sequence -1 and those behind the last as sequence S (they only get
// their zero gradient), and the piece of sequence s in chunk b has the number b + s + 1:
// neighbouring pieces differ in one of the two, so numbers do not meet, those of a sequence
// lie together, and no sum over the sequences before is needed.  Without offsets the pieces
// are the chunks.
struct Piece {
  int seq, begin, end;  // begin == end: no piece has the number
};

__device__ __forceinline__ int begin_of(const int32_t *off, int T, int s) {  // s in [-1, S]
  return s < 0 ? 0 : min(max(off[s], 0), T);
}

// The piece numbered x: the last sequence whose first piece's number is not past x, looked for
// by one wavefront in 64 places at a time.  Equal in every lane.
__device__ __forceinline__ Piece find_piece(const int32_t *off, int S, int T, int chunk, int x) {
  if (!off) return Piece{0, min(x * chunk, T), (int)min((int64_t)(x + 1) * chunk, (int64_t)T)};
  const int lane = threadIdx.x & 63;
  int lo = -1, n = S + 2;  // among sequences lo .. lo + n - 1
  int b = 0;
  while (n > 1) {
    const int step = (n + 63) / 64, s = lo + lane * step;
    b = s <= S && lane * step < n ? begin_of(off, T, s) : 0;
    const bool at = s <= S && lane * step < n && b / chunk + s + 1 <= x;
    const int last = max(__popcll(__ballot(at)) - 1, 0);
    n = min(step, n - last * step);
    lo += last * step;
  }
  b = begin_of(off, T, lo);
  const int e = lo == S ? T : max(min(off[lo + 1], T), b);
  const int64_t c0 = (int64_t)(x - lo - 1) * chunk;  // the piece's chunk
  const int begin = (int)min(max(c0, (int64_t)b), (int64_t)T);
  return Piece{lo, begin, max((int)min(c0 + chunk, (int64_t)e), begin)};
}

// The numbers of sequence s's pieces (s in [0, S)): first .. first + n - 1.
__device__ __forceinline__ void seq_pieces(const int32_t *off, int T, int s, int chunk, int &first, int &n) {
  int b, e;
  seq_range(off, T, s, b, e);
  first = b / chunk + (off ? s + 1 : 0);
  n = e > b ? (e - 1) / chunk - b / chunk + 1 : 0;
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

// Sum of column values p[q * stride] over q = from, from + step, ... < n, eight loads in flight.
template <typename Sum, typename T>
__device__ __forceinline__ Sum column_sum(const T *p, size_t stride, int from, int n, int step) {
  Sum sum = 0;
  if (from >= n) return sum;
  p += (size_t)from * stride;
  const uint32_t inc = (uint32_t)step * (uint32_t)stride;
  int left = (n - from + step - 1) / step;  // values
  for (; left > 0; left -= 8, p += 8 * (size_t)inc) {
    T v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = p[(uint32_t)min(j, left - 1) * inc];  // (the last value again past the end)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += j < left ? (Sum)v[j] : Sum(0);
  }
  return sum;
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
    for (int j = 0; j < B; ++j) e[j] = src[min(i0 + j * THREADS, n - 1)];  // (no load waits for a condition)
    if (mask) {
      uint8_t in[B];
#pragma unroll
      for (int j = 0; j < B; ++j) in[j] = mask[begin + min(i0 + j * THREADS, n - 1) / (uint32_t)k];
#pragma unroll
      for (int j = 0; j < B; ++j) e[j] = in[j] ? e[j] : -1;
    }
#pragma unroll
    for (int j = 0; j < B; ++j)
      if (i0 + j * THREADS < n && e[j] >= 0 && e[j] < E) atomicAdd(&mine[e[j]], 1);
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

// What a counting block found: counted tokens, and the bit of their sequence (up to 64).
struct PieceTokens {
  int32_t tokens, pad;
  uint64_t seq;
};

// Counts of one piece: choices in part[piece][0..E-1], tokens in tokens[piece].
__global__ __launch_bounds__(BL_COUNT_THREADS) void balance_count_kernel(const int32_t *__restrict__ ids,
                                                                         const uint8_t *__restrict__ mask,
                                                                         const int32_t *__restrict__ off, int T, int E,
                                                                         int k, int S, int chunk, int copies,
                                                                         int32_t *__restrict__ part,
                                                                         PieceTokens *__restrict__ tokens) {
  extern __shared__ int32_t s_mem[];
  const Piece pc = find_piece(off, S, T, chunk, blockIdx.x);
  if (pc.begin >= pc.end || pc.seq < 0 || pc.seq >= S) {  // equal in every thread
    if (threadIdx.x == 0) tokens[blockIdx.x] = PieceTokens{0, 0, 0};
    return;
  }
  count_chunk_lds<BL_COUNT_THREADS>(s_mem, copies, ids, mask, pc.begin, pc.end, E, k);
  for (int e = threadIdx.x; e < E; e += BL_COUNT_THREADS) part[(size_t)blockIdx.x * E + e] = s_mem[e];
  if (threadIdx.x == 0) {
    const int n = s_mem[copies * E];
    tokens[blockIdx.x] = PieceTokens{n, 0, n > 0 && pc.seq < 64 ? 1ull << pc.seq : 0};
  }
}

// Counted tokens of a sequence from its pieces', in every lane.
__device__ __forceinline__ int seq_count(const PieceTokens *tokens, int first, int n) {
  int c = 0;
  for (int q = threadIdx.x & 63; q < n; q += 64) c += tokens[first + q].tokens;
  return group_reduce<64>(c, add);
}
// Counted tokens of the whole batch and sequences that count any (up to 64).
__device__ __forceinline__ void batch_count(const PieceTokens *tokens, int n, int &all, int &live) {
  int c = 0;
  uint64_t seen = 0;
  for (int q = threadIdx.x & 63; q < n; q += 64) {
    const PieceTokens p = tokens[q];
    c += p.tokens;
    seen |= p.seq;
  }
  all = group_reduce<64>(c, add);
  const auto either = [](uint32_t x, uint32_t y) { return x | y; };
  live = __popc(group_reduce<64>((uint32_t)seen, either)) + __popc(group_reduce<64>((uint32_t)(seen >> 32), either));
}

// The sums of the counting blocks' results.  Block s * parts + q: 64 experts of sequence s, four
// threads an expert.  The last block: sequences that count a token, and tokens in all.
__global__ __launch_bounds__(256) void balance_tables_kernel(const int32_t *__restrict__ off, int T, int E, int S,
                                                             int chunk, int parts, int blocks,
                                                             const int32_t *__restrict__ part,
                                                             const PieceTokens *__restrict__ tokens,
                                                             int32_t *__restrict__ counts,
                                                             int32_t *__restrict__ seq_tokens,
                                                             int32_t *__restrict__ totals) {
  __shared__ int s_c[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int first, n, c = 0;
  if (blockIdx.x == (unsigned)(S * parts)) {
    int live = 0;
    for (int s = threadIdx.x; s < S; s += 256) {
      seq_pieces(off, T, s, chunk, first, n);
      n = min(n, blocks - first);  // (offsets that run backwards could name more pieces)
      int mine = 0;
      for (int q = 0; q < n; ++q) mine += tokens[first + q].tokens;
      c += mine;
      live += mine > 0;
    }
    c = group_reduce<64>(c, add);
    live = group_reduce<64>(live, add);
    if (lane == 0) {
      s_c[wave][0] = live;
      s_c[wave][1] = c;
    }
    __syncthreads();
    if (threadIdx.x < 2)
      totals[threadIdx.x] = s_c[0][threadIdx.x] + s_c[1][threadIdx.x] + s_c[2][threadIdx.x] + s_c[3][threadIdx.x];
    return;
  }
  const int s = blockIdx.x / parts, q0 = blockIdx.x - s * parts, e = q0 * 64 + lane;
  seq_pieces(off, T, s, chunk, first, n);
  n = min(n, blocks - first);
  if (e < E) c = column_sum<int>(part + (size_t)first * E + e, E, wave, n, 4);
  s_c[wave][lane] = c;
  __syncthreads();
  if (wave == 0) {
    if (e < E) counts[(size_t)s * E + e] = s_c[0][lane] + s_c[1][lane] + s_c[2][lane] + s_c[3][lane];
    if (q0 == 0) {
      const int t = seq_count(tokens, first, n);
      if (lane == 0) seq_tokens[s] = t;
    }
  }
}

// ------------------------------------------------------------------------------- main pass

struct BalanceArgs {
  const float *logits;
  const int32_t *ids;  // the block counts for itself (one sequence of few choices), or NULL
  const uint8_t *mask;
  const int32_t *off;
  int32_t *counts;
  int32_t *seq_tokens;
  const float *dloss;  // upstream gradients of the two losses, or NULL (ones)
  float *dlogits;      // or NULL
  float *part;         // [pieces][E]: column sums of p
  double *sums;        // [blocks][2]: sum of sum_i f_i p_ti / N_s, sum of z^2 (a finite z's square can pass
                       // the largest float)
  // the counting blocks' results, added up by each block for itself, or NULL: counts,
  // seq_tokens and totals (NULL: seq_tokens) hold the sums
  const int32_t *cpart;
  const PieceTokens *ctokens;
  int cblocks, cchunk;
  const int32_t *totals;
  float *mean_probs, *losses;
  int T, E, k, S, chunk, copies, cols;
  int one;  // the only block: it finishes too
  float alpha, beta;
};

// Values of a lane that every row of such a kernel has (values LPT apart; see values_per_lane).
constexpr int sure_values(int lpt, int values) {
  return values > 12 ? 12 : values > 4 ? values - 2 : lpt > 1 ? 3 : 0;
}
constexpr int at_once(int values) { return values <= 4 ? 4 : values <= 8 ? 2 : 1; }

// A token's row in LPT lanes of VPL values each, 64 / LPT tokens a wavefront, at_once(VPL) such
// groups of tokens at a time (their loads and lane moves in flight together).  With VEC (E a
// multiple of 4) a lane's values are 16-byte groups; otherwise they lie LPT apart, so that
// each load still covers neighbouring words.
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
  const Piece pc = find_piece(a.off, a.S, a.T, a.chunk, blockIdx.x);
  const bool rows = pc.begin < pc.end && pc.seq >= 0 && pc.seq < a.S;
  const bool self = LOSS && a.ids;
  if (!rows) {
    if (a.dlogits) {  // of no sequence: a zero gradient
      const int64_t to = (int64_t)pc.end * E;
      for (int64_t i = (int64_t)pc.begin * E + threadIdx.x; i < to; i += BL_THREADS) a.dlogits[i] = 0.f;
    }
    if (LOSS && !a.one && threadIdx.x == 0) a.sums[2 * (size_t)blockIdx.x] = a.sums[2 * (size_t)blockIdx.x + 1] = 0.;
    if (!(self && blockIdx.x == 0)) return;  // block 0 counts also where it has no rows
  }
  float l[NT][VPL];
  bool counted[NT];
  // No load waits for a condition: rows of uncounted tokens are read and not looked at, tokens
  // past the piece and values past the row read the last ones.
  auto load = [&](int t0) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int t = min(t0 + n * TPW + sub, pc.end - 1);
      const float *row = a.logits + (size_t)t * E;
      if constexpr (VEC) {
#pragma unroll
        for (int v = 0; v < VPL; v += 4) {
          const f32x4 q = *reinterpret_cast<const f32x4 *>(row + min(expert(v), E - 4));
#pragma unroll
          for (int i = 0; i < 4; ++i) l[n][v + i] = q[i];
        }
      } else {
#pragma unroll
        for (int v = 0; v < VPL; ++v) l[n][v] = row[v < sure_values(LPT, VPL) ? expert(v) : min(expert(v), E - 1)];
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int t = t0 + n * TPW + sub;
      counted[n] = t < pc.end;
      if (a.mask) counted[n] = counted[n] && a.mask[min(t, pc.end - 1)] != 0;
    }
  };
  const int t_first = pc.begin + wave * (NT * TPW);
  if (rows) load(t_first);  // in flight while the tables are read
  // sequences that count a token, tokens in all
  int live = 0, all = 0;
  if (self) {
    int b, e;
    seq_range(a.off, a.T, 0, b, e);
    count_chunk_lds<BL_THREADS>(s_mem, a.copies, a.ids, a.mask, b, e, E, a.k);
    all = s_mem[a.copies * E];
    live = all > 0;
    if (blockIdx.x == 0) {
      for (int i = threadIdx.x; i < E; i += BL_THREADS) a.counts[i] = s_mem[i];
      if (threadIdx.x == 0) a.seq_tokens[0] = all;
      if (!rows) return;  // equal in every thread
    }
  } else if (LOSS && a.ctokens) {
    batch_count(a.ctokens, a.cblocks, all, live);
  } else if (LOSS) {
    live = a.totals[0];
    all = a.totals[1];
  } else {
    if (a.S <= 64) {
      if (lane < a.S) all = a.seq_tokens[lane];
      live = group_reduce<64>(all > 0 ? 1 : 0, add);
      all = group_reduce<64>(all, add);
    } else {
      __shared__ int s_tot[BL_WAVES][2];
      for (int s = threadIdx.x; s < a.S; s += BL_THREADS) {
        const int n = a.seq_tokens[s];
        live += n > 0;
        all += n;
      }
      live = group_reduce<64>(live, add);
      all = group_reduce<64>(all, add);
      if (lane == 0) {
        s_tot[wave][0] = live;
        s_tot[wave][1] = all;
      }
      __syncthreads();
      live = all = 0;
#pragma unroll
      for (int w = 0; w < BL_WAVES; ++w) {
        live += s_tot[w][0];
        all += s_tot[w][1];
      }
    }
  }
  const float up0 = a.dloss ? a.dloss[0] : 1.f, up1 = a.dloss ? a.dloss[1] : 1.f;
  const float cb = up1 * (2.f * a.beta / (float)max(all, 1));
  // the sequence's counted tokens, and its experts' shares of the choices
  int ns = all;
  float f[VPL], acc[VPL];
  if (self) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) f[v] = expert(v) < E ? (float)s_mem[expert(v)] : 0.f;
    __syncthreads();
  } else if (LOSS && a.ctokens) {
    int first, n;
    seq_pieces(a.off, a.T, pc.seq, a.cchunk, first, n);
    n = min(n, a.cblocks - first);
    if (a.S > 1) ns = seq_count(a.ctokens, first, n);
    for (int e = threadIdx.x; e < E; e += BL_THREADS) s_mem[e] = 0;
    __syncthreads();
    // threads on neighbouring experts (cols: a power of two), the others on further pieces
    const int col = threadIdx.x & (a.cols - 1), row = threadIdx.x / a.cols, step = BL_THREADS / a.cols;
    for (int e = col; e < E; e += a.cols)
      atomicAdd(&s_mem[e], column_sum<int>(a.cpart + (size_t)first * E + e, E, row, n, step));
    __syncthreads();
#pragma unroll
    for (int v = 0; v < VPL; ++v) f[v] = expert(v) < E ? (float)s_mem[expert(v)] : 0.f;
    __syncthreads();
  } else {
    ns = a.seq_tokens[pc.seq];
#pragma unroll
    for (int v = 0; v < VPL; ++v) f[v] = expert(v) < E ? (float)a.counts[(size_t)pc.seq * E + expert(v)] : 0.f;
  }
  const float ca = up0 * (a.alpha * (float)E / ((float)max(live, 1) * (float)max(ns, 1)));
  const float fden = (float)max(ns, 1) * (float)a.k;
  double bacc = 0., zacc = 0.;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    f[v] /= fden;
    acc[v] = 0.f;
  }
  for (int t0 = t_first; t0 < pc.end; t0 += BL_WAVES * NT * TPW) {
    if (t0 != t_first) load(t0);
    float base[NT], sum[NT], dot[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float m = -INFINITY;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        l[n][v] = counted[n] && expert(v) < E ? l[n][v] : -INFINITY;
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
      const bool none = sum[n] == 0.f;
      const float inv = none ? 0.f : __builtin_amdgcn_rcpf(sum[n]);  // sum is in [1, E]
      const float z = none ? 0.f : base[n] + __logf(sum[n]);
      const float mean_f = dot[n] * inv;  // sum_i f_i p_i
      // factors of zero too: upstream gradients may be infinite or NaN
      const float can = none ? 0.f : ca;
      const float shift = none ? 0.f : __builtin_fmaf(ca, mean_f, -(cb * z));
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
      // written once and not read here: past the caches (16384 x 256: 13.0 -> 11.5 us)
      if (a.dlogits && t < pc.end) {
        float *drow = a.dlogits + (size_t)t * E;
        if constexpr (VEC) {
#pragma unroll
          for (int v = 0; v < VPL; v += 4) {
            f32x4 q;
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = l[n][v + i] * __builtin_fmaf(can, f[v + i], -shift);
            if (expert(v) < E) __builtin_nontemporal_store(q, reinterpret_cast<f32x4 *>(drow + expert(v)));
          }
        } else {
#pragma unroll
          for (int v = 0; v < VPL; ++v)
            if (expert(v) < E)
              __builtin_nontemporal_store(l[n][v] * __builtin_fmaf(can, f[v], -shift), drow + expert(v));
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
  const int32_t *cpart;  // the counting blocks' results, or NULL: counts, seq_tokens and totals
  const PieceTokens *ctokens;  // (NULL: one sequence) hold the sums
  const int32_t *totals;
  int32_t *counts, *seq_tokens;
  float *mean_probs, *losses;
  int T, E, S, chunk, blocks, cchunk, cblocks, cols, parts;
  float alpha, beta;
};

// Block s < S * parts: `cols` (a power of two, at most 32) of a sequence's mean probabilities,
// threads on neighbouring experts and on further pieces of the main pass.  The last block: the
// two losses, since sum_i f_si P_si is the mean over the sequence's tokens of sum_i f_si p_ti.
__global__ __launch_bounds__(BL_FIN_THREADS) void balance_finish_kernel(FinishArgs a) {
  __shared__ double s_p[BL_FIN_WAVES][32];
  __shared__ int s_c[BL_FIN_WAVES][32];
  __shared__ double s_red[BL_FIN_WAVES][2];
  const int S = a.S, E = a.E;
  if (blockIdx.x == (unsigned)(S * a.parts)) {
    double bal = 0, z = 0;
    for (int b = threadIdx.x; b < a.blocks; b += BL_FIN_THREADS) {
      bal += a.sums[2 * (size_t)b];
      z += a.sums[2 * (size_t)b + 1];
    }
    int live, all;
    if (a.ctokens) {
      batch_count(a.ctokens, a.cblocks, all, live);
    } else if (a.totals) {
      live = a.totals[0];
      all = a.totals[1];
    } else {
      all = a.seq_tokens[0];
      live = 1;
    }
    block_sum2<BL_FIN_WAVES>(bal, z, s_red);
    if (threadIdx.x == 0) {
      a.losses[0] = (float)((double)a.alpha * E * bal / max(live, 1));
      a.losses[1] = (float)((double)a.beta * z / max(all, 1));
    }
    return;
  }
  const int s = blockIdx.x / a.parts;
  const int col = threadIdx.x & (a.cols - 1), row = threadIdx.x / a.cols, rows = BL_FIN_THREADS / a.cols;
  const int part = blockIdx.x - s * a.parts, e = part * a.cols + col;
  int first, n, cfirst = 0, cn = 0, tokens, c = 0;
  seq_pieces(a.off, a.T, s, a.chunk, first, n);
  n = min(n, a.blocks - first);  // (offsets that run backwards could name more pieces)
  if (a.ctokens) {
    seq_pieces(a.off, a.T, s, a.cchunk, cfirst, cn);
    cn = min(cn, a.cblocks - cfirst);
    tokens = seq_count(a.ctokens, cfirst, cn);
    if (part == 0 && threadIdx.x == 0) a.seq_tokens[s] = tokens;
  } else {
    tokens = a.seq_tokens[s];
  }
  double p = 0;
  if (e < E) {
    p = column_sum<double>(a.part + (size_t)first * E + e, E, row, n, rows);
    if (a.ctokens) c = column_sum<int>(a.cpart + (size_t)cfirst * E + e, E, row, cn, rows);
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
    a.mean_probs[(size_t)s * E + e] = (float)(p / max(tokens, 1));
    if (a.ctokens) a.counts[(size_t)s * E + e] = c;
  }
}

// Values a lane takes at most (16 past 64 lanes).  One 16-byte load where rows allow it: 8 values
// measured 5.9 against 5.1 us on 16 x 32 and 9.5 against 9.3 on 16384 x 256 (gradient alone),
// 16 values 8.4 and 13.0.  Odd rows, where a value is a load and few lanes save reductions, up to 4,
// 6, 8 and 12 values (gradient alone): 52103 x 161 19.3, 15.6, 15.6, 16.6 us; 43919 x 191 17.9,
// 15.5, 15.7, 16.7; 129055 x 65 19.3, 17.8, 18.9, 37.9.  Large batches of 17 to 47 experts are the
// exception: 254200 x 33 19.6, 36.6, 36.9, 86.4 (4000 rows: the same for all but 12).
constexpr int kVecValues = 4, kOddValues = 6;
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

// Tokens of a counting block: at most 128 results to add up (256 tokens a block: 16384 x 256 21.4
// against 20.0 us; 1024: 19.7, but 25.3 against 24.0 in nine sequences).
int count_chunk(int T) { return std::max(512, (T + 127) / 128); }
// Tokens of a block of the main pass: one round of its wavefronts at least.  With the losses
// each block leaves its column sums (512 blocks: 16384 x 256 20.0 us; 256 or 1024: 21.4).
int main_chunk(int T, int E, bool loss) {
  const int blocks = loss ? 512 : 2048;
  return std::max(BL_WAVES * tokens_at_once(E), (T + blocks - 1) / blocks);
}

// Numbers of the pieces of T tokens in chunks, with S sequences.
int pieces(int T, int chunk, int S, bool off) { return (T + chunk - 1) / chunk + (off ? S + 1 : 0); }

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
  // fewer than 64 lanes: as few values as lanes_per_token() asks for, no more
#define BL_CASE(L)                                     \
  case L:                                              \
    if (E % 4 == 0 && v == 4) BL_LAUNCH(L, 4, true);   \
    if (E % 4 != 0 && v == 4) BL_LAUNCH(L, 4, false);  \
    if (E % 4 != 0 && v == 6) BL_LAUNCH(L, 6, false);  \
    if (L < 64) return hipErrorInvalidValue;
  switch (lanes_per_token(E)) {
    BL_CASE(1)
    BL_CASE(2)
    BL_CASE(4)
    BL_CASE(8)
    BL_CASE(16)
    BL_CASE(32)
    BL_CASE(64)
      if (E % 4 == 0) {
        if (v == 8) BL_LAUNCH(64, 8, true);
        if (v == 12) BL_LAUNCH(64, 12, true);
        BL_LAUNCH(64, 16, true);
      }
      if (v == 8) BL_LAUNCH(64, 8, false);
      if (v == 10) BL_LAUNCH(64, 10, false);
      if (v == 12) BL_LAUNCH(64, 12, false);
      BL_LAUNCH(64, 16, false);
  }
  return hipErrorInvalidValue;
#undef BL_CASE
#undef BL_LAUNCH
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

struct BalanceWs {
  size_t count_part, count_tokens, totals, main_part, sums, total;
};
BalanceWs balance_ws(int T, int E, int S) {
  BalanceWs w;
  const size_t cb = pieces(T, count_chunk(T), S, true), mb = pieces(T, main_chunk(T, E, true), S, true);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  w.count_part = take(cb * E * 4);
  w.count_tokens = take(cb * sizeof(PieceTokens));
  w.totals = take(8);
  w.main_part = take(mb * E * 4);
  w.sums = take(mb * 16);
  w.total = at;
  return w;
}

// One sequence with at most this many choices is counted by every block of the main pass for
// itself, against a launch that counts: 8192 x 64, one choice, 9.6 against 11.9 us; 16384 choices
// of 16384 x 64 11.4 against 12.2, of 2048 x 256 11.6 against 12.0, of 8192 x 256 13.2 against
// 14.5; 32768 of 32768 x 64 16.5 against 14.1, of 4096 x 256 15.3 against 12.4.
constexpr int64_t kSelfCount = 16384;
// Up to 64 sequences, and at most this many partial counts: every block of the main pass adds
// up its sequence's for itself, and no launch for the tables is made: 65536 x 32 15.9 against
// 27.1 us, 16384 x 256 20.0 against 21.5, 65536 x 256 (the most) 40.0 against 47.0.
constexpr int64_t kSelfTables = 32768;

}  // namespace

size_t balance_workspace_bytes(int T, int E, int S) { return balance_ws(T, E, S).total; }

hipError_t launch_balance_loss(const BalanceCall &c, int32_t *counts, int32_t *seq_tokens, float *mean_probs,
                               float *losses, void *ws, hipStream_t s) {
  const BalanceWs w = balance_ws(c.T, c.E, c.S);
  uint8_t *base = static_cast<uint8_t *>(ws);
  int32_t *cpart = reinterpret_cast<int32_t *>(base + w.count_part);
  PieceTokens *ctokens = reinterpret_cast<PieceTokens *>(base + w.count_tokens);
  int32_t *totals = reinterpret_cast<int32_t *>(base + w.totals);
  const int cc = count_chunk(c.T), mc = main_chunk(c.T, c.E, true);
  const int cb = pieces(c.T, cc, c.S, c.off != nullptr), mb = pieces(c.T, mc, c.S, c.off != nullptr);
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
  if (c.S == 1 && (int64_t)c.T * c.k <= kSelfCount) {
    a.ids = c.ids;
    a.one = mb == 1;
  } else {
    hipLaunchKernelGGL(balance_count_kernel, dim3((unsigned)cb), dim3(BL_COUNT_THREADS), (copies * c.E + 1) * 4, s,
                       c.ids, c.mask, c.off, c.T, c.E, c.k, c.S, cc, copies, cpart, ctokens);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (c.S <= 64 && (int64_t)cb * c.E <= kSelfTables) {
      a.cpart = cpart;
      a.ctokens = ctokens;
      a.cblocks = cb;
      a.cchunk = cc;
      a.cols = 1;
      while (a.cols < BL_THREADS && a.cols < c.E) a.cols *= 2;
    } else {
      const int parts = (c.E + 63) / 64;
      hipLaunchKernelGGL(balance_tables_kernel, dim3((unsigned)(c.S * parts + 1)), dim3(256), 0, s, c.off, c.T, c.E,
                         c.S, cc, parts, cb, cpart, ctokens, counts, seq_tokens, totals);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      a.totals = totals;
    }
  }
  if ((e = launch_main<true>(a, mb, s)) != hipSuccess || a.one) return e;
  FinishArgs f{};
  f.part = a.part;
  f.sums = a.sums;
  f.off = c.off;
  f.cpart = a.cpart;
  f.ctokens = a.ctokens;
  f.cblocks = a.cblocks;
  f.cchunk = a.cchunk;
  f.totals = a.totals;
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
  while (f.cols < 16 && f.cols < c.E) f.cols *= 2;
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
  return launch_main<false>(a, pieces(c.T, a.chunk, c.S, c.off != nullptr), s);
}

}  // namespace moe
