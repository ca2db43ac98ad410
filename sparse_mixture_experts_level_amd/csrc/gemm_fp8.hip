// Grouped products in 8-bit floating point with a scale for each block of 128 (layouts in fp8.hpp):
//   out[r][n] = sum_b 2^(sx[r][b] + sw[n / 128][b]) sum_{k in block b} x8[r][k] w8[n][k]
// for the rows r of each group, bf16; and the gate_up form, whose epilogue forms
//   H[r][n] = silu(G[r][n]) U[r][n],  silu(z) = z / (1 + exp(-z))
// from the float sums and quantises it again, a scale for each 128 columns of a row.
//
// Few rows a group: bound by the weights' bytes.  Weights go from memory straight to registers (their
// layout is the matrix instruction's), whole lines, non-temporal, several steps ahead; codes become
// bf16 times their scale there (an exact conversion, two values an instruction) and meet the rows in the bf16 matrix
// instruction: at half the 8-bit one's rate it still has time to spare, and its sums are those of
// floats, where the 8-bit instruction drops what lies 2^-14 below the largest of 16 products (1.5e-5 of a
// sum: enough to move one code of H in two thousand).
#include <algorithm>
#include <climits>
#include <cstdlib>

#include "fp8.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

// Where row m0 + r of a group stands: byte offsets of its codes and scales in xres and sres, kOob past the group's
// end and for an index outside the rows.
struct Fp8Rows {
  rsrc_t xres, sres;
  bool gather;
  __device__ __forceinline__ Fp8Rows(const Fp8GemmArgs &a, int m0, int rows) : gather(a.row_index != nullptr) {
    const int kp = fp8_row_bytes(a.K), ks = fp8_scale_bytes(a.K);
    const int64_t first = gather ? 0 : m0, n = gather ? a.x_rows : rows;
    xres = make_rsrc(a.x8 + first * kp, (uint32_t)(n * kp));
    sres = make_rsrc(a.x_scale + first * ks, (uint32_t)(n * ks));
  }
  // (the index of a row past the end is read from the last row's place, so that no load waits for a branch)
  __device__ __forceinline__ uint32_t row(const Fp8GemmArgs &a, int m0, int r, int n) const {
    uint32_t src = (uint32_t)r, most = (uint32_t)n;
    if (gather) {
      src = (uint32_t)a.row_index[m0 + min(r, n - 1)];
      most = (uint32_t)a.x_rows;
    }
    return r < n && src < most ? src : kOob;
  }
};

// H's 8 bits from a lane's four columns of one row: `top` is the largest magnitude of the row's 128.
__device__ __forceinline__ void store_h(const Fp8GemmArgs &a, const float *h, float top, int64_t row, int nb, int col,
                                        bool first) {
  const uint32_t byte = fp8_scale_byte(top);
  const float inv = fp8_inverse(byte);
  *reinterpret_cast<uint32_t *>(a.h8 + row * fp8_row_bytes(a.n_out) + col) =
      fp8_codes(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv);
  if (first) a.h_scale[row * fp8_scale_bytes(a.n_out) + nb] = (uint8_t)byte;
}

// A lane's four columns of one output row.
__device__ __forceinline__ void store_y(const Fp8GemmArgs &a, f32x4 v, int64_t row, int col) {
  uint16_t *o = a.y + row * a.n_out + col;
  if (a.n_out % 4 == 0) {
    if (col < a.n_out) *reinterpret_cast<uint2 *>(o) = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (col + j < a.n_out) o[j] = f32_to_bf16(v[j]);
  }
}

// Few rows: 16 of them at a time, one block after the other.  A workgroup has 16 U output columns; each wave 16
// of them (for gate_up the 16 gate and the 16 up rows) and one of KS parts of K, whose sums the first
// part's waves add in order.  Rows are read from the caches in the operand layout, two steps ahead, with the weights,
// R steps of 128 ahead, all in registers: no LDS, no barrier.  The weights are the
// matrix instruction's first operand, so that a lane holds four consecutive columns of one row.
template <bool SWIGLU, int U, int KS>
__global__ __launch_bounds__(64 * U * KS, 4) void fp8_small_kernel(const Fp8GemmArgs a) {
  constexpr int NB = SWIGLU ? 2 : 1, R = SWIGLU ? 4 : 8, XR = 2;
  constexpr bool QUANTISE = SWIGLU && U == 8;  // a block of H's columns a workgroup
  __shared__ float tops[QUANTISE ? 8 : 1][16];
  __shared__ f32x4 parts[KS > 1 ? (KS - 1) * U * NB * 64 : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lr = lane & 15,
            lg = lane >> 4;
  const int u = wave % U, part = wave / U;
  int begin, end;
  const int nb = blockIdx.x, g = fp8_nth_group(a, blockIdx.y, INT_MAX, begin, end);
  if (g < 0) return;
  const int kt = fp8_blocks(a.K), kp = fp8_row_bytes(a.K), ks = fp8_scale_bytes(a.K);
  // parts of K are whole words of scales: four steps
  const int quads = ks / 4, tb = 4 * (quads * part / KS), te = min(kt, 4 * (quads * (part + 1) / KS));
  const int unit = nb * U + u, units = (a.n_out + 15) / 16;
  const int64_t wbytes = fp8_group_bytes(a.n_out, a.K, SWIGLU);
  const rsrc_t wres = make_rsrc(a.w8 + g * wbytes, (uint32_t)wbytes);
  uint32_t half;  // (gate and up blocks are neighbours)
  const uint32_t wbase = fp8_block_offset(unit * NB, units * NB, kt, half) + (uint32_t)lane * 16u;
  const int tw = unit < units ? te : 0;  // no weights past the last block
  const uint8_t *wscale = a.w_scale + ((int64_t)g * fp8_blocks(a.n_out) + min(unit, units - 1) / 8) * NB * ks;
  for (int m0 = begin; m0 < end; m0 += 16) {
    u32x4 w[R][NB][2], x[XR][2];
    uint32_t sx, nx, sw[NB], nw[NB];
    auto load_w = [&](int j, int t) {  // steps past the part's end read zeros
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t o = t < tw ? wbase + (uint32_t)(2 * t) * half + (uint32_t)b * 1024u : kOob;
        w[j][b][0] = buf_ld16_nt(wres, o);
        w[j][b][1] = buf_ld16_nt(wres, t < tw ? o + half : kOob);
      }
    };
#pragma unroll
    for (int j = 0; j < R; ++j) load_w(j, tb + j);
    const Fp8Rows rows(a, m0, min(16, end - m0));
    const uint32_t src = rows.row(a, m0, lr, min(16, end - m0));
    const uint32_t xoff = src != kOob ? src * (uint32_t)kp + (uint32_t)lg * 16u : kOob;
    const uint32_t soff = src != kOob ? src * (uint32_t)ks : kOob;
    auto load_x = [&](int j, int t) {
      const uint32_t o = t < te && xoff != kOob ? xoff + (uint32_t)t * 128u : kOob;
      x[j][0] = buf_ld16(rows.xres, o);
      x[j][1] = buf_ld16(rows.xres, o == kOob ? kOob : o + 64u);
    };
    auto load_scales = [&](int t) {  // of four steps; past K those of the last four again (their codes are zeros)
      const int at = min(t, ks - 4);
      nx = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rows.sres, soff == kOob ? kOob : soff + (uint32_t)at, 0, 0);
#pragma unroll
      for (int b = 0; b < NB; ++b) nw[b] = scalar_load(wscale + b * ks + at);
    };
    load_scales(tb);
#pragma unroll
    for (int j = 0; j < XR; ++j) load_x(j, tb + j);
    // All of the first loads, by a wait that the compiler counts: it would otherwise take the loop's entry, where few
    // loads follow those of step 0, for the rule, and wait for nearly all in flight on every trip.
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    f32x4 acc[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int t0 = tb; t0 < te; t0 += R) {
      auto step = [&](auto jc) {
        constexpr int J = decltype(jc)::value, S = J % 4;
        const int t = t0 + J;
        if constexpr (S == 0) {
          const int left = te - t;  // blocks of this part: the padding's scales are not looked at
          const uint32_t keep = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
          sx = nx & keep;
#pragma unroll
          for (int b = 0; b < NB; ++b) sw[b] = nw[b] & keep;
          load_scales(t + 4);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {  // 32 of K: eight of each lane's 32 codes
          const u32x4 xb = fp8_to_bf16(x[J % XR][m / 2][2 * (m % 2)], x[J % XR][m / 2][2 * (m % 2) + 1], fp8_scale<S>(sx));
#pragma unroll
          for (int b = 0; b < NB; ++b)
            acc[b] = mfma16(fp8_to_bf16(w[J][b][m / 2][2 * (m % 2)], w[J][b][m / 2][2 * (m % 2) + 1], fp8_scale<S>(sw[b])), xb,
                            acc[b]);
        }
        __builtin_amdgcn_sched_barrier(0);  // loads into registers still in use would get others, copied after a wait
        load_x(J % XR, t + XR);
        load_w(J, t + R);
      };
      step(std::integral_constant<int, 0>{});
      step(std::integral_constant<int, 1>{});
      step(std::integral_constant<int, 2>{});
      step(std::integral_constant<int, 3>{});
      if constexpr (R == 8) {
        step(std::integral_constant<int, 4>{});
        step(std::integral_constant<int, 5>{});
        step(std::integral_constant<int, 6>{});
        step(std::integral_constant<int, 7>{});
      }
    }
    if constexpr (KS > 1) {
      if (part > 0)
#pragma unroll
        for (int b = 0; b < NB; ++b) parts[(((part - 1) * U + u) * NB + b) * 64 + lane] = acc[b];
      __syncthreads();
      if (part == 0)
#pragma unroll
        for (int p = 1; p < KS; ++p)
#pragma unroll
          for (int b = 0; b < NB; ++b) acc[b] += parts[(((p - 1) * U + u) * NB + b) * 64 + lane];
    }
    const int col = unit * 16 + lg * 4;
    const int64_t row = m0 + lr;
    if constexpr (QUANTISE) {
      float h[4], top = 0.0f;
      if (part == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[j] = silu_f32(acc[0][j]) * acc[1][j];
          top = fmaxf(top, fp8_magnitude(h[j]));
        }
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        if (lg == 0) tops[u][lr] = top;
      }
      __syncthreads();
      if (part == 0 && row < end) {
#pragma unroll
        for (int v = 0; v < 8; ++v) top = fmaxf(top, tops[v][lr]);
        store_h(a, h, top, row, nb, col, u == 0 && lg == 0);
      }
    } else if constexpr (SWIGLU) {
      if (part == 0 && row < end) {
        f32x4 h;
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = silu_f32(acc[0][j]) * acc[1][j];
        if (col < fp8_row_bytes(a.n_out)) *reinterpret_cast<f32x4 *>(a.h32 + row * (int64_t)fp8_row_bytes(a.n_out) + col) = h;
      }
    } else if (part == 0 && row < end) {
      store_y(a, acc[0], row, col);
    }
    if (QUANTISE || KS > 1) __syncthreads();  // the next rows use the same LDS
  }
}

// Some rows, up to 128 at a time: a workgroup has 128 columns of H or 256 of y, each of its eight waves two
// blocks of 16 weight rows (gate and up, or neighbours).  The rows are read by all eight waves from LDS, where
// loads without registers put them as codes, a step of 128 of K a stage, in the operand layout (2 KB for 16 rows:
// sixteen lanes read 256 consecutive bytes); four stages, three steps ahead, one barrier a step.  The 8-bit matrix
// instruction: converted to bf16 by each wave, 128 rows took 1.7 us a step of the 1.2 that its weights take.
constexpr int MD_R = 4, MD_D = 3, MD_ROWS = 128, MD_STAGE = MD_ROWS * 128;

// One block of n <= 16 MS rows from m0 on; MS is exact, so that no branch is in the loop.
template <bool SWIGLU, int MS>
__device__ __forceinline__ void medium_rows(const Fp8GemmArgs &a, int g, int nb, int m0, int n, uint8_t *s0, uint8_t *s1,
                                            uint8_t *s2, uint8_t *s3, float (*tops)[MD_ROWS]) {
  constexpr int R = MD_R, D = MD_D;
  auto stage = [&](int b) -> uint8_t * { return b == 0 ? s0 : b == 1 ? s1 : b == 2 ? s2 : s3; };
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lr = lane & 15,
            lg = lane >> 4;
  const int kt = fp8_blocks(a.K), kp = fp8_row_bytes(a.K), ks = fp8_scale_bytes(a.K);
  const int units = (a.n_out + 15) / 16 * (SWIGLU ? 2 : 1), unit = nb * 16 + wave * 2;  // blocks of 16 weight rows
  const int64_t wbytes = fp8_group_bytes(a.n_out, a.K, SWIGLU);
  const rsrc_t wres = make_rsrc(a.w8 + g * wbytes, (uint32_t)wbytes);
  uint32_t half;
  const uint32_t wbase = fp8_block_offset(unit, units, kt, half) + (uint32_t)lane * 16u;
  const int sblocks = fp8_blocks(a.n_out);
  const uint8_t *wscale =
      a.w_scale + ((int64_t)g * sblocks + (SWIGLU ? nb : min(nb * 2 + wave / 4, sblocks - 1))) * (SWIGLU ? 2 : 1) * ks;
  i32x8 w[R][2];
  auto load_w = [&](int j, int t) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const bool in = t < kt && unit + b < units;
      const uint32_t o = wbase + (uint32_t)(2 * t) * half + (uint32_t)b * 1024u;
      w[j][b] = fp8_operand(buf_ld16_nt(wres, in ? o : kOob), buf_ld16_nt(wres, in ? o + half : kOob));
    }
  };
  const Fp8Rows rows(a, m0, n);
  // this wave's pieces of a stage, one for each half of K's 128: subtile `wave`, row lr, codes 64 p + 16 lg ..
  const uint32_t src = rows.row(a, m0, wave * 16 + lr, n);
  const uint32_t xoff = src != kOob ? src * (uint32_t)kp + (uint32_t)lg * 16u : kOob;
  auto load_x = [&](int t, int b) {
    const uint32_t o = t < kt && xoff != kOob ? xoff + (uint32_t)t * 128u : kOob;
    buf_ld16_lds(rows.xres, o, stage(b) + wave * 2048);
    buf_ld16_lds(rows.xres, o == kOob ? kOob : o + 64u, stage(b) + wave * 2048 + 1024);
  };
  uint32_t soff[MS], sx[MS], nx[MS], sw[2], nw[2];
#pragma unroll
  for (int i = 0; i < MS; ++i) {
    const uint32_t r = rows.row(a, m0, i * 16 + lr, n);
    soff[i] = r != kOob ? r * (uint32_t)ks : kOob;
  }
  auto load_scales = [&](int t) {  // of four steps; past K those of the last four again (their codes are zeros)
    const int at = min(t, ks - 4);
#pragma unroll
    for (int i = 0; i < MS; ++i)
      nx[i] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rows.sres, soff[i] == kOob ? kOob : soff[i] + (uint32_t)at, 0, 0);
#pragma unroll
    for (int b = 0; b < 2; ++b) nw[b] = scalar_load(wscale + (SWIGLU ? b * ks : 0) + at);
  };
  f32x4 acc[MS][2];
#pragma unroll
  for (int i = 0; i < MS; ++i)
#pragma unroll
    for (int b = 0; b < 2; ++b) acc[i][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  load_scales(0);
#pragma unroll
  for (int b = 0; b < D; ++b) load_x(b, b);
  __builtin_amdgcn_sched_barrier(0);  // the waits count on rows before weights
#pragma unroll
  for (int j = 0; j < R; ++j) load_w(j, j);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(4 * R) : "memory");  // the first stages are there
  auto bar = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  bar();
  for (int t0 = 0; t0 < kt; t0 += R) {
    const uint32_t keep = kt - t0 >= 4 ? ~0u : (1u << (8 * (kt - t0))) - 1u;  // the padding's scales are not looked at
#pragma unroll
    for (int i = 0; i < MS; ++i) sx[i] = nx[i] & keep;
#pragma unroll
    for (int b = 0; b < 2; ++b) sw[b] = nw[b] & keep;
    load_scales(t0 + R);
    auto step = [&](auto jc) {
      constexpr int J = decltype(jc)::value;
      const int t = t0 + J;
      load_x(t + D, (J + D) % R);  // the stage read in step t - 1, which every wave has left
      __builtin_amdgcn_sched_barrier(0);
      const uint8_t *st = stage(J) + lane * 16;
#pragma unroll
      for (int i = 0; i < MS; ++i) {
        const i32x8 x = fp8_operand(*reinterpret_cast<const u32x4 *>(st + i * 2048),
                                    *reinterpret_cast<const u32x4 *>(st + i * 2048 + 1024));
#pragma unroll
        for (int b = 0; b < 2; ++b) acc[i][b] = mfma_fp8_16<J>(w[J][b], x, acc[i][b], sw[b], sx[i]);
      }
      __builtin_amdgcn_sched_barrier(0);  // loads into registers still in use would get others, copied after a wait
      load_w(J, t + R);
      // step t + 1's rows, loaded in step t + 1 - D, are there when at most the loads behind them are in flight
      // (weights of that step, rows and weights of the steps since; the scales may lie between as well)
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(4 + 6 * (D - 1)) : "memory");
      bar();
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no write to LDS may outlive its rows
  __syncthreads();
  if constexpr (SWIGLU) {
    const int col = nb * 128 + wave * 16 + lg * 4;
#pragma unroll
    for (int i = 0; i < MS; ++i) {
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][0][j] = silu_f32(acc[i][0][j]) * acc[i][1][j];
        top = fmaxf(top, fp8_magnitude(acc[i][0][j]));
      }
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      if (lg == 0) tops[wave][i * 16 + lr] = top;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MS; ++i) {
      float top = 0.0f;
#pragma unroll
      for (int v = 0; v < 8; ++v) top = fmaxf(top, tops[v][i * 16 + lr]);
      const int64_t row = m0 + i * 16 + lr;
      const float h[4] = {acc[i][0][0], acc[i][0][1], acc[i][0][2], acc[i][0][3]};
      if (row < m0 + n) store_h(a, h, top, row, nb, col, wave == 0 && lg == 0);
    }
    __syncthreads();
  } else {
#pragma unroll
    for (int i = 0; i < MS; ++i) {
      const int64_t row = m0 + i * 16 + lr;
      if (row < m0 + n)
#pragma unroll
        for (int b = 0; b < 2; ++b) store_y(a, acc[i][b], row, (unit + b) * 16 + lg * 4);
    }
  }
}

template <bool SWIGLU>
__global__ __launch_bounds__(512) void fp8_medium_kernel(const Fp8GemmArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t s0[MD_STAGE], s1[MD_STAGE], s2[MD_STAGE], s3[MD_STAGE];
  __shared__ float tops[SWIGLU ? 8 : 1][MD_ROWS];
  int begin, end;
  const int nb = blockIdx.x, g = fp8_nth_group(a, blockIdx.y, a.xp ? kFp8FewRows : INT_MAX, begin, end);
  if (g < 0) return;  // (groups of more rows: the large kernel's)
  for (int m0 = begin; m0 < end; m0 += MD_ROWS) {
    const int n = min(MD_ROWS, end - m0);
    switch ((n + 15) / 16) {
#define MOE_ROWS(MS) \
  case MS: medium_rows<SWIGLU, MS>(a, g, nb, m0, n, s0, s1, s2, s3, tops); break
      MOE_ROWS(1);
      MOE_ROWS(2);
      MOE_ROWS(3);
      MOE_ROWS(4);
      MOE_ROWS(5);
      MOE_ROWS(6);
      MOE_ROWS(7);
      MOE_ROWS(8);
#undef MOE_ROWS
    }
  }
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8GemmArgs &a, hipStream_t s) {
  const bool swiglu = a.h8 != nullptr;
  const int groups = std::min(a.num_groups, a.rows_max);
  auto grid = [&](int cols) { return dim3((unsigned)((a.n_out + cols - 1) / cols), (unsigned)groups); };
  if (a.xp) {
    const hipError_t e = launch_fp8_gemm_large(a, s);
    if (e != hipSuccess) return e;
  }
  if (std::min(a.group_rows_max, a.rows_max) <= 16) {
    const int ss = getenv("SS") ? atoi(getenv("SS")) : 1;
    if (swiglu && ss == 2)
      hipLaunchKernelGGL((fp8_small_kernel<true, 8, 2>), grid(128), dim3(1024), 0, s, a);
    else if (swiglu)
      hipLaunchKernelGGL((fp8_small_kernel<true, 8, 1>), grid(128), dim3(512), 0, s, a);
    else if ((int64_t)groups * ((a.n_out + 63) / 64) < 128)
      hipLaunchKernelGGL((fp8_small_kernel<false, 2, 2>), grid(32), dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL((fp8_small_kernel<false, 4, 1>), grid(64), dim3(256), 0, s, a);
  } else {
    if (swiglu)
      hipLaunchKernelGGL((fp8_medium_kernel<true>), grid(128), dim3(512), 0, s, a);
    else
      hipLaunchKernelGGL((fp8_medium_kernel<false>), grid(256), dim3(512), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace moe
