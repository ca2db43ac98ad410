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
// sum: enough to move one code of H in two thousand, which takes the FFN's error from 1.7e-3 of its norm to 1.8 .. 2.1e-3).
#include <algorithm>
#include <climits>

#include "gemm_fp8.hpp"

namespace moe {

namespace {

// Few rows: 16 of them at a time, one block after the other.  A workgroup has 16 U columns of H (each wave 16, NB = 2
// blocks of weights: gate and up) or 16 U NB of y; each wave one of KS parts of K, whose sums the first part's waves add
// in order.  Rows are read from the caches in the operand layout, two steps ahead, with the weights, R steps of 128
// ahead (8 KB a wave; twice as many made the FFN of 32 x 8 rows x 2880 x 2880 147 us for 141, one token's gate_up
// 21.1 for 20.1: memory serves fewer requests at a time better), all in registers: no LDS, no barrier.  The weights are the
// matrix instruction's first operand, so that a lane holds four consecutive columns of one row.
// Measured: one token, 4 of 32 experts of 2880 x 2880, gate_up 20.1 us and down 11.0 (66 and 33 MB: 3.3 and 3.0 TB/s from 92 and
// 180 workgroups, of which one CU takes in 50 GB/s at most, after 4.5 us of launch and lookups); 16 tokens 5.6 TB/s.
template <bool SWIGLU, int U, int KS, int NB, int R>
__global__ __launch_bounds__(64 * U * KS, 4) void fp8_small_kernel(const Fp8GemmArgs a) {
  constexpr int XR = 2, NS = SWIGLU ? 2 : 1;  // NS: scales a wave
  static_assert(!SWIGLU || (U == 8 && NB == 2), "a block of H's columns a workgroup");
  static_assert(4 % R == 0, "a word of scales a trip");
  __shared__ float tops[SWIGLU ? 8 : 1][16];
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
  const int unit = nb * U + u, blocks = (a.n_out + 15) / 16 * NS;  // of 16 weight rows
  const int64_t wbytes = fp8_group_bytes(a.n_out, a.K, SWIGLU);
  const rsrc_t wres = make_rsrc(a.w8 + g * wbytes, (uint32_t)wbytes);
  uint32_t half;  // (gate and up blocks are neighbours)
  const uint32_t wbase = fp8_block_offset(unit * NB, blocks, kt, half) + (uint32_t)lane * 16u;
  const int tw0 = unit * NB < blocks ? te : 0, tw1 = unit * NB + 1 < blocks ? te : 0;  // no weights past the last block
  const int sblocks = fp8_blocks(a.n_out);
  const uint8_t *wscale = a.w_scale + ((int64_t)g * sblocks + min(unit * NB / NS / 8, sblocks - 1)) * NS * ks;
  for (int left = end - begin; left > 0; left -= 16) {  // (m0 + 16 may pass 2^31)
    const int m0 = end - left, n = min(16, left);
    u32x4 w[R][NB][2], x[XR][2];
    uint32_t sx, nx, sw[NS], nw[NS];
    auto load_w = [&](int j, int t) {  // steps past the part's end read zeros
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int tw = SWIGLU || b == 0 ? tw0 : tw1;
        const uint32_t o = t < tw ? wbase + (uint32_t)(2 * t) * half + (uint32_t)b * 1024u : kOob;
        w[j][b][0] = buf_ld16_nt(wres, o);
        w[j][b][1] = buf_ld16_nt(wres, t < tw ? o + half : kOob);
      }
    };
#pragma unroll
    for (int j = 0; j < R; ++j) load_w(j, tb + j);
    const Fp8Rows rows(a, m0, n);
    const uint32_t src = rows.row(a, m0, lr, n);
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
      for (int b = 0; b < NS; ++b) nw[b] = scalar_load(wscale + b * ks + at);
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
    for (int t0 = tb; t0 < te; t0 += 4) {
      auto step = [&](auto jc) {
        constexpr int J = decltype(jc)::value;
        const int t = t0 + J;
        if constexpr (J == 0) {
          const int left = te - t;  // blocks of this part: the padding's scales are not looked at
          const uint32_t keep = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
          sx = nx & keep;
#pragma unroll
          for (int b = 0; b < NS; ++b) sw[b] = nw[b] & keep;
          load_scales(t + 4);
        }
        const int shift = fp8_shift<J>(sw[0], sw[NS - 1]);
        const float fx = fp8_shifted<J>(sx, shift);
        float fw[NS];
#pragma unroll
        for (int b = 0; b < NS; ++b) fw[b] = fp8_shifted<J>(sw[b], -shift);
#pragma unroll
        for (int m = 0; m < 4; ++m) {  // 32 of K: eight of each lane's 32 codes
          const u32x4 xb = fp8_to_bf16(x[J % XR][m / 2][2 * (m % 2)], x[J % XR][m / 2][2 * (m % 2) + 1], fx);
#pragma unroll
          for (int b = 0; b < NB; ++b)
            acc[b] = mfma16(fp8_to_bf16(w[J % R][b][m / 2][2 * (m % 2)], w[J % R][b][m / 2][2 * (m % 2) + 1], fw[b % NS]), xb,
                            acc[b]);
        }
        __builtin_amdgcn_sched_barrier(0);  // loads into registers still in use would get others, copied after a wait
        load_x(J % XR, t + XR);
        load_w(J % R, t + R);
      };
      step(std::integral_constant<int, 0>{});
      step(std::integral_constant<int, 1>{});
      step(std::integral_constant<int, 2>{});
      step(std::integral_constant<int, 3>{});
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
    const int col = unit * 16 * NB / NS + lg * 4;
    const int64_t row = (int64_t)m0 + lr;
    if constexpr (SWIGLU) {
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
      if (part == 0 && lr < n) {
#pragma unroll
        for (int v = 0; v < 8; ++v) top = fmaxf(top, tops[v][lr]);
        store_h(a, h, top, row, nb, col, u == 0 && lg == 0);
      }
    } else if (part == 0 && lr < n) {
#pragma unroll
      for (int b = 0; b < NB; ++b) store_y(a, acc[b], row, col + b * 16);
    }
    if (SWIGLU || KS > 1) __syncthreads();  // the next rows use the same LDS
  }
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8GemmArgs &a, hipStream_t s) {
  if (std::min(a.group_rows_max, a.rows_max) > kFp8SmallRows) return launch_fp8_gemm_rows(a, s);
  const int groups = std::min(a.num_groups, a.rows_max);
  auto grid = [&](int cols) { return dim3((unsigned)((a.n_out + cols - 1) / cols), (unsigned)groups); };
  // Linear: a wave takes two blocks of 16 columns, so that the rows are read half as often, where that leaves a workgroup a
  // CU (32 groups of 16 rows, 2048 x 7168: 114 -> 101 us; of one row: 83 -> 79; but 4 groups, 2880 x 2880, 92 workgroups:
  // 11.0 -> 12.2), and a part of K where even one block leaves half of them idle (1 x 2048 x 7168: 8.6 -> 7.9).
  if (a.h8)
    hipLaunchKernelGGL((fp8_small_kernel<true, 8, 1, 2, 2>), grid(128), dim3(512), 0, s, a);
  else if ((int64_t)groups * ((a.n_out + 63) / 64) < 128)
    hipLaunchKernelGGL((fp8_small_kernel<false, 2, 2, 1, 4>), grid(32), dim3(256), 0, s, a);
  else if ((int64_t)groups * ((a.n_out + 127) / 128) < 256)
    hipLaunchKernelGGL((fp8_small_kernel<false, 4, 1, 1, 4>), grid(64), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((fp8_small_kernel<false, 4, 1, 2, 2>), grid(128), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
