// Grouped products in 8-bit floating point with a scale for each block of 128 (layouts in fp8.hpp):
//   out[r][n] = sum_b 2^(sx[r][b] + sw[n / 128][b]) sum_{k in block b} x8[r][k] w8[n][k]
// for the rows r of each group, bf16; and the gate_up form, whose epilogue forms
//   H[r][n] = silu(G[r][n]) U[r][n],  silu(z) = z / (1 + exp(-z))
// from the float sums and quantises it again, a scale for each 128 columns of a row.
#include <algorithm>

#include "fp8.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

// One workgroup: 128 output columns of one group, eight waves of 16 columns (and, for gate_up, the 16 gate
// and the 16 up rows of each), row blocks of 16 MS rows one after the other.  The weights are the
// matrix instruction's first operand, so that a lane holds four consecutive columns of one row.
template <bool SWIGLU, int MS>
__global__ __launch_bounds__(512) void fp8_stream_kernel(const Fp8GemmArgs a) {
  constexpr int NB = SWIGLU ? 2 : 1;
  __shared__ float tops[8][16 * MS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lr = lane & 15, lg = lane >> 4;
  const int n_blocks = fp8_blocks(a.n_out);
  const int g = blockIdx.x / n_blocks, nb = blockIdx.x - g * n_blocks;
  const int begin = min(max(a.offsets[g], 0), a.rows_max), end = min(max(a.offsets[g + 1], begin), a.rows_max);
  if (begin >= end) return;
  const int kt = fp8_blocks(a.K), kp = fp8_row_bytes(a.K), ks = fp8_scale_bytes(a.K);
  const int unit = nb * 8 + wave, units = (a.n_out + 15) / 16;
  const int64_t wbytes = (int64_t)units * NB * kt * kFp8Tile;
  const rsrc_t wres = make_rsrc(a.w8 + g * wbytes, (uint32_t)wbytes);
  const uint32_t woff = unit < units ? (uint32_t)(unit * NB * kt * kFp8Tile + lane * 16) : kOob;
  const uint8_t *wscale = a.w_scale + (int64_t)(g * n_blocks + nb) * NB * ks;
  for (int m0 = begin; m0 < end; m0 += 16 * MS) {
    const bool gather = a.row_index != nullptr;
    const rsrc_t xres = gather ? make_rsrc(a.x8, (uint32_t)((int64_t)a.x_rows * kp))
                               : make_rsrc(a.x8 + (int64_t)m0 * kp, (uint32_t)(min(16 * MS, end - m0) * kp));
    const rsrc_t sres = gather ? make_rsrc(a.x_scale, (uint32_t)((int64_t)a.x_rows * ks))
                               : make_rsrc(a.x_scale + (int64_t)m0 * ks, (uint32_t)(min(16 * MS, end - m0) * ks));
    uint32_t xoff[MS], soff[MS];
#pragma unroll
    for (int i = 0; i < MS; ++i) {
      const int r = i * 16 + lr;
      uint32_t src = (uint32_t)r;
      bool ok = m0 + r < end;
      if (gather && ok) {
        src = (uint32_t)a.row_index[m0 + r];
        ok = src < (uint32_t)a.x_rows;
      }
      xoff[i] = ok ? src * (uint32_t)kp + (uint32_t)lg * 16u : kOob;
      soff[i] = ok ? src * (uint32_t)ks : kOob;
    }
    f32x4 acc[MS][NB];
#pragma unroll
    for (int i = 0; i < MS; ++i)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[i][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < kt; k0 += 4) {
      const uint32_t keep = kt - k0 >= 4 ? ~0u : (1u << (8 * (kt - k0))) - 1u;  // scales of blocks that exist
      uint32_t sx[MS], sw[NB];
#pragma unroll
      for (int i = 0; i < MS; ++i)
        sx[i] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(sres, soff[i] == kOob ? kOob : soff[i] + k0, 0, 0) & keep;
#pragma unroll
      for (int b = 0; b < NB; ++b) sw[b] = *reinterpret_cast<const uint32_t *>(wscale + b * ks + k0) & keep;
      auto step = [&](auto jc) {
        constexpr int J = decltype(jc)::value;
        const bool in = k0 + J < kt;
        i32x8 w[NB], x[MS];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint32_t o = in && woff != kOob ? woff + (uint32_t)((b * kt + k0 + J) * kFp8Tile) : kOob;
          w[b] = fp8_operand(buf_ld16_nt(wres, o), buf_ld16_nt(wres, o == kOob ? kOob : o + 1024u));
        }
#pragma unroll
        for (int i = 0; i < MS; ++i) {
          const uint32_t o = in && xoff[i] != kOob ? xoff[i] + (uint32_t)((k0 + J) * 128) : kOob;
          x[i] = fp8_operand(buf_ld16(xres, o), buf_ld16(xres, o == kOob ? kOob : o + 64u));
        }
#pragma unroll
        for (int i = 0; i < MS; ++i)
#pragma unroll
          for (int b = 0; b < NB; ++b) acc[i][b] = mfma_fp8_16<J>(w[b], x[i], acc[i][b], sw[b], sx[i]);
      };
      step(std::integral_constant<int, 0>{});
      step(std::integral_constant<int, 1>{});
      step(std::integral_constant<int, 2>{});
      step(std::integral_constant<int, 3>{});
    }
    const int col = nb * 128 + wave * 16 + lg * 4;
    if constexpr (SWIGLU) {
      float h[MS][4];
#pragma unroll
      for (int i = 0; i < MS; ++i) {
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[i][j] = silu_f32(acc[i][0][j]) * acc[i][1][j];
          top = fmaxf(top, fp8_magnitude(h[i][j]));
        }
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        if (lg == 0) tops[wave][i * 16 + lr] = top;
      }
      __syncthreads();
      const int hp = fp8_row_bytes(a.n_out), hs = fp8_scale_bytes(a.n_out);
#pragma unroll
      for (int i = 0; i < MS; ++i) {
        float top = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) top = fmaxf(top, tops[w][i * 16 + lr]);
        const uint32_t byte = fp8_scale_byte(top);
        const float inv = fp8_inverse(byte);
        const int64_t row = m0 + i * 16 + lr;
        if (row < end) {
          *reinterpret_cast<uint32_t *>(a.h8 + row * hp + col) =
              fp8_codes(h[i][0] * inv, h[i][1] * inv, h[i][2] * inv, h[i][3] * inv);
          if (wave == 0 && lg == 0) a.h_scale[row * hs + nb] = (uint8_t)byte;
        }
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int i = 0; i < MS; ++i) {
        const int64_t row = m0 + i * 16 + lr;
        if (row >= end) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (col + j < a.n_out) a.y[row * a.n_out + col + j] = f32_to_bf16(acc[i][0][j]);
      }
    }
  }
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8GemmArgs &a, hipStream_t s) {
  const unsigned grid = (unsigned)(a.num_groups * fp8_blocks(a.n_out));
  if (a.h8)
    hipLaunchKernelGGL((fp8_stream_kernel<true, 2>), dim3(grid), dim3(512), 0, s, a);
  else
    hipLaunchKernelGGL((fp8_stream_kernel<false, 2>), dim3(grid), dim3(512), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
