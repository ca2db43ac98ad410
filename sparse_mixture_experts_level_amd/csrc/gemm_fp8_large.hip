// Grouped products in 8 bits for groups of many rows (layouts in fp8.hpp), bound by the matrix cores.
//
// 256 rows x 256 weight rows a workgroup (for gate_up 128 columns of H: 16 gate and 16 up rows in turn), eight
// waves of 128 x 64, 32x32x64 instructions with their operands' scales (the
// blocks' scales cost nothing).  Both operands go from memory to LDS without registers, a step of 64 of K as
// 1 KB pieces that are consecutive in memory and lie in LDS as the instruction reads them: for 16 rows, [4 chunks of
// 16 codes][16 rows], so that sixteen lanes read 256 consecutive bytes.  The rows are copied into that
// layout beforehand (fp8_pack_rows_kernel); H is written in it.  Four stages, three steps ahead; the
// two waves of each SIMD take turns, one computing while the other loads and reads
// (the bf16 kernel's schedule for groups of many rows: the same bytes and cycles a step, twice the products).
#include <algorithm>

#include "fp8.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr int LG_TILE = kFp8LargeRows * 64;  // bytes of an operand's stage: 256 rows, 64 of K

__device__ __forceinline__ int large_tiles(const Fp8GemmArgs &a, int g) {
  int begin, end;
  fp8_group_rows(a, g, begin, end);
  return fp8_large_tiles(end - begin);
}

// Tile m -> its group (-1 past the last), the group's first tile and count, and the number of all tiles; the
// same in every lane.
__device__ __forceinline__ void find_tile(const Fp8GemmArgs &a, int m, int &group, int &first, int &count) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  group = -1;
  first = count = 0;
  for (int g0 = 0; g0 < a.num_groups; g0 += 64) {
    const int mine = g0 + lane < a.num_groups ? large_tiles(a, g0 + lane) : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o, 64);
      if (lane >= o) incl += v;
    }
    const uint64_t hit = __ballot(base + incl > m);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      group = g0 + l;
      first = base + __shfl(incl - mine, l, 64);
      count = __shfl(mine, l, 64);
      return;
    }
    base += __shfl(incl, 63, 64);
  }
}

__device__ __forceinline__ int all_tiles(const Fp8GemmArgs &a) {
  int sum = 0;
  for (int g = threadIdx.x & 63; g < a.num_groups; g += 64) sum += large_tiles(a, g);
  return __builtin_amdgcn_readfirstlane(group_reduce<64>(sum, [](int x, int y) { return x + y; }));
}

__device__ __forceinline__ f32x16 mfma_fp8_32(i32x8 a, i32x8 b, f32x16 c, uint32_t sa, uint32_t sb, int byte) {
  switch (byte) {
    case 0: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, (int)sa, 0, (int)sb);
    case 1: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 1, (int)sa, 1, (int)sb);
    case 2: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 2, (int)sa, 2, (int)sb);
    default: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 3, (int)sa, 3, (int)sb);
  }
}

template <bool SWIGLU>
__global__ __launch_bounds__(512, 1) void fp8_large_kernel(const Fp8GemmArgs a, int n_tiles) {
  constexpr int NBUF = 4;
  __shared__ __attribute__((aligned(1024))) uint8_t sA0[LG_TILE], sA1[LG_TILE], sA2[LG_TILE], sA3[LG_TILE];
  __shared__ __attribute__((aligned(1024))) uint8_t sB0[LG_TILE], sB1[LG_TILE], sB2[LG_TILE], sB3[LG_TILE];
  auto bufA = [&](int b) -> uint8_t * { return b == 0 ? sA0 : b == 1 ? sA1 : b == 2 ? sA2 : sA3; };
  auto bufB = [&](int b) -> uint8_t * { return b == 0 ? sB0 : b == 1 ? sB1 : b == 2 ? sB2 : sB3; };
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / 4, wn = wave % 4, lr = lane & 31, lh = lane >> 5;
  // (offsets that decrease could count rows twice: no tile past those that the packed copies have room for)
  const int tiles_max = gridDim.x / n_tiles, tiles = min(all_tiles(a), tiles_max), blocks = tiles * n_tiles;
  if ((int)blockIdx.x >= blocks) return;
  const int lin = xcd_remap(blockIdx.x, blocks);
  int g, mt_first, mt_count;
  find_tile(a, lin / n_tiles, g, mt_first, mt_count);
  if (g < 0) return;
  g = __builtin_amdgcn_readfirstlane(g);
  mt_first = __builtin_amdgcn_readfirstlane(mt_first);
  mt_count = __builtin_amdgcn_readfirstlane(mt_count);
  const int local = lin - mt_first * n_tiles;
  int begin, end;
  fp8_group_rows_uniform(a, g, begin, end);
  int mt, nt;
  if (end - begin <= (SWIGLU ? 2 : 1) * a.n_out) {  // the weights are larger: their tile outermost
    nt = local / mt_count;
    mt = local - nt * mt_count;
  } else {  // bands of four row tiles, weight tile outer within a band
    constexpr int BAND = 4;
    const int band = local / (BAND * n_tiles), r = local - band * BAND * n_tiles;
    const int bm = min(BAND, mt_count - band * BAND);
    nt = r / bm;
    mt = band * BAND + (r - nt * bm);
  }
  mt = __builtin_amdgcn_readfirstlane(mt);
  nt = __builtin_amdgcn_readfirstlane(nt);
  const int per = fp8_tile_rows(end - begin, mt_count);
  const int m0 = begin + mt * per, rows = min(per, end - m0), m_tile = mt_first + mt;
  if (m_tile >= tiles_max) return;
  const int row_blocks = (rows + 31) / 32, mine = max(0, min(4, row_blocks - wm * 4));  // of 32 rows: the tile's, this wave's
  const int kt = fp8_blocks(a.K), nk = 2 * kt, ks = fp8_scale_bytes(a.K);
  const int64_t abytes = (int64_t)kFp8LargeRows * kt * kFp8Block;
  const int64_t wbytes = fp8_group_bytes(a.n_out, a.K, SWIGLU);
  const rsrc_t ares = make_rsrc(a.xp + m_tile * abytes, (uint32_t)abytes);
  const rsrc_t wres = make_rsrc(a.w8 + g * wbytes, (uint32_t)wbytes);
  const rsrc_t sres = make_rsrc(a.xp_scale + (int64_t)m_tile * kFp8LargeRows * ks, (uint32_t)(kFp8LargeRows * ks));
  // this wave's pieces of a stage: 16-row blocks 2 wave and 2 wave + 1 of both operands
  uint32_t aoff[2], boff[2], wstep;
  const int wblocks = (a.n_out + 15) / 16 * (SWIGLU ? 2 : 1);
  const uint32_t wtile = fp8_block_offset(nt * 16, wblocks, kt, wstep);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t at = (uint32_t)(2 * wave + i) * 1024u + (uint32_t)lane * 16u;
    aoff[i] = wave < row_blocks ? at : kOob;
    boff[i] = nt * 16 + 2 * wave + i < wblocks ? wtile + at : kOob;
  }
  auto issue = [&](int s, int b) {
    const uint32_t ka = (uint32_t)s * (uint32_t)LG_TILE, kb = (uint32_t)s * wstep;
    const bool in = s < nk;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      buf_ld16_lds(ares, in && aoff[i] != kOob ? aoff[i] + ka : kOob, bufA(b) + (2 * wave + i) * 1024);
      buf_ld16_lds(wres, in && boff[i] != kOob ? boff[i] + kb : kOob, bufB(b) + (2 * wave + i) * 1024);
    }
  };
  const int sblocks = fp8_blocks(a.n_out);
  const uint8_t *wscale = a.w_scale + ((int64_t)g * sblocks + (SWIGLU ? nt : min(nt * 2 + wn / 2, sblocks - 1))) *
                                          (SWIGLU ? 2 : 1) * ks;
  uint32_t sx[4], sw[2];
  // four blocks of K, eight steps; past K zeros, or the last ones again
  auto load_scales = [&](int q) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sx[i] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(
          sres, (uint32_t)(q * kFp8LargeRows + wm * 128 + i * 32 + lr) * 4u, 0, 0);
#pragma unroll
    for (int j = 0; j < 2; ++j) sw[j] = scalar_load(wscale + (SWIGLU ? j * ks : 0) + min(4 * q, ks - 4));
  };

  f32x16 acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x16{};
  // This lane's 32 codes of a row, chunks 2 lh and 2 lh + 1, in the first of the wave's row and weight blocks (one offset
  // and constants from there: with the sums formed anew for each read the compiler lost track of which
  // stage a read is of, and waited for every load in flight).
  const int half = (lane >> 4) & 1, at = (2 * lh) * 256 + (lane & 15) * 16;
  const int a_at = (wm * 8 + half) * 1024 + at, b_at = (wn * 4 + (SWIGLU ? 2 : 1) * half) * 1024 + at;
  {
    // A wave in mem(s) issues step s + 3 and completes its own loads of step s + 1, before the barrier that
    // precedes every read of them; a stage is refilled only after the barrier that follows both groups' reads.
    const bool second = wave >= 4;
    u32x4 af[4][2], bf[2][2];
    uint32_t cx[4], cw[2];
    auto mem = [&](int s, int b) {
      issue(s + 3, (b + 3) % NBUF);
      asm volatile("s_waitcnt vmcnt(8)" ::: "memory");  // the two younger steps' may stay in flight
      const uint8_t *la = bufA(b % NBUF), *lb = bufB(b % NBUF);
      const uint8_t *pa = la + a_at, *pb = lb + b_at;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= mine) break;
        af[i][0] = *reinterpret_cast<const u32x4 *>(pa + i * 2048);
        af[i][1] = *reinterpret_cast<const u32x4 *>(pa + i * 2048 + 256);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        bf[j][0] = *reinterpret_cast<const u32x4 *>(pb + j * (SWIGLU ? 1024 : 2048));
        bf[j][1] = *reinterpret_cast<const u32x4 *>(pb + j * (SWIGLU ? 1024 : 2048) + 256);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    };
    auto comp = [&](int b) {
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= mine) break;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = mfma_fp8_32(fp8_operand(bf[j][0], bf[j][1]), fp8_operand(af[i][0], af[i][1]), acc[i][j], cw[j], cx[i],
                                  b / 2);
      }
      __builtin_amdgcn_s_setprio(0);
    };
    auto bar = [&]() {
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
    };
    auto next_scales = [&](int q) {  // those of the eight steps that begin; the following ones are loaded
#pragma unroll
      for (int i = 0; i < 4; ++i) cx[i] = sx[i];
#pragma unroll
      for (int j = 0; j < 2; ++j) cw[j] = sw[j];
      load_scales(q + 1);
    };
    load_scales(0);
#pragma unroll
    for (int b = 0; b < 3; ++b) issue(b, b);
    asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
    bar();
    if (second) bar();
    int s0 = 0;
    for (; s0 + 8 <= nk; s0 += 8) {
      next_scales(s0 / 8);
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        mem(s0 + b, b);
        bar();
        comp(b);
        bar();
      }
    }
    if (s0 < nk) {
      next_scales(s0 / 8);
#pragma unroll
      for (int b = 0; b < 7; ++b) {
        if (s0 + b >= nk) break;
        mem(s0 + b, b);
        bar();
        comp(b);
        bar();
      }
    }
    if (!second) bar();
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no LDS write may outlive the block
  __syncthreads();

  // Block (i, j): lane l holds row wm * 128 + i * 32 + l % 32 and, per q = 0..3, columns 8 q + 4 (l / 32) .. + 3 of its 32.
  if constexpr (SWIGLU) {
    float *tops = reinterpret_cast<float *>(sB0);  // [4 waves of columns][256 rows]
    float top[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      top[i] = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        acc[i][0][e] = silu_f32(acc[i][0][e]) * acc[i][1][e];
        top[i] = fmaxf(top[i], fp8_magnitude(acc[i][0][e]));
      }
      top[i] = fmaxf(top[i], __shfl_xor(top[i], 32, 64));
      if (lh == 0) tops[wn * 256 + wm * 128 + i * 32 + lr] = top[i];
    }
    __syncthreads();
    // the tile's 256 x 128 codes in H's packed layout: 16-row blocks' first KB (columns below 64) in sA0, second in sA1
    const int hs = fp8_scale_bytes(a.n_out), ht = fp8_blocks(a.n_out);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = wm * 128 + i * 32 + lr;
      const float t = fmaxf(fmaxf(tops[row], tops[256 + row]), fmaxf(tops[512 + row], tops[768 + row]));
      const uint32_t byte = fp8_scale_byte(t);
      const float inv = fp8_inverse(byte);
      uint8_t *o = (wn < 2 ? sA0 : sA1) + (row >> 4) * 1024 + (wn & 1) * 512 + (row & 15) * 16 + lh * 4;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint32_t *>(o + (q >> 1) * 256 + (q & 1) * 8) =
            fp8_codes(acc[i][0][4 * q] * inv, acc[i][0][4 * q + 1] * inv, acc[i][0][4 * q + 2] * inv,
                      acc[i][0][4 * q + 3] * inv);
      if (wn == 0 && lh == 0)
        a.hp_scale[(int64_t)m_tile * kFp8LargeRows * hs + ((nt / 4) * kFp8LargeRows + row) * 4 + nt % 4] = (uint8_t)byte;
    }
    __syncthreads();
    uint8_t *hp = a.hp + ((int64_t)m_tile * ht + nt) * (2 * LG_TILE);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const int q = threadIdx.x + 512 * v;  // 16-byte piece of the 16 KB
        stg16(hp + p * LG_TILE + q * 16, *reinterpret_cast<const u32x4 *>((p ? sA1 : sA0) + q * 16));
      }
  } else {
    // bf16: each wave's 128 rows x 64 columns through its own 16 KB, 128-byte rows, 16-byte chunk c of row r at
    // c ^ ((r >> 1) & 7), out as whole pieces along the rows
    uint8_t *stage = wave < 4 ? bufA(wave) : bufB(wave - 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = i * 32 + lr;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint2 *>(stage + row * 128 + (((j * 4 + q) ^ ((row >> 1) & 7)) << 4) + lh * 8) =
              uint2{pack_bf16x2(acc[i][j][4 * q], acc[i][j][4 * q + 1]), pack_bf16x2(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3])};
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const int c = lane & 7, col = nt * 256 + wn * 64 + c * 8;
#pragma unroll
    for (int it = 0; it < 16; ++it) {
      const int row = it * 8 + (lane >> 3), grow = wm * 128 + row;
      const u32x4 v = *reinterpret_cast<const u32x4 *>(stage + row * 128 + ((c ^ ((row >> 1) & 7)) << 4));
      if (grow >= rows) continue;
      bf16_t *o = a.y + (int64_t)(m0 + grow) * a.n_out + col;
      if (col + 8 <= a.n_out) {
        *reinterpret_cast<u32x4_any *>(o) = v;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + e < a.n_out) o[e] = (bf16_t)(v[e / 2] >> (16 * (e % 2)));
      }
    }
  }
}

// The rows of the tiles, and their scales as [4 blocks of K][256 rows] words, for fp8_large_kernel: one
// workgroup a tile and four blocks of K, 512 bytes of a row by 32 threads.
__global__ __launch_bounds__(256) void fp8_pack_rows_kernel(const Fp8GemmArgs a, uint8_t *__restrict__ xp,
                                                            uint8_t *__restrict__ xp_scale) {
  const int kt = fp8_blocks(a.K), kp = fp8_row_bytes(a.K), ks = fp8_scale_bytes(a.K), quads = ks / 4;
  const int b0 = (blockIdx.x % quads) * 4, m_tile = blockIdx.x / quads;
  int g, first, count, begin, end;
  find_tile(a, m_tile, g, first, count);
  if (g < 0) return;
  fp8_group_rows(a, g, begin, end);
  const int per = fp8_tile_rows(end - begin, count), m0 = begin + (m_tile - first) * per, rows = min(per, end - m0);
  auto source = [&](int r) -> int64_t {  // -1: zeros
    if (r >= rows) return -1;
    if (!a.row_index) return m0 + r;
    const int s = a.row_index[m0 + r];
    return (uint32_t)s < (uint32_t)a.x_rows ? s : -1;
  };
  const int r0 = threadIdx.x >> 5, c = threadIdx.x & 31, b = b0 + (c >> 3);  // a block's 16-byte piece c & 7
  for (int i0 = 0; i0 < rows; i0 += 64) {
    u32x4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t s = source(i0 + i * 8 + r0);
      v[i] = u32x4{0u, 0u, 0u, 0u};
      if (s >= 0 && b < kt) v[i] = ldg16(a.x8 + s * kp + b0 * 128 + c * 16);
    }
    if (b < kt) {
      uint8_t *o = xp + (((int64_t)m_tile * kt + b) * 2 + (c >> 2 & 1)) * LG_TILE + (c & 3) * 256;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = i0 + i * 8 + r0;
        if (r < 256) stg16(o + (r >> 4) * 1024 + (r & 15) * 16, v[i]);
      }
    }
  }
  const int64_t s = source(threadIdx.x);
  const uint32_t w = s >= 0 ? *reinterpret_cast<const uint32_t *>(a.x_scale + s * ks + b0) : 0u;
  reinterpret_cast<uint32_t *>(xp_scale)[((int64_t)m_tile * quads + b0 / 4) * kFp8LargeRows + threadIdx.x] = w;
}

}  // namespace

hipError_t launch_fp8_pack_rows(const Fp8GemmArgs &a, uint8_t *xp, uint8_t *xp_scale, hipStream_t s) {
  const int64_t grid = fp8_large_tiles_max(a.rows_max, a.num_groups) * (fp8_scale_bytes(a.K) / 4);
  if (grid == 0) return hipSuccess;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL(fp8_pack_rows_kernel, dim3((unsigned)grid), dim3(256), 0, s, a, xp, xp_scale);
  return hipGetLastError();
}

hipError_t launch_fp8_gemm_large(const Fp8GemmArgs &a, hipStream_t s) {
  const bool swiglu = a.hp != nullptr;
  const int n_tiles = (a.n_out + (swiglu ? 127 : 255)) / (swiglu ? 128 : 256);
  const int64_t grid = fp8_large_tiles_max(a.rows_max, a.num_groups) * n_tiles;
  if (grid == 0) return hipSuccess;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  if (swiglu)
    hipLaunchKernelGGL((fp8_large_kernel<true>), dim3((unsigned)grid), dim3(512), 0, s, a, n_tiles);
  else
    hipLaunchKernelGGL((fp8_large_kernel<false>), dim3((unsigned)grid), dim3(512), 0, s, a, n_tiles);
  return hipGetLastError();
}

}  // namespace moe
