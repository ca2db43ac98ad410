// Grouped products in 8 bits for groups of more than 16 rows (layouts in fp8.hpp).
//
// Many rows, bound by the matrix cores (4096 x 4096 x 14336: 177 us, 2.7 PFLOP/s beside packing; 8 x 1024 rows, 4096 x
// 14336 gate_up 847 us, 2.3 PFLOP/s at the clock that this long a launch leaves; a tile's begin and end 10 us of its 53):
// 256 rows x 256 weight rows a workgroup (for gate_up 128 columns of H: 16 gate and 16 up rows in turn), eight
// waves of 128 x 64, 32x32x64 instructions with their operands' scales (the
// blocks' scales cost nothing).  Both operands go from memory to LDS without registers, a step of 64 of K as
// 1 KB pieces that are consecutive in memory and lie in LDS as the instruction reads them: for 16 rows, [4 chunks of
// 16 codes][16 rows], so that sixteen lanes read 256 consecutive bytes.  The rows are copied into that
// layout beforehand (fp8_pack_rows_kernel) or, for few column tiles, taken as they are, half a line at a time; H is written in
// it.  Four stages, three steps ahead; the
// two waves of each SIMD take turns, one computing while the other loads and reads
// (the bf16 kernel's schedule for groups of many rows: the same bytes and cycles a step, twice the products).
#include <algorithm>
#include <climits>

#include "gemm_fp8.hpp"

namespace moe {

namespace {

constexpr int LG_TILE = kFp8LargeRows * 64;  // bytes of an operand's stage: 256 rows, 64 of K

// Block `block` of a launch of per_tile column tiles: the tiles of the groups of many rows, group after group, a block for
// each column tile; then the groups of few (any number of rows where none is announced to have many), a block for each of
// `chunks` ranges of column tiles; all of them, or those past the last whole 256, again for each further part of K.  One
// pass over the offsets, two for more than 64 groups; all results in scalar registers.
struct Fp8Tile {
  int g, begin, end;  // -1: there is no such tile
  int first, count;   // the group's tiles, numbered over all groups (count 0: few rows)
  int lin;            // the block's number among the tiles' (many rows: after the spreading)
  int tiles;          // of many rows, in all
  int part, parts;
  int col0, col1;     // few rows: the column tiles
  int slot, cut;      // the tile's place among the `cut` tiles that are cut, where those are the last round's; -1: by rows
};
enum Fp8Blocks { kPack, kProduct, kAdd };  // block: a tile; of the product's launch; of the tiles that are cut
__device__ __forceinline__ Fp8Tile find_tile(const Fp8GemmArgs &a, int tiles_max, int block, int per_tile, Fp8Blocks kind) {
  const bool spread = kind != kPack;
  const int lane = threadIdx.x & 63, G = a.num_groups;
  const int few = a.large ? kFp8FewRows : INT_MAX;
  Fp8Tile t{-1, 0, 0, 0, 0, 0, 0, 0, 1, 0, 0, -1, 0};
  int b = 0, e = 0, all = 0;
#pragma unroll 1
  for (int g0 = 0; g0 < G; g0 += 64) {
    b = e = 0;
    if (g0 + lane < G) fp8_group_rows(a, g0 + lane, b, e);
    // (offsets that decrease could count rows twice: no tile past those that the packed copies have room for, nor a sum of
    // 1024 groups past 2^31)
    t.tiles = min(t.tiles + group_reduce<64>(a.large ? fp8_large_tiles(e - b) : 0, [](int x, int y) { return x + y; }), tiles_max);
    all += __popcll(__ballot(e > b && e - b <= few));
  }
  t.tiles = __builtin_amdgcn_readfirstlane(t.tiles);
  all = __builtin_amdgcn_readfirstlane(all);
  int chunks = per_tile, columns = 1;
  if (spread && a.few_chunks && all > 0) {  // more, where fewer groups than there can be leave CUs idle
    chunks = min(per_tile, max(a.few_chunks, 256 / all));
    columns = (per_tile + chunks - 1) / chunks;
    chunks = (per_tile + columns - 1) / columns;
  }
  const int large = t.tiles * per_tile;
  all = large + all * chunks;
  if (all == 0) return t;
  int whole = 0;  // tiles of the whole rounds
  if (spread && (a.parts_cap > 1 || a.rounds)) {
    const int full = a.rounds && all == large ? all / 256 * 256 : 0, rest = all - full;
    if (full > 0 && rest > 0)
      t.parts = fp8_parts(rest, rest, 256, a.K, kFp8Parts);
    else if (full == 0 && a.parts_cap > 1)
      t.parts = fp8_parts(all, a.rows_max, per_tile, a.K, a.parts_cap);
    if (kind == kAdd) block += full;
    if (t.parts > 1) {
      whole = full;
      if (block < whole) {
        t.parts = 1;
      } else {
        t.part = (block - whole) / rest;
        block -= t.part * rest;
        t.cut = rest;
        if (full > 0) t.slot = block - whole;
      }
    }
  }
  if (block >= all || t.part >= t.parts) return t;
  // the first tiles' blocks in one contiguous range an XCD, as neighbours share operands
  const bool many = block < large;
  const int spreads = whole > 0 ? whole : large;
  const int lin = spread && block < spreads ? xcd_remap(block, spreads) : block;
  const int v = many ? lin / per_tile : t.tiles + (lin - large) / chunks;
  t.lin = lin;
  t.col0 = __builtin_amdgcn_readfirstlane((lin - large) % chunks * columns);
  t.col1 = min(per_tile, t.col0 + __builtin_amdgcn_readfirstlane(columns));
  int seen = 0;
#pragma unroll 1
  for (int g0 = 0; g0 < G; g0 += 64) {
    if (G > 64) {
      b = e = 0;
      if (g0 + lane < G) fp8_group_rows(a, g0 + lane, b, e);
    }
    const int mine = many ? fp8_large_tiles(e - b) : e > b && e - b <= few ? 1 : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int x = __shfl_up(incl, o, 64);
      if (lane >= o) incl += x;
    }
    const int want = many ? v : v - t.tiles;
    const uint64_t hit = __ballot(seen + incl > want);
    if (hit) {
      const int l = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)hit) - 1);
      t.g = g0 + l;
      t.begin = __builtin_amdgcn_readlane(b, l);
      t.end = __builtin_amdgcn_readlane(e, l);
      t.first = __builtin_amdgcn_readfirstlane(seen) + __builtin_amdgcn_readlane(incl - mine, l);
      t.count = many ? __builtin_amdgcn_readlane(mine, l) : 0;
      return t;
    }
    seen += __builtin_amdgcn_readlane(incl, 63);
  }
  return t;
}

// Row and column tile of a block of a group of many rows.
__device__ __forceinline__ void place(const Fp8GemmArgs &a, const Fp8Tile &t, int n_tiles, int weight_rows, int &mt, int &nt) {
  const int local = t.lin - t.first * n_tiles;
  if (t.end - t.begin <= weight_rows) {  // the weights are larger: their tile outermost
    nt = local / t.count;
    mt = local - nt * t.count;
  } else {  // bands of four row tiles, weight tile outer within a band
    constexpr int BAND = 4;
    const int band = local / (BAND * n_tiles), r = local - band * BAND * n_tiles;
    const int bm = min(BAND, t.count - band * BAND);
    nt = r / bm;
    mt = band * BAND + (r - nt * bm);
  }
  mt = __builtin_amdgcn_readfirstlane(mt);
  nt = __builtin_amdgcn_readfirstlane(nt);
}

// A part's words of scales (four blocks of K each): first and past the last.
__device__ __forceinline__ void part_of_k(const Fp8GemmArgs &a, const Fp8Tile &t, int &q0, int &q1) {
  const int words = fp8_scale_bytes(a.K) / 4;
  q0 = words * t.part / t.parts;
  q1 = words * (t.part + 1) / t.parts;
}

// Some rows, up to 128 at a time: a workgroup has 128 columns of H or 256 of y, each of its eight waves two
// blocks of 16 weight rows (gate and up, or neighbours).  The rows are read by all eight waves from LDS, where
// loads without registers put them as codes, a step of 128 of K a stage, in the operand layout (2 KB for 16 rows:
// sixteen lanes read 256 consecutive bytes); four stages, three steps ahead, one barrier a step.  The 8-bit matrix
// instruction: converted to bf16 by each wave, 128 rows took 1.7 us a step of the 1.2 that its weights take.
// Bound by the weights' bytes: 32 x 80 rows, 7168 x 2048, gate_up 160 us (5.9 TB/s), down 104 (4.5, of 224 CUs; with
// rows read again for each column tile 5.9 beyond L2); 32 x 4 rows both in 234 (6.0).
constexpr int MD_R = 4, MD_D = 3, MD_ROWS = 128;

// One block of n <= 16 MS rows from m0 on, column tiles nb0 .. nb1 - 1 one after the other without a pause of the loads: in a
// tile's last four steps those of the next one's first are loaded.  MS is exact, so that no branch is in the loop.
template <bool SWIGLU, int MS>
__device__ __forceinline__ void medium_rows(const Fp8GemmArgs &a, const Fp8Tile &tile, int n_tiles, int m0, int n,
                                            uint8_t *s0, uint8_t *s1, uint8_t *s2, uint8_t *s3, uint8_t *row_scales,
                                            float (*tops)[MD_ROWS]) {
  constexpr int R = MD_R, D = MD_D;
  static_assert(R == 4 && D == 3, "a word of scales and the stages");
  auto stage = [&](int b) -> uint8_t * { return b == 0 ? s0 : b == 1 ? s1 : b == 2 ? s2 : s3; };
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lr = lane & 15,
            lg = lane >> 4;
  const int kt = fp8_blocks(a.K), kp = fp8_row_bytes(a.K), ks = fp8_scale_bytes(a.K);
  const int units = (a.n_out + 15) / 16 * (SWIGLU ? 2 : 1);  // blocks of 16 weight rows
  int tb, te;  // this part's steps
  part_of_k(a, tile, tb, te);
  tb *= 4;
  te = min(kt, te * 4);
  const int g = tile.g;
  const int64_t wbytes = fp8_group_bytes(a.n_out, a.K, SWIGLU);
  const rsrc_t wres = make_rsrc(a.w8 + g * wbytes, (uint32_t)wbytes);
  const int sblocks = fp8_blocks(a.n_out);
  // the column tile that is loaded
  uint32_t half, wbase;
  int end0, end1;  // its steps, of this wave's two blocks
  const uint8_t *wscale;
  auto columns = [&](int nb) {
    const int unit = nb * 16 + wave * 2;
    wbase = fp8_block_offset(unit, units, kt, half) + (uint32_t)lane * 16u;
    end0 = nb < tile.col1 && unit < units ? te : 0;
    end1 = nb < tile.col1 && unit + 1 < units ? te : 0;
    wscale = a.w_scale + ((int64_t)g * sblocks + min(SWIGLU ? nb : nb * 2 + wave / 4, sblocks - 1)) * (SWIGLU ? 2 : 1) * ks;
  };
  i32x8 w[R][2];
  auto load_w = [&](int j, int t) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const bool in = t < (b ? end1 : end0);
      const uint32_t o = wbase + (uint32_t)(2 * t) * half + (uint32_t)b * 1024u;
      w[j][b] = fp8_operand(buf_ld16_nt(wres, in ? o : kOob), buf_ld16_nt(wres, in ? o + half : kOob));
    }
  };
  const Fp8Rows rows(a, m0, n);
  // this wave's pieces of a stage, one for each half of K's 128: subtile `wave`, row lr, codes 64 p + 16 lg ..
  const uint32_t src = rows.row(a, m0, wave * 16 + lr, n);
  const uint32_t xoff = src != kOob ? src * (uint32_t)kp + (uint32_t)lg * 16u : kOob;
  auto load_x = [&](int t, int end, int b) {
    const uint32_t o = t < end && xoff != kOob ? xoff + (uint32_t)t * 128u : kOob;
    buf_ld16_lds(rows.xres, o, stage(b) + wave * 2048);
    buf_ld16_lds(rows.xres, o == kOob ? kOob : o + 64u, stage(b) + wave * 2048 + 1024);
  };
  // The rows' scales of four steps go through LDS too, each wave's 16 rows by one load: read by every wave from memory they
  // are MS loads of 16 lines each, behind which the waits below found too few weights still in flight.
  const uint32_t soff = src != kOob && lg == 0 ? src * (uint32_t)ks : kOob;
  uint32_t sx[MS], sw[2], nw[2];
  // of four steps; past K those of the last four again (their codes are zeros)
  auto load_row_scales = [&](int t) {
    buf_ld4_lds(rows.sres, soff == kOob ? kOob : soff + (uint32_t)min(t, ks - 4), row_scales + wave * 256);
  };
  auto load_scales = [&](int t) {
#pragma unroll
    for (int b = 0; b < 2; ++b) nw[b] = scalar_load(wscale + (SWIGLU ? b * ks : 0) + min(t, ks - 4));
  };
  f32x4 acc[MS][2];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < MS; ++i)
#pragma unroll
      for (int b = 0; b < 2; ++b) acc[i][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  clear();
  auto bar = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  auto lds_bar = [&]() {  // and LDS written before it can be read after it; loads stay in flight
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    bar();
    asm volatile("" ::: "memory");
  };
  auto finish = [&](int nb) {
    int first = m0, some = n;
    asm volatile("" : "+s"(first), "+s"(some));  // no rows' addresses, nor which there are, kept in registers over the loop
    if (tile.parts > 1) {
#pragma unroll
      for (int i = 0; i < MS; ++i) {
        const int64_t row = (int64_t)first + i * 16 + lr;
        if (i * 16 + lr < some)
#pragma unroll
          for (int b = 0; b < 2; ++b)
            *reinterpret_cast<f32x4 *>(a.parts + (tile.part * (int64_t)a.rows_max + row) * n_tiles * 256 + nb * 256 +
                                       (SWIGLU ? b * 128 + wave * 16 : wave * 32 + b * 16) + lg * 4) = acc[i][b];
      }
    } else if constexpr (SWIGLU) {
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
      lds_bar();
#pragma unroll
      for (int i = 0; i < MS; ++i) {
        float top = 0.0f;
#pragma unroll
        for (int v = 0; v < 8; ++v) top = fmaxf(top, tops[v][i * 16 + lr]);
        const int64_t row = (int64_t)first + i * 16 + lr;
        const float h[4] = {acc[i][0][0], acc[i][0][1], acc[i][0][2], acc[i][0][3]};
        if (i * 16 + lr < some) store_h(a, h, top, row, nb, col, wave == 0 && lg == 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < MS; ++i) {
        const int64_t row = (int64_t)first + i * 16 + lr;
        if (i * 16 + lr < some)
#pragma unroll
          for (int b = 0; b < 2; ++b) store_y(a, acc[i][b], row, (nb * 16 + wave * 2 + b) * 16 + lg * 4);
      }
    }
  };
  int nb = tile.col0, t0 = tb;
  columns(nb);
  load_scales(tb);
  load_row_scales(tb);
#pragma unroll
  for (int b = 0; b < D; ++b) load_x(tb + b, te, b);
  __builtin_amdgcn_sched_barrier(0);  // the waits count on rows before weights
#pragma unroll
  for (int j = 0; j < R; ++j) load_w(j, tb + j);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(4 * R) : "memory");  // the first stages are there
  bar();
  for (;;) {
    const uint32_t keep = kt - t0 >= 4 ? ~0u : (1u << (8 * (kt - t0))) - 1u;  // the padding's scales are not looked at
#pragma unroll
    for (int i = 0; i < MS; ++i) sx[i] = *reinterpret_cast<const uint32_t *>(row_scales + i * 256 + lr * 4) & keep;
#pragma unroll
    for (int b = 0; b < 2; ++b) sw[b] = nw[b] & keep;
    // the four steps that are loaded meanwhile
    const bool last = t0 + R >= te;
    const int next = nb + (last ? 1 : 0), n0 = last ? tb : t0 + R, nend = next < tile.col1 ? te : 0;
    if (last) columns(next);
    load_scales(n0);
    auto step = [&](auto jc) {
      constexpr int J = decltype(jc)::value;
      if constexpr (J == 1) {  // every wave has read the former ones
        load_row_scales(n0);
        __builtin_amdgcn_sched_barrier(0);
      }
      // the stage read in the step before, which every wave has left
      if constexpr (J == 0)
        load_x(t0 + D, te, D);
      else
        load_x(n0 + J - 1, nend, J - 1);
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
      load_w(J, n0 + J);
      // step t + 1's rows, loaded in step t + 1 - D, are there when at most the loads behind them are in flight
      // (weights of that step, rows and weights of the steps since, and the scales where those lie behind; stores of a tile
      // that ended among them only make it wait for more)
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(4 + 6 * (D - 1) + (J == 1 || J == 2)) : "memory");
      bar();
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
    t0 = n0;
    if (last) {
      finish(nb);
      if (next == tile.col1) break;
      nb = next;
      clear();
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no write to LDS may outlive its rows
  __syncthreads();
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
__global__ __launch_bounds__(512, 1) void fp8_rows_kernel(const Fp8GemmArgs a, int n_tiles, int tiles_max) {
  constexpr int NBUF = 4;
  __shared__ __attribute__((aligned(1024))) uint8_t sA0[LG_TILE], sA1[LG_TILE], sA2[LG_TILE], sA3[LG_TILE];
  __shared__ __attribute__((aligned(1024))) uint8_t sB0[LG_TILE], sB1[LG_TILE], sB2[LG_TILE], sB3[LG_TILE];
  __shared__ uint8_t row_scales[8 * 256];
  auto bufA = [&](int b) -> uint8_t * { return b == 0 ? sA0 : b == 1 ? sA1 : b == 2 ? sA2 : sA3; };
  auto bufB = [&](int b) -> uint8_t * { return b == 0 ? sB0 : b == 1 ? sB1 : b == 2 ? sB2 : sB3; };
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / 4, wn = wave % 4, lr = lane & 31, lh = lane >> 5;
  const Fp8Tile tile = find_tile(a, tiles_max, a.first_block + (int)blockIdx.x, n_tiles, kProduct);
  if (tile.g < 0) return;
  const int g = tile.g, begin = tile.begin, end = tile.end, mt_first = tile.first, mt_count = tile.count;
  if (mt_count == 0) {
    for (int left = end - begin; left > 0; left -= MD_ROWS) {  // (m0 + MD_ROWS may pass 2^31)
      const int m0 = end - left, n = min(MD_ROWS, left);
      switch ((n + 15) / 16) {
#define MOE_ROWS(MS)                                                                       \
  case MS:                                                                                 \
    medium_rows<SWIGLU, MS>(a, tile, n_tiles, m0, n, sA0, sA1, sA2, sA3, row_scales,       \
                            reinterpret_cast<float(*)[MD_ROWS]>(sB0));                     \
    break
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
    return;
  }
  int mt, nt;
  place(a, tile, n_tiles, (SWIGLU ? 2 : 1) * a.n_out, mt, nt);
  const int per = fp8_tile_rows(end - begin, mt_count);
  const int m0 = begin + mt * per, rows = min(per, end - m0), m_tile = mt_first + mt;
  if (m_tile >= tiles_max) return;
  const int row_blocks = (rows + 31) / 32, mine = max(0, min(4, row_blocks - wm * 4));  // of 32 rows: the tile's, this wave's
  const int kt = fp8_blocks(a.K), ks = fp8_scale_bytes(a.K);
  int q0, q1;  // this part's words of scales, and its steps of 64
  part_of_k(a, tile, q0, q1);
  const int kfirst = 8 * q0, nk = min(2 * kt, 8 * q1) - kfirst;
  const int64_t abytes = (int64_t)kFp8LargeRows * kt * kFp8Block;
  const int64_t wbytes = fp8_group_bytes(a.n_out, a.K, SWIGLU);
  // the rows as they are, or packed
  const Fp8Rows from(a, m0, rows);
  const bool packed = a.xp != nullptr;
  const rsrc_t ares = packed ? make_rsrc(a.xp + m_tile * abytes, (uint32_t)abytes) : from.xres;
  const rsrc_t sres = packed ? make_rsrc(a.xp_scale + (int64_t)m_tile * kFp8LargeRows * ks, (uint32_t)(kFp8LargeRows * ks))
                             : from.sres;
  const uint32_t astep = packed ? (uint32_t)LG_TILE : 64u, sstep = packed ? kFp8LargeRows * 4u : 4u;
  const rsrc_t wres = make_rsrc(a.w8 + g * wbytes, (uint32_t)wbytes);
  // this wave's pieces of a stage: 16-row blocks 2 wave and 2 wave + 1 of both operands
  uint32_t aoff[2], boff[2], wstep;
  const int wblocks = (a.n_out + 15) / 16 * (SWIGLU ? 2 : 1);
  const uint32_t wtile = fp8_block_offset(nt * 16, wblocks, kt, wstep);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t at = (uint32_t)(2 * wave + i) * 1024u + (uint32_t)lane * 16u;
    if (packed) {
      aoff[i] = wave < row_blocks ? at : kOob;
    } else {
      const uint32_t src = from.row(a, m0, (2 * wave + i) * 16 + (lane & 15), rows);
      aoff[i] = src != kOob ? src * (uint32_t)fp8_row_bytes(a.K) + (uint32_t)(lane >> 4) * 16u : kOob;
    }
    boff[i] = nt * 16 + 2 * wave + i < wblocks ? wtile + at : kOob;
  }
  auto issue = [&](int s, int b) {
    const uint32_t ka = (uint32_t)(kfirst + s) * astep, kb = (uint32_t)(kfirst + s) * wstep;
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
  // four blocks of K, eight steps; past K zeros, or the last ones again.  The rows' go through LDS, one load a wave for 64
  // rows (two waves write the same): each wave's own 128 were four loads, behind which the waits counted too few others.
  uint32_t sw[2];
  const int srow = (wave & 3) * 64 + lane;
  uint32_t soff = (uint32_t)srow * 4u;
  if (!packed) {
    const uint32_t src = from.row(a, m0, srow, rows);
    soff = src != kOob ? src * (uint32_t)ks : kOob;
  }
  auto load_row_scales = [&](int q) {
    buf_ld4_lds(sres, soff != kOob ? soff + (uint32_t)q * sstep : kOob, row_scales + (wave & 3) * 256);
  };
  auto load_scales = [&](int q) {
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
    auto mem = [&](int q, int s, auto bc) {
      constexpr int b = decltype(bc)::value;
      if constexpr (b == 2) {  // both groups have read the former ones
        load_row_scales(q + 1);
        __builtin_amdgcn_sched_barrier(0);
      }
      issue(s + 3, (b + 3) % NBUF);
      // the two younger steps' may stay in flight, and the scales where they lie between
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(8 + (b == 2 || b == 3)) : "memory");
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
      for (int i = 0; i < 4; ++i) cx[i] = *reinterpret_cast<const uint32_t *>(row_scales + (wm * 128 + i * 32 + lr) * 4);
#pragma unroll
      for (int j = 0; j < 2; ++j) cw[j] = sw[j];
      load_scales(q + 1);
    };
    load_scales(q0);
    load_row_scales(q0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int b = 0; b < 3; ++b) issue(b, b);
    asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
    bar();
    if (second) bar();
    int s0 = 0, q = q0;
    auto step = [&](auto bc) {
      mem(q, s0 + decltype(bc)::value, bc);
      bar();
      comp(decltype(bc)::value);
      bar();
    };
#define MOE_STEP(B) step(std::integral_constant<int, B>{})
    for (; s0 + 8 <= nk; s0 += 8, ++q) {
      next_scales(q);
      MOE_STEP(0);
      MOE_STEP(1);
      MOE_STEP(2);
      MOE_STEP(3);
      MOE_STEP(4);
      MOE_STEP(5);
      MOE_STEP(6);
      MOE_STEP(7);
    }
    if (s0 < nk) {  // two, four or six: K is whole blocks of 128
      next_scales(q);
      MOE_STEP(0);
      MOE_STEP(1);
      if (s0 + 2 < nk) {
        MOE_STEP(2);
        MOE_STEP(3);
        if (s0 + 4 < nk) {
          MOE_STEP(4);
          MOE_STEP(5);
        }
      }
    }
#undef MOE_STEP
    if (!second) bar();
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no LDS write may outlive the block
  __syncthreads();

  // Block (i, j): lane l holds row wm * 128 + i * 32 + l % 32 and, per q = 0..3, columns 8 q + 4 (l / 32) .. + 3 of its 32.
  if (tile.parts > 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = wm * 128 + i * 32 + lr;
      if (row >= rows) continue;
      float *o = (tile.slot < 0 ? a.parts + (tile.part * (int64_t)a.rows_max + m0 + row) * n_tiles * 256 + nt * 256
                                : a.parts + ((int64_t)(tile.part * tile.cut + tile.slot) * kFp8LargeRows + row) * 256) +
                 lh * 4 + (SWIGLU ? wn * 32 : wn * 64);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<f32x4 *>(o + j * (SWIGLU ? 128 : 32) + q * 8) =
              f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    }
    return;
  }
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

// The parts' sums in order, and what the product's own epilogue does with them: sixteen workgroups a tile of
// fp8_rows_kernel.
template <bool SWIGLU>
__global__ __launch_bounds__(256) void fp8_add_parts_kernel(const Fp8GemmArgs a, int n_tiles, int tiles_max) {
  const Fp8Tile tile = find_tile(a, tiles_max, blockIdx.x, n_tiles, kAdd);
  if (tile.g < 0 || tile.parts == 1 || tile.part > 0) return;
  int nt, mt = 0, m0 = tile.begin, n = tile.end - tile.begin, last = n;
  if (tile.count) {
    place(a, tile, n_tiles, (SWIGLU ? 2 : 1) * a.n_out, mt, nt);
    const int per = fp8_tile_rows(n, tile.count);
    m0 += mt * per;
    n = min(per, tile.end - m0);
    last = (n + 31) / 32 * 32;  // packed tiles are read by whole 32s
  } else {
    nt = tile.col0;
  }
  const int m_tile = tile.first + mt;
  if (tile.count && m_tile >= tiles_max) return;
  constexpr int LANES = SWIGLU ? 16 : 32;  // of eight columns each, a row
  const int l = threadIdx.x % LANES;
  for (int r = blockIdx.y * (256 / LANES) + threadIdx.x / LANES; r < (SWIGLU ? last : n); r += gridDim.y * (256 / LANES)) {
    float v[SWIGLU ? 2 : 1][8] = {};
    if (r < n)
#pragma unroll 2
      for (int s = 0; s < tile.parts; ++s) {
        const float *p = (tile.slot < 0 ? a.parts + (s * (int64_t)a.rows_max + m0 + r) * n_tiles * 256 + nt * 256
                                        : a.parts + ((int64_t)(s * tile.cut + tile.slot) * kFp8LargeRows + r) * 256) + l * 8;
#pragma unroll
        for (int h = 0; h < (SWIGLU ? 2 : 1); ++h) {
          const f32x4 x = *reinterpret_cast<const f32x4 *>(p + h * 128), y = *reinterpret_cast<const f32x4 *>(p + h * 128 + 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[h][e] += x[e];
            v[h][4 + e] += y[e];
          }
        }
      }
    if constexpr (SWIGLU) {
      float top = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[0][e] = silu_f32(v[0][e]) * v[1][e];
        top = fmaxf(top, fp8_magnitude(v[0][e]));
      }
      top = group_reduce<16>(top, [](float x, float y) { return fmaxf(x, y); });
      const uint32_t byte = fp8_scale_byte(top);
      const float inv = fp8_inverse(byte);
      const uint2 codes{fp8_codes(v[0][0] * inv, v[0][1] * inv, v[0][2] * inv, v[0][3] * inv),
                        fp8_codes(v[0][4] * inv, v[0][5] * inv, v[0][6] * inv, v[0][7] * inv)};
      const int ht = fp8_blocks(a.n_out), hs = fp8_scale_bytes(a.n_out);
      if (tile.count) {
        uint8_t *o = a.hp + (((int64_t)m_tile * ht + nt) * 2 + l / 8) * LG_TILE;
        *reinterpret_cast<uint2 *>(o + (r >> 4) * 1024 + (l / 2 % 4) * 256 + (r & 15) * 16 + l % 2 * 8) = codes;
        if (l == 0) a.hp_scale[(int64_t)m_tile * kFp8LargeRows * hs + ((nt / 4) * kFp8LargeRows + r) * 4 + nt % 4] = (uint8_t)byte;
      } else {
        *reinterpret_cast<uint2 *>(a.h8 + (int64_t)(m0 + r) * fp8_row_bytes(a.n_out) + nt * 128 + l * 8) = codes;
        if (l == 0) a.h_scale[(int64_t)(m0 + r) * hs + nt] = (uint8_t)byte;
      }
    } else {
      const int col = nt * 256 + l * 8;
      store8<bf16_t, false>(a.y + (int64_t)(m0 + r) * a.n_out + col, a.n_out - col, v[0]);
    }
  }
}

// The rows of the tiles, and their scales as [4 blocks of K][256 rows] words, for fp8_rows_kernel: one
// workgroup 64 rows of a tile and four blocks of K; a wave reads 64 bytes of its 16 rows at a time, the other half of
// each line next, and writes them as one piece of 1 KB (whole rows a wave, 16 bytes of each written apart: 36 us for
// 27 at 4096 x 14336).
__global__ __launch_bounds__(256) void fp8_pack_rows_kernel(const Fp8GemmArgs a, uint8_t *__restrict__ xp,
                                                            uint8_t *__restrict__ xp_scale, int tiles_max) {
  const int kt = fp8_blocks(a.K), kp = fp8_row_bytes(a.K), ks = fp8_scale_bytes(a.K), quads = ks / 4;
  const int b0 = blockIdx.y * 4, m_tile = blockIdx.x / 4;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int block = (blockIdx.x % 4) * 4 + wave, r = block * 16 + (lane & 15), c = lane >> 4;  // of 16 rows; row, chunk
  const Fp8Tile t = find_tile(a, tiles_max, m_tile, 1, kPack);
  if (t.count == 0) return;
  const int per = fp8_tile_rows(t.end - t.begin, t.count), m0 = t.begin + (m_tile - t.first) * per;
  const int rows = min(per, t.end - m0);
  if (block * 16 >= (rows + 31) / 32 * 32) return;  // the kernel reads whole 32s
  const Fp8Rows from(a, m0, rows);
  const uint32_t src = from.row(a, m0, r, rows);
  u32x4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = buf_ld16(from.xres, src != kOob && b0 + i / 2 < kt ? src * (uint32_t)kp + (uint32_t)(b0 * 128 + i * 64 + c * 16) : kOob);
  const uint32_t scales = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(
      from.sres, src != kOob ? src * (uint32_t)ks + (uint32_t)b0 : kOob, 0, 0);
  uint8_t *o = xp + ((int64_t)m_tile * kt + b0) * 2 * LG_TILE + block * 1024 + lane * 16;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (b0 + i / 2 < kt) stg16(o + i * LG_TILE, v[i]);
  if (lane < 16)
    reinterpret_cast<uint32_t *>(xp_scale)[((int64_t)m_tile * quads + blockIdx.y) * kFp8LargeRows + r] = scales;
}

}  // namespace

hipError_t launch_fp8_pack_rows(const Fp8GemmArgs &a, uint8_t *xp, uint8_t *xp_scale, hipStream_t s) {
  const int64_t tiles = fp8_large_tiles_max(a.rows_max, a.num_groups);
  const int quads = fp8_scale_bytes(a.K) / 4;
  if (tiles >= (1 << 22) || quads > 65535) return hipErrorInvalidValue;  // 2^32 threads
  if (tiles > 0)
    hipLaunchKernelGGL(fp8_pack_rows_kernel, dim3((unsigned)tiles * (kFp8LargeRows / 64), (unsigned)quads), dim3(256), 0, s, a,
                       xp, xp_scale, (int)tiles);
  return hipGetLastError();
}

// Ranges of column tiles, a block each, for the groups of few rows: of as many tiles, up to 64 steps of 128 of K, as cost least
// in rounds of 256 blocks for as many groups as there can be, counted in steps, of which a block's begin and end take
// eight (10 us); a tenth has to be won.  Longer ones end unevenly.  us with 1, 2, 4, 7 and all tiles a block: 212 of 256
// groups of up to 80 rows, 7168 x 2048, 28 tiles of 16 steps, 580, -, 552, 593, 692; 2048 gate_up, 16 of 56 steps, 927, 972,
// 1017, -, 1069; 32 x 80 rows, 28 of 16 steps, 115 and, with four, 104.  0: a block for each tile.
static int few_chunks(int groups, int n_tiles, int k) {
  const int64_t steps = fp8_scale_bytes(k);
  int64_t least = ((int64_t)groups * n_tiles + 255) / 256 * (steps + 8) * 9 / 10;
  int best = 0;
  for (int columns = 2; columns <= n_tiles && columns * steps <= 64; ++columns) {
    const int64_t chunks = (n_tiles + columns - 1) / columns, cost = (groups * chunks + 255) / 256 * (columns * steps + 8);
    if (cost < least) {
      best = (int)chunks;
      least = cost;
    }
  }
  return best;
}

hipError_t launch_fp8_gemm_rows(const Fp8GemmArgs &call, hipStream_t s) {
  Fp8GemmArgs a = call;
  const bool swiglu = a.h8 != nullptr;
  const int n_tiles = (a.n_out + (swiglu ? 127 : 255)) / (swiglu ? 128 : 256);
  const int64_t tiles = a.large ? fp8_large_tiles_max(a.rows_max, a.num_groups) : 0;
  const int groups = std::min(a.num_groups, a.rows_max);
  a.few_chunks = a.parts_cap > 1 ? 0 : few_chunks(groups, n_tiles, a.K);
  // A group has one tile, few rows or many, and one more for each further 256 rows; in ranges, as many as there can be of each.
  const int64_t blocks = a.few_chunks ? tiles * n_tiles + std::max<int64_t>((int64_t)groups * a.few_chunks, 256)
                                      : (groups + (a.large ? a.rows_max / kFp8LargeRows : 0)) * (int64_t)n_tiles;
  // parts are one round at most
  const int64_t grid = a.rounds ? blocks + 256 : a.parts_cap > 1 ? std::max<int64_t>(blocks, 256) : blocks;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  constexpr int64_t kBlocks = 1 << 22;  // a launch: its threads are counted in 32 bits
  for (int64_t first = 0; first < grid; first += kBlocks) {
    a.first_block = (int)first;
    const dim3 some((unsigned)std::min(kBlocks, grid - first));
    if (swiglu)
      hipLaunchKernelGGL((fp8_rows_kernel<true>), some, dim3(512), 0, s, a, n_tiles, (int)tiles);
    else
      hipLaunchKernelGGL((fp8_rows_kernel<false>), some, dim3(512), 0, s, a, n_tiles, (int)tiles);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (a.parts_cap == 1 && !a.rounds)) return e;
  const dim3 adding((unsigned)std::min<int64_t>(blocks, 128), 16);  // tiles that are cut: half a round at most
  if (swiglu)
    hipLaunchKernelGGL((fp8_add_parts_kernel<true>), adding, dim3(256), 0, s, a, n_tiles, (int)tiles);
  else
    hipLaunchKernelGGL((fp8_add_parts_kernel<false>), adding, dim3(256), 0, s, a, n_tiles, (int)tiles);
  return hipGetLastError();
}

}  // namespace moe
