// What the products in 8 bits share: where a group's rows stand, and how results leave.
#pragma once

#include "fp8.hpp"

namespace moe {

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

}  // namespace moe
