// pad16.hpp -- copies of a product's operands with aligned rows.
#pragma once
#include "gated_core.hpp"

namespace fp8dp {

// Copies with aligned rows of up to three matrices of `cols` columns, zeros behind them, in one launch: rows of a K that
// is no multiple of 8 start anywhere, and the tiles that are filled by copies are then worth more than the copies cost.
struct PadArgs {
  const uint16_t* from[3];
  uint16_t* to[3];
  int64_t rows[3];   // ends of the three, in rows of all
  int cols, ld;
};
static __global__ __launch_bounds__(256) void k_pad16(PadArgs a) {
  const uint32_t nvec = (uint32_t)a.ld / 8;
  const uint64_t total = (uint64_t)a.rows[2] * nvec, step = (uint64_t)gridDim.x * 256;
  for (uint64_t at = (uint64_t)blockIdx.x * 256 + threadIdx.x; at < total; at += step) {
    const int64_t row = total >> 32 ? at / nvec : (uint32_t)at / nvec;
    const int c = (int)(at - (uint64_t)row * nvec) * 8, which = (row >= a.rows[0]) + (row >= a.rows[1]);
    const int64_t r = row - (which == 0 ? 0 : which == 1 ? a.rows[0] : a.rows[1]);
    const uint16_t* const from = which == 0 ? a.from[0] : which == 1 ? a.from[1] : a.from[2];
    uint16_t* const to = which == 0 ? a.to[0] : which == 1 ? a.to[1] : a.to[2];
    const Raw8<bf16_t> v = load_raw(reinterpret_cast<const bf16_t*>(from) + r * a.cols + c, a.cols - c);
    *reinterpret_cast<u32x4_t*>(to + r * a.ld + c) = u32x4_t{v.w[0], v.w[1], v.w[2], v.w[3]};
  }
}
// x [M x cols], w0 and w1 [N x cols] to `to`, one behind the other; pad_bytes() of them.
inline int64_t pad_ld(int64_t cols) { return round_up(cols, 8); }
inline int64_t pad_bytes(int64_t M, int64_t N, int64_t cols) {
  return round_up((M + 2 * N) * pad_ld(cols) * 2, 256);
}
inline int pad_operands(const char* what, const uint16_t* x, const uint16_t* w0, const uint16_t* w1, int64_t M,
                        int64_t N, int64_t cols, uint16_t* to, hipStream_t stream) {
  const int64_t ld = pad_ld(cols);
  const PadArgs a = {{x, w0, w1}, {to, to + M * ld, to + (M + N) * ld}, {M, M + N, M + 2 * N}, (int)cols, (int)ld};
  hipLaunchKernelGGL(k_pad16, dim3(grid_for((M + 2 * N) * (ld / 8), 256, 32)), dim3(256), 0, stream, a);
  return check_launch(what);
}
// Whether the copies pay for themselves, by M N K (measured, copied / as they are, us): forward 777 x 1023 x 1001 21.2 /
// 25.8, 777 x 1023 x 101 10.9 / 9.5, 300 x 600 x 301 12.5 / 11.7; backward, where two products share
// them, 777 x 1023 x 1001 46.8 / 58.1, 777 x 1023 x 101 39.8 / 44.5, 100 x 300 x 1001 25.7 / 30.9, 300 x 300 x 301 28.9 / 35.2.
inline bool pad_pays(int64_t M, int64_t N, int64_t K, bool backward) {
  return K % 8 != 0 && (double)M * (double)N * (double)K >= (backward ? 8e6 : 256e6);
}

}  // namespace fp8dp
