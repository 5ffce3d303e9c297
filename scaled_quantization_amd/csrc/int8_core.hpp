// int8_core.hpp -- pieces shared by the INT8 matrix kernels: argument block,
// MFMA types and the epilogue that applies the scales of token and channel.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_core.hpp"
#include "row_core.hpp"

namespace fp8dp {

typedef int v4i_t __attribute__((ext_vector_type(4)));
typedef int v16i_t __attribute__((ext_vector_type(16)));
typedef unsigned int u32x4_b_t __attribute__((ext_vector_type(4), aligned(1)));

struct I8Args {
  const int8_t *a, *b;          // rows of lda / ldb bytes
  int M, N, K;
  int64_t lda, ldb;
  const float *sa, *sb;
  const void* bias;
  bool bias_f32;
  void* y;
  int first = 0;                // tile (or group of channels) of workgroup 0: for_blocks()
};

// Whether the rows of both operands start at multiples of 16 bytes and K is one too.
inline bool rows16(const I8Args& g) {
  return g.K % 16 == 0 && g.lda % 16 == 0 && g.ldb % 16 == 0 && aligned16(g.a) && aligned16(g.b);
}

// A launch has at most 2^32 - 1 threads, which workgroups of 512 reach at 2^23: more of them
// go in several launches, each with the index of its first one.  launch(first, count).
template <typename F>
inline int for_blocks(int64_t blocks, F&& launch) {
  constexpr int64_t kMost = (int64_t)1 << 22;   // (a multiple of 8: the XCDs' turns go on)
  for (int64_t first = 0; first < blocks; first += kMost) {
    const int rc = launch((int)first, (unsigned)std::min(blocks - first, kMost));
    if (rc) return rc;
  }
  return FP8DP_OK;
}

// What chunks past K are copied from.
__device__ const u32x4_t kZeroChunk = {0, 0, 0, 0};

// 16 bytes at any byte address.
__device__ __forceinline__ v4i_t load16(const int8_t* p) {
  const u32x4_b_t v = *reinterpret_cast<const u32x4_b_t*>(p);
  return v4i_t{(int)v.x, (int)v.y, (int)v.z, (int)v.w};
}

// v with its first d bytes zero (d >= 16: all).
__device__ __forceinline__ v4i_t zero_first(v4i_t v, int d) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int s = 8 * d - 32 * w;
    v[w] &= s >= 32 ? 0 : s <= 0 ? -1 : (int)(0xFFFFFFFFu << s);
  }
  return v;
}

// A chunk of 16 bytes that K may cut.  The sum takes K in any order as long as
// both operands agree, so a cut chunk is read as the row's last 16 bytes,
// without reading past the row, and the bytes that earlier chunks hold already
// are cleared in one operand (ONCE).  Rows below 16 bytes are read byte by byte.
template <bool ONCE>
__device__ __forceinline__ v4i_t load_chunk(const int8_t* row, int k, int K) {
  if (K >= 16) {
    const int at = k < K - 16 ? k : K - 16;
    const v4i_t v = load16(row + at);
    return ONCE ? zero_first(v, k - at) : v;
  }
  uint64_t lo = 0, hi = 0;
#pragma unroll 1
  for (int j = 15; j >= 0; --j) {
    hi = hi << 8 | lo >> 56;
    lo = lo << 8 | (k + j < K ? (uint8_t)row[k + j] : 0);
  }
  return v4i_t{(int)lo, (int)(lo >> 32), (int)hi, (int)(hi >> 32)};
}

// Four outputs of row m, columns n .. n + 3, from their integer sums:
// (sum sa) sb + bias in binary32, one rounding to T.  Columns at or past N are
// not stored.
template <typename T>
__device__ __forceinline__ void store_out4(const I8Args& g, int64_t m, int n, float sa,
                                           const float sb[4], const float bias[4], const v4i_t& c) {
  float v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = __builtin_fmaf((float)c[j] * sa, sb[j], bias[j]);
  T* const p = static_cast<T*>(g.y) + m * g.N + n;
  if (n + 4 <= g.N) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<f32x4_e_t*>(p) = f32x4_e_t{v[0], v[1], v[2], v[3]};
    } else {
      const float w[8] = {v[0], v[1], v[2], v[3], 0.0f, 0.0f, 0.0f, 0.0f};
      const Raw8<T> r = round8(w, T{});
      typedef unsigned int pair_t __attribute__((ext_vector_type(2), aligned(2)));
      *reinterpret_cast<pair_t*>(p) = pair_t{r.w[0], r.w[1]};
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < g.N) p[j] = from_f32<T>(v[j]);
  }
}
// Weight scales and bias of columns n .. n + 3, as loaded (clamped to the last
// column) and widened, so that the loads can be issued long before their use.
struct RawCols4 {
  float sb[4];
  uint32_t bias[4];
};
template <typename T>
__device__ __forceinline__ RawCols4 load_cols4(const I8Args& g, int n) {
  RawCols4 r = {};
  int c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    c[j] = n + j < g.N ? n + j : g.N - 1;
    r.sb[j] = g.sb[c[j]];
  }
  if (g.bias != nullptr) {
    if (sizeof(T) == 4 || g.bias_f32) {
#pragma unroll
      for (int j = 0; j < 4; ++j) r.bias[j] = static_cast<const uint32_t*>(g.bias)[c[j]];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) r.bias[j] = static_cast<const uint16_t*>(g.bias)[c[j]];
    }
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void widen_bias4(const I8Args& g, const RawCols4& r, float bias[4]) {
  if (sizeof(T) == 4 || g.bias_f32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) bias[j] = __uint_as_float(r.bias[j]);
  } else if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) bias[j] = to_f32(T{(uint16_t)r.bias[j]});
  }
}

// What the outputs of a tile of BM tokens x BN channels need beside its sums, in LDS: loaded
// while the first stages travel, so that the epilogue waits for nothing from memory.
template <int BM, int BN>
struct TileScales {
  float sa[BM], sb[BN], bias[BN];
};
template <typename T, int BM, int BN>
__device__ __forceinline__ void load_scales(const I8Args& g, TileScales<BM, BN>& s, int m0, int n0,
                                            int tid, int threads) {
  for (int i = tid; i < BM; i += threads) s.sa[i] = g.sa[m0 + i < g.M ? m0 + i : g.M - 1];
  for (int i = tid; i < BN; i += threads) {
    const int n = n0 + i < g.N ? n0 + i : g.N - 1;
    s.sb[i] = g.sb[n];
    s.bias[i] = g.bias == nullptr ? 0.0f
                : sizeof(T) == 4 || g.bias_f32 ? static_cast<const float*>(g.bias)[n]
                                               : to_f32(static_cast<const T*>(g.bias)[n]);
  }
}

// Epilogue of a wave's TM x TN tiles of 32 x 32 at row wr, column wc of a tile at m0, n0.  In such a
// tile the lane holds token lane % 32 and register r channel 8 (r / 4) + 4 (lane / 32) + r % 4:
// stored from there, a row gets 8 bytes at a time.  The wave turns its tiles in its own
// 32 x 32 TN words of LDS, 32 tokens at a time as binary32 (sum times token scale), and reads them
// back with 8 consecutive channels per lane, whose scales and bias it then holds for
// all rows, and whole cache lines per row to store.  16-byte chunks are swizzled by row
// against bank conflicts.
typedef float f32x4_t __attribute__((ext_vector_type(4)));
template <typename T, int TM, int TN, int BM, int BN>
__device__ __forceinline__ void turn_out(const I8Args& g, const v16i_t (&acc)[TM][TN],
                                         uint8_t* part, const TileScales<BM, BN>& scales, int m0,
                                         int n0, int wr, int wc, int lane) {
  constexpr int CW = TN * 32, LPR = CW / 8, RPI = 64 / LPR;   // columns, lanes per row, rows per step
  const int frow = lane & 31, fhalf = lane >> 5;
  auto at = [&](int r, int c) {   // byte of chunk c (4 channels) of row r
    return r * CW * 4 + ((c ^ (TN == 1 ? (r >> 1) & 7 : r & 15)) << 4);
  };
  const int col = wc + (lane % LPR) * 8, n = n0 + col, row = wr + lane / LPR;
  float sb[8], bias[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    sb[k] = scales.sb[col + k];
    bias[k] = scales.bias[col + k];
  }
  T* out = static_cast<T*>(g.y) + (int64_t)(m0 + row) * g.N + n;
  const int left = n < g.N ? g.M - m0 - row : 0, wide = g.N - n;   // rows and columns to the edge
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const float sa = scales.sa[wr + 32 * i + frow];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4_t v;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = (float)acc[i][j][4 * q + r] * sa;
        *reinterpret_cast<f32x4_t*>(part + at(frow, j * 8 + 2 * q + fhalf)) = v;
      }
#pragma unroll
    for (int s = 0; s < 32 / RPI; ++s) {
      const int r = s * RPI + lane / LPR, c = (lane % LPR) * 2;
      const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(part + at(r, c));
      const f32x4_t hi = *reinterpret_cast<const f32x4_t*>(part + at(r, c + 1));
      float v[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = __builtin_fmaf(lo[k], sb[k], bias[k]);
        v[k + 4] = __builtin_fmaf(hi[k], sb[k + 4], bias[k + 4]);
      }
      if (32 * i + s * RPI < left) store8(out, wide, v);
      out += (int64_t)RPI * g.N;
    }
  }
}

}  // namespace fp8dp
