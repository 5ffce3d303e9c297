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
};

// Four outputs of row m, columns n .. n + 3, from their integer sums:
// (sum sa) sb + bias in binary32, one rounding to T.  Columns at or past N are
// not stored.
template <typename T>
__device__ __forceinline__ void store_out4(const I8Args& g, int64_t m, int n, float sa,
                                           const float sb[4], const float bias[4], const v4i_t& c) {
  float v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = (float)c[j] * sa * sb[j] + bias[j];
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
template <typename T>
__device__ __forceinline__ void load_cols4(const I8Args& g, int n, float sb[4], float bias[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = n + j < g.N ? n + j : g.N - 1;
    sb[j] = g.sb[c];
    bias[j] = g.bias == nullptr ? 0.0f
              : g.bias_f32      ? static_cast<const float*>(g.bias)[c]
                                : to_f32(static_cast<const T*>(g.bias)[c]);
  }
}

}  // namespace fp8dp
