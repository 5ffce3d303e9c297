// int8_skinny.hpp -- the INT8 product for few tokens, as its callers see it.
#pragma once
#include "int8_core.hpp"

namespace fp8dp {

// Bytes between the rows of codes in LDS: K rounded up to whole 128-byte pieces,
// plus 16 so that the 16 rows of a fragment read start 16 bytes apart in the banks.
__host__ __device__ constexpr int skinny_stride(int K) { return (K + 127) / 128 * 128 + 16; }

// x: tokens of the output's type to cast in the kernel (int8_linear), or NULL: codes in g.a.
int skinny_i8(const char* what, fp8dp_dtype yt, const I8Args& g, const void* x,
              hipStream_t stream);

// Whether the casting form takes these tokens: one tile of 16, their codes in LDS.
inline bool skinny_casts(int64_t M, int64_t K) {
  return M <= 16 && K >= 128 && M * skinny_stride((int)K) <= 128 * 1024;
}

}  // namespace fp8dp
