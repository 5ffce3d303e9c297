// int8_skinny.hpp -- the INT8 product for few tokens, as its callers see it.
#pragma once
#include "int8_core.hpp"

namespace fp8dp {

constexpr int kFewTokens = 64;

// Bytes between the rows of codes in LDS: K rounded up to whole 128-byte pieces,
// plus 16 so that the rows of a fragment read start 16 bytes apart in the banks.
__host__ __device__ constexpr int skinny_stride(int K) { return (K + 127) / 128 * 128 + 16; }

// LDS of the casting form beside its ring: codes, tokens (in copies of 1 KB), 16 scales and the
// largest magnitudes of up to 4 waves parts.
constexpr size_t skinny_cast_bytes(int M, int K, int size, int waves) {
  const int64_t chunks = (int64_t)M * K * size / 16, group = 64 * waves;
  return (size_t)M * skinny_stride(K) + (size_t)((chunks + group - 1) / group) * group * 16 +
         4 * (16 + 4 * waves);
}

// x: tokens of the output's type to cast in the kernel (int8_linear), or NULL: codes in g.a.
// At most kFewTokens tokens.
int skinny_i8(const char* what, fp8dp_dtype yt, const I8Args& g, const void* x,
              hipStream_t stream);

// Whether the casting form takes the tokens at x: up to 16 of 16384 values together, or one; rows of
// whole chunks; at most 64 KB of LDS beside the ring of 64 KB, which is 12288 values of FP32 and one token of
// 20480 in 16 bits.  Every workgroup casts all of them, which against a launch of its own (in a graph,
// where a launch costs least) gains at few values and breaks even at 16384: 1 x 4096 x 4096 4.8 us
// for 6.2, 4 x 4096 x 4096 5.7 for 6.3, 8 x 1024 x 1024 4.1 for 5.2, 16 x 4096 x 1024 5.5 for 5.4.
constexpr size_t kCastBytes = 64 * 1024;
static_assert(skinny_cast_bytes(1, 20480, 2, 8) <= kCastBytes && skinny_cast_bytes(1, 20496, 2, 8) > kCastBytes &&
                  skinny_cast_bytes(1, 12288, 4, 8) <= kCastBytes && skinny_cast_bytes(1, 12304, 4, 8) > kCastBytes &&
                  skinny_cast_bytes(16, 768, 4, 8) <= kCastBytes && skinny_cast_bytes(16, 784, 4, 8) > kCastBytes &&
                  skinny_cast_bytes(16, 1024, 2, 8) <= kCastBytes,
              "the limits that the comment names");
inline bool skinny_casts(const I8Args& g, const void* x, int size) {
  return g.M <= 16 && (g.M == 1 || (int64_t)g.M * g.K <= 16384) && g.K % 16 == 0 &&
         g.ldb % 16 == 0 && aligned16(x) && aligned16(g.b) &&
         skinny_cast_bytes(g.M, g.K, size, 8) <= kCastBytes;
}

}  // namespace fp8dp
