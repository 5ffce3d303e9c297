// gated_core.hpp -- pieces shared by the gated linear layer's kernels: the activations with their
// derivatives, argument checks and the choice of tiles.
#pragma once
#include "fp8dp_gated.h"
#include "mma16.hpp"

namespace fp8dp {

__device__ __forceinline__ float sigmoid_of(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-g));   // (1 ulp each; exp of a large -g is infinite, its inverse 0)
}
// f(g), and f'(g) where GRAD.  The tails are formed without cancelling: sigmoid(v) for (1 + tanh(v / 2)) / 2
// and the complementary error function for 1 + erf.
template <int ACT, bool GRAD>
__device__ __forceinline__ float gate_of(float g, float* slope) {
  switch (ACT) {
    case FP8DP_GATE_SILU: {
      const float p = sigmoid_of(g);
      if (GRAD) *slope = __builtin_fmaf(g * p, 1.0f - p, p);
      return g * p;
    }
    case FP8DP_GATE_GELU: {
      const float p = 0.5f * erfcf(g * -0.70710678118654752f);
      if (GRAD) *slope = __builtin_fmaf(g * 0.39894228040143268f, __expf(-0.5f * g * g), p);
      return g * p;
    }
    case FP8DP_GATE_GELU_TANH: {
      // beyond 20 the sigmoid is 0 or 1, and the cube would leave binary32
      const float c = g < -20.0f ? -20.0f : g > 20.0f ? 20.0f : g;
      const float p = sigmoid_of(1.5957691216057308f * __builtin_fmaf(0.044715f * c * c, c, c));
      if (GRAD)
        *slope = __builtin_fmaf(g * p * (1.0f - p),
                                1.5957691216057308f * __builtin_fmaf(0.134145f * c, c, 1.0f), p);
      return g * p;
    }
    case FP8DP_GATE_SIGMOID: {
      const float p = sigmoid_of(g);
      if (GRAD) *slope = p * sigmoid_of(-g);   // (1 - p would cancel: nothing was left of it from g = 17 on)
      return p;
    }
    case FP8DP_GATE_RELU:
      if (GRAD) *slope = g > 0.0f ? 1.0f : 0.0f;
      return g <= 0.0f ? 0.0f : g;   // (a NaN stays one)
    case FP8DP_GATE_RELU2: {
      const float r = g <= 0.0f ? 0.0f : g;
      if (GRAD) *slope = 2.0f * r;
      return r * r;
    }
    default:
      if (GRAD) *slope = 1.0f;
      return g;
  }
}

// f(std::integral_constant<int, act>): one branch for a whole tile or kernel.  (A branch per element made 64 times seven
// pieces of code of a tile's outputs, which the instruction cache does not hold: 16384 x 8192 x 128, 180 us
// against 126.)
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case FP8DP_GATE_SILU: return f(std::integral_constant<int, FP8DP_GATE_SILU>{});
    case FP8DP_GATE_GELU: return f(std::integral_constant<int, FP8DP_GATE_GELU>{});
    case FP8DP_GATE_GELU_TANH: return f(std::integral_constant<int, FP8DP_GATE_GELU_TANH>{});
    case FP8DP_GATE_SIGMOID: return f(std::integral_constant<int, FP8DP_GATE_SIGMOID>{});
    case FP8DP_GATE_RELU: return f(std::integral_constant<int, FP8DP_GATE_RELU>{});
    case FP8DP_GATE_RELU2: return f(std::integral_constant<int, FP8DP_GATE_RELU2>{});
    default: return f(std::integral_constant<int, FP8DP_GATE_IDENTITY>{});
  }
}

inline int check_gated(const char* what, int64_t M, int64_t N, int64_t K, fp8dp_dtype dt, fp8dp_gate act,
                       const void* workspace, int64_t workspace_bytes) {
  if (M < 1 || N < 1 || K < 1 || M > FP8DP_GATED_MAX_ROWS || N > FP8DP_GATED_MAX_WIDTH ||
      K > FP8DP_GATED_MAX_WIDTH) {
    set_error("%s: M must be 1 .. %d, N and K 1 .. %d (got %lld, %lld, %lld)", what,
              FP8DP_GATED_MAX_ROWS, FP8DP_GATED_MAX_WIDTH, (long long)M, (long long)N, (long long)K);
    return FP8DP_EINVAL;
  }
  if (dt != FP8DP_BF16 && dt != FP8DP_F16) {
    set_error("%s: the type must be bfloat16 or float16", what);
    return FP8DP_EINVAL;
  }
  if (act < FP8DP_GATE_SILU || act > FP8DP_GATE_IDENTITY) {
    set_error("%s: unknown activation %d", what, (int)act);
    return FP8DP_EINVAL;
  }
  if (workspace_bytes < 0 || !aligned_to(workspace, 16)) {
    set_error("%s: workspace must be 16-byte aligned, its size not negative", what);
    return FP8DP_EINVAL;
  }
  return FP8DP_OK;
}

// Whether an operand's rows can be copied in chunks of 16 bytes.
inline bool rows16(const Operand& o, int64_t width) {
  return o.ld % 8 == 0 && width % 8 == 0 && aligned16(o.p[0]) && aligned16(o.p[1]);
}

// Tiles of a product of m x n outputs over `stages` of K, and over how many workgroups K is split.
enum TileShape { kTile256, kTile192, kTile128, kTileAny };   // 256 x 256, 256 x 192, 128 x 128, the same at any alignment
struct ProductPlan {
  TileShape shape;
  int splits;
};
inline int64_t tiles_of(TileShape t, int64_t m, int64_t n) {
  const int64_t bm = t == kTile256 || t == kTile192 ? 256 : 128;
  const int64_t bn = t == kTile256 ? 256 : t == kTile192 ? 192 : 128;
  return ((m + bm - 1) / bm) * ((n + bn - 1) / bn);
}
// The plan of the least estimate, in us: a workgroup's stages of 64 of K and, for each tile, its ends (the first copies,
// the outputs).  The stages' times were measured, as the difference of K = 4096 and 1024 over 48, with every compute unit busy
// with one tile or two: 256 x 256 1.40 .. 1.72 (4096 x 4096), 256 x 192 1.02 .. 1.04, 128 x 128 0.44 .. 0.49 where it has a
// compute unit to itself, 0.80 .. 0.85 for two, at any alignment 1.04 .. 1.30 and 1.35 .. 1.56.  A K that is
// shared costs a join.  With estimates that favoured shares by a third more, gradients of 1025 x 1023 x 1001 took 50.5 us
// for 45.9 (dx from three shares, now one), 8192 x 2048 x 768 169 for 161, one forward of 100 x 1024 x 1024 14.1 for 11.6;
// 1000 x 8192 x 4096 is the worst loss that was found (302, now 312).
inline ProductPlan plan_product(int64_t m, int64_t n, int64_t stages, bool dual, bool direct) {
  const double cus = num_cus();
  ProductPlan best = {direct ? kTile256 : kTileAny, 1};
  double least = 1e30;
  auto offer = [&](TileShape t, double per_stage, double alone, int per_cu, double ends) {
    const double tiles = (double)tiles_of(t, m, n);
    for (int s = 1; s <= 8 && (s == 1 || stages / s >= 4); ++s) {
      const double groups = tiles * s, turns = std::ceil(groups / (cus * per_cu));
      const double each = (double)((stages + s - 1) / s) * (groups <= cus ? alone : per_stage) + ends;
      const double join = s == 1 ? 0.0 : 4.0 + s * (double)m * (double)n * 8.0 / 4e6;
      const double us = turns * each + join;
      if (us < least) {
        least = us;
        best = {t, s};
      }
    }
  };
  if (direct) {
    offer(kTile256, 1.45, 1.45, 1, 5.0);
    if (!dual) offer(kTile192, 1.05, 1.05, 1, 4.5);
    offer(kTile128, 0.82, 0.45, 2, 3.5);
  } else {
    offer(kTileAny, 1.45, 1.15, 2, 3.5);
  }
  return best;
}

inline int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

}  // namespace fp8dp
