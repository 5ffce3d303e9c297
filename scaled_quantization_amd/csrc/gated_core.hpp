// gated_core.hpp -- pieces shared by the gated linear layer's kernels: the activations with their
// derivatives and argument checks.
#pragma once
#include "fp8dp_gated.h"
#include "mma16.hpp"
#include "product_plan.hpp"

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

inline ProductPlan plan_product(int64_t m, int64_t n, int64_t stages, bool dual, bool direct) {
  return plan_product(m, n, stages, dual, direct, num_cus());
}

inline int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

}  // namespace fp8dp
