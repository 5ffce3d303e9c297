// row_norm.hip -- forward kernels over whole rows: dropout with the residual
// sum, layer norm, the INT8 cast with one scale per row, and their fusions
// (one template, k_row).
//
// A row of up to 16384 elements stays in registers from its one read to its
// outputs: a wave per row up to 2048 elements (4 rows per workgroup, no LDS, no
// barrier), a workgroup of 256 or 1024 threads above; longer rows are read
// again by each step (mean, variance, output), from cache where they fit.  The
// variance is the mean of squared distances from the mean, taken after the
// mean from the registers, so it costs no second read and does not cancel.
// All of it is bound by memory: per element one read of each input and one write
// of each output.
#include <hip/hip_runtime.h>

#include "row_core.hpp"

namespace fp8dp {

struct RowArgs {
  const void *x, *residual, *weight, *bias;
  int64_t rows;
  int cols;
  bool wf32;
  DropRule rule;
  const uint64_t* rng;
  float eps;
  void *z, *y;
  float *mean, *rstd;
  int8_t* q;
  int64_t ldq;          // bytes between rows of q; beyond cols they are zeros
  float* scale;
};

// T: element type.  NV vectors of 8 per thread in registers (0: a loop over longer
// rows, and rows of less than 8).  THR threads per row.  DROP: apply the mask.  NORM / QUANT:
// the norm, the cast.  Without both, z (or out) is all there is to write.
template <typename T, int NV, int THR, bool DROP, bool NORM, bool QUANT>
__global__ __launch_bounds__(THR < 256 ? 256 : THR) void k_row(RowArgs a) {
  constexpr int RPB = THR < 256 ? 256 / THR : 1;   // rows per workgroup
  constexpr bool REG = NV > 0;
  constexpr int HELD = REG ? NV : 1;
  constexpr int WAVES = THR / 64;
  __shared__ float scratch[THR > 64 ? 2 * 3 * WAVES : 1];
  const int t = THR > 64 ? (int)threadIdx.x : (int)(threadIdx.x & 63);
  const int sub = THR > 64 ? 0 : (int)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cols = a.cols;
  const int nvec = (int)(((QUANT ? a.ldq : (int64_t)cols) + 7) / 8);
  const int steps = REG ? NV : (nvec + THR - 1) / THR;
  const float fcols = (float)cols;
  const T* const x = static_cast<const T*>(a.x);
  const T* const residual = static_cast<const T*>(a.residual);
  DropKey key = {};
  if constexpr (DROP) key = drop_key(a.rng);

  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPB + sub; row < a.rows;
       row += (int64_t)gridDim.x * RPB, turn ^= 1) {
    float* const sc = scratch + (THR > 64 ? turn * 3 * WAVES : 0);
    const int64_t base = row * cols;
    auto column = [&](int i) { return (i * THR + t) * 8; };
    float v[HELD][8];
    float sum = 0.0f;
    uint32_t top = 0;

    // one vector of the row: mask, residual sum, z, and its part of the first statistic
    auto begin = [&](int i, float* w, const float* r) {
      const int c = column(i), n = cols - c;
      if constexpr (DROP) drop8(key, a.rule, (uint32_t)(i * THR + t), (uint32_t)row, w);
      if (residual != nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] += r[j];
      }
      if (a.z != nullptr) {
        through8<T>(w);
        store8(static_cast<T*>(a.z) + base + c, n, w);
      }
      if constexpr (NORM) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += w[j];
      } else if constexpr (QUANT) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t b = __float_as_uint(w[j]) & 0x7FFFFFFFu;
          top = b > top ? b : top;
        }
      }
    };
    // parameters of a vector: held as loaded (issued ahead of the row), or loaded at their use
    RawParam pw[HELD], pb[HELD];
    auto params = [&](int i, int n, float* g, float* b) {
      if constexpr (REG) {
        widen_param<T>(pw[i], a.weight, a.wf32, n, 1.0f, g);
        widen_param<T>(pb[i], a.bias, a.wf32, n, 0.0f, b);
      } else {
        load_param8<T>(a.weight, a.wf32, column(i), n, 1.0f, g);
        load_param8<T>(a.bias, a.wf32, column(i), n, 0.0f, b);
      }
    };
    if constexpr (REG) {
      // every load of the row first, without a branch, then the arithmetic
      Raw8<T> rx[NV], rr[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) rx[i] = load_row(x + base, column(i), cols);
      if (residual != nullptr) {
#pragma unroll
        for (int i = 0; i < NV; ++i) rr[i] = load_row(residual + base, column(i), cols);
      }
      if constexpr (NORM) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          pw[i] = load_param<T>(a.weight, a.wf32, column(i), cols);
          pb[i] = load_param<T>(a.bias, a.wf32, column(i), cols);
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int n = cols - column(i);
        float r[8] = {};
        settle(rx[i], n);
        widen8f(rx[i], v[i]);
        if (residual != nullptr) {
          settle(rr[i], n);
          widen8f(rr[i], r);
        }
        begin(i, v[i], r);
      }
    } else {
      for (int i = 0; i < steps; ++i) {
        const int c = column(i), n = cols - c;
        float r[8] = {};
        load8(x + base + c, n, v[0]);
        if (residual != nullptr) load8(residual + base + c, n, r);
        begin(i, v[0], r);
      }
    }
    // f(i, values): from the registers, or read again
    auto each = [&](auto&& f) {
      if constexpr (REG) {
#pragma unroll
        for (int i = 0; i < NV; ++i) f(i, v[i]);
      } else {
        const T* const from = a.z != nullptr ? static_cast<const T*>(a.z) : x;
        for (int i = 0; i < steps; ++i) {
          load8(from + base + column(i), cols - column(i), v[0]);
          f(i, v[0]);
        }
      }
    };

    float mean = 0.0f, rstd = 0.0f;
    if constexpr (NORM) {
      mean = row_sum<THR>(sum, sc) / fcols;
      float sq = 0.0f;
      each([&](int i, float* w) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] -= mean;
        zero_from8(cols - column(i), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) sq = __builtin_fmaf(w[j], w[j], sq);
      });
      const float var = row_sum<THR>(sq, sc + WAVES) / fcols;
      rstd = 1.0f / __fsqrt_rn(var + a.eps);
      if (t == 0) {
        if (a.mean != nullptr) a.mean[row] = mean;
        if (a.rstd != nullptr) a.rstd[row] = rstd;
      }
      // in registers the row is now x - mean; read again it is x
      each([&](int i, float* w) {
        const int c = column(i), n = cols - c;
        float g[8], b[8];
        params(i, n, g, b);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          w[j] = __builtin_fmaf((REG ? w[j] : w[j] - mean) * rstd, g[j], b[j]);
        if constexpr (QUANT) {
          zero_from8(n, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t m = __float_as_uint(w[j]) & 0x7FFFFFFFu;
            top = m > top ? m : top;
          }
        } else {
          store8(static_cast<T*>(a.y) + base + c, n, w);
        }
      });
    }

    if constexpr (QUANT) {
      top = row_umax<THR>(top, reinterpret_cast<uint32_t*>(sc) + 2 * WAVES);
      const bool plain = top != 0 && top < 0x7F800000u;
      const RowScale s = row_scale(plain ? top : 0x3F800000u);
      if (t == 0)
        a.scale[row] = plain ? __uint_as_float(top) / 127.0f
                             : (top == 0 ? 0.0f : __builtin_nanf(""));
      int8_t* const q = a.q + row * a.ldq;
      each([&](int i, float* w) {
        const int c = column(i), n = cols - c;
        if constexpr (NORM && !REG) {
          float g[8], b[8];
          params(i, n, g, b);
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = __builtin_fmaf((w[j] - mean) * rstd, g[j], b[j]);
          zero_from8(n, w);
        }
        uint2 code = {0u, 0u};
        if (plain) code = codes8<NORM || sizeof(T) == 4>(w, s);
        const int64_t room = a.ldq - c;
        store_codes8(q + c, room < 8 ? (int)room : 8, code);
      });
    }
  }
}

template <typename T, int NV, int THR, bool DROP, bool NORM, bool QUANT>
static int launch_row(const RowArgs& a, const char* what, hipStream_t stream) {
  constexpr int RPB = THR < 256 ? 256 / THR : 1;
  const int64_t need = (a.rows + RPB - 1) / RPB;
  const unsigned grid = grid_for(need * 256, 256, 64);
  hipLaunchKernelGGL((k_row<T, NV, THR, DROP, NORM, QUANT>), dim3(grid),
                     dim3(THR < 256 ? 256 : THR), 0, stream, a);
  return check_launch(what);
}

// Threads and registers per row by its vectors of 8 elements.
template <typename T, bool DROP, bool NORM, bool QUANT>
static int launch_width(const RowArgs& a, const char* what, hipStream_t stream) {
  const int64_t nvec = ((QUANT ? a.ldq : (int64_t)a.cols) + 7) / 8;
  if (a.cols < 8) return launch_row<T, 0, 64, DROP, NORM, QUANT>(a, what, stream);
  if (nvec <= 64) return launch_row<T, 1, 64, DROP, NORM, QUANT>(a, what, stream);
  if (nvec <= 128) return launch_row<T, 2, 64, DROP, NORM, QUANT>(a, what, stream);
  if (nvec <= 256) return launch_row<T, 4, 64, DROP, NORM, QUANT>(a, what, stream);
  if (nvec <= 512) return launch_row<T, 2, 256, DROP, NORM, QUANT>(a, what, stream);
  if (nvec <= 1024) return launch_row<T, 4, 256, DROP, NORM, QUANT>(a, what, stream);
  if (nvec <= 2048) return launch_row<T, 2, 1024, DROP, NORM, QUANT>(a, what, stream);
  return launch_row<T, 0, 1024, DROP, NORM, QUANT>(a, what, stream);
}

template <bool DROP, bool NORM, bool QUANT>
static int launch_type(fp8dp_dtype dt, const RowArgs& a, const char* what, hipStream_t stream) {
  if (dt == FP8DP_BF16) return launch_width<bf16_t, DROP, NORM, QUANT>(a, what, stream);
  if (dt == FP8DP_F16) return launch_width<f16_t, DROP, NORM, QUANT>(a, what, stream);
  return launch_width<float, DROP, NORM, QUANT>(a, what, stream);
}

static int check_eps(const char* what, float eps) {
  if (eps >= 0.0f && eps <= 3.402823466e38f) return FP8DP_OK;
  set_error("%s: eps must not be negative, and finite", what);
  return FP8DP_EINVAL;
}

static int check_drop(const char* what, float p, const uint64_t* rng, DropRule* rule) {
  if (!drop_rule(p, rule)) {
    set_error("%s: p must be 0 .. 1", what);
    return FP8DP_EINVAL;
  }
  if (p > 0.0f && rng == nullptr) {
    set_error("%s: p > 0 needs rng (seed and offset on the device)", what);
    return FP8DP_EINVAL;
  }
  return FP8DP_OK;
}

// The cast into rows of ldq bytes (at least cols), for int8_linear as well.
int quantize_rows(const char* what, const void* x, int64_t rows, int64_t cols, fp8dp_dtype dt,
                  int8_t* q, int64_t ldq, float* scale, hipStream_t stream) {
  RowArgs a = {};
  a.x = x;
  a.rows = rows;
  a.cols = (int)cols;
  a.q = q;
  a.ldq = ldq;
  a.scale = scale;
  return launch_type<false, false, true>(dt, a, what, stream);
}

}  // namespace fp8dp

using namespace fp8dp;

extern "C" int layer_norm(const void* x, const void* weight, const void* bias, int64_t rows,
                          int64_t cols, fp8dp_dtype dt, fp8dp_dtype wt, float eps, void* y,
                          float* mean, float* rstd, hipStream_t stream) {
  const char* what = "layer_norm";
  int rc = check_rows(what, rows, cols);   // first: an empty tensor has no address
  if (rc) return rc;
  if (x == nullptr || y == nullptr) {
    set_error("%s: x and y must be non-NULL", what);
    return FP8DP_EINVAL;
  }
  if ((rc = check_types(what, dt, wt)) ||
      (rc = check_eps(what, eps)))
    return rc;
  const int64_t e = dtype_size(dt), we = dtype_size(wt);
  if (!aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(weight, we) || !aligned_to(bias, we) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return bad_align(what);
  RowArgs a = {};
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.rows = rows;
  a.cols = (int)cols;
  a.wf32 = wt == FP8DP_F32;
  a.eps = eps;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  return launch_type<false, true, false>(dt, a, what, stream);
}

extern "C" int dropout_add(const void* x, const void* residual, int64_t rows, int64_t cols,
                           fp8dp_dtype dt, float p, const uint64_t* rng, void* out,
                           hipStream_t stream) {
  const char* what = "dropout_add";
  int rc = check_rows(what, rows, cols);   // first: an empty tensor has no address
  if (rc) return rc;
  if (x == nullptr || out == nullptr) {
    set_error("%s: x and out must be non-NULL", what);
    return FP8DP_EINVAL;
  }
  RowArgs a = {};
  if ((rc = check_types(what, dt, dt)) ||
      (rc = check_drop(what, p, rng, &a.rule)))
    return rc;
  const int64_t e = dtype_size(dt);
  if (!aligned_to(x, e) || !aligned_to(residual, e) || !aligned_to(out, e) || !aligned_to(rng, 8))
    return bad_align(what);
  a.x = x;
  a.residual = residual;
  a.rows = rows;
  a.cols = (int)cols;
  a.rng = rng;
  a.z = out;
  return a.rule.threshold > 0 ? launch_type<true, false, false>(dt, a, what, stream)
                              : launch_type<false, false, false>(dt, a, what, stream);
}

extern "C" int dropout_add_layer_norm(const void* x, const void* residual, const void* weight,
                                      const void* bias, int64_t rows, int64_t cols, fp8dp_dtype dt,
                                      fp8dp_dtype wt, float p, const uint64_t* rng, float eps,
                                      void* z, void* y, float* mean, float* rstd,
                                      hipStream_t stream) {
  const char* what = "dropout_add_layer_norm";
  int rc = check_rows(what, rows, cols);   // first: an empty tensor has no address
  if (rc) return rc;
  if (x == nullptr || z == nullptr || y == nullptr) {
    set_error("%s: x, z and y must be non-NULL", what);
    return FP8DP_EINVAL;
  }
  RowArgs a = {};
  if ((rc = check_types(what, dt, wt)) ||
      (rc = check_drop(what, p, rng, &a.rule)) || (rc = check_eps(what, eps)))
    return rc;
  const int64_t e = dtype_size(dt), we = dtype_size(wt);
  if (!aligned_to(x, e) || !aligned_to(residual, e) || !aligned_to(z, e) || !aligned_to(y, e) ||
      !aligned_to(weight, we) || !aligned_to(bias, we) || !aligned_to(mean, 4) ||
      !aligned_to(rstd, 4) || !aligned_to(rng, 8))
    return bad_align(what);
  if (y == z) {
    set_error("%s: y and z must not be the same buffer", what);
    return FP8DP_EINVAL;
  }
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.bias = bias;
  a.rows = rows;
  a.cols = (int)cols;
  a.wf32 = wt == FP8DP_F32;
  a.rng = rng;
  a.eps = eps;
  a.z = z;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  return a.rule.threshold > 0 ? launch_type<true, true, false>(dt, a, what, stream)
                              : launch_type<false, true, false>(dt, a, what, stream);
}

extern "C" int quantize_int8(const void* x, int64_t rows, int64_t cols, fp8dp_dtype dt, int8_t* q,
                             float* scale, hipStream_t stream) {
  const char* what = "quantize_int8";
  int rc = check_rows(what, rows, cols);   // first: an empty tensor has no address
  if (rc) return rc;
  if (x == nullptr || q == nullptr || scale == nullptr) {
    set_error("%s: x, q and scale must be non-NULL", what);
    return FP8DP_EINVAL;
  }
  if ((rc = check_types(what, dt, dt))) return rc;
  if (!aligned_to(x, dtype_size(dt)) || !aligned_to(scale, 4)) return bad_align(what);
  return quantize_rows(what, x, rows, cols, dt, q, cols, scale, stream);
}

extern "C" int layer_norm_quantize_int8(const void* x, const void* residual, const void* weight,
                                        const void* bias, int64_t rows, int64_t cols,
                                        fp8dp_dtype dt, fp8dp_dtype wt, float eps, void* z,
                                        int8_t* q, float* scale, hipStream_t stream) {
  const char* what = "layer_norm_quantize_int8";
  int rc = check_rows(what, rows, cols);   // first: an empty tensor has no address
  if (rc) return rc;
  if (x == nullptr || q == nullptr || scale == nullptr) {
    set_error("%s: x, q and scale must be non-NULL", what);
    return FP8DP_EINVAL;
  }
  if ((residual == nullptr) != (z == nullptr)) {
    set_error("%s: residual and z go together", what);
    return FP8DP_EINVAL;
  }
  if ((rc = check_types(what, dt, wt)) ||
      (rc = check_eps(what, eps)))
    return rc;
  const int64_t e = dtype_size(dt), we = dtype_size(wt);
  if (!aligned_to(x, e) || !aligned_to(residual, e) || !aligned_to(z, e) ||
      !aligned_to(weight, we) || !aligned_to(bias, we) || !aligned_to(scale, 4))
    return bad_align(what);
  RowArgs a = {};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.bias = bias;
  a.rows = rows;
  a.cols = (int)cols;
  a.wf32 = wt == FP8DP_F32;
  a.eps = eps;
  a.z = z;
  a.q = q;
  a.ldq = cols;
  a.scale = scale;
  return launch_type<false, true, true>(dt, a, what, stream);
}
