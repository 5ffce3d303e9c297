// row_norm.hip -- forward kernels: dropout with the residual sum, layer norm, the
// INT8 cast with one scale per row, and their fusions over whole rows (one template, k_row).
//
// A row of up to 16384 elements stays in registers from its one read to its
// outputs: a wave per row up to 2048 elements (4 rows per workgroup, no LDS, no
// barrier), a workgroup of 256 or 1024 threads above; longer rows are read
// again by each step (mean, variance, output), from cache where they fit.  The
// variance is the mean of squared distances from the mean, taken after the
// mean from the registers, so it costs no second read and does not cancel.
// Tensors beyond the caches are bound by memory (per element one read of each input and one write
// of each output), rows that come from cache by their instructions.
#include <hip/hip_runtime.h>

#include "row_core.hpp"

namespace fp8dp {

// Dropout and residual sum alone, where no row needs its other elements: a thread per
// vector, rows and vectors in one index, so that odd lengths leave no thread idle (with a
// workgroup per row 1023 x 4097 FP32 took 10.6 us, this 10.2) and a single long row fills the device.
template <typename T, bool DROP>
__global__ __launch_bounds__(256) void k_drop(const T* x, const T* residual, int64_t rows, int cols,
                                              DropRule rule, const uint64_t* rng, T* out) {
  DropKey key = {};
  if constexpr (DROP) key = drop_key(rng);
  const uint32_t nvec = ((uint32_t)cols + 7) / 8;
  const uint64_t total = (uint64_t)rows * nvec, step = (uint64_t)gridDim.x * 256;
  const uint64_t step_rows = step / nvec;
  const uint32_t step_vecs = (uint32_t)(step - step_rows * nvec);
  uint64_t at = (uint64_t)blockIdx.x * 256 + threadIdx.x;
  uint64_t row = total >> 32 ? at / nvec : (uint32_t)at / nvec;
  uint32_t vec = (uint32_t)(at - row * nvec);
  for (; at < total; at += step) {
    const int c = (int)vec * 8, n = cols - c;
    const int64_t o = (int64_t)row * cols + c;
    float v[8], r[8];
    const Raw8<T> rx = load_raw(x + o, n);
    Raw8<T> rr = {};
    if (residual != nullptr) rr = load_raw(residual + o, n);
    widen8f(rx, v);
    if constexpr (DROP) drop8(key, rule, vec, (uint32_t)row, v);
    if (residual != nullptr) {
      widen8f(rr, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += r[j];
    }
    store8(out + o, n, v);
    row += step_rows;
    vec += step_vecs;
    if (vec >= nvec) {
      vec -= nvec;
      ++row;
    }
  }
}

template <typename T, bool DROP>
static int launch_drop(const void* x, const void* residual, int64_t rows, int64_t cols,
                       DropRule rule, const uint64_t* rng, void* out, hipStream_t stream) {
  // one vector per thread (a loop of 16 workgroups per compute unit: 65536 x 4096 BF16 335 us, this 266)
  const unsigned grid = grid_for(rows * ((cols + 7) / 8), 256, 1024);
  hipLaunchKernelGGL((k_drop<T, DROP>), dim3(grid), dim3(256), 0, stream, static_cast<const T*>(x),
                     static_cast<const T*>(residual), rows, (int)cols, rule, rng,
                     static_cast<T*>(out));
  return check_launch("dropout_add");
}

template <bool DROP>
static int launch_drop_type(fp8dp_dtype dt, const void* x, const void* residual, int64_t rows,
                            int64_t cols, DropRule rule, const uint64_t* rng, void* out,
                            hipStream_t stream) {
  if (dt == FP8DP_BF16)
    return launch_drop<bf16_t, DROP>(x, residual, rows, cols, rule, rng, out, stream);
  if (dt == FP8DP_F16)
    return launch_drop<f16_t, DROP>(x, residual, rows, cols, rule, rng, out, stream);
  return launch_drop<float, DROP>(x, residual, rows, cols, rule, rng, out, stream);
}

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

// T: element type.  NV: vectors of 8 per thread, ceil(cols / 8 / THR).  THR: threads per row.
// DROP: apply the mask.  NORM / QUANT: the norm, the cast, one of them at least.
//
// A wave costs 4 cycles an instruction on its SIMD, so rows that come from cache are
// bound by the instructions per element, not by memory: the parameters are widened
// once for all rows of a wave, the masks of the last vector are kept in registers, and
// the next row is loaded while one is in hand (the last one loads itself again).
template <typename T, int NV, int THR, bool DROP, bool NORM, bool QUANT>
__global__ __launch_bounds__(THR == 64 ? 256 : THR) void k_row(RowArgs a) {
  constexpr int RPB = THR == 64 ? 4 : 1;   // rows per workgroup
  constexpr int WAVES = THR / 64;
  __shared__ float scratch[THR > 64 ? 2 * 3 * WAVES : 1];
  const int t = THR > 64 ? (int)threadIdx.x : (int)(threadIdx.x & 63);
  const int sub = THR > 64 ? 0 : (int)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cols = a.cols;
  const bool ragged = cols % 8 != 0;
  const float inv_cols = 1.0f / (float)cols;
  const T* const x = static_cast<const T*>(a.x);
  const T* const residual = static_cast<const T*>(a.residual);
  DropKey key = {};
  if constexpr (DROP) key = drop_key(a.rng);
  auto column = [&](int i) { return (i * THR + t) * 8; };
  const int n_last = cols - column(NV - 1);
  auto count = [&](int i) { return i < NV - 1 ? 8 : n_last; };   // elements of vector i
  const Mask8 mask(n_last);

  struct Row {
    Raw8<T> x[NV], r[NV];
  };
  auto load = [&](int64_t row, Row& o) {
    const int64_t base = row * cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) o.x[i] = load_row(x + base, column(i), cols);
    if (residual != nullptr) {
#pragma unroll
      for (int i = 0; i < NV; ++i) o.r[i] = load_row(residual + base, column(i), cols);
    }
  };
  const int64_t step = (int64_t)gridDim.x * RPB, begin = (int64_t)blockIdx.x * RPB + sub;
  if (begin >= a.rows) return;   // (whole waves, or with THR > 64 whole workgroups)
  Row next;
  load(begin, next);

  float g[NORM ? NV : 1][8], b[NORM ? NV : 1][8];
  if constexpr (NORM) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      load_param8<T>(a.weight, a.wf32, column(i), count(i), 1.0f, g[i]);
      load_param8<T>(a.bias, a.wf32, column(i), count(i), 0.0f, b[i]);
    }
    mask.clear(g[NV - 1]);   // (NULL parameters fill all 8)
    mask.clear(b[NV - 1]);
  }

  int turn = 0;
  for (int64_t row = begin; row < a.rows; row += step, turn ^= 1) {
    float* const sc = scratch + (THR > 64 ? turn * 3 * WAVES : 0);
    const int64_t base = row * cols;
    const Row now = next;
    load(row + step < a.rows ? row + step : row, next);

    float v[NV][8];
    float sum = 0.0f;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float* const w = v[i];
      Raw8<T> raw = now.x[i];
      if (i == NV - 1) {
        settle(raw, n_last, ragged);
        mask.clear_empty(raw);
      }
      widen8f(raw, w);
      if constexpr (DROP) drop8(key, a.rule, (uint32_t)(i * THR + t), (uint32_t)row, w);
      if (residual != nullptr) {
        float r[8];
        raw = now.r[i];
        if (i == NV - 1) {
          settle(raw, n_last, ragged);
          mask.clear_empty(raw);
        }
        widen8f(raw, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] += r[j];
      }
      if (a.z != nullptr) {
        const Raw8<T> out = round8(w, T{});
        store_row(element(static_cast<T*>(a.z) + base, column(i)), count(i), out);
        widen8f(out, w);
      }
      if constexpr (NORM) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += w[j];
      } else if constexpr (QUANT) {
        top = magnitude8(w, top);
      }
    }

    if constexpr (NORM) {
      const float mean = row_sum<THR>(sum, sc) * inv_cols;
      float sq = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] -= mean;
        if (i == NV - 1) mask.clear(v[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) sq = __builtin_fmaf(v[i][j], v[i][j], sq);
      }
      const float rstd = rsqrtf(row_sum<THR>(sq, sc + WAVES) * inv_cols + a.eps);
      if (t == 0) {
        if (a.mean != nullptr) a.mean[row] = mean;
        if (a.rstd != nullptr) a.rstd[row] = rstd;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = __builtin_fmaf(v[i][j] * rstd, g[i][j], b[i][j]);
        if constexpr (QUANT) {
          if (i == NV - 1) mask.clear(v[i]);   // (a NaN row's padding too)
          top = magnitude8(v[i], top);
        } else {
          store_row(element(static_cast<T*>(a.y) + base, column(i)), count(i), round8(v[i], T{}));
        }
      }
    }

    if constexpr (QUANT) {
      top = row_umax<THR>(top, reinterpret_cast<uint32_t*>(sc) + 2 * WAVES);
      const bool plain = top != 0 && top < 0x7F800000u;
      const RowScale s = row_scale(plain ? top : 0x3F800000u);
      if (t == 0)
        a.scale[row] = plain ? __uint_as_float(top) / 127.0f
                             : (top == 0 ? 0.0f : __builtin_nanf(""));
      int8_t* const q = a.q + row * a.ldq;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = column(i);
        uint2 code = {0u, 0u};
        if (plain) code = codes8<NORM || sizeof(T) == 4>(v[i], s);
        // rows of q may be padded by up to 15 bytes of zeros
        if (i < NV - 1) store_codes8(element(q, c), 8, code);
        else store_codes8(q + c, a.ldq - c < 8 ? (int)(a.ldq - c) : 8, code);
      }
    }
  }
}

// Rows of more than 16384 elements, or less than 8: a loop that reads the row
// again for each statistic and for the output.  A thread's sums may be of 2^17 vectors: LongSum.
template <typename T, int THR, bool DROP, bool NORM, bool QUANT>
__global__ __launch_bounds__(THR == 64 ? 256 : THR) void k_row_loop(RowArgs a) {
  constexpr int RPB = THR == 64 ? 4 : 1;
  constexpr int WAVES = THR / 64;
  __shared__ float scratch[THR > 64 ? 2 * 3 * WAVES : 1];
  const int t = THR > 64 ? (int)threadIdx.x : (int)(threadIdx.x & 63);
  const int sub = THR > 64 ? 0 : (int)(threadIdx.x >> 6);
  const int cols = a.cols;
  const int wide = (int)(QUANT ? a.ldq : (int64_t)cols);
  const float inv_cols = 1.0f / (float)cols;
  const T* const x = static_cast<const T*>(a.x);
  const T* const residual = static_cast<const T*>(a.residual);
  DropKey key = {};
  if constexpr (DROP) key = drop_key(a.rng);

  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPB + sub; row < a.rows;
       row += (int64_t)gridDim.x * RPB, turn ^= 1) {
    float* const sc = scratch + (THR > 64 ? turn * 3 * WAVES : 0);
    const int64_t base = row * cols;
    const T* const again = (a.z != nullptr ? static_cast<const T*>(a.z) : x) + base;
    float w[8], mean = 0.0f, rstd = 0.0f;
    LongSum sum;
    uint32_t top = 0;
    auto normed = [&](int c) {
      float g[8], b[8];
      load8(again + c, cols - c, w);
      load_param8<T>(a.weight, a.wf32, c, cols - c, 1.0f, g);
      load_param8<T>(a.bias, a.wf32, c, cols - c, 0.0f, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = __builtin_fmaf((w[j] - mean) * rstd, g[j], b[j]);
      zero_from8(cols - c, w);
    };
    for (int c = t * 8; c < cols; c += THR * 8) {
      const int n = cols - c;
      load8(x + base + c, n, w);
      if constexpr (DROP) drop8(key, a.rule, (uint32_t)(c / 8), (uint32_t)row, w);
      if (residual != nullptr) {
        float r[8];
        load8(residual + base + c, n, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] += r[j];
      }
      if (a.z != nullptr) {
        through8<T>(w);
        store8(static_cast<T*>(a.z) + base + c, n, w);
      }
      if constexpr (NORM) {
        zero_from8(n, w);
        sum.add(sum8(w));
      } else if constexpr (QUANT) {
        top = magnitude8(w, top);
      }
    }
    if constexpr (NORM) {
      mean = row_sum<THR>(sum.total(), sc) * inv_cols;
      LongSum sq;
      for (int c = t * 8; c < cols; c += THR * 8) {
        load8(again + c, cols - c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] -= mean;
        zero_from8(cols - c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] *= w[j];
        sq.add(sum8(w));
      }
      rstd = rsqrtf(row_sum<THR>(sq.total(), sc + WAVES) * inv_cols + a.eps);
      if (t == 0) {
        if (a.mean != nullptr) a.mean[row] = mean;
        if (a.rstd != nullptr) a.rstd[row] = rstd;
      }
      for (int c = t * 8; c < cols; c += THR * 8) {
        normed(c);
        if constexpr (QUANT) top = magnitude8(w, top);
        else store8(static_cast<T*>(a.y) + base + c, cols - c, w);
      }
    }
    if constexpr (QUANT) {
      top = row_umax<THR>(top, reinterpret_cast<uint32_t*>(sc) + 2 * WAVES);
      const bool plain = top != 0 && top < 0x7F800000u;
      const RowScale s = row_scale(plain ? top : 0x3F800000u);
      if (t == 0)
        a.scale[row] = plain ? __uint_as_float(top) / 127.0f
                             : (top == 0 ? 0.0f : __builtin_nanf(""));
      for (int c = t * 8; c < wide; c += THR * 8) {
        if constexpr (NORM) normed(c);
        else load8(again + c, cols - c, w);
        uint2 code = {0u, 0u};
        if (plain) code = codes8<NORM || sizeof(T) == 4>(w, s);
        store_codes8(a.q + row * a.ldq + c, wide - c, code);
      }
    }
  }
}

// Waves per compute unit that the grid is made for.  Tensors that the caches hold (512 MB
// moved in all: the last-level cache has 256 MB) do best with few waves that walk many rows,
// which spares them the parameters and masks; streams from memory with many
// short ones, whose reads and writes the scheduler keeps apart.  Measured, 16 against
// 256 waves: layer norm 16384 x 768 10.4 / 13.9 us, dropout + residual + norm 30001 x 1600 74 / 95;
// layer norm 65536 x 4096 206 / 179, with dropout and residual 444 / 382.  The norm
// with the cast is bound by its instructions and keeps to few waves: 65536 x 4096 190 / 202 us,
// 4096 x 16384 55.4 / 55.2.  (With the residual, which it also writes back, 401 / 325.)
constexpr int64_t kRowStreamBytes = (int64_t)512 << 20;

template <typename T, int NV, int THR, bool DROP, bool NORM, bool QUANT>
static int launch_row(const RowArgs& a, const char* what, hipStream_t stream) {
  constexpr int RPB = THR == 64 ? 4 : 1, BLOCK = THR == 64 ? 256 : THR;
  const int64_t need = (a.rows + RPB - 1) / RPB;
  const int64_t per = sizeof(T) * (1 + (a.residual != nullptr) + (a.z != nullptr) + (a.y != nullptr)) +
                      (QUANT ? 1 : 0);
  const bool streams = a.rows * a.cols * per > kRowStreamBytes && !(NORM && QUANT);
  const unsigned grid = grid_for(need * BLOCK, BLOCK, std::max(1, (streams ? 256 : 16) * 64 / BLOCK));
  if constexpr (NV > 0)
    hipLaunchKernelGGL((k_row<T, NV, THR, DROP, NORM, QUANT>), dim3(grid), dim3(BLOCK), 0, stream,
                       a);
  else
    hipLaunchKernelGGL((k_row_loop<T, THR, DROP, NORM, QUANT>), dim3(grid), dim3(BLOCK), 0, stream,
                       a);
  return check_launch(what);
}

// Threads and registers per row by its vectors of 8 elements.
template <typename T, bool DROP, bool NORM, bool QUANT>
static int launch_width(const RowArgs& a, const char* what, hipStream_t stream) {
  const int64_t nvec = ((QUANT ? a.ldq : (int64_t)a.cols) + 7) / 8;
  if (a.cols < 8) return launch_row<T, 0, 64, DROP, NORM, QUANT>(a, what, stream);
  if (nvec <= 64) return launch_row<T, 1, 64, DROP, NORM, QUANT>(a, what, stream);
  if (nvec <= 128) return launch_row<T, 2, 64, DROP, NORM, QUANT>(a, what, stream);
  if (nvec <= 192) return launch_row<T, 3, 64, DROP, NORM, QUANT>(a, what, stream);
  if (nvec <= 256) return launch_row<T, 4, 64, DROP, NORM, QUANT>(a, what, stream);
  if (nvec <= 512) return launch_row<T, 2, 256, DROP, NORM, QUANT>(a, what, stream);
  if (nvec <= 768) return launch_row<T, 3, 256, DROP, NORM, QUANT>(a, what, stream);
  if (nvec <= 1024) return launch_row<T, 1, 1024, DROP, NORM, QUANT>(a, what, stream);
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
  DropRule rule;
  if ((rc = check_types(what, dt, dt)) || (rc = check_drop(what, p, rng, &rule))) return rc;
  const int64_t e = dtype_size(dt);
  if (!aligned_to(x, e) || !aligned_to(residual, e) || !aligned_to(out, e) || !aligned_to(rng, 8))
    return bad_align(what);
  return rule.threshold > 0 ? launch_drop_type<true>(dt, x, residual, rows, cols, rule, rng, out, stream)
                            : launch_drop_type<false>(dt, x, residual, rows, cols, rule, rng, out, stream);
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
