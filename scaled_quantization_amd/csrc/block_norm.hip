// block_norm.hip -- the norms after a block and before the next one, with the block's gate and the
// residual sum between them, in one pass over the rows.
//
//   post_rstd = 1 / sqrt(mean(x^2) + eps),  z = a residual + b gate x post_rstd post_weight
//   pre_rstd = 1 / sqrt(mean(z^2) + eps),   y = z pre_rstd pre_weight
//
// A row of 8 to 16384 elements stays in registers from its one read to its outputs: a wave per row
// up to 2048 elements, a workgroup above; other rows are read again by each step.  A gate per
// channel is folded into the weight behind the first norm once per wave, so it costs a row nothing.
// The second norm reads z as stored, so that the backward pass agrees with it.
// Bound by memory: 16384 x 768 18 us (5.6 TB/s; floor 15), 16384 x 4096 101 us (5.3 TB/s); the norm alone 9.2 and 48.
// Binary32 rows, read and stored as two halves of 16 bytes a lane: 8192 x 2048 62 us (4.3 TB/s).
#include <hip/hip_runtime.h>

#include "row_core.hpp"

namespace fp8dp {

struct BlockNormArgs {
  const void *x, *residual, *post, *gate, *pre;
  int64_t rows;
  int cols;
  bool wf32, gate_f32;
  float a, b, eps;
  void *z, *y;
  float *post_rstd, *pre_rstd;
};

// Weight behind the first norm with what else is the same for all rows: b gate post.
template <typename T, bool TOKEN>
__device__ __forceinline__ void load_branch8(const BlockNormArgs& a, int64_t c, int n, float w[8]) {
  load_param8<T>(a.post, a.wf32, c, n, 1.0f, w);
  float g[8];
  load_param8<T>(TOKEN ? nullptr : a.gate, a.gate_f32, c, n, 1.0f, g);
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] *= a.b * g[j];
}

// TOKEN: a gate per token and channel.  BRANCH: there is an x (else z is the residual as it is).
template <typename T, int NV, int THR, bool TOKEN, bool BRANCH>
__global__ __launch_bounds__(THR == 64 ? 256 : THR) void k_block_norm(BlockNormArgs a) {
  constexpr int RPB = THR == 64 ? 4 : 1;
  constexpr int WAVES = THR / 64;
  __shared__ float scratch[THR > 64 ? 2 * 2 * WAVES : 1];
  const int t = THR > 64 ? (int)threadIdx.x : (int)(threadIdx.x & 63);
  const int sub = THR > 64 ? 0 : (int)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cols = a.cols;
  const bool ragged = cols % 8 != 0;
  const float inv_cols = 1.0f / (float)cols;
  const T *const x = static_cast<const T*>(a.x), *const residual = static_cast<const T*>(a.residual),
          *const gate = static_cast<const T*>(a.gate);
  auto column = [&](int i) { return (i * THR + t) * 8; };
  const int n_last = cols - column(NV - 1);
  auto count = [&](int i) { return i < NV - 1 ? 8 : n_last; };
  const Mask8 mask(n_last);

  struct Row {
    Raw8<T> x[BRANCH ? NV : 1], r[NV], g[TOKEN ? NV : 1];
  };
  auto load = [&](int64_t row, Row& o) {
    const int64_t base = row * cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (BRANCH) o.x[i] = load_row(x + base, column(i), cols);
      o.r[i] = load_row(residual + base, column(i), cols);
      if constexpr (TOKEN) o.g[i] = load_row(gate + base, column(i), cols);
    }
  };
  auto widen = [&](Raw8<T> raw, int i, float v[8]) {
    if (i == NV - 1) {
      settle(raw, n_last, ragged);
      mask.clear_empty(raw);
    }
    widen8f(raw, v);
  };
  const int64_t step = (int64_t)gridDim.x * RPB, begin = (int64_t)blockIdx.x * RPB + sub;
  if (begin >= a.rows) return;   // (whole waves, or with THR > 64 whole workgroups)
  Row next;
  load(begin, next);

  float w[BRANCH ? NV : 1][8], p[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (BRANCH) load_branch8<T, TOKEN>(a, column(i), count(i), w[i]);
    load_param8<T>(a.pre, a.wf32, column(i), count(i), 1.0f, p[i]);
  }

  int turn = 0;
  for (int64_t row = begin; row < a.rows; row += step, turn ^= 1) {
    float* const sc = scratch + (THR > 64 ? turn * 2 * WAVES : 0);
    const int64_t base = row * cols;
    const Row now = next;
    load(row + step < a.rows ? row + step : row, next);

    float v[NV][8], rstd = 0.0f;
    if constexpr (BRANCH) {
      float sq = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        widen(now.x[i], i, v[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) sq = __builtin_fmaf(v[i][j], v[i][j], sq);
      }
      rstd = rsqrtf(row_sum<THR>(sq, sc) * inv_cols + a.eps);
      if (t == 0 && a.post_rstd != nullptr) a.post_rstd[row] = rstd;
    }
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float r[8];
      widen(now.r[i], i, r);
      if constexpr (BRANCH) {
        float g[8];
        if constexpr (TOKEN) widen(now.g[i], i, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float u = v[i][j] * rstd * w[i][j];
          if constexpr (TOKEN) u *= g[j];
          v[i][j] = __builtin_fmaf(a.a, r[j], u);
        }
        if (i == NV - 1) mask.clear(v[i]);   // (0 times a weight that is not there)
        const Raw8<T> out = round8(v[i], T{});
        store_row(element(static_cast<T*>(a.z) + base, column(i)), count(i), out);
        widen8f(out, v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = r[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sq = __builtin_fmaf(v[i][j], v[i][j], sq);
    }
    if (a.y == nullptr) continue;
    rstd = rsqrtf(row_sum<THR>(sq, sc + WAVES) * inv_cols + a.eps);
    if (t == 0 && a.pre_rstd != nullptr) a.pre_rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= rstd * p[i][j];
      store_row(element(static_cast<T*>(a.y) + base, column(i)), count(i), round8(v[i], T{}));
    }
  }
}

// Rows of more than 16384 elements, or less than 8: read again by each step.
template <typename T, int THR, bool TOKEN, bool BRANCH>
__global__ __launch_bounds__(THR == 64 ? 256 : THR) void k_block_norm_loop(BlockNormArgs a) {
  constexpr int RPB = THR == 64 ? 4 : 1;
  constexpr int WAVES = THR / 64;
  __shared__ float scratch[THR > 64 ? 2 * 2 * WAVES : 1];
  const int t = THR > 64 ? (int)threadIdx.x : (int)(threadIdx.x & 63);
  const int sub = THR > 64 ? 0 : (int)(threadIdx.x >> 6);
  const int cols = a.cols;
  const float inv_cols = 1.0f / (float)cols;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPB + sub; row < a.rows;
       row += (int64_t)gridDim.x * RPB, turn ^= 1) {
    float* const sc = scratch + (THR > 64 ? turn * 2 * WAVES : 0);
    const int64_t base = row * cols;
    const T* const residual = static_cast<const T*>(a.residual) + base;
    const T* const again = BRANCH ? static_cast<const T*>(a.z) + base : residual;
    float v[8], rstd = 0.0f;
    auto square = [&]() {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= v[j];
    };
    LongSum sq;
    if constexpr (BRANCH) {
      const T* const x = static_cast<const T*>(a.x) + base;
      for (int c = t * 8; c < cols; c += THR * 8) {
        load8(x + c, cols - c, v);
        square();
        sq.add(sum8(v));
      }
      rstd = rsqrtf(row_sum<THR>(sq.total(), sc) * inv_cols + a.eps);
      if (t == 0 && a.post_rstd != nullptr) a.post_rstd[row] = rstd;
      sq = LongSum{};
      for (int c = t * 8; c < cols; c += THR * 8) {
        const int n = cols - c;
        float r[8], w[8], g[8];
        load8(x + c, n, v);
        load8(residual + c, n, r);
        load_branch8<T, TOKEN>(a, c, n, w);
        if constexpr (TOKEN) load8(static_cast<const T*>(a.gate) + base + c, n, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float u = v[j] * rstd * w[j];
          if constexpr (TOKEN) u *= g[j];
          v[j] = __builtin_fmaf(a.a, r[j], u);
        }
        through8<T>(v);
        store8(static_cast<T*>(a.z) + base + c, n, v);
        zero_from8(n, v);
        square();
        sq.add(sum8(v));
      }
    } else {
      for (int c = t * 8; c < cols; c += THR * 8) {
        load8(residual + c, cols - c, v);
        square();
        sq.add(sum8(v));
      }
    }
    if (a.y == nullptr) continue;
    rstd = rsqrtf(row_sum<THR>(sq.total(), sc + WAVES) * inv_cols + a.eps);
    if (t == 0 && a.pre_rstd != nullptr) a.pre_rstd[row] = rstd;
    for (int c = t * 8; c < cols; c += THR * 8) {
      float p[8];
      load8(again + c, cols - c, v);
      load_param8<T>(a.pre, a.wf32, c, cols - c, 1.0f, p);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= rstd * p[j];
      store8(static_cast<T*>(a.y) + base + c, cols - c, v);
    }
  }
}

template <typename T, int NV, int THR, bool TOKEN, bool BRANCH>
static int launch_block(const BlockNormArgs& a, hipStream_t stream) {
  constexpr int RPB = THR == 64 ? 4 : 1, BLOCK = THR == 64 ? 256 : THR;
  const int64_t need = (a.rows + RPB - 1) / RPB;
  // 16 waves per compute unit walk the rows (256 short-lived ones take the same time on streams from memory: 16384 x 4096 102
  // us against 101, with a gate per token 129 / 127)
  const unsigned grid = grid_for(need * BLOCK, BLOCK, std::max(1, 16 * 64 / BLOCK));
  if constexpr (NV > 0)
    hipLaunchKernelGGL((k_block_norm<T, NV, THR, TOKEN, BRANCH>), dim3(grid), dim3(BLOCK), 0, stream, a);
  else
    hipLaunchKernelGGL((k_block_norm_loop<T, THR, TOKEN, BRANCH>), dim3(grid), dim3(BLOCK), 0, stream, a);
  return check_launch("block_norm");
}

template <typename T, bool TOKEN, bool BRANCH>
static int launch_width(const BlockNormArgs& a, hipStream_t stream) {
  const int nvec = (a.cols + 7) / 8;
  if (a.cols < 8) return launch_block<T, 0, 64, TOKEN, BRANCH>(a, stream);
  if (nvec <= 64) return launch_block<T, 1, 64, TOKEN, BRANCH>(a, stream);
  if (nvec <= 128) return launch_block<T, 2, 64, TOKEN, BRANCH>(a, stream);
  // (all vectors of a thread but the last are whole)
  if (nvec <= 192) return launch_block<T, 3, 64, TOKEN, BRANCH>(a, stream);
  if (nvec <= 256) return launch_block<T, 4, 64, TOKEN, BRANCH>(a, stream);
  if (nvec <= 512) return launch_block<T, 2, 256, TOKEN, BRANCH>(a, stream);
  if (nvec <= 1024) return launch_block<T, 1, 1024, TOKEN, BRANCH>(a, stream);
  if (nvec <= 2048) return launch_block<T, 2, 1024, TOKEN, BRANCH>(a, stream);
  return launch_block<T, 0, 1024, TOKEN, BRANCH>(a, stream);
}

template <typename T>
static int launch_kind(const BlockNormArgs& a, bool token, hipStream_t stream) {
  if (a.x == nullptr) return launch_width<T, false, false>(a, stream);
  return token ? launch_width<T, true, true>(a, stream) : launch_width<T, false, true>(a, stream);
}

}  // namespace fp8dp

using namespace fp8dp;

extern "C" int block_norm(const void* x, const void* residual, const void* post_weight,
                          const void* gate, int32_t gate_per_token, const void* pre_weight,
                          int64_t rows, int64_t cols, fp8dp_dtype dt, fp8dp_dtype wt,
                          fp8dp_dtype gt, float residual_scale, float branch_scale, float eps,
                          void* z, void* y, float* post_rstd, float* pre_rstd, hipStream_t stream) {
  const char* what = "block_norm";
  int rc = check_rows(what, rows, cols);   // first: an empty tensor has no address
  if (rc) return rc;
  if (residual == nullptr || (x == nullptr) != (z == nullptr) || (x == nullptr && y == nullptr)) {
    set_error("%s: residual must be non-NULL, x and z go together, and one of z and y is written", what);
    return FP8DP_EINVAL;
  }
  if (x == nullptr && (post_weight != nullptr || gate != nullptr || post_rstd != nullptr)) {
    set_error("%s: post_weight, gate and post_rstd belong to x", what);
    return FP8DP_EINVAL;
  }
  if (y == nullptr && pre_rstd != nullptr) {
    set_error("%s: pre_rstd belongs to y", what);
    return FP8DP_EINVAL;
  }
  const bool token = gate != nullptr && gate_per_token != 0;
  if ((rc = check_types(what, dt, wt)) || (rc = check_types(what, dt, gt))) return rc;
  if (token && gt != dt) {
    set_error("%s: a gate per token has the activations' type", what);
    return FP8DP_EINVAL;
  }
  const float top = 3.402823466e38f;
  if (!(eps >= 0.0f && eps <= top) || !(std::fabs(residual_scale) <= top) ||
      !(std::fabs(branch_scale) <= top)) {
    set_error("%s: eps must not be negative, and eps and the scales finite", what);
    return FP8DP_EINVAL;
  }
  const int64_t e = dtype_size(dt), we = dtype_size(wt);
  if (!aligned_to(x, e) || !aligned_to(residual, e) || !aligned_to(z, e) || !aligned_to(y, e) ||
      !aligned_to(post_weight, we) || !aligned_to(pre_weight, we) ||
      !aligned_to(gate, dtype_size(gt)) || !aligned_to(post_rstd, 4) || !aligned_to(pre_rstd, 4))
    return bad_align(what);
  if (shared_buffers({y, post_rstd, pre_rstd}, {z, x, residual, gate, post_weight, pre_weight}) ||
      shared_buffers({z}, {token ? nullptr : gate, post_weight, pre_weight})) {
    set_error("%s: y and the statistics must not be z, an input or each other, nor z a parameter", what);
    return FP8DP_EINVAL;
  }
  BlockNormArgs a = {};
  a.x = x;
  a.residual = residual;
  a.post = post_weight;
  a.gate = gate;
  a.pre = pre_weight;
  a.rows = rows;
  a.cols = (int)cols;
  a.wf32 = wt == FP8DP_F32;
  a.gate_f32 = gt == FP8DP_F32;
  a.a = residual_scale;
  a.b = branch_scale;
  a.eps = eps;
  a.z = z;
  a.y = y;
  a.post_rstd = post_rstd;
  a.pre_rstd = pre_rstd;
  if (dt == FP8DP_BF16) return launch_kind<bf16_t>(a, token, stream);
  if (dt == FP8DP_F16) return launch_kind<f16_t>(a, token, stream);
  return launch_kind<float>(a, token, stream);
}
