// int8_gemm.hip -- y[m, n] = (sum over k of a[m, k] b[n, k]) sa[m] sb[n] + bias[n]
// for INT8 codes with one scale per token and one per output channel.
//
// The sum is exact in 32-bit integers, so the order of K is free: tiles, splits and
// instruction shapes give the same bits.  All kernels feed the matrix
// instruction with the weight as its first operand, which leaves a lane with one
// token and four consecutive channels per register group: one token scale per
// lane and stores of four outputs.
#include <hip/hip_runtime.h>

#include "int8_core.hpp"
#include "int8_skinny.hpp"
#include "int8_tile.hpp"

namespace fp8dp {

// ------------------------------------------------------------------ any shape
// 64 x 64 outputs per workgroup of 4 waves (32 x 32 each, 2 x 2 of the
// 16 x 16 x 64 instruction), K in stages of 128 bytes through registers into a
// double-buffered LDS tile.  Rows may start at any byte and end at any.
template <typename T>
__global__ __launch_bounds__(256) void k_i8_any(I8Args g) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][2][64 * kBK];
  const int tiles_n = (g.N + 63) / 64;
  const int ntiles = ((g.M + 63) / 64) * tiles_n;
  const int tile = tile_of_block(blockIdx.x, ntiles);
  const int m0 = (tile / tiles_n) * 64, n0 = (tile % tiles_n) * 64;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  const int stages = (g.K + kBK - 1) / kBK;

  // thread t moves chunk t % 8 of rows t / 8 and t / 8 + 32 of both tiles
  const int srow = tid >> 3, sch = tid & 7;
  const int8_t *pa[2], *pb[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int ra = m0 + srow + 32 * i, rb = n0 + srow + 32 * i;
    pa[i] = g.a + (int64_t)(ra < g.M ? ra : g.M - 1) * g.lda;
    pb[i] = g.b + (int64_t)(rb < g.N ? rb : g.N - 1) * g.ldb;
  }
  v4i_t ra[2], rb[2];
  auto load = [&](int s) {
    const int k = s * kBK + sch * 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ra[i] = load_chunk<true>(pa[i], k, g.K);
      rb[i] = load_chunk<false>(pb[i], k, g.K);
    }
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      *reinterpret_cast<v4i_t*>(&lds[buf][0][swz(srow + 32 * i, sch)]) = ra[i];
      *reinterpret_cast<v4i_t*>(&lds[buf][1][swz(srow + 32 * i, sch)]) = rb[i];
    }
  };

  v4i_t acc[2][2] = {};
  const int frow = lane & 15, fch = lane >> 4;
  load(0);
  put(0);
  __syncthreads();
  for (int s = 0; s < stages; ++s) {
    const int buf = s & 1;
    if (s + 1 < stages) load(s + 1);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      v4i_t fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fa[i] = *reinterpret_cast<const v4i_t*>(&lds[buf][0][swz(wm + 16 * i + frow, ks * 4 + fch)]);
        fb[i] = *reinterpret_cast<const v4i_t*>(&lds[buf][1][swz(wn + 16 * i + frow, ks * 4 + fch)]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
    if (s + 1 < stages) put(buf ^ 1);
    __syncthreads();
  }
  // a 16 x 16 tile: lane holds token lane % 16 and channels 4 (lane / 16) .. + 3
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int n = n0 + wn + 16 * j + 4 * fch;
    const RawCols4 cols = load_cols4<T>(g, n);
    float bias[4];
    widen_bias4<T>(g, cols, bias);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = m0 + wm + 16 * i + frow;
      if (m < g.M) store_out4<T>(g, m, n, g.sa[m], cols.sb, bias, acc[i][j]);
    }
  }
}

template <typename T>
static int launch_i8(const char* what, const I8Args& g, void* workspace, int64_t workspace_bytes,
                     hipStream_t stream) {
  const int64_t tiles = (((int64_t)g.M + 63) / 64) * (((int64_t)g.N + 63) / 64);
  if (tiles > 0x7FFFFFFF) {
    set_error("%s: shape too large", what);
    return FP8DP_EINVAL;
  }
  hipLaunchKernelGGL((k_i8_any<T>), dim3((unsigned)tiles), dim3(256), 0, stream, g);
  return check_launch(what);
}

static int dispatch_i8(const char* what, fp8dp_dtype yt, const I8Args& g, void* workspace,
                       int64_t workspace_bytes, hipStream_t stream) {
  if (g.M <= kFewTokens) return skinny_i8(what, yt, g, nullptr, stream);
  if (rows16(g)) return tile_i8(what, yt, g, stream);
  if (yt == FP8DP_BF16) return launch_i8<bf16_t>(what, g, workspace, workspace_bytes, stream);
  if (yt == FP8DP_F16) return launch_i8<f16_t>(what, g, workspace, workspace_bytes, stream);
  return launch_i8<float>(what, g, workspace, workspace_bytes, stream);
}

static int check_i8(const char* what, int64_t M, int64_t N, int64_t K, fp8dp_dtype yt,
                    fp8dp_dtype bt, const void* workspace, int64_t workspace_bytes) {
  if (M < 1 || N < 1 || K < 1 || M > (1 << 30) || N > (1 << 30) || K > FP8DP_INT8_MAX_K) {
    set_error("%s: M and N must be 1 .. 2^30 and K 1 .. %d (got %lld, %lld, %lld)", what,
              FP8DP_INT8_MAX_K, (long long)M, (long long)N, (long long)K);
    return FP8DP_EINVAL;
  }
  if (workspace_bytes < 0 || !aligned_to(workspace, 16)) {
    set_error("%s: workspace must be 16-byte aligned, its size not negative", what);
    return FP8DP_EINVAL;
  }
  return check_types(what, yt, bt);
}

static int64_t padded_k(int64_t K) { return (K + 15) / 16 * 16; }

// quantize_rows: row_norm.hip
int quantize_rows(const char* what, const void* x, int64_t rows, int64_t cols, fp8dp_dtype dt,
                  int8_t* q, int64_t ldq, float* scale, hipStream_t stream);

}  // namespace fp8dp

using namespace fp8dp;

extern "C" int int8_gemm(const int8_t* a, const int8_t* b, int64_t M, int64_t N, int64_t K,
                         const float* a_scale, const float* b_scale, const void* bias,
                         fp8dp_dtype yt, fp8dp_dtype bt, void* y, void* workspace,
                         int64_t workspace_bytes, hipStream_t stream) {
  const char* what = "int8_gemm";
  const int rc = check_i8(what, M, N, K, yt, bt, workspace, workspace_bytes);
  if (rc) return rc;
  if (a == nullptr || b == nullptr || a_scale == nullptr || b_scale == nullptr || y == nullptr) {
    set_error("%s: NULL pointer argument", what);
    return FP8DP_EINVAL;
  }
  if (!aligned_to(a_scale, 4) || !aligned_to(b_scale, 4) || !aligned_to(y, dtype_size(yt)) ||
      !aligned_to(bias, dtype_size(bt)))
    return bad_align(what);
  const I8Args g = {a,  b,       (int)M,  (int)N, (int)K, K, K, a_scale,
                    b_scale, bias, bt == FP8DP_F32, y};
  return dispatch_i8(what, yt, g, workspace, workspace == nullptr ? 0 : workspace_bytes, stream);
}

extern "C" int64_t int8_linear_workspace(int64_t M, int64_t K) {
  if (M < 1 || K < 1) return 0;
  return M * padded_k(K) + (4 * M + 15) / 16 * 16;
}

extern "C" int int8_linear(const void* x, const int8_t* w8, const float* w_scale, const void* bias,
                           int64_t M, int64_t N, int64_t K, fp8dp_dtype dt, fp8dp_dtype bt, void* y,
                           void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  const char* what = "int8_linear";
  int rc = check_i8(what, M, N, K, dt, bt, workspace, workspace_bytes);
  if (rc) return rc;
  if (x == nullptr || w8 == nullptr || w_scale == nullptr || y == nullptr || workspace == nullptr) {
    set_error("%s: NULL pointer argument", what);
    return FP8DP_EINVAL;
  }
  const int64_t need = int8_linear_workspace(M, K);
  if (workspace_bytes < need) {
    set_error("%s: workspace needs %lld bytes, got %lld", what, (long long)need,
              (long long)workspace_bytes);
    return FP8DP_EINVAL;
  }
  if (!aligned_to(x, dtype_size(dt)) || !aligned_to(w_scale, 4) || !aligned_to(y, dtype_size(dt)) ||
      !aligned_to(bias, dtype_size(bt)))
    return bad_align(what);
  I8Args g = {nullptr, w8, (int)M, (int)N, (int)K, K, K, nullptr, w_scale, bias, bt == FP8DP_F32, y};
  if (skinny_casts(g, x, (int)dtype_size(dt))) return skinny_i8(what, dt, g, x, stream);
  const int64_t ld = padded_k(K);
  int8_t* const q = static_cast<int8_t*>(workspace);
  float* const scale = reinterpret_cast<float*>(q + M * ld);
  rc = quantize_rows(what, x, M, K, dt, q, ld, scale, stream);
  if (rc) return rc;
  g.a = q;
  g.lda = ld;
  g.sa = scale;
  return dispatch_i8(what, dt, g, static_cast<uint8_t*>(workspace) + need, workspace_bytes - need,
                     stream);
}
