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

// Bytes from one row of padded codes to the next.
static int64_t padded_k(int64_t K) { return (K + 15) / 16 * 16; }

// What of a workspace the ranges of K use at most.
constexpr int64_t kSplitBytes = (int64_t)16 << 20;

// ------------------------------------------------------------------ any shape
// Tiles of 64 TW x 64 TW outputs for rows that start and end at any byte: 16-byte loads at
// any alignment into registers, then into double-buffered LDS tiles of 128 bytes of K
// (the layout of gemm_core.hpp).  Four waves own TW x TW tiles of 32 x 32 each.
// PF stages are in flight in registers: a stage's loads take microseconds to arrive, its
// products a fraction of one.  Four ahead against one (in a graph): operands from memory 128 x 2048 x 4096
// 12.5 / 13.3 us, 777 x 1023 x 1001 9.4 / 9.1, 300 x 2049 x 640 7.6 / 6.7; from cache 12.1 / 11.8,
// 8.3 / 7.7 and 6.7 / 5.5: the depth serves long rows only.
// They are issued without a branch (a chunk past K is read as the row's last 16 bytes and
// cleared when it is put into LDS), or the compiler would have to wait for all of them.
// TINY: rows of less than 16 bytes, in one stage.
// gridDim.y > 1 (SPLIT): workgroup (t, s) takes the s-th range of stages and leaves its integer sums in
// `partial`, [range][tile][4 registers][thread], for k_i8_join.
template <int TW, bool TINY>
constexpr bool kSplits = TW == 1 && !TINY;   // larger tiles are for many of them, tiny rows are one stage

template <typename T, int TW, int PF, bool TINY>
__global__ __launch_bounds__(256) void k_i8_any(I8Args g, v4i_t* partial) {
  constexpr bool SPLIT = kSplits<TW, TINY>;
  constexpr int R = 64 * TW, TILE = R * kBK, L = R / 32;   // rows, bytes of a tile, chunks per thread
  __shared__ __attribute__((aligned(16))) uint8_t lds[4 * TILE];
  __shared__ TileScales<R, R> scales;
  const int tiles_n = (g.N + R - 1) / R;
  const int ntiles = ((g.M + R - 1) / R) * tiles_n;
  const int tile = tile_of_block(g.first + (int)blockIdx.x, ntiles);
  const int m0 = (tile / tiles_n) * R, n0 = (tile % tiles_n) * R;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wave >> 1) * 32 * TW, wn = (wave & 1) * 32 * TW;
  const int stages = (g.K + kBK - 1) / kBK;
  const int first = SPLIT ? (int)((int64_t)stages * blockIdx.y / gridDim.y) : 0;
  const int turns = SPLIT ? (int)((int64_t)stages * (blockIdx.y + 1) / gridDim.y) - first : stages;

  // thread t moves chunk t % 8 of rows t / 8 + 32 i of both tiles
  const int srow = tid >> 3, sch = tid & 7;
  const int8_t *pa[L], *pb[L];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int ra = m0 + srow + 32 * i, rb = n0 + srow + 32 * i;
    pa[i] = g.a + (int64_t)(ra < g.M ? ra : g.M - 1) * g.lda;
    pb[i] = g.b + (int64_t)(rb < g.N ? rb : g.N - 1) * g.ldb;
  }
  v4i_t ra[PF][L], rb[PF][L];
  auto load = [&](int u, int s) {
    const int k = s * kBK + sch * 16, at = k < g.K - 16 ? k : g.K - 16;
#pragma unroll
    for (int i = 0; i < L; ++i) {
      ra[u][i] = TINY ? load_chunk<true>(pa[i], k, g.K) : load16(pa[i] + at);
      rb[u][i] = TINY ? load_chunk<false>(pb[i], k, g.K) : load16(pb[i] + at);
    }
  };
  // (turns past the last of the range add nothing)
  auto put = [&](int u, int t, int buf) {
    const int s = first + t;
    if (t >= turns) {
#pragma unroll
      for (int i = 0; i < L; ++i) ra[u][i] = v4i_t{0, 0, 0, 0};
    } else if (!TINY && (s + 1) * kBK > g.K) {
      const int k = s * kBK + sch * 16, at = k < g.K - 16 ? k : g.K - 16;
#pragma unroll
      for (int i = 0; i < L; ++i) ra[u][i] = zero_first(ra[u][i], k - at);
    }
#pragma unroll
    for (int i = 0; i < L; ++i) {
      *reinterpret_cast<v4i_t*>(lds + buf * 2 * TILE + swz(srow + 32 * i, sch)) = ra[u][i];
      *reinterpret_cast<v4i_t*>(lds + buf * 2 * TILE + TILE + swz(srow + 32 * i, sch)) = rb[u][i];
    }
  };

  v16i_t acc[TW][TW];
#pragma unroll
  for (int i = 0; i < TW; ++i)
#pragma unroll
    for (int j = 0; j < TW; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
  const int frow = lane & 31, fhalf = lane >> 5;
  // turn t multiplies the range's t-th stage out of LDS, puts the next one there and loads the one
  // PF later
#pragma unroll
  for (int u = 0; u < PF; ++u) load(u, first + u);
  if (!SPLIT || gridDim.y == 1) load_scales<T>(g, scales, m0, n0, tid, 256);
  put(0, 0, 0);
  load(0, first + PF);
  __syncthreads();
  auto turn = [&](int t, int u) {   // u = (t + 1) % PF
    const uint8_t* const sA = lds + (t & 1) * 2 * TILE;
    const uint8_t* const sB = sA + TILE;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      v4i_t fa[TW], fb[TW];
#pragma unroll
      for (int i = 0; i < TW; ++i) {
        fa[i] = *reinterpret_cast<const v4i_t*>(sA + swz(wm + 32 * i + frow, ks * 2 + fhalf));
        fb[i] = *reinterpret_cast<const v4i_t*>(sB + swz(wn + 32 * i + frow, ks * 2 + fhalf));
      }
#pragma unroll
      for (int i = 0; i < TW; ++i)
#pragma unroll
        for (int j = 0; j < TW; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
    put(u, t + 1, (t + 1) & 1);
    load(u, first + t + 1 + PF);
    __syncthreads();
  };
  for (int t = 0; t < turns; t += PF)
    static_for<PF>([&](auto U) { turn(t + decltype(U)::value, (decltype(U)::value + 1) % PF); });
  if constexpr (SPLIT) {
    if (gridDim.y > 1) {
      v4i_t* const o = partial + ((int64_t)blockIdx.y * ntiles + tile) * (4 * 256) + tid;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const v16i_t& c = acc[0][0];
        o[i * 256] = v4i_t{c[4 * i], c[4 * i + 1], c[4 * i + 2], c[4 * i + 3]};
      }
      return;
    }
  }
  turn_out<T>(g, acc, lds + wave * 32 * TW * 128, scales, m0, n0, wm, wn, lane);
}

// Joins the ranges' sums of a tile of 64 x 64 and writes its outputs.
template <typename T>
__global__ __launch_bounds__(256) void k_i8_join(I8Args g, const v4i_t* partial, int ranges) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[4 * 32 * 128];
  __shared__ TileScales<64, 64> scales;
  const int tiles_n = (g.N + 63) / 64, tile = blockIdx.x;
  const int m0 = (tile / tiles_n) * 64, n0 = (tile % tiles_n) * 64;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  load_scales<T>(g, scales, m0, n0, tid, 256);
  v16i_t acc[1][1];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v4i_t sum = {};
    const v4i_t* p = partial + ((int64_t)tile * 4 + i) * 256 + tid;
#pragma unroll 4
    for (int s = 0; s < ranges; ++s, p += (int64_t)gridDim.x * (4 * 256)) sum += *p;
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[0][0][4 * i + r] = sum[r];
  }
  __syncthreads();
  turn_out<T>(g, acc, lds + wave * 32 * 128, scales, m0, n0, (wave >> 1) * 32, (wave & 1) * 32, lane);
}

template <typename T, int TW, int PF, bool TINY = false>
static int launch_any(const char* what, const I8Args& g, void* workspace, int64_t workspace_bytes,
                      hipStream_t stream) {
  const int64_t tiles = (((int64_t)g.M + 64 * TW - 1) / (64 * TW)) *
                        (((int64_t)g.N + 64 * TW - 1) / (64 * TW));
  // K in ranges of at least 4 stages, as long as there are compute units without a tile
  int64_t ranges = 1;
  if constexpr (kSplits<TW, TINY>) {
    const int64_t stages = (g.K + kBK - 1) / kBK, bytes = tiles * 64 * 64 * 4;
    ranges = std::min({stages / 4, num_cus() / tiles, std::min(workspace_bytes, kSplitBytes) / bytes,
                       (int64_t)16});
    // (the join is a launch of 2 to 3 us: 128 x 1024 x 8191 28.0 -> 14.8 us, 128 x 2048 x 4096 13.9 ->
    // 12.7, but 256 x 512 x 2048 8.6 -> 9.3)
    if (stages < 32 || ranges < 2) ranges = 1;
  }
  v4i_t* const partial = static_cast<v4i_t*>(workspace);
  const int rc = for_blocks(tiles, [&](int first, unsigned count) {
    I8Args part = g;
    part.first = first;
    hipLaunchKernelGGL((k_i8_any<T, TW, PF, TINY>), dim3(count, (unsigned)ranges), dim3(256), 0, stream,
                       part, partial);
    return check_launch(what);
  });
  if constexpr (kSplits<TW, TINY>) {
    if (rc || ranges == 1) return rc;
    hipLaunchKernelGGL((k_i8_join<T>), dim3((unsigned)tiles), dim3(256), 0, stream, g, partial,
                       (int)ranges);
    return check_launch(what);
  }
  return rc;
}

// Rows of K bytes at any alignment -> rows of ld bytes, a multiple of 16, zeros behind K.
__global__ __launch_bounds__(256) void k_pad_rows(const int8_t* src, int64_t lds_src, int K, int rows,
                                                  int8_t* dst, int64_t ld) {
  const int chunks = (int)(ld / 16);
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const int8_t* const from = src + row * lds_src;
    for (int c = blockIdx.x * 256 + threadIdx.x; c < chunks; c += gridDim.x * 256) {
      const int k = c * 16;
      v4i_t v;
      if (k + 16 <= K) {
        v = load16(from + k);
      } else {
        uint32_t w[4] = {};
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (k + j < K) w[j >> 2] |= (uint32_t)(uint8_t)from[k + j] << (8 * (j & 3));
        v = v4i_t{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
      }
      *reinterpret_cast<v4i_t*>(dst + row * ld + k) = v;
    }
  }
}

static int pad_rows(const char* what, const int8_t* src, int64_t ld_src, int K, int rows, int8_t* dst,
                    int64_t ld, hipStream_t stream) {
  const unsigned wide = (unsigned)((ld / 16 + 255) / 256);
  const unsigned tall = (unsigned)std::min<int64_t>(rows, 65535);
  hipLaunchKernelGGL(k_pad_rows, dim3(wide, tall), dim3(256), 0, stream, src, ld_src, K, rows, dst,
                     ld);
  return check_launch(what);
}

// Which tiles, from what a product with K = 4096 takes per round of workgroups (us, measured):
// 256 x 256 one workgroup per compute unit, 64; 128 x 128 two, 40 (one alone 26; with rows at any
// byte 62 and 25); 64 x 64 four, 57 (one 13, two 22).  K scales all of them alike and leaves the ranking:
// what a tile costs beside K (prologue, epilogue) is not in it, nor was it measured below K = 500 or N = 100.
struct TileCost {
  double c256, c128, c64, c128_any;
  explicit TileCost(const I8Args& g) {
    const int64_t cus = num_cus();
    auto tiles = [&](int64_t r) { return ((g.M + r - 1) / r) * ((g.N + r - 1) / r); };
    auto rounds = [&](int64_t t, int64_t per) { return (double)((t + per * cus - 1) / (per * cus)); };
    const int64_t t256 = tiles(256), t128 = tiles(128), t64 = tiles(64);
    c256 = 64.0 * rounds(t256, 1);
    c128 = t128 <= cus ? 26.0 : 40.0 * rounds(t128, 2);
    c128_any = t128 <= cus ? 25.0 : 62.0 * rounds(t128, 2);
    c64 = t64 <= cus ? 13.0 : t64 <= 2 * cus ? 22.0 : 57.0 * t64 / (4.0 * cus);
  }
};

// More than kFewTokens tokens; `padded`: the codes in g.a have zeros behind K up to a multiple of 16.
static int dispatch_i8(const char* what, fp8dp_dtype yt, I8Args g, bool padded, void* workspace,
                       int64_t workspace_bytes, hipStream_t stream) {
  if (g.M <= kFewTokens) return skinny_i8(what, yt, g, nullptr, stream);
  const TileCost cost(g);
  const double tile = std::min(cost.c256, cost.c128), any = std::min(cost.c128_any, cost.c64);
  bool aligned = rows16(g);
  if (!aligned && g.K >= 1024) {
    // copies of the operands with aligned rows, where the tiles then gain more than the
    // copies take (3 us each and 4 bytes a ns): 4096 x 4096 x 4095 125 -> 81 us, 3000 x 3000 x 1500
    // 48 -> 39.  Below K = 1024 the outputs weigh more than this reckons: 5000 x 5000 x 500 39 -> 45
    const int64_t ld = padded_k(g.K);
    const bool pad_a = !(padded && g.lda == ld && aligned16(g.a));
    const int64_t bytes_b = g.N * ld, bytes_a = pad_a ? g.M * ld : 0;
    const double copies = (pad_a ? 6.0 : 3.0) + (bytes_a + bytes_b) / 2e6;
    if (bytes_a + bytes_b <= workspace_bytes && (any - tile) * g.K / 4096.0 > copies) {
      int8_t* const to = static_cast<int8_t*>(workspace);
      int rc = pad_rows(what, g.b, g.ldb, g.K, g.N, to, ld, stream);
      if (!rc && pad_a) rc = pad_rows(what, g.a, g.lda, g.K, g.M, to + bytes_b, ld, stream);
      if (rc) return rc;
      g.b = to;
      if (pad_a) g.a = to + bytes_b;
      g.lda = g.ldb = ld;
      g.K = (int)ld;
      aligned = true;
    }
  }
  if (aligned && tile < cost.c64) return tile_i8(what, yt, g, cost.c256 <= cost.c128, stream);
  auto run = [&](auto t) -> int {
    using T = decltype(t);
    if (g.K < 16) return launch_any<T, 1, 1, true>(what, g, nullptr, 0, stream);
    if (!aligned && cost.c128_any < cost.c64)
      return launch_any<T, 2, 2>(what, g, nullptr, 0, stream);
    return launch_any<T, 1, 4>(what, g, workspace, workspace_bytes, stream);
  };
  if (yt == FP8DP_BF16) return run(bf16_t{});
  if (yt == FP8DP_F16) return run(f16_t{});
  return run(float{});
}

static int check_i8(const char* what, int64_t M, int64_t N, int64_t K, fp8dp_dtype yt,
                    fp8dp_dtype bt, const void* workspace, int64_t workspace_bytes) {
  if (M < 1 || N < 1 || K < 1 || M > (1 << 30) || N > (1 << 30) || K > FP8DP_INT8_MAX_K) {
    set_error("%s: M and N must be 1 .. 2^30 and K 1 .. %d (got %lld, %lld, %lld)", what,
              FP8DP_INT8_MAX_K, (long long)M, (long long)N, (long long)K);
    return FP8DP_EINVAL;
  }
  // (tiles of 64 x 64 then count in 32 bits)
  if (M * N > (int64_t)1 << 40) {
    set_error("%s: M * N must be at most 2^40 (got %lld, %lld)", what, (long long)M, (long long)N);
    return FP8DP_EINVAL;
  }
  if (workspace_bytes < 0 || !aligned_to(workspace, 16)) {
    set_error("%s: workspace must be 16-byte aligned, its size not negative", what);
    return FP8DP_EINVAL;
  }
  return check_types(what, yt, bt);
}

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
  return dispatch_i8(what, yt, g, false, workspace, workspace == nullptr ? 0 : workspace_bytes,
                     stream);
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
  return dispatch_i8(what, dt, g, true, static_cast<uint8_t*>(workspace) + need,
                     workspace_bytes - need, stream);
}
