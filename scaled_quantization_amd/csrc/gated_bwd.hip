// gated_bwd.hip -- gradients of the gated linear layer.
//
//   (x and the weights copied to aligned rows where K is no multiple of 8)
//   dg = dh u f'(g), du = dh f(g)          one pass, D = [dg | du] of the operands' type
//   dx = dg Wg + du Wu = D [Wg; Wu]        contraction over the channels, W lies down
//   [dWg; dWu] = D^T x                     contraction over the tokens, both operands lie down
//
// D is in the workspace: rows of 2 Np values, Np = N to a multiple of 64, and as many rows as M to a
// multiple of 64; what pads it is zeros, so that every stage of K is whole on D's side.  Rounding
// dg and du to 16 bits, as the matrix instructions take them, is off by half a step of the type per term;
// the products sum them in binary32.  (One pass forms dg and du for both products: formed
// in the products' loads they would be computed once per tile of K, 4 times each at the size below.)
//
// In float16 dg and du may leave the type's range where the gradients do not.  The pass that forms them leaves the largest
// finite magnitude of each workgroup; a kernel behind it looks at these, and where the largest of all is outside [2^-6,
// 2^15] forms dg and du again times a power of two, which the products' outputs take back.  (In that range the smallest
// step of the type, half of it 2^-25, is 2^-19 of the largest or less: gradients whose typical value is 2^-5 of their
// largest keep 2^-14.)
//
// 16384 x 2048 x 768: the pass over dh, gate and up 50 us (6.7 TB/s), dx 104, the weights' 105 and 10 for their join: 206
// GFLOP in two products, 0.99 PFLOP/s, whose waves wait for their operands half of the time.
#include "gated_core.hpp"
#include "pad16.hpp"

namespace fp8dp {

struct GradArgs {
  const void *dh, *gate, *up;
  int M, N, Np, act;
  uint32_t rows;
  void* d;
};
// Calls f(dg, du, where they go) for each of this thread's vectors; `threads` of a workgroup.
template <typename T, typename F>
__device__ __forceinline__ void gate_grad(const GradArgs& a, uint32_t threads, F&& f) {
  const T *const dh = static_cast<const T*>(a.dh), *const gate = static_cast<const T*>(a.gate),
          *const up = static_cast<const T*>(a.up);
  const uint32_t nvec = (uint32_t)a.Np / 8;
  const uint64_t total = (uint64_t)a.rows * nvec, step = (uint64_t)gridDim.x * threads;
  for (uint64_t at = (uint64_t)blockIdx.x * threads + threadIdx.x; at < total; at += step) {
    const uint32_t row = total >> 32 ? (uint32_t)(at / nvec) : (uint32_t)at / nvec;
    const int c = (int)((uint32_t)(at - (uint64_t)row * nvec) * 8);
    const int n = (int)row < a.M ? a.N - c : 0;
    const int64_t from = (int64_t)row * a.N + c;
    const Raw8<T> rd = load_raw(dh + from, n), rg = load_raw(gate + from, n), ru = load_raw(up + from, n);
    float vd[8], g[8], u[8];
    widen8f(rd, vd);
    widen8f(rg, g);
    widen8f(ru, u);
    with_act(a.act, [&](auto ACT) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float slope;
        const float f = gate_of<decltype(ACT)::value, true>(g[j], &slope);
        g[j] = vd[j] * u[j] * slope;
        u[j] = vd[j] * f;
      }
    });
    f(g, u, static_cast<T*>(a.d) + (int64_t)row * 2 * a.Np + c);
  }
}
template <typename T>
__device__ __forceinline__ void store_grad(const float g[8], const float u[8], int Np, T* to) {
  const Raw8<T> dg = round8(g, T{}), du = round8(u, T{});
  *reinterpret_cast<u32x4_t*>(to) = u32x4_t{dg.w[0], dg.w[1], dg.w[2], dg.w[3]};
  *reinterpret_cast<u32x4_t*>(to + Np) = u32x4_t{du.w[0], du.w[1], du.w[2], du.w[3]};
}

// In float16 also tops[workgroup]: the bits of its largest finite magnitude.
template <typename T>
__global__ __launch_bounds__(256) void k_gate_grad(GradArgs a, uint32_t* tops) {
  float top = 0.0f;
  gate_grad<T>(a, 256, [&](const float g[8], const float u[8], T* to) {
    store_grad(g, u, a.Np, to);
    if constexpr (std::is_same<T, f16_t>::value) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float vg = __builtin_fabsf(g[j]), vu = __builtin_fabsf(u[j]);
        top = vg > top && vg < INFINITY ? vg : top;   // (a NaN is not larger)
        top = vu > top && vu < INFINITY ? vu : top;
      }
    }
  });
  if constexpr (std::is_same<T, f16_t>::value) {
    __shared__ uint32_t scratch[4];
    const uint32_t most = row_umax<256>(__float_as_uint(top), scratch);
    if (threadIdx.x == 0) tops[blockIdx.x] = most;
  }
}

// Float16: *back = what the products' outputs are multiplied with; dg and du once more where that is not 1.
constexpr int kGradTops = 4096;   // most workgroups of the pass before
static __global__ __launch_bounds__(1024) void k_gate_grad_again(GradArgs a, const uint32_t* tops, int n, float* back) {
  __shared__ uint32_t scratch[16];
  uint32_t top = 0;
  for (int i = threadIdx.x; i < n; i += 1024) top = tops[i] > top ? tops[i] : top;
  top = row_umax<1024>(top, scratch);
  const int e = (int)(top >> 23);   // (of a binary32 from 2^(e - 127) on; at most 2^49, what three float16 can reach)
  const int shift = top == 0 || (e >= 127 - 6 && e < 127 + 15) ? 0 : std::min(127 + 14 - e, 100);
  if (blockIdx.x == 0 && threadIdx.x == 0) *back = __uint_as_float((uint32_t)(127 - shift) << 23);
  if (shift == 0) return;
  const float by = __uint_as_float((uint32_t)(127 + shift) << 23);
  gate_grad<f16_t>(a, 1024, [&](float g[8], float u[8], f16_t* to) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[j] *= by;
      u[j] *= by;
    }
    store_grad(g, u, a.Np, to);
  });
}

// Rows m of a product in one piece or two: row m of piece m / seg at y[piece] + (m % seg) N, of
// which `valid` are stored.
template <typename T>
struct Rows2 {
  T *y0, *y1;
  int seg, valid, N;
  const float* back;   // what float16 outputs are multiplied with, a power of two
  __device__ __forceinline__ float back_of() const { return std::is_same<T, f16_t>::value ? *back : 1.0f; }
  __device__ __forceinline__ float scaled(float v, float by) const { return std::is_same<T, f16_t>::value ? v * by : v; }
  __device__ __forceinline__ T* at(int m) const {
    const bool second = m >= seg;
    const int r = second ? m - seg : m;
    if (r >= valid || (second && y1 == nullptr)) return nullptr;
    return (second ? y1 : y0) + (int64_t)r * N;
  }
};

template <typename T, int TM, int TN>
struct PlainOut {
  Rows2<T> rows;
  __device__ __forceinline__ void operator()(const v4f_t (&acc)[TM][TN], uint8_t* part, int m, int n,
                                             int lane, int) const {
    const float back = rows.back_of();
#pragma unroll
    for (int i0 = 0; i0 < TM; i0 += 2)
      static_for<(TN + 3) / 4>([&](auto P) {
        constexpr int j0 = 4 * decltype(P)::value;
        turn16<T, (TN - j0 > 2 ? 2 : 1)>(
            part, lane, [&](int i, int j, int r) { return rows.scaled(acc[i0 + i][j0 + j][r], back); },
            [&](int r, int c, const Raw8<T>& v) {
              T* const y = rows.at(m + 16 * i0 + r);
              const int col = n + 16 * j0 + c, left = rows.N - col;
              if (y != nullptr && left > 0) store_row(y + col, left, v);
            });
      });
  }
};

// Sums of a range of K: parts[split][m][N].
template <int TM, int TN>
struct PlainParts {
  float* parts;
  int M, N;
  __device__ __forceinline__ void operator()(const v4f_t (&acc)[TM][TN], uint8_t* part, int m, int n,
                                             int lane, int split) const {
    float* const to = parts + (int64_t)split * M * N;
#pragma unroll
    for (int i0 = 0; i0 < TM; i0 += 2)
#pragma unroll
      for (int j0 = 0; j0 < TN; j0 += 2)
        turn32(
            part, lane, [&](int i, int j) { return acc[i0 + i][j0 + j]; },
            [&](int r, int c, const Raw8<float>& v) {
              const int row = m + 16 * i0 + r, col = n + 16 * j0 + c, left = N - col;
              if (row < M && left > 0) store_row(to + (int64_t)row * N + col, left, v);
            });
  }
};

template <typename T>
__global__ __launch_bounds__(256) void k_plain_join(const float* parts, int splits, int M, Rows2<T> rows) {
  const uint32_t nvec = ((uint32_t)rows.N + 7) / 8;
  const uint64_t total = (uint64_t)M * nvec, step = (uint64_t)gridDim.x * 256;
  const float back = rows.back_of();
  for (uint64_t at = (uint64_t)blockIdx.x * 256 + threadIdx.x; at < total; at += step) {
    const uint32_t row = total >> 32 ? (uint32_t)(at / nvec) : (uint32_t)at / nvec;
    const int c = (int)((uint32_t)(at - (uint64_t)row * nvec) * 8), n = rows.N - c;
    T* const y = rows.at((int)row);
    if (y == nullptr) continue;
    float sum[8] = {};
    for (int s = 0; s < splits; ++s) {
      float v[8];
      load8(parts + ((int64_t)s * M + row) * rows.N + c, n, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += v[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] = rows.scaled(sum[j], back);
    store8(y + c, n, sum);
  }
}

template <typename T, int WM, int WN, int TM, int TN, int S, bool ADOWN, bool DIRECT>
static int launch_plain(const char* what, MmaArgs g, int m, int splits, Rows2<T> rows, float* parts,
                        hipStream_t stream) {
  g.tiles_m = (m + WM * TM * 16 - 1) / (WM * TM * 16);
  g.tiles_n = (rows.N + WN * TN * 16 - 1) / (WN * TN * 16);
  g.splits = splits;
  return for_work<DIRECT>((int64_t)g.tiles_m * g.tiles_n * splits, WM * WN == 8 || S > 2 ? 1 : 2, [&](int first, unsigned count) {
    g.first = first;
    const dim3 grid(count), block(64 * WM * WN);
    if (splits > 1) {
      const PlainParts<TM, TN> out = {parts, m, rows.N};
      hipLaunchKernelGGL((k_mma<T, WM, WN, TM, TN, S, ADOWN, true, false, DIRECT, PlainParts<TM, TN>>), grid,
                         block, 0, stream, g, out);
    } else {
      const PlainOut<T, TM, TN> out = {rows};
      hipLaunchKernelGGL((k_mma<T, WM, WN, TM, TN, S, ADOWN, true, false, DIRECT, PlainOut<T, TM, TN>>), grid,
                         block, 0, stream, g, out);
    }
    return check_launch(what);
  });
}

// m rows of outputs, of which `rows` says where they go; B lies down.
template <typename T, bool ADOWN>
static int run_product(const char* what, const MmaArgs& g, int m, const ProductPlan& p, Rows2<T> rows,
                       float* parts, hipStream_t stream) {
  int rc;
  if (p.shape == kTile256) rc = launch_plain<T, 4, 2, 4, 8, 2, ADOWN, true>(what, g, m, p.splits, rows, parts, stream);
  else if (p.shape == kTile192) rc = launch_plain<T, 4, 2, 4, 6, 2, ADOWN, true>(what, g, m, p.splits, rows, parts, stream);
  else if (p.shape == kTile128 && tiles_of(kTile128, m, rows.N) * p.splits <= num_cus())
    rc = launch_plain<T, 2, 2, 4, 4, 4, ADOWN, true>(what, g, m, p.splits, rows, parts, stream);
  else if (p.shape == kTile128) rc = launch_plain<T, 2, 2, 4, 4, 2, ADOWN, true>(what, g, m, p.splits, rows, parts, stream);
  else rc = launch_plain<T, 2, 2, 4, 4, 2, ADOWN, false>(what, g, m, p.splits, rows, parts, stream);
  if (rc || p.splits == 1) return rc;
  const int64_t nvec = ((int64_t)rows.N + 7) / 8;
  hipLaunchKernelGGL((k_plain_join<T>), dim3(grid_for(m * nvec, 256, 16)), dim3(256), 0, stream, parts, p.splits,
                     m, rows);
  return check_launch(what);
}

// What the workspace holds behind copies of operands: D, the largest magnitudes and `back`, sums of ranges of K.
constexpr int64_t kTopsBytes = (kGradTops + 64) * 4;   // (whole cache lines: sums that start amid one cost 25 us in 16384 x 2048 x 768)
struct BwdSizes {
  int64_t Mp, Np, d_bytes;
  ProductPlan dx, dw;
  BwdSizes(int64_t M, int64_t N, int64_t K, bool direct)
      : Mp(round_up(M, kStageK)), Np(round_up(N, kStageK)), d_bytes(Mp * 2 * Np * 2),
        dx(plan_product(M, K, 2 * Np / kStageK, false, direct)),
        dw(plan_product(2 * Np, K, Mp / kStageK, false, direct)) {}
  int64_t parts_bytes(int64_t M, int64_t K) const {
    return std::max<int64_t>(dx.splits > 1 ? dx.splits * M * K * 4 : 0,
                             dw.splits > 1 ? dw.splits * 2 * Np * K * 4 : 0);
  }
};

template <typename T>
static int run_gated_bwd(const char* what, const T* dh, const T* gate, const T* up, const T* x, const T* wg,
                         const T* wu, int M, int N, int K, int act, T* dx, T* dwg, T* dwu, void* workspace,
                         hipStream_t stream) {
  auto words = [](const T* p) { return reinterpret_cast<const uint16_t*>(p); };
  Operand w = {{words(wg), words(wu)}, K, K}, xs = {{words(x), words(x)}, K, K};
  bool direct_w = rows16(w, K), direct_x = rows16(xs, K);
  if (pad_pays(M, N, K, true)) {   // (columns of zeros behind K are multiplied and not stored)
    uint16_t* const to = static_cast<uint16_t*>(workspace);
    const int rc = pad_operands(what, xs.p[0], w.p[0], w.p[1], M, N, K, to, stream);
    if (rc) return rc;
    const int64_t ld = pad_ld(K);
    xs = {{to, to}, ld, (int)ld};
    w = {{to + M * ld, to + (M + N) * ld}, ld, (int)ld};
    direct_w = direct_x = true;
    workspace = static_cast<uint8_t*>(workspace) + pad_bytes(M, N, K);
  }
  const BwdSizes sw(M, N, K, direct_w), sx(M, N, K, direct_x);
  const int Np = (int)sw.Np, Mp = (int)sw.Mp;
  T* const d = static_cast<T*>(workspace);
  uint32_t* const tops = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + sw.d_bytes);
  float* const back = reinterpret_cast<float*>(tops + kGradTops);
  float* const parts = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(tops) + kTopsBytes);
  const int64_t vecs = (int64_t)Mp * (Np / 8);
  const GradArgs grad = {dh, gate, up, M, N, Np, act, (uint32_t)Mp, d};
  constexpr bool narrow = std::is_same<T, f16_t>::value;
  const unsigned grid = narrow ? std::min<unsigned>(grid_for(vecs, 256, 16), kGradTops) : grid_for(vecs, 256, 1024);
  hipLaunchKernelGGL((k_gate_grad<T>), dim3(grid), dim3(256), 0, stream, grad, tops);
  int rc = check_launch(what);
  if (rc) return rc;
  if constexpr (narrow) {
    hipLaunchKernelGGL(k_gate_grad_again, dim3(grid_for(vecs, 1024, 1)), dim3(1024), 0, stream, grad, tops, (int)grid,
                       back);
    if ((rc = check_launch(what))) return rc;
  }
  if (dx != nullptr) {
    MmaArgs g = {};
    g.a = {{words(d), words(d) + Np}, 2 * (int64_t)Np, M};
    g.b = w;
    g.seg_stages = Np / kStageK;
    g.stages = 2 * g.seg_stages;
    g.valid_a = Np;
    g.valid_b = N;
    const Rows2<T> rows = {dx, nullptr, M, M, K, back};
    if ((rc = run_product<T, false>(what, g, M, sw.dx, rows, parts, stream))) return rc;
  }
  if (dwg != nullptr) {
    MmaArgs g = {};
    g.a = {{words(d), words(d)}, 2 * (int64_t)Np, 2 * Np};
    g.b = xs;
    g.stages = g.seg_stages = Mp / kStageK;
    g.valid_a = Mp;
    g.valid_b = M;
    const Rows2<T> rows = {dwg, dwu, Np, N, K, back};
    if ((rc = run_product<T, true>(what, g, 2 * Np, sx.dw, rows, parts, stream))) return rc;
  }
  return FP8DP_OK;
}

}  // namespace fp8dp

using namespace fp8dp;

extern "C" int64_t gated_linear_backward_workspace(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || N < 1 || K < 1 || M > FP8DP_GATED_MAX_ROWS || N > FP8DP_GATED_MAX_WIDTH ||
      K > FP8DP_GATED_MAX_WIDTH)
    return 0;
  const BwdSizes d(M, N, K, true), a(M, N, K, false);
  return (pad_pays(M, N, K, true) ? pad_bytes(M, N, K) : 0) + d.d_bytes + kTopsBytes +
         std::max(d.parts_bytes(M, K), a.parts_bytes(M, K));
}

extern "C" int gated_linear_backward(const void* dh, const void* gate, const void* up, const void* x,
                                     const void* w_gate, const void* w_up, int64_t M, int64_t N, int64_t K,
                                     fp8dp_dtype dt, fp8dp_gate act, void* dx, void* dw_gate, void* dw_up,
                                     void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  const char* what = "gated_linear_backward";
  const int rc = check_gated(what, M, N, K, dt, act, workspace, workspace_bytes);
  if (rc) return rc;
  if (dh == nullptr || gate == nullptr || up == nullptr || x == nullptr || w_gate == nullptr ||
      w_up == nullptr || workspace == nullptr) {
    set_error("%s: dh, gate, up, x, w_gate, w_up and workspace must be non-NULL", what);
    return FP8DP_EINVAL;
  }
  if ((dw_gate == nullptr) != (dw_up == nullptr) || (dw_gate == nullptr && dx == nullptr)) {
    set_error("%s: dw_gate and dw_up go together, and dx or they are computed", what);
    return FP8DP_EINVAL;
  }
  const int64_t need = gated_linear_backward_workspace(M, N, K);
  if (workspace_bytes < need) {
    set_error("%s: workspace needs %lld bytes, got %lld", what, (long long)need, (long long)workspace_bytes);
    return FP8DP_EINVAL;
  }
  const void* const all[] = {dh, gate, up, x, w_gate, w_up, dx, dw_gate, dw_up};
  for (const void* p : all)
    if (!aligned_to(p, 2)) return bad_align(what);
  for (int i = 6; i < 9; ++i)
    for (int j = 0; j < i; ++j)
      if (all[i] != nullptr && all[i] == all[j]) {
        set_error("%s: outputs must not be inputs, nor each other", what);
        return FP8DP_EINVAL;
      }
  auto run = [&](auto t) {
    using T = decltype(t);
    return run_gated_bwd<T>(what, static_cast<const T*>(dh), static_cast<const T*>(gate),
                            static_cast<const T*>(up), static_cast<const T*>(x), static_cast<const T*>(w_gate),
                            static_cast<const T*>(w_up), (int)M, (int)N, (int)K, act, static_cast<T*>(dx),
                            static_cast<T*>(dw_gate), static_cast<T*>(dw_up), workspace, stream);
  };
  return dt == FP8DP_BF16 ? run(bf16_t{}) : run(f16_t{});
}
