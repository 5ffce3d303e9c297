// gated.hip -- the gated linear layer: h = f(x Wg^T) * (x Wu^T).
//
// Both projections are one product whose columns alternate between gate and up, 32 of each: a
// wave then holds a token's g and u of the same channel in two accumulators, and the activation and the
// product are the epilogue; neither projection goes to memory unless the backward pass wants it.
//
// Many tokens are bound by the matrix pipes and their power: 16384 x 8192 x 4096 takes 1540 us (1.43 PFLOP/s; a library's
// product of the same size alone reaches 1.57) and 1650 where both projections are kept.  Few tokens are bound by the weights'
// bytes: 48 x 16384 x 4096 58 us, 4.6 TB/s (the tokens, brought in again for every 16 channels, are more bytes, from L2).  The
// erf form of GELU is not hidden behind the products: 1750 for 1560.  Small ones by launch, first copies and outputs: 777 x 1023 x 1001
// 18 us behind 4.6 for the aligned copies.
#include "gated_core.hpp"
#include "pad16.hpp"

namespace fp8dp {

// Outputs of a wave's TM x TN tiles: columns n .. of the dual product are channels n / 2 ..  Of four column tiles
// two are gate and two are up.
template <typename T, int TM, int TN>
struct GatedOut {
  T *h, *gate, *up;
  int M, N, act;
  __device__ __forceinline__ void operator()(const v4f_t (&acc)[TM][TN], uint8_t* part, int m, int n,
                                             int lane, int) const {
    constexpr int JT = TN / 4;   // 32 channels each
    const int c0 = n / 2;
    auto of = [](int j) { return j / 2 * 4 + j % 2; };   // gate's tile of channel tile j
#pragma unroll
    for (int i0 = 0; i0 < TM; i0 += 2) {
      auto emit = [&](T* to) {
        return [=](int r, int c, const Raw8<T>& v) {
          const int row = m + 16 * i0 + r, left = N - c0 - c;
          if (row < M && left > 0) store_row(to + (int64_t)row * N + c0 + c, left, v);
        };
      };
      with_act(act, [&](auto ACT) {
        turn16<T, JT>(
            part, lane,
            [&](int i, int j, int r) {
              return gate_of<decltype(ACT)::value, false>(acc[i0 + i][of(j)][r], nullptr) *
                     acc[i0 + i][of(j) + 2][r];
            },
            emit(h));
      });
      if (gate != nullptr) {
        turn16<T, JT>(part, lane, [&](int i, int j, int r) { return acc[i0 + i][of(j)][r]; }, emit(gate));
        turn16<T, JT>(part, lane, [&](int i, int j, int r) { return acc[i0 + i][of(j) + 2][r]; }, emit(up));
      }
    }
  }
};

// Sums of a range of K: parts[split][gate, up][M][N].
template <int TM, int TN>
struct GatedParts {
  float* parts;
  int M, N;
  __device__ __forceinline__ void operator()(const v4f_t (&acc)[TM][TN], uint8_t* part, int m, int n,
                                             int lane, int split) const {
    const int c0 = n / 2;
#pragma unroll
    for (int i0 = 0; i0 < TM; i0 += 2)
#pragma unroll
      for (int j0 = 0; j0 < TN; j0 += 2) {
        float* const to = parts + (int64_t)(2 * split + j0 / 2 % 2) * M * N;
        turn32(
            part, lane, [&](int i, int j) { return acc[i0 + i][j0 + j]; },
            [=](int r, int c, const Raw8<float>& v) {
              const int row = m + 16 * i0 + r, col = c0 + j0 / 4 * 32 + c, left = N - col;
              if (row < M && left > 0) store_row(to + (int64_t)row * N + col, left, v);
            });
      }
  }
};

// h (and g, u) from the sums of `splits` ranges.
template <typename T>
__global__ __launch_bounds__(256) void k_gated_join(const float* parts, int splits, int64_t total, T* h,
                                                    T* gate, T* up, int act) {
  const int64_t step = (int64_t)gridDim.x * 2048;
  for (int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; at < total; at += step) {
    const int n = (int)std::min<int64_t>(total - at, 8);
    float g[8] = {}, u[8] = {};
    for (int s = 0; s < splits; ++s) {
      float a[8], b[8];
      load8(parts + (2 * s) * total + at, n, a);
      load8(parts + (2 * s + 1) * total + at, n, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        g[j] += a[j];
        u[j] += b[j];
      }
    }
    if (gate != nullptr) {
      store8(gate + at, n, g);
      store8(up + at, n, u);
    }
    with_act(act, [&](auto ACT) {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = gate_of<decltype(ACT)::value, false>(g[j], nullptr) * u[j];
    });
    store8(h + at, n, g);
  }
}

// ------------------------------------------------------------------ few tokens
// Up to 16 MT tokens: bound by the weights, which are read once.  A workgroup owns 16 channels; its waves take
// the blocks of 128 k in turn and their sums are joined in LDS.  The matrix instruction 16 x 16 x 32 has the
// weight's rows as its first operand, so a lane ends with one token and four channels.  Rows may start and
// end at any byte: a chunk that K cuts is read as the row's last 8 values and shifted.
constexpr int kFewWaves = 8, kFewTokens16 = 64;
// Groups of 16 channels x K from which on rings are used.  Rings / straight from memory (us): 1 x 4096 x 4096 13.4 / 14.1,
// 1 x 16384 x 4096 47.8 / 51.9, 16 x 1024 x 4096 8.8 / 13.1, 64 x 16384 x 4096 63.6 / 101.7; below, one stage of K or two a wave
// fill no ring.
constexpr int64_t kRingWork = (int64_t)256 * 1024;

template <typename T>
__device__ __forceinline__ v8s_t as_frag(const Raw8<T>& r) {
  return __builtin_bit_cast(v8s_t, u32x4_t{r.w[0], r.w[1], r.w[2], r.w[3]});
}

// Outputs of one token and four channels c0 ..
template <typename T>
__device__ __forceinline__ void store_few(v4f_t g, v4f_t u, int token, int c0, int M, int N, int act, T* h, T* gate,
                                          T* up) {
  if (token >= M) return;
  float v[4];
  with_act(act, [&](auto ACT) {
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = gate_of<decltype(ACT)::value, false>(g[r], nullptr) * u[r];
  });
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (c0 + r >= N) continue;
    const int64_t at = (int64_t)token * N + c0 + r;
    h[at] = from_f32<T>(v[r]);
    if (gate != nullptr) {
      gate[at] = from_f32<T>(g[r]);
      up[at] = from_f32<T>(u[r]);
    }
  }
}

template <typename T, int MT>
__global__ __launch_bounds__(64 * kFewWaves) void k_gated_few(const T* x, const T* w_gate, const T* w_up,
                                                              int M, int N, int K, int act, T* h, T* gate,
                                                              T* up) {
  __shared__ v4f_t sums[kFewWaves][2][MT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16, row = lane & 15, part = lane >> 4;
  const int n = n0 + row < N ? n0 + row : N - 1;
  const T *const wg = w_gate + (int64_t)n * K, *const wu = w_up + (int64_t)n * K;
  const T* xr[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) xr[i] = x + (int64_t)(16 * i + row < M ? 16 * i + row : M - 1) * K;
  v4f_t ag[MT], au[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) ag[i] = au[i] = v4f_t{0.0f, 0.0f, 0.0f, 0.0f};

  auto block = [&](int k0, auto WHOLE) {
    constexpr bool whole = decltype(WHOLE)::value;
    Raw8<T> g[4], u[4], v[MT][4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k = k0 + 32 * s + 8 * part;
      auto load = [&](const T* p) {
        if constexpr (whole) return load_raw8(p + k);
        else return load_raw(p + k, K - k);
      };
      g[s] = load(wg);
      u[s] = load(wu);
#pragma unroll
      for (int i = 0; i < MT; ++i) v[i][s] = load(xr[i]);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        ag[i] = mma16(T{}, as_frag(g[s]), as_frag(v[i][s]), ag[i]);
        au[i] = mma16(T{}, as_frag(u[s]), as_frag(v[i][s]), au[i]);
      }
  };
  int k0 = wave * 128;
  for (; k0 + 128 <= K; k0 += kFewWaves * 128) block(k0, std::true_type{});
  if (k0 < K) block(k0, std::false_type{});

#pragma unroll
  for (int i = 0; i < MT; ++i) {
    sums[wave][0][i][lane] = ag[i];
    sums[wave][1][i][lane] = au[i];
  }
  __syncthreads();
  if (wave >= MT) return;
  v4f_t g = {0.0f, 0.0f, 0.0f, 0.0f}, u = g;
#pragma unroll
  for (int w = 0; w < kFewWaves; ++w) {
    g += sums[w][0][wave][lane];
    u += sums[w][1][wave][lane];
  }
  store_few(g, u, 16 * wave + row, n0 + 4 * part, M, N, act, h, gate, up);
}

// The same for rows that start at multiples of 16 bytes.  Fragments read straight from memory have 16 rows in consecutive
// lanes, which the compute unit takes one 16-byte piece a cycle; here each wave copies whole cache lines into a ring of its
// own in LDS, 8 rows x 128 bytes a copy, four times the rate (48 tokens x 16384 x 4096: 85 -> 59 us).  Stages of 64 k go to the waves
// in turn; the grid is resident, and a wave's ring runs on into the workgroup's next 16 channels while their sums
// are joined.  W waves and S slots: 64 KiB or more under way in each compute unit.
template <typename T, int MT, int W, int S>
__global__ __launch_bounds__(64 * W) void k_gated_ring(const T* x, const T* w_gate, const T* w_up, int M, int N,
                                                       int K, int act, T* h, T* gate, T* up) {
  constexpr int TILES = 2 + MT, STAGE = TILES * 2048, NC = 2 * TILES;   // tiles of 16 rows x 64 k; copies a stage
  __shared__ __attribute__((aligned(1024))) uint8_t rings[W * S * STAGE];
  __shared__ v4f_t sums[W][2][MT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint8_t* const ring = rings + wave * S * STAGE;
  const int row = lane & 15, part = lane >> 4;
  const int stages = (K + kStageK - 1) / kStageK, mine = stages > wave ? (stages - wave + W - 1) / W : 0;
  const int groups = (N + 15) / 16, turns = ((int)gridDim.x + groups - 1 - (int)blockIdx.x) / (int)gridDim.x;
  // copy c of a stage: rows 8 (c % 2) + lane / 8 of tile c / 2, the chunk that swz() puts there
  const int crow = lane >> 3, cchunk = lane & 7;
  uint32_t xoff[2 * MT];
#pragma unroll
  for (int c = 0; c < 2 * MT; ++c) {
    const int r = 16 * (c / 2) + 8 * (c % 2) + crow;
    xoff[c] = (uint32_t)(r < M ? r : M - 1) * (uint32_t)K * 2;
  }
  int to = blockIdx.x, to_stage = 0;   // the next to be copied: the group's channels, and its place among this wave's
  auto issue = [&](int slot) {
    const int k0 = (wave + to_stage * W) * kStageK, left = K - k0;
    static_for<NC>([&](auto C) {
      constexpr int c = decltype(C)::value, tile = c / 2;
      const int chunk = cchunk ^ ((4 * (c % 2) + (crow >> 1)) & 7);
      const T* base;
      uint32_t from;
      if constexpr (tile < 2) {
        const int n = to * 16 + 8 * (c % 2) + crow;
        base = (tile == 0 ? w_gate : w_up) + (int64_t)to * 16 * K + k0;
        from = (uint32_t)((n < N ? n : N - 1) - to * 16) * (uint32_t)K * 2;
      } else {
        base = x + k0;
        from = xoff[c - 4];
      }
      from += chunk * 16;
      uint8_t* const l = ring + slot * STAGE + c * 1024;
      if (left >= kStageK)
        copy16_to_lds_from(base, from, l);
      else
        copy16_to_lds(chunk * 8 < left ? reinterpret_cast<const uint8_t*>(base) + from
                                       : reinterpret_cast<const uint8_t*>(&kZeroChunk16), l);
    });
    if (++to_stage == mine) {
      to_stage = 0;
      to += gridDim.x;
    }
  };
  const int total = mine * turns;   // stages of this wave
#pragma unroll
  for (int s = 0; s < S - 1; ++s)
    if (s < total) issue(s);
  int at = 0, slot = 0;             // the stage in hand
  for (int group = blockIdx.x; group < groups; group += gridDim.x) {
    v4f_t ag[MT], au[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) ag[i] = au[i] = v4f_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int j = 0; j < mine; ++j, ++at) {
      __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): the slot to be filled has been read
      if (at + S - 1 < total) issue(slot == 0 ? S - 1 : slot - 1);
      // the copies of the stage in hand have landed: of those behind it as many may be under way as there are
      const int behind = total - 1 - at;
      if (behind >= S - 1) wait_vmcnt<(S - 1) * NC>();
      else if (S > 2 && behind == S - 2) wait_vmcnt<(S - 2) * NC>();
      else if (S > 3 && behind == S - 3) wait_vmcnt<(S > 3 ? S - 3 : 0) * NC>();
      else wait_vmcnt<0>();
      __builtin_amdgcn_sched_barrier(0);
      __asm__ volatile("" ::: "memory");
      const uint8_t* const from = ring + slot * STAGE;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int f = swz(row, 4 * q + part);
        const v8s_t g = *reinterpret_cast<const v8s_t*>(from + f), u = *reinterpret_cast<const v8s_t*>(from + 2048 + f);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const v8s_t v = *reinterpret_cast<const v8s_t*>(from + (2 + i) * 2048 + f);
          ag[i] = mma16(T{}, g, v, ag[i]);
          au[i] = mma16(T{}, u, v, au[i]);
        }
      }
      slot = slot == S - 1 ? 0 : slot + 1;
    }
    // (barriers alone, not __syncthreads(): the copies under way stay so)
    if (group != (int)blockIdx.x) {   // the sums of the channels before have been read
      __builtin_amdgcn_s_waitcnt(0xC07F);
      stage_barrier();
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      sums[wave][0][i][lane] = ag[i];
      sums[wave][1][i][lane] = au[i];
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);
    stage_barrier();
    if (wave < MT) {
      v4f_t g = {0.0f, 0.0f, 0.0f, 0.0f}, u = g;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        g += sums[w][0][wave][lane];
        u += sums[w][1][wave][lane];
      }
      store_few(g, u, 16 * wave + row, group * 16 + 4 * part, M, N, act, h, gate, up);
    }
  }
}

// ------------------------------------------------------------------ launch
static ProductPlan plan_gated(int64_t M, int64_t N, int64_t K, bool direct) {
  return plan_product(M, 2 * N, (K + kStageK - 1) / kStageK, true, direct);
}

template <typename T, int WM, int WN, int TM, int TN, int S, bool DIRECT>
static int launch_gated(const char* what, MmaArgs g, int M, int N, int splits, int act, T* h, T* gate, T* up,
                        float* parts, hipStream_t stream) {
  g.tiles_m = (M + WM * TM * 16 - 1) / (WM * TM * 16);
  g.tiles_n = (N + WN * TN * 8 - 1) / (WN * TN * 8);
  g.splits = splits;
  return for_work<DIRECT>((int64_t)g.tiles_m * g.tiles_n * splits, WM * WN == 8 || S > 2 ? 1 : 2, [&](int first, unsigned count) {
    g.first = first;
    const dim3 grid(count), block(64 * WM * WN);
    if (splits > 1) {
      const GatedParts<TM, TN> out = {parts, M, N};
      hipLaunchKernelGGL((k_mma<T, WM, WN, TM, TN, S, false, false, true, DIRECT, GatedParts<TM, TN>>), grid,
                         block, 0, stream, g, out);
    } else {
      const GatedOut<T, TM, TN> out = {h, gate, up, M, N, act};
      hipLaunchKernelGGL((k_mma<T, WM, WN, TM, TN, S, false, false, true, DIRECT, GatedOut<T, TM, TN>>), grid,
                         block, 0, stream, g, out);
    }
    return check_launch(what);
  });
}

template <typename T>
static int run_gated(const char* what, const T* x, const T* wg, const T* wu, int M, int N, int K, int act, T* h,
                     T* gate, T* up, float* parts, int64_t parts_bytes, hipStream_t stream) {
  MmaArgs g = {};
  g.a = {{reinterpret_cast<const uint16_t*>(x), reinterpret_cast<const uint16_t*>(x)}, K, M};
  g.b = {{reinterpret_cast<const uint16_t*>(wg), reinterpret_cast<const uint16_t*>(wu)}, K, N};
  g.stages = g.seg_stages = (K + kStageK - 1) / kStageK;
  g.valid_a = g.valid_b = K;
  bool direct = rows16(g.a, K) && rows16(g.b, K);
  if (M <= kFewTokens16) {
    const int64_t groups = ((int64_t)N + 15) / 16;
    if (direct && K >= 256 && groups * K >= kRingWork) {
      const dim3 grid((unsigned)std::min<int64_t>(groups, num_cus()));
      auto ring = [&](auto mt, auto w, auto s) {
        constexpr int W = decltype(w)::value;
        hipLaunchKernelGGL((k_gated_ring<T, decltype(mt)::value, W, decltype(s)::value>), grid, dim3(64 * W), 0, stream,
                           x, wg, wu, M, N, K, act, h, gate, up);
        return check_launch(what);
      };
      using std::integral_constant;
      if (M <= 16) return ring(integral_constant<int, 1>{}, integral_constant<int, 8>{}, integral_constant<int, 3>{});
      if (M <= 32) return ring(integral_constant<int, 2>{}, integral_constant<int, 4>{}, integral_constant<int, 4>{});
      if (M <= 48) return ring(integral_constant<int, 3>{}, integral_constant<int, 4>{}, integral_constant<int, 3>{});
      return ring(integral_constant<int, 4>{}, integral_constant<int, 4>{}, integral_constant<int, 2>{});
    }
    const dim3 grid((unsigned)groups), block(64 * kFewWaves);
    auto few = [&](auto mt) {
      hipLaunchKernelGGL((k_gated_few<T, decltype(mt)::value>), grid, block, 0, stream, x, wg, wu, M, N, K, act,
                         h, gate, up);
      return check_launch(what);
    };
    if (M <= 16) return few(std::integral_constant<int, 1>{});
    if (M <= 32) return few(std::integral_constant<int, 2>{});
    if (M <= 48) return few(std::integral_constant<int, 3>{});
    return few(std::integral_constant<int, 4>{});
  }
  if (!direct && pad_pays(M, N, K, false) && parts_bytes >= pad_bytes(M, N, K)) {
    uint16_t* const to = reinterpret_cast<uint16_t*>(parts);
    const int rc = pad_operands(what, g.a.p[0], g.b.p[0], g.b.p[1], M, N, K, to, stream);
    if (rc) return rc;
    const int64_t ld = pad_ld(K);
    g.a = {{to, to}, ld, M};
    g.b = {{to + M * ld, to + (M + N) * ld}, ld, N};
    direct = true;
    parts += pad_bytes(M, N, K) / 4;
    parts_bytes -= pad_bytes(M, N, K);
  }
  ProductPlan p = plan_gated(M, N, K, direct);
  if ((int64_t)p.splits * 2 * M * N * 4 > parts_bytes) p.splits = 1;
  int rc;
  if (p.shape == kTile256) rc = launch_gated<T, 4, 2, 4, 8, 2, true>(what, g, M, N, p.splits, act, h, gate, up, parts, stream);
  else if (direct && tiles_of(kTile128, M, 2 * (int64_t)N) * p.splits <= num_cus())
    rc = launch_gated<T, 2, 2, 4, 4, 4, true>(what, g, M, N, p.splits, act, h, gate, up, parts, stream);
  else if (direct) rc = launch_gated<T, 2, 2, 4, 4, 2, true>(what, g, M, N, p.splits, act, h, gate, up, parts, stream);
  else rc = launch_gated<T, 2, 2, 4, 4, 2, false>(what, g, M, N, p.splits, act, h, gate, up, parts, stream);
  if (rc || p.splits == 1) return rc;
  const int64_t total = (int64_t)M * N;
  hipLaunchKernelGGL((k_gated_join<T>), dim3(grid_for((total + 7) / 8, 256, 16)), dim3(256), 0, stream, parts,
                     p.splits, total, h, gate, up, act);
  return check_launch(what);
}

}  // namespace fp8dp

using namespace fp8dp;

extern "C" int64_t gated_linear_workspace(int64_t M, int64_t N, int64_t K) {
  if (M <= kFewTokens16 || N < 1 || K < 1 || M > FP8DP_GATED_MAX_ROWS || N > FP8DP_GATED_MAX_WIDTH ||
      K > FP8DP_GATED_MAX_WIDTH)
    return 0;
  auto parts = [&](bool direct) {
    const int splits = plan_gated(M, N, K, direct).splits;
    return splits > 1 ? (int64_t)splits * 2 * M * N * 4 : (int64_t)0;
  };
  const int64_t padded = pad_pays(M, N, K, false) ? pad_bytes(M, N, K) + parts(true) : 0;
  return std::max({padded, parts(false), K % 8 == 0 ? parts(true) : (int64_t)0});
}

extern "C" int gated_linear(const void* x, const void* w_gate, const void* w_up, int64_t M, int64_t N,
                            int64_t K, fp8dp_dtype dt, fp8dp_gate act, void* h, void* gate, void* up,
                            void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  const char* what = "gated_linear";
  const int rc = check_gated(what, M, N, K, dt, act, workspace, workspace_bytes);
  if (rc) return rc;
  if (x == nullptr || w_gate == nullptr || w_up == nullptr || h == nullptr) {
    set_error("%s: x, w_gate, w_up and h must be non-NULL", what);
    return FP8DP_EINVAL;
  }
  if ((gate == nullptr) != (up == nullptr)) {
    set_error("%s: gate and up go together", what);
    return FP8DP_EINVAL;
  }
  if (!aligned_to(x, 2) || !aligned_to(w_gate, 2) || !aligned_to(w_up, 2) || !aligned_to(h, 2) ||
      !aligned_to(gate, 2) || !aligned_to(up, 2))
    return bad_align(what);
  const void* const all[] = {x, w_gate, w_up, h, gate, up};
  for (int i = 3; i < 6; ++i)
    for (int j = 0; j < i; ++j)
      if (all[i] != nullptr && all[i] == all[j]) {
        set_error("%s: h, gate and up must be different buffers, and no inputs", what);
        return FP8DP_EINVAL;
      }
  auto run = [&](auto t) {
    using T = decltype(t);
    return run_gated<T>(what, static_cast<const T*>(x), static_cast<const T*>(w_gate),
                        static_cast<const T*>(w_up), (int)M, (int)N, (int)K, act, static_cast<T*>(h),
                        static_cast<T*>(gate), static_cast<T*>(up), static_cast<float*>(workspace),
                        workspace == nullptr ? 0 : workspace_bytes, stream);
  };
  return dt == FP8DP_BF16 ? run(bf16_t{}) : run(f16_t{});
}
