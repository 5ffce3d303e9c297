// lora.hip -- low-rank adapters of many requests beside a shared projection.
//
//   v[t] = a_i x[t],   y[t] = base[t] + scale_i b_i v[t],   i the adapter of token t
//
// A plan, made once per step, orders the tokens by adapter and cuts each adapter's into tiles of up to
// 32, so that an adapter's weights are read once per tile.  Two kernels follow: the first gathers a
// tile's tokens and leaves v in binary32, K split over workgroups where there are few tiles; the second adds
// the ranges up and multiplies by b.  v goes to the matrix instructions as a sum of two 16-bit
// values, scaled by a power of two per token: 16 ranks fill half of an instruction's 32, so the low parts
// take the other half and cost nothing.
#include "gated_core.hpp"

namespace fp8dp {

constexpr int kLoraTile = 32;
constexpr int kLoraHead = 4;   // words: tiles, tokens, adapters, 0

inline int64_t lora_most_tiles(int64_t tokens, int64_t adapters) {
  return tokens / kLoraTile + std::min(tokens, adapters + 1);
}

// A plan's parts.
struct LoraPlan {
  const int32_t* p;
  int tokens;
  __device__ __forceinline__ const int32_t* order() const { return p + kLoraHead; }
  __device__ __forceinline__ const int32_t* tiles() const { return p + kLoraHead + tokens; }
};
struct LoraTile {
  int start, adapter, count;   // adapter -1: none
};
// Whether workgroup `b` has a tile of a plan for these sizes.
__device__ __forceinline__ bool lora_tile(const LoraPlan& plan, int adapters, int b, LoraTile* t) {
  if (plan.p[1] != plan.tokens || plan.p[2] != adapters || b >= plan.p[0]) return false;
  const int32_t* const e = plan.tiles() + 2 * (int64_t)b;
  t->start = e[0];
  t->adapter = e[1] >> 8;
  t->count = e[1] & 255;
  return true;
}

// One workgroup: counts per wave and adapter in LDS (each wave has a range of the tokens), their sums over
// adapters, then every wave hands out its tokens' places in order, so that the order is stable.
constexpr int kPlanWaves = 16;
__global__ __launch_bounds__(64 * kPlanWaves) void k_lora_plan(const int32_t* index, int tokens, int adapters,
                                                               int32_t* plan) {
  extern __shared__ int32_t shared[];
  const int groups = adapters + 1;                  // the last: no adapter
  int32_t* const counts = shared;                   // [wave][group]
  int32_t* const firsts = counts + kPlanWaves * groups;   // first place of a group, after its scan
  int32_t* const tiles = firsts + groups;           // first tile of a group
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, threads = 64 * kPlanWaves;
  for (int i = tid; i < kPlanWaves * groups; i += threads) counts[i] = 0;
  __syncthreads();
  const int64_t per = ((int64_t)tokens + threads - 1) / threads * 64;
  const int64_t begin = wave * per, end = begin + per < tokens ? begin + per : tokens;
  int32_t* const mine = counts + wave * groups;
  auto group = [&](int64_t t) {
    const int32_t i = index[t];
    return i >= 0 && i < adapters ? i : adapters;
  };
  for (int64_t t = begin + lane; t < end; t += 64) atomicAdd(&mine[group(t)], 1);
  __syncthreads();
  for (int g = tid; g < groups; g += threads) {
    int sum = 0;
    for (int w = 0; w < kPlanWaves; ++w) sum += counts[w * groups + g];
    firsts[g] = sum;
    tiles[g] = (sum + kLoraTile - 1) / kLoraTile;
  }
  __syncthreads();
  // inclusive sums over the groups, at most three of them a thread
  for (int d = 1; d < groups; d <<= 1) {
    int a[3], b[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int g = tid + i * threads;
      a[i] = g < groups && g >= d ? firsts[g - d] : 0;
      b[i] = g < groups && g >= d ? tiles[g - d] : 0;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int g = tid + i * threads;
      if (g < groups) {
        firsts[g] += a[i];
        tiles[g] += b[i];
      }
    }
    __syncthreads();
  }
  // counts become the first place of each wave's tokens of a group
  for (int g = tid; g < groups; g += threads) {
    int at = g > 0 ? firsts[g - 1] : 0;
    for (int w = 0; w < kPlanWaves; ++w) {
      const int n = counts[w * groups + g];
      counts[w * groups + g] = at;
      at += n;
    }
  }
  __syncthreads();
  int32_t* const order = plan + kLoraHead;
  for (int64_t t0 = begin; t0 < end; t0 += 64) {
    const int64_t t = t0 + lane;
    const int g = t < end ? group(t) : -1;
    uint64_t left = __ballot(g >= 0);
    while (left != 0) {   // (one group of the wave's tokens a turn)
      const int lead = __builtin_amdgcn_readlane(g, __builtin_ctzll(left));
      const uint64_t same = __ballot(g == lead);
      const int at = mine[lead];
      if (g == lead) order[at + __popcll(same & ((1ull << lane) - 1))] = (int32_t)t;
      if (lane == 0) mine[lead] = at + __popcll(same);
      left &= ~same;
    }
  }
  const int total = tiles[groups - 1];
  int32_t* const out = plan + kLoraHead + tokens;
  for (int b = tid; b < total; b += threads) {
    int lo = 0, hi = groups - 1;   // the first group whose tiles reach past b
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (tiles[mid] > b) hi = mid;
      else lo = mid + 1;
    }
    const int first = lo > 0 ? firsts[lo - 1] : 0, j = b - (lo > 0 ? tiles[lo - 1] : 0);
    const int start = first + j * kLoraTile, left = firsts[lo] - start;
    out[2 * (int64_t)b] = start;
    out[2 * (int64_t)b + 1] = (lo == adapters ? -256 : lo * 256) + (left < kLoraTile ? left : kLoraTile);
  }
  if (tid == 0) {
    plan[0] = total;
    plan[1] = tokens;
    plan[2] = adapters;
    plan[3] = 0;
  }
}

struct LoraArgs {
  LoraPlan plan;
  const void *x, *a, *b, *base;
  const float* scale;
  const int32_t* ranks;
  int N, K, rank, adapters, splits, k_range;
  void* y;
  float* v;   // [split][place][ranks to a multiple of 16]
};

__device__ __forceinline__ int lora_rank(const LoraArgs& a, int adapter) {
  if (a.ranks == nullptr) return a.rank;
  const int r = a.ranks[adapter];
  return r < 0 ? 0 : r < a.rank ? r : a.rank;
}

template <typename T>
__device__ __forceinline__ v8s_t as_lora(const Raw8<T>& r) {
  return __builtin_bit_cast(v8s_t, u32x4_t{r.w[0], r.w[1], r.w[2], r.w[3]});
}

// v of a tile, up to 16 RB ranks and a range of K; four waves take its blocks of 64 in turn.
constexpr int kLoraWaves = 4;
template <typename T, int RB>
__global__ __launch_bounds__(64 * kLoraWaves) void k_lora_down(LoraArgs a) {
  __shared__ v4f_t sums[kLoraWaves][RB][2][64];
  LoraTile tile;
  if (!lora_tile(a.plan, a.adapters, blockIdx.x, &tile) || tile.adapter < 0) return;
  const int rank = lora_rank(a, tile.adapter), r0 = blockIdx.z * 16 * RB;
  if (r0 >= rank) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, part = lane >> 4;
  const bool second = tile.count > 16;
  const T* xr[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int at = 16 * i + row < tile.count ? 16 * i + row : tile.count - 1;
    xr[i] = static_cast<const T*>(a.x) + (int64_t)a.plan.order()[tile.start + at] * a.K;
  }
  const T* ar[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int r = r0 + 16 * b + row < rank ? r0 + 16 * b + row : rank - 1;   // (spare ranks meet no one)
    ar[b] = static_cast<const T*>(a.a) + ((int64_t)tile.adapter * a.rank + r) * a.K;
  }
  v4f_t acc[RB][2];
#pragma unroll
  for (int b = 0; b < RB; ++b) acc[b][0] = acc[b][1] = v4f_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int begin = blockIdx.y * a.k_range, end = begin + a.k_range < a.K ? begin + a.k_range : a.K;
  auto block = [&](int k0, auto WHOLE) {
    constexpr bool whole = decltype(WHOLE)::value;
    Raw8<T> w[RB][2], x[2][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int k = k0 + 32 * s + 8 * part;
      auto load = [&](const T* p) {
        if constexpr (whole) return load_raw8(p + k);
        else return load_raw(p + k, end - k);
      };
#pragma unroll
      for (int b = 0; b < RB; ++b) w[b][s] = load(ar[b]);
      x[0][s] = load(xr[0]);
      if (second) x[1][s] = load(xr[1]);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        acc[b][0] = mma16(T{}, as_lora(w[b][s]), as_lora(x[0][s]), acc[b][0]);
        if (second) acc[b][1] = mma16(T{}, as_lora(w[b][s]), as_lora(x[1][s]), acc[b][1]);
      }
  };
  int k0 = begin + wave * 64;
  for (; k0 + 64 <= end; k0 += kLoraWaves * 64) block(k0, std::true_type{});
  if (k0 < end) block(k0, std::false_type{});
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int i = 0; i < 2; ++i) sums[wave][b][i][lane] = acc[b][i];
  __syncthreads();
  const int rp = (a.rank + 15) / 16 * 16;
  for (int i = threadIdx.x; i < RB * 2 * 64; i += 64 * kLoraWaves) {
    const int l = i & 63, half = (i >> 6) & 1, b = i >> 7;
    const int token = 16 * half + (l & 15), r = r0 + 16 * b + 4 * (l >> 4);
    if (token >= tile.count || r >= rp) continue;
    v4f_t s = sums[0][b][half][l];
#pragma unroll
    for (int w = 1; w < kLoraWaves; ++w) s += sums[w][b][half][l];
    *reinterpret_cast<v4f_t*>(a.v + ((int64_t)blockIdx.y * a.plan.tokens + tile.start + token) * rp + r) = s;
  }
}

// y of a tile and 32 channels a turn of each wave.  v is staged in LDS as 16-bit pairs [token][16 ranks: 16
// high parts, 16 low parts].  Two instructions give a lane one token and 8 consecutive channels.
constexpr int kLoraChannels = 512;   // of a workgroup
template <typename T>
__global__ __launch_bounds__(64 * kLoraWaves) void k_lora_up(LoraArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint16_t pairs[];
  __shared__ float factor[kLoraTile];
  LoraTile tile;
  if (!lora_tile(a.plan, a.adapters, blockIdx.x, &tile)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rank = tile.adapter < 0 ? 0 : lora_rank(a, tile.adapter);
  const int n_end = std::min<int>(a.N, (blockIdx.y + 1) * kLoraChannels);
  const int32_t* const order = a.plan.order() + tile.start;
  const T* const base = static_cast<const T*>(a.base);
  T* const y = static_cast<T*>(a.y);
  if (rank == 0) {
    if (y == base) return;
    const int n = n_end - blockIdx.y * kLoraChannels, vecs = (n + 7) / 8;
    for (int i = threadIdx.x; i < tile.count * vecs; i += 64 * kLoraWaves) {
      const int c = blockIdx.y * kLoraChannels + i % vecs * 8;
      const int64_t at = (int64_t)order[i / vecs] * a.N + c;
      Raw8<T> r = {};
      if (base != nullptr) r = load_raw(base + at, n_end - c);
      store_row(y + at, n_end - c, r);
    }
    return;
  }
  const int blocks = (rank + 15) / 16, rp = (a.rank + 15) / 16 * 16, pitch = blocks * 32 + 8;
  // 8 threads a token
  {
    const int token = threadIdx.x >> 3, sub = threadIdx.x & 7;
    const bool live = token < tile.count;
    const float* const from = a.v + (int64_t)(tile.start + (live ? token : 0)) * rp;
    const int64_t step = (int64_t)a.plan.tokens * rp;
    auto value = [&](int r) {
      float s = 0.0f;
      if (live && r < rank)
        for (int p = 0; p < a.splits; ++p) s += from[p * step + r];
      return s;
    };
    float top = 0.0f;
    for (int r = sub; r < blocks * 16; r += 8) {
      const float m = __builtin_fabsf(value(r));
      top = m > top ? m : top;
    }
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) {
      const float o = __shfl_xor(top, d);
      top = o > top ? o : top;
    }
    // a power of two that brings the largest to [1, 2), where there is one
    const int e = (int)(__float_as_uint(top) >> 23);
    const bool plain = e > 0 && e < 255;
    const int shift = plain ? (e < 2 ? 125 : e > 252 ? -125 : 127 - e) : 0;
    const float down = __uint_as_float((uint32_t)(127 + shift) << 23);
    for (int r = sub; r < blocks * 16; r += 8) {
      const float v = value(r) * down;
      const T hi = from_f32<T>(v);
      const float rest = v - to_f32(hi);
      uint16_t* const at = pairs + token * pitch + r / 16 * 32 + r % 16;
      at[0] = hi.bits;
      at[16] = from_f32<T>(rest == rest ? rest : 0.0f).bits;   // (an infinite v has no low part)
    }
    if (sub == 0)
      factor[token] = a.scale[tile.adapter] * __uint_as_float((uint32_t)(127 - shift) << 23);
  }
  __syncthreads();
  const int row = lane & 15, part = lane >> 4;
  const bool second = tile.count > 16;
  const T* const b = static_cast<const T*>(a.b) + (int64_t)tile.adapter * a.N * a.rank;
  for (int n0 = blockIdx.y * kLoraChannels + wave * 32; n0 < n_end; n0 += kLoraWaves * 32) {
    const int c = n0 + 8 * part, left = n_end - c;
    int64_t at[2];
    Raw8<T> old[2] = {};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int token = 16 * i + row;
      at[i] = token < tile.count ? (int64_t)order[token] * a.N + c : -1;
      if (at[i] >= 0 && base != nullptr) old[i] = load_raw(base + at[i], left);
    }
    v4f_t acc[2][2] = {};
    // row i of instruction j is channel 8 (i / 4) + 4 j + i % 4
    const T* br[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int n = n0 + 8 * (row >> 2) + 4 * j + (row & 3);
      br[j] = b + (int64_t)(n < a.N ? n : a.N - 1) * a.rank;
    }
    for (int k = 0; k < blocks; ++k) {
      const int r = 16 * k + 8 * (part & 1);
      Raw8<T> w[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) w[j] = load_raw(br[j] + r, rank - r);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (i == 1 && !second) continue;
        const uint16_t* const from = pairs + (16 * i + row) * pitch + 32 * k + 8 * part;
        const v8s_t v = *reinterpret_cast<const v8s_t*>(from);
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mma16(T{}, as_lora(w[j]), v, acc[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (at[i] < 0 || left <= 0) continue;
      const float f = factor[16 * i + row];
      float o[8], s[8];
      widen8f(old[i], o);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = __builtin_fmaf(acc[i][j >> 2][j & 3], f, o[j]);
      store8(y + at[i], left, s);
    }
  }
}

// Over how many ranges K is split: workgroups for every compute unit four times, ranges of 256 or more.
struct LoraSplit {
  int splits, range;
};
static LoraSplit lora_split(int64_t tokens, int64_t K, int64_t rank, int64_t adapters) {
  const int64_t tiles = tokens / kLoraTile + std::min(tokens, adapters), groups = tiles * ((rank + 63) / 64);
  int64_t s = (4 * (int64_t)num_cus() + groups - 1) / groups;
  s = std::max<int64_t>(1, std::min<int64_t>({s, K / 256, 16}));
  const int64_t range = round_up((K + s - 1) / s, 64);
  return {(int)((K + range - 1) / range), (int)range};
}

template <typename T>
static int run_lora(const LoraArgs& a, int64_t most, hipStream_t stream) {
  const char* what = "lora_add";
  const int rb = a.rank <= 16 ? 1 : a.rank <= 32 ? 2 : 4;
  const dim3 block(64 * kLoraWaves);
  const dim3 down((unsigned)most, (unsigned)a.splits, (unsigned)((a.rank + 16 * rb - 1) / (16 * rb)));
  if (rb == 1) hipLaunchKernelGGL((k_lora_down<T, 1>), down, block, 0, stream, a);
  else if (rb == 2) hipLaunchKernelGGL((k_lora_down<T, 2>), down, block, 0, stream, a);
  else hipLaunchKernelGGL((k_lora_down<T, 4>), down, block, 0, stream, a);
  const int rc = check_launch(what);
  if (rc) return rc;
  const dim3 up((unsigned)most, (unsigned)((a.N + kLoraChannels - 1) / kLoraChannels));
  const size_t lds = (size_t)kLoraTile * ((a.rank + 15) / 16 * 32 + 8) * 2;
  hipLaunchKernelGGL((k_lora_up<T>), up, block, lds, stream, a);
  return check_launch(what);
}

static bool lora_sizes(int64_t tokens, int64_t adapters) {
  return tokens >= 1 && tokens <= FP8DP_LORA_MAX_TOKENS && adapters >= 1 &&
         adapters <= FP8DP_LORA_MAX_ADAPTERS;
}
static int check_lora_sizes(const char* what, int64_t tokens, int64_t adapters) {
  if (lora_sizes(tokens, adapters)) return FP8DP_OK;
  set_error("%s: tokens must be 1 .. %d and adapters 1 .. %d (got %lld, %lld)", what, FP8DP_LORA_MAX_TOKENS,
            FP8DP_LORA_MAX_ADAPTERS, (long long)tokens, (long long)adapters);
  return FP8DP_EINVAL;
}

}  // namespace fp8dp

using namespace fp8dp;

extern "C" int64_t lora_plan_size(int64_t tokens, int64_t adapters) {
  return lora_sizes(tokens, adapters) ? kLoraHead + tokens + 2 * lora_most_tiles(tokens, adapters) : -1;
}

extern "C" int lora_plan(const int32_t* index, int64_t tokens, int64_t adapters, int32_t* plan,
                         hipStream_t stream) {
  const char* what = "lora_plan";
  const int rc = check_lora_sizes(what, tokens, adapters);
  if (rc) return rc;
  if (index == nullptr || plan == nullptr) {
    set_error("%s: index and plan must be non-NULL", what);
    return FP8DP_EINVAL;
  }
  if (!aligned_to(index, 4) || !aligned_to(plan, 4)) return bad_align(what);
  const size_t lds = (size_t)(kPlanWaves + 2) * (adapters + 1) * 4;
  if (lds > 65536) {
    static const hipError_t allowed = hipFuncSetAttribute(
        reinterpret_cast<const void*>(&k_lora_plan), hipFuncAttributeMaxDynamicSharedMemorySize,
        (kPlanWaves + 2) * (FP8DP_LORA_MAX_ADAPTERS + 1) * 4);
    if (allowed != hipSuccess) {
      set_error("%s: %s", what, hipGetErrorString(allowed));
      return FP8DP_EHIP;
    }
  }
  hipLaunchKernelGGL(k_lora_plan, dim3(1), dim3(64 * kPlanWaves), lds, stream, index, (int)tokens, (int)adapters,
                     plan);
  return check_launch(what);
}

extern "C" int64_t lora_add_workspace(int64_t tokens, int64_t N, int64_t K, int64_t rank, int64_t adapters) {
  if (!lora_sizes(tokens, adapters) || N < 1 || K < 1 || rank < 1 || N > FP8DP_GATED_MAX_WIDTH ||
      K > FP8DP_GATED_MAX_WIDTH || rank > FP8DP_LORA_MAX_RANK)
    return -1;
  return (int64_t)lora_split(tokens, K, rank, adapters).splits * tokens * round_up(rank, 16) * 4;
}

extern "C" int lora_add(const void* x, const void* a, const void* b, const float* scale, const int32_t* ranks,
                        const int32_t* plan, const void* base, int64_t tokens, int64_t N, int64_t K,
                        int64_t rank, int64_t adapters, fp8dp_dtype dt, void* y, void* workspace,
                        int64_t workspace_bytes, hipStream_t stream) {
  const char* what = "lora_add";
  const int rc = check_lora_sizes(what, tokens, adapters);
  if (rc) return rc;
  if (N < 1 || K < 1 || rank < 1 || N > FP8DP_GATED_MAX_WIDTH || K > FP8DP_GATED_MAX_WIDTH ||
      rank > FP8DP_LORA_MAX_RANK) {
    set_error("%s: N and K must be 1 .. %d and rank 1 .. %d (got %lld, %lld, %lld)", what,
              FP8DP_GATED_MAX_WIDTH, FP8DP_LORA_MAX_RANK, (long long)N, (long long)K, (long long)rank);
    return FP8DP_EINVAL;
  }
  if (dt != FP8DP_BF16 && dt != FP8DP_F16) {
    set_error("%s: the type must be bfloat16 or float16", what);
    return FP8DP_EINVAL;
  }
  if (x == nullptr || a == nullptr || b == nullptr || scale == nullptr || plan == nullptr || y == nullptr ||
      workspace == nullptr) {
    set_error("%s: x, a, b, scale, plan, y and workspace must be non-NULL", what);
    return FP8DP_EINVAL;
  }
  if (!aligned_to(x, 2) || !aligned_to(a, 2) || !aligned_to(b, 2) || !aligned_to(base, 2) || !aligned_to(y, 2) ||
      !aligned_to(scale, 4) || !aligned_to(ranks, 4) || !aligned_to(plan, 4))
    return bad_align(what);
  const int64_t need = lora_add_workspace(tokens, N, K, rank, adapters);
  if (!aligned16(workspace) || workspace_bytes < need) {
    set_error("%s: workspace must be 16-byte aligned and of %lld bytes, got %lld", what, (long long)need,
              (long long)workspace_bytes);
    return FP8DP_EINVAL;
  }
  if (y == x || y == a || y == b) {
    set_error("%s: y must not be x, a or b", what);
    return FP8DP_EINVAL;
  }
  const LoraSplit s = lora_split(tokens, K, rank, adapters);
  LoraArgs g = {};
  g.plan = {plan, (int)tokens};
  g.x = x;
  g.a = a;
  g.b = b;
  g.base = base;
  g.scale = scale;
  g.ranks = ranks;
  g.N = (int)N;
  g.K = (int)K;
  g.rank = (int)rank;
  g.adapters = (int)adapters;
  g.splits = s.splits;
  g.k_range = s.range;
  g.y = y;
  g.v = static_cast<float*>(workspace);
  const int64_t most = lora_most_tiles(tokens, adapters);
  return dt == FP8DP_BF16 ? run_lora<bf16_t>(g, most, stream) : run_lora<f16_t>(g, most, stream);
}
