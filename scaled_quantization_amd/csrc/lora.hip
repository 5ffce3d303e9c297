// lora.hip -- low-rank adapters of many requests beside a shared projection.
//
//   v[t] = a_i x[t],   y[t] = base[t] + scale_i b_i v[t],   i the adapter of token t
//
// A plan, made once per step, orders the tokens by adapter and cuts each adapter's into tiles of up to
// 32, so that an adapter's weights are read once per tile.  It takes one workgroup, whose waves hand out places to one adapter
// of their 64 tokens a turn: 10 us for 64 tokens, 11 for 5003 of 8 adapters, 85 for 70000 in runs, 370 for 70000 mixed of 64.  Two kernels follow: the first gathers a
// tile's tokens and leaves v in binary32, K split over workgroups where there are few tiles; the second adds
// the ranges up and multiplies by b.  Each reads its weights once a tile; what bounds both is the way from the plan to the
// data (entry, order, rows, weights: one waits for the other), so as many workgroups as fit are under way and each loads
// ahead.  64 tokens of 64 adapters, ranks of 16, 4096 x 4096: 4.7 and 8 us; 5003 tokens of 8, ranks of 64: 16 and 36 us,
// where 131 MB at the rate of a large copy would be 20 in all.  v goes to the matrix instructions as a sum of two 16-bit
// values, scaled by a power of two per token: of up to 16 ranks, which fill half of an instruction's 32, the low parts
// take the other half; more have an instruction for each part.
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
  // (the entry is there for every workgroup, and read along with the head)
  const int32_t* const e = plan.tiles() + 2 * (int64_t)b;
  const int start = e[0], info = e[1], count = plan.p[0], tokens = plan.p[1], made_for = plan.p[2];
  t->start = start;
  t->adapter = info >> 8;
  t->count = info & 255;
  return tokens == plan.tokens && made_for == adapters && b < count;
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

// Ranks as the matrix instructions take them.
__host__ __device__ inline int lora_pitch(int rank) { return rank <= 16 ? 16 : (rank + 31) / 32 * 32; }

struct LoraArgs {
  LoraPlan plan;
  const void *x, *a, *b, *base;
  const float* scale;
  const int32_t* ranks;
  int N, K, rank, adapters, splits, k_range, most;   // most: tiles that the plan has room for
  void* y;
  float* v;   // [split][place][lora_pitch(rank)]
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

// v of a tile, up to 16 RB ranks and a range of K; eight waves take its blocks of 64 in turn.
constexpr int kDownWaves = 8, kLoraWaves = 4;   // of the first kernel's workgroups, and of the second's
template <typename T, int RB>
__global__ __launch_bounds__(64 * kDownWaves) void k_lora_down(LoraArgs a) {
  __shared__ v4f_t sums[kDownWaves][RB][2][64];
  LoraTile tile;
  const uint32_t at_tile = blockIdx.x / (uint32_t)a.splits, split = blockIdx.x - at_tile * (uint32_t)a.splits;
  if (!lora_tile(a.plan, a.adapters, (int)at_tile, &tile) || tile.adapter < 0) return;
  const int rank = lora_rank(a, tile.adapter), r0 = blockIdx.y * 16 * RB;
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
  const int begin = (int)split * a.k_range, end = begin + a.k_range < a.K ? begin + a.k_range : a.K;
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
  for (; k0 + 64 <= end; k0 += kDownWaves * 64) block(k0, std::true_type{});
  if (k0 < end) block(k0, std::false_type{});
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int i = 0; i < 2; ++i) sums[wave][b][i][lane] = acc[b][i];
  __syncthreads();
  const int rp = lora_pitch(a.rank);
  for (int i = threadIdx.x; i < RB * 2 * 64; i += 64 * kDownWaves) {
    const int l = i & 63, half = (i >> 6) & 1, b = i >> 7;
    const int token = 16 * half + (l & 15), r = r0 + 16 * b + 4 * (l >> 4);
    if (token >= tile.count || r >= rp) continue;
    v4f_t s = sums[0][b][half][l];
#pragma unroll
    for (int w = 1; w < kDownWaves; ++w) s += sums[w][b][half][l];
    *reinterpret_cast<v4f_t*>(a.v + ((int64_t)split * a.plan.tokens + tile.start + token) * rp + r) = s;
  }
}

// y of a tile.  A wave takes 32 channels a step; pairs of instructions give a lane one token and 8 consecutive
// channels.  What a step reads (base and b, up to 16 RB ranks) is loaded DEPTH steps ahead, the first of them
// before v is there (of 64 ranks two steps: a third no longer fits the registers of four waves, 51 us for 42 with 5003
// tokens).  v is staged in LDS as 16-bit pairs [token][GR ranks: GR high parts, GR low parts].
// Channels of a workgroup, 64 lanes x 8.  (1024, which stage v half as often: 16 us for 13 with 64 tokens and 57 for 53
// with 5003, both kernels.)  A wave's are in a row: the halves of a cache line are read, and stored, one after the other by
// the same wave.  The workgroups of a tile follow each other, so that whole rows are under way (both together: 20000
// tokens 170 us, now 157).
constexpr int kLoraChannels = 512;
constexpr int kLoraSplits = 8;       // most ranges of K
constexpr int kLoraGridY = 32768;    // tiles of the grid's second dimension
template <typename T, int RB, int DEPTH>
__global__ __launch_bounds__(64 * kLoraWaves, 4) void k_lora_up(LoraArgs a) {
  constexpr int GR = RB == 1 ? 16 : 32, GN = RB == 1 ? 1 : RB / 2;   // ranks of a group, groups of a chunk
  extern __shared__ __attribute__((aligned(16))) uint8_t shared_up[];
  __shared__ float factor[kLoraTile];
  LoraTile tile;
  const int at_tile = blockIdx.y + blockIdx.z * kLoraGridY;
  if (at_tile >= a.most || !lora_tile(a.plan, a.adapters, at_tile, &tile)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rank = tile.adapter < 0 ? 0 : lora_rank(a, tile.adapter);
  const int n_begin = blockIdx.x * kLoraChannels, n_end = std::min<int>(a.N, n_begin + kLoraChannels);
  const int32_t* const order = a.plan.order() + tile.start;
  const T* const base = static_cast<const T*>(a.base);
  T* const y = static_cast<T*>(a.y);
  if (rank == 0) {
    if (y == base) return;
    // 64 lanes a row of up to 512 channels, four rows of a wave under way
    const int c = n_begin + lane * 8, left = n_end - c;
    for (int t0 = 0; t0 < tile.count; t0 += 4 * kLoraWaves) {
      Raw8<T> r[4] = {};
      int64_t at[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = t0 + i * kLoraWaves + wave;
        at[i] = (int64_t)order[t < tile.count ? t : t0] * a.N + c;
        if (base != nullptr && t < tile.count) r[i] = load_raw(base + at[i], left);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t0 + i * kLoraWaves + wave < tile.count && left > 0) store_row(y + at[i], left, r[i]);
    }
    return;
  }
  const int row = lane & 15, part = lane >> 4;
  const bool second = tile.count > 16;
  const int groups = (rank + GR - 1) / GR, chunks = (groups + GN - 1) / GN, wide = groups * GR;
  auto rank_at = [&](int g) { return g * GR + 8 * (RB == 1 ? part & 1 : part); };   // of this lane's 8 in group g
  const T* const b = static_cast<const T*>(a.b) + (int64_t)tile.adapter * a.N * a.rank;
  int64_t token[2];   // first element of this lane's rows of base and y
  bool live[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    live[i] = 16 * i + row < tile.count;
    token[i] = (int64_t)order[live[i] ? 16 * i + row : 0] * a.N;
  }
  struct Step {
    Raw8<T> old[2], w[GN][2];
  };
  const int per = (n_end - n_begin + kLoraWaves * 32 - 1) / (kLoraWaves * 32) * 32, first = n_begin + wave * per;
  const int turns = first < n_end ? (std::min(n_end - first, per) + 31) / 32 : 0, steps = turns * chunks;
  auto load = [&](int s, Step& o) {
    if (s >= steps) return;
    const int turn = chunks == 1 ? s : s / chunks, chunk = s - turn * chunks;
    const int n0 = first + turn * 32, c = n0 + 8 * part;
    if (chunk == 0 && base != nullptr) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (live[i]) o.old[i] = load_raw(base + token[i] + c, n_end - c);
    }
    // row i of instruction j is channel 8 (i / 4) + 4 j + i % 4
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int n = n0 + 8 * (row >> 2) + 4 * j + (row & 3);
      const T* const br = b + (uint32_t)(n < a.N ? n : a.N - 1) * (uint32_t)a.rank;   // (below 2^28)
#pragma unroll
      for (int k = 0; k < GN; ++k) {
        const int r = rank_at(chunk * GN + k);
        if (a.rank >= 8) o.w[k][j] = load_raw8(br + (r < a.rank - 8 ? r : a.rank - 8));
        else load_cut(br, a.rank, o.w[k][j]);
      }
    }
  };
  Step ahead[DEPTH];
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) {
    ahead[d] = Step{};
    load(d, ahead[d]);
  }

  // v: the ranges' sums in binary32 (rows of 8 words more: 8 tokens are read at once), then the pairs (8 threads a token)
  const int rp = lora_pitch(a.rank), pitch = wide * 2 + 8;
  float* const sums = reinterpret_cast<float*>(shared_up);                       // [token][wide]
  uint16_t* const pairs = reinterpret_cast<uint16_t*>(sums + kLoraTile * (wide + 8));
  {
    const int64_t step = (int64_t)a.plan.tokens * rp;
    for (int i = threadIdx.x; i < tile.count * (wide / 4); i += 64 * kLoraWaves) {
      const int t = i / (wide / 4), r = (i - t * (wide / 4)) * 4;
      const float* const from = a.v + (int64_t)(tile.start + t) * rp + r;
      v4f_t s = *reinterpret_cast<const v4f_t*>(from);
#pragma unroll 7
      for (int p = 1; p < a.splits; ++p) s += *reinterpret_cast<const v4f_t*>(from + p * step);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (r + j >= rank) s[j] = 0.0f;
      *reinterpret_cast<v4f_t*>(sums + t * (wide + 8) + r) = s;
    }
  }
  __syncthreads();
  {
    const int t = threadIdx.x >> 3, sub = threadIdx.x & 7;
    const float* const from = sums + t * (wide + 8);
    const bool mine = t < tile.count;
    float top = 0.0f;
    for (int r = sub; r < wide; r += 8) {
      const float m = mine ? __builtin_fabsf(from[r]) : 0.0f;
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
    for (int r = sub; r < wide; r += 8) {
      const float v = mine ? from[r] * down : 0.0f;
      const T hi = from_f32<T>(v);
      const float rest = v - to_f32(hi);
      uint16_t* const at = pairs + t * pitch + r / GR * (2 * GR) + r % GR;
      at[0] = hi.bits;
      at[GR] = from_f32<T>(rest == rest ? rest : 0.0f).bits;   // (an infinite v has no low part)
    }
    if (sub == 0) factor[t] = a.scale[tile.adapter] * __uint_as_float((uint32_t)(127 - shift) << 23);
  }
  __syncthreads();

  v4f_t acc[2][2] = {};
  Raw8<T> old[2] = {};
  // A vector of b's ranks r .. r + 7 as read: what is beyond the rank is cleared (it may be anything, and meets zeros).  A row
  // of b that the vector would leave was read as its last 8.
  auto settled = [&](Raw8<T> w, int r) {
    const int from = a.rank < 8 ? 0 : r < a.rank - 8 ? r : a.rank - 8;
    if (r > from) w.w = shift_down(w.w, 16 * (r - from));
    const int n = rank - r;
#pragma unroll
    for (int j = 0; j < 4; ++j) w.w[j] &= (2 * j < n ? 0xFFFFu : 0u) | (2 * j + 1 < n ? 0xFFFF0000u : 0u);
    return w;
  };
  auto multiply = [&](int s, const Step& o) {
    const int turn = chunks == 1 ? s : s / chunks, chunk = s - turn * chunks;
    if (chunk == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        old[i] = o.old[i];
        acc[i][0] = acc[i][1] = v4f_t{0.0f, 0.0f, 0.0f, 0.0f};
      }
    }
#pragma unroll
    for (int k = 0; k < GN; ++k) {
      const int at = chunk * GN + k;
      if (at >= groups) break;
      Raw8<T> w[2] = {o.w[k][0], o.w[k][1]};
      if (at * GR + GR > rank) {
        w[0] = settled(w[0], rank_at(at));
        w[1] = settled(w[1], rank_at(at));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (i == 1 && !second) continue;
        const uint16_t* const from = pairs + (16 * i + row) * pitch + 2 * GR * at + 8 * part;
        // (of 16 ranks the lanes of the upper two parts hold the low parts)
        const v8s_t hi = *reinterpret_cast<const v8s_t*>(from);
        v8s_t lo;
        if constexpr (RB > 1) lo = *reinterpret_cast<const v8s_t*>(from + GR);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          acc[i][j] = mma16(T{}, as_lora(w[j]), hi, acc[i][j]);
          if constexpr (RB > 1) acc[i][j] = mma16(T{}, as_lora(w[j]), lo, acc[i][j]);
        }
      }
    }
    if (chunk + 1 < chunks) return;
    const int c = first + turn * 32 + 8 * part, left = n_end - c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!live[i] || left <= 0) continue;
      const float f = factor[16 * i + row];
      float was[8], sum[8];
      widen8f(old[i], was);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] = __builtin_fmaf(acc[i][j >> 2][j & 3], f, was[j]);
      store8(y + token[i] + c, left, sum);
    }
  };
  for (int s = 0; s < steps; s += DEPTH) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      if (s + d >= steps) break;
      multiply(s + d, ahead[d]);
      load(s + d + DEPTH, ahead[d]);
    }
  }
}

// Over how many ranges K is split: two workgroups for every compute unit, each of 512 or more of K (a step of its eight
// waves).  Every workgroup of the second kernel adds the ranges up: for four per compute unit 5003 tokens take 59 us, for
// two 55, for one 56 and ranks of 128 81 instead of 70.
struct LoraSplit {
  int splits, range;
};
static LoraSplit lora_split(int64_t tokens, int64_t K, int64_t rank, int64_t adapters) {
  const int64_t tiles = tokens / kLoraTile + std::min(tokens, adapters), groups = tiles * ((rank + 63) / 64);
  int64_t s = (2 * (int64_t)num_cus() + groups - 1) / groups;
  s = std::max<int64_t>(1, std::min<int64_t>({s, K / 512, kLoraSplits}));
  const int64_t range = round_up((K + s - 1) / s, 64);
  return {(int)((K + range - 1) / range), (int)range};
}

template <typename T>
static int run_lora(const LoraArgs& a, hipStream_t stream) {
  const char* what = "lora_add";
  const int rb = a.rank <= 16 ? 1 : a.rank <= 32 ? 2 : 4;
  const dim3 block(64 * kLoraWaves);
  const dim3 down((unsigned)(a.most * a.splits), (unsigned)((a.rank + 16 * rb - 1) / (16 * rb)));
  if (rb == 1) hipLaunchKernelGGL((k_lora_down<T, 1>), down, dim3(64 * kDownWaves), 0, stream, a);
  else if (rb == 2) hipLaunchKernelGGL((k_lora_down<T, 2>), down, dim3(64 * kDownWaves), 0, stream, a);
  else hipLaunchKernelGGL((k_lora_down<T, 4>), down, dim3(64 * kDownWaves), 0, stream, a);
  const int rc = check_launch(what);
  if (rc) return rc;
  const dim3 up((unsigned)((a.N + kLoraChannels - 1) / kLoraChannels), (unsigned)std::min(a.most, kLoraGridY),
                (unsigned)((a.most + kLoraGridY - 1) / kLoraGridY));
  const size_t wide = lora_pitch(a.rank), lds = kLoraTile * ((wide + 8) * 4 + (wide * 2 + 8) * 2);
  if (rb == 1) hipLaunchKernelGGL((k_lora_up<T, 1, 4>), up, block, lds, stream, a);
  else if (rb == 2) hipLaunchKernelGGL((k_lora_up<T, 2, 4>), up, block, lds, stream, a);
  else hipLaunchKernelGGL((k_lora_up<T, 4, 2>), up, block, lds, stream, a);
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
  return (int64_t)lora_split(tokens, K, rank, adapters).splits * tokens * lora_pitch((int)rank) * 4;
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
  g.most = (int)lora_most_tiles(tokens, adapters);
  return dt == FP8DP_BF16 ? run_lora<bf16_t>(g, stream) : run_lora<f16_t>(g, stream);
}
