// int8_tile.hip -- the INT8 product in LDS tiles, for operands whose rows start at
// multiples of 16 bytes (K itself a multiple of 16).
//
// A workgroup of WM x WN waves owns BM x BN outputs; a wave TM x TN tiles of
// the 32 x 32 x 32 matrix instruction.  K advances 128 bytes per stage through a
// ring of S slots in LDS, which global_load_lds fills without passing registers
// (16-byte chunks swizzled as gemm_core.hpp describes, so that fragment reads
// meet no bank twice).  Software pipeline by half stages, fragments
// double-buffered: the first half of a stage reads its second 64 bytes of K while
// the first are multiplied; then one barrier shows that every wave's copies of
// the next stage have landed and that this stage's slot has been read; the
// second half refills the slot, reads the next stage's first 64 bytes and
// multiplies the second.
// Rows past M or N are read as the last row and not stored; chunks past K come as
// zeros for the tokens and as any chunk of the row for the weight.
#include <hip/hip_runtime.h>

#include "int8_core.hpp"
#include "int8_tile.hpp"

#include <type_traits>

namespace fp8dp {

// Lane i's 16 bytes at base + off[i] land at l + 16 i; as copy16_to_lds, with
// the wave's base in scalar registers.
__device__ __forceinline__ void copy16_to_lds_at(const int8_t* base, uint32_t off, uint8_t* l) {
  const uint32_t la = (uint32_t)(uintptr_t)(lds_void_t*)l;
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(off), "s"(base), "{m0}"(la)
               : "memory");
}

template <typename T, int WM, int WN, int TM, int TN, int S>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_i8_tile(I8Args g) {
  constexpr int W = WM * WN, BM = WM * TM * 32, BN = WN * TN * 32;
  constexpr int ASZ = BM * kBK, SLOT = (BM + BN) * kBK;
  static_assert(W % 2 == 0, "the swizzle of a copy");
  constexpr int LA = BM / 8 / W, LB = BN / 8 / W, NCOPY = LA + LB;   // copies of a wave per stage
  __shared__ __attribute__((aligned(16))) uint8_t lds[S * SLOT + sizeof(TileScales<BM, BN>)];
  TileScales<BM, BN>& scales = *reinterpret_cast<TileScales<BM, BN>*>(lds + S * SLOT);

  const int tiles_n = (g.N + BN - 1) / BN;
  const int ntiles = ((g.M + BM - 1) / BM) * tiles_n;
  const int tile = tile_of_block(g.first + (int)blockIdx.x, ntiles);
  // bands 4 tiles wide: the 32 tiles that an XCD has in hand are 8 x 4, whose operands are 12
  // tiles in all, not 2 x 16
  const int tiles_m = (g.M + BM - 1) / BM, band = tile / (4 * tiles_m);
  const int in_band = tile - band * 4 * tiles_m, wide = tiles_n - band * 4 < 4 ? tiles_n - band * 4 : 4;
  const int m0 = in_band / wide * BM, n0 = (band * 4 + in_band % wide) * BN;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = (wave / WN) * TM * 32, wc = (wave % WN) * TN * 32;
  const int KT = (g.K + kBK - 1) / kBK;

  // copy i of this wave: rows 8 (wave + W i) .. + 7 of the tile, lane l the logical chunk that
  // swz() places at chunk l % 8 of row l / 8
  const int lrow = lane >> 3;
  const int8_t* const baseA = g.a + (int64_t)m0 * g.lda;
  const int8_t* const baseB = g.b + (int64_t)n0 * g.ldb;
  uint32_t offA[LA], offB[LB];
  // (r / 2) % 8 of row r = 8 (wave + W i) + l / 8 does not depend on i
  const int chunk = (lane & 7) ^ ((4 * wave + (lrow >> 1)) & 7);
#pragma unroll
  for (int i = 0; i < LA; ++i) {
    const int r = 8 * (wave + W * i) + lrow;
    offA[i] = (uint32_t)((r < g.M - m0 ? r : g.M - 1 - m0) * (uint32_t)g.lda + chunk * 16);
  }
#pragma unroll
  for (int i = 0; i < LB; ++i) {
    const int r = 8 * (wave + W * i) + lrow;
    offB[i] = (uint32_t)((r < g.N - n0 ? r : g.N - 1 - n0) * (uint32_t)g.ldb + chunk * 16);
  }
  auto issue = [&](int kt) {
    uint8_t* const base = lds + (kt % S) * SLOT + wave * 1024;
    const int k0 = kt * kBK;
    if (k0 + kBK <= g.K) {
#pragma unroll
      for (int i = 0; i < LA; ++i)
        copy16_to_lds_at(baseA + k0, offA[i], base + i * W * 1024);
#pragma unroll
      for (int i = 0; i < LB; ++i)
        copy16_to_lds_at(baseB + k0, offB[i], base + ASZ + i * W * 1024);
    } else {
      const int left = (g.K - k0) / 16;   // chunks of this stage inside K, 1 .. 7
#pragma unroll
      for (int i = 0; i < LA; ++i)
        copy16_to_lds(chunk < left
                          ? reinterpret_cast<const uint8_t*>(baseA + k0 + offA[i])
                          : reinterpret_cast<const uint8_t*>(&kZeroChunk),
                      base + i * W * 1024);
#pragma unroll
      for (int i = 0; i < LB; ++i)
        copy16_to_lds(reinterpret_cast<const uint8_t*>(
                          baseB + k0 + offB[i] - (chunk < left ? 0 : chunk * 16)),
                      base + ASZ + i * W * 1024);
    }
  };

  // one copy of a whole stage
  auto copy_one = [&](auto C, const int8_t* a, const int8_t* b, uint8_t* base) {
    constexpr int c = decltype(C)::value;
    if constexpr (c < LA) copy16_to_lds_at(a, offA[c], base + c * W * 1024);
    else copy16_to_lds_at(b, offB[c - LA], base + ASZ + (c - LA) * W * 1024);
  };

  // fragments of 64 bytes of K (half h of a stage) in two 32-byte steps: one read of the 2 (TM + TN)
  struct Frags {
    v4i_t a[2][TM], b[2][TN];
  };
  const int frow = lane & 31, fhalf = lane >> 5;
  auto read_one = [&](auto X, const uint8_t* slot, int h, Frags& f) {
    constexpr int x = decltype(X)::value, q = x / (TM + TN), i = x % (TM + TN);
    const int c = h * 4 + q * 2 + fhalf;
    if constexpr (i < TM)
      f.a[q][i] = *reinterpret_cast<const v4i_t*>(slot + swz(wr + 32 * i + frow, c));
    else
      f.b[q][i - TM] =
          *reinterpret_cast<const v4i_t*>(slot + ASZ + swz(wc + 32 * (i - TM) + frow, c));
  };
  constexpr int READS = 2 * (TM + TN), PRODUCTS = 2 * TM * TN;
  v16i_t acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
  // the products of a half stage, with between(0), between(1), ... after one each: reads and
  // copies issue while a product runs, instead of before the first one
  auto multiply = [&](const Frags& f, auto&& between) {
    static_for<PRODUCTS>([&](auto X) {
      constexpr int x = decltype(X)::value, q = x / (TM * TN), i = x / TN % TM, j = x % TN;
      acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.b[q][j], f.a[q][i], acc[i][j], 0, 0, 0);
      between(X);
      __builtin_amdgcn_sched_barrier(0);
    });
  };

#pragma unroll
  for (int s = 0; s < S; ++s)
    if (s < KT) issue(s);
  load_scales<T>(g, scales, m0, n0, threadIdx.x, 64 * W);
  if (KT >= S) wait_vmcnt<(S - 1) * NCOPY>();
  else wait_vmcnt<0>();
  stage_barrier();

  static_assert(READS <= PRODUCTS + 8 && NCOPY <= PRODUCTS, "what fits between the products");
  constexpr int EACH = (READS + PRODUCTS - 1) / PRODUCTS;   // reads after a product
  Frags f0, f1;
  static_for<READS>([&](auto X) { read_one(X, lds, 0, f0); });
  // one stage; COPY: the stage S later is whole and copied between the products (else, near the end of K,
  // ahead of them); NEXT: there is a next stage
  auto stage = [&](int kt, auto COPY, auto NEXT) {
    constexpr bool copy = decltype(COPY)::value, next = decltype(NEXT)::value;
    const uint8_t* const slot = lds + (kt % S) * SLOT;
    const uint8_t* const after = lds + ((kt + 1) % S) * SLOT;
    auto reads = [&](auto X, const uint8_t* from, int h, Frags& f) {
      static_for<EACH>([&](auto E) {
        constexpr int x = decltype(X)::value * EACH + decltype(E)::value;
        if constexpr (x < READS) read_one(std::integral_constant<int, x>{}, from, h, f);
      });
    };
    multiply(f0, [&](auto X) { reads(X, slot, 1, f1); });
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): this wave's reads of stage kt are done
    // its copies of stage kt + 1 have landed
    if (copy || kt + S - 1 < KT) wait_vmcnt<(S - 2) * NCOPY>();
    else wait_vmcnt<0>();
    stage_barrier();
    if constexpr (!copy) {
      if (kt + S < KT) issue(kt + S);
    }
    const int k0 = (kt + S) * kBK;
    uint8_t* const base = lds + (kt % S) * SLOT + wave * 1024;
    multiply(f1, [&](auto X) {
      if constexpr (next) reads(X, after, 0, f0);
      if constexpr (copy && decltype(X)::value < NCOPY) copy_one(X, baseA + k0, baseB + k0, base);
    });
  };
  using yes = std::true_type;
  using no = std::false_type;
  int kt = 0;
  for (; (kt + S + 1) * kBK <= g.K; ++kt) stage(kt, yes{}, yes{});
  for (; kt + 1 < KT; ++kt) stage(kt, no{}, yes{});
  stage(kt, no{}, no{});

  static_assert(W * 32 * TN * 128 <= S * SLOT, "the waves' parts fit the ring");
  turn_out<T>(g, acc, lds + wave * 32 * TN * 128, scales, m0, n0, wr, wc, lane);
}

template <typename T, int WM, int WN, int TM, int TN, int S>
static int launch_tile(const char* what, const I8Args& g, hipStream_t stream) {
  constexpr int BM = WM * TM * 32, BN = WN * TN * 32;
  const int64_t tiles = (((int64_t)g.M + BM - 1) / BM) * (((int64_t)g.N + BN - 1) / BN);
  return for_blocks(tiles, [&](int first, unsigned count) {
    I8Args part = g;
    part.first = first;
    hipLaunchKernelGGL((k_i8_tile<T, WM, WN, TM, TN, S>), dim3(count), dim3(64 * WM * WN), 0, stream, part);
    return check_launch(what);
  });
}

int tile_i8(const char* what, fp8dp_dtype yt, const I8Args& g, bool wide, hipStream_t stream) {
  auto run = [&](auto t) -> int {
    using T = decltype(t);
    return wide ? launch_tile<T, 4, 2, 2, 4, 2>(what, g, stream)
                : launch_tile<T, 2, 2, 2, 2, 2>(what, g, stream);
  };
  if (yt == FP8DP_BF16) return run(bf16_t{});
  if (yt == FP8DP_F16) return run(f16_t{});
  return run(float{});
}

}  // namespace fp8dp
