// mma16.hpp -- matrix products of 16-bit operands in LDS tiles (gfx950), for operands whose
// contraction runs along rows or down columns.
//
//   C[m, n] = sum over k of A(m, k) B(n, k)
//
// An operand lies "along" (a row of m holds its k) or "down" (a row of k holds its m).  K advances
// 64 values a stage.  In LDS a tile that lies along has rows of 128 bytes, swizzled as gemm_core.hpp
// describes; one that lies down keeps its rows of k, and the transposing LDS read (16 lanes
// read 4 rows of 16 values, each lane gets a column) makes fragments of it, so that no operand
// is transposed in memory.  Its 16-byte chunks are swizzled so that the 4 rows x 64 bytes that half a wave
// reads at once are in different banks.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gemm_core.hpp"
#include "row_core.hpp"

namespace fp8dp {

typedef __bf16 v8bf16_t __attribute__((ext_vector_type(8)));
typedef _Float16 v8f16_t __attribute__((ext_vector_type(8)));
typedef short v4s_t __attribute__((ext_vector_type(4)));
typedef short v8s_t __attribute__((ext_vector_type(8)));
typedef float v4f_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v16f_t mma32(bf16_t, v8s_t a, v8s_t b, v16f_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf16_t, a),
                                                 __builtin_bit_cast(v8bf16_t, b), c, 0, 0, 0);
}
__device__ __forceinline__ v16f_t mma32(f16_t, v8s_t a, v8s_t b, v16f_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8f16_t, a),
                                                __builtin_bit_cast(v8f16_t, b), c, 0, 0, 0);
}
__device__ __forceinline__ v4f_t mma16(bf16_t, v8s_t a, v8s_t b, v4f_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf16_t, a),
                                                 __builtin_bit_cast(v8bf16_t, b), c, 0, 0, 0);
}
__device__ __forceinline__ v4f_t mma16(f16_t, v8s_t a, v8s_t b, v4f_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8f16_t, a),
                                                __builtin_bit_cast(v8f16_t, b), c, 0, 0, 0);
}

constexpr int kStageK = 64;   // values of K per stage

// What chunks past an operand's end are copied from.
__device__ const u32x4_t kZeroChunk16 = {0, 0, 0, 0};

// Lane i's 16 bytes at base + off[i] land at l + 16 i, the base in scalar registers.
__device__ __forceinline__ void copy16_to_lds_from(const void* base, uint32_t off, uint8_t* l) {
  const uint32_t la = (uint32_t)(uintptr_t)(lds_void_t*)l;
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(off), "s"(base), "{m0}"(la) : "memory");
}

// An operand of a product: `rows` of the output's dimension, in one piece or in two.
//   along: row r at p[piece] + r ld; DUAL: a tile's rows alternate between the pieces, 32 of each.
//   down: row k of a piece at p[piece] + k ld.
// K in two pieces: p[1] holds the second half of its stages.  ld in elements.
struct Operand {
  const uint16_t* p[2];
  int64_t ld;
  int rows;
};

struct MmaArgs {
  Operand a, b;
  int seg_stages;        // stages per piece of K (all of them where K is in one piece)
  int valid_a, valid_b;  // k of a piece that count, the others are zeros
  int stages;            // of all pieces
  int tiles_m, tiles_n;
  int first = 0;         // tile of workgroup 0
};

// Byte of 16-byte chunk c of row k of a tile that lies down, R rows of the output's dimension wide.
template <int R>
__device__ __forceinline__ int down_swizzle(int k) {
  return R % 128 == 0 ? (k & 3) << 2 : ((k >> 1) & 1) << 2;
}
template <int R>
__device__ __forceinline__ int down_at(int k, int c) {
  return k * (R * 2) + ((c ^ down_swizzle<R>(k)) << 4);
}

// Moves tiles of R x 64 values into LDS with W waves.  DIRECT: rows start at multiples of 16 bytes
// and are whole chunks, copied without passing registers; else through registers at any alignment.
template <typename T, int R, int W, bool DOWN, bool DUAL, bool DIRECT>
struct Loader {
  static constexpr int SIZE = R * 128;             // bytes of a tile
  static constexpr int L = SIZE / 1024 / W;        // copies of a wave per stage
  static_assert(SIZE % (1024 * W) == 0 && !(DUAL && DOWN), "whole copies");
  uint32_t off[L];                                 // bytes from the stage's base
  Raw8<T> reg[DIRECT ? 1 : L];
  int cut[DIRECT ? 1 : L];                         // elements of the chunk inside the row (down)
  int wave, lane;

  __device__ __forceinline__ void init(const Operand& o, int r0, int wave_, int lane_) {
    wave = wave_;
    lane = lane_;
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int pos = (wave + W * i) * 64 + lane;   // chunk of the tile in LDS
      if constexpr (DOWN) {
        constexpr int CH = R / 8;
        const int k = pos / CH, c = (pos % CH) ^ down_swizzle<R>(k);
        int m = r0 + c * 8;
        if constexpr (DIRECT) {
          if (m > o.rows - 8) m = o.rows - 8;      // (columns past the end are not stored)
        } else {
          cut[i] = o.rows - m;
          if (m > o.rows - 8) m = o.rows >= 8 ? o.rows - 8 : 0;
        }
        off[i] = (uint32_t)k * (uint32_t)(o.ld * 2) + (uint32_t)m * 2;
      } else {
        const int r = pos / 8, c = (pos % 8) ^ ((r >> 1) & 7);
        int m = DUAL ? r0 / 2 + (r >> 6) * 32 + (r & 31) : r0 + r;
        if (m > o.rows - 1) m = o.rows - 1;        // (rows past the end are not stored)
        // from the tile's first row, so that 32 bits hold it
        off[i] = (uint32_t)(m - (DUAL ? r0 / 2 : r0)) * (uint32_t)(o.ld * 2) + (uint32_t)c * 16;
      }
    }
  }
  // the tile's first row, or for DOWN the first column
  static __device__ __forceinline__ const uint8_t* base(const Operand& o, int piece, int r0, int k) {
    const uint16_t* const p = piece ? o.p[1] : o.p[0];
    if constexpr (DOWN) return reinterpret_cast<const uint8_t*>(p + (int64_t)k * o.ld);
    else return reinterpret_cast<const uint8_t*>(p + (int64_t)(DUAL ? r0 / 2 : r0) * o.ld + k);
  }
  // First k of copy i's chunk (along), or its row of k (down).  For the last stage only: the lane is
  // made opaque so that the result takes no registers in the loop.
  __device__ __forceinline__ int first_k(int i) const {
    int l = lane;
    asm volatile("" : "+v"(l));
    const int pos = (wave + W * i) * 64 + l;
    if constexpr (DOWN) return pos / (R / 8);
    else return ((pos % 8) ^ ((pos >> 4) & 7)) * 8;
  }
  // Which piece copy i's rows belong to (the same for its 8 rows, so for the wave).
  __device__ __forceinline__ int dual_piece(int i) const { return ((wave + W * i) >> 2) & 1; }

  // Stage at k of the piece, of which `left` values of K count (64 or more: all).
  __device__ __forceinline__ void copy(const Operand& o, int piece, int r0, int k, int left, uint8_t* slot) {
    static_for<L>([&](auto I) { copy_one<decltype(I)::value>(o, piece, r0, k, left, slot); });
  }
  template <int I>
  __device__ __forceinline__ void copy_one(const Operand& o, int piece, int r0, int k, int left,
                                           uint8_t* slot) {
    static_assert(DIRECT, "");
    const uint8_t* const b = base(o, DUAL ? dual_piece(I) : piece, r0, k);
    uint8_t* const l = slot + (wave + W * I) * 1024;
    if (left >= kStageK) {
      copy16_to_lds_from(b, off[I], l);
    } else {
      copy16_to_lds(first_k(I) < left ? b + off[I] : reinterpret_cast<const uint8_t*>(&kZeroChunk16), l);
    }
  }
  // The same through registers: fetch starts the loads, put stores them to LDS.
  __device__ __forceinline__ void fetch(const Operand& o, int piece, int r0, int k, int left) {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const uint8_t* const b = base(o, DUAL ? dual_piece(i) : piece, r0, k);
      if constexpr (DOWN) {
        const T* const p = reinterpret_cast<const T*>(b + off[i]);
        if (first_k(i) >= left) {
          reg[i] = Raw8<T>{};
        } else if (o.rows >= 8) {
          reg[i] = load_raw8(p);
        } else {
          load_cut(p, o.rows, reg[i]);
        }
      } else {
        reg[i] = load_raw(reinterpret_cast<const T*>(b + off[i]), left - first_k(i));
      }
    }
  }
  __device__ __forceinline__ void put(const Operand& o, uint8_t* slot) {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      if constexpr (DOWN) {
        if (o.rows >= 8) settle(reg[i], cut[i]);
      }
      *reinterpret_cast<u32x4_t*>(slot + (wave + W * i) * 1024 + lane * 16) =
          u32x4_t{reg[i].w[0], reg[i].w[1], reg[i].w[2], reg[i].w[3]};
    }
  }
};

// Fragment of 32 rows (tile `ti` of 32) and 16 values of K (step q of 4) of a tile of R rows at `slot`:
// lane l holds row l % 32 and k 8 (l / 32) .. + 7.
template <int R, bool DOWN>
__device__ __forceinline__ v8s_t fragment(const uint8_t* slot, int ti, int q, int lane) {
  if constexpr (DOWN) {
    typedef __attribute__((address_space(3))) v4s_t lds_v4s_t;
    const int p = lane & 15;
    const int k = 8 * (lane >> 5) + (p >> 2), c = 4 * ti + 2 * ((lane >> 4) & 1) + ((p & 3) >> 1);
    const uint8_t* const at = slot + down_at<R>(k, c) + (p & 1) * 8 + q * 16 * R * 2;
    const v4s_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t*)at);
    const v4s_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t*)(at + 4 * R * 2));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  } else {
    return *reinterpret_cast<const v8s_t*>(slot + swz(32 * ti + (lane & 31), 2 * q + (lane >> 5)));
  }
}

// ------------------------------------------------------------------ the product
// A workgroup of WM x WN waves owns BM x BN outputs, a wave TM x TN tiles of 32 x 32.  The product is
// issued with B first, so a lane holds one m and register r the n 8 (r / 4) + 4 (lane / 32) + r % 4.
// gridDim.y > 1: workgroup (t, s) takes the s-th range of stages.
// out(acc, lds of the wave, m of the wave, n of the wave, split): stores the tile.
//
// DIRECT: two LDS slots filled by copies that pass no registers.  A stage goes in halves, with
// fragments double-buffered: the first half of a stage is multiplied while its second is read, then one barrier
// shows that all copies of the next stage have landed and that this slot has been read; the second
// half is multiplied while the slot is refilled and the next stage's first half is read.
// Else: loads of the next stage travel in registers while one is multiplied.
template <typename T, int WM, int WN, int TM, int TN, bool ADOWN, bool BDOWN, bool DUAL, bool DIRECT,
          typename Out>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_mma(MmaArgs g, Out out) {
  constexpr int W = WM * WN, BM = WM * TM * 32, BN = WN * TN * 32;
  using LoadA = Loader<T, BM, W, ADOWN, false, DIRECT>;
  using LoadB = Loader<T, BN, W, BDOWN, DUAL, DIRECT>;
  constexpr int SLOT = LoadA::SIZE + LoadB::SIZE, NCOPY = LoadA::L + LoadB::L;
  constexpr int kTurn = 32 * 32 * TN * 4;   // bytes of a wave's part of LDS for the outputs
  constexpr int LDS = 2 * SLOT > W * kTurn ? 2 * SLOT : W * kTurn;
  __shared__ __attribute__((aligned(16))) uint8_t lds[LDS];

  const int ntiles = g.tiles_m * g.tiles_n;
  const int tile = tile_of_block(g.first + (int)blockIdx.x, ntiles);
  // bands 4 tiles wide: the 32 tiles that an XCD has in hand are 8 x 4, whose operands are 12 tiles
  const int band = tile / (4 * g.tiles_m), in_band = tile - band * 4 * g.tiles_m;
  const int wide = g.tiles_n - band * 4 < 4 ? g.tiles_n - band * 4 : 4;
  const int m0 = in_band / wide * BM, n0 = (band * 4 + in_band % wide) * BN;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / WN * TM, wc = wave % WN * TN;   // in tiles of 32
  const int begin = (int)((int64_t)g.stages * blockIdx.y / gridDim.y);
  const int end = (int)((int64_t)g.stages * (blockIdx.y + 1) / gridDim.y);

  LoadA la;
  LoadB lb;
  la.init(g.a, m0, wave, lane);
  lb.init(g.b, n0, wave, lane);
  struct At {
    int piece, k;
  };
  auto at = [&](int kt) -> At {
    const int piece = kt >= g.seg_stages;
    return {piece, (kt - (piece ? g.seg_stages : 0)) * kStageK};
  };

  v16f_t acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  if constexpr (DIRECT) {
    // fragments of two of a stage's four steps: one read of the 2 (TM + TN)
    struct Frags {
      v8s_t a[2][TM], b[2][TN];
    };
    auto read_one = [&](auto X, const uint8_t* slot, int h, Frags& f) {
      constexpr int x = decltype(X)::value, q = x / (TM + TN), i = x % (TM + TN);
      if constexpr (i < TM) f.a[q][i] = fragment<BM, ADOWN>(slot, wr + i, 2 * h + q, lane);
      else f.b[q][i - TM] = fragment<BN, BDOWN>(slot + LoadA::SIZE, wc + i - TM, 2 * h + q, lane);
    };
    constexpr int READS = 2 * (TM + TN), PRODUCTS = 2 * TM * TN;
    constexpr int EACH = (READS + PRODUCTS - 1) / PRODUCTS, CEACH = (NCOPY + PRODUCTS - 1) / PRODUCTS;
    // the products of a half stage, with between(0), between(1), ... after one each: reads and copies
    // issue while a product runs
    auto multiply = [&](const Frags& f, auto&& between) {
      static_for<PRODUCTS>([&](auto X) {
        constexpr int x = decltype(X)::value, q = x / (TM * TN), i = x / TN % TM, j = x % TN;
        acc[i][j] = mma32(T{}, f.b[q][j], f.a[q][i], acc[i][j]);
        between(X);
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    auto issue = [&](int kt) {
      const At s = at(kt);
      uint8_t* const slot = lds + ((kt - begin) & 1) * SLOT;
      la.copy(g.a, s.piece, m0, s.k, g.valid_a - s.k, slot);
      lb.copy(g.b, s.piece, n0, s.k, g.valid_b - s.k, slot + LoadA::SIZE);
    };
    // the first stage from begin + 2 on that is not whole, or the end: the last one of a piece
    const int least = g.valid_a < g.valid_b ? g.valid_a : g.valid_b;
    int whole = end;
    if (least < g.seg_stages * kStageK) {
      const int last = begin + 2 < g.seg_stages ? g.seg_stages - 1 : g.stages - 1;
      if (last < whole) whole = last;
    }
    if (begin < end) issue(begin);
    if (begin + 1 < end) issue(begin + 1);
    if (begin + 1 < end) wait_vmcnt<NCOPY>();
    else wait_vmcnt<0>();
    stage_barrier();
    Frags f0, f1;
    if (begin < end) static_for<READS>([&](auto X) { read_one(X, lds, 0, f0); });
    // one stage; COPY: the stage two later is whole and copied between the products (else ahead of
    // them); NEXT: there is a next stage
    auto stage = [&](int kt, auto COPY, auto NEXT) {
      constexpr bool copy = decltype(COPY)::value, next = decltype(NEXT)::value;
      uint8_t* const slot = lds + ((kt - begin) & 1) * SLOT;
      const uint8_t* const after = lds + ((kt + 1 - begin) & 1) * SLOT;
      auto reads = [&](auto X, const uint8_t* from, int h, Frags& f) {
        static_for<EACH>([&](auto E) {
          constexpr int x = decltype(X)::value * EACH + decltype(E)::value;
          if constexpr (x < READS) read_one(std::integral_constant<int, x>{}, from, h, f);
        });
      };
      multiply(f0, [&](auto X) { reads(X, slot, 1, f1); });
      __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): this wave's reads of the stage are done
      wait_vmcnt<0>();                      // its copies of the next one have landed
      stage_barrier();
      const At s = at(kt + 2);
      if constexpr (!copy) {
        if (kt + 2 < end) issue(kt + 2);
      }
      multiply(f1, [&](auto X) {
        if constexpr (next) reads(X, after, 0, f0);
        if constexpr (copy) {
          static_for<CEACH>([&](auto E) {
            constexpr int c = decltype(X)::value * CEACH + decltype(E)::value;
            if constexpr (c < LoadA::L)
              la.template copy_one<c>(g.a, s.piece, m0, s.k, kStageK, slot);
            else if constexpr (c < NCOPY)
              lb.template copy_one<c - LoadA::L>(g.b, s.piece, n0, s.k, kStageK, slot + LoadA::SIZE);
          });
        }
      });
    };
    using yes = std::true_type;
    using no = std::false_type;
    int kt = begin;
    for (; kt < whole - 2; ++kt) stage(kt, yes{}, yes{});
    for (; kt + 1 < end; ++kt) stage(kt, no{}, yes{});
    if (kt < end) stage(kt, no{}, no{});
  } else {
    auto fetch = [&](int kt) {
      const At s = at(kt);
      la.fetch(g.a, s.piece, m0, s.k, g.valid_a - s.k);
      lb.fetch(g.b, s.piece, n0, s.k, g.valid_b - s.k);
    };
    auto put = [&](int kt) {
      uint8_t* const slot = lds + ((kt - begin) & 1) * SLOT;
      la.put(g.a, slot);
      lb.put(g.b, slot + LoadA::SIZE);
    };
    if (begin < end) {
      fetch(begin);
      put(begin);
    }
    __syncthreads();
    for (int kt = begin; kt < end; ++kt) {
      if (kt + 1 < end) fetch(kt + 1);
      const uint8_t* const slot = lds + ((kt - begin) & 1) * SLOT;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v8s_t fa[TM], fb[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[i] = fragment<BM, ADOWN>(slot, wr + i, q, lane);
#pragma unroll
        for (int j = 0; j < TN; ++j) fb[j] = fragment<BN, BDOWN>(slot + LoadA::SIZE, wc + j, q, lane);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[i][j] = mma32(T{}, fb[j], fa[i], acc[i][j]);
      }
      if (kt + 1 < end) put(kt + 1);
      __syncthreads();
    }
  }
  // (all waves have read their last fragments: of DIRECT after the last stage's barrier nothing is read)
  out(acc, lds + wave * kTurn, m0 + wr * 32, n0 + wc * 32, lane, (int)blockIdx.y);
}

// Turns 32 rows x 32 JT columns of a wave through its part of LDS: value(j, r) is register r of column
// tile j in the layout above; emit(row, column, v) gets 8 consecutive columns, so that rows are
// stored in whole cache lines.  16-byte chunks are swizzled by row against bank conflicts.
template <int JT, typename Value, typename Emit>
__device__ __forceinline__ void turn_tile(uint8_t* part, int lane, Value&& value, Emit&& emit) {
  constexpr int CW = JT * 32, LPR = CW / 8;   // columns, lanes per row
  auto at = [&](int r, int c) {               // byte of chunk c (4 columns) of row r
    return r * CW * 4 + ((c ^ (JT == 1 ? (r >> 1) & 7 : JT == 3 ? r & 7 : r & 15)) << 4);
  };
  const int frow = lane & 31, fhalf = lane >> 5;
#pragma unroll
  for (int j = 0; j < JT; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v4f_t v;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = value(j, 4 * q + r);
      *reinterpret_cast<v4f_t*>(part + at(frow, j * 8 + 2 * q + fhalf)) = v;
    }
#pragma unroll
  for (int s = 0; s < LPR / 2; ++s) {
    const int x = s * 64 + lane, r = x / LPR, c = x % LPR * 2;
    const v4f_t lo = *reinterpret_cast<const v4f_t*>(part + at(r, c));
    const v4f_t hi = *reinterpret_cast<const v4f_t*>(part + at(r, c + 1));
    const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    emit(r, c * 4, v);
  }
}

// A launch has at most 2^32 - 1 threads; launch(first, count) in parts of a multiple of 8 tiles.
template <typename F>
inline int for_tiles(int64_t tiles, F&& launch) {
  constexpr int64_t kMost = (int64_t)1 << 22;
  for (int64_t first = 0; first < tiles; first += kMost) {
    const int rc = launch((int)first, (unsigned)std::min(tiles - first, kMost));
    if (rc) return rc;
  }
  return FP8DP_OK;
}

}  // namespace fp8dp
