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

// The 16 x 16 x 32 instruction: its accumulators are read and written once per 32 k, those of 32 x 32 x 16 once per
// 16, and the matrix pipes are bound by power: bare loops of them on normal data reach 2.06 and 1.83 PFLOP/s.
__device__ __forceinline__ v4f_t mma16(bf16_t, v8s_t a, v8s_t b, v4f_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf16_t, a),
                                                 __builtin_bit_cast(v8bf16_t, b), c, 0, 0, 0);
}
__device__ __forceinline__ v4f_t mma16(f16_t, v8s_t a, v8s_t b, v4f_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8f16_t, a),
                                                __builtin_bit_cast(v8f16_t, b), c, 0, 0, 0);
}

constexpr int kStageK = 64;   // values of K per stage

// The value, of which the compiler knows nothing: what is computed from it is not moved out of a loop, where it would
// take registers from the products.
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

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
  int tiles_m, tiles_n, splits;
  int first = 0;         // piece of work of workgroup 0
};

// Byte of 16-byte chunk c of row k of a tile that lies down, R rows of the output's dimension wide.
template <int R>
__device__ __forceinline__ int down_swizzle(int k) {
  return (R % 128 == 0 ? (k & 3) << 2 : ((k >> 1) & 1) << 2) | ((k >> 3) & 1) << 1;
}
template <int R>
__device__ __forceinline__ int down_at(int k, int c) {
  return k * (R * 2) + ((c ^ down_swizzle<R>(k)) << 4);
}

// Where a wave's copies of a tile's stage come from: the tile's first row of each piece (down: k = 0) and the
// bytes to the next k, held in scalar registers.  (Read from the arguments by the piece's number they came as scalar
// loads in the loop, each of which waited for all LDS reads under way.)
template <int W, bool DOWN, bool DUAL>
struct Source {
  const uint8_t* base;
  int64_t second, per_k;   // bytes from the first piece to the second, and to the next k
  int wave;
  __device__ __forceinline__ void init(const Operand& o, int r0, int wave_) {
    wave = wave_;
    const int64_t skip = DOWN ? 0 : (int64_t)(DUAL ? r0 / 2 : r0) * o.ld * 2;
    base = reinterpret_cast<const uint8_t*>(o.p[0]) + skip;
    second = reinterpret_cast<const uint8_t*>(o.p[1]) - reinterpret_cast<const uint8_t*>(o.p[0]);
    per_k = DOWN ? o.ld * 2 : 2;
  }
  // Copy i's base at k of a piece.  DUAL: a copy's 8 rows are all of one piece.
  __device__ __forceinline__ const uint8_t* at(int i, int piece, int k, int64_t more = 0) const {
    const int64_t which = DUAL ? ((wave + W * i) >> 2) & 1 : piece;
    return base + ((-which & second) + k * per_k + more);
  }
};

// Moves tiles of R x 64 values into LDS with W waves, L copies of 1 KiB a wave and stage.
// DIRECT: rows start at multiples of 16 bytes and are whole chunks, copied without passing registers.  Along, rows past
// the end are read as the last one; down, columns past the end are read as the last chunk.  Neither is stored.
template <typename T, int R, int W, bool DOWN, bool DUAL, bool DIRECT>
struct Loader {
  static constexpr int SIZE = R * 128, L = SIZE / 1024 / W, CH = R / 8;
  static constexpr bool EVEN = DOWN && 64 * W % CH == 0;   // copies are a fixed number of whole rows of k apart
  static_assert(DIRECT && SIZE % (1024 * W) == 0 && (W == 4 || W == 8) && !(DUAL && DOWN), "whole copies");
  const uint8_t *base, *here;    // of the tile, and of the stage to be copied
  int64_t second, per_k;         // bytes from the first piece to the second, and to the next k
  uint32_t off[EVEN ? 1 : L];
  int wave, lane;

  __device__ __forceinline__ void init(const Operand& o, int r0, int wave_, int lane_) {
    wave = wave_;
    lane = lane_;
    const int l = opaque(lane_);
    const uint32_t row = (uint32_t)(o.ld * 2);
    per_k = DOWN ? o.ld * 2 : 2;
    base = reinterpret_cast<const uint8_t*>(o.p[0]);
    second = reinterpret_cast<const uint8_t*>(o.p[1]) - base;
    if constexpr (DOWN) {
#pragma unroll
      for (int i = 0; i < (EVEN ? 1 : L); ++i) {
        const int pos = (wave + W * i) * 64 + l, k = pos / CH;
        const int m = r0 + ((pos % CH) ^ down_swizzle<R>(k)) * 8;
        off[i] = (uint32_t)k * row + (uint32_t)(m > o.rows - 8 ? o.rows - 8 : m) * 2;
      }
    } else {
      const int first = DUAL ? r0 / 2 : r0, most = o.rows - 1 - first;
      base += (int64_t)first * o.ld * 2;
      // a copy's 8 rows are all of one piece: of eight waves the upper four have the second's, of four the odd copies
      if (DUAL && W == 8) base += (wave >> 2) * second;
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const int pos = (wave + W * i) * 64 + l, r = pos / 8, m = DUAL ? (r >> 6) * 32 + (r & 31) : r;
        off[i] = (uint32_t)(m > most ? most : m) * row + (uint32_t)((pos % 8) ^ ((r >> 1) & 7)) * 16;
      }
    }
  }
  // On to the stage at k of a piece, and to the one behind it.
  __device__ __forceinline__ void go(int piece, int k) { here = base + (DUAL ? 0 : piece * second) + k * per_k; }
  __device__ __forceinline__ void step() { here += kStageK * per_k; }
  // First k of copy i's chunk (along), or its row of k (down).
  __device__ __forceinline__ int first_k(int i) const {
    const int pos = (wave + W * i) * 64 + opaque(lane);
    if constexpr (DOWN) return pos / CH;
    else return ((pos % 8) ^ ((pos >> 4) & 7)) * 8;
  }
  // Copy I of the stage, of which `left` values of K count (64 or more: all).
  template <int I>
  __device__ __forceinline__ void copy_one(int left, uint8_t* slot) {
    const uint8_t* b = here;
    if constexpr (DUAL && W == 4) b += I % 2 * second;
    if constexpr (EVEN) b += I * (64 * W / CH) * per_k;
    const uint32_t from = off[EVEN ? 0 : I];
    uint8_t* const l = slot + (wave + W * I) * 1024;
    if (left >= kStageK) {
      copy16_to_lds_from(b, from, l);
    } else {
      copy16_to_lds(first_k(I) < left ? b + from : reinterpret_cast<const uint8_t*>(&kZeroChunk16), l);
    }
  }
  __device__ __forceinline__ void copy(int left, uint8_t* slot) {
    static_for<L>([&](auto I) { copy_one<decltype(I)::value>(left, slot); });
  }
};

// The same through registers at any alignment: fetch starts the loads, put stores them to LDS.
template <typename T, int R, int W, bool DOWN, bool DUAL>
struct Loader<T, R, W, DOWN, DUAL, false> {
  static constexpr int SIZE = R * 128, L = SIZE / 1024 / W, CH = R / 8;
  static_assert(SIZE % (1024 * W) == 0 && !(DUAL && DOWN), "whole copies");
  Source<W, DOWN, DUAL> source;
  uint32_t off[L];   // bytes from the stage's base
  int cut[L];        // down: elements of the chunk inside the row
  Raw8<T> reg[L];
  int lane;

  __device__ __forceinline__ void init(const Operand& o, int r0, int wave, int lane_) {
    source.init(o, r0, wave);
    lane = lane_;
    const uint32_t row = (uint32_t)(o.ld * 2);
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int pos = (wave + W * i) * 64 + lane;
      if constexpr (DOWN) {
        const int k = pos / CH, m = r0 + ((pos % CH) ^ down_swizzle<R>(k)) * 8, most = o.rows >= 8 ? o.rows - 8 : 0;
        cut[i] = o.rows - m;
        off[i] = (uint32_t)k * row + (uint32_t)(m > most ? most : m) * 2;
      } else {
        const int r = pos / 8, first = DUAL ? r0 / 2 : r0, c = (pos % 8) ^ ((r >> 1) & 7);
        const int m = DUAL ? (r >> 6) * 32 + (r & 31) : r, most = o.rows - 1 - first;
        off[i] = (uint32_t)(m > most ? most : m) * row + (uint32_t)c * 16;
      }
    }
  }
  __device__ __forceinline__ int first_k(int i) const {
    const int pos = (source.wave + W * i) * 64 + lane;
    if constexpr (DOWN) return pos / CH;
    else return ((pos % 8) ^ ((pos >> 4) & 7)) * 8;
  }
  __device__ __forceinline__ void fetch(const Operand& o, int piece, int k, int left) {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const T* const p = reinterpret_cast<const T*>(source.at(i, piece, k) + off[i]);
      if constexpr (DOWN) {
        if (first_k(i) >= left) {
          reg[i] = Raw8<T>{};
        } else if (o.rows >= 8) {
          reg[i] = load_raw8(p);
        } else {
          load_cut(p, o.rows, reg[i]);
        }
      } else {
        reg[i] = load_raw(p, left - first_k(i));
      }
    }
  }
  __device__ __forceinline__ void put(const Operand& o, uint8_t* slot) {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      if constexpr (DOWN) {
        if (o.rows >= 8) settle(reg[i], cut[i]);
      }
      *reinterpret_cast<u32x4_t*>(slot + (source.wave + W * i) * 1024 + lane * 16) =
          u32x4_t{reg[i].w[0], reg[i].w[1], reg[i].w[2], reg[i].w[3]};
    }
  }
};

// Fragments of 16 rows and 32 values of K (half h of a stage): lane l holds row l % 16 and k 8 (l / 16) .. + 7.
// start() is the LDS address of a wave's first tile (of 16 rows, tile t0 of the workgroup's R / 16) in the tile at `slot`;
// read() that of its j-th.  The offsets are constants, or one exclusive-or away.
typedef __attribute__((address_space(3))) v4s_t lds_v4s_t;
typedef __attribute__((address_space(3))) v8s_t lds_v8s_t;
template <int R, bool DOWN>
struct Fragments {
  static __device__ __forceinline__ uint32_t start(const uint8_t* slot, int t0, int h, int lane) {
    const uint32_t at = (uint32_t)(uintptr_t)(lds_void_t*)slot;
    if constexpr (DOWN) {
      const int p = lane & 15, k = 8 * (lane >> 4) + (p >> 2);
      const uint32_t lead = at + (h * 32 + k) * (R * 2) + (down_swizzle<R>(k) << 4) + ((p & 3) >> 1) * 16 + (p & 1) * 8;
      return R % 128 == 0 ? lead ^ (uint32_t)(t0 << 5) : lead;
    } else {
      return at + swz(16 * t0 + (lane & 15), 4 * h + (lane >> 4));
    }
  }
  static __device__ __forceinline__ v8s_t read(uint32_t start, int t0, int j) {
    if constexpr (DOWN) {
      // (a slot is a multiple of a row of k and of 512 bytes; rows of 192 values are not: there the swizzle stays within 128)
      uint32_t at;
      if constexpr (R % 128 == 0) at = start ^ (uint32_t)(j << 5);
      else at = (start ^ (uint32_t)(((t0 + j) & 3) << 5)) + (uint32_t)((t0 + j) >> 2) * 128;
      const v4s_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t*)(uintptr_t)at);
      const v4s_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t*)(uintptr_t)(at + 4 * R * 2));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      return *(const lds_v8s_t*)(uintptr_t)(start + j * 2048);
    }
  }
};

// ------------------------------------------------------------------ the product
// A workgroup of WM x WN waves owns BM x BN outputs, a wave 16 TM x 16 TN as tiles of 16 x 16.  The product is
// issued with B first, so a lane holds m lane % 16 of a tile, and register r its n 4 (lane / 16) + r.
// A piece of work is a tile and a range of K, of which there are `splits`.
// out(acc, LDS of the wave, m of the wave, n of the wave, lane, split): stores the tile.
//
// DIRECT: S LDS slots filled by copies that pass no registers, two for the large tiles (64 KiB a stage), four where a
// compute unit has one small tile and its stages would wait for memory.  A stage goes in halves, with
// fragments double-buffered: the first half of a stage is multiplied while its second is read, then one barrier
// shows that all copies of the next stage have landed and that this slot has been read; the second
// half is multiplied while the slot is refilled and the next stage's first half is read.  The copies are
// spread over the half: the compute unit takes one in 16 cycles, and eight waves that issue theirs
// at once wait for each other.
// The grid is resident: a workgroup goes from one piece of work to the next in one pipeline, the last stages
// of one refill the slots with the first of the next, so that its outputs are stored while they travel (outputs have
// LDS of their own).  Stores count like copies where a wave waits for its copies: the ones under way before the outputs
// are waited for ahead of the first store, and the first stage behind the outputs waits for none.
// Else: loads of the next stage travel in registers while one is multiplied, a workgroup per piece of work.
constexpr int kOutBytes = 4096;   // a wave's LDS for its outputs

// Piece of work `i` of `n` in the order of workgroups b = i % grid: each XCD (workgroup b runs on XCD b % 8)
// has consecutive ones in hand, of the last, cut pass too where that is a multiple of 8.
__device__ __forceinline__ int work_of(int i, int n, int grid) {
  const int pass = i / grid, b = i - pass * grid, left = n - pass * grid < grid ? n - pass * grid : grid;
  return pass * grid + (left % 8 == 0 ? b % 8 * (left / 8) + b / 8 : b);
}

template <typename T, int WM, int WN, int TM, int TN, int S, bool ADOWN, bool BDOWN, bool DUAL, bool DIRECT,
          typename Out>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_mma(MmaArgs g, Out out) {
  constexpr int W = WM * WN, BM = WM * TM * 16, BN = WN * TN * 16;
  using LoadA = Loader<T, BM, W, ADOWN, false, DIRECT>;
  using LoadB = Loader<T, BN, W, BDOWN, DUAL, DIRECT>;
  constexpr int SLOT = LoadA::SIZE + LoadB::SIZE, NCOPY = LoadA::L + LoadB::L;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S * SLOT + W * kOutBytes];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / WN * TM, wc = wave % WN * TN;   // in tiles of 16
  uint8_t* const part = lds + S * SLOT + wave * kOutBytes;
  const int ntiles = g.tiles_m * g.tiles_n, total = ntiles * g.splits;

  struct Work {
    int m0, n0, begin, end, split;
  };
  auto work = [&](int i) -> Work {
    const int w = work_of(i, total, DIRECT ? (int)gridDim.x : total);
    const int split = w / ntiles, tile = w - split * ntiles;
    // bands 4 tiles wide: the 32 tiles that an XCD has in hand are 8 x 4, whose operands are 12 tiles
    const int band = tile / (4 * g.tiles_m), in_band = tile - band * 4 * g.tiles_m;
    const int wide = g.tiles_n - band * 4 < 4 ? g.tiles_n - band * 4 : 4;
    // (divisions leave their results in vector registers)
    auto s = [](int v) { return (int)__builtin_amdgcn_readfirstlane(v); };
    const int each = g.stages / g.splits, more = g.stages - each * g.splits;   // the first `more` ranges have one more
    const int begin = split * each + (split < more ? split : more);
    return {s(in_band / wide * BM), s((band * 4 + in_band % wide) * BN), s(begin),
            s(begin + each + (split < more ? 1 : 0)), s(split)};
  };
  struct At {
    int piece, k;
  };
  auto at = [&](int kt) -> At {
    const int piece = kt >= g.seg_stages;
    return {piece, (kt - (piece ? g.seg_stages : 0)) * kStageK};
  };

  LoadA la;
  LoadB lb;
  v4f_t acc[TM][TN];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = v4f_t{0.0f, 0.0f, 0.0f, 0.0f};
  };
  clear();

  if constexpr (DIRECT) {
    // fragments of half a stage: one read of the TM + TN
    using FragA = Fragments<BM, ADOWN>;
    using FragB = Fragments<BN, BDOWN>;
    struct Frags {
      v8s_t a[TM], b[TN];
    };
    // addresses of the second halves in the slot in hand, and of the first halves in the next one
    uint32_t a1 = FragA::start(lds, wr, 1, lane), b1 = FragB::start(lds + LoadA::SIZE, wc, 1, lane);
    uint32_t a0 = FragA::start(lds + SLOT, wr, 0, lane), b0 = FragB::start(lds + SLOT + LoadA::SIZE, wc, 0, lane);
    auto read_one = [&](auto X, uint32_t a, uint32_t b, Frags& f) {
      constexpr int x = decltype(X)::value;
      if constexpr (x < TM) f.a[x] = FragA::read(a, wr, x);
      else f.b[x - TM] = FragB::read(b, wc, x - TM);
    };
    constexpr int READS = TM + TN, PRODUCTS = TM * TN;
    static_assert(READS <= PRODUCTS, "a read behind a product");
    // the products of a half stage, with between(0), between(1), ... after one each: reads and copies
    // issue while a product runs
    auto multiply = [&](const Frags& f, auto&& between) {
      static_for<PRODUCTS>([&](auto X) {
        constexpr int x = decltype(X)::value, i = x / TN, j = x % TN;
        acc[i][j] = mma16(T{}, f.b[j], f.a[i], acc[i][j]);
        between(X);
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    // the stage to be copied next: to_kt of piece of work `to`, S stages ahead of the one that is multiplied
    int to = blockIdx.x, to_kt = 0, to_end = 0;
    int later = -1;   // stages that have been copied or are under way behind the one in hand

    auto issue = [&](uint8_t* slot, bool first) {
      if (first || to_kt == to_end) {   // on to the next piece of work
        if (!first) to += gridDim.x;
        if (to >= total) return;
        const Work w = work(to);
        la.init(g.a, w.m0, wave, lane);
        lb.init(g.b, w.n0, wave, lane);
        to_kt = w.begin;
        to_end = w.end;
      }
      const At s = at(to_kt++);
      la.go(s.piece, s.k);
      lb.go(s.piece, s.k);
      la.copy(g.valid_a - s.k, slot);
      lb.copy(g.valid_b - s.k, slot + LoadA::SIZE);
      ++later;
    };
#pragma unroll 1
    for (int s = 0; s < S; ++s) issue(lds + s * SLOT, s == 0);
    // all but the copies of the last `n` stages have landed
    auto landed_but = [&](int n) {
      if (S > 3 && n >= 3) wait_vmcnt<(S > 3 ? 3 : 0) * NCOPY>();
      else if (S > 2 && n == 2) wait_vmcnt<(S > 2 ? 2 : 0) * NCOPY>();
      else if (n == 1) wait_vmcnt<NCOPY>();
      else wait_vmcnt<0>();
    };
    landed_but(later);
    stage_barrier();
    Frags f0, f1;
    uint32_t hand = 0, next = SLOT;   // the slots of the stage in hand and of the next one, in bytes
    int landed = 0;                   // stages behind the one in hand that have been waited for
    // One stage.  COPY: the stage to be copied is whole and the one behind the last copied, and copied between the
    // products; else it is any, or none, and copied ahead of them.  The next stage's first half is read even where
    // there is no next stage: nothing looks at it then.
    auto stage = [&](auto COPY) {
      constexpr bool copy = decltype(COPY)::value;
      uint8_t* const slot = lds + hand;
      multiply(f0, [&](auto X) {
        if constexpr (decltype(X)::value < READS) read_one(X, a1, b1, f1);
      });
      __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): this wave's reads of the stage are done
      // its copies of the next one have landed
      if (landed > 0) --landed;
      else if constexpr (copy) wait_vmcnt<(S - 2) * NCOPY>();
      else landed_but(later - 1);
      stage_barrier();
      if constexpr (!copy) {
        issue(slot, false);
        --later;
      }
      multiply(f1, [&](auto X) {
        constexpr int x = decltype(X)::value, c0 = x * NCOPY / PRODUCTS, c1 = (x + 1) * NCOPY / PRODUCTS;
        if constexpr (x < READS) read_one(X, a0, b0, f0);
        if constexpr (copy) {
          static_for<c1 - c0>([&](auto C) {
            constexpr int c = c0 + decltype(C)::value;
            if constexpr (c < LoadA::L) la.template copy_one<c>(kStageK, slot);
            else lb.template copy_one<c - LoadA::L>(kStageK, slot + LoadA::SIZE);
          });
        }
      });
      if constexpr (copy) {
        la.step();
        lb.step();
      }
      const uint32_t after = next + SLOT == S * SLOT ? 0 : next + SLOT;
      a1 += next - hand;
      b1 += next - hand;
      a0 += after - next;
      b0 += after - next;
      hand = next;
      next = after;
    };
    const int least = g.valid_a < g.valid_b ? g.valid_a : g.valid_b;
    const int cut = least < g.seg_stages * kStageK ? 1 : 0;   // the last stage of a piece of K is not whole
    for (int i = blockIdx.x; i < total; i += gridDim.x) {
      const Work now = work(i);
      // (the first half is read again behind the outputs, which need its registers)
      static_for<READS>([&](auto X) { read_one(X, a0 + (hand - next), b0 + (hand - next), f0); });
      int kt = now.begin;
      while (kt < now.end) {
        // stages that are copied between products: whole, and of the same piece of K and of work
        const int piece_end = kt + S < g.seg_stages ? g.seg_stages : g.stages;
        const int stop = piece_end - cut < now.end ? piece_end - cut : now.end;
        if (kt + S < stop) {
          const At s = at(kt + S);
          la.go(s.piece, s.k);
          lb.go(s.piece, s.k);
          to_kt = stop;
          for (; kt + S < stop; ++kt) stage(std::true_type{});
        }
        stage(std::false_type{});
        ++kt;
      }
      wait_vmcnt<0>();
      landed = S - 1;
      out(acc, part, now.m0 + wr * 16, now.n0 + wc * 16, opaque(lane), now.split);
      clear();
    }
  } else {
    const Work now = work(g.first + blockIdx.x);
    la.init(g.a, now.m0, wave, lane);
    lb.init(g.b, now.n0, wave, lane);
    auto fetch = [&](int kt) {
      const At s = at(kt);
      la.fetch(g.a, s.piece, s.k, g.valid_a - s.k);
      lb.fetch(g.b, s.piece, s.k, g.valid_b - s.k);
    };
    auto put = [&](int kt) {
      uint8_t* const slot = lds + ((kt - now.begin) & 1) * SLOT;
      la.put(g.a, slot);
      lb.put(g.b, slot + LoadA::SIZE);
    };
    fetch(now.begin);
    put(now.begin);
    __syncthreads();
    for (int kt = now.begin; kt < now.end; ++kt) {
      if (kt + 1 < now.end) fetch(kt + 1);
      const uint8_t* const slot = lds + ((kt - now.begin) & 1) * SLOT;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        v8s_t fa[TM], fb[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i)
          fa[i] = Fragments<BM, ADOWN>::read(Fragments<BM, ADOWN>::start(slot, wr, q, lane), wr, i);
#pragma unroll
        for (int j = 0; j < TN; ++j)
          fb[j] = Fragments<BN, BDOWN>::read(Fragments<BN, BDOWN>::start(slot + LoadA::SIZE, wc, q, lane), wc, j);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[i][j] = mma16(T{}, fb[j], fa[i], acc[i][j]);
      }
      if (kt + 1 < now.end) put(kt + 1);
      __syncthreads();
    }
    out(acc, part, now.m0 + wr * 16, now.n0 + wc * 16, lane, now.split);
  }
}

// Outputs of a wave, 32 rows (two tiles) at a time, turned through its LDS so that rows are stored in whole pieces of
// 8 columns.  In 16 bits: 32 JT columns; value(i, j, r) is register r of row tile i (0, 1) and column tile j in
// the layout above; emit(row, column, v) gets 8 consecutive columns, a row's from 4 JT lanes.  16-byte chunks are
// swizzled by row against bank conflicts.
template <typename T, int JT, typename Value, typename Emit>
__device__ __forceinline__ void turn16(uint8_t* part, int lane, Value&& value, Emit&& emit) {
  static_assert(JT == 1 || JT == 2, "");
  constexpr int PITCH = JT * 64, LPR = JT * 4;   // bytes and lanes per row
  auto at = [&](int r, int c) {                  // byte of chunk c (8 columns) of row r
    return r * PITCH + ((c ^ (JT == 2 ? r & 7 : (r >> 1) & 3)) << 4);
  };
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2 * JT; ++j) {
      float v[8] = {};
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = value(i, j, r);
      const Raw8<T> w = round8(v, T{});
      *reinterpret_cast<uint2*>(part + at(16 * i + (lane & 15), 2 * j + (lane >> 5)) + ((lane >> 4) & 1) * 8) =
          make_uint2(w.w[0], w.w[1]);
    }
#pragma unroll
  for (int s = 0; s < LPR / 2; ++s) {
    const int x = s * 64 + lane, r = x / LPR, c = x % LPR;
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(part + at(r, c));
    Raw8<T> w;
    w.w = u32x4_e_t{v[0], v[1], v[2], v[3]};
    emit(r, c * 8, w);
  }
}
// In 32 bits: 32 columns, a row's from 4 lanes.
template <typename Value, typename Emit>
__device__ __forceinline__ void turn32(uint8_t* part, int lane, Value&& value, Emit&& emit) {
  auto at = [&](int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); };   // chunk c: 4 columns
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      *reinterpret_cast<v4f_t*>(part + at(16 * i + (lane & 15), 4 * j + (lane >> 4))) = value(i, j);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int r = s * 16 + (lane >> 2), c = (lane & 3) * 2;
    const v4f_t lo = *reinterpret_cast<const v4f_t*>(part + at(r, c));
    const v4f_t hi = *reinterpret_cast<const v4f_t*>(part + at(r, c + 1));
    Raw8<float> w;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w.lo[j] = lo[j];
      w.hi[j] = hi[j];
    }
    emit(r, c * 4, w);
  }
}

// Runs a product's pieces of work: a resident grid where DIRECT, else a workgroup each (in launches of at most 2^32 - 1
// threads).
template <bool DIRECT, typename F>
inline int for_work(int64_t total, int per_cu, F&& launch) {
  if (DIRECT) return launch(0, (unsigned)std::min<int64_t>(total, (int64_t)num_cus() * per_cu));
  constexpr int64_t kMost = (int64_t)1 << 22;
  for (int64_t first = 0; first < total; first += kMost) {
    const int rc = launch((int)first, (unsigned)std::min(total - first, kMost));
    if (rc) return rc;
  }
  return FP8DP_OK;
}

}  // namespace fp8dp
