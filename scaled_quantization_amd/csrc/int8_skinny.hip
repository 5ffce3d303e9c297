// int8_skinny.hip -- the INT8 product for few tokens (decoding): bound by the weight's bytes and
// by latency.  A workgroup owns 16 channels and all tokens (up to 64); its waves split K
// and join their integer sums in LDS, so a product of 4096 channels fills 256 compute units.
//
// A matrix instruction wants 16 rows side by side, and loading such fragments
// from global memory touches 64 cache lines per instruction.  k_i8_few therefore copies whole
// 128-byte lines (8 rows per instruction) straight into LDS, into a ring of SL pieces
// of 128 bytes of K that belongs to the wave alone: no barrier, each wave waits for its
// own copies.  k_i8_few_any, for rows that start at any byte, loads fragments from memory.
//
// CAST (int8_linear): the tokens come as T, go to LDS ahead of the weights and are cast there
// (quantize_int8's rule) by every workgroup for itself while the weights travel: for a
// few tokens that costs less than a launch of its own.
#include <hip/hip_runtime.h>

#include "int8_core.hpp"
#include "int8_skinny.hpp"

namespace fp8dp {

// Joins the waves' sums ([wave][tile][lane] of 4 integers in `join`) and stores the outputs of
// MT tiles of 16 tokens x 16 channels; lane: token lane % 16, channels 4 (lane / 16) .. + 3.
template <typename T, int MT, int WAVES>
__device__ __forceinline__ void join_out(const I8Args& g, v4i_t* join, const v4i_t (&acc)[MT],
                                         const float (&sa)[MT], const RawCols4& cols, int n,
                                         int wave, int lane) {
#pragma unroll
  for (int i = 0; i < MT; ++i) join[(wave * MT + i) * 64 + lane] = acc[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    if (i % WAVES != wave) continue;
    v4i_t sum = {};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += join[(w * MT + i) * 64 + lane];
    const int m = 16 * i + (lane & 15);
    if (m < g.M && n < g.N) {
      float bias[4];
      widen_bias4<T>(g, cols, bias);
      store_out4<T>(g, m, n, sa[i], cols.sb, bias, sum);
    }
  }
}

// AG: groups of 8 tokens.  SL: pieces in a wave's ring.
template <typename T, int AG, int WAVES, int SL, bool CAST>
__global__ __launch_bounds__(64 * WAVES) void k_i8_few(I8Args g, const T* x) {
  constexpr int MT = (AG + 1) / 2, NA = CAST ? 0 : AG, NC = NA + 2;   // copies per piece
  constexpr int SLOT = NC * 1024;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int frow = lane & 15, fch = lane >> 4;
  const int n0 = (g.first + (int)blockIdx.x) * 16, K = g.K, M = g.M;
  uint8_t* const ring = lds + wave * SL * SLOT;

  // what the epilogue needs, ahead of everything
  const int n = n0 + 4 * fch;
  const RawCols4 cols = load_cols4<T>(g, n);
  float sa[MT];
  if constexpr (!CAST) {
#pragma unroll
    for (int i = 0; i < MT; ++i) sa[i] = g.sa[16 * i + frow < M ? 16 * i + frow : M - 1];
  }

  // copy c of a piece: 8 rows, lane l row 8 c + l / 8 and the chunk that swz() keeps at l % 8
  const uint8_t* row[NC];
  int chunk[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) chunk[c] = (lane & 7) ^ ((4 * c + (lane >> 4)) & 7);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int r = 8 * (c < NA ? c : c - NA) + (lane >> 3);
    row[c] = reinterpret_cast<const uint8_t*>(
                 c < NA ? g.a + (r < M ? r : M - 1) * g.lda
                        : g.b + (int64_t)(n0 + r < g.N ? n0 + r : g.N - 1) * g.ldb);
  }
  const int pieces = (K + 127) / 128;
  const int mine = pieces > wave ? (pieces - wave + WAVES - 1) / WAVES : 0;
  auto issue = [&](int j) {
    uint8_t* const slot = ring + (j % SL) * SLOT;
    const int k = (wave + j * WAVES) * 128, left = (K - k) / 16;   // chunks inside K
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int ch = chunk[(c < NA ? c : c - NA) & 1];
      // past K: zeros for the tokens (CAST clears its codes instead), any chunk for the weight
      const uint8_t* p = row[c] + k + (left >= 8 || ch < left ? ch * 16 : 0);
      if (c < NA && left < 8 && ch >= left) p = reinterpret_cast<const uint8_t*>(&kZeroChunk);
      copy16_to_lds(p, slot + c * 1024);
    }
  };
  auto issue_first = [&] {
#pragma unroll
    for (int j = 0; j < SL; ++j)
      if (j < mine) issue(j);
  };

  const int stride = skinny_stride(K);
  uint8_t* const codes = lds + WAVES * SL * SLOT;
  uint8_t* const tokens = codes + M * stride;
  if constexpr (!CAST) {
    issue_first();
  } else {
    // the tokens' chunks, one copy of 64 per wave in turn
    const int chunks = M * K * (int)sizeof(T) / 16, steps = (chunks + 64 * WAVES - 1) / (64 * WAVES);
    float* const scale = reinterpret_cast<float*>(tokens + steps * 1024 * WAVES);
    uint32_t* const top = reinterpret_cast<uint32_t*>(scale + 16);
    for (int s = 0; s < steps; ++s) {
      const int q = (s * WAVES + wave) * 64 + lane;
      copy16_to_lds(reinterpret_cast<const uint8_t*>(x) + (size_t)(q < chunks ? q : chunks - 1) * 16,
                    tokens + (s * WAVES + wave) * 1024);
    }
    issue_first();
    // copies return in order: the tokens are there when only the weights' are left
    static_for<SL + 1>([&](auto J) {
      if ((mine < SL ? mine : SL) == decltype(J)::value) wait_vmcnt<decltype(J)::value * NC>();
    });
    stage_barrier();
    // a wave takes one of `parts` ranges of a token's vectors at a time
    const int parts = M == 1 ? WAVES : M == 2 ? WAVES / 2 : M <= 4 ? WAVES / 4 : 1, items = M * parts;
    const int nvec = K / 8, per = (nvec + parts - 1) / parts;
    auto vector = [&](int i, int v, float* w) {
      const T* const p = reinterpret_cast<const T*>(tokens) + (i / parts) * K + v * 8;
      Raw8<T> raw;
      __builtin_memcpy(&raw, __builtin_assume_aligned(p, 16), sizeof(raw));
      widen8f(raw, w);
    };
    for (int i = wave; i < items; i += WAVES) {
      const int p = i % parts, v1 = (p + 1) * per < nvec ? (p + 1) * per : nvec;
      uint32_t m = 0;
      for (int v = p * per + lane; v < v1; v += 64) {
        float w[8];
        vector(i, v, w);
        m = magnitude8(w, m);
      }
      m = wave_umax(m);
      if (lane == 0) top[i] = m;
    }
    __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    stage_barrier();
    for (int i = wave; i < items; i += WAVES) {
      const int r = i / parts, p = i % parts;
      const uint32_t m = wave_umax(top[r * parts + (lane & (parts - 1))]);
      const bool plain = m != 0 && m < 0x7F800000u;
      const RowScale s = row_scale(plain ? m : 0x3F800000u);
      if (p == 0 && lane == 0)
        scale[r] = plain ? __uint_as_float(m) / 127.0f : m == 0 ? 0.0f : __builtin_nanf("");
      const int v1 = (p + 1) * per < nvec ? (p + 1) * per : nvec;
      for (int v = p * per + lane; v < v1; v += 64) {
        uint2 code = {0u, 0u};
        if (plain) {
          float w[8];
          vector(i, v, w);
          code = codes8<sizeof(T) == 4>(w, s);
        }
        *reinterpret_cast<uint2*>(codes + r * stride + v * 8) = code;
      }
      // the wave of the first range also clears the codes from K to the end of the LDS row (16 vectors
      // at most); the others may be empty, with nvec anywhere among their starts
      if (p == 0 && nvec + lane < stride / 8)
        *reinterpret_cast<uint2*>(codes + r * stride + (nvec + lane) * 8) = uint2{0u, 0u};
    }
    __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    stage_barrier();
    sa[0] = scale[frow < M ? frow : M - 1];
  }

  const uint8_t* const code_row = codes + (frow < M ? frow : M - 1) * stride;   // CAST
  v4i_t acc[MT] = {};
  for (int j = 0; j < mine; ++j) {
    // piece j has landed when at most the later ones in flight are left
    const int later = mine - 1 - j < SL - 1 ? mine - 1 - j : SL - 1;
    static_for<SL>([&](auto J) {
      if (later == decltype(J)::value) wait_vmcnt<decltype(J)::value * NC>();
    });
    __asm__ volatile("" ::: "memory");
    const uint8_t* const slot = ring + (j % SL) * SLOT;
    const int k = (wave + j * WAVES) * 128;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = h * 4 + fch;
      const v4i_t fb = *reinterpret_cast<const v4i_t*>(slot + NA * 1024 + swz(frow, c));
      v4i_t fa[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i)
        fa[i] = CAST ? *reinterpret_cast<const v4i_t*>(code_row + k + c * 16)
                     : *reinterpret_cast<const v4i_t*>(
                           slot + swz(16 * i + (2 * i + 1 < NA ? frow : frow & 7), c));
#pragma unroll
      for (int i = 0; i < MT; ++i)
        acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb, fa[i], acc[i], 0, 0, 0);
    }
    __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the slot has been read
    if (j + SL < mine) issue(j + SL);
  }
  __syncthreads();
  join_out<T, MT, WAVES>(g, reinterpret_cast<v4i_t*>(lds), acc, sa, cols, n, wave, lane);
}

// Rows that start at any byte: fragments straight from memory, UNITS pieces in flight.
template <typename T, int MT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_i8_few_any(I8Args g) {
  constexpr int UNITS = 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[WAVES * MT * 1024];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int frow = lane & 15, fch = lane >> 4;
  const int n0 = (g.first + (int)blockIdx.x) * 16, K = g.K, M = g.M;

  const int n = n0 + 4 * fch;
  const RawCols4 cols = load_cols4<T>(g, n);
  float sa[MT];
  const int8_t* pa[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = 16 * i + frow < M ? 16 * i + frow : M - 1;
    sa[i] = g.sa[m];
    pa[i] = g.a + m * g.lda;
  }
  const int8_t* const pb = g.b + (int64_t)(n0 + frow < g.N ? n0 + frow : g.N - 1) * g.ldb;

  // The whole pieces of K, p = wave, wave + WAVES, ...; the cut one at the end comes after them.
  // A wave with fewer pieces than UNITS reads its last one again: no load stands behind a
  // branch, so waiting for one of them never waits for the later ones.
  const int pieces = K / 128;
  v4i_t fb[UNITS][2], fa[UNITS][2][MT];
  auto load = [&](int u, int p) {
    const int k = (p < pieces ? p : pieces - 1) * 128 + fch * 16;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      fb[u][h] = load16(pb + k + h * 64);
#pragma unroll
      for (int i = 0; i < MT; ++i) fa[u][h][i] = load16(pa[i] + k + h * 64);
    }
  };
  v4i_t acc[MT] = {};
  auto multiply = [&](int u) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < MT; ++i)
        acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[u][h], fa[u][h][i], acc[i], 0, 0, 0);
  };
  if (pieces > 0) {
#pragma unroll
    for (int u = 0; u < UNITS; ++u) load(u, wave + u * WAVES);
    int p0 = wave;
    for (; p0 + UNITS * WAVES < pieces; p0 += UNITS * WAVES) {
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        multiply(u);
        load(u, p0 + (u + UNITS) * WAVES);
      }
    }
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
      if (p0 + u * WAVES < pieces) multiply(u);
  }
  if (K % 128 != 0 && wave == pieces % WAVES) {
#pragma unroll 1
    for (int k = pieces * 128 + fch * 16; k < pieces * 128 + 128; k += 64) {
      const v4i_t w = load_chunk<false>(pb, k, K);
#pragma unroll
      for (int i = 0; i < MT; ++i)
        acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, load_chunk<true>(pa[i], k, K), acc[i], 0,
                                                       0, 0);
    }
  }
  join_out<T, MT, WAVES>(g, reinterpret_cast<v4i_t*>(lds), acc, sa, cols, n, wave, lane);
}

template <typename T, int AG, int WAVES, int SL, bool CAST>
static int launch_few(const char* what, const I8Args& g, const void* x, hipStream_t stream) {
  constexpr size_t ring = (size_t)WAVES * SL * ((CAST ? 0 : AG) + 2) * 1024;
  static_assert(ring >= (size_t)WAVES * ((AG + 1) / 2) * 1024, "the joined sums fit the ring");
  const size_t bytes = ring + (CAST ? skinny_cast_bytes(g.M, g.K, sizeof(T), WAVES) : 0);
  return for_blocks((g.N + 15) / 16, [&](int first, unsigned count) {
    I8Args part = g;
    part.first = first;
    hipLaunchKernelGGL((k_i8_few<T, AG, WAVES, SL, CAST>), dim3(count), dim3(64 * WAVES), bytes, stream,
                       part, static_cast<const T*>(x));
    return check_launch(what);
  });
}

template <typename T, int MT>
static int launch_few_any(const char* what, const I8Args& g, hipStream_t stream) {
  return for_blocks((g.N + 15) / 16, [&](int first, unsigned count) {
    I8Args part = g;
    part.first = first;
    hipLaunchKernelGGL((k_i8_few_any<T, MT, 8>), dim3(count), dim3(512), 0, stream, part);
    return check_launch(what);
  });
}

template <typename T>
static int skinny_type(const char* what, const I8Args& g, const void* x, hipStream_t stream) {
  if (x != nullptr) return launch_few<T, 2, 8, 4, true>(what, g, x, stream);
  if (!rows16(g)) {
    if (g.M <= 16) return launch_few_any<T, 1>(what, g, stream);
    if (g.M <= 32) return launch_few_any<T, 2>(what, g, stream);
    return launch_few_any<T, 4>(what, g, stream);
  }
  // rings of 96 to 128 KB: what a compute unit has in flight
  if (g.M <= 8) return launch_few<T, 1, 8, 4, false>(what, g, x, stream);
  if (g.M <= 16) return launch_few<T, 2, 8, 4, false>(what, g, x, stream);
  if (g.M <= 32) return launch_few<T, 4, 8, 2, false>(what, g, x, stream);
  if (g.M <= 48) return launch_few<T, 6, 8, 2, false>(what, g, x, stream);
  return launch_few<T, 8, 4, 3, false>(what, g, x, stream);
}

int skinny_i8(const char* what, fp8dp_dtype yt, const I8Args& g, const void* x,
              hipStream_t stream) {
  if (yt == FP8DP_BF16) return skinny_type<bf16_t>(what, g, x, stream);
  if (yt == FP8DP_F16) return skinny_type<f16_t>(what, g, x, stream);
  return skinny_type<float>(what, g, x, stream);
}

}  // namespace fp8dp
