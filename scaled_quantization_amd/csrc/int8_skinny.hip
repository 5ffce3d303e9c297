// int8_skinny.hip -- the INT8 product for few tokens (decoding): bound by the
// weight's bytes and by latency, so every weight byte is loaded once, straight
// from memory into the registers that feed the matrix instruction, and K is split over
// the waves of a workgroup (the integer partial sums are joined in LDS).
//
// A workgroup of WAVES waves owns 16 NT channels and 16 MT tokens.  Wave w takes
// the 128-byte pieces w, w + WAVES, ... of K, whole cache lines of each
// weight row, and keeps UNITS pieces in flight.  Rows may start at any byte.
//
// FUSED: the tokens come as T and are cast here (quantize_int8's rule), by
// every workgroup for itself, into LDS: for a few tokens that costs less than a
// launch of its own.  The first weight loads are issued before the cast, which
// runs while they travel.
#include <hip/hip_runtime.h>

#include "int8_core.hpp"
#include "int8_skinny.hpp"

namespace fp8dp {

template <typename T, int MT, int NT, int WAVES, bool FUSED>
__global__ __launch_bounds__(64 * WAVES) void k_i8_skinny(I8Args g, const T* x) {
  constexpr int UNITS = 4;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int frow = lane & 15, fch = lane >> 4;
  const int n0 = blockIdx.x * 16 * NT, m0 = blockIdx.y * 16 * MT;
  const int K = g.K;
  const int stride = skinny_stride(K);       // of the codes in LDS
  const int mrows = g.M - m0 < 16 * MT ? g.M - m0 : 16 * MT;
  uint32_t* const top = reinterpret_cast<uint32_t*>(lds + (FUSED ? mrows * stride : 0));
  float* const scale = reinterpret_cast<float*>(top + 16 * MT * WAVES);
  const int parts = mrows == 1 ? WAVES : mrows == 2 ? WAVES / 2 : mrows <= 4 ? WAVES / 4 : 1;

  const int8_t* pb[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int n = n0 + 16 * j + frow;
    pb[j] = g.b + (int64_t)(n < g.N ? n : g.N - 1) * g.ldb;
  }
  const int8_t* pa[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = 16 * i + frow < mrows ? 16 * i + frow : mrows - 1;
    pa[i] = FUSED ? reinterpret_cast<const int8_t*>(lds) + m * stride
                  : g.a + (int64_t)(m0 + m) * g.lda;
  }

  // what the epilogue needs, ahead of everything
  RawCols4 cols[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) cols[j] = load_cols4<T>(g, n0 + 16 * j + 4 * fch);

  // The whole pieces of K, p = wave, wave + WAVES, ...; the cut one at the end comes after them.
  // Weights always, codes too unless they are in LDS.
  // K is at least 128, and a wave with fewer pieces than UNITS reads its last one again: no load
  // stands behind a branch, so waiting for one of them never waits for the later ones.
  const int pieces = K / 128;
  v4i_t fb[UNITS][2][NT], fa[FUSED ? 1 : UNITS][2][MT];
  auto load = [&](int u, int p) {
    const int k = (p < pieces ? p : pieces - 1) * 128 + fch * 16;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < NT; ++j) fb[u][h][j] = load16(pb[j] + k + h * 64);
      if constexpr (!FUSED) {
#pragma unroll
        for (int i = 0; i < MT; ++i) fa[u][h][i] = load16(pa[i] + k + h * 64);
      }
    }
  };
  auto load_first = [&] {
#pragma unroll
    for (int u = 0; u < UNITS; ++u) load(u, wave + u * WAVES);
  };

  if constexpr (!FUSED) {
    load_first();
  } else {
    // item i: part i % parts of token i / parts, a wave each.  Where every lane has one vector at
    // most, it is loaded ahead of the weights (loads return in order) and cast while they travel;
    // otherwise the weights follow the cast, which reads the tokens twice.
    const int nvec = (K + 7) / 8, per = (nvec + parts - 1) / parts, items = mrows * parts;
    auto absmax = [](const Raw8<T>& raw, uint32_t m) {
      float w[8];
      widen8f(raw, w);
      return magnitude8(w, m);
    };
    // the rule of item i's token, once all parts of its largest magnitude are in `top`
    auto rule = [&](int i, bool& plain) {
      const int r = i / parts;
      const uint32_t m = wave_umax(top[r * parts + (lane & (parts - 1))]);
      plain = m != 0 && m < 0x7F800000u;
      if (i % parts == 0 && lane == 0)
        scale[r] = plain ? __uint_as_float(m) / 127.0f : m == 0 ? 0.0f : __builtin_nanf("");
      return row_scale(plain ? m : 0x3F800000u);
    };
    auto put = [&](int i, int v, const Raw8<T>& raw, const RowScale& s, bool plain) {
      float w[8];
      widen8f(raw, w);
      uint2 code = {0u, 0u};
      if (plain) code = codes8<sizeof(T) == 4>(w, s);
      *reinterpret_cast<uint2*>(lds + (i / parts) * stride + v * 8) = code;
    };
    bool plain;
    if (items <= WAVES && per <= 64) {
      const int i = wave < items ? wave : items - 1, v = (i % parts) * per + lane;
      const bool has = wave < items && lane < per && v < nvec;
      Raw8<T> raw = load_row(x + (int64_t)(m0 + i / parts) * K, v * 8, K);
      load_first();
      settle(raw, has ? K - v * 8 : 0);
      const uint32_t m = wave_umax(absmax(raw, 0));
      if (lane == 0 && wave < items) top[i] = m;
      __syncthreads();
      const RowScale s = rule(i, plain);
      if (has) put(i, v, raw, s, plain);
    } else {
      for (int i = wave; i < items; i += WAVES) {
        const T* const row = x + (int64_t)(m0 + i / parts) * K;
        const int v1 = (i % parts + 1) * per < nvec ? (i % parts + 1) * per : nvec;
        uint32_t m = 0;
        for (int v = (i % parts) * per + lane; v < v1; v += 64) {
          Raw8<T> raw = load_row(row, v * 8, K);
          settle(raw, K - v * 8);
          m = absmax(raw, m);
        }
        m = wave_umax(m);
        if (lane == 0) top[i] = m;
      }
      __syncthreads();
      for (int i = wave; i < items; i += WAVES) {
        const T* const row = x + (int64_t)(m0 + i / parts) * K;
        const RowScale s = rule(i, plain);
        const int v1 = (i % parts + 1) * per < nvec ? (i % parts + 1) * per : nvec;
        for (int v = (i % parts) * per + lane; v < v1; v += 64) {
          Raw8<T> raw = load_row(row, v * 8, K);
          settle(raw, K - v * 8);
          put(i, v, raw, s, plain);
        }
      }
      load_first();
    }
    __syncthreads();
  }

  v4i_t acc[MT][NT] = {};
  auto multiply = [&](int u, int p) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v4i_t now[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if constexpr (FUSED)
          now[i] = *reinterpret_cast<const v4i_t*>(pa[i] + p * 128 + h * 64 + fch * 16);
        else
          now[i] = fa[u][h][i];
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[u][h][j], now[i], acc[i][j], 0, 0, 0);
    }
  };
  int p0 = wave;
  for (; p0 + UNITS * WAVES < pieces; p0 += UNITS * WAVES) {
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      multiply(u, p0 + u * WAVES);
      load(u, p0 + (u + UNITS) * WAVES);
    }
  }
#pragma unroll
  for (int u = 0; u < UNITS; ++u)
    if (p0 + u * WAVES < pieces) multiply(u, p0 + u * WAVES);
  if (K % 128 != 0 && wave == pieces % WAVES) {
#pragma unroll 1
    for (int k = pieces * 128 + fch * 16; k < pieces * 128 + 128; k += 64) {
      v4i_t now[MT], w[NT];
#pragma unroll
      for (int i = 0; i < MT; ++i) now[i] = load_chunk<true>(pa[i], k, K);
#pragma unroll
      for (int j = 0; j < NT; ++j) w[j] = load_chunk<false>(pb[j], k, K);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[j], now[i], acc[i][j], 0, 0, 0);
    }
  }

  // join the waves' sums: [wave][tile][lane] of 4 integers
  float sa_row[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int r = 16 * i + frow < mrows ? 16 * i + frow : mrows - 1;
    sa_row[i] = FUSED ? scale[r] : g.sa[m0 + r];
  }
  if constexpr (FUSED) __syncthreads();
  v4i_t* const join = reinterpret_cast<v4i_t*>(lds);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) join[(wave * MT * NT + i * NT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if ((i * NT + j) % WAVES != wave) continue;
      v4i_t sum = {};
#pragma unroll
      for (int w = 0; w < WAVES; ++w) sum += join[(w * MT * NT + i * NT + j) * 64 + lane];
      const int n = n0 + 16 * j + 4 * fch;
      if (16 * i + frow < mrows && n < g.N) {
        float bias[4];
        widen_bias4<T>(g, cols[j], bias);
        store_out4<T>(g, m0 + 16 * i + frow, n, sa_row[i], cols[j].sb, bias, sum);
      }
    }
}

template <typename T, int MT, int NT, int WAVES, bool FUSED>
static int launch_skinny(const char* what, const I8Args& g, const void* x, hipStream_t stream) {
  const int64_t blocks = ((int64_t)g.N + 16 * NT - 1) / (16 * NT);
  const int64_t tall = ((int64_t)g.M + 16 * MT - 1) / (16 * MT);
  const int rows = g.M < 16 * MT ? g.M : 16 * MT;
  size_t bytes = (size_t)WAVES * MT * NT * 1024;
  if (FUSED) bytes = std::max(bytes, (size_t)rows * skinny_stride(g.K) + 4u * 16 * MT * (WAVES + 1));
  hipLaunchKernelGGL((k_i8_skinny<T, MT, NT, WAVES, FUSED>), dim3((unsigned)blocks, (unsigned)tall),
                     dim3(64 * WAVES), bytes, stream, g, static_cast<const T*>(x));
  return check_launch(what);
}

template <typename T>
static int skinny_type(const char* what, const I8Args& g, const void* x, hipStream_t stream) {
  if (x != nullptr) return launch_skinny<T, 1, 1, 8, true>(what, g, x, stream);
  if (g.M <= 16) return launch_skinny<T, 1, 1, 8, false>(what, g, x, stream);
  if (g.M <= 32) return launch_skinny<T, 2, 1, 8, false>(what, g, x, stream);
  return launch_skinny<T, 4, 1, 8, false>(what, g, x, stream);
}

int skinny_i8(const char* what, fp8dp_dtype yt, const I8Args& g, const void* x,
              hipStream_t stream) {
  if (yt == FP8DP_BF16) return skinny_type<bf16_t>(what, g, x, stream);
  if (yt == FP8DP_F16) return skinny_type<f16_t>(what, g, x, stream);
  return skinny_type<float>(what, g, x, stream);
}

}  // namespace fp8dp
