// row_core.hpp -- pieces shared by the kernels that work on whole rows (layer
// norm, dropout, INT8 quantizer): vectors of 8 elements at the alignment of an
// element, row statistics over a wave or a workgroup, the Philox mask, and
// the exact INT8 rounding.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "codec.hpp"
#include "common.hpp"
#include "fp8dp_block.h"

namespace fp8dp {

// ------------------------------------------------------------------ vectors
// 16 and 8 bytes at the alignment of one element: gfx950 takes global accesses
// of any alignment, so rows of odd length need no path of their own.
typedef unsigned int u32x4_e_t __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned int u32x2_b_t __attribute__((ext_vector_type(2), aligned(1)));
typedef float f32x4_e_t __attribute__((ext_vector_type(4), aligned(4)));

struct bf16_t { uint16_t bits; };
struct f16_t { uint16_t bits; };

template <typename T> struct Raw8 { u32x4_e_t w; };          // 8 elements as loaded
template <> struct Raw8<float> { f32x4_e_t lo, hi; };

__device__ __forceinline__ float to_f32(bf16_t x) { return __uint_as_float((uint32_t)x.bits << 16); }
__device__ __forceinline__ float to_f32(f16_t x) {
  return (float)__builtin_bit_cast(_Float16, x.bits);
}
__device__ __forceinline__ float to_f32(float x) { return x; }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ bf16_t from_f32<bf16_t>(float v) {
  return {(uint16_t)(pack2_bf16_hw(v, 0.0f) & 0xFFFFu)};
}
template <> __device__ __forceinline__ f16_t from_f32<f16_t>(float v) {
  return {__builtin_bit_cast(uint16_t, (_Float16)v)};
}
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }

template <bool STREAM = false, typename T>
__device__ __forceinline__ Raw8<T> load_raw8(const T* p) {
  Raw8<T> r;
  if constexpr (sizeof(T) == 4) {
    const f32x4_e_t* const q = reinterpret_cast<const f32x4_e_t*>(p);
    r.lo = STREAM ? __builtin_nontemporal_load(q) : q[0];
    r.hi = STREAM ? __builtin_nontemporal_load(q + 1) : q[1];
  } else {
    const u32x4_e_t* const q = reinterpret_cast<const u32x4_e_t*>(p);
    r.w = STREAM ? __builtin_nontemporal_load(q) : q[0];
  }
  return r;
}

__device__ __forceinline__ void widen8f(const Raw8<bf16_t>& r, float v[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(r.w[j] << 16);
    v[2 * j + 1] = __uint_as_float(r.w[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void widen8f(const Raw8<f16_t>& r, float v[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = (float)__builtin_bit_cast(_Float16, (uint16_t)(r.w[j] & 0xFFFFu));
    v[2 * j + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(r.w[j] >> 16));
  }
}
__device__ __forceinline__ void widen8f(const Raw8<float>& r, float v[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = r.lo[j];
    v[j + 4] = r.hi[j];
  }
}

__device__ __forceinline__ Raw8<bf16_t> round8(const float v[8], bf16_t) {
  Raw8<bf16_t> r;
#pragma unroll
  for (int j = 0; j < 4; ++j) r.w[j] = pack2_bf16_hw(v[2 * j], v[2 * j + 1]);
  return r;
}
__device__ __forceinline__ Raw8<f16_t> round8(const float v[8], f16_t) {
  Raw8<f16_t> r;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    r.w[j] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[2 * j]) |
             (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[2 * j + 1]) << 16;
  return r;
}
__device__ __forceinline__ Raw8<float> round8(const float v[8], float) {
  Raw8<float> r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r.lo[j] = v[j];
    r.hi[j] = v[j + 4];
  }
  return r;
}
// Outputs are stored non-temporally: this kernel does not read them again, and they
// displace fewer of the inputs from L2 (layer norm 16384 x 768 11.3 -> 10.4 us, with
// dropout and residual 22.0 -> 19.0, layer norm 65536 x 4096 186 -> 179).  Loads are left alone:
// inputs often come out of the cache that an earlier kernel filled (non-temporal loads at
// 16384 x 768: 14.4 us).
template <typename T>
__device__ __forceinline__ void store_raw8(T* p, const Raw8<T>& r) {
  __builtin_nontemporal_store(r.w, reinterpret_cast<u32x4_e_t*>(p));
}
template <>
__device__ __forceinline__ void store_raw8<float>(float* p, const Raw8<float>& r) {
  __builtin_nontemporal_store(r.lo, reinterpret_cast<f32x4_e_t*>(p));
  __builtin_nontemporal_store(r.hi, reinterpret_cast<f32x4_e_t*>(p + 4));
}

// The n elements at p (n >= 8: 8 of them; n <= 0: none), the rest zeros, still as loaded:
// nothing waits for them before they are widened, so several vectors travel
// together.  A cut vector takes 8 loads of single elements, clamped instead of branched over.
__device__ __forceinline__ void load_cut(const bf16_t* p, int n, Raw8<bf16_t>& r) {
  const uint16_t* const q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = q[2 * j < n ? 2 * j : 0], hi = q[2 * j + 1 < n ? 2 * j + 1 : 0];
    r.w[j] = (2 * j < n ? lo : 0u) | (2 * j + 1 < n ? hi << 16 : 0u);
  }
}
__device__ __forceinline__ void load_cut(const f16_t* p, int n, Raw8<f16_t>& r) {
  Raw8<bf16_t> b;
  load_cut(reinterpret_cast<const bf16_t*>(p), n, b);
  r.w = b.w;
}
__device__ __forceinline__ void load_cut(const float* p, int n, Raw8<float>& r) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float lo = p[j < n ? j : 0], hi = p[j + 4 < n ? j + 4 : 0];
    r.lo[j] = j < n ? lo : 0.0f;
    r.hi[j] = j + 4 < n ? hi : 0.0f;
  }
}
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw(const T* p, int n) {
  Raw8<T> r = {};
  if (n >= 8) r = load_raw8(p);
  else if (n > 0) load_cut(p, n, r);
  return r;
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, float v[8]) {
  widen8f(load_raw(p, n), v);
}

template <typename T>
__device__ __forceinline__ void store8(T* p, int n, const float v[8]) {
  if (n >= 8) {
    store_raw8(p, round8(v, T{}));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = from_f32<T>(v[j]);
  }
}
// Element c of a row whose address is the same for the wave: the address stays in scalar
// registers and the offset is one 32-bit register.
template <typename T>
__device__ __forceinline__ const T* element(const T* row, int c) {
  return reinterpret_cast<const T*>(reinterpret_cast<const char*>(row) +
                                    (uint32_t)c * (uint32_t)sizeof(T));
}
template <typename T>
__device__ __forceinline__ T* element(T* row, int c) {
  return reinterpret_cast<T*>(reinterpret_cast<char*>(row) + (uint32_t)c * (uint32_t)sizeof(T));
}

// n elements of a vector already rounded.
template <typename T>
__device__ __forceinline__ void store_row(T* p, int n, const Raw8<T>& r) {
  if (n >= 8) {
    store_raw8(p, r);
  } else {
    float v[8];
    widen8f(r, v);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = from_f32<T>(v[j]);
  }
}

// Rows of at least 8 elements, without a branch: vector i of thread t starts at column
// 8 (i THR + t) and is read at most 8 before the row's end.  Only the last vector
// (i = NV - 1) can be cut or empty: settle() moves its n elements to the front
// once they have arrived (`ragged`: cols is no multiple of 8, the same for all threads), and
// its mask, kept over all rows, clears the rest.
// STREAM: not to be kept in the caches.
template <bool STREAM = false, typename T>
__device__ __forceinline__ Raw8<T> load_row(const T* row, int c, int cols) {
  return load_raw8<STREAM>(element(row, c < cols - 8 ? c : cols - 8));
}
__device__ __forceinline__ u32x4_e_t shift_down(u32x4_e_t w, int s) {   // by s bits, s > 0
  uint64_t lo = (uint64_t)w[1] << 32 | w[0], hi = (uint64_t)w[3] << 32 | w[2];
  lo = s < 64 ? lo >> s | hi << (64 - s) : s < 128 ? hi >> (s - 64) : 0;
  hi = s < 64 ? hi >> s : 0;
  return u32x4_e_t{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}
__device__ __forceinline__ void settle(Raw8<bf16_t>& r, int n, bool ragged = true) {
  if (ragged && n < 8) r.w = shift_down(r.w, n > 0 ? 16 * (8 - n) : 128);
}
__device__ __forceinline__ void settle(Raw8<f16_t>& r, int n, bool ragged = true) {
  if (ragged && n < 8) r.w = shift_down(r.w, n > 0 ? 16 * (8 - n) : 128);
}
__device__ __forceinline__ void settle(Raw8<float>& r, int n, bool ragged = true) {
  if (ragged && n < 8) {
    float v[8] = {r.lo[0], r.lo[1], r.lo[2], r.lo[3], r.hi[0], r.hi[1], r.hi[2], r.hi[3]};
    const int s = n > 0 ? 8 - n : 8;
#pragma unroll
    for (int b = 1; b <= 8; b <<= 1)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (s & b) v[j] = j + b < 8 ? v[j + b] : 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r.lo[j] = v[j];
      r.hi[j] = v[j + 4];
    }
  }
}
struct Mask8 {
  uint32_t bits[8];
  __device__ explicit Mask8(int n) {
#pragma unroll
    for (int j = 0; j < 8; ++j) bits[j] = j < n ? 0xFFFFFFFFu : 0u;
  }
  __device__ __forceinline__ void clear(float v[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(__float_as_uint(v[j]) & bits[j]);
  }
  // of a vector as loaded and settled: cut ones end in zeros already
  template <typename T>
  __device__ __forceinline__ void clear_empty(Raw8<T>& r) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) r.w[j] &= bits[0];
  }
  __device__ __forceinline__ void clear_empty(Raw8<float>& r) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r.lo[j] = __uint_as_float(__float_as_uint(r.lo[j]) & bits[0]);
      r.hi[j] = __uint_as_float(__float_as_uint(r.hi[j]) & bits[0]);
    }
  }
};
// Rounds 8 values to T and back (what a later read of the stored tensor sees).
template <typename T>
__device__ __forceinline__ void through8(float v[8]) {
  widen8f(round8(v, T{}), v);
}
// The parameters of columns c .. c + 7: type T, or float where wf32; NULL: fill.
template <typename T>
__device__ __forceinline__ void load_param8(const void* w, bool wf32, int64_t c, int n, float fill,
                                            float v[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = fill;
  } else if (wf32) {
    load8(static_cast<const float*>(w) + c, n, v);
  } else {
    load8(static_cast<const T*>(w) + c, n, v);
  }
}
__device__ __forceinline__ void zero_from8(int n, float v[8]) {
  if (n < 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j >= n) v[j] = 0.0f;
  }
}

// ------------------------------------------------------------------ reductions
// Wave-wide sum / unsigned max on the DPP network (no LDS): shifts inside rows
// of 16 lanes, then the row broadcasts; the total lands in lane 63 and
// comes back as a wave-uniform value.  Lanes without a source add zero.
__device__ __forceinline__ float wave_sum(float x) {
#define FP8DP_STEP(ctrl, rows)                                                              \
  x += __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(x), ctrl, rows, 0xF, \
                                                   false))
  FP8DP_STEP(0x111, 0xF);   // row_shr:1
  FP8DP_STEP(0x112, 0xF);   // row_shr:2
  FP8DP_STEP(0x114, 0xF);   // row_shr:4
  FP8DP_STEP(0x118, 0xF);   // row_shr:8
  FP8DP_STEP(0x142, 0xA);   // row_bcast:15
  FP8DP_STEP(0x143, 0xC);   // row_bcast:31
#undef FP8DP_STEP
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), 63));
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t x) {
#define FP8DP_STEP(ctrl, rows)                                                        \
  do {                                                                                \
    const uint32_t o = __builtin_amdgcn_update_dpp(0u, x, ctrl, rows, 0xF, false);    \
    x = o > x ? o : x;                                                                \
  } while (0)
  FP8DP_STEP(0x111, 0xF);
  FP8DP_STEP(0x112, 0xF);
  FP8DP_STEP(0x114, 0xF);
  FP8DP_STEP(0x118, 0xF);
  FP8DP_STEP(0x142, 0xA);
  FP8DP_STEP(0x143, 0xC);
#undef FP8DP_STEP
  return __builtin_amdgcn_readlane(x, 63);
}

// Totals over the THR threads of a row: a wave alone, or a workgroup through
// LDS (scratch: one slot of THR / 64 values per call site).  Every thread
// of the workgroup calls these together when THR > 64.
template <int THR>
__device__ __forceinline__ float row_sum(float x, float* scratch) {
  x = wave_sum(x);
  if constexpr (THR > 64) {
    if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0.0f;
#pragma unroll
    for (int i = 0; i < THR / 64; ++i) x += scratch[i];
  }
  return x;
}
template <int THR>
__device__ __forceinline__ uint32_t row_umax(uint32_t x, uint32_t* scratch) {
  x = wave_umax(x);
  if constexpr (THR > 64) {
    if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int i = 0; i < THR / 64; ++i) x = scratch[i] > x ? scratch[i] : x;
  }
  return x;
}

// A running sum of any length: what each addition rounds off is kept beside it (Knuth's exact
// error of a sum), so the total is off by 2 roundings instead of one per term.  An infinity
// or a NaN comes out as the plain sum's.
struct LongSum {
  float s = 0.0f, e = 0.0f;
  __device__ __forceinline__ void add(float v) {
    const float t = s + v, b = t - s;
    e += (s - (t - b)) + (v - b);
    s = t;
  }
  __device__ __forceinline__ float total() const { return e == e ? s + e : s; }
};
__device__ __forceinline__ float sum8(const float v[8]) {
  return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}

// ------------------------------------------------------------------ dropout
// Philox4x32 (Salmon et al., SC 2011), 10 rounds: per round two 32 x 32 -> 64
// products and four XORs, the key advanced by the two Weyl constants.
struct DropRule {
  uint32_t threshold;     // kept: number >= threshold; 65536 drops all
  float scale;            // 65536 / (65536 - threshold)
};
struct DropKey {
  uint32_t k0, k1, c2, c3;
};
__device__ __forceinline__ DropKey drop_key(const uint64_t* rng) {
  const uint64_t seed = rng[0], offset = rng[1];
  return {(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)offset, (uint32_t)(offset >> 32)};
}
// x[j] = kept ? x[j] * scale : 0 for the 8 elements of vector `vec` of `row`.
__device__ __forceinline__ void drop8(const DropKey& key, DropRule rule, uint32_t vec, uint32_t row,
                                      float x[8]) {
  uint32_t c0 = vec, c1 = row, c2 = key.c2, c3 = key.c3, k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)b;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  const uint32_t w[4] = {c0, c1, c2, c3};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = (w[j] & 0xFFFFu) >= rule.threshold ? x[2 * j] * rule.scale : 0.0f;
    x[2 * j + 1] = (w[j] >> 16) >= rule.threshold ? x[2 * j + 1] * rule.scale : 0.0f;
  }
}
// Host: the rule for p, and whether p is one.
inline bool drop_rule(float p, DropRule* r) {
  if (!(p >= 0.0f && p <= 1.0f)) return false;
  r->threshold = (uint32_t)std::nearbyint((double)p * 65536.0);
  r->scale = r->threshold < 65536u ? 65536.0f / (float)(65536u - r->threshold) : 0.0f;
  return true;
}

// ------------------------------------------------------------------ INT8 codes
// q = rint(127 x / m) for the row's largest magnitude m, ties to even.  The quotient t
// of p = 127 x by m is formed as t0 = p y, t = t0 + (p - t0 m) y with y = fl(1 / m): the
// remainder in the middle is exact, so t is the quotient itself wherever that is
// a binary32 value, halves among them, and within an ulp elsewhere.  For x of 16 bits p is
// exact and a quotient that is no half is at least 2^-12 from one, so the
// rounding of t decides as the exact quotient would.
// The magic addend rounds to nearest even and leaves the code in the low byte.
// A row with very large or small m is scaled by a power of two first (`up`), which
// keeps p and y in range.
struct RowScale {
  float m, inv, up;
};
__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {
  RowScale s;
  const float m = __uint_as_float(amax_bits);
  s.up = m > 0x1p100f ? 0x1p-100f : (m < 0x1p-20f ? 0x1p100f : 1.0f);
  s.m = m * s.up;
  s.inv = 1.0f / s.m;
  return s;
}
// Packs the codes of 8 values (bytes in order).  The row's amax is finite and not zero.
// EXACT32: x has 32 bits (FP32 tensors and a norm's values), so p is rounded and a quotient may be
// as close to a half as p's rounding error e: values next to a border (one in some thousands) are
// decided by the sign of |p - q m| + e - m / 2, whose terms are exact there.
template <bool EXACT32>
__device__ __forceinline__ uint2 codes8(const float x[8], const RowScale& s) {
  constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23
  uint32_t b[8];
  float v[8], worst = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = x[j];
  if (s.up != 1.0f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= s.up;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float p = v[j] * 127.0f, t0 = p * s.inv;
    const float t = __builtin_fmaf(__builtin_fmaf(-t0, s.m, p), s.inv, t0) + kMagic;
    b[j] = __float_as_uint(t);
    if constexpr (EXACT32)
      worst = __builtin_fmaxf(worst, __builtin_fabsf(__builtin_fmaf(kMagic - t, s.m, p)));
  }
  if constexpr (EXACT32) {
    const float half = s.m * 0.5f;
    if (worst >= half * 0.9999f) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float p = v[j] * 127.0f, e = __builtin_fmaf(v[j], 127.0f, -p);
        const float r = __builtin_fmaf(kMagic - __uint_as_float(b[j]), s.m, p);
        const float over = (__builtin_fabsf(r) - half) + (r < 0.0f ? -e : e);
        // past the border, or on it with an odd code (2^-149 stands for "more than zero")
        const bool move = over >= __uint_as_float(~b[j] & 1u);
        b[j] += move ? (r < 0.0f ? -1 : 1) : 0;
      }
    }
  }
  uint2 q;
  q.x = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400u),
                              __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), 0x05040100u);
  q.y = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[7], b[6], 0x0C0C0400u),
                              __builtin_amdgcn_perm(b[5], b[4], 0x0C0C0400u), 0x05040100u);
  return q;
}
// Largest magnitude of 8 values, as bits that order NaN above infinity above the rest;
// `top` is the running maximum.
__device__ __forceinline__ uint32_t magnitude8(const float w[8], uint32_t top) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t m = __float_as_uint(w[j]) & 0x7FFFFFFFu;
    top = m > top ? m : top;
  }
  return top;
}
__device__ __forceinline__ void store_codes8(int8_t* p, int n, uint2 q) {
  if (n >= 8) {
    __builtin_nontemporal_store(u32x2_b_t{q.x, q.y}, reinterpret_cast<u32x2_b_t*>(p));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = (int8_t)((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
  }
}

// ------------------------------------------------------------------ host checks
inline int64_t dtype_size(fp8dp_dtype t) { return t == FP8DP_F32 ? 4 : 2; }
inline bool known_dtype(fp8dp_dtype t) {
  return t == FP8DP_BF16 || t == FP8DP_F16 || t == FP8DP_F32;
}
inline bool aligned_to(const void* p, int64_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(n - 1)) == 0;
}
inline int check_rows(const char* what, int64_t rows, int64_t cols) {
  if (rows < 1 || cols < 1 || rows > 0x7FFFFFFF || cols > (1 << 30)) {
    set_error("%s: rows must be 1 .. 2^31 - 1 and cols 1 .. 2^30 (got %lld, %lld)", what, (long long)rows,
              (long long)cols);
    return FP8DP_EINVAL;
  }
  return FP8DP_OK;
}
inline int check_types(const char* what, fp8dp_dtype dt, fp8dp_dtype wt) {
  if (!known_dtype(dt) || !(wt == dt || wt == FP8DP_F32)) {
    set_error("%s: unknown type, or parameters neither of the activations' type nor binary32", what);
    return FP8DP_EINVAL;
  }
  return FP8DP_OK;
}
inline int bad_align(const char* what) {
  set_error("%s: every pointer must be aligned to its elements", what);
  return FP8DP_EINVAL;
}

}  // namespace fp8dp
