// block_norm_bwd.hip -- gradients of block_norm.hip's pass, in one pass over the rows.
//
//   xh = x post_rstd, zh = z pre_rstd, c = dy pre_weight
//   dz = dz_add + pre_rstd (c - zh mean(c zh)),       dresidual = a dz
//   dw_pre = sum over rows of dy zh
//   e = b gate dz,   dx = post_rstd (e w_post - xh mean(e w_post xh))
//   dw_post = sum over rows of e xh,   dgate = b dz xh w_post, summed over rows where they share it
//
// With a gate per channel both of its sums are one: P = sum over rows of dz xh, dw_post = b gate P and
// dgate = b w_post P; with one per token the sum is of gate dz xh.  So every form has two sums per column.
// Rows of 8 to 8192 elements (of up to 16384 where there are at most 64 for each compute unit) are read once: a grid of resident workgroups walks the rows, each thread keeps the sums of its own columns, and
// the workgroups' sums are added by a second kernel in a fixed order (no atomics: the same
// call gives the same bits).  dz stays in registers between the row's two reductions.
// Bound by memory with as many writes as reads nearly: 16384 x 4096 with a gate per token 205 us (5.2 TB/s), with one per
// channel 155, 16384 x 768 36 (a quarter of the slots for vectors is empty).  Rows of 8193 to 16384 are bound by registers: the
// compiler moves their parameters out of the loop over rows, and of the 128 registers a thread has it then spills up to 123
// more (488 bytes a lane in bfloat16 with both norms and a gate per channel, 416 with one per token, 496 and 428 in float16,
// 388 and 420 in binary32, whose 512-thread forms spill 44 and 200): 2048 x 16384 132 us for 60 of bytes.  What is left to
// the kernel that reads a row again by each step is slow: 16384 x 12288 572 us, one row more 3290; 65536 x 7 2100.
#include <hip/hip_runtime.h>

#include "row_core.hpp"

namespace fp8dp {

struct BlockNormBwdArgs {
  const void *dy, *dz_add, *x, *z, *post, *gate, *pre;
  const float *post_rstd, *pre_rstd;
  int64_t rows;
  int cols;
  bool wf32, gate_f32, sums;
  float a, b;
  void *dresidual, *dx, *dgate;   // dgate: per token only
  float* parts;                   // [workgroups][2][cols]: P or its form with the gate, dw_pre
};

// One vector behind the first reduction: dz, stored as the residual's gradient.
template <typename T>
__device__ __forceinline__ void block_dz(const BlockNormBwdArgs& a, int64_t at, int n, const float dy[8],
                                         const float zh[8], const float p[8], const float add[8],
                                         float rstd, float mean, float dz[8]) {
  float out[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    dz[j] = __builtin_fmaf(rstd, dy[j] * p[j] - zh[j] * mean, add[j]);
    out[j] = a.a * dz[j];
  }
  if (n > 0) store8(static_cast<T*>(a.dresidual) + at, n, out);
}

constexpr int kBlockWaves = 4;
constexpr int kBlockHeld = 64;   // rows whose sums stay in registers before they join those of earlier rows

// TOKEN: a gate per token and channel.  BRANCH: gradients of x, its norm and gate.  NORM: there is a dy.
template <typename T, int NV, int THR, bool TOKEN, bool BRANCH, bool NORM, bool STREAM>
__global__ __launch_bounds__(THR == 64 ? 64 * kBlockWaves : THR) void k_block_bwd(BlockNormBwdArgs a) {
  // HELD: parameters, sums and the next row in registers; 1024 threads have 128 registers each, and keep their sums in LDS
  constexpr bool HELD = THR < 1024;
  constexpr int RPB = THR == 64 ? kBlockWaves : 1, THREADS = RPB * THR, WAVES = THR / 64;
  __shared__ float lds[NV * 16 * THREADS + (THR == 64 ? 0 : 2 * 2 * WAVES)];
  float* const earlier = lds + threadIdx.x;
  float* const scratch = lds + NV * 16 * THREADS;
  const int t = THR > 64 ? (int)threadIdx.x : (int)(threadIdx.x & 63);
  const int sub = THR > 64 ? 0 : (int)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cols = a.cols;
  const bool ragged = cols % 8 != 0;
  const float inv_cols = 1.0f / (float)cols;
  const T *const dy = static_cast<const T*>(a.dy), *const z = static_cast<const T*>(a.z),
          *const add = static_cast<const T*>(a.dz_add), *const x = static_cast<const T*>(a.x),
          *const gate = static_cast<const T*>(a.gate);
  auto column = [&](int i) { return (i * THR + t) * 8; };
  const int n_last = cols - column(NV - 1);
  auto count = [&](int i) { return i < NV - 1 ? 8 : n_last; };
  const Mask8 mask(n_last);

  // the row in hand and the next one, still as loaded
  struct Row {
    Raw8<T> dy[NORM ? NV : 1], z[NORM ? NV : 1], add[NV], x[BRANCH ? NV : 1], g[TOKEN ? NV : 1];
    float r1, r2;
  };
  auto load = [&](int64_t row, Row& o) {
    const int64_t base = row * cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (NORM) {
        o.dy[i] = load_row<STREAM>(dy + base, column(i), cols);
        o.z[i] = load_row<STREAM>(z + base, column(i), cols);
      }
      if (add != nullptr) o.add[i] = load_row<STREAM>(add + base, column(i), cols);
      if constexpr (BRANCH) o.x[i] = load_row<STREAM>(x + base, column(i), cols);
      if constexpr (TOKEN) o.g[i] = load_row<STREAM>(gate + base, column(i), cols);
    }
    if constexpr (BRANCH) o.r1 = a.post_rstd[row];
    if constexpr (NORM) o.r2 = a.pre_rstd[row];
  };
  auto widen = [&](Raw8<T> raw, int i, float v[8]) {
    if (i == NV - 1) {
      settle(raw, n_last, ragged);
      mask.clear_empty(raw);
    }
    widen8f(raw, v);
  };
  const int64_t step = (int64_t)gridDim.x * RPB, first = (int64_t)blockIdx.x * RPB + sub;
  Row next;
  if constexpr (HELD) load(first < a.rows ? first : a.rows - 1, next);   // (a spare wave loads the last row)

  constexpr int HV = HELD ? NV : 1;
  float held_w[HV][8], held_p[HV][8], s1[HV][8], s2[HV][8];
  // what e w_post is of dz: b gate w_post, or b w_post with a gate per token
  auto load_w = [&](int i, float w[8]) {
    load_param8<T>(a.post, a.wf32, column(i), count(i), 1.0f, w);
    float g[8];
    load_param8<T>(TOKEN ? nullptr : a.gate, a.gate_f32, column(i), count(i), 1.0f, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] *= a.b * g[j];
  };
  auto load_p = [&](int i, float p[8]) { load_param8<T>(a.pre, a.wf32, column(i), count(i), 1.0f, p); };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (HELD) {
      if constexpr (BRANCH) load_w(i, held_w[i]);
      if constexpr (NORM) load_p(i, held_p[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) s1[i][j] = s2[i][j] = 0.0f;
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) earlier[(i * 16 + j) * THREADS] = 0.0f;
    }
  }
  auto weight = [&](int i, float w[8]) {
    if constexpr (HELD) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = held_w[i][j];
    } else {
      load_w(i, w);
    }
  };
  auto pre = [&](int i, float p[8]) {
    if constexpr (HELD) {
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = held_p[i][j];
    } else {
      load_p(i, p);
    }
  };
  // adds x y to the first or second sum of column j of vector i
  auto add1 = [&](int i, int j, float x, float y) {
    if constexpr (HELD) s1[i][j] = __builtin_fmaf(x, y, s1[i][j]);
    else earlier[(i * 16 + j) * THREADS] = __builtin_fmaf(x, y, earlier[(i * 16 + j) * THREADS]);
  };
  auto add2 = [&](int i, int j, float x, float y) {
    if constexpr (HELD) s2[i][j] = __builtin_fmaf(x, y, s2[i][j]);
    else earlier[(i * 16 + 8 + j) * THREADS] = __builtin_fmaf(x, y, earlier[(i * 16 + 8 + j) * THREADS]);
  };

  // (A cut vector is read as its row's last 8 elements, the first of which another wave may have written in place already: these
  // are shifted out, so that no order is needed between the two.)
  int turn = 0;
  bool more = false;   // there are sums of earlier rows
  for (int64_t row = first;;) {
    const int64_t stop = HELD ? std::min(row + kBlockHeld * step, a.rows) : a.rows;
    for (; row < stop; row += step, turn ^= 1) {
      float* const sc = scratch + (THR > 64 ? turn * 2 * WAVES : 0);
      const int64_t base = row * cols;
      if constexpr (!HELD) load(row, next);
      const Row now = next;
      if constexpr (HELD) load(row + step < a.rows ? row + step : row, next);
      float mean = 0.0f, dz[NV][8];
      if constexpr (NORM) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float vd[8], zh[8], p[8];
          widen(now.dy[i], i, vd);
          widen(now.z[i], i, zh);
          pre(i, p);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            zh[j] *= now.r2;
            mean = __builtin_fmaf(vd[j] * p[j], zh[j], mean);
            add2(i, j, vd[j], zh[j]);
          }
        }
        mean = row_sum<THR>(mean, sc) * inv_cols;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float vd[8] = {}, zh[8] = {}, va[8] = {}, p[8] = {};
        if constexpr (NORM) {
          pre(i, p);
          widen(now.dy[i], i, vd);
          widen(now.z[i], i, zh);
#pragma unroll
          for (int j = 0; j < 8; ++j) zh[j] *= now.r2;
        }
        if (add != nullptr) widen(now.add[i], i, va);
        block_dz<T>(a, base + column(i), count(i), vd, zh, p, va, NORM ? now.r2 : 0.0f, mean, dz[i]);
      }
      if constexpr (BRANCH) {
        mean = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (i == NV - 1) mask.clear(dz[i]);   // (0 times a row's infinity)
          float xh[8], g[8], dg[8], w[8];
          weight(i, w);
          widen(now.x[i], i, xh);
          if constexpr (TOKEN) widen(now.g[i], i, g);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            xh[j] *= now.r1;
            if constexpr (TOKEN) {
              dg[j] = dz[i][j] * w[j] * xh[j];
              dz[i][j] *= g[j];
            }
            add1(i, j, dz[i][j], xh[j]);
            dz[i][j] *= w[j];
            mean = __builtin_fmaf(dz[i][j], xh[j], mean);
          }
          if constexpr (TOKEN)
            if (a.dgate != nullptr && count(i) > 0)
              store8(static_cast<T*>(a.dgate) + base + column(i), count(i), dg);
        }
        mean = row_sum<THR>(mean, sc + WAVES) * inv_cols;
        if (a.dx != nullptr) {
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            float xh[8];
            widen(now.x[i], i, xh);
#pragma unroll
            for (int j = 0; j < 8; ++j) dz[i][j] = now.r1 * (dz[i][j] - xh[j] * now.r1 * mean);
            if (count(i) > 0) store8(static_cast<T*>(a.dx) + base + column(i), count(i), dz[i]);
          }
        }
      }
    }
    if (row >= a.rows) break;
    if constexpr (HELD) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float *const e1 = earlier + (i * 16 + j) * THREADS, *const e2 = e1 + 8 * THREADS;
          *e1 = more ? *e1 + s1[i][j] : s1[i][j];
          *e2 = more ? *e2 + s2[i][j] : s2[i][j];
          s1[i][j] = s2[i][j] = 0.0f;
        }
      more = true;
    }
  }
  if (!a.sums) return;
  if constexpr (HELD) {
    if (more) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s1[i][j] += earlier[(i * 16 + j) * THREADS];
          s2[i][j] += earlier[(i * 16 + 8 + j) * THREADS];
        }
    }
  }
  if constexpr (THR == 64) {
    // the waves' sums, halved in two steps through LDS (lane-major: no conflicts)
#pragma unroll
    for (int s = kBlockWaves / 2; s > 0; s >>= 1) {
      __syncthreads();
      if (sub >= s && sub < 2 * s) {
        float* const o = lds + (sub - s) * NV * 16 * 64 + t;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            o[(i * 16 + j) * 64] = s1[i][j];
            o[(i * 16 + 8 + j) * 64] = s2[i][j];
          }
      }
      __syncthreads();
      if (sub < s) {
        const float* const o = lds + sub * NV * 16 * 64 + t;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            s1[i][j] += o[(i * 16 + j) * 64];
            s2[i][j] += o[(i * 16 + 8 + j) * 64];
          }
      }
    }
    if (sub != 0) return;
  }
  float* const out = a.parts + (int64_t)blockIdx.x * 2 * cols;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (count(i) > 0) {
      float v1[8], v2[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v1[j] = HELD ? s1[HELD ? i : 0][j] : earlier[(i * 16 + j) * THREADS];
        v2[j] = HELD ? s2[HELD ? i : 0][j] : earlier[(i * 16 + 8 + j) * THREADS];
      }
      store8(out + column(i), count(i), v1);
      store8(out + cols + column(i), count(i), v2);
    }
}

// Rows beyond the registers, or below one vector: a workgroup per row, read once per reduction and
// once for the outputs.  The sums live in the workgroup's own words of the workspace (they stay in
// L2); with several rows a workgroup, what an addition rounds off is kept in a second set of
// them, `halves` sets behind, so that the error does not grow with the rows.
template <typename T, bool TOKEN>
__global__ __launch_bounds__(1024) void k_block_bwd_long(BlockNormBwdArgs a, int64_t halves) {
  __shared__ float lds[2 * 2 * 16];
  const int t = threadIdx.x, cols = a.cols;
  const float inv_cols = 1.0f / (float)cols;
  const T *const dy = static_cast<const T*>(a.dy), *const z = static_cast<const T*>(a.z),
          *const add = static_cast<const T*>(a.dz_add), *const x = static_cast<const T*>(a.x);
  float* const sums = a.parts + (int64_t)blockIdx.x * 2 * cols;
  float* const lost = sums + halves * 2 * cols;
  int turn = 0;
  bool more = false;
  auto join = [&](int64_t c, int n, const float v[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= n) continue;
      float s = v[j], e = 0.0f;
      if (more) {
        LongSum l;
        l.s = sums[c + j];
        l.e = lost[c + j];
        l.add(v[j]);
        s = l.s;
        e = l.e == l.e ? l.e : 0.0f;   // (an infinite sum stays one)
      }
      sums[c + j] = s;
      if (halves > 0) lost[c + j] = e;
    }
  };
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1, more = true) {
    const float r1 = x != nullptr ? a.post_rstd[row] : 0.0f, r2 = dy != nullptr ? a.pre_rstd[row] : 0.0f;
    const int64_t base = row * cols;
    float m1 = 0.0f, m2 = 0.0f;
    // dy, zh and pre_weight of the vector at c
    auto normed = [&](int64_t c, int n, float vd[8], float zh[8], float p[8]) {
      load8(dy + base + c, n, vd);
      load8(z + base + c, n, zh);
      load_param8<T>(a.pre, a.wf32, c, n, 1.0f, p);
#pragma unroll
      for (int j = 0; j < 8; ++j) zh[j] *= r2;
    };
    if (dy != nullptr) {
      LongSum s;
      for (int64_t c = (int64_t)t * 8; c < cols; c += 8192) {
        const int n = (int)(cols - c);
        float vd[8], zh[8], p[8];
        normed(c, n, vd, zh, p);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] *= vd[j] * zh[j];
        s.add(sum8(p));
        if (a.sums) {
#pragma unroll
          for (int j = 0; j < 8; ++j) vd[j] *= zh[j];
          join(cols + c, n, vd);
        }
      }
      m1 = row_sum<1024>(s.total(), lds + turn * 32) * inv_cols;
    }
    LongSum s;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      for (int64_t c = (int64_t)t * 8; c < cols; c += 8192) {
        const int n = (int)(cols - c);
        float dz[8] = {};
        if (add != nullptr) load8(add + base + c, n, dz);
        if (dy != nullptr) {
          float vd[8], zh[8], p[8];
          normed(c, n, vd, zh, p);
#pragma unroll
          for (int j = 0; j < 8; ++j) dz[j] = __builtin_fmaf(r2, vd[j] * p[j] - zh[j] * m1, dz[j]);
        }
        float xh[8], w[8], g[8], dg[8];
        if (x != nullptr) {
          load8(x + base + c, n, xh);
          load_param8<T>(a.post, a.wf32, c, n, 1.0f, w);
          if constexpr (TOKEN) load8(static_cast<const T*>(a.gate) + base + c, n, g);
          else load_param8<T>(a.gate, a.gate_f32, c, n, 1.0f, g);
          zero_from8(n, dz);
        }
        if (pass == 0) {
          if (x == nullptr) continue;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            xh[j] *= r1;
            dg[j] = a.b * dz[j] * w[j] * xh[j];
            w[j] = dg[j] * g[j];
            xh[j] *= TOKEN ? g[j] * dz[j] : dz[j];
          }
          s.add(sum8(w));
          if (a.sums) join(c, n, xh);
        } else {
          // in place of dy or dz_add: this thread has read both at c for the last time
          if (x != nullptr && TOKEN && a.dgate != nullptr) {
#pragma unroll
            for (int j = 0; j < 8; ++j) dg[j] = a.b * dz[j] * w[j] * (xh[j] * r1);
            store8(static_cast<T*>(a.dgate) + base + c, n, dg);
          }
          if (x != nullptr && a.dx != nullptr) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              w[j] = r1 * (a.b * g[j] * w[j] * dz[j] - xh[j] * r1 * m2);
            store8(static_cast<T*>(a.dx) + base + c, n, w);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) dz[j] *= a.a;
          store8(static_cast<T*>(a.dresidual) + base + c, n, dz);
        }
      }
      if (pass == 0 && x != nullptr) m2 = row_sum<1024>(s.total(), lds + turn * 32 + 16) * inv_cols;
    }
  }
}

// The gradients of the weights and of a gate per channel, from `nparts` partial sums of 2 * cols values:
// 32 columns and 32 ranges of the sums per workgroup, joined in LDS in a fixed order.
struct BlockPartsArgs {
  const float* parts;
  int nparts, cols;
  const void *post, *gate;   // gate: per channel only
  bool wf32, gate_f32;
  float b;
  float *dpost, *dpre, *dgate;
};
template <typename T>
__global__ __launch_bounds__(1024) void k_block_parts(BlockPartsArgs a) {
  __shared__ float lds[32][33];
  const int col = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int64_t width = 2 * (int64_t)a.cols;
  for (int64_t c0 = (int64_t)blockIdx.x * 32; c0 < width; c0 += (int64_t)gridDim.x * 32) {
    const int64_t c = c0 + col;
    float s = 0.0f;
    if (c < width) {
#pragma unroll 8
      for (int i = part; i < a.nparts; i += 32) s += a.parts[i * width + c];
    }
    lds[part][col] = s;
    __syncthreads();
    if (part == 0 && c < width) {
      float v[4] = {};
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i & 3] += lds[i][col];
      const float total = (v[0] + v[1]) + (v[2] + v[3]);
      if (c >= a.cols) {
        if (a.dpre != nullptr) a.dpre[c - a.cols] = total;
      } else {
        auto one = [&](const void* p, bool f32) {
          return p == nullptr ? 1.0f : f32 ? static_cast<const float*>(p)[c] : to_f32(static_cast<const T*>(p)[c]);
        };
        if (a.dpost != nullptr) a.dpost[c] = a.b * one(a.gate, a.gate_f32) * total;
        if (a.dgate != nullptr) a.dgate[c] = a.b * one(a.post, a.wf32) * total;
      }
    }
    __syncthreads();
  }
}

template <typename T>
static int launch_block_parts(const BlockPartsArgs& p, hipStream_t stream) {
  const int64_t blocks = std::min<int64_t>((2 * (int64_t)p.cols + 31) / 32, 1 << 16);
  hipLaunchKernelGGL((k_block_parts<T>), dim3((unsigned)blocks), dim3(1024), 0, stream, p);
  return check_launch("block_norm_backward");
}

template <typename T, int NV, int THR, bool TOKEN, bool BRANCH, bool NORM, bool STREAM>
static int launch_block_bwd_as(const BlockNormBwdArgs& a, BlockPartsArgs p, hipStream_t stream) {
  constexpr int RPB = THR == 64 ? kBlockWaves : 1;
  static const int resident = [] {
    int n = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, (k_block_bwd<T, NV, THR, TOKEN, BRANCH, NORM, STREAM>),
                                                     RPB * THR, 0) != hipSuccess || n < 1)
      n = 1;
    return std::min(n, std::max(1, 16 * 64 / (NV * RPB * THR)));
  }();
  const int64_t cap = std::min<int64_t>(FP8DP_NORM_PARTS, (int64_t)num_cus() * resident);
  const int64_t grid = std::min<int64_t>((a.rows + RPB - 1) / RPB, cap);
  hipLaunchKernelGGL((k_block_bwd<T, NV, THR, TOKEN, BRANCH, NORM, STREAM>), dim3((unsigned)grid), dim3(RPB * THR), 0,
                     stream, a);
  const int rc = check_launch("block_norm_backward");
  if (rc || !a.sums) return rc;
  p.nparts = (int)grid;
  return launch_block_parts<T>(p, stream);
}

// Beyond the 256 MB of the last-level cache: read past the caches (16384 x 4096 with a gate per token 213 us, now 205).
template <typename T, int NV, int THR, bool TOKEN, bool BRANCH, bool NORM>
static int launch_block_bwd(const BlockNormBwdArgs& a, const BlockPartsArgs& p, hipStream_t stream) {
  const int64_t tensors = 1 + 2 * NORM + (a.dz_add != nullptr) + (BRANCH ? 1 + (a.dx != nullptr) : 0) +
                          (TOKEN ? 1 + (a.dgate != nullptr) : 0);
  if (a.rows * a.cols * tensors * (int64_t)sizeof(T) > ((int64_t)256 << 20))
    return launch_block_bwd_as<T, NV, THR, TOKEN, BRANCH, NORM, true>(a, p, stream);
  return launch_block_bwd_as<T, NV, THR, TOKEN, BRANCH, NORM, false>(a, p, stream);
}

template <typename T, bool TOKEN, bool BRANCH, bool NORM>
static int launch_block_width(const BlockNormBwdArgs& a, BlockPartsArgs p, hipStream_t stream) {
  const int nvec = (a.cols + 7) / 8;
  if (a.cols >= 8) {
    if (nvec <= 64) return launch_block_bwd<T, 1, 64, TOKEN, BRANCH, NORM>(a, p, stream);
    if (nvec <= 128) return launch_block_bwd<T, 2, 64, TOKEN, BRANCH, NORM>(a, p, stream);
    if (nvec <= 256) return launch_block_bwd<T, 1, 256, TOKEN, BRANCH, NORM>(a, p, stream);
    if (nvec <= 512) return launch_block_bwd<T, 2, 256, TOKEN, BRANCH, NORM>(a, p, stream);
    if (nvec <= 1024) return launch_block_bwd<T, 2, 512, TOKEN, BRANCH, NORM>(a, p, stream);
    // sums of up to 64 rows each, one after another, and no more: what they round off is not kept (2048 x 16384: 558 us by
    // the kernel below)
    if (nvec <= 2048 && a.rows <= 64 * (int64_t)num_cus())
      return launch_block_bwd<T, 2, 1024, TOKEN, BRANCH, NORM>(a, p, stream);
  }
  // below FP8DP_NORM_PARTS rows each has a workgroup; of more, half the parts are sums and half what they lost
  const bool one = a.rows < FP8DP_NORM_PARTS;
  const int64_t grid = one ? a.rows : FP8DP_NORM_PARTS / 2;
  hipLaunchKernelGGL((k_block_bwd_long<T, TOKEN>), dim3((unsigned)grid), dim3(1024), 0, stream, a,
                     one ? (int64_t)0 : grid);
  const int rc = check_launch("block_norm_backward");
  if (rc || !a.sums) return rc;
  p.nparts = (int)(one ? grid : 2 * grid);
  return launch_block_parts<T>(p, stream);
}

template <typename T>
static int launch_block_kind(const BlockNormBwdArgs& a, const BlockPartsArgs& p, bool token,
                             hipStream_t stream) {
  if (a.x == nullptr) return launch_block_width<T, false, false, true>(a, p, stream);
  if (a.dy == nullptr)
    return token ? launch_block_width<T, true, true, false>(a, p, stream)
                   : launch_block_width<T, false, true, false>(a, p, stream);
  return token ? launch_block_width<T, true, true, true>(a, p, stream)
                 : launch_block_width<T, false, true, true>(a, p, stream);
}

}  // namespace fp8dp

using namespace fp8dp;

extern "C" int block_norm_backward(const void* dy, const void* dz_add, const void* x, const void* z,
                                   const void* post_weight, const void* gate, int32_t gate_per_token,
                                   const void* pre_weight, const float* post_rstd,
                                   const float* pre_rstd, int64_t rows, int64_t cols, fp8dp_dtype dt,
                                   fp8dp_dtype wt, fp8dp_dtype gt, float residual_scale,
                                   float branch_scale, void* dresidual, void* dx, void* dgate,
                                   float* dpost_weight, float* dpre_weight, float* workspace,
                                   hipStream_t stream) {
  const char* what = "block_norm_backward";
  int rc = check_rows(what, rows, cols);   // first: an empty tensor has no address
  if (rc) return rc;
  if (dresidual == nullptr || (dy == nullptr && dz_add == nullptr) || (dy == nullptr && x == nullptr)) {
    set_error("%s: dresidual, dy or dz_add, and dy or x must be non-NULL", what);
    return FP8DP_EINVAL;
  }
  if (dy != nullptr ? z == nullptr || pre_rstd == nullptr
                    : pre_weight != nullptr || dpre_weight != nullptr) {
    set_error("%s: dy comes with z and pre_rstd, and pre_weight and its gradient with dy", what);
    return FP8DP_EINVAL;
  }
  if (x != nullptr ? post_rstd == nullptr
                   : post_weight != nullptr || gate != nullptr || dx != nullptr || dgate != nullptr ||
                         dpost_weight != nullptr) {
    set_error("%s: x comes with post_rstd, and post_weight, gate and the gradients of the three with x", what);
    return FP8DP_EINVAL;
  }
  if (dgate != nullptr && gate == nullptr) {
    set_error("%s: dgate needs the gate", what);
    return FP8DP_EINVAL;
  }
  const bool token = gate != nullptr && gate_per_token != 0;
  if ((rc = check_types(what, dt, wt)) || (rc = check_types(what, dt, gt))) return rc;
  if (token && gt != dt) {
    set_error("%s: a gate per token has the activations' type", what);
    return FP8DP_EINVAL;
  }
  const float top = 3.402823466e38f;
  if (!(std::fabs(residual_scale) <= top) || !(std::fabs(branch_scale) <= top)) {
    set_error("%s: the scales must be finite", what);
    return FP8DP_EINVAL;
  }
  const bool sums = dpost_weight != nullptr || dpre_weight != nullptr || (dgate != nullptr && !token);
  if (sums && workspace == nullptr) {
    set_error("%s: gradients of weights and of a gate per channel need a workspace", what);
    return FP8DP_EINVAL;
  }
  const int64_t e = dtype_size(dt), we = dtype_size(wt);
  if (!aligned_to(dy, e) || !aligned_to(dz_add, e) || !aligned_to(x, e) || !aligned_to(z, e) ||
      !aligned_to(post_weight, we) || !aligned_to(gate, dtype_size(gt)) || !aligned_to(pre_weight, we) ||
      !aligned_to(post_rstd, 4) || !aligned_to(pre_rstd, 4) || !aligned_to(dresidual, e) ||
      !aligned_to(dx, e) || !aligned_to(dgate, token ? e : 4) || !aligned_to(dpost_weight, 4) ||
      !aligned_to(dpre_weight, 4) || !aligned_to(workspace, 4))
    return bad_align(what);
  const void* const gates = token ? nullptr : dgate;
  if (shared_buffers({dresidual, dx, dgate, dpost_weight, dpre_weight},
                     {x, z, gate, post_weight, pre_weight, post_rstd, pre_rstd, sums ? workspace : nullptr}) ||
      shared_buffers({gates, dpost_weight, dpre_weight}, {dy, dz_add})) {
    set_error("%s: gradients and inputs must be different buffers, but for dresidual, dx and a dgate per token in place of "
              "dy or dz_add", what);
    return FP8DP_EINVAL;
  }
  BlockNormBwdArgs a = {};
  a.dy = dy;
  a.dz_add = dz_add;
  a.x = x;
  a.z = z;
  a.post = post_weight;
  a.gate = gate;
  a.pre = pre_weight;
  a.post_rstd = post_rstd;
  a.pre_rstd = pre_rstd;
  a.rows = rows;
  a.cols = (int)cols;
  a.wf32 = wt == FP8DP_F32;
  a.gate_f32 = gt == FP8DP_F32;
  a.sums = sums;
  a.a = x != nullptr ? residual_scale : 1.0f;   // without x, z is the residual
  a.b = branch_scale;
  a.dresidual = dresidual;
  a.dx = dx;
  a.dgate = token ? dgate : nullptr;
  a.parts = workspace;
  BlockPartsArgs p = {};
  p.parts = workspace;
  p.cols = (int)cols;
  p.post = post_weight;
  p.gate = token ? nullptr : gate;
  p.wf32 = a.wf32;
  p.gate_f32 = a.gate_f32;
  p.b = branch_scale;
  p.dpost = dpost_weight;
  p.dpre = dpre_weight;
  p.dgate = token ? nullptr : static_cast<float*>(dgate);
  if (dt == FP8DP_BF16) return launch_block_kind<bf16_t>(a, p, token, stream);
  if (dt == FP8DP_F16) return launch_block_kind<f16_t>(a, p, token, stream);
  return launch_block_kind<float>(a, p, token, stream);
}
