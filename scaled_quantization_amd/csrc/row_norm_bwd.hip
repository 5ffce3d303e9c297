// row_norm_bwd.hip -- layer norm's backward pass, with the residual stream's
// gradient added and the dropout mask applied again where asked.
//
//   g = dy w, h = (z - mean) rstd
//   dz = rstd (g - mean(g) - h mean(g h)) + dz_add,  dx = keep dz / (1 - p)
//   dw = sum over rows of dy h,  db = sum over rows of dy
//
// Rows of 8 to 8192 elements in one pass, which reads dy and z once: a persistent grid walks the rows,
// a wave or workgroup per row as in the forward kernels, and each thread keeps the weight
// gradients of its own columns over all its rows.  The partial sums of a workgroup go to the
// workspace once, and a second kernel adds them in a fixed order (no atomics, so the same
// call gives the same bits).  Other rows are read three times: by a kernel for the weight
// gradients, and twice by one for dz.
#include <hip/hip_runtime.h>

#include "row_core.hpp"

namespace fp8dp {

struct NormBwdArgs {
  const void *dy, *z, *weight, *dz_add;
  const float *mean, *rstd;
  int64_t rows;
  int cols;
  bool wf32, sums;
  DropRule rule;
  const uint64_t* rng;
  void *dz, *dx;
  float* parts;        // [workgroups][2][cols]
};

// h and g of one vector.  h takes the difference first, whatever the type: a fused z rstd - mean rstd
// would round mean rstd, which a row far from zero makes many times h, and dweight, which is
// binary32, would show it.
__device__ __forceinline__ void norm_hg(const float z[8], const float dy[8], const float w[8],
                                        float mean, float rstd, float h[8], float g[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    h[j] = (z[j] - mean) * rstd;
    g[j] = dy[j] * w[j];
  }
}

template <typename T, bool DROP>
__device__ __forceinline__ void norm_out(const NormBwdArgs& a, const DropKey& key, int64_t row,
                                         int vec, int n, const float h[8], const float g[8],
                                         const float add[8], float rstd, float mg, float mgh) {
  const int64_t base = row * a.cols;
  float d[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    d[j] = __builtin_fmaf(h[j], -mgh * rstd, __builtin_fmaf(g[j], rstd, -mg * rstd));
  if (a.dz_add != nullptr) {
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j] += add[j];
  }
  store8(element(static_cast<T*>(a.dz) + base, vec * 8), n, d);
  if (a.dx != nullptr) {
    if constexpr (DROP) drop8(key, a.rule, (uint32_t)vec, (uint32_t)row, d);
    store8(element(static_cast<T*>(a.dx) + base, vec * 8), n, d);
  }
}

// Sums of two values over the THR threads of a row, one barrier.
template <int THR>
__device__ __forceinline__ void row_sum2(float& x, float& y, float* scratch) {
  x = wave_sum(x);
  y = wave_sum(y);
  if constexpr (THR > 64) {
    if ((threadIdx.x & 63) == 0) {
      scratch[2 * (threadIdx.x >> 6)] = x;
      scratch[2 * (threadIdx.x >> 6) + 1] = y;
    }
    __syncthreads();
    x = y = 0.0f;
#pragma unroll
    for (int i = 0; i < THR / 64; ++i) {
      x += scratch[2 * i];
      y += scratch[2 * i + 1];
    }
  }
}

constexpr int kBwdWaves = 4;   // waves of a workgroup whose waves own rows

// Rows whose weight gradients a thread sums in registers before that sum joins those of its earlier
// rows in its own words of LDS: 2^24 rows are two sums of 64 terms each, not one of 4096 whose
// roundings fall to one side (dbias of nearly equal gradients was off by 400 roundings).
constexpr int kBwdHeld = 64;

// STREAM: tensors beyond the caches, read past them.
template <typename T, int NV, int THR, bool DROP, bool STREAM>
__global__ __launch_bounds__(THR == 64 ? 64 * kBwdWaves : THR) void k_norm_bwd(NormBwdArgs a) {
  constexpr int RPB = THR == 64 ? kBwdWaves : 1, THREADS = RPB * THR;
  // the weight gradients of earlier rows, [16 NV][thread], and the scratch of a row's sums
  __shared__ float lds[NV * 16 * THREADS + (THR == 64 ? 0 : 2 * 2 * (THR / 64))];
  float* const earlier = lds + threadIdx.x;
  float* const scratch = lds + NV * 16 * THREADS;
  const int t = THR > 64 ? (int)threadIdx.x : (int)(threadIdx.x & 63);
  const int sub = THR > 64 ? 0 : (int)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cols = a.cols;
  const bool ragged = cols % 8 != 0;
  const float inv_cols = 1.0f / (float)cols;
  const T *const z = static_cast<const T*>(a.z), *const dy = static_cast<const T*>(a.dy),
          *const add = static_cast<const T*>(a.dz_add);
  DropKey key = {};
  if constexpr (DROP) key = drop_key(a.rng);
  auto column = [&](int i) { return (i * THR + t) * 8; };

  const int n_last = cols - column(NV - 1);
  const Mask8 mask(n_last);

  // the row in hand and the next one, still as loaded: a row's loads have a whole
  // row of arithmetic to arrive
  struct Row {
    Raw8<T> z[NV], dy[NV], add[NV];
    float mean, rstd;
  };
  auto load = [&](int64_t row, Row& r) {
    const int64_t base = row * cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      r.z[i] = load_row<STREAM>(z + base, column(i), cols);
      r.dy[i] = load_row<STREAM>(dy + base, column(i), cols);
      if (add != nullptr) r.add[i] = load_row<STREAM>(add + base, column(i), cols);
    }
    r.mean = a.mean[row];
    r.rstd = a.rstd[row];
  };
  const int64_t step = (int64_t)gridDim.x * RPB, first = (int64_t)blockIdx.x * RPB + sub;
  Row next;
  load(first < a.rows ? first : a.rows - 1, next);   // (a spare wave loads the last row)

  float w[NV][8], dw[NV][8], db[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_param8<T>(a.weight, a.wf32, column(i), cols - column(i), 1.0f, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = db[i][j] = 0.0f;
  }

  int turn = 0;
  bool more = false;   // there are sums of earlier rows
  for (int64_t row = first;;) {
    const int64_t stop = std::min(row + kBwdHeld * step, a.rows);
    for (; row < stop; row += step, turn ^= 1) {
      const Row r = next;
      load(row + step < a.rows ? row + step : row, next);
      float sg = 0.0f, sgh = 0.0f;
      // h and g of vector i (the compiler keeps them over the reduction where registers allow)
      auto make = [&](int i, float* h, float* g, float* vd) {
        float vz[8];
        Raw8<T> raw = r.z[i];
        if (i == NV - 1) settle(raw, n_last, ragged);
        widen8f(raw, vz);
        raw = r.dy[i];
        if (i == NV - 1) {
          settle(raw, n_last, ragged);
          mask.clear_empty(raw);
        }
        widen8f(raw, vd);
        norm_hg(vz, vd, w[i], r.mean, r.rstd, h, g);
      };
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float h[8], g[8], vd[8];
        make(i, h, g, vd);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          sg += g[j];
          sgh = __builtin_fmaf(g[j], h[j], sgh);
          dw[i][j] = __builtin_fmaf(vd[j], h[j], dw[i][j]);
          db[i][j] += vd[j];
        }
      }
      row_sum2<THR>(sg, sgh, scratch + (THR > 64 ? turn * 2 * (THR / 64) : 0));
      const float mg = sg * inv_cols, mgh = sgh * inv_cols;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int n = i < NV - 1 ? 8 : n_last;
        float va[8] = {};
        if (add != nullptr) {
          Raw8<T> raw = r.add[i];
          if (i == NV - 1) settle(raw, n_last, ragged);
          widen8f(raw, va);
        }
        float h[8], g[8], vd[8];
        make(i, h, g, vd);
        if (i < NV - 1 || n > 0)
          norm_out<T, DROP>(a, key, row, column(i) / 8, n, h, g, va, r.rstd, mg, mgh);
      }
    }
    if (row >= a.rows) break;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float *const ew = earlier + (i * 16 + j) * THREADS, *const eb = ew + 8 * THREADS;
        *ew = more ? *ew + dw[i][j] : dw[i][j];
        *eb = more ? *eb + db[i][j] : db[i][j];
        dw[i][j] = db[i][j] = 0.0f;
      }
    more = true;
  }
  if (!a.sums) return;
  if (more) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dw[i][j] += earlier[(i * 16 + j) * THREADS];
        db[i][j] += earlier[(i * 16 + 8 + j) * THREADS];
      }
  }

  if constexpr (THR == 64) {
    // the waves' sums, halved in two steps through LDS (lane-major: no conflicts)
#pragma unroll
    for (int s = kBwdWaves / 2; s > 0; s >>= 1) {
      __syncthreads();
      if (sub >= s && sub < 2 * s) {
        float* const o = lds + (sub - s) * NV * 16 * 64 + t;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            o[(i * 16 + j) * 64] = dw[i][j];
            o[(i * 16 + 8 + j) * 64] = db[i][j];
          }
      }
      __syncthreads();
      if (sub < s) {
        const float* const o = lds + sub * NV * 16 * 64 + t;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            dw[i][j] += o[(i * 16 + j) * 64];
            db[i][j] += o[(i * 16 + 8 + j) * 64];
          }
      }
    }
    if (sub != 0) return;
  }
  float* const p = a.parts + (int64_t)blockIdx.x * 2 * cols;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * THR + t) * 8, n = cols - c;
    if (n > 0) {
      store8(p + c, n, dw[i]);
      store8(p + cols + c, n, db[i]);
    }
  }
}

// Rows beyond the registers (and below one vector): dz by a workgroup per row, two reads of it; the
// weight gradients by k_norm_bwd_cols, a thread per 8 columns down a range of rows.
template <typename T, bool DROP>
__global__ __launch_bounds__(1024) void k_norm_bwd_long(NormBwdArgs a) {
  __shared__ float lds[2 * 2 * 16];
  const int t = threadIdx.x, cols = a.cols;
  const float inv_cols = 1.0f / (float)cols;
  DropKey key = {};
  if constexpr (DROP) key = drop_key(a.rng);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    float mg = 0.0f, mgh = 0.0f;
    LongSum sg, sgh;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      for (int64_t c = (int64_t)t * 8; c < cols; c += 8192) {
        const int n = (int)(cols - c);
        const int64_t at = row * cols + c;
        float z[8], dy[8], w[8], h[8], g[8];
        load8(static_cast<const T*>(a.z) + at, n, z);
        load8(static_cast<const T*>(a.dy) + at, n, dy);
        load_param8<T>(a.weight, a.wf32, c, n, 1.0f, w);
        norm_hg(z, dy, w, mean, rstd, h, g);
        if (pass == 0) {
          sg.add(sum8(g));
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] *= h[j];
          sgh.add(sum8(g));
        } else {
          float add[8] = {};
          if (a.dz_add != nullptr) load8(static_cast<const T*>(a.dz_add) + at, n, add);
          norm_out<T, DROP>(a, key, row, (int)(c / 8), n, h, g, add, rstd, mg, mgh);
        }
      }
      if (pass == 0) {
        mg = sg.total();
        mgh = sgh.total();
        row_sum2<1024>(mg, mgh, lds + turn * 32);
        mg *= inv_cols;
        mgh *= inv_cols;
      }
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_norm_bwd_cols(NormBwdArgs a) {
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  const int cols = a.cols, n = (int)(cols - c);
  if (c >= cols) return;
  LongSum dw[8], db[8];
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    float z[8], dy[8];
    load8(static_cast<const T*>(a.z) + row * cols + c, n, z);
    load8(static_cast<const T*>(a.dy) + row * cols + c, n, dy);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dw[j].add(dy[j] * ((z[j] - mean) * rstd));
      db[j].add(dy[j]);
    }
  }
  float sw[8], sb[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    sw[j] = dw[j].total();
    sb[j] = db[j].total();
  }
  float* const p = a.parts + (int64_t)blockIdx.y * 2 * cols;
  store8(p + c, n, sw);
  store8(p + cols + c, n, sb);
}

// dweight and dbias from `nparts` partial sums of 2 * cols values: 32 columns (a cache
// line of pairs) and 64 ranges of the sums per workgroup; the ranges are joined in LDS in a fixed order.
__global__ __launch_bounds__(1024) void k_norm_parts(const float* parts, int nparts, int cols,
                                                     float* dweight, float* dbias) {
  typedef float pair_t __attribute__((ext_vector_type(2), aligned(4)));
  __shared__ float lds[64][33];
  const int lane = threadIdx.x & 15, group = threadIdx.x >> 4;
  const int col = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int64_t width = 2 * (int64_t)cols;
  for (int64_t c0 = (int64_t)blockIdx.x * 32; c0 < width; c0 += (int64_t)gridDim.x * 32) {
    const int64_t c = c0 + 2 * lane;
    pair_t s = {0.0f, 0.0f};
    if (c < width) {
#pragma unroll 8
      for (int i = group; i < nparts; i += 64)
        s += *reinterpret_cast<const pair_t*>(parts + i * width + c);
    }
    lds[group][2 * lane] = s.x;
    lds[group][2 * lane + 1] = s.y;
    __syncthreads();
    // 32 columns x 8 ranges of 8, then the 8
    float v = 0.0f;
    if (part < 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v += lds[part * 8 + i][col];
    }
    __syncthreads();
    if (part < 8) lds[part][col] = v;
    __syncthreads();
    if (part == 0 && c0 + col < width) {
      float total = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) total += lds[i][col];
      if (c0 + col < cols) dweight[c0 + col] = total;
      else dbias[c0 + col - cols] = total;
    }
    __syncthreads();
  }
}

static int launch_parts(const NormBwdArgs& a, int nparts, float* dweight, float* dbias,
                        hipStream_t stream) {
  const int64_t blocks = std::min<int64_t>((2 * (int64_t)a.cols + 31) / 32, 1 << 16);
  hipLaunchKernelGGL(k_norm_parts, dim3((unsigned)blocks), dim3(1024), 0, stream, a.parts,
                     nparts, a.cols, dweight, dbias);
  return check_launch("layer_norm_backward");
}

template <typename T, int NV, int THR, bool DROP, bool STREAM>
static int launch_bwd_as(const NormBwdArgs& a, float* dweight, float* dbias, hipStream_t stream) {
  constexpr int RPB = THR == 64 ? kBwdWaves : 1;
  // A compute unit gets waves for 16 vectors of a row and no more: each has two rows of loads in
  // flight, and more of them only spread the reads and writes over more of memory (per
  // compute unit 8 waves of 2 vectors against 12: 65536 x 4096 270 / 303 us, 262144 x 768
  // 200 / 207, 16384 x 768 19.9 / 21.6; 16 waves of 1 against 8: 30001 x 1600 60 / 70).  All are
  // resident at once and walk the same number of rows.
  static const int resident = [] {
    int n = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, (k_norm_bwd<T, NV, THR, DROP, STREAM>),
                                                     RPB * THR, 0) != hipSuccess || n < 1)
      n = 1;
    return std::min(n, std::max(1, 16 * 64 / (NV * RPB * THR)));
  }();
  const int64_t cap = std::min<int64_t>(FP8DP_NORM_PARTS, (int64_t)num_cus() * resident);
  const int64_t grid = std::min<int64_t>((a.rows + RPB - 1) / RPB, cap);
  hipLaunchKernelGGL((k_norm_bwd<T, NV, THR, DROP, STREAM>), dim3((unsigned)grid), dim3(RPB * THR), 0,
                     stream, a);
  const int rc = check_launch("layer_norm_backward");
  if (rc || !a.sums) return rc;
  return launch_parts(a, (int)grid, dweight, dbias, stream);
}

// Beyond the 256 MB of the last-level cache: read past the caches (measured, with and without:
// 65536 x 4096 270 / 286 us, 262144 x 768 199 / 214; 16384 x 768, which they hold, 20.9 / 20.3
// and with dropout and residual 31.2 / 28.5).
template <typename T, int NV, int THR, bool DROP>
static int launch_bwd(const NormBwdArgs& a, float* dweight, float* dbias, hipStream_t stream) {
  const int64_t tensors = 3 + (a.dz_add != nullptr) + (a.dx != nullptr);
  if (a.rows * a.cols * tensors * (int64_t)sizeof(T) > ((int64_t)256 << 20))
    return launch_bwd_as<T, NV, THR, DROP, true>(a, dweight, dbias, stream);
  return launch_bwd_as<T, NV, THR, DROP, false>(a, dweight, dbias, stream);
}

template <typename T, bool DROP>
static int launch_bwd_long(const NormBwdArgs& a, float* dweight, float* dbias,
                           hipStream_t stream) {
  // the sums first: dz or dx may be written over dy
  if (a.sums) {
    const int64_t blocks = ((int64_t)a.cols + 2047) / 2048;
    const int64_t want = std::max<int64_t>(1, (int64_t)num_cus() * 8 / blocks);
    const int64_t parts = std::min<int64_t>({want, a.rows, FP8DP_NORM_PARTS});
    hipLaunchKernelGGL((k_norm_bwd_cols<T>), dim3((unsigned)blocks, (unsigned)parts), dim3(256), 0,
                       stream, a);
    int rc = check_launch("layer_norm_backward");
    if (rc || (rc = launch_parts(a, (int)parts, dweight, dbias, stream))) return rc;
  }
  hipLaunchKernelGGL((k_norm_bwd_long<T, DROP>),
                     dim3((unsigned)std::min<int64_t>(a.rows, (int64_t)num_cus() * 8)), dim3(1024),
                     0, stream, a);
  return check_launch("layer_norm_backward");
}

template <typename T, bool DROP>
static int launch_bwd_width(const NormBwdArgs& a, float* dweight, float* dbias,
                            hipStream_t stream) {
  const int64_t nvec = ((int64_t)a.cols + 7) / 8;
  if (a.cols < 8) return launch_bwd_long<T, DROP>(a, dweight, dbias, stream);
  if (nvec <= 64) return launch_bwd<T, 1, 64, DROP>(a, dweight, dbias, stream);
  if (nvec <= 128) return launch_bwd<T, 2, 64, DROP>(a, dweight, dbias, stream);
  if (nvec <= 256) return launch_bwd<T, 1, 256, DROP>(a, dweight, dbias, stream);
  if (nvec <= 512) return launch_bwd<T, 2, 256, DROP>(a, dweight, dbias, stream);
  // 128 registers a thread: 8 to 56 bytes a thread go to scratch with dropout, 12 in FP32, and it is
  // still the better side (against the two kernels below: 4096 x 8192 46 / 97 us, with dropout and
  // residual 71 / 116, FP32 84 / 149 and 157 / 195; 1024 x 4104 16 / 29)
  if (nvec <= 1024) return launch_bwd<T, 1, 1024, DROP>(a, dweight, dbias, stream);
  // two vectors per thread of 1024 spill all through: 4096 x 16384 took 299 us, this 155
  return launch_bwd_long<T, DROP>(a, dweight, dbias, stream);
}

template <bool DROP>
static int launch_bwd_type(fp8dp_dtype dt, const NormBwdArgs& a, float* dweight, float* dbias,
                           hipStream_t stream) {
  if (dt == FP8DP_BF16) return launch_bwd_width<bf16_t, DROP>(a, dweight, dbias, stream);
  if (dt == FP8DP_F16) return launch_bwd_width<f16_t, DROP>(a, dweight, dbias, stream);
  return launch_bwd_width<float, DROP>(a, dweight, dbias, stream);
}

}  // namespace fp8dp

using namespace fp8dp;

extern "C" int layer_norm_backward(const void* dy, const void* z, const void* weight,
                                   const float* mean, const float* rstd, const void* dz_add,
                                   int64_t rows, int64_t cols, fp8dp_dtype dt, fp8dp_dtype wt,
                                   float p, const uint64_t* rng, void* dz, void* dx,
                                   float* dweight, float* dbias, float* workspace,
                                   hipStream_t stream) {
  const char* what = "layer_norm_backward";
  int rc = check_rows(what, rows, cols);   // first: an empty tensor has no address
  if (rc) return rc;
  if (dy == nullptr || z == nullptr || mean == nullptr || rstd == nullptr || dz == nullptr) {
    set_error("%s: dy, z, mean, rstd and dz must be non-NULL", what);
    return FP8DP_EINVAL;
  }
  if ((dweight == nullptr) != (dbias == nullptr) || (dweight != nullptr && workspace == nullptr)) {
    set_error("%s: dweight and dbias go together, and need a workspace", what);
    return FP8DP_EINVAL;
  }
  NormBwdArgs a = {};
  if ((rc = check_types(what, dt, wt))) return rc;
  if (!drop_rule(p, &a.rule)) {
    set_error("%s: p must be 0 .. 1", what);
    return FP8DP_EINVAL;
  }
  if (dx != nullptr && p > 0.0f && rng == nullptr) {
    set_error("%s: p > 0 needs rng (seed and offset on the device)", what);
    return FP8DP_EINVAL;
  }
  const int64_t e = dtype_size(dt);
  if (!aligned_to(dy, e) || !aligned_to(z, e) || !aligned_to(dz_add, e) || !aligned_to(dz, e) ||
      !aligned_to(dx, e) || !aligned_to(weight, dtype_size(wt)) || !aligned_to(mean, 4) ||
      !aligned_to(rstd, 4) || !aligned_to(dweight, 4) || !aligned_to(dbias, 4) ||
      !aligned_to(workspace, 4) || !aligned_to(rng, 8))
    return bad_align(what);
  if (dz == dx || dz == z || dx == z) {
    set_error("%s: dz, dx and z must be different buffers", what);
    return FP8DP_EINVAL;
  }
  a.dy = dy;
  a.z = z;
  a.weight = weight;
  a.dz_add = dz_add;
  a.mean = mean;
  a.rstd = rstd;
  a.rows = rows;
  a.cols = (int)cols;
  a.wf32 = wt == FP8DP_F32;
  a.sums = dweight != nullptr;
  a.rng = rng;
  a.dz = dz;
  a.dx = dx;
  a.parts = workspace;
  return dx != nullptr && a.rule.threshold > 0
             ? launch_bwd_type<true>(dt, a, dweight, dbias, stream)
             : launch_bwd_type<false>(dt, a, dweight, dbias, stream);
}
