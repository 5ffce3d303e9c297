/*
 * fp8dp_block.h -- C ABI of libfp8dp.so, second part: the operators around the
 * MLP in a transformer block.  Layer norm and its backward pass, dropout with
 * the residual sum, and the INT8 linear layer with one scale per token and one
 * per output channel.
 *
 * The conventions are fp8dp.h's: device pointers, caller-owned memory, calls
 * enqueued on `stream` without waiting, nothing allocated, 0 or a negative
 * FP8DP_E* code with fp8dp_last_error(), and nothing enqueued when a check
 * fails.  Two differences: tensors here need only the alignment of their
 * elements (rows of odd length have no more), and cols, N and K may be any
 * positive size.  Matrices are dense and row-major.  Outputs must not overlap
 * inputs, except where a call says so.
 *
 * Sums, statistics and the norm's arithmetic are binary32 (integers for the
 * INT8 product); long sums are joined so that their error hardly grows with
 * their length.  Each output is rounded once, to its own type.
 */
#ifndef FP8DP_BLOCK_H
#define FP8DP_BLOCK_H

#include "fp8dp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of activations, their gradients and outputs. */
typedef enum { FP8DP_BF16 = 0, FP8DP_F16 = 1, FP8DP_F32 = 2 } fp8dp_dtype;

/* Most partial sums per column of a weight gradient: the workspace of
   layer_norm_backward is 2 * min(rows, FP8DP_NORM_PARTS) * cols floats. */
#define FP8DP_NORM_PARTS 1024

/* Largest K of int8_gemm and int8_linear: K products of magnitude up to 2^14
   (-128 * -128) stay below 2^31. */
#define FP8DP_INT8_MAX_K 131071

/* Layer norm over the last dimension:
     mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps),
     y = (x - mu) * rstd * weight + bias.
   x, y: [rows x cols] of type dt.  weight, bias: [cols] of type wt, which is dt
   or FP8DP_F32; NULL stands for ones / zeros.  mean, rstd: [rows] floats that
   backward reads, or NULL.  A row that holds a NaN or an infinity gives NaN;
   other rows are not touched by it.
   Errors: EINVAL for a NULL x or y, rows outside 1 .. 2^31 - 1, cols
   outside 1 .. 2^30, an unknown type, wt neither dt nor FP8DP_F32, a misaligned pointer, or an eps
   that is negative or not finite. */
int layer_norm(const void* x, const void* weight, const void* bias, int64_t rows, int64_t cols,
               fp8dp_dtype dt, fp8dp_dtype wt, float eps, void* y, float* mean, float* rstd,
               hipStream_t stream);

/* out = residual + keep * x / (1 - p) on [rows x cols] of type dt; residual NULL: no sum.
   The random numbers come from Philox4x32 with 10 rounds (Salmon, Moraes, Dror
   and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011).  The
   block with key (rng[0] low, high word) and counter (c / 8, row, rng[1] low,
   high word) gives 8 numbers of 16 bits, low half of a word first; element
   (row, c) takes number c % 8 and is kept when it is at least
   T = rint(65536 p); x / (1 - p) is x * (65536 / (65536 - T)), so the expected
   value is x exactly, and T = 65536 drops all.  No mask is stored: the same call on
   the gradient of out, with the same p and rng and no residual, is the
   backward pass.
   rng: two 64-bit words on the device, seed and offset, read by the kernel (a
   captured graph may change them between replays); NULL only with p = 0.  The words
   alone decide the mask: two uses with the same words drop the same elements,
   so each layer, step and rank has its own (the offset step * layers + layer, say, and a
   seed per rank), and a backward pass those of its forward.
   out may be x or residual.  A dropped element contributes +0, also where x is
   not finite.
   Errors: EINVAL for a NULL x or out, rows or cols out of range, an unknown
   type, p outside [0, 1], rng NULL with p > 0, or a misaligned pointer. */
int dropout_add(const void* x, const void* residual, int64_t rows, int64_t cols, fp8dp_dtype dt,
                float p, const uint64_t* rng, void* out, hipStream_t stream);

/* z = dropout_add(x, residual), rounded to dt and stored, and y = layer_norm(z),
   in one pass.  The norm reads z as stored, so layer_norm_backward on z agrees.
   Errors: those of the two calls; z must not be NULL.  z may be x or residual. */
int dropout_add_layer_norm(const void* x, const void* residual, const void* weight,
                           const void* bias, int64_t rows, int64_t cols, fp8dp_dtype dt,
                           fp8dp_dtype wt, float p, const uint64_t* rng, float eps, void* z,
                           void* y, float* mean, float* rstd, hipStream_t stream);

/* Backward of layer_norm at its input z, from dy and the forward's mean and rstd:
     g = dy * weight, h = (z - mean) * rstd,
     dz = rstd * (g - mean(g) - h * mean(g * h)) + dz_add,
     dweight = sum over rows of dy * h, dbias = sum over rows of dy.
   dz_add: the gradient that reaches z past the norm (the residual stream), or
   NULL.  dz: [rows x cols] of type dt: with dropout_add_layer_norm also the residual's gradient.
   dx: that of its x, keep * dz / (1 - p) from the unrounded dz with the
   forward's p and rng, or NULL (p and rng are then not used).
   dweight, dbias: [cols] floats, both or neither; with them workspace is 2 * min(rows,
   FP8DP_NORM_PARTS) * cols floats.  The sums have a fixed order: the same call
   gives the same bits.  dz may be dy or dz_add; dx may be dy or dz_add where
   dz is not.
   Errors: EINVAL for a NULL dy, z, mean, rstd or dz, one of dweight and dbias
   without the other or without a workspace, and as above. */
int layer_norm_backward(const void* dy, const void* z, const void* weight, const float* mean,
                        const float* rstd, const void* dz_add, int64_t rows, int64_t cols,
                        fp8dp_dtype dt, fp8dp_dtype wt, float p, const uint64_t* rng, void* dz,
                        void* dx, float* dweight, float* dbias, float* workspace,
                        hipStream_t stream);

/* INT8 codes with one scale per row: scale = amax(|x|) / 127 and
   q = x * 127 / amax(|x|) rounded to the nearest whole number, ties to even, decided
   exactly; x is about q * scale.  x: [rows x cols] of type dt, q: [rows x cols]
   int8 in -127 .. 127, scale: [rows] floats.  For activations a row is a
   token, for a weight [N x K] an output channel.  A row of zeros has scale 0 and
   codes 0; a row that holds a NaN or an infinity has scale NaN and codes 0, so
   that a product with it is NaN. */
int quantize_int8(const void* x, int64_t rows, int64_t cols, fp8dp_dtype dt, int8_t* q,
                  float* scale, hipStream_t stream);

/* quantize_int8 of layer_norm(x), whose binary32 values are cast without a
   rounding to dt in between.  With residual (type dt) the norm reads z = x +
   residual, rounded to dt and stored to z; residual and z go together. */
int layer_norm_quantize_int8(const void* x, const void* residual, const void* weight,
                             const void* bias, int64_t rows, int64_t cols, fp8dp_dtype dt,
                             fp8dp_dtype wt, float eps, void* z, int8_t* q, float* scale,
                             hipStream_t stream);

/* y[m, n] = (sum over k of a[m, k] * b[n, k]) * a_scale[m] * b_scale[n] + bias[n],
   the sum exact in 32-bit integers.  a: [M x K], b: [N x K] int8 (all of
   -128 .. 127), bias: [N] of type bt, which is yt or FP8DP_F32, or NULL; y: [M x N] of type yt.
   workspace: scratch that lets the library split K over workgroups when there
   are few tiles of y (16 MiB is all that takes), and copy operands whose rows do not start
   at multiples of 16 bytes into rows that do (K rounded up to 16 bytes a row of each); NULL
   or any size is fine.  Calls that share a workspace must not overlap in time.
   Errors: EINVAL for a NULL operand, scale or y, M or N outside 1 .. 2^30, M * N
   above 2^40, K outside 1 .. FP8DP_INT8_MAX_K, unknown types, a misaligned pointer
   (workspace: 16 bytes), or workspace_bytes < 0. */
int int8_gemm(const int8_t* a, const int8_t* b, int64_t M, int64_t N, int64_t K,
              const float* a_scale, const float* b_scale, const void* bias, fp8dp_dtype yt,
              fp8dp_dtype bt, void* y, void* workspace, int64_t workspace_bytes,
              hipStream_t stream);

/* Least workspace of int8_linear, in bytes: the tokens' codes, their rows padded to a
   multiple of 16 bytes, and their scales.  What is beyond it serves int8_gemm as its workspace. */
int64_t int8_linear_workspace(int64_t M, int64_t K);

/* quantize_int8 of x [M x K] (type dt) and int8_gemm with w8 [N x K] and w_scale
   [N]; y and bias as there, y of type dt.  workspace: 16-byte aligned, at least
   int8_linear_workspace(M, K) bytes.  Errors: as int8_gemm's. */
int int8_linear(const void* x, const int8_t* w8, const float* w_scale, const void* bias, int64_t M,
                int64_t N, int64_t K, fp8dp_dtype dt, fp8dp_dtype bt, void* y, void* workspace,
                int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8DP_BLOCK_H */
