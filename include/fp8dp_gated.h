/*
 * fp8dp_gated.h -- C ABI of libfp8dp.so, third part: the operators of a gated
 * feed-forward block.  Its two first projections with the activation and the
 * product, the norms before and after a block with the block's gate and residual
 * scale, and low-rank adapters of many requests beside a shared projection.
 *
 * The conventions are fp8dp_block.h's: device pointers, caller-owned memory, calls
 * enqueued on `stream` without waiting, nothing allocated, 0 or a negative
 * FP8DP_E* code with fp8dp_last_error(), and nothing enqueued when a check
 * fails.  Tensors need only the alignment of their elements, sizes may be any
 * positive numbers within the stated limits, matrices are dense and row-major, and outputs
 * must not overlap inputs, except where a call says so.  Calls that share a workspace must
 * not overlap in time; what a workspace holds does not matter before a call, nor after it.
 * Sums and statistics are binary32, and each output is rounded once, to its own type.
 */
#ifndef FP8DP_GATED_H
#define FP8DP_GATED_H

#include "fp8dp_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* f of the gated linear layer: g sigmoid(g); g Phi(g) with the normal distribution's Phi;
   g sigmoid(2 sqrt(2 / pi) (g + 0.044715 g^3)), which is its tanh form; sigmoid(g);
   max(g, 0); max(g, 0)^2; g.  The derivative of max(g, 0) is 0 at 0. */
typedef enum {
  FP8DP_GATE_SILU = 0,
  FP8DP_GATE_GELU = 1,
  FP8DP_GATE_GELU_TANH = 2,
  FP8DP_GATE_SIGMOID = 3,
  FP8DP_GATE_RELU = 4,
  FP8DP_GATE_RELU2 = 5,
  FP8DP_GATE_IDENTITY = 6
} fp8dp_gate;

/* Largest N and K of the gated linear layer, and its most tokens. */
#define FP8DP_GATED_MAX_WIDTH 1048576
#define FP8DP_GATED_MAX_ROWS 16777216

/* Bytes of workspace with which gated_linear splits K over workgroups where there are few
   tiles of h, and copies operands whose rows K cuts to aligned ones; 0 where it would do neither. */
int64_t gated_linear_workspace(int64_t M, int64_t N, int64_t K);

/* The first half of a gated feed-forward layer:
     g = x w_gate^T, u = x w_up^T, h = f(g) u, with f and the product on the binary32 sums.
   x: [M x K], w_gate, w_up: [N x K], h: [M x N], all of type dt, FP8DP_BF16 or FP8DP_F16.
   gate, up: [M x N] of type dt, g and u rounded, for the backward pass; both or neither.
   workspace: 16-byte aligned scratch, or NULL; with less than gated_linear_workspace()
   bytes K is not split and nothing copied.
   Errors: EINVAL for a NULL x, w_gate, w_up or h, one of gate and up without the other, M
   outside 1 .. FP8DP_GATED_MAX_ROWS, N or K outside 1 .. FP8DP_GATED_MAX_WIDTH, another type, an unknown
   act, a misaligned pointer, an output that is an input or another output, or workspace_bytes < 0. */
int gated_linear(const void* x, const void* w_gate, const void* w_up, int64_t M, int64_t N,
                 int64_t K, fp8dp_dtype dt, fp8dp_gate act, void* h, void* gate, void* up,
                 void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace that gated_linear_backward needs. */
int64_t gated_linear_backward_workspace(int64_t M, int64_t N, int64_t K);

/* Backward of gated_linear from dh and the forward's x, gate and up:
     dg = dh u f'(g), du = dh f(g),
     dx = dg w_gate + du w_up, dw_gate = dg^T x, dw_up = du^T x.
   dg and du are rounded to dt, the matrix instructions' operand type; in float16 they may be past that type's range:
   where the largest finite magnitude of them all is outside [2^-6, 2^15), all are held times one power of two
   that brings it to [2^14, 2^15) and that the outputs take back.  What float16 then holds as a subnormal is off by up to
   2^-25, or 2^-39 of that largest magnitude where it was outside.  The sums are
   binary32 and have a fixed order: the same call gives the same bits.  All tensors are of
   type dt, dx [M x K], dw_gate and dw_up [N x K].  dx, or dw_gate and dw_up together, may be
   NULL and are then not computed.
   workspace: 16-byte aligned, at least gated_linear_backward_workspace() bytes.
   Errors: as gated_linear's, and EINVAL for a workspace that is NULL or too small. */
int gated_linear_backward(const void* dh, const void* gate, const void* up, const void* x,
                          const void* w_gate, const void* w_up, int64_t M, int64_t N, int64_t K,
                          fp8dp_dtype dt, fp8dp_gate act, void* dx, void* dw_gate, void* dw_up,
                          void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* From one block to the next in one pass over [rows x cols] tensors of type dt: the norm behind
   the block, its gate, the residual sum, and the norm in front of the next block.
     post_rstd = 1 / sqrt(mean(x^2) + eps),
     z = residual_scale * residual + branch_scale * gate * x * post_rstd * post_weight,
     pre_rstd = 1 / sqrt(mean(z^2) + eps),  y = z * pre_rstd * pre_weight;
   the second norm reads z as stored.
   x NULL: the norm alone, of the residual as it is (z, post_weight, gate and post_rstd are
   NULL then).  y NULL: no second norm; pre_weight is not read then, and pre_rstd is NULL.
   post_weight, pre_weight: [cols] of type wt, dt or FP8DP_F32; NULL stands for ones.
   gate: NULL stands for ones; gate_per_token 0: [cols] of type gt, dt or FP8DP_F32; else
   [rows x cols] of type dt, and gt is dt.
   post_rstd, pre_rstd: [rows] floats that backward reads, or NULL.
   z may be x, residual or a gate per token.  A row that holds a NaN or an infinity gives NaN or 0
   where the formula does; other rows are not touched by it.  The squares are binary32 too: a row whose squares
   add up to more than 3.4e38 has an inverse of 0, and one of values below 1e-19 counts as zeros (which shows with an eps of 0
   alone).
   Errors: EINVAL for a NULL residual, z without x or x without z, neither z nor y, what belongs to
   an x that is NULL, pre_rstd without y, rows or cols out of layer_norm's range, unknown types, a misaligned pointer, an eps that is
   negative or not finite, a scale that is not finite, y or the statistics the same
   buffer as z, an input or each other, or z the same as a weight, a gate per channel or a statistic. */
int block_norm(const void* x, const void* residual, const void* post_weight, const void* gate,
               int32_t gate_per_token, const void* pre_weight, int64_t rows, int64_t cols,
               fp8dp_dtype dt, fp8dp_dtype wt, fp8dp_dtype gt, float residual_scale,
               float branch_scale, float eps, void* z, void* y, float* post_rstd, float* pre_rstd,
               hipStream_t stream);

/* Backward of block_norm from dy, the gradient dz_add that reaches z past the second norm, and the
   forward's x, z, post_rstd and pre_rstd.  With xh = x post_rstd, zh = z pre_rstd, c = dy pre_weight:
     dz = dz_add + pre_rstd * (c - zh * mean(c * zh)),  dresidual = residual_scale * dz,
     dpre_weight = sum over rows of dy * zh,  e = branch_scale * gate * dz,
     dpost_weight = sum over rows of e * xh,
     dx = post_rstd * (e * post_weight - xh * mean(e * post_weight * xh)),
     dgate = branch_scale * dz * xh * post_weight, summed over rows for a gate per channel.
   dy NULL: block_norm was called without y.  dz_add NULL: zeros.  x NULL: block_norm was called
   without x; dresidual is dz then.
   dresidual, dx: [rows x cols] of type dt; dgate: [rows x cols] of type dt for a gate per token,
   [cols] floats for one per channel; dpost_weight, dpre_weight: [cols] floats.  All but dresidual may be NULL.
   workspace: 2 * min(rows, FP8DP_NORM_PARTS) * cols floats where a sum over rows is asked for.  The
   sums have a fixed order: the same call gives the same bits.
   dresidual may be dy or dz_add; dx and a dgate per token too where no other output is.
   Errors: EINVAL for a NULL dresidual, neither dy nor dz_add, neither dy nor x, an argument without what it belongs
   to, outputs that are the same buffer or an input (but for those above) or the workspace, a missing workspace, and as
   above. */
int block_norm_backward(const void* dy, const void* dz_add, const void* x, const void* z,
                        const void* post_weight, const void* gate, int32_t gate_per_token,
                        const void* pre_weight, const float* post_rstd, const float* pre_rstd,
                        int64_t rows, int64_t cols, fp8dp_dtype dt, fp8dp_dtype wt, fp8dp_dtype gt,
                        float residual_scale, float branch_scale, void* dresidual, void* dx,
                        void* dgate, float* dpost_weight, float* dpre_weight, float* workspace,
                        hipStream_t stream);

/* Most tokens and adapters of a plan, and the largest rank. */
#define FP8DP_LORA_MAX_TOKENS 4194304
#define FP8DP_LORA_MAX_ADAPTERS 2048
#define FP8DP_LORA_MAX_RANK 256

/* 32-bit words of a plan; -1 for sizes out of range. */
int64_t lora_plan_size(int64_t tokens, int64_t adapters);

/* Groups a step's tokens by their adapters, for any number of lora_add calls.
   index: [tokens] 32-bit integers on the device; a negative one, or one at or past `adapters`,
   stands for no adapter.  plan: lora_plan_size() 32-bit integers.
   Errors: EINVAL for NULL or misaligned pointers, tokens outside 1 .. FP8DP_LORA_MAX_TOKENS, or
   adapters outside 1 .. FP8DP_LORA_MAX_ADAPTERS. */
int lora_plan(const int32_t* index, int64_t tokens, int64_t adapters, int32_t* plan,
              hipStream_t stream);

/* Bytes of workspace that lora_add needs; -1 for sizes out of range. */
int64_t lora_add_workspace(int64_t tokens, int64_t N, int64_t K, int64_t rank, int64_t adapters);

/* Adds the low-rank products of the tokens' adapters to the output of a shared projection:
     y[t] = base[t] + scale[i] * b_i (a_i x[t]) with i = index[t]; y[t] = base[t] without an adapter.
   x: [tokens x K], a: [adapters x rank x K], b: [adapters x N x rank], base, y: [tokens x N], all of
   type dt, FP8DP_BF16 or FP8DP_F16; scale: [adapters] floats; the products a_i x[t] are summed in
   binary32 and multiplied by b_i as two 16-bit parts each, 16 bits of them in bfloat16 and 22 in float16.
   ranks: [adapters] 32-bit integers, of adapter i the first ranks[i] rows of a and columns of b count
   (what the others hold does not matter; below 0 is 0, above rank is rank), or NULL: all.
   plan: lora_plan's for the same tokens and adapters.  With one made for other numbers of them, or none, which only the
   device can see, the call returns 0 and y stays as it is.  base NULL: zeros.  y may be base.
   A token or a row of b that holds an infinity or a NaN gives infinities or NaN (NaN also where the formula has an
   infinity: its parts are added), and no other token or channel is touched.
   workspace: 16-byte aligned, at least lora_add_workspace() bytes.
   Errors: EINVAL for a NULL x, a, b, scale, plan, y or workspace, tokens, adapters or rank out of range,
   N or K outside 1 .. FP8DP_GATED_MAX_WIDTH, another type, a misaligned pointer, or a workspace that is
   too small. */
int lora_add(const void* x, const void* a, const void* b, const float* scale, const int32_t* ranks,
             const int32_t* plan, const void* base, int64_t tokens, int64_t N, int64_t K,
             int64_t rank, int64_t adapters, fp8dp_dtype dt, void* y, void* workspace,
             int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8DP_GATED_H */
