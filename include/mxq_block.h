/*
 * mxq_block.h - C ABI of libmxq, the operators around the quantized linears
 * of a transformer block: what a block computes between one quantized
 * product and the next, fused with the quantizer before the product or with
 * the product's epilogue.
 *
 *   mxq_norm_quantize   residual add with gate, norm (before the next linear,
 *                       and after the branch), weight and modulation, then
 *                       the activation format of the next linear
 *   mxq_gemm_residual   scaled GEMM with bias, GELU, gate and residual
 *   mxq_gemm_gated      both first projections of a gated feed-forward block,
 *                       the activation and the product, in one kernel
 *   mxq_quantize_weight_gated_mxfp4   packs the two projections for it
 *
 * Formats, status codes, quantization rules and the conventions of every
 * entry point (pointers, streams, validation before anything is enqueued,
 * empty problems, alignment, MXQ_CHECK_FINITE) are those of mxq.h. No call
 * here needs a workspace or synchronizes, every call can be captured into a
 * graph, calls may overlap on one device, and results do not depend on the
 * schedule (no floating-point atomics).
 *
 * With MXQ_CHECK_FINITE set the calls also scan their vectors (weights and
 * biases, modulation vectors of the groups that the rows use, act_mult) before
 * anything is written, and report values that overflowed bf16 in an output or
 * before its quantization (by the scales, which are then past any finite
 * block's or row's). Token scales and codes of an operand are not scanned.
 *
 * Modulation vectors (gate, scale, shift) belong to groups of rows: a vector
 * is [groups][ld_mod], row m uses row m / rows_per_group of it (a batch item's
 * tokens, or 1 for a vector per token); rows_per_group = 0 means one group
 * for all rows. All vectors of a call share mod_type, ld_mod and the grouping;
 * ld_mod >= the vector's length lets them be slices of one [groups][6 K] table.
 */
#ifndef MXQ_BLOCK_H
#define MXQ_BLOCK_H

#include "mxq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Norms: v / sqrt(mean v^2 + eps), and (v - mean) / sqrt(mean (v - mean)^2 + eps). */
enum { MXQ_NORM_NONE = 0, MXQ_NORM_RMS = 1, MXQ_NORM_LAYER = 2 };

/* Element types of modulation vectors. */
enum { MXQ_MOD_F32 = 0, MXQ_MOD_BF16 = 1 };

/* Activations of a gated feed-forward block: v / (1 + exp(-v)), and tanh-GELU. */
enum { MXQ_GATED_SILU = 0, MXQ_GATED_GELU_TANH = 1 };

/* Longest row of mxq_norm_quantize (a row stays in one workgroup's registers). */
#define MXQ_NORM_MAX_K 32768

/*
 * mxq_norm_quantize: per row m, in fp32,
 *   b   = branch, or post_norm(branch) * post_weight + post_bias
 *   h   = RN_bf16( x + branch_scale * gate * b )    (h = x without a branch)
 *   n   = norm(h) * weight + bias
 *   n   = n * (1 + scale) + shift
 * and out = RN_bf16(n) in the activation format of the next linear's `mode`:
 *   MXQ_W4A4                 MXFP4 codes and scales, as mxq_quantize_act
 *   MXQ_W4A8                 FP8 codes and per-token scales, as mxq_quantize_act
 *   MXQ_POLICY_TRANSFORM_ON  MXFP4 codes and scales, as mxq_quantize_mxfp4_hadamard
 *   MXQ_POLICY_BF16          the bf16 values (a linear outside this library)
 * The norm is taken of the rounded h, the value that the next residual add
 * reads. The codes are exactly those of the bf16 output's quantizer.
 *   x, branch   device bf16 [M][ldx], [M][ldb]; branch null for none
 *   post_norm   MXQ_NORM_NONE, _RMS or _LAYER of the branch, with post_weight
 *               and post_bias (device bf16 [K] or null; null without a norm)
 *   gate        modulation vector or null (all ones); branch_scale: host factor
 *   norm        MXQ_NORM_RMS or _LAYER; weight, bias: device bf16 [K] or null
 *   scale,shift modulation vectors or null (zeros)
 *   eps         positive and finite, for both norms
 *   act_mult    device float32 [K]: MXQ_POLICY_TRANSFORM_ON only (K % 128 == 0),
 *               null in the other modes
 *   h           device bf16 [M][ldh] (output) or null; may be x or branch
 *               itself (same pointer and stride), else may not overlap an input
 *   out         device: bf16 [M][K], or codes; out_scales: scales (null for
 *               bf16). A bf16 out may be x or branch itself where those are
 *               dense; else outputs may not overlap an input or each other
 *   M, K        K a multiple of 32, at most MXQ_NORM_MAX_K (MXQ_ERR_SHAPE)
 * gate, post_norm, branch_scale != 1 or h without a branch: MXQ_ERR_NULL.
 * act_mult or out_scales in a mode that does not take them: MXQ_ERR_MODE.
 * Values whose squares sum past fp32's range (|v| about 1e18) are not finite
 * inputs of a norm: the row's output is NaN (and its h, for the branch's norm),
 * which MXQ_CHECK_FINITE reports.
 */
typedef struct mxq_norm_args {
  const void* x;
  const void* branch;
  const void* gate;
  const void* post_weight;
  const void* post_bias;
  const void* weight;
  const void* bias;
  const void* scale;
  const void* shift;
  const float* act_mult;
  void* h;
  void* out;
  void* out_scales;
  int64_t M, K;
  int64_t ldx, ldb, ldh;
  int64_t ld_mod, rows_per_group;
  int32_t post_norm, norm, mod_type;
  float eps, branch_scale;
} mxq_norm_args;
int mxq_norm_quantize(int mode, const mxq_norm_args* args, hipStream_t stream);

/*
 * mxq_gemm_residual: y [M][N] =
 *   RN_bf16( residual + gate * epilogue( sum_k deqA[m][k] deqW[n][k] + bias[n] ) )
 * in fp32 up to the one rounding (mxq_gemm into memory and a residual add
 * after it round the product to bf16 first).
 *   a_codes .. epilogue  as for mxq_gemm, MXQ_W4A4 or MXQ_W4A8
 *   residual  device bf16 [M][N] (dense)
 *   gate      modulation vector [groups][ld_mod >= N] of mod_type, or null
 *             (ones; ld_mod, rows_per_group and mod_type are then not read)
 *   y         device bf16 [M][N] (output); may be residual itself, else may not
 *             overlap an input
 * Any M, N at most 2^28 - 32, K a multiple of 32. Rows in the tens run a kernel
 * that splits K over a workgroup's waves; its sums are taken in another order
 * than mxq_gemm's. So do, at any M and then far slower than the pipelined
 * kernel, N below 256 or no multiple of 8, K below 512 (W4A8: 384), codes of 2
 * GiB or more, and a gate of several groups (rows_per_group > 0) whose ld_mod is
 * no multiple of 8.
 */
int mxq_gemm_residual(int mode, const void* a_codes, const void* a_scales, const void* w_codes, const void* w_scales,
                      const void* bias, int epilogue, const void* residual, const void* gate, int mod_type,
                      int64_t ld_mod, int64_t rows_per_group, void* y, int64_t M, int64_t N, int64_t K,
                      hipStream_t stream);

/*
 * Offline round-to-nearest MXFP4 packing of a gated feed-forward block's two
 * first projections (each [H][K] bf16, nn.Linear layout) for mxq_gemm_gated:
 * the codes and scales are those of mxq_quantize_weight_mxfp4 on the [2H][K]
 * matrix whose rows 64 b .. 64 b + 31 are rows 32 b .. 32 b + 31 of w_gate and
 * whose next 32 rows are those of w_up. H a multiple of 32.
 *   w_gate, w_up  device bf16 [H][ldw]
 *   codes         device uint8, 2H * K/2 bytes in code panels (output)
 *   scales        device uint8 [ceil(K/128)][2H][4] (output)
 */
int mxq_quantize_weight_gated_mxfp4(const void* w_gate, const void* w_up, int64_t H, int64_t K, int64_t ldw,
                                    void* codes, void* scales, hipStream_t stream);

/*
 * mxq_gemm_gated: hidden [M][H] = RN_bf16( act( g ) * u ), in fp32 from
 *   g = sum_k deqA[m][k] deqWg[h][k] + bias_gate[h]
 *   u = sum_k deqA[m][k] deqWu[h][k] + bias_up[h].
 *   a_codes/a_scales  device, from mxq_quantize_act(mode, ...) or mxq_norm_quantize
 *   w_codes/w_scales  device, from mxq_quantize_weight_gated_mxfp4
 *   bias_gate, bias_up  device bf16 [H], each or both null for none
 *   act               MXQ_GATED_SILU or MXQ_GATED_GELU_TANH
 *   y_scales null:    y is device bf16 [M][H] (output)
 *   y_scales given:   MXQ_W4A4 only: y and y_scales are the MXFP4 activation
 *                     of the second projection (M * H/2 code bytes in panels,
 *                     scales [ceil(H/128)][M][4]): the codes of
 *                     mxq_quantize_act(MXQ_W4A4, the bf16 hidden state)
 * H and K multiples of 32, H at most 2^28 - 32, any M.
 */
int mxq_gemm_gated(int mode, const void* a_codes, const void* a_scales, const void* w_codes, const void* w_scales,
                   const void* bias_gate, const void* bias_up, int act, void* y, void* y_scales, int64_t M, int64_t H,
                   int64_t K, hipStream_t stream);

/* Name of the kernel that mxq_gemm_residual (gated = 0, N columns) or
 * mxq_gemm_gated (N = H, gated = 1) runs, as a static string: "pipe_..." for
 * the LDS-pipelined kernel, "tokens_..." for the split-K kernel, "invalid" for
 * another mode. The choice goes by measured times; the environment variable
 * MXQ_BLOCK_KERNEL=pipe or tokens, read at every call, fixes it where the
 * pipelined kernel takes the shape. The name goes by the shape: a residual
 * product whose gate has several groups (rows_per_group > 0) with ld_mod no
 * multiple of 8 runs the split-K kernel at any size. Host only. */
const char* mxq_block_kernel_name(int mode, int gated, int mxfp4_out, int64_t M, int64_t N, int64_t K);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_BLOCK_H */
