// mxq_block_api.cpp - the extern "C" boundary of the operators around the
// quantized linears (declared in include/mxq_block.h): validation on the host,
// before anything is enqueued, then dispatch to the gfx950 kernels.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "mxq_block.h"
#include "mxq_host.h"
#include "mxq_internal.h"

using namespace mxq;

namespace {

bool aligned16_or_null(const void* p) { return p == nullptr || aligned16(p); }

// A call's modulation vectors of length n: element type, stride and grouping.
int check_modulation(int mod_type, int64_t ld_mod, int64_t rows_per_group, int64_t n) {
  if (mod_type != MXQ_MOD_F32 && mod_type != MXQ_MOD_BF16) return MXQ_ERR_MODE;
  if (ld_mod < n || ld_mod >= kMaxDim || rows_per_group < 0 || rows_per_group >= kMaxDim) return MXQ_ERR_SHAPE;
  return MXQ_OK;
}

// MXQ_CHECK_FINITE on a modulation vector of length n: the groups that m rows use.
int modulation_guard(const char* what, const void* p, int mod_type, int64_t ld_mod, int64_t rows_per_group, int64_t m,
                     int64_t n, hipStream_t stream) {
  if (p == nullptr) return MXQ_OK;
  const int64_t groups = rows_per_group > 0 ? (m + rows_per_group - 1) / rows_per_group : 1;
  return mod_type == MXQ_MOD_BF16 ? finite_guard(what, p, groups, n, ld_mod, stream)
                                  : finite_guard_f32(what, p, groups, n, ld_mod, stream);
}

// The same on a bf16 vector.
int vector_guard(const char* what, const void* p, int64_t n, hipStream_t stream) {
  return p == nullptr ? MXQ_OK : finite_guard(what, p, 1, n, n, stream);
}

const char* kernel_name(int mode, bool pipelined) {
  if (pipelined) return mode == MXQ_W4A4 ? "pipe_w4a4" : "pipe_w4a8";
  return mode == MXQ_W4A4 ? "tokens_w4a4" : "tokens_w4a8";
}

}  // namespace

extern "C" {

int mxq_norm_quantize(int mode, const mxq_norm_args* args, hipStream_t stream) {
  if (mode != MXQ_W4A4 && mode != MXQ_W4A8 && mode != MXQ_POLICY_BF16 && mode != MXQ_POLICY_TRANSFORM_ON)
    return MXQ_ERR_MODE;
  if (args == nullptr) return MXQ_ERR_NULL;
  const mxq_norm_args& a = *args;
  if (a.norm != MXQ_NORM_RMS && a.norm != MXQ_NORM_LAYER) return MXQ_ERR_MODE;
  if (a.post_norm != MXQ_NORM_NONE && a.post_norm != MXQ_NORM_RMS && a.post_norm != MXQ_NORM_LAYER) return MXQ_ERR_MODE;
  if (!(a.eps > 0.0f) || !isfinite(a.eps) || !isfinite(a.branch_scale)) return MXQ_ERR_MODE;
  int st = check_mk(a.M, a.K, a.ldx);
  if (st != MXQ_OK) return st;
  if (a.K > MXQ_NORM_MAX_K || (mode == MXQ_POLICY_TRANSFORM_ON && a.K % 128 != 0)) return MXQ_ERR_SHAPE;
  if (a.branch != nullptr && (st = check_mk(a.M, a.K, a.ldb)) != MXQ_OK) return st;
  if (a.h != nullptr && (st = check_mk(a.M, a.K, a.ldh)) != MXQ_OK) return st;
  const bool modulated = a.gate != nullptr || a.scale != nullptr || a.shift != nullptr;
  if (modulated && (st = check_modulation(a.mod_type, a.ld_mod, a.rows_per_group, a.K)) != MXQ_OK) return st;
  if (a.M == 0) return MXQ_OK;
  if (a.x == nullptr || a.out == nullptr) return MXQ_ERR_NULL;
  if (mode != MXQ_POLICY_BF16 && a.out_scales == nullptr) return MXQ_ERR_NULL;
  if (mode == MXQ_POLICY_TRANSFORM_ON && a.act_mult == nullptr) return MXQ_ERR_NULL;
  if (a.branch == nullptr &&
      (a.gate != nullptr || a.post_norm != MXQ_NORM_NONE || a.branch_scale != 1.0f || a.h != nullptr))
    return MXQ_ERR_NULL;
  if (a.post_norm == MXQ_NORM_NONE && (a.post_weight != nullptr || a.post_bias != nullptr)) return MXQ_ERR_MODE;
  for (const void* p : {a.x, a.branch, a.gate, a.post_weight, a.post_bias, a.weight, a.bias, a.scale, a.shift,
                        (const void*)a.act_mult, (const void*)a.h, (const void*)a.out, (const void*)a.out_scales})
    if (!aligned16_or_null(p)) return MXQ_ERR_ALIGN;
  if (a.ldx % 8 != 0 || (a.branch != nullptr && a.ldb % 8 != 0) || (a.h != nullptr && a.ldh % 8 != 0) ||
      (modulated && a.ld_mod % 8 != 0))
    return MXQ_ERR_ALIGN;
  // operands that the mode does not read
  if ((a.act_mult != nullptr && mode != MXQ_POLICY_TRANSFORM_ON) || (a.out_scales != nullptr && mode == MXQ_POLICY_BF16))
    return MXQ_ERR_MODE;
  if (log_enabled())
    fprintf(stderr, "[mxq] norm_quantize mode=%d norm=%d post=%d M=%lld K=%lld\n", mode, a.norm, a.post_norm,
            (long long)a.M, (long long)a.K);
  if ((st = finite_guard("norm input", a.x, a.M, a.K, a.ldx, stream)) != MXQ_OK) return st;
  if (a.branch != nullptr && (st = finite_guard("branch", a.branch, a.M, a.K, a.ldb, stream)) != MXQ_OK) return st;
  const struct { const char* what; const void* p; } vectors[] = {
      {"post_weight", a.post_weight}, {"post_bias", a.post_bias}, {"norm weight", a.weight}, {"norm bias", a.bias}};
  for (const auto& v : vectors)
    if ((st = vector_guard(v.what, v.p, a.K, stream)) != MXQ_OK) return st;
  const struct { const char* what; const void* p; } modulation[] = {{"gate", a.gate}, {"scale", a.scale}, {"shift", a.shift}};
  for (const auto& v : modulation)
    if ((st = modulation_guard(v.what, v.p, a.mod_type, a.ld_mod, a.rows_per_group, a.M, a.K, stream)) != MXQ_OK) return st;
  if (mode == MXQ_POLICY_TRANSFORM_ON &&
      (st = finite_guard_f32("transform factors", a.act_mult, 1, a.K, a.K, stream)) != MXQ_OK)
    return st;
  st = hip_status(launch_norm_quant(mode, a, stream));
  if (st != MXQ_OK) return st;
  if (a.h != nullptr && (st = finite_guard("residual stream", a.h, a.M, a.K, a.ldh, stream)) != MXQ_OK) return st;
  // An h or an output that overflowed bf16 (h need not be stored: its row's norm
  // is not finite either) leaves its mark in the scales of the quantized formats.
  if (mode == MXQ_POLICY_BF16) return finite_guard("norm output", a.out, a.M, a.K, a.K, stream);
  if (mode == MXQ_W4A8) return finite_guard_f32("norm output", a.out_scales, 1, a.M, a.M, stream);
  return finite_guard_mx("norm output", a.out_scales, a.M, a.K, stream);
}

int mxq_gemm_residual(int mode, const void* a_codes, const void* a_scales, const void* w_codes, const void* w_scales,
                      const void* bias, int epilogue, const void* residual, const void* gate, int mod_type,
                      int64_t ld_mod, int64_t rows_per_group, void* y, int64_t M, int64_t N, int64_t K,
                      hipStream_t stream) {
  if (mode != MXQ_W4A4 && mode != MXQ_W4A8) return MXQ_ERR_MODE;
  if (epilogue != MXQ_EPI_NONE && epilogue != MXQ_EPI_GELU_TANH) return MXQ_ERR_MODE;
  int st = check_mk(M, K, K);
  if (st != MXQ_OK) return st;
  if (N < 0 || N > kMaxBlockCols) return MXQ_ERR_SHAPE;
  if (gate != nullptr && (st = check_modulation(mod_type, ld_mod, rows_per_group, N)) != MXQ_OK) return st;
  if (M == 0 || N == 0) return MXQ_OK;
  if (a_codes == nullptr || a_scales == nullptr || w_codes == nullptr || w_scales == nullptr || residual == nullptr ||
      y == nullptr)
    return MXQ_ERR_NULL;
  if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(w_codes) || !aligned16(w_scales) ||
      !aligned16_or_null(bias) || !aligned16(residual) || !aligned16_or_null(gate) || !aligned16(y))
    return MXQ_ERR_ALIGN;
  const ResidualEpi e{residual, gate, ld_mod, rows_per_group, mod_type == MXQ_MOD_BF16};
  if (log_enabled())
    fprintf(stderr, "[mxq] gemm_residual %s M=%lld N=%lld K=%lld epi=%d kernel=%s\n", mode == MXQ_W4A4 ? "w4a4" : "w4a8",
            (long long)M, (long long)N, (long long)K, epilogue, kernel_name(mode, gemm_residual_pipelined(mode, M, N, K, e)));
  if ((st = finite_guard("residual", residual, M, N, N, stream)) != MXQ_OK) return st;
  if ((st = vector_guard("bias", bias, N, stream)) != MXQ_OK) return st;
  if ((st = modulation_guard("gate", gate, mod_type, ld_mod, rows_per_group, M, N, stream)) != MXQ_OK) return st;
  return output_guard(launch_gemm_residual(mode, a_codes, a_scales, w_codes, w_scales, bias, epilogue, e, y, M, N, K,
                                             stream),
                      "output", y, M, N, stream);
}

int mxq_quantize_weight_gated_mxfp4(const void* w_gate, const void* w_up, int64_t H, int64_t K, int64_t ldw,
                                    void* codes, void* scales, hipStream_t stream) {
  int st = check_mk(H, K, ldw);
  if (st != MXQ_OK) return st;
  if (H % 32 != 0) return MXQ_ERR_SHAPE;
  if (H == 0) return MXQ_OK;
  if (w_gate == nullptr || w_up == nullptr || codes == nullptr || scales == nullptr) return MXQ_ERR_NULL;
  if (!aligned16(w_gate) || !aligned16(w_up) || !aligned16(codes) || !aligned16(scales) || ldw % 8 != 0)
    return MXQ_ERR_ALIGN;
  if (log_enabled()) fprintf(stderr, "[mxq] quantize_weight_gated_mxfp4 H=%lld K=%lld\n", (long long)H, (long long)K);
  if ((st = finite_guard("gate weight", w_gate, H, K, ldw, stream)) != MXQ_OK) return st;
  if ((st = finite_guard("up weight", w_up, H, K, ldw, stream)) != MXQ_OK) return st;
  return hip_status(launch_mxfp4_quant_gated(w_gate, w_up, H, K, ldw, codes, scales, stream));
}

int mxq_gemm_gated(int mode, const void* a_codes, const void* a_scales, const void* w_codes, const void* w_scales,
                   const void* bias_gate, const void* bias_up, int act, void* y, void* y_scales, int64_t M, int64_t H,
                   int64_t K, hipStream_t stream) {
  if (mode != MXQ_W4A4 && mode != MXQ_W4A8) return MXQ_ERR_MODE;
  if (act != MXQ_GATED_SILU && act != MXQ_GATED_GELU_TANH) return MXQ_ERR_MODE;
  if (y_scales != nullptr && mode != MXQ_W4A4) return MXQ_ERR_MODE;
  int st = check_mk(M, K, K);
  if (st != MXQ_OK) return st;
  if (H < 0 || H > kMaxBlockCols || H % 32 != 0) return MXQ_ERR_SHAPE;
  if (M == 0 || H == 0) return MXQ_OK;
  if (a_codes == nullptr || a_scales == nullptr || w_codes == nullptr || w_scales == nullptr || y == nullptr)
    return MXQ_ERR_NULL;
  if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(w_codes) || !aligned16(w_scales) ||
      !aligned16_or_null(bias_gate) || !aligned16_or_null(bias_up) || !aligned16(y) || !aligned16_or_null(y_scales))
    return MXQ_ERR_ALIGN;
  if (log_enabled())
    fprintf(stderr, "[mxq] gemm_gated %s%s M=%lld H=%lld K=%lld act=%d kernel=%s\n", mode == MXQ_W4A4 ? "w4a4" : "w4a8",
            y_scales != nullptr ? " -> mxfp4" : "", (long long)M, (long long)H, (long long)K, act,
            mxq_block_kernel_name(mode, 1, y_scales != nullptr, M, H, K));
  if ((st = vector_guard("gate bias", bias_gate, H, stream)) != MXQ_OK) return st;
  if ((st = vector_guard("up bias", bias_up, H, stream)) != MXQ_OK) return st;
  const hipError_t e = launch_gemm_gated(mode, a_codes, a_scales, w_codes, w_scales, bias_gate, bias_up, act, y,
                                           y_scales, M, H, K, stream);
  if (y_scales == nullptr) return output_guard(e, "output", y, M, H, stream);
  if (e != hipSuccess) return MXQ_ERR_HIP;
  return finite_guard_mx("output", y_scales, M, H, stream);
}

const char* mxq_block_kernel_name(int mode, int gated, int mxfp4_out, int64_t M, int64_t N, int64_t K) {
  if (mode != MXQ_W4A4 && mode != MXQ_W4A8) return "invalid";
  return kernel_name(mode, gated ? gemm_gated_pipelined(mode, M, N, K, mxfp4_out != 0)
                                 : gemm_residual_pipelined(mode, M, N, K, ResidualEpi{}));
}

}  // extern "C"
