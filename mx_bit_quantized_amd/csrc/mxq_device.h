// mxq_device.h - device-only helpers shared by the gfx950 kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq_convert.h"

namespace mxq {

// tanh-GELU in fp32, 0.5 y (1 + tanh(u)) with u = sqrt(2/pi) (y + 0.044715 y^3),
// written as y / (1 + exp(-2u)) and exp(-2u) = 2^(y (c0 + c1 y^2)) with the
// constants folded: 5 VALU operations and 2 transcendental ones per element.
__device__ __forceinline__ float gelu_tanh_dev(float y) {
  constexpr float kL = -2.0f * 1.4426950408889634f * 0.7978845608028654f;  // -2 log2(e) sqrt(2/pi)
  const float e = __builtin_amdgcn_exp2f(y * __builtin_fmaf(y * y, kL * 0.044715f, kL));
  return y * __builtin_amdgcn_rcpf(1.0f + e);
}

// v / (1 + exp(-v)): exp2 overflows to infinity for v below about -88, whose
// reciprocal is the limit 0.
__device__ __forceinline__ float silu_dev(float v) {
  return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f));
}

// MXFP4 block helpers (the quantizers' rule, OCP MX: scale byte from the
// block's largest magnitude, elements rounded by the scaled conversion).
//
// Largest magnitude bit pattern (sign cleared) of 8 bf16: exact for finite
// bf16, no float compare and no denormal flush.
__device__ __forceinline__ uint32_t chunk_amax(const uint4 c) {
  uint32_t m0 = umax(c.x & 0x7FFFu, (c.x >> 16) & 0x7FFFu);
  uint32_t m1 = umax(c.y & 0x7FFFu, (c.y >> 16) & 0x7FFFu);
  uint32_t m2 = umax(c.z & 0x7FFFu, (c.z >> 16) & 0x7FFFu);
  uint32_t m3 = umax(c.w & 0x7FFFu, (c.w >> 16) & 0x7FFFu);
  return umax(umax(m0, m1), umax(m2, m3));
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// 8 bf16 -> 8 E2M1 codes (element 2t in the low nibble of byte t) of a block
// with scale byte sb, with gfx950's scaled conversion: it divides by the
// power of two whose exponent field is sb and rounds to nearest even,
// saturating at 6, keeping the sign (also of zeros). For every finite bf16
// and every scale byte of a block that can hold it this equals
// e2m1_code_bf16 (an exhaustive GPU test checks it).
__device__ __forceinline__ uint32_t pack8_fp4(const uint4 c, uint32_t sb) {
  const float scale = as_float(sb << 23);
  uint32_t out = 0;
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, __builtin_bit_cast(bf16x2_t, c.x), scale, 0);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, __builtin_bit_cast(bf16x2_t, c.y), scale, 1);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, __builtin_bit_cast(bf16x2_t, c.z), scale, 2);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(out, __builtin_bit_cast(bf16x2_t, c.w), scale, 3);
  return out;
}

// 16-byte load of 8 bf16 input elements; with NT, with the non-temporal hint
// (inputs larger than the last-level cache, read once: see mxfp4_quant_kernel).
template <bool NT>
__device__ __forceinline__ uint4 load_chunk(const uint4* p) {
  if constexpr (NT) {
    typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
    const u32x4 q = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
    return make_uint4(q.x, q.y, q.z, q.w);
  } else {
    return *p;
  }
}

// Max over the 4 lanes of a quad, by DPP quad permutations (lane ^ 1, lane ^ 2).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = umax(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));
  v = umax(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));
  return v;
}

// Max over the 16 lanes of a DPP row, in every lane of it: the quad, then the
// other quad (mirrored in 8) and the other half (mirrored in 16).
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = quad_max(v);
  v = umax(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));
  v = umax(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));
  return v;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = umax(v, (uint32_t)__shfl_xor((int)v, off));
  return v;
}

// FP8 helpers (the per-token quantizers' rule).
//
// Signed IEEE quotient x / s of a bf16 element: formed from |x| (rounding to
// nearest is symmetric; the FMA correction would lose the sign of -0) with
// x's sign attached. A row of zeros has s = 0: its quotients are signed zeros
// (the reciprocal is infinite there, and 0 * inf would be NaN).
__device__ __forceinline__ float fp8_signed_quotient(uint32_t bits16, const Fp8Row& r) {
  const float q = r.s == 0.0f ? 0.0f : fp8_quotient(as_float((bits16 & 0x7FFFu) << 16), r);
  return as_float(as_uint(q) | ((bits16 & 0x8000u) << 16));
}

// 8 bf16 -> 8 E4M3FN codes. The quotients are correctly rounded fp32 with
// |q| <= 448 (1 + 2^-22); gfx950's packed conversion rounds them to nearest
// even, signs and subnormals included: for every fp32 with |q| <= 464 it
// equals e4m3fn_code (an exhaustive GPU test checks it).
__device__ __forceinline__ uint2 pack8_fp8(const uint4 c, const Fp8Row& r) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t out[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float q0 = fp8_signed_quotient(w[2 * i] & 0xFFFFu, r), q1 = fp8_signed_quotient(w[2 * i] >> 16, r);
    const float q2 = fp8_signed_quotient(w[2 * i + 1] & 0xFFFFu, r), q3 = fp8_signed_quotient(w[2 * i + 1] >> 16, r);
    uint32_t o = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q0, q1, 0, false);
    o = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q2, q3, (int)o, true);
    out[i] = o;
  }
  return make_uint2(out[0], out[1]);
}

__device__ __forceinline__ void bf16x8_to_f32(const uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = as_float(w[i] << 16);
    f[2 * i + 1] = as_float(w[i] & 0xFFFF0000u);
  }
}

typedef float f32x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t bf16x2_rne(float a, float b) {
  const f32x2_t f = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2_t));
}

// 128-point transform of one row panel held by 16 lanes, 8 elements each:
// lane chunk c holds elements 8c .. 8c + 7. Every lane of the wave takes part
// in the exchanges (no lane may be inactive here).
//
// Stages h = 1, 2, 4 run inside the lane. Stages h = 8, 16, 32, 64 pair the
// lanes whose chunk index differs in bit 1, 2, 4, 8 (lane ^ 1, ^ 2, ^ 4, ^ 8
// within the 16-lane row). They keep a known sign per lane: afterwards the
// lane holds (-1)^popcount(c) times the transform (callers fold that sign
// into the channel factor, an exact change). In that form each stage is one
// fused multiply-add of the partner's value, read through DPP, into the
// lane's own: with u = s v (the partner's sign equal to the lane's s before
// the stage), the lane whose bit is clear computes u_p + u = s (a + b) and
// keeps its sign, the other computes u - u_p = -s (a - b) and flips it. Each
// is one rounding of a + b or a - b, up to that sign; only the sign of an
// exact zero is lost, and callers turn every exact zero into +0.
// The DPP patterns: lane ^ 1 and ^ 2 are quad permutations, ^ 8 the row
// rotation by 8, ^ 4 the half-row mirror (lane ^ 7) then the quad
// permutation lane ^ 3. All are their own inverses, so no direction
// convention matters. A DPP read of a register needs two wait states after
// a VALU write of it: the block opens with them, and inside it every DPP
// source was written eight instructions earlier.
__device__ __forceinline__ void fwht128_lanes(float (&f)[8], int c) {
#pragma unroll
  for (int h = 1; h < 8; h <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if ((e & h) == 0) {
        const float a = f[e], b = f[e + h];
        f[e] = a + b;
        f[e + h] = a - b;
      }
  const float s1 = (c & 1) ? -1.0f : 1.0f, s2 = (c & 2) ? -1.0f : 1.0f;
  const float s4 = (c & 4) ? -1.0f : 1.0f, s8 = (c & 8) ? -1.0f : 1.0f;
  float t0, t1, t2, t3, t4, t5, t6, t7;
#define MXQ_DPP_FMAC(D, S, SG, PAT) "v_fmac_f32_dpp " D ", " S ", " SG " " PAT " row_mask:0xf bank_mask:0xf bound_ctrl:1\n\t"
#define MXQ_DPP_MOV(D, S, PAT) "v_mov_b32_dpp " D ", " S " " PAT " row_mask:0xf bank_mask:0xf bound_ctrl:1\n\t"
#define MXQ_STAGE8(SG, PAT)                                                                                   \
  MXQ_DPP_FMAC("%0", "%0", SG, PAT) MXQ_DPP_FMAC("%1", "%1", SG, PAT) MXQ_DPP_FMAC("%2", "%2", SG, PAT)      \
  MXQ_DPP_FMAC("%3", "%3", SG, PAT) MXQ_DPP_FMAC("%4", "%4", SG, PAT) MXQ_DPP_FMAC("%5", "%5", SG, PAT)      \
  MXQ_DPP_FMAC("%6", "%6", SG, PAT) MXQ_DPP_FMAC("%7", "%7", SG, PAT)
  asm volatile(
      "s_nop 1\n\t"
      MXQ_STAGE8("%16", "quad_perm:[1,0,3,2]")
      MXQ_STAGE8("%17", "quad_perm:[2,3,0,1]")
      MXQ_DPP_MOV("%8", "%0", "row_half_mirror") MXQ_DPP_MOV("%9", "%1", "row_half_mirror")
      MXQ_DPP_MOV("%10", "%2", "row_half_mirror") MXQ_DPP_MOV("%11", "%3", "row_half_mirror")
      MXQ_DPP_MOV("%12", "%4", "row_half_mirror") MXQ_DPP_MOV("%13", "%5", "row_half_mirror")
      MXQ_DPP_MOV("%14", "%6", "row_half_mirror") MXQ_DPP_MOV("%15", "%7", "row_half_mirror")
      MXQ_DPP_FMAC("%0", "%8", "%18", "quad_perm:[3,2,1,0]") MXQ_DPP_FMAC("%1", "%9", "%18", "quad_perm:[3,2,1,0]")
      MXQ_DPP_FMAC("%2", "%10", "%18", "quad_perm:[3,2,1,0]") MXQ_DPP_FMAC("%3", "%11", "%18", "quad_perm:[3,2,1,0]")
      MXQ_DPP_FMAC("%4", "%12", "%18", "quad_perm:[3,2,1,0]") MXQ_DPP_FMAC("%5", "%13", "%18", "quad_perm:[3,2,1,0]")
      MXQ_DPP_FMAC("%6", "%14", "%18", "quad_perm:[3,2,1,0]") MXQ_DPP_FMAC("%7", "%15", "%18", "quad_perm:[3,2,1,0]")
      MXQ_STAGE8("%19", "row_ror:8")
      : "+v"(f[0]), "+v"(f[1]), "+v"(f[2]), "+v"(f[3]), "+v"(f[4]), "+v"(f[5]), "+v"(f[6]), "+v"(f[7]),
        "=&v"(t0), "=&v"(t1), "=&v"(t2), "=&v"(t3), "=&v"(t4), "=&v"(t5), "=&v"(t6), "=&v"(t7)
      : "v"(s1), "v"(s2), "v"(s4), "v"(s8));
#undef MXQ_STAGE8
#undef MXQ_DPP_MOV
#undef MXQ_DPP_FMAC
}

// Softmax statistics of the attention kernels. A weight is 2^(s c + shift) in one fma, with
// shift = -round(m c) for a running maximum m: the rounding is common to a row's weights and
// leaves their ratios, but moves them all by up to half a step of m c. Below 2^30 that is a
// factor 2^32, inside fp32's range; past it all weights may become zeros or infinities. There
// they are zeros (a later score inside the range takes over), and a row that ends there is
// NaN, not the zeros of a row that sees nothing.
constexpr float kMaxScore = 0x1p30f;  // in units of log2

__device__ __forceinline__ float score_shift(float m, float scale_log2) {
  const float t = m * scale_log2;
  return __builtin_fabsf(t) < kMaxScore ? -t : -__builtin_inff();  // (m = -infinity: nothing seen, all weights 0)
}
// A row's largest score in units of log2, -infinity only if that is what it is.
__device__ __forceinline__ float row_top(float m, float scale_log2) {
  return m == -__builtin_inff() ? m : fmaxf(m * scale_log2, -3.4e38f);
}
// 1 / the sum of a row's weights.
__device__ __forceinline__ float row_inverse(float top, float sum) {
  if (top > -__builtin_inff() && !(__builtin_fabsf(top) < kMaxScore)) return __builtin_nanf("");
  return sum == 0.0f ? 0.0f : 1.0f / sum;
}

}  // namespace mxq
