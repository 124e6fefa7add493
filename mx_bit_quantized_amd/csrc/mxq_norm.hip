// mxq_norm.hip - residual add, norm, modulation and the next linear's
// activation quantizer in one pass over the rows (mxq_norm_quantize).
//
// Per row, in fp32: h = RN_bf16(x + g (b - mu_b) r_b), with mu_b, r_b the
// branch's own statistics for a post-norm (0 and 1 without one) and g the gate
// times branch_scale and post-norm weight; then n = (h - mu) r A + B with
// A = weight (1 + scale), B = bias (1 + scale) + shift, rounded to bf16 and
// quantized by the rules of mxq_quantize_act. mu and the mean square are those
// of the rounded h: it is what the next residual add reads, and a caller that
// keeps only h in memory computes the same norm. The variance is the mean
// square of the centred values, a second reduction over registers rather than
// E[v^2] - mu^2, which loses the variance of rows with a large mean.
//
// Bound by memory: x, branch in, h and codes out, each once. A workgroup holds
// whole rows in registers, thread t the 8-element chunks t + T c (c < CH) of R
// rows at a time, so that the per-channel factors A, B, g (fp32, up to 10x a
// row's bytes) are read and combined once per workgroup, not once per row: a
// wave per row, which needs no barrier, would pull them through the L2 for
// every row. Workgroups take contiguous runs of rows. Where their number is a
// multiple of 8, the runs of one XCD are adjacent, so that the 64-byte pieces of a
// code panel's lines meet in one L2; other grids, the 511 workgroups of 75600 x
// 5120 too, keep the launch's order.
// 75600 x 5120, layer norm with gate and modulation: 628 us in bf16 (4.93 TB/s
// over x, branch, h and out; a 2 GiB copy reaches 4.92), MXFP4 543 us (4.65), FP8
// 603 us (4.49, three reductions a row), transformed MXFP4 835 us (3.03: the
// transform's arithmetic and lane exchanges come on top). A vector per token, 18900
// x 5120: 400 us with fp32 vectors and 285 us with bf16 ones, 4.84 and 4.75 TB/s with
// the vectors' bytes. One row of 5120: 2.7 - 4.3 us.
// Spills: from K = 8193 on with a post-norm to MXFP4 (8 registers, transformed 16),
// past 16384 in every form but FP8 (20 to 72): 4000 x 28672 takes 103 us as a plain
// RMS norm, 223 us with a branch and its norm and 305 us to MXFP4.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq_block.h"
#include "mxq_convert.h"
#include "mxq_device.h"
#include "mxq_internal.h"

namespace mxq {

constexpr int kOutBf16 = 0, kOutMxfp4 = 1, kOutFp8 = 2, kOutHadamard = 3;

struct NormArgs {
  const uint16_t* x;
  const uint16_t* branch;
  const void* gate;
  const uint16_t* post_weight;
  const uint16_t* post_bias;
  const uint16_t* weight;
  const uint16_t* bias;
  const void* scale;
  const void* shift;
  const float* act_mult;
  uint16_t* h;
  uint8_t* out;
  uint32_t* out_scales;
  int64_t M, ldx, ldb, ldh, ld_mod, rows_per_group, rows_per_wg;
  int K, post_norm, norm, mod_bf16;
  float eps, branch_scale, k, inv_k;
};

// Sum over the 16 lanes of a DPP row, in every lane of it.
template <int CTRL>
__device__ __forceinline__ float row_get(float v) {
  return as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)as_uint(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float row_sum(float v) {
  v += row_get<0xB1>(v);   // lane ^ 1
  v += row_get<0x4E>(v);   // lane ^ 2
  v += row_get<0x141>(v);  // mirrored in 8: the other quad
  v += row_get<0x140>(v);  // mirrored in 16: the other half
  return v;
}

// The wave's total in lane 63, from the totals of its four 16-lane rows: row
// broadcasts of lane 15 into rows 1 and 3, then of lane 31 into rows 2 and 3
// (masked rows add the zero of the first operand).
__device__ __forceinline__ float wave_total_63(float v) {
  v = row_sum(v);
  v += as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)as_uint(v), 0x142, 0xA, 0xF, false));
  v += as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)as_uint(v), 0x143, 0xC, 0xF, false));
  return v;
}
__device__ __forceinline__ uint32_t wave_max_63(uint32_t v) {
  v = row_max(v);
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));
  return v;
}

// sum / k, correctly rounded: the product with the rounded reciprocal, then one
// step with its exact remainder (Markstein's quotient). The product alone is one
// step off for some k (multiples of 7, 13, 41 among them), and a row of one value c
// then keeps c 2^-24 of it, whose square competes with eps: a layer norm of 28672
// values of 1e5 gave -0.99 in place of 0. Two operations a row.
__device__ __forceinline__ float mean_of(float sum, float k, float inv_k) {
  const float q = sum * inv_k;
  return __builtin_fmaf(__builtin_fmaf(-q, k, sum), inv_k, q);
}

// 8 consecutive modulation values of a group's vector, in fp32.
__device__ __forceinline__ void load_mod8(const void* p, int64_t at, int bf16, float (&f)[8]) {
  if (bf16) {
    bf16x8_to_f32(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at), f);
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 a = q[0], b = q[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
}

// x, branch and h carry no __restrict__: h may be either of the two (a thread
// reads its chunks of a row before it writes them, and no other thread's).
// POST: with a norm of the branch (its statistics and post_bias). HOLD: the factors
// stay in registers for all rows of a group, else they are read at their use.
// AHEAD: the next rows' loads are issued before the arithmetic on the present
// ones, the first ones' before the factors' (at a group's last rows, whose batch
// may be cut short, rows are read again). WPE: waves per SIMD to leave room for.
template <int CH, int R, int OUT, bool POST, bool HOLD, bool AHEAD, int WPE>
__global__ __launch_bounds__(1024) __attribute__((amdgpu_waves_per_eu(WPE))) void norm_quant_kernel(const NormArgs a) {
  // sums of the workgroup's waves, double-buffered: a reduction's reads are
  // over for every wave before the barrier of the next one, so the buffer is
  // free for the one after that
  __shared__ __attribute__((aligned(16))) uint32_t red[2][16][R];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int T = blockDim.x, NW = T >> 6;
  const int chunks = a.K >> 3;
  const int grid = gridDim.x;
  const int lin = (grid & 7) == 0 ? (blockIdx.x & 7) * (grid >> 3) + (blockIdx.x >> 3) : blockIdx.x;
  const int64_t begin = (int64_t)lin * a.rows_per_wg;
  const int64_t end = begin + a.rows_per_wg < a.M ? begin + a.rows_per_wg : a.M;

  bool ok[CH];
  int64_t at[CH];  // first element of the thread's chunks in a row
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    ok[c] = tid + T * c < chunks;
    at[c] = 8 * (int64_t)(tid + T * c);
  }

  int buf = 0;
  // totals over the workgroup of R per-thread values, in every thread
  auto total = [&](float (&v)[R]) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      v[i] = wave_total_63(v[i]);
      if (lane == 63) red[buf][wave][i] = as_uint(v[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] = (lane & 15) < NW ? as_float(red[buf][lane & 15][i]) : 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] = row_sum(v[i]);
    buf ^= 1;
  };
  auto total_max = [&](uint32_t (&v)[R]) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      v[i] = wave_max_63(v[i]);
      if (lane == 63) red[buf][wave][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] = (lane & 15) < NW ? red[buf][lane & 15][i] : 0u;
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] = row_max(v[i]);
    buf ^= 1;
  };
  // Several chunks per thread: the values are unpacked again after a reduction
  // (the compiler would keep all of them in fp32 across it, and spill).
  auto keep_packed = [](uint4 (&v)[CH][R]) {
    if constexpr (CH > 1)
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < R; ++i) asm volatile("" : "+v"(v[c][i].x), "+v"(v[c][i].y), "+v"(v[c][i].z), "+v"(v[c][i].w));
  };
  // mean (layer norm, else 0) and 1 / sqrt(mean square + eps) of R rows of bf16 chunks
  auto stats = [&](uint4 (&v)[CH][R], int kind, float (&mu)[R], float (&rs)[R]) {
#pragma unroll
    for (int i = 0; i < R; ++i) mu[i] = 0.0f;
    if (kind == MXQ_NORM_LAYER) {
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          float f[8];
          bf16x8_to_f32(v[c][i], f);  // zeros past the row's end
          mu[i] += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
        }
      total(mu);
      keep_packed(v);
#pragma unroll
      for (int i = 0; i < R; ++i) mu[i] = mean_of(mu[i], a.k, a.inv_k);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      rs[i] = 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float f[8], s = 0.0f;
        bf16x8_to_f32(v[c][i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = f[e] - mu[i];
          s = __builtin_fmaf(d, d, s);
        }
        rs[i] += ok[c] ? s : 0.0f;
      }
    }
    total(rs);
    keep_packed(v);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      // (a sum past fp32's range is no norm: 0 times its infinity makes the row NaN,
      // where 1 / sqrt(infinity) = 0 would leave finite values, the bias)
      const float v = __builtin_fmaf(rs[i], a.inv_k, a.eps);
      rs[i] = __builtin_fmaf(v, 0.0f, 1.0f / __builtin_sqrtf(v));
    }
  };

  // the factors of one chunk: gate side (GW, GB), then norm side (A, B)
  auto gate_factors = [&](int64_t base, int64_t col, bool live, float (&gw)[8], float (&gb)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      gw[e] = a.branch_scale;
      gb[e] = 0.0f;
    }
    if (!live) return;
    float f[8];
    if (a.gate != nullptr) {
      load_mod8(a.gate, base + col, a.mod_bf16, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) gw[e] *= f[e];
    }
    if (POST && a.post_bias != nullptr) {
      bf16x8_to_f32(*reinterpret_cast<const uint4*>(a.post_bias + col), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) gb[e] = gw[e] * f[e];
    }
    if (POST && a.post_weight != nullptr) {
      bf16x8_to_f32(*reinterpret_cast<const uint4*>(a.post_weight + col), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) gw[e] *= f[e];
    }
  };
  auto norm_factors = [&](int64_t base, int64_t col, bool live, float (&fa)[8], float (&fb)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      fa[e] = 1.0f;
      fb[e] = 0.0f;
    }
    if (!live) return;
    float f[8];
    if (a.weight != nullptr) bf16x8_to_f32(*reinterpret_cast<const uint4*>(a.weight + col), fa);
    if (a.bias != nullptr) bf16x8_to_f32(*reinterpret_cast<const uint4*>(a.bias + col), fb);
    if (a.scale != nullptr) {
      load_mod8(a.scale, base + col, a.mod_bf16, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        fa[e] *= 1.0f + f[e];
        fb[e] *= 1.0f + f[e];
      }
    }
    if (a.shift != nullptr) {
      load_mod8(a.shift, base + col, a.mod_bf16, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) fb[e] += f[e];
    }
  };

  float GW[HOLD ? CH : 1][8], GB[HOLD ? CH : 1][8], A[HOLD ? CH : 1][8], B[HOLD ? CH : 1][8];
  // rows r .. r + R - 1 (those before `end`) into registers
  auto load_rows = [&](int64_t r, uint4 (&x)[CH][R], uint4 (&b)[CH][R]) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const bool live = r + i < end && ok[c];
        x[c][i] = live ? *reinterpret_cast<const uint4*>(a.x + (r + i) * a.ldx + at[c]) : make_uint4(0, 0, 0, 0);
        if (a.branch != nullptr)
          b[c][i] = live ? *reinterpret_cast<const uint4*>(a.branch + (r + i) * a.ldb + at[c]) : make_uint4(0, 0, 0, 0);
      }
  };
  uint4 xn[CH][R], bn[CH][R];
  if constexpr (AHEAD) load_rows(begin, xn, bn);
  int64_t base = 0;           // the group's vectors
  int64_t group_end = begin;  // rows from here on need another group's factors
  // (every thread of the workgroup takes the same path: the loop's bounds and
  // the barriers inside depend on the row range and the arguments only)
  for (int64_t r0 = begin; r0 < end;) {
    if (r0 >= group_end) {
      const int64_t group = a.rows_per_group > 0 ? r0 / a.rows_per_group : 0;
      base = group * a.ld_mod;
      if constexpr (HOLD) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          gate_factors(base, at[c], ok[c], GW[c], GB[c]);
          norm_factors(base, at[c], ok[c], A[c], B[c]);
        }
      }
      group_end = a.rows_per_group > 0 ? (group + 1) * a.rows_per_group : a.M;
      group_end = group_end < end ? group_end : end;
    }
    const int nr = (int)(group_end - r0 < R ? group_end - r0 : R);

    uint4 h[CH][R], b[CH][R];
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          h[c][i] = xn[c][i];
          b[c][i] = bn[c][i];
        }
      load_rows(r0 + nr, xn, bn);
    } else {
      load_rows(r0, h, b);
    }
    float mu[R], rs[R];
    if (a.branch != nullptr) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        mu[i] = 0.0f;
        rs[i] = 1.0f;
      }
      if constexpr (POST) stats(b, a.post_norm, mu, rs);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int f = HOLD ? c : 0;
        if constexpr (!HOLD) gate_factors(base, at[c], ok[c], GW[0], GB[0]);
#pragma unroll
        for (int i = 0; i < R; ++i) {
          float fx[8], fb[8];
          bf16x8_to_f32(h[c][i], fx);
          bf16x8_to_f32(b[c][i], fb);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if constexpr (POST) {
              const float t = __builtin_fmaf((fb[e] - mu[i]) * rs[i], GW[f][e], GB[f][e]);
              fx[e] += ok[c] ? t : 0.0f;
            } else {
              fx[e] = __builtin_fmaf(fb[e], GW[f][e], fx[e]);  // zeros past the row's end
            }
          }
          h[c][i] = make_uint4(bf16x2_rne(fx[0], fx[1]), bf16x2_rne(fx[2], fx[3]), bf16x2_rne(fx[4], fx[5]),
                               bf16x2_rne(fx[6], fx[7]));
          if (a.h != nullptr && i < nr && ok[c]) *reinterpret_cast<uint4*>(a.h + (r0 + i) * a.ldh + at[c]) = h[c][i];
        }
        if constexpr (CH > 2) __builtin_amdgcn_sched_barrier(0);  // one chunk's values at a time
      }
    }
    stats(h, a.norm, mu, rs);

    // n, in bf16, over h
    uint32_t amax[R];
#pragma unroll
    for (int i = 0; i < R; ++i) amax[i] = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int fc = HOLD ? c : 0;
      if constexpr (!HOLD) norm_factors(base, at[c], ok[c], A[0], B[0]);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float f[8];
        bf16x8_to_f32(h[c][i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __builtin_fmaf((f[e] - mu[i]) * rs[i], A[fc][e], B[fc][e]);
        h[c][i] = make_uint4(bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]),
                             bf16x2_rne(f[6], f[7]));
        if constexpr (OUT == kOutFp8) amax[i] = umax(amax[i], ok[c] ? chunk_amax(h[c][i]) : 0u);
      }
      if constexpr (CH > 2) __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (OUT == kOutFp8) total_max(amax);
    keep_packed(h);

#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t row = r0 + i;
      [[maybe_unused]] Fp8Row fr;
      if constexpr (OUT == kOutFp8) {
        fr = fp8_row_setup(amax[i]);
        if (tid == 0 && i < nr) a.out_scales[row] = as_uint(fr.s);
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const bool live = i < nr && ok[c];
        if constexpr (OUT == kOutBf16) {
          if (live) *reinterpret_cast<uint4*>(a.out + 2 * (row * a.K + at[c])) = h[c][i];
        } else if constexpr (OUT == kOutFp8) {
          if (live) *reinterpret_cast<uint2*>(a.out + row * a.K + at[c]) = pack8_fp8(h[c][i], fr);
        } else {
          // lane chunk within its panel of 128 elements: 16 lanes of a DPP row
          const int pc = lane & 15;
          uint4 v = h[c][i];
          if constexpr (OUT == kOutHadamard) {
            // the transformed quantizer's arithmetic: butterflies, RN(t * mult
            // + 0) with the lane's sign in the factor, bf16 (every lane takes
            // part in the exchanges; K is a multiple of 128, so a panel's 16
            // lanes are all in or all out of the row)
            float f[8], m[8];
            bf16x8_to_f32(v, f);
            fwht128_lanes(f, pc);
            const uint32_t neg = (uint32_t)(__builtin_popcount(pc) & 1) << 31;
#pragma unroll
            for (int e = 0; e < 8; ++e) m[e] = 0.0f;
            if (ok[c]) load_mod8(a.act_mult, at[c], 0, m);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = __builtin_fmaf(f[e], as_float(as_uint(m[e]) ^ neg), 0.0f);
            v = make_uint4(bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]),
                           bf16x2_rne(f[6], f[7]));
          }
          // chunks is a multiple of 4: a block's 4 lanes are in the row or out of it together
          const uint32_t am = quad_max(chunk_amax(v));
          const uint32_t sb = ok[c] ? mx_scale_byte(am) : 0u;
          const uint32_t packed = pack8_fp4(v, sb);
          const uint32_t s1 = (uint32_t)__builtin_amdgcn_mov_dpp((int)sb, 0x104, 0xF, 0xF, true);
          const uint32_t s2 = (uint32_t)__builtin_amdgcn_mov_dpp((int)sb, 0x108, 0xF, 0xF, true);
          const uint32_t s3 = (uint32_t)__builtin_amdgcn_mov_dpp((int)sb, 0x10C, 0xF, 0xF, true);
          if (live) {
            const int p = (int)(at[c] >> 7);
            const int w = a.K - 128 * p < 128 ? a.K - 128 * p : 128;
            *reinterpret_cast<uint32_t*>(a.out + (int64_t)p * 64 * a.M + row * (w >> 1) + 4 * pc) = packed;
            if (pc == 0) a.out_scales[(int64_t)p * a.M + row] = sb | (s1 << 8) | (s2 << 16) | (s3 << 24);
          }
        }
        if constexpr (CH > 2) __builtin_amdgcn_sched_barrier(0);
      }
    }
    r0 += nr;
  }
}

template <int CH, int R, bool POST, bool HOLD, bool AHEAD, int WPE>
static void launch_norm_out(int out, const NormArgs& a, int grid, int threads, hipStream_t s) {
  const dim3 g(grid), t(threads);
  switch (out) {
    case kOutMxfp4: hipLaunchKernelGGL((norm_quant_kernel<CH, R, kOutMxfp4, POST, HOLD, AHEAD, WPE>), g, t, 0, s, a); break;
    case kOutFp8: hipLaunchKernelGGL((norm_quant_kernel<CH, R, kOutFp8, POST, HOLD, AHEAD, WPE>), g, t, 0, s, a); break;
    case kOutHadamard: hipLaunchKernelGGL((norm_quant_kernel<CH, R, kOutHadamard, POST, HOLD, AHEAD, WPE>), g, t, 0, s, a); break;
    default: hipLaunchKernelGGL((norm_quant_kernel<CH, R, kOutBf16, POST, HOLD, AHEAD, WPE>), g, t, 0, s, a); break;
  }
}

hipError_t launch_norm_quant(int mode, const mxq_norm_args& g, hipStream_t s) {
  NormArgs a{};
  a.x = static_cast<const uint16_t*>(g.x);
  a.branch = static_cast<const uint16_t*>(g.branch);
  a.gate = g.gate;
  a.post_weight = static_cast<const uint16_t*>(g.post_weight);
  a.post_bias = static_cast<const uint16_t*>(g.post_bias);
  a.weight = static_cast<const uint16_t*>(g.weight);
  a.bias = static_cast<const uint16_t*>(g.bias);
  a.scale = g.scale;
  a.shift = g.shift;
  a.act_mult = g.act_mult;
  a.h = static_cast<uint16_t*>(g.h);
  a.out = static_cast<uint8_t*>(g.out);
  a.out_scales = static_cast<uint32_t*>(g.out_scales);
  a.M = g.M;
  a.K = (int)g.K;
  a.ldx = g.ldx;
  a.ldb = g.ldb;
  a.ldh = g.ldh;
  a.ld_mod = g.ld_mod;
  a.rows_per_group = g.rows_per_group;
  a.post_norm = g.post_norm;
  a.norm = g.norm;
  a.mod_bf16 = g.mod_type == MXQ_MOD_BF16;
  a.eps = g.eps;
  a.branch_scale = g.branch_scale;
  a.k = (float)g.K;
  a.inv_k = 1.0f / a.k;
  const int out = mode == MXQ_W4A4                   ? kOutMxfp4
                  : mode == MXQ_W4A8                 ? kOutFp8
                  : mode == MXQ_POLICY_TRANSFORM_ON  ? kOutHadamard
                                                     : kOutBf16;
  const int chunks = a.K >> 3;
  const int ch = chunks <= 1024 ? 1 : chunks <= 2048 ? 2 : 4;
  const int threads = (chunks + 64 * ch - 1) / (64 * ch) * 64;
  const int waves = threads >> 6;
  // about 20 waves per CU in one round of workgroups, so that the factors are read
  // as seldom as the chip can be filled (75600 x 5120: 512 workgroups 625 us, 1024
  // 670 us; 20000 x 512, one wave each: 5120 workgroups 14 us, 1024 25 us)
  const int64_t wgs = 256 * (20 / waves > 0 ? 20 / waves : 1);
  const int64_t per = (g.M + wgs - 1) / wgs;
  a.rows_per_wg = per;
  const int grid = (int)((g.M + per - 1) / per);
  const bool post = g.post_norm != MXQ_NORM_NONE;
  // Two rows at a time fill the 128-byte lines of a code panel in one workgroup
  // (MXFP4 75600 x 5120: 539 us against 585); with few rows per workgroup one row,
  // its loads issued ahead of the factors' (2048 x 5120: 14.9 us against 16.2); with
  // the branch's statistics one row, two would not fit the registers.
  if (ch == 1) {
    if (post) launch_norm_out<1, 1, true, true, false, 5>(out, a, grid, threads, s);
    else if (per >= 8) launch_norm_out<1, 2, false, true, false, 5>(out, a, grid, threads, s);
    else launch_norm_out<1, 1, false, true, true, 5>(out, a, grid, threads, s);
  } else if (ch == 2) {
    if (post) launch_norm_out<2, 1, true, true, false, 4>(out, a, grid, threads, s);
    else launch_norm_out<2, 1, false, true, false, 4>(out, a, grid, threads, s);
  } else {
    // (four chunks per thread and their factors do not fit: read at their use)
    if (post) launch_norm_out<4, 1, true, false, false, 4>(out, a, grid, threads, s);
    else launch_norm_out<4, 1, false, false, false, 4>(out, a, grid, threads, s);
  }
  return hipGetLastError();
}

}  // namespace mxq
