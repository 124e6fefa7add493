// mxq_tokens.hip - the scaled GEMMs of mxq_gemm_residual and mxq_gemm_gated
// for few rows (decoding: one token per sequence), and for the shapes that
// the pipelined kernel does not take.
//
// With a few rows the product reads the MXFP4 weight once, N K 17/32 bytes,
// and does little else: it is bound by how fast the whole chip pulls that
// stream in. A workgroup owns 32 output columns (for the gated pair the 32
// gate rows and 32 up rows of the same hidden columns, adjacent in the packed
// weight) and its waves (8 or 16) split K: wave w of W takes the 128-element code panels
// w, w + W, ... A wave's load of a panel's 32 rows is 2 KiB of consecutive
// memory. It loads BATCH panels (one, or two with two token tiles), waits and
// multiplies, so that what overlaps loads with arithmetic is the other waves.
// Nothing goes through LDS on the way to the matrix cores: no row is shared
// between waves. The tokens are
// the MFMA's second operand, 32 at a time, from L2; rows past M repeat the last
// one (their columns are not written). The waves' partial sums meet in LDS,
// in wave order, so a result depends on the shape only.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mxq_block.h"
#include "mxq_convert.h"
#include "mxq_device.h"
#include "mxq_internal.h"

namespace mxq {

typedef int v8i_t __attribute__((ext_vector_type(8)));
typedef float v16f_t __attribute__((ext_vector_type(16)));

constexpr int kTokPitch = 36;  // floats per token of a staged 32 x 32 tile (16-byte aligned, banks spread)

// One lane's operands of a panel for a 32-row tile: lane (r, g) holds blocks
// 2g and 2g + 1 of row r (MFMA step kk takes block 2g + kk of both operands),
// scale bytes in the low half of sc. FP8 operands as the mixed instruction
// pairs them: slot g carries half g of block kk, then half g of block 2 + kk.
template <int CHUNKS>
struct TokFrag {
  uint4 d[CHUNKS];
  uint32_t sc;
};

__device__ __forceinline__ void tok_load_fp4(TokFrag<2>& f, const uint8_t* q, const uint32_t* sc, int64_t rows, int64_t row,
                                             int p, int K, int g) {
  const int w = K - 128 * p < 128 ? K - 128 * p : 128;
  const uint4* src = reinterpret_cast<const uint4*>(q + (int64_t)p * 64 * rows + row * (w >> 1)) + 2 * g;
  const int blocks = (w >> 5) - 2 * g;  // of the lane's two
  f.d[0] = blocks > 0 ? src[0] : make_uint4(0, 0, 0, 0);
  f.d[1] = blocks > 1 ? src[1] : make_uint4(0, 0, 0, 0);
  f.sc = sc[(int64_t)p * rows + row] >> (16 * g);
}

__device__ __forceinline__ void tok_load_fp8(TokFrag<4>& f, const uint8_t* q, int64_t row, int p, int K, int g) {
  const int blocks = (K >> 5) - 4 * p;  // blocks in the panel, 4 but for a ragged last one
  const uint4* src = reinterpret_cast<const uint4*>(q + row * K + 128 * (int64_t)p) + g;
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
    f.d[2 * kk] = kk < blocks ? src[2 * kk] : make_uint4(0, 0, 0, 0);
    f.d[2 * kk + 1] = 2 + kk < blocks ? src[2 * (2 + kk)] : make_uint4(0, 0, 0, 0);
  }
  f.sc = 0x7F7Fu;  // 2^0: the per-token scale is applied to the sums
}

__device__ __forceinline__ v8i_t tok_op(const uint4 lo) {
  return v8i_t{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, 0, 0, 0, 0};
}
__device__ __forceinline__ v8i_t tok_op(const uint4 lo, const uint4 hi) {
  return v8i_t{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

__device__ __forceinline__ float mod_value(const void* p, int64_t at, int bf16) {
  return bf16 ? as_float((uint32_t)static_cast<const uint16_t*>(p)[at] << 16) : static_cast<const float*>(p)[at];
}

constexpr int kTokResidual = 0, kTokGated = 1, kTokGatedMxfp4 = 2;

struct TokArgs {
  const uint8_t* wq;
  const uint32_t* ws;
  const uint8_t* aq;
  const void* as;
  const uint16_t* bias;   // gated: of the gate projection
  const uint16_t* bias2;  // gated: of the up projection
  const uint16_t* residual;
  const void* gate;
  uint16_t* y;
  uint8_t* y_scales;
  int64_t ld_mod, rows_per_group;
  int M, N, K;  // N: output columns (gated: the hidden size)
  int mod_bf16, act;
};

// TM: 32-token tiles per workgroup, which share each load of the weight. BATCH:
// panels that a wave has in flight.
template <int MODE, int TM, int KIND, int WAVES, int BATCH, int WPE>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(WPE))) void gemm_tokens_kernel(const TokArgs a) {
  constexpr bool GATED = KIND != kTokResidual;
  constexpr int TN = GATED ? 2 : 1;
  constexpr int XC = MODE == 0 ? 2 : 4;
  __shared__ __attribute__((aligned(16))) float red[WAVES][32 * kTokPitch];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 31, g = lane >> 5;
  const int n0 = blockIdx.x * 32;
  const int m_tiles = (int)(((int64_t)a.M + 32 * TM - 1) / (32 * TM));
  const int n_panels = (a.K + 127) >> 7;
  const int64_t w_rows = GATED ? 2 * (int64_t)a.N : a.N;
  int64_t wrow[TN], xrow[TM];
#pragma unroll
  for (int i = 0; i < TN; ++i) {
    wrow[i] = GATED ? 2 * (int64_t)n0 + 32 * i + r : n0 + r;  // H is a multiple of 32: in range
    if (!GATED && wrow[i] >= a.N) wrow[i] = a.N - 1;
  }
  for (int mt = blockIdx.y; mt < m_tiles; mt += gridDim.y) {
  const int m0 = mt * (32 * TM);
#pragma unroll
  for (int j = 0; j < TM; ++j) xrow[j] = (int64_t)m0 + 32 * j + r < a.M ? m0 + 32 * j + r : a.M - 1;

  v16f_t acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;

  for (int p0 = wave; p0 < n_panels; p0 += WAVES * BATCH) {
    TokFrag<2> wf[BATCH][TN];
    TokFrag<XC> xf[BATCH][TM];
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int p = p0 + WAVES * u;
      if (p < n_panels) {  // the same for the whole wave
#pragma unroll
        for (int i = 0; i < TN; ++i) tok_load_fp4(wf[u][i], a.wq, a.ws, w_rows, wrow[i], p, a.K, g);
#pragma unroll
        for (int j = 0; j < TM; ++j) {
          if constexpr (MODE == 0)
            tok_load_fp4(xf[u][j], a.aq, static_cast<const uint32_t*>(a.as), a.M, xrow[j], p, a.K, g);
          else
            tok_load_fp8(xf[u][j], a.aq, xrow[j], p, a.K, g);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      if (p0 + WAVES * u < n_panels) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
          for (int j = 0; j < TM; ++j) {
            if constexpr (MODE == 0) {
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                  tok_op(wf[u][i].d[0]), tok_op(xf[u][j].d[0]), acc[i][j], 4, 4, 0, (int)wf[u][i].sc, 0, (int)xf[u][j].sc);
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                  tok_op(wf[u][i].d[1]), tok_op(xf[u][j].d[1]), acc[i][j], 4, 4, 1, (int)wf[u][i].sc, 1, (int)xf[u][j].sc);
            } else {
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                  tok_op(wf[u][i].d[0]), tok_op(xf[u][j].d[0], xf[u][j].d[1]), acc[i][j], 4, 0, 0, (int)wf[u][i].sc, 0,
                  (int)xf[u][j].sc);
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                  tok_op(wf[u][i].d[1]), tok_op(xf[u][j].d[2], xf[u][j].d[3]), acc[i][j], 4, 0, 1, (int)wf[u][i].sc, 0,
                  (int)xf[u][j].sc);
            }
          }
      }
    }
  }

  // Tile by tile through LDS: wave w's 32 x 32 sums as [token][column], then
  // thread t < 512 adds the waves' for token t / 16, columns 2 (t % 16), + 1.
  const bool adds = threadIdx.x < 512;
  const int tm = adds ? threadIdx.x >> 4 : 0, tn = (threadIdx.x & 15) * 2;
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    float v[TN][2];
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      if (i + j > 0) __syncthreads();  // the tile before has been read
#pragma unroll
      for (int qq = 0; qq < 4; ++qq)
        *reinterpret_cast<float4*>(&red[wave][r * kTokPitch + 8 * qq + 4 * g]) =
            make_float4(acc[i][j][4 * qq], acc[i][j][4 * qq + 1], acc[i][j][4 * qq + 2], acc[i][j][4 * qq + 3]);
      __syncthreads();
      v[i][0] = v[i][1] = 0.0f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const float2 s = *reinterpret_cast<const float2*>(&red[w][tm * kTokPitch + tn]);
        v[i][0] += s.x;
        v[i][1] += s.y;
      }
    }
    const int64_t m = (int64_t)m0 + 32 * j + tm;
    const bool live = adds && m < a.M;  // whole 16-lane rows at once: the block maximum below stays uniform
    const int n = n0 + tn;
    if constexpr (MODE == 1) {
      const float s = live ? static_cast<const float*>(a.as)[m] : 0.0f;
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        v[i][0] *= s;
        v[i][1] *= s;
      }
    }
    if constexpr (KIND == kTokResidual) {
      if (!live) continue;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (a.bias != nullptr && n + e < a.N) v[0][e] += as_float((uint32_t)a.bias[n + e] << 16);
      if (a.act == MXQ_EPI_GELU_TANH) {
        v[0][0] = gelu_tanh_dev(v[0][0]);
        v[0][1] = gelu_tanh_dev(v[0][1]);
      }
      const int64_t at = (int64_t)m * a.N + n;
      const int64_t gat = a.gate == nullptr ? 0 : (a.rows_per_group > 0 ? m / a.rows_per_group : 0) * a.ld_mod + n;
      float o[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        o[e] = 0.0f;
        if (n + e < a.N) {
          const float res = as_float((uint32_t)a.residual[at + e] << 16);
          o[e] = a.gate == nullptr ? res + v[0][e] : __builtin_fmaf(mod_value(a.gate, gat + e, a.mod_bf16), v[0][e], res);
        }
      }
      const uint32_t o2 = bf16x2_rne(o[0], o[1]);
      if ((a.N & 1) == 0) {
        if (n < a.N) *reinterpret_cast<uint32_t*>(a.y + at) = o2;
      } else {
        if (n < a.N) a.y[at] = (uint16_t)o2;
        if (n + 1 < a.N) a.y[at + 1] = (uint16_t)(o2 >> 16);
      }
    } else {
      float hid[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float gv = v[0][e], uv = v[1][e];
        if (a.bias != nullptr) gv += as_float((uint32_t)a.bias[n + e] << 16);
        if (a.bias2 != nullptr) uv += as_float((uint32_t)a.bias2[n + e] << 16);
        hid[e] = (a.act == MXQ_GATED_SILU ? silu_dev(gv) : gelu_tanh_dev(gv)) * uv;
      }
      const uint32_t h2 = bf16x2_rne(hid[0], hid[1]);
      if constexpr (KIND == kTokGated) {
        if (live) *reinterpret_cast<uint32_t*>(a.y + (int64_t)m * a.N + n) = h2;
      } else {
        // the 16 lanes of a DPP row hold one 32-element block of token m
        uint32_t am = umax(h2 & 0x7FFFu, (h2 >> 16) & 0x7FFFu);
        am = row_max(am);
        const uint32_t sb = mx_scale_byte(am);
        uint32_t byte = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(0u, __builtin_bit_cast(bf16x2_t, h2), as_float(sb << 23), 0) & 0xFFu;
        // four lanes' bytes to one dword, in the quad's first lane
        byte |= (uint32_t)__builtin_amdgcn_mov_dpp((int)byte, 0xB1, 0xF, 0xF, false) << 8;
        byte |= (uint32_t)__builtin_amdgcn_mov_dpp((int)byte, 0x4E, 0xF, 0xF, false) << 16;
        if (live) {
          const int block = n0 >> 5, p = n0 >> 7;
          const int w = a.N - 128 * p < 128 ? a.N - 128 * p : 128;
          uint8_t* codes = reinterpret_cast<uint8_t*>(a.y) + (int64_t)p * 64 * a.M + (int64_t)m * (w >> 1);
          if ((lane & 3) == 0) *reinterpret_cast<uint32_t*>(codes + 16 * (block & 3) + (tn >> 1)) = byte;
          if (tn == 0) {
            uint8_t* sc = a.y_scales + ((int64_t)p * a.M + m) * 4;
            sc[block & 3] = (uint8_t)sb;
            // bytes of blocks past the row's end are zero
            if (block + 1 == a.N >> 5)
              for (int q = (block & 3) + 1; q < 4; ++q) sc[q] = 0;
          }
        }
      }
    }
  }
  __syncthreads();  // the last tile has been read
  }
}

template <int MODE, int KIND>
static hipError_t launch_tokens_kind(const TokArgs& a, hipStream_t s) {
  const unsigned gx = (unsigned)(((int64_t)a.N + 31) / 32);
  auto go = [&](auto tm, auto waves, auto wpe) {
    constexpr int TM = decltype(tm)::value, W = decltype(waves)::value;
    const unsigned gy = (unsigned)(((int64_t)a.M + 32 * TM - 1) / (32 * TM));
    hipLaunchKernelGGL((gemm_tokens_kernel<MODE, TM, KIND, W, TM, decltype(wpe)::value>),
                       dim3(gx, gy < 65535u ? gy : 65535u), dim3(64 * W), 0, s, a);  // row tiles loop beyond
  };
  constexpr std::integral_constant<int, 1> c1;
  constexpr std::integral_constant<int, 2> c2;
  constexpr std::integral_constant<int, 4> c4;
  constexpr std::integral_constant<int, 8> c8;
  constexpr std::integral_constant<int, 16> c16;
  // Loads in flight come from many waves of one panel rather than few of several.
  // One token tile: the narrow outputs of a residual product (160 workgroups at N =
  // 5120) take 16 waves (W4A4 1 x 5120 x 13824: 9.1 us, 8 waves of two panels 10.6), the
  // gated pair 8 waves, two workgroups to a CU (1 x 13824 x 5120: 15.3 us, three panels
  // and one workgroup 16.6, measured side by side). With three sets of weights in
  // turn, which the Infinity Cache holds, the two products take
  // 8.6 and 13.5 us now, from HBM (24 and 16 sets) 11.3 us (3.3 TB/s) and 17.1 us (4.4).
  // More rows: the residual product takes a workgroup per 32 rows, which read the
  // weight again out of the L2 (W4A8 96 x 5120 x 5120 15.8 us, with two tiles per
  // workgroup 21.4; 64 x 5120 x 13824 34.3 and 32.2), the gated pair, whose weight is
  // the larger part, two tiles and two panels (64 x 13824 x 5120: 23.7 us, four
  // panels 42.2).
  if constexpr (KIND == kTokResidual) {
    if (a.M <= 32 && gx < (1u << 22)) go(c1, c16, c4);  // (a grid's threads: kMaxBlockCols)
    else go(c1, c8, c4);
  } else {
    if (a.M <= 32) go(c1, c8, c4);
    else go(c2, c8, c2);
  }
  return hipGetLastError();
}

hipError_t launch_tokens_residual(int mode, const void* a_codes, const void* a_scales, const void* w_codes,
                                  const void* w_scales, const void* bias, int epilogue, const ResidualEpi& e, void* y,
                                  int64_t M, int64_t N, int64_t K, hipStream_t s) {
  TokArgs a{};
  a.wq = static_cast<const uint8_t*>(w_codes);
  a.ws = static_cast<const uint32_t*>(w_scales);
  a.aq = static_cast<const uint8_t*>(a_codes);
  a.as = a_scales;
  a.bias = static_cast<const uint16_t*>(bias);
  a.residual = static_cast<const uint16_t*>(e.residual);
  a.gate = e.gate;
  a.y = static_cast<uint16_t*>(y);
  a.ld_mod = e.ld_mod;
  a.rows_per_group = e.rows_per_group;
  a.mod_bf16 = e.mod_bf16;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.act = epilogue;
  return mode == 0 ? launch_tokens_kind<0, kTokResidual>(a, s) : launch_tokens_kind<1, kTokResidual>(a, s);
}

hipError_t launch_tokens_gated(int mode, const void* a_codes, const void* a_scales, const void* w_codes,
                               const void* w_scales, const void* bias_gate, const void* bias_up, int act, void* y,
                               void* y_scales, int64_t M, int64_t H, int64_t K, hipStream_t s) {
  TokArgs a{};
  a.wq = static_cast<const uint8_t*>(w_codes);
  a.ws = static_cast<const uint32_t*>(w_scales);
  a.aq = static_cast<const uint8_t*>(a_codes);
  a.as = a_scales;
  a.bias = static_cast<const uint16_t*>(bias_gate);
  a.bias2 = static_cast<const uint16_t*>(bias_up);
  a.y = static_cast<uint16_t*>(y);
  a.y_scales = static_cast<uint8_t*>(y_scales);
  a.M = (int)M;
  a.N = (int)H;
  a.K = (int)K;
  a.act = act;
  if (y_scales != nullptr) return launch_tokens_kind<0, kTokGatedMxfp4>(a, s);
  return mode == 0 ? launch_tokens_kind<0, kTokGated>(a, s) : launch_tokens_kind<1, kTokGated>(a, s);
}

}  // namespace mxq
