// mxq_rotary.hip - RMS norm of q and k, rotary positions and the key-value
// cache's rows, in one pass over the stacked q/k/v rows (mxq_rotary_qkv).
//
// A pair of elements is a complex number and its rotation a product with
// exp(i t), t = position * frequency. t is formed in fp64 and reduced there to
// revolutions in [-1/2, 1/2]: in fp32 a position of 10^6 would leave an angle
// error of 0.06. Everything after it (norm, sine, cosine, rotation) is fp32 with
// one rounding to bf16.
//
// Bound by memory: each row in, q and k (and the cache's rows) out, once. A
// workgroup holds R whole rows in registers, thread t the units t + T u of each:
// a unit is 8 pairs of one head, two 16-byte chunks (side by side, or `pairs`
// elements apart when the two halves of a head are paired), so a rotation needs
// no other thread, and outputs may be the inputs' own memory. The angles of a
// token are shared by all its heads: they are computed once per token by the
// first threads and read from LDS. Norm weights stay in registers over the rows
// of a workgroup. The next rows' loads are issued before the arithmetic on these.
//
// 75600 rows of 120 heads of 128, norm over the row, three axes: 620 us, 5.0 TB/s
// (1754 us with loads where they are needed and a thread's 16 bytes 256 apart). 8195
// rows of 56 heads, norm per head, into the cache and dense: 50 us, 5.0 TB/s; into the
// cache alone 49 us, into an MXFP8 one 58, whose codes leave in pieces of 8 bytes and whose
// scales leave as single bytes. One row: 3.3 us, 12 with the call.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq_attention.h"
#include "mxq_convert.h"
#include "mxq_device.h"
#include "mxq_internal.h"

namespace mxq {

constexpr int kMaxPairs = 64;

struct RotaryArgs {
  const uint16_t* qkv;
  const int32_t* positions;
  const double* freqs;
  const int32_t* axis;
  const uint16_t* q_weight;
  const uint16_t* k_weight;
  uint16_t* q;
  uint16_t* k;
  const int32_t* slots;
  uint8_t* ck;
  uint8_t* cv;
  uint8_t* cks;
  uint8_t* cvs;
  int64_t M, ldx, ldq, ldk, ld_pos, capacity, rows_per_wg;
  int heads, kv_heads, dshift, axes, pairs, interleaved, norm, page_shift, mxfp8, units;
  float eps, inv_q, inv_k;  // (inverse elements of a row's q and k)
};

// Sum and maximum over the 8 (head size 128) or 4 (64) lanes of a head.
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)as_uint(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float head_sum(float v, bool wide) {
  v += dpp_f32<0xB1>(v);  // lane ^ 1
  v += dpp_f32<0x4E>(v);  // lane ^ 2
  const float o = dpp_f32<0x141>(v);  // mirrored in 8: the other quad
  return wide ? v + o : v;
}
__device__ __forceinline__ uint32_t head_max(uint32_t v, bool wide) {
  v = quad_max(v);
  const uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false);
  return wide ? umax(v, o) : v;
}

// 8 bf16 -> 8 E4M3 codes of a block with scale 2^(sb - 127), saturating at 448. A NaN is kept,
// in a branch of its own: the median of it and the two bounds would be a bound, and a key of
// -infinity drops out of attention without a trace. (Only a block that holds an infinity or a
// NaN has a scale of 2^120. Without the branch: 58.3 us for 8195 rows of 40 + 8 + 8 heads, 57.7
// so, 57.3 with the bounds alone.)
__device__ __forceinline__ uint2 pack8_mxfp8(const uint4 c, uint32_t sb) {
  float f[8], r[8];
  bf16x8_to_f32(c, f);
  const float inv = as_float((254u - sb) << 23);
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = __builtin_amdgcn_fmed3f(f[i] * inv, -448.0f, 448.0f);
  if (__any(sb >= 247u)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = f[i] != f[i] ? f[i] : r[i];
  }
  uint2 o;
  o.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(r[0], r[1], 0, false);
  o.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(r[2], r[3], (int)o.x, true);
  o.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(r[4], r[5], 0, false);
  o.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(r[6], r[7], (int)o.y, true);
  return o;
}

// E8M0 byte of an MXFP8 block from its largest bf16 magnitude: floor(log2) - 8.
__device__ __forceinline__ uint32_t mxfp8_scale_byte(uint32_t amax_bits) {
  const int b = (int)(amax_bits >> 7) - 8;
  return b < 0 ? 0u : (uint32_t)b;
}

// 1 / sqrt(mean square + eps). A sum of squares past fp32's range is no norm: 0 times its
// infinity makes the row NaN, where 1 / sqrt(infinity) = 0 would leave zeros.
__device__ __forceinline__ float inverse_norm(float sum, float inv_n, float eps) {
  const float v = sum * inv_n + eps;
  return __builtin_fmaf(v, 0.0f, __builtin_amdgcn_rsqf(v));
}

// Rotations of 8 elements by the pairs' cosines and sines: four pairs side by side,
// or eight pairs of one chunk with the other.
__device__ __forceinline__ void turn_interleaved(float (&f)[8], const float* cs, const float* sn) {
  const float4 c = *reinterpret_cast<const float4*>(cs), s = *reinterpret_cast<const float4*>(sn);
  const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float x = f[2 * p], y = f[2 * p + 1];
    f[2 * p] = x * cc[p] - y * ss[p];
    f[2 * p + 1] = x * ss[p] + y * cc[p];
  }
}
__device__ __forceinline__ void turn_halves(float (&f)[8], float (&g)[8], const float* cs, const float* sn) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float4 c = *reinterpret_cast<const float4*>(cs + 4 * h), s = *reinterpret_cast<const float4*>(sn + 4 * h);
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float x = f[4 * h + p], y = g[4 * h + p];
      f[4 * h + p] = x * cc[p] - y * ss[p];
      g[4 * h + p] = x * ss[p] + y * cc[p];
    }
  }
}

template <int U, int R>
__global__ __launch_bounds__(1024) void rotary_qkv_kernel(const RotaryArgs a) {
  // cosines and sines of R tokens, and the waves' sums of q and of k: double-buffered, so
  // that the one barrier of a step also frees the buffer of the step before
  __shared__ __attribute__((aligned(16))) float turn[2][R][2][kMaxPairs];
  __shared__ float red[2][R][2][16];
  const int tid = threadIdx.x, T = blockDim.x, lane = tid & 63, wave = tid >> 6, waves = T >> 6;
  const int D = 1 << a.dshift, per_head = D >> 4;
  const bool wide = per_head == 8;
  const int qn = a.heads * per_head, kn = a.kv_heads * per_head;  // units of q, of k (and of v)
  const int64_t begin = (int64_t)blockIdx.x * a.rows_per_wg;
  const int64_t end = begin + a.rows_per_wg < a.M ? begin + a.rows_per_wg : a.M;

  // the thread's units: part (0 q, 1 k, 2 v, 3 none), head, first elements of the two
  // chunks, first pairs of the chunks (interleaved) or of the unit; -1: not turned
  int part[U], head[U], c0[U], c1[U], p0[U], p1[U];
  int64_t from[U];
  uint4 w0[U], w1[U];
  const uint4 ones = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    int at = (int)blockIdx.y * T + tid + T * u;
    part[u] = at >= a.units ? 3 : at < qn ? 0 : at < qn + kn ? 1 : 2;
    at -= part[u] == 1 ? qn : part[u] == 2 ? qn + kn : 0;
    const int sub = at & (per_head - 1);
    head[u] = part[u] == 3 ? 0 : at / per_head;
    c0[u] = 8 * sub;
    c1[u] = D / 2 + 8 * sub;
    p0[u] = p1[u] = -1;
    if (a.interleaved) {
      if (c0[u] < 2 * a.pairs) p0[u] = c0[u] / 2;
      if (c1[u] < 2 * a.pairs) p1[u] = c1[u] / 2;
    } else if (8 * sub < a.pairs) {
      c1[u] = a.pairs + 8 * sub;
      p0[u] = 8 * sub;
    } else {
      c0[u] = 16 * sub;
      c1[u] = 16 * sub + 8;
    }
    if (part[u] >= 2) p0[u] = p1[u] = -1;
    from[u] = (int64_t)(head[u] + (part[u] == 1 ? a.heads : part[u] == 2 ? a.heads + a.kv_heads : 0)) << a.dshift;
    w0[u] = w1[u] = ones;
    const uint16_t* w = part[u] == 0 ? a.q_weight : part[u] == 1 ? a.k_weight : nullptr;
    if (w != nullptr) {
      w += a.norm == MXQ_ROTARY_NORM_ROW ? (int64_t)head[u] << a.dshift : 0;
      w0[u] = *reinterpret_cast<const uint4*>(w + c0[u]);
      w1[u] = *reinterpret_cast<const uint4*>(w + c1[u]);
    }
  }
  // the pair (and row of a step) whose angle this thread computes
  const int mine = tid % kMaxPairs, mine_row = tid / kMaxPairs;
  const bool turns = mine_row < R && mine < a.pairs;
  double freq = 0.0;
  const int32_t* pos = nullptr;
  if (turns) {
    const int axis = a.axis == nullptr ? 0 : a.axis[mine];
    if ((unsigned)axis < (unsigned)a.axes) {
      freq = a.freqs[mine];
      pos = a.positions + axis * a.ld_pos;
    }
  }
  auto position = [&](int64_t m0) {
    const int64_t m = m0 + mine_row < end ? m0 + mine_row : end - 1;
    return pos != nullptr ? pos[m] : 0;
  };
  auto load = [&](int64_t m0, uint4 (&x0)[U][R], uint4 (&x1)[U][R]) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint16_t* row = a.qkv + (m0 + r < end ? m0 + r : end - 1) * a.ldx;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        x0[u][r] = x1[u][r] = make_uint4(0, 0, 0, 0);
        if (part[u] < 3) {
          x0[u][r] = *reinterpret_cast<const uint4*>(row + from[u] + c0[u]);
          x1[u][r] = *reinterpret_cast<const uint4*>(row + from[u] + c1[u]);
        }
      }
    }
  };

  uint4 x0[U][R], x1[U][R], n0[U][R], n1[U][R];
  load(begin, x0, x1);
  int at_pos = position(begin), next_pos = 0;
  int buf = 0;
  for (int64_t m0 = begin; m0 < end; m0 += R, buf ^= 1) {
    // the next rows' loads are under way during the arithmetic on these (the last step's
    // are its own again; in place that is safe: nothing of them is used)
    const int64_t next = m0 + R < end ? m0 + R : m0;
    load(next, n0, n1);
    next_pos = position(next);
    if (turns) {
      const double rev = (double)at_pos * freq * 0.15915494309189533577;
      float s, c;
      sincospif(2.0f * (float)(rev - __builtin_rint(rev)), &s, &c);
      turn[buf][mine_row][0][mine] = c;
      turn[buf][mine_row][1][mine] = s;
    }
    if (a.norm == MXQ_ROTARY_NORM_ROW) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float sq = 0.0f, sk = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float f[8], g[8], s = 0.0f;
          bf16x8_to_f32(x0[u][r], f);
          bf16x8_to_f32(x1[u][r], g);
#pragma unroll
          for (int e = 0; e < 8; ++e) s += f[e] * f[e] + g[e] * g[e];
          sq += part[u] == 0 ? s : 0.0f;
          sk += part[u] == 1 ? s : 0.0f;
        }
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
          sq += __shfl_xor(sq, off);
          sk += __shfl_xor(sk, off);
        }
        if (lane == 0) {
          red[buf][r][0][wave] = sq;
          red[buf][r][1][wave] = sk;
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t m = m0 + r;
      if (m >= end) break;
      float iq = 1.0f, ik = 1.0f;
      if (a.norm == MXQ_ROTARY_NORM_ROW) {
        float sq = 0.0f, sk = 0.0f;
        for (int w = 0; w < waves; ++w) {
          sq += red[buf][r][0][w];
          sk += red[buf][r][1][w];
        }
        iq = inverse_norm(sq, a.inv_q, a.eps);
        ik = inverse_norm(sk, a.inv_k, a.eps);
      }
      int64_t slot = -1;
      if (a.ck != nullptr) {
        slot = a.slots[m];
        if (slot >= a.capacity) slot = -1;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[8], g[8];
        bf16x8_to_f32(x0[u][r], f);
        bf16x8_to_f32(x1[u][r], g);
        float inv = part[u] == 0 ? iq : ik;
        if (a.norm == MXQ_ROTARY_NORM_HEAD) {
          float s = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) s += f[e] * f[e] + g[e] * g[e];
          inv = inverse_norm(head_sum(s, wide), wide ? 1.0f / 128.0f : 1.0f / 64.0f, a.eps);
        }
        uint4 y0 = x0[u][r], y1 = x1[u][r];
        if (part[u] < 2) {
          if (a.norm != MXQ_ROTARY_NORM_NONE) {
            float v[8], w[8];
            bf16x8_to_f32(w0[u], v);
            bf16x8_to_f32(w1[u], w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              f[e] = f[e] * inv * v[e];
              g[e] = g[e] * inv * w[e];
            }
          }
          const float* cs = turn[buf][r][0];
          const float* sn = turn[buf][r][1];
          if (a.interleaved) {
            if (p0[u] >= 0) turn_interleaved(f, cs + p0[u], sn + p0[u]);
            if (p1[u] >= 0) turn_interleaved(g, cs + p1[u], sn + p1[u]);
          } else if (p0[u] >= 0) {
            turn_halves(f, g, cs + p0[u], sn + p0[u]);
          }
          y0 = make_uint4(bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]), bf16x2_rne(f[6], f[7]));
          y1 = make_uint4(bf16x2_rne(g[0], g[1]), bf16x2_rne(g[2], g[3]), bf16x2_rne(g[4], g[5]), bf16x2_rne(g[6], g[7]));
          uint16_t* out = part[u] == 0 ? a.q : a.k;
          if (out != nullptr) {
            out += m * (part[u] == 0 ? a.ldq : a.ldk) + ((int64_t)head[u] << a.dshift);
            *reinterpret_cast<uint4*>(out + c0[u]) = y0;
            *reinterpret_cast<uint4*>(out + c1[u]) = y1;
          }
        }
        if (slot < 0) continue;  // (all lanes of the workgroup alike)
        uint32_t sb0 = 0, sb1 = 0, kept = 0;
        if (a.mxfp8) {
          // largest magnitudes of the head's blocks of 32; lane j of a head keeps block j's
          const uint32_t m0b = chunk_amax(y0), m1b = chunk_amax(y1);
          for (int b = 0; b < D / 32; ++b) {
            const uint32_t here = head_max(umax(c0[u] >> 5 == b ? m0b : 0u, c1[u] >> 5 == b ? m1b : 0u), wide);
            const uint32_t byte = mxfp8_scale_byte(here);
            sb0 = c0[u] >> 5 == b ? byte : sb0;
            sb1 = c1[u] >> 5 == b ? byte : sb1;
            kept = (lane & (per_head - 1)) == b ? byte : kept;
          }
        }
        if (part[u] == 1 || part[u] == 2) {
          const int64_t page = int64_t(1) << a.page_shift;
          const int64_t line = ((slot >> a.page_shift) * a.kv_heads + head[u]) * page + (slot & (page - 1));
          uint8_t* codes = part[u] == 1 ? a.ck : a.cv;
          if (a.mxfp8) {
            *reinterpret_cast<uint2*>(codes + line * D + c0[u]) = pack8_mxfp8(y0, sb0);
            *reinterpret_cast<uint2*>(codes + line * D + c1[u]) = pack8_mxfp8(y1, sb1);
            const int j = lane & (per_head - 1);
            if (j < D / 32) (part[u] == 1 ? a.cks : a.cvs)[line * (D / 32) + j] = (uint8_t)kept;
          } else {
            uint16_t* out = reinterpret_cast<uint16_t*>(codes) + line * D;
            *reinterpret_cast<uint4*>(out + c0[u]) = y0;
            *reinterpret_cast<uint4*>(out + c1[u]) = y1;
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        x0[u][r] = n0[u][r];
        x1[u][r] = n1[u][r];
      }
    at_pos = next_pos;
  }
}

template <int U, int R>
static hipError_t launch(const RotaryArgs& a, dim3 grid, int threads, hipStream_t s) {
  hipLaunchKernelGGL((rotary_qkv_kernel<U, R>), grid, dim3(threads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_rotary_qkv(const mxq_rotary_args& g, const mxq_kv_cache* cache, hipStream_t s) {
  RotaryArgs a{};
  a.qkv = static_cast<const uint16_t*>(g.qkv);
  a.positions = g.positions;
  a.freqs = g.freqs;
  a.axis = g.axis;
  a.q_weight = static_cast<const uint16_t*>(g.q_weight);
  a.k_weight = static_cast<const uint16_t*>(g.k_weight);
  a.q = static_cast<uint16_t*>(g.q);
  a.k = static_cast<uint16_t*>(g.k);
  a.M = g.M; a.ldx = g.ldx; a.ldq = g.ldq; a.ldk = g.ldk; a.ld_pos = g.ld_pos;
  a.heads = g.heads; a.kv_heads = g.kv_heads; a.dshift = __builtin_ctz((unsigned)g.head_dim);
  a.axes = g.axes; a.pairs = g.pairs; a.interleaved = g.interleaved; a.norm = g.norm; a.eps = g.eps;
  a.inv_q = 1.0f / (float)(g.heads > 0 ? g.heads * g.head_dim : 1);
  a.inv_k = 1.0f / (float)(g.kv_heads > 0 ? g.kv_heads * g.head_dim : 1);
  const int per_head = g.head_dim / 16;
  a.units = (g.heads + g.kv_heads) * per_head;
  if (cache != nullptr) {
    a.slots = g.slots;
    a.ck = static_cast<uint8_t*>(cache->k);
    a.cv = static_cast<uint8_t*>(cache->v);
    a.cks = static_cast<uint8_t*>(cache->k_scales);
    a.cvs = static_cast<uint8_t*>(cache->v_scales);
    a.capacity = cache->pages * cache->page_size;
    a.page_shift = __builtin_ctzll((unsigned long long)cache->page_size);
    a.mxfp8 = cache->format == MXQ_KV_MXFP8;
    a.units += g.kv_heads * per_head;
  }
  // A row's sums need the whole row in one workgroup, which then holds up to four units a
  // thread; heads on their own (or no norm) go to workgroups of 512 units. Two and four units
  // spill registers: 4096 rows, row norm, 64 + 64 (one unit), 65 + 65, 128 + 128 (two), 170 +
  // 170 heads of 128 (four) 49, 245, 327, 617 us.
  const bool row_norm = g.norm == MXQ_ROTARY_NORM_ROW;
  const int parts = row_norm ? 1 : (a.units + 511) / 512;
  const int units = (a.units + parts - 1) / parts;
  const int U = units <= 1024 ? 1 : units <= 2048 ? 2 : 4;
  // Two rows a step pay where many workgroups stream; few rows need as many workgroups as they
  // can get. One row a step against two, us: 1 row of 40 + 8 + 8 heads of 128 3.2, 3.4, 1536
  // rows 9.5, 10.9, 8192 rows 35.4, 36.0; 64 + 8 + 8 heads 1536 rows 16.5, 16.9, 4096 rows 36.2,
  // 32.6, 8192 rows 62.6, 58.8.
  const int R = g.M < 2048 || U > 1 ? 1 : 2;
  int threads = ((units + U - 1) / U + 63) / 64 * 64;
  if (threads < R * kMaxPairs) threads = R * kMaxPairs;
  const int64_t steps = (g.M + R - 1) / R;
  const int64_t most = 256 * (1024 / threads);
  const int64_t grid = steps < most ? steps : most;
  a.rows_per_wg = (steps + grid - 1) / grid * R;
  const dim3 wgs((unsigned)((g.M + a.rows_per_wg - 1) / a.rows_per_wg), (unsigned)parts);
  if (U == 1) return R == 1 ? launch<1, 1>(a, wgs, threads, s) : launch<1, 2>(a, wgs, threads, s);
  if (U == 2) return launch<2, 1>(a, wgs, threads, s);
  return launch<4, 1>(a, wgs, threads, s);
}

}  // namespace mxq
