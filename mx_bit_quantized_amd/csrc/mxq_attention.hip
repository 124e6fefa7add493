// mxq_attention.hip - attention of ragged sequences (mxq_attention).
//
// One pass over the keys with a running maximum and sum per query. A workgroup
// holds 32 QT NW rows of one key head and sequence: row R is query R / G, head
// R % G of the G query heads that share the key head, so that all of them read a
// key tile once. Tiles of 64 keys and their values go to LDS by asynchronous
// copies, one tile ahead.
//
// Both products are 32x32x16 bf16 MFMAs on transposed operands: S^T = K Q^T puts a
// query's scores into one lane (and the lane 32 further), so that its maximum and
// sum need one exchange, and its 16 scores of 32 keys are, packed to bf16, the
// operand B of O^T = V^T P^T without a move between lanes: the product may take
// the keys in any order, and the transposing LDS reads of V take them in the order
// that the scores are held in.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq_attention.h"
#include "mxq_convert.h"
#include "mxq_device.h"
#include "mxq_internal.h"

namespace mxq {

typedef __bf16 bf16x8_v __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4_v __attribute__((ext_vector_type(4)));
typedef unsigned u32x2_v __attribute__((ext_vector_type(2)));

constexpr int kKeys = 64;  // keys of a tile

struct AttnArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* starts_q;
  const int32_t* starts_k;
  uint16_t* out;
  float* part;
  int64_t ldq, ldk, ldv, ldo;
  int sequences, Mq, Mk, left, right, sinks, kv_heads, group, slots, items, splits;
  float scale_log2;
};

// A copy of 16 bytes a lane from memory to LDS: lane i's lands at lds + 16 i.
__device__ __forceinline__ void copy16(const void* src, void* lds) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
}

__device__ __forceinline__ float other_half_max(float v) {
  const u32x2_v r = __builtin_amdgcn_permlane32_swap(as_uint(v), as_uint(v), false, false);
  return fmaxf(as_float(r[0]), as_float(r[1]));
}
__device__ __forceinline__ float other_half_sum(float v) {
  const u32x2_v r = __builtin_amdgcn_permlane32_swap(as_uint(v), as_uint(v), false, false);
  return as_float(r[0]) + as_float(r[1]);
}

// Chunk (16 bytes) of a tile row at which chunk c of key `row` is kept. K rows are
// read by 32 lanes at one chunk, V rows by 8 keys at 64 bytes: either way the lanes
// of one LDS pass meet all banks.
template <int D>
__device__ __forceinline__ int k_chunk(int row, int c) {
  return D == 128 ? c ^ (row & 15) : c ^ ((row >> 1) & 7);
}
template <int D>
__device__ __forceinline__ int v_chunk(int row, int c) {
  return D == 128 ? c ^ ((row & 3) << 2) : c ^ (((row >> 1) & 1) << 2);
}

template <int D, int QT, int NW>
__global__ __launch_bounds__(64 * NW) void attention_kernel(const AttnArgs a) {
  constexpr int ROWS = 32 * QT * NW, CH = D / 8, TILE = kKeys * D * 2;
  constexpr int COPIES = TILE / 1024 / NW;  // of 1 KiB, per wave and tensor
  extern __shared__ __attribute__((aligned(128))) uint8_t lds[];  // K, V of one tile, K, V of the next
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, half = lane >> 5, l32 = lane & 31;

  // work item: XCDs take runs of neighbouring items (tiles of one key head meet in one L2)
  const int per_xcd = (a.items + 7) >> 3;
  const int lin = (int)(blockIdx.x & 7) * per_xcd + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per_xcd || lin >= a.items) return;
  const int split = lin % a.splits, item = lin / a.splits;
  const int hk = item / a.slots, slot = a.slots - 1 - item % a.slots;

  // the sequence and tile of a slot: sequence b owns the slots from
  // floor(starts_q[b] G / ROWS) + b on, enough of them for its rows
  int b = 0, q0 = 0, nq = a.Mq, k0 = 0, nk = a.Mk, tile = slot;
  if (a.starts_q != nullptr) {
    int lo = 0, hi = a.sequences;  // first slot of lo <= slot < that of hi
    while (hi - lo > 1) {
      const int step = (hi - lo + 63) >> 6, probe = lo + lane * step;
      const bool in = probe < hi;
      const int64_t s = in ? min(max(a.starts_q[probe], 0), a.Mq) : 0;
      const uint64_t ok = __ballot(in && (lane == 0 || s * a.group / ROWS + probe <= slot));
      const int last = 63 - __builtin_clzll(ok | 1);
      hi = min(hi, lo + (last + 1) * step);
      lo += last * step;
    }
    b = __builtin_amdgcn_readfirstlane(lo);
    q0 = min(max(a.starts_q[b], 0), a.Mq);
    nq = min(max(a.starts_q[b + 1], q0), a.Mq) - q0;
    k0 = min(max(a.starts_k[b], 0), a.Mk);
    nk = min(max(a.starts_k[b + 1], k0), a.Mk) - k0;
    tile = slot - (int)((int64_t)q0 * a.group / ROWS) - b;
  }
  const int64_t rows = (int64_t)nq * a.group;
  const int64_t row0 = (int64_t)tile * ROWS;
  if (tile < 0 || row0 >= rows) return;

  // positions of the workgroup's first and last query, and the keys they see
  const int ta = (int)(row0 / a.group), tb = (int)((min(row0 + ROWS, rows) - 1) / a.group);
  const int pa = nk - nq + ta, pb = nk - nq + tb;
  const int jend = a.right < 0 ? nk : min(nk, max(0, (int)min((int64_t)pb + a.right + 1, (int64_t)nk)));
  const int jbeg = a.left < 0 ? 0 : min(max(0, pa - a.left), jend);
  const int tend = (jend + kKeys - 1) / kKeys;
  const int tbeg = jbeg / kKeys;
  const int nsink = min(tbeg, (min(a.sinks, jend) + kKeys - 1) / kKeys);  // tiles of sinks before the window's
  const int ntiles = nsink + tend - tbeg;
  const int t_first = (int)((int64_t)ntiles * split / a.splits), t_last = (int)((int64_t)ntiles * (split + 1) / a.splits);
  auto tile_key = [&](int t) { return (t < nsink ? t : tbeg + t - nsink) * kKeys; };

  // this wave's rows
  int64_t row[QT];
  int pos[QT];
  const uint16_t* kbase = a.k + (int64_t)k0 * a.ldk + hk * D;
  const uint16_t* vbase = a.v + (int64_t)k0 * a.ldv + hk * D;
  bf16x8_v qf[QT][D / 16];
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    row[i] = row0 + (wave * QT + i) * 32 + l32;
    const int64_t r = min(row[i], rows - 1);
    const int t = (int)(r / a.group), g = (int)(r - (int64_t)t * a.group);
    pos[i] = nk - nq + t;
    const uint16_t* src = a.q + (int64_t)(q0 + t) * a.ldq + (hk * a.group + g) * D + 8 * half;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) qf[i][c] = *reinterpret_cast<const bf16x8_v*>(src + 16 * c);
  }
  const int64_t wrow = row0 + wave * QT * 32;  // positions of the wave's rows
  const int wpa = nk - nq + (int)(min(wrow, rows - 1) / a.group);
  const int wpb = nk - nq + (int)(min(wrow + QT * 32 - 1, rows - 1) / a.group);

  f32x16 o[QT][D / 32];
  float m[QT], l[QT];
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    m[i] = -__builtin_inff();
    l[i] = 0.0f;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[i][d][r] = 0.0f;
  }

  // copies of one tile: rows past the last key repeat it
  auto fetch = [&](int key, int buf) {
    uint8_t* base = lds + buf * 2 * TILE;
#pragma unroll
    for (int c = 0; c < COPIES; ++c) {
      const int piece = wave * COPIES + c;
      const int r = (piece * 64 + lane) / CH, at = (piece * 64 + lane) % CH;
      const int64_t key_row = min(key + r, nk - 1);
      copy16(kbase + key_row * a.ldk + 8 * k_chunk<D>(r, at), base + piece * 1024);
      copy16(vbase + key_row * a.ldv + 8 * v_chunk<D>(r, at), base + TILE + piece * 1024);
    }
  };

  if (t_first < t_last) fetch(tile_key(t_first), 0);
  for (int t = t_first; t < t_last; ++t) {
    const int key = tile_key(t), buf = (t - t_first) & 1;
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (t + 1 < t_last) fetch(tile_key(t + 1), buf ^ 1);
    // whether the wave's rows see the tile at all, and all of it
    const bool none = wrow >= rows || (a.right >= 0 && key > (int64_t)wpb + a.right) ||
                      (a.left >= 0 && key + kKeys - 1 < wpa - a.left && key >= a.sinks);
    if (none) continue;
    const bool whole = key + kKeys <= nk && (a.right < 0 || key + kKeys - 1 <= (int64_t)wpa + a.right) &&
                       (a.left < 0 || key >= wpb - a.left || key + kKeys <= a.sinks);
    const uint8_t* kt = lds + buf * 2 * TILE;
    const uint8_t* vt = kt + TILE;
    f32x16 s[QT][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int i = 0; i < QT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[i][j][r] = 0.0f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const int r = 32 * j + l32;
        const bf16x8_v kf = *reinterpret_cast<const bf16x8_v*>(kt + r * D * 2 + 16 * k_chunk<D>(r, 2 * c + half));
#pragma unroll
        for (int i = 0; i < QT; ++i) s[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[i][c], s[i][j], 0, 0, 0);
      }
    }
    u32x4_v p[QT][2][2];
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      if (!whole) {
        const int hi = a.right < 0 ? nk - 1 : (int)min((int64_t)nk - 1, (int64_t)pos[i] + a.right);
        const int lo = a.left < 0 ? 0 : pos[i] - a.left;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int at = key + 32 * j + 8 * (r >> 2) + 4 * half + (r & 3);
            const bool seen = at <= hi && (at >= lo || at < a.sinks);
            s[i][j][r] = seen ? s[i][j][r] : -__builtin_inff();
          }
      }
      float top = s[i][0][0];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, s[i][j][r]);
      top = fmaxf(other_half_max(top), m[i]);
      if (__any(top > m[i])) {
        const float alpha = top == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f((m[i] - top) * a.scale_log2);
        m[i] = top;
        l[i] *= alpha;
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
          for (int r = 0; r < 16; ++r) o[i][d][r] *= alpha;
      }
      const float shift = m[i] == -__builtin_inff() ? 0.0f : -m[i] * a.scale_log2;
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; r += 2) {
          const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][j][r], a.scale_log2, shift));
          const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][j][r + 1], a.scale_log2, shift));
          sum += e0 + e1;
          p[i][j][r >> 3][(r & 7) >> 1] = bf16x2_rne(e0, e1);
        }
      l[i] += sum;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int d = 0; d < D / 32; ++d) {
          // lanes 16 e .. 16 e + 15 (e = lane / 16) transpose keys 4 (e / 2) .. + 3 at columns 16 (e % 2) ..
          const int r0 = 32 * j + 16 * c + 4 * half + ((lane & 15) >> 2);
          const int col = 32 * d + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);  // element
          const uint8_t* at0 = vt + r0 * D * 2 + 16 * v_chunk<D>(r0, col >> 3) + 2 * (col & 7);
          const uint8_t* at1 = vt + (r0 + 8) * D * 2 + 16 * v_chunk<D>(r0 + 8, col >> 3) + 2 * (col & 7);
          const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)at0);
          const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)at1);
          const bf16x8_v vf = __builtin_bit_cast(bf16x8_v, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
          for (int i = 0; i < QT; ++i)
            o[i][d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, __builtin_bit_cast(bf16x8_v, p[i][j][c]), o[i][d], 0, 0, 0);
        }
  }

#pragma unroll
  for (int i = 0; i < QT; ++i) {
    l[i] = other_half_sum(l[i]);
    if (row[i] >= rows) continue;
    const int t = (int)(row[i] / a.group), g = (int)(row[i] - (int64_t)t * a.group);
    if (a.splits > 1) {
      // unnormalised part: D sums, the maximum (in units of log2) and the sum of weights
      const int64_t at = ((int64_t)split * a.Mq + q0 + t) * (a.kv_heads * a.group) + hk * a.group + g;
      float* dst = a.part + at * D;
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int r = 0; r < 16; r += 4)
          *reinterpret_cast<float4*>(dst + 32 * d + 2 * r + 4 * half) = make_float4(o[i][d][r], o[i][d][r + 1], o[i][d][r + 2], o[i][d][r + 3]);
      if (half == 0) {
        float* ml = a.part + (int64_t)a.splits * a.Mq * (a.kv_heads * a.group) * D + 2 * at;
        ml[0] = m[i] * a.scale_log2;
        ml[1] = l[i];
      }
    } else {
      const float inv = l[i] == 0.0f ? 0.0f : 1.0f / l[i];
      uint16_t* dst = a.out + (int64_t)(q0 + t) * a.ldo + (hk * a.group + g) * D;
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int r = 0; r < 16; r += 4)
          *reinterpret_cast<uint2*>(dst + 32 * d + 2 * r + 4 * half) =
              make_uint2(bf16x2_rne(o[i][d][r] * inv, o[i][d][r + 1] * inv), bf16x2_rne(o[i][d][r + 2] * inv, o[i][d][r + 3] * inv));
    }
  }
}

// Joins the parts of a row: weights 2^(m_s - max). A wave per 64 / (D / 4) rows.
template <int D>
__global__ __launch_bounds__(256) void attention_join_kernel(const AttnArgs a) {
  constexpr int LANES = D / 4;
  const int heads = a.kv_heads * a.group;
  const int end = a.starts_q != nullptr ? min(max(a.starts_q[a.sequences], 0), a.Mq) : a.Mq;
  const int begin = a.starts_q != nullptr ? min(max(a.starts_q[0], 0), a.Mq) : 0;
  const int64_t r = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LANES;
  const int c = (threadIdx.x % LANES) * 4;
  const int64_t row = r / heads;
  if (row < begin || row >= end) return;
  const int64_t total = (int64_t)a.Mq * heads;
  const float* ml = a.part + a.splits * total * D;
  float top = -__builtin_inff();
  for (int s = 0; s < a.splits; ++s) top = fmaxf(top, ml[2 * (s * total + r)]);
  const float at = top == -__builtin_inff() ? 0.0f : top;
  float l = 0.0f;
  float4 o = make_float4(0, 0, 0, 0);
  for (int s = 0; s < a.splits; ++s) {
    const float w = __builtin_amdgcn_exp2f(ml[2 * (s * total + r)] - at);
    const float4 v = *reinterpret_cast<const float4*>(a.part + (s * total + r) * D + c);
    l += w * ml[2 * (s * total + r) + 1];
    o.x += w * v.x;
    o.y += w * v.y;
    o.z += w * v.z;
    o.w += w * v.w;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  *reinterpret_cast<uint2*>(a.out + row * a.ldo + (r - row * heads) * D + c) =
      make_uint2(bf16x2_rne(o.x * inv, o.y * inv), bf16x2_rne(o.z * inv, o.w * inv));
}

constexpr int kQT = 1, kNW = 8, kRows = 32 * kQT * kNW;

static int64_t attention_slots(const mxq_attention_args& g) {
  return g.Mq * (g.heads / g.kv_heads) / kRows + g.sequences;
}

static int attention_splits(const mxq_attention_args& g) {
  const int64_t items = attention_slots(g) * g.kv_heads;
  const int64_t tiles = (g.Mk + kKeys - 1) / kKeys;
  if (items == 0) return 1;
  int64_t s = 512 / items;
  if (s > tiles / 8) s = tiles / 8;
  return s < 2 ? 1 : (int)s;
}

size_t attention_workspace(const mxq_attention_args& g) {
  const int splits = attention_splits(g);
  return splits < 2 ? 0 : (size_t)splits * g.Mq * g.heads * (g.head_dim + 2) * 4;
}

bool attention_fits(const mxq_attention_args& g) {
  return (attention_slots(g) * g.kv_heads * attention_splits(g) + 8) * 64 * kNW < (int64_t(1) << 32);
}

template <int D>
static hipError_t launch(const AttnArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)((a.items + 7) / 8 * 8);
  hipLaunchKernelGGL((attention_kernel<D, kQT, kNW>), dim3(grid), dim3(64 * kNW), 4 * kKeys * D * 2, s, a);
  if (a.splits > 1) {
    const int64_t rows = (int64_t)a.Mq * a.kv_heads * a.group;
    hipLaunchKernelGGL((attention_join_kernel<D>), dim3((unsigned)((rows * (D / 4) + 255) / 256)), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

hipError_t launch_attention(const mxq_attention_args& g, void* workspace, hipStream_t s) {
  auto limit = [](int64_t v) { return (int)(v < 0 ? -1 : v < (1 << 30) ? v : (1 << 30)); };
  AttnArgs a{};
  a.q = static_cast<const uint16_t*>(g.q);
  a.k = static_cast<const uint16_t*>(g.k);
  a.v = static_cast<const uint16_t*>(g.v);
  a.starts_q = g.starts_q;
  a.starts_k = g.starts_k;
  a.out = static_cast<uint16_t*>(g.out);
  a.part = static_cast<float*>(workspace);
  a.ldq = g.ldq; a.ldk = g.ldk; a.ldv = g.ldv; a.ldo = g.ldo;
  a.sequences = (int)g.sequences; a.Mq = (int)g.Mq; a.Mk = (int)g.Mk;
  a.left = limit(g.left); a.right = limit(g.right); a.sinks = limit(g.sinks);
  a.kv_heads = g.kv_heads; a.group = g.heads / g.kv_heads;
  a.slots = (int)attention_slots(g);
  a.splits = attention_splits(g);
  a.items = a.slots * a.kv_heads * a.splits;
  a.scale_log2 = g.scale * 1.4426950408889634f;
  return g.head_dim == 128 ? launch<128>(a, s) : launch<64>(a, s);
}

}  // namespace mxq
