// mxq_paged.hip - attention of one new token per sequence over a paged
// key-value cache (mxq_attention_paged).
//
// Bound by memory: every visible key and value once. The work is cut on the
// device: units of 16 keys of all sequences and key heads in one row, of which
// each workgroup takes an equal run, whatever the lengths. A workgroup forms the
// running sum of the sequences' units for itself, finds its first sequence and
// walks on from there; a run that holds a whole sequence writes its output, the
// pieces of a cut one go to the workspace and a second kernel joins them. A
// workgroup has at most two pieces (its first and its last run), so the workspace
// does not grow with the batch.
//
// Within a run the four waves take 32 keys at a time (two units; a page holds at
// least one), each with a running maximum and sum of its own, joined in LDS. Keys
// go from memory straight into operand A of S^T = K Q^T (16x16x32 MFMAs, up to 16
// query heads of a key head as columns); values pass through the wave's own LDS
// for the transposing read that makes them operand A of O^T = V^T P^T, so the loop
// has no barrier. Scores, maxima, sums and O are fp32; the weights are rounded to bf16
// for the second product (the sum takes them unrounded), out once. MXFP8 values are
// exact in bf16 (4 bits of significand, the scale a power of two), so both formats
// share the products; the scale is multiplied in on the way to them.
//
// One sequence of 131071, 40 + 8 heads of 128: 101 us, 5.3 TB/s (a copy: 4.9; a read
// has no writes to turn the memory round for). 64 sequences, 262147 tokens in all, MXFP8:
// 118 to 120 us, 4.7 TB/s. Both with the loads of a step issued before the arithmetic on the
// step before: 102 and 124 us without. 9 sequences, window of 2048, heads of 64: 17.6 us
// for 38 MB, 14 of them in this kernel: two steps a wave, so the chain of lengths,
// table, keys, values and joins is what takes the time; then 3.9 us of join.
//
// More than 16 query heads to a key head are pieces of their own, which read the cache
// again: 32 sequences of 8000, one key head of 128, 16, 20, 33 query heads 33, 49, 67 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq_attention.h"
#include "mxq_convert.h"
#include "mxq_device.h"
#include "mxq_internal.h"

namespace mxq {

typedef __bf16 bf16x8_v __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4_v __attribute__((ext_vector_type(4)));
typedef unsigned u32x2_v __attribute__((ext_vector_type(2)));

constexpr int kPagedThreads = 256, kPagedWaves = 4;
// Least run of a workgroup: 32 keys for each wave. Runs of 4, 8, 16 units at least, us, 40 + 8
// heads of 128: 1 sequence of 500 9.5, 10.0, 11.8, 16 of 200 14.9, 13.5, 18.9.
constexpr int kMinUnits = 8;
constexpr int kPartRows = 16;    // query heads of a piece

// Workgroups that share a CU: what the registers of the loads ahead leave (128-long heads
// with three spill and take twice the time). Heads of 64, 9 sequences with a window of
// 2048: 18.1 us with two, 17.5 with three, 20.7 with four.
constexpr int workgroups_per_cu(int head_dim) { return head_dim == 64 ? 3 : 2; }

struct PagedArgs {
  const uint16_t* q;
  const uint8_t* ck;
  const uint8_t* cv;
  const uint8_t* cks;
  const uint8_t* cvs;
  const int32_t* table;
  const int32_t* lengths;
  uint16_t* out;
  float* part;
  int32_t* sums;
  int64_t ldq, ldo, width, pages;
  int sequences, kv_heads, group, qgroups, page_shift, left, sinks, workgroups;
  float scale_log2;
};

// Units of a sequence of n tokens: those of the sinks, then those of the window.
struct Span {
  int sink_units, first_unit, units;
};
__device__ __forceinline__ int full_length(const PagedArgs& a, int b) { return min(max(a.lengths[b], 0), 1 << 30); }
// What the table can hold of it.
__device__ __forceinline__ int held_length(const PagedArgs& a, int full) {
  const int64_t cap = a.width << a.page_shift;
  return (int)(full < cap ? full : cap);
}
__device__ __forceinline__ Span paged_span(const PagedArgs& a, int full) {
  const int n = held_length(a, full);
  Span s;
  const int begin = a.left < 0 ? 0 : max(0, full - 1 - a.left);
  const int end = (n + 15) >> 4;
  s.first_unit = min(begin >> 4, end);
  s.sink_units = min(s.first_unit, (min(a.sinks, n) + 15) >> 4);
  s.units = s.sink_units + end - s.first_unit;
  return s;
}

// Running sums of the sequences' units in LDS (pre[b], b <= sequences) with their lengths,
// and the units' total.
__device__ __forceinline__ int unit_sums(const PagedArgs& a, int* pre, int* len, int* waves) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int before = 0;
  if (tid == 0) pre[0] = 0;
  for (int b0 = 0; b0 < a.sequences; b0 += kPagedThreads) {
    const int b = b0 + tid;
    const int full = b < a.sequences ? full_length(a, b) : 0;
    int v = b < a.sequences ? paged_span(a, full).units : 0;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int u = __shfl_up(v, off);
      if (lane >= off) v += u;
    }
    if (lane == 63) waves[wave] = v;
    __syncthreads();
    int sum = before, all = 0;
#pragma unroll
    for (int w = 0; w < kPagedWaves; ++w) {
      sum += w < wave ? waves[w] : 0;
      all += waves[w];
    }
    if (b < a.sequences) {
      pre[b + 1] = sum + v;
      len[b] = full;
    }
    before += all;
    __syncthreads();
  }
  return before;
}

// Units of each workgroup's run, from the total over sequences and heads.
__device__ __forceinline__ int64_t run_units(const PagedArgs& a, int64_t total) {
  const int64_t c = (total + a.workgroups - 1) / a.workgroups;
  return c > kMinUnits ? c : kMinUnits;
}

__device__ __forceinline__ float quarter_max(float v) {  // over lanes l, l ^ 16, l ^ 32, l ^ 48
  const u32x2_v r = __builtin_amdgcn_permlane32_swap(as_uint(v), as_uint(v), false, false);
  v = fmaxf(as_float(r[0]), as_float(r[1]));
  const u32x2_v t = __builtin_amdgcn_permlane16_swap(as_uint(v), as_uint(v), false, false);
  return fmaxf(as_float(t[0]), as_float(t[1]));
}
__device__ __forceinline__ float quarter_sum(float v) {
  const u32x2_v r = __builtin_amdgcn_permlane32_swap(as_uint(v), as_uint(v), false, false);
  v = as_float(r[0]) + as_float(r[1]);
  const u32x2_v t = __builtin_amdgcn_permlane16_swap(as_uint(v), as_uint(v), false, false);
  return as_float(t[0]) + as_float(t[1]);
}

// 4 E4M3 codes of a block with scale byte sb -> 4 bf16, exact (but below 2^-126).
__device__ __forceinline__ uint2 unpack4_mxfp8(uint32_t codes, uint32_t sb) {
  const float scale = sb == 0 ? as_float(0x00400000u) : as_float(sb << 23);
  uint2 o;
  o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, false));
  o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, true));
  return o;
}

template <int D, bool FP8>
__global__ __launch_bounds__(kPagedThreads, workgroups_per_cu(D)) void paged_kernel(const PagedArgs a) {
  constexpr int UNIT = 16 * D * 2;                  // bytes of a unit's values in LDS
  constexpr int LOADS = FP8 ? D / 64 : D / 32;      // 16-byte loads a lane for a unit of keys (or values)
  constexpr int LINE = FP8 ? D : 2 * D;             // bytes of a key in the cache
  constexpr int CHUNKS = LINE / 16;
  extern __shared__ __attribute__((aligned(128))) uint8_t lds[];  // values [wave][2 units], later the join; then sums
  constexpr int AREA = kPagedWaves * 16 * D * 4;
  __shared__ float join_ml[kPagedWaves][16][2];
  __shared__ int waves[kPagedWaves];
  int* const pre = reinterpret_cast<int*>(lds + AREA);
  int* const len = pre + a.sequences + 1;

  const int tid = threadIdx.x, lane = tid & 63, n16 = lane & 15, g4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int per_seq = unit_sums(a, pre, len, waves);
  const int64_t total = (int64_t)per_seq * a.kv_heads * a.qgroups;
  const int64_t run = run_units(a, total);
  __syncthreads();
  if (blockIdx.x == 0)  // for the second kernel
    for (int i = tid; i <= a.sequences; i += kPagedThreads) a.sums[i] = pre[i];
  int64_t at = (int64_t)blockIdx.x * run;
  const int64_t stop = min(at + run, total);
  if (at >= stop) return;
  int h = (int)(at / per_seq);  // key head and group of query heads
  int b;
  {
    const int x = (int)(at - (int64_t)h * per_seq);
    int lo = 0, hi = a.sequences;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= x)
        lo = mid;
      else
        hi = mid;
    }
    b = lo;
  }
  uint8_t* const vlds = lds + wave * 2 * UNIT;

  while (at < stop) {
    const int64_t head_at = (int64_t)h * per_seq;
    while (pre[b + 1] == pre[b]) ++b;  // (at < stop: a sequence with units follows)
    const int u_first = (int)(at - head_at) - pre[b];
    const int u_all = pre[b + 1] - pre[b];
    const int u_last = (int)min((int64_t)u_all, stop - head_at - pre[b]);
    const int hk = h / a.qgroups, qg = h - hk * a.qgroups;
    const int full = len[b], n = held_length(a, full);
    const Span span = paged_span(a, full);
    const int lo_key = a.left < 0 ? 0 : full - 1 - a.left;
    const int heads_here = min(kPartRows, a.group - qg * kPartRows);
    const int head0 = hk * a.group + qg * kPartRows;

    bf16x8_v qf[D / 32];
    {
      const uint16_t* src = a.q + (int64_t)b * a.ldq + (int64_t)(head0 + min(n16, heads_here - 1)) * D;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        // the elements of a head in the order in which a lane's key loads bring them
        const int e = FP8 ? 16 * (4 * (j >> 1) + g4) + 8 * (j & 1) : 8 * (4 * j + g4);
        qf[j] = *reinterpret_cast<const bf16x8_v*>(src + e);
      }
    }
    f32x4 o[D / 16];
#pragma unroll
    for (int d = 0; d < D / 16; ++d) o[d] = f32x4{0, 0, 0, 0};
    float m = -__builtin_inff(), l = 0.0f;

    // Two units of the wave: their first keys, whether their pages exist, and what the lane
    // loads of them. The page numbers of a step are read one step before its loads, and the
    // loads are issued before the arithmetic on the step before.
    struct Units {
      int key[2], page[2];
      bool live[2];
      uint4 kr[2][LOADS], vr[2][LOADS];
      uint32_t ksc[2][LOADS], vsc[2][LOADS];
    };
    auto look = [&](int u0, Units& x) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int u = min(u0 + i, u_last - 1);
        x.key[i] = 16 * (u < span.sink_units ? u : span.first_unit + u - span.sink_units);
        x.page[i] = a.table[(int64_t)b * a.width + (x.key[i] >> a.page_shift)];
      }
    };
    auto load = [&](int u0, Units& x) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x.live[i] = u0 + i < u_last && (unsigned)x.page[i] < (uint64_t)a.pages;
        const int page = x.live[i] ? x.page[i] : 0;
        const int64_t line = (((int64_t)page * a.kv_heads + hk) << a.page_shift) + (x.key[i] & ((1 << a.page_shift) - 1));
        const uint8_t* kb = a.ck + line * LINE;
        const uint8_t* vb = a.cv + line * LINE;
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
          const int piece = 64 * j + lane;
          x.kr[i][j] = *reinterpret_cast<const uint4*>(kb + n16 * LINE + 16 * (4 * j + g4));
          x.vr[i][j] = *reinterpret_cast<const uint4*>(vb + piece * 16);
          if constexpr (FP8) {
            x.ksc[i][j] = a.cks[(line + n16) * (D / 32) + ((4 * j + g4) >> 1)];
            x.vsc[i][j] = a.cvs[(line + piece / CHUNKS) * (D / 32) + ((piece % CHUNKS) >> 1)];
          }
        }
      }
    };
    auto attend = [&](const Units& x) {
      f32x4 s[2];
      bool part_unit = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s[i] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
          const uint4 k = x.kr[i][j];
          if constexpr (FP8) {
            const uint2 x0 = unpack4_mxfp8(k.x, x.ksc[i][j]), x1 = unpack4_mxfp8(k.y, x.ksc[i][j]);
            const uint2 x2 = unpack4_mxfp8(k.z, x.ksc[i][j]), x3 = unpack4_mxfp8(k.w, x.ksc[i][j]);
            s[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_v, make_uint4(x0.x, x0.y, x1.x, x1.y)),
                                                          qf[2 * j], s[i], 0, 0, 0);
            s[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_v, make_uint4(x2.x, x2.y, x3.x, x3.y)),
                                                          qf[2 * j + 1], s[i], 0, 0, 0);
          } else {
            s[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_v, k), qf[j], s[i], 0, 0, 0);
          }
        }
        // a unit with keys that the query does not see
        const bool all = x.live[i] && x.key[i] + 16 <= n && (x.key[i] >= lo_key || x.key[i] + 16 <= a.sinks);
        part_unit |= !all;
        if (!all) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int k = x.key[i] + 4 * g4 + r;
            const bool seen = x.live[i] && k < n && (k >= lo_key || k < a.sinks);
            s[i][r] = seen ? s[i][r] : -__builtin_inff();
          }
        }
      }
      // values into the wave's LDS: row (key) r of a unit, 32-byte pairs of chunks permuted
      // so that the 16 rows of a transposing read meet all banks
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
          const int piece = 64 * j + lane, r = piece / CHUNKS, c = piece % CHUNKS;
          const uint4 v = x.vr[i][j];
          uint4 lo = v, hi = v;
          if constexpr (FP8) {
            const uint2 x0 = unpack4_mxfp8(v.x, x.vsc[i][j]), x1 = unpack4_mxfp8(v.y, x.vsc[i][j]);
            const uint2 x2 = unpack4_mxfp8(v.z, x.vsc[i][j]), x3 = unpack4_mxfp8(v.w, x.vsc[i][j]);
            lo = make_uint4(x0.x, x0.y, x1.x, x1.y);
            hi = make_uint4(x2.x, x2.y, x3.x, x3.y);
          }
          if (part_unit) {
            const int k = x.key[i] + r;
            if (!(x.live[i] && k < n && (k >= lo_key || k < a.sinks))) lo = hi = make_uint4(0, 0, 0, 0);
          }
          const int swz = D == 128 ? r & 7 : (r >> 1) & 3;
          uint8_t* dst = vlds + i * UNIT + r * D * 2;
          if constexpr (FP8) {
            *reinterpret_cast<uint4*>(dst + 32 * (c ^ swz)) = lo;
            *reinterpret_cast<uint4*>(dst + 32 * (c ^ swz) + 16) = hi;
          } else {
            *reinterpret_cast<uint4*>(dst + 32 * ((c >> 1) ^ swz) + 16 * (c & 1)) = lo;
          }
        }
      float top = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                        fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
      top = fmaxf(quarter_max(top), m);
      if (__any(top > m)) {
        const float alpha = top == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f((m - top) * a.scale_log2);
        m = top;
        l *= alpha;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) o[d] *= alpha;
      }
      const float shift = score_shift(m, a.scale_log2);
      float e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i >> 2][i & 3], a.scale_log2, shift));
        l += e[i];
      }
      const u32x4_v p = {bf16x2_rne(e[0], e[1]), bf16x2_rne(e[2], e[3]), bf16x2_rne(e[4], e[5]), bf16x2_rne(e[6], e[7])};
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        const int r = 4 * g4 + (n16 >> 2);
        const int swz = D == 128 ? r & 7 : (r >> 1) & 3;
        const uint8_t* src = vlds + r * D * 2 + 32 * (d ^ swz) + 8 * (n16 & 3);
        const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)src);
        const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(src + UNIT));
        const bf16x8_v vf = __builtin_bit_cast(bf16x8_v, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
        o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, __builtin_bit_cast(bf16x8_v, p), o[d], 0, 0, 0);
      }
    };

    constexpr int STEP = 2 * kPagedWaves;
    int u0 = u_first + 2 * wave;
    if (u0 < u_last) {
      Units x, y;
      look(u0, x);
      look(u0 + STEP, y);  // (past the run: its last unit, not used)
      load(u0, x);
      for (;;) {
        const bool more = u0 + STEP < u_last;
        if (more) load(u0 + STEP, y);
        Units z;
        look(u0 + 2 * STEP, z);
        attend(x);
        if (!more) break;
        u0 += STEP;
        x = y;
        y.key[0] = z.key[0];
        y.key[1] = z.key[1];
        y.page[0] = z.page[0];
        y.page[1] = z.page[1];
      }
    }

    // join of the waves
    l = quarter_sum(l);
    __syncthreads();
    if (g4 == 0) {
      join_ml[wave][n16][0] = row_top(m, a.scale_log2);
      join_ml[wave][n16][1] = l;
    }
    float* const jo = reinterpret_cast<float*>(lds) + wave * 16 * D;
#pragma unroll
    for (int d = 0; d < D / 16; ++d)
      *reinterpret_cast<float4*>(jo + n16 * D + 16 * d + 4 * g4) = make_float4(o[d][0], o[d][1], o[d][2], o[d][3]);
    __syncthreads();
    const bool whole = u_first == 0 && u_last == u_all;
    // piece 0: a sequence that begins in an earlier run, piece 1: one that begins here
    const int64_t slot = 2 * (int64_t)blockIdx.x + (u_first == 0 ? 1 : 0);
    for (int i = tid; i < heads_here * (D / 4); i += kPagedThreads) {
      const int row = i / (D / 4), c = i % (D / 4) * 4;
      float top = -__builtin_inff();
#pragma unroll
      for (int w = 0; w < kPagedWaves; ++w) top = fmaxf(top, join_ml[w][row][0]);
      const float base = top == -__builtin_inff() ? 0.0f : top;
      float sum = 0.0f;
      float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int w = 0; w < kPagedWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(join_ml[w][row][0] - base);
        const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(lds) + (w * 16 + row) * D + c);
        sum += f * join_ml[w][row][1];
        v.x += f * x.x;
        v.y += f * x.y;
        v.z += f * x.z;
        v.w += f * x.w;
      }
      if (whole) {
        const float inv = row_inverse(top, sum);
        *reinterpret_cast<uint2*>(a.out + (int64_t)b * a.ldo + (int64_t)(head0 + row) * D + c) =
            make_uint2(bf16x2_rne(v.x * inv, v.y * inv), bf16x2_rne(v.z * inv, v.w * inv));
      } else {
        *reinterpret_cast<float4*>(a.part + (slot * kPartRows + row) * D + c) = v;
        if (c == 0) {
          float* ml = a.part + 2 * (int64_t)a.workgroups * kPartRows * D + 2 * (slot * kPartRows + row);
          ml[0] = top;
          ml[1] = sum;
        }
      }
    }
    __syncthreads();
    at = head_at + pre[b] + u_last;
    if (u_last == u_all) {
      ++b;
      if (at == head_at + per_seq) {
        b = 0;
        ++h;
      }
    }
  }
}

// Joins the pieces of cut sequences, and writes the zeros of empty ones. HEADS query heads
// to a workgroup, the pieces of each over 256 / HEADS / (D / 4) groups of threads.
template <int D, int HEADS>
__global__ __launch_bounds__(kPagedThreads) void paged_join_kernel(const PagedArgs a) {
  constexpr int LANES = D / 4, AHEAD = kPagedThreads / HEADS / LANES;
  __shared__ __attribute__((aligned(16))) float so[HEADS][AHEAD][D];
  __shared__ float sml[HEADS][AHEAD][2];
  const int heads = a.kv_heads * a.group;
  const int mine = threadIdx.x / (LANES * AHEAD);
  const int lane = threadIdx.x % LANES, which = threadIdx.x / LANES % AHEAD;
  const int item = min((int)(blockIdx.x * HEADS) + mine, a.sequences * heads - 1);  // (the last one again, past the end)
  const int b = item / heads, head = item - b * heads;
  const int hk = head / a.group, qg = (head - hk * a.group) / kPartRows;
  const int row = head - hk * a.group - qg * kPartRows;
  uint16_t* out = a.out + (int64_t)b * a.ldo + (int64_t)head * D + 4 * lane;
  const int before = a.sums[b], per_seq = a.sums[a.sequences];
  const int units = a.sums[b + 1] - before;
  int64_t i0 = 0, i1 = 0;
  if (units > 0) {
    const int64_t run = run_units(a, (int64_t)per_seq * a.kv_heads * a.qgroups);
    const int64_t f0 = (int64_t)(hk * a.qgroups + qg) * per_seq + before;
    i0 = f0 / run;
    i1 = (f0 + units - 1) / run;
  }
  const float* ml = a.part + 2 * (int64_t)a.workgroups * kPartRows * D;
  float top = -__builtin_inff(), sum = 0.0f;
  float4 v = make_float4(0, 0, 0, 0);
  auto add = [&](float pm, float pl, const float4& x) {
    const float now = fmaxf(top, pm);
    const float base = now == -__builtin_inff() ? 0.0f : now;
    const float f = __builtin_amdgcn_exp2f(top - base), w = __builtin_amdgcn_exp2f(pm - base);
    top = now;
    sum = sum * f + pl * w;
    v.x = v.x * f + x.x * w;
    v.y = v.y * f + x.y * w;
    v.z = v.z * f + x.z * w;
    v.w = v.w * f + x.w * w;
  };
  if (i0 < i1)
#pragma unroll 4  // loads under way together: 64 pieces a head 4.9 us, by two 5.5, by eight 8.7
    for (int64_t i = i0 + which; i <= i1; i += AHEAD) {
      const int64_t at = (2 * i + (i == i0 ? 1 : 0)) * kPartRows + row;
      const float2 p = *reinterpret_cast<const float2*>(ml + 2 * at);
      add(p.x, p.y, *reinterpret_cast<const float4*>(a.part + at * D + 4 * lane));
    }
  if constexpr (AHEAD > 1) {
    *reinterpret_cast<float4*>(&so[mine][which][4 * lane]) = v;
    if (lane == 0) {
      sml[mine][which][0] = top;
      sml[mine][which][1] = sum;
    }
    __syncthreads();
    if (which != 0) return;
#pragma unroll
    for (int i = 1; i < AHEAD; ++i) add(sml[mine][i][0], sml[mine][i][1], *reinterpret_cast<const float4*>(&so[mine][i][4 * lane]));
  }
  if (units > 0 && i0 == i1) return;  // written by the first kernel
  const float inv = row_inverse(top, sum);
  *reinterpret_cast<uint2*>(out) = make_uint2(bf16x2_rne(v.x * inv, v.y * inv), bf16x2_rne(v.z * inv, v.w * inv));
}

static int paged_workgroups(int head_dim) { return 256 * workgroups_per_cu(head_dim); }

static size_t part_bytes(int head_dim) { return (size_t)2 * paged_workgroups(head_dim) * kPartRows * (head_dim + 2) * 4; }

size_t paged_workspace(const mxq_paged_args& g, const mxq_kv_cache& c) {
  return part_bytes(c.head_dim) + (size_t)(g.sequences + 1) * 4;
}

template <int D>
static hipError_t launch(const PagedArgs& a, bool fp8, hipStream_t s) {
  const size_t bytes = kPagedWaves * 16 * D * 4 + (size_t)(2 * a.sequences + 1) * 4;
  if (fp8)
    hipLaunchKernelGGL((paged_kernel<D, true>), dim3(a.workgroups), dim3(kPagedThreads), bytes, s, a);
  else
    hipLaunchKernelGGL((paged_kernel<D, false>), dim3(a.workgroups), dim3(kPagedThreads), bytes, s, a);
  // Few pieces to a sequence: a wave per head; many: a workgroup. The two against each other,
  // us, 40 heads of 128: 1 sequence of 131071 107, 101; 16 of 8000 100, 100; 256 of 1000 188, 196.
  const int heads = a.sequences * a.kv_heads * a.group;
  if (a.sequences * a.kv_heads * a.qgroups * 4 > a.workgroups)
    hipLaunchKernelGGL((paged_join_kernel<D, 4>), dim3((heads + 3) / 4), dim3(kPagedThreads), 0, s, a);
  else
    hipLaunchKernelGGL((paged_join_kernel<D, 1>), dim3(heads), dim3(kPagedThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_attention_paged(const mxq_paged_args& g, const mxq_kv_cache& c, void* workspace, hipStream_t s) {
  auto limit = [](int64_t v) { return (int)(v < 0 ? -1 : v < (1 << 30) ? v : (1 << 30)); };
  PagedArgs a{};
  a.q = static_cast<const uint16_t*>(g.q);
  a.ck = static_cast<const uint8_t*>(c.k);
  a.cv = static_cast<const uint8_t*>(c.v);
  a.cks = static_cast<const uint8_t*>(c.k_scales);
  a.cvs = static_cast<const uint8_t*>(c.v_scales);
  a.table = g.block_table;
  a.lengths = g.lengths;
  a.out = static_cast<uint16_t*>(g.out);
  a.part = static_cast<float*>(workspace);
  a.sums = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + part_bytes(c.head_dim));
  a.ldq = g.ldq; a.ldo = g.ldo; a.width = g.width; a.pages = c.pages;
  a.sequences = (int)g.sequences; a.kv_heads = c.kv_heads; a.group = g.heads / c.kv_heads;
  a.qgroups = (a.group + kPartRows - 1) / kPartRows;
  a.page_shift = __builtin_ctzll((unsigned long long)c.page_size);
  a.left = limit(g.left); a.sinks = limit(g.sinks);
  a.workgroups = paged_workgroups(c.head_dim);
  a.scale_log2 = g.scale * 1.4426950408889634f;
  return c.head_dim == 128 ? launch<128>(a, c.format == MXQ_KV_MXFP8, s) : launch<64>(a, c.format == MXQ_KV_MXFP8, s);
}

}  // namespace mxq
