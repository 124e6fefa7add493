// mxq_attention.hip - attention of ragged sequences (mxq_attention).
//
// One pass over the keys with a running maximum m and sum l per query:
//   m' = max(m, max_j s_j), l' = l 2^(m - m') + sum_j 2^(s_j - m'),
//   o' = o 2^(m - m') + sum_j 2^(s_j - m') v_j, out = o / l,
// s in units of log2. Scores, m, l and o are fp32; the weights 2^(s - m') are
// rounded to bf16 for the second product (the sum takes them unrounded), and out
// once: a relative error of .0020 to .0024 against 64 bits, .0017 of it out's own.
//
// A workgroup holds 32 NW rows of one key head and sequence: row R is query R / G,
// head R % G of the G query heads that share the key head, so that all of them read
// a key tile once. Tiles of 64 keys and their values go to LDS by asynchronous
// copies, one to two tiles ahead, double-buffered.
//
// Both products are 32x32x16 bf16 MFMAs on transposed operands: S^T = K Q^T puts a
// query's scores into one lane (and the lane 32 further), so that its maximum and
// sum need one exchange, and its 16 scores of 32 keys are, packed to bf16, the
// operand B of O^T = V^T P^T without a move between lanes: the product may take
// the keys in any order, and the transposing LDS reads of V take them in the order
// that the scores are held in.
//
// A wave issues MFMAs and vector instructions one after the other, and the two
// pipes work side by side only if they alternate. So a step takes the scores of
// tile t + 1 and, slot by slot between their MFMAs and those of O, the exponentials,
// sums, packing and maxima of tile t, fixed in place by scheduling barriers; operand
// A is read from LDS eight fragments ahead, and a step has one barrier.
//
// 32760 x 32760, 40 heads of 128: 17.1 to 18.4 ms by the card, 1.19 to 1.29 PFLOP/s,
// against 1.41 to 1.65 PFLOP/s of large library products. There the MFMAs are busy
// 73 to 74% of the cycles and the power cap holds the clock at 1.6 GHz (all-zero operands:
// 12.95 ms). 65520 queries against 741 keys (6.5 tiles a workgroup): 656 to 684 us,
// 0.81 to 0.84 PFLOP/s; of a workgroup's 28000 cycles 15500 are steps, 5700 the first
// loads (rows of q from HBM, as the output's on their way there: 2.0 TB/s), 3300 the
// first scores and the last product without their counterparts, 2800 the way out.
// Causal prompts with a window of 1024: 326 to 343 us, 0.88 PFLOP/s, the same ends and the
// tiles that the window cuts (a fifth of them). Heads of 64, 296 rows, 30011 keys:
// 37 us, 0.49 PFLOP/s: as many exponentials for half the products, 23% of the last
// tile's rows empty, and the join (5 us).
//
// Slower, and not kept (before against after, in us or ms): two query tiles a wave at
// one wave per SIMD 17.5, 22 ms; the sum from the rounded weights by dot products
// 17.5, 18.2 ms; workgroups that stay and take the next tile 1% faster in the text
// case, 4% slower with the window; rows of q brought to the L2 by the workgroup
// before 667, 690; key heads in turn instead of one after the other 692, 699.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>

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

// n / d for n < 2^31 as a product: mul = ceil(2^(32 + shift) / d), 2^shift < d <= 2^(shift + 1).
struct Divider {
  uint32_t mul, shift, d;
};
static Divider divider(uint32_t d) {
  if (d == 1) return {0, 0, 1};
  const uint32_t shift = 31 - __builtin_clz(d - 1);
  return {(uint32_t)(((uint64_t(1) << (32 + shift)) + d - 1) / d), shift, d};
}
__device__ __forceinline__ int divide(int n, const Divider& by) {
  return by.d == 1 ? n : (int)(__umulhi((uint32_t)n, by.mul) >> by.shift);
}

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
  Divider by_group, by_slots, by_splits;
  float scale_log2, slack;  // slack: how far a score may lie above the running maximum
};

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

// What a workgroup works on: a tile of rows of one sequence and key head, and the key
// tiles that its queries see.
struct Work {
  int hk, split, q0, k0, nq, nk;
  int row0, rows;  // of queries and heads (below 2^31)
  int tbeg, nsink, t_first, t_last;
};

template <int ROWS>
__device__ __forceinline__ bool find_work(const AttnArgs& a, int lane, Work& w) {
  // XCDs take runs of neighbouring items (tiles of one key head meet in one L2)
  const int per_xcd = (a.items + 7) >> 3;
  const int lin = (int)(blockIdx.x & 7) * per_xcd + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per_xcd || lin >= a.items) return false;
  const int item = divide(lin, a.by_splits);
  w.split = lin - item * a.splits;
  w.hk = divide(item, a.by_slots);
  const int slot = a.slots - 1 - (item - w.hk * a.slots);

  // the sequence and tile of a slot: sequence b owns the slots from
  // floor(starts_q[b] G / ROWS) + b on, enough of them for its rows
  w.q0 = 0; w.nq = a.Mq; w.k0 = 0; w.nk = a.Mk;
  int tile = slot;
  if (a.starts_q != nullptr) {
    int lo = 0, hi = a.sequences;  // first slot of lo <= slot < that of hi
    auto first_slot = [&](int b, int s) { return s * a.group / ROWS + b; };
    while (hi - lo > 64) {
      const int step = (hi - lo + 63) >> 6, probe = lo + lane * step;
      const bool in = probe < hi;
      const int s = in ? min(max(a.starts_q[probe], 0), a.Mq) : 0;
      const uint64_t ok = __ballot(in && (lane == 0 || first_slot(probe, s) <= slot));
      const int last = 63 - __builtin_clzll(ok | 1);
      hi = min(hi, lo + (last + 1) * step);
      lo += last * step;
    }
    // of up to 64 sequences all that is needed, one a lane
    const int probe = min(lo + lane, hi - 1);
    const int q0 = min(max(a.starts_q[probe], 0), a.Mq), q1 = min(max(a.starts_q[probe + 1], q0), a.Mq);
    const int k0 = min(max(a.starts_k[probe], 0), a.Mk), k1 = min(max(a.starts_k[probe + 1], k0), a.Mk);
    const uint64_t ok = __ballot(lane < hi - lo && (lane == 0 || first_slot(probe, q0) <= slot));
    const int at = 63 - __builtin_clzll(ok | 1), b = lo + at;
    w.q0 = __builtin_amdgcn_readlane(q0, at);
    w.nq = __builtin_amdgcn_readlane(q1, at) - w.q0;
    w.k0 = __builtin_amdgcn_readlane(k0, at);
    w.nk = __builtin_amdgcn_readlane(k1, at) - w.k0;
    tile = slot - w.q0 * a.group / ROWS - b;
  }
  w.rows = w.nq * a.group;
  if (tile < 0 || tile > (w.rows - 1) / ROWS || w.rows == 0) return false;
  w.row0 = tile * ROWS;

  // positions of the first and last query, and the tiles of the keys they see: those of
  // the sinks that lie before the window's, then the window's
  const int pa = w.nk - w.nq + divide(w.row0, a.by_group);
  const int pb = w.nk - w.nq + divide(min(w.row0 + (ROWS - 1), w.rows - 1), a.by_group);
  const int jend = a.right < 0 ? w.nk : max(0, (int)min((int64_t)pb + a.right + 1, (int64_t)w.nk));
  const int jbeg = a.left < 0 ? 0 : min(max(0, pa - a.left), jend);
  w.tbeg = jbeg / kKeys;
  w.nsink = min(w.tbeg, (min(a.sinks, jend) + kKeys - 1) / kKeys);
  const int tiles = w.nsink + (jend + kKeys - 1) / kKeys - w.tbeg;
  w.t_first = divide(tiles * w.split, a.by_splits);  // (below 2^24 tiles, and 2^6 splits)
  w.t_last = divide(tiles * (w.split + 1), a.by_splits);
  return true;
}

typedef int i32x4 __attribute__((ext_vector_type(4)));

// A copy of 16 bytes a lane from a buffer to LDS: lane i's, at byte off, lands at lds + 16 i;
// past the buffer's end it is zeros. In asm, so that the compiler's waits for it (it would
// wait for all copies before the next LDS read) stay out of the loop, which waits before its
// barrier. M0 needs one wait state before the copy. A resource that a vector instruction
// wrote (the compiler brings spilled ones back so) would need five; none is spilled here, and
// a test reads the distance off the built code. ONCE: data that is read once leaves the caches
// to the rest (q so, and out stored so: 15 MB of keys and values, 1.3 GB of q and out, 691 us without
// and 676 with).
template <bool ONCE = false>
__device__ __forceinline__ void copy16(const i32x4& rs, uint32_t off, uint32_t lds) {
  if constexpr (ONCE)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
                 :: "s"(lds), "v"(off), "s"(rs) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :: "s"(lds), "v"(off), "s"(rs) : "memory", "m0");
}
__device__ __forceinline__ void tile_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ void read_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ uint32_t lds_word(uint32_t at) {
  return *reinterpret_cast<const __attribute__((address_space(3))) uint32_t*>(at);
}
// Two bf16 values, infinities and NaNs replaced by zeros.
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t v) {
  if ((v & 0x7F80u) == 0x7F80u) v &= 0xFFFF0000u;
  if ((v & 0x7F800000u) == 0x7F800000u) v &= 0xFFFFu;
  return v;
}
__device__ __forceinline__ bf16x8_v lds_row(uint32_t at) {
  return *reinterpret_cast<const __attribute__((address_space(3))) bf16x8_v*>(at);
}
__device__ __forceinline__ s16x4 lds_columns(uint32_t at) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<__attribute__((address_space(3))) s16x4*>(at));
}

template <int N, class F>
__device__ __forceinline__ void unroll(F&& f) {
  [&]<int... I>(std::integer_sequence<int, I...>) { (f(std::integral_constant<int, I>{}), ...); }(std::make_integer_sequence<int, N>{});
}

// (heads of 64: three workgroups on a CU where there are as many)
template <int D, int NW>
__global__ __launch_bounds__(64 * NW, D == 64 ? 3 : 2) void attention_kernel(const AttnArgs a) {
  constexpr int ROWS = 32 * NW, CH = D / 8, TILE = kKeys * D * 2, DC = D / 16, DT = D / 32;
  constexpr int COPIES = TILE / 1024 / NW;  // of 1 KiB, per wave and tensor
  extern __shared__ __attribute__((aligned(128))) uint8_t lds[];  // [2] of a tile's K, V
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, l32 = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  Work w;
  if (!find_work<ROWS>(a, lane, w)) return;
  const int nk = w.nk, ntiles = w.t_last - w.t_first;
  auto tile_key = [&](int t) {
    t += w.t_first;
    return (t < w.nsink ? t : w.tbeg + t - w.nsink) * kKeys;
  };

  // copies of a tile; rows past the last key are zeros
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const uint16_t* kbase = a.k + (int64_t)w.k0 * a.ldk + w.hk * D;
  const uint16_t* vbase = a.v + (int64_t)w.k0 * a.ldv + w.hk * D;
  uint32_t koff[COPIES], voff[COPIES];
#pragma unroll
  for (int c = 0; c < COPIES; ++c) {
    const int piece = (wave * COPIES + c) * 64 + lane, r = piece / CH, at = piece % CH;
    koff[c] = (uint32_t)(2 * (r * a.ldk + 8 * k_chunk<D>(r, at)));
    voff[c] = (uint32_t)(2 * (r * a.ldv + 8 * v_chunk<D>(r, at)));
  }
  // the rows of tile t; past the last tile nothing (zeros, to a place that is not read any more)
  auto tile_rows = [&](const uint16_t* base, int64_t ld, int t) {
    const int key = tile_key(t);
    const uint64_t at = (uint64_t)(base + key * ld);
    const int last = min(nk - key, kKeys) - 1;  // (64 rows of 2^24 elements stay below 2^31 bytes)
    i32x4 r;
    r.x = (int)(uint32_t)at;
    r.y = (int)(uint32_t)(at >> 32) & 0xFFFF;
    r.z = t < ntiles ? last * (int)ld * 2 + 2 * D : 0;
    r.w = 0x00020000;
    return r;
  };
  auto copy_k = [&](const i32x4& rs, int c, int buf) { copy16(rs, koff[c], lds0 + buf * 2 * TILE + (wave * COPIES + c) * 1024); };
  auto copy_v = [&](const i32x4& rs, int c, int buf) {
    copy16(rs, voff[c], lds0 + buf * 2 * TILE + TILE + (wave * COPIES + c) * 1024);
  };
  auto fetch_k = [&](int t, int buf) {
    const i32x4 rs = tile_rows(kbase, a.ldk, t);
#pragma unroll
    for (int c = 0; c < COPIES; ++c) copy_k(rs, c, buf);
  };
  auto fetch_v = [&](int t, int buf) {
    const i32x4 rs = tile_rows(vbase, a.ldv, t);
#pragma unroll
    for (int c = 0; c < COPIES; ++c) copy_v(rs, c, buf);
  };

  // The loop takes two steps a turn (scores and buffers change places without moves): of an
  // odd number of steps the first one precedes it.
  const int odd = (ntiles - 1) & 1;

  // Token, head and position of the lane's row; the place of the wave's first token in q or
  // out, and how far behind it the lane's row begins, in bytes (32 rows of 2^24 elements).
  const int wrow = min(w.row0 + wave * 32, w.rows - 1), row = w.row0 + wave * 32 + l32;
  const int token0 = divide(wrow, a.by_group), token = divide(min(row, w.rows - 1), a.by_group);
  const int head = min(row, w.rows - 1) - token * a.group, pos = nk - w.nq + token;
  auto base = [&](int64_t ld) { return (int64_t)(w.q0 + token0) * ld + w.hk * a.group * D; };
  auto offset = [&](int64_t ld) { return (uint32_t)((token - token0) * (int)ld + head * D) * 2; };

  // The wave's rows of q. With four waves they come as whole rows through LDS, through the
  // places that the wave itself fills with the second tile (its fragments straight from memory
  // are 32 bytes of 32 rows at a time: with the way out through LDS 695 us, 682 so, for 65520
  // queries and 741 keys); eight waves have no such room, and a longer run to spread it over.
  constexpr int QPIECES = D / 16;  // of 1 KiB: 64 / CH rows each
  constexpr bool STAGED = QPIECES == 2 * COPIES;
  bf16x8_v qf[DC];
  auto staged = [&](int c) { return lds0 + (odd ^ 1) * 2 * TILE + (c < COPIES ? 0 : TILE - COPIES * 1024) + (wave * COPIES + c) * 1024; };
  if (ntiles > 0) {
    if constexpr (STAGED) {
      const uint64_t at = (uint64_t)(a.q + base(a.ldq));
      const i32x4 rs = {(int)(uint32_t)at, (int)(uint32_t)(at >> 32) & 0xFFFF, 0x7FFFFFFF, 0x00020000};
#pragma unroll
      for (int c = 0; c < QPIECES; ++c) {
        const int r = (c * 64 + lane) / CH;
        copy16<true>(rs, __shfl(offset(a.ldq), r) + 16 * k_chunk<D>(r, lane % CH), staged(c));
      }
    } else {
      const uint16_t* src = a.q + base(a.ldq) + offset(a.ldq) / 2 + 8 * half;
#pragma unroll
      for (int c = 0; c < DC; ++c) qf[c] = *reinterpret_cast<const bf16x8_v*>(src + 16 * c);
    }
    fetch_k(0, odd);
    fetch_v(0, odd);
    if constexpr (!STAGED) fetch_k(1, odd ^ 1);
  }
  const int wpa = nk - w.nq + token0;  // positions of the wave's first and last row
  const int wpb = nk - w.nq + divide(min(wrow + 31, w.rows - 1), a.by_group);

  f32x16 o[DT];
  // per query: the running maximum, what raises it, the exponents' shift that it makes, sums of weights
  float m, bar, shift, l, sum[2];
  auto reset = [&] {
    m = bar = -__builtin_inff();
    shift = l = sum[0] = sum[1] = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[d][r] = 0.0f;
  };
  reset();

  // LDS addresses of the lane's operand reads in buffer 0
  uint32_t ka[DC], va[DT];
#pragma unroll
  for (int c = 0; c < DC; ++c) ka[c] = lds0 + l32 * D * 2 + 16 * k_chunk<D>(l32, 2 * c + half);
#pragma unroll
  for (int d = 0; d < DT; ++d) {
    // lanes 16 e .. 16 e + 15 (e = lane / 16) transpose keys 4 (e / 2) .. + 3 at columns 16 (e % 2) ..
    const int r = 4 * half + ((lane & 15) >> 2), col = 32 * d + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    va[d] = lds0 + TILE + r * D * 2 + 16 * v_chunk<D>(r, col >> 3) + 2 * (col & 7);
  }

  // scores of a tile
  auto scores = [&](f32x16 (&s)[2], uint32_t buf) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int c = 0; c < DC; ++c) {
        const bf16x8_v kf = lds_row(ka[c] + buf + j * 32 * D * 2);
        f32x16 z;
#pragma unroll
        for (int r = 0; r < 16; ++r) z[r] = 0.0f;
        s[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[c], c == 0 ? z : s[j], 0, 0, 0);
      }
  };
  auto maxima = [&](const f32x16 (&s)[2], float& top) {
    float x = s[0][0];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) x = fmaxf(x, s[j][r]);
    top = x;
  };
  // the tiles of the window that all of the wave's rows see whole: whole_from .. + whole_count - 1
  const int whole_key = a.left < 0 ? 0 : max(0, wpb - a.left);
  const int whole_end = a.right < 0 ? nk : (int)min((int64_t)nk, (int64_t)wpa + a.right + 1);
  const int whole_from = max((whole_key + kKeys - 1) / kKeys - w.tbeg, 0) + w.nsink - w.t_first;
  const int whole_count = max(0, (whole_end < 0 ? 0 : whole_end / kKeys) - w.tbeg + w.nsink - w.t_first - whole_from);
  // hides what the wave's rows do not see of tile t; false if that is nothing
  auto hide = [&](f32x16 (&s)[2], int t) {
    if ((unsigned)(t - whole_from) < (unsigned)whole_count) return false;
    const int key = tile_key(t);
    int first = key + 4 * half;  // the lane's keys are first + 32 j + 8 (r / 4) + r % 4
    asm volatile("" : "+v"(first));  // (what follows stays out of the loop's registers)
    const bool high = key + kKeys > whole_end, low = key < whole_key;
    if (high) {
      const int last = (a.right < 0 ? nk - 1 : (int)min((int64_t)nk - 1, (int64_t)pos + a.right)) - first;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          s[j][r] = 32 * j + 8 * (r >> 2) + (r & 3) <= last ? s[j][r] : -__builtin_inff();
    }
    if (low) {
      const int begin = pos - a.left - first, sinks = a.sinks - first;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int at = 32 * j + 8 * (r >> 2) + (r & 3);
          s[j][r] = at >= begin || at < sinks ? s[j][r] : -__builtin_inff();
        }
    }
    return true;
  };
  // raises the running maximum where the tile's is far above it (top: of the lane's keys)
  auto raise = [&](float top) {
    if (!__any(top > bar)) return;
    const float now = fmaxf(other_half_max(top), m);
    const float alpha = now == m ? 1.0f : __builtin_amdgcn_exp2f((m - now) * a.scale_log2);
    m = now;
    bar = now + a.slack;
    shift = score_shift(now, a.scale_log2);
    sum[0] *= alpha;
    sum[1] *= alpha;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[d][r] *= alpha;
  };

  // operand A of a step: its key fragments (of the next tile), then its value fragments
  constexpr int F1 = 2 * DC, F2 = 4 * DT, F = F1 + F2;
  // (the two halves of the keys in turn: an MFMA then does not wait for the one right before)
  auto key_fragment = [&](int f, uint32_t buf) { return lds_row(ka[f / 2] + buf + (f % 2) * 32 * D * 2); };
  auto value_fragment = [&](int f, uint32_t buf) {
    const uint32_t at = va[f % DT] + buf + (f / DT) * 16 * D * 2;
    const s16x4 v0 = lds_columns(at), v1 = lds_columns(at + 8 * D * 2);
    return __builtin_bit_cast(bf16x8_v, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  // vector work of a step, instruction by instruction: per pair of scores the exponents'
  // arguments, the weights, and (of the pair before) their sums and bf16 values; then the
  // maxima of the next tile's scores
  constexpr int PER_PAIR = 7, PAIRS = 16, OPS_W = PER_PAIR * (PAIRS + 1), OPS_M = 16;
  // the weights of the last 16 keys are needed in slot W: all weights come before it,
  // evenly, and the maxima after them
  constexpr int W = F1 + 3 * DT;
  static_assert(PER_PAIR * 13 * W < (F1 + 2 * DT) * OPS_W && PER_PAIR * 9 * W < (F1 + DT) * OPS_W && PER_PAIR * 5 * W < F1 * OPS_W);
  auto ops_before = [](int slot) constexpr {
    return slot <= W ? slot * OPS_W / W : OPS_W + (slot - W) * OPS_M / (F - W);
  };
  float e[2][2], arg[2];
  u32x4_v p[4];
  float top;
  auto vector_op = [&](auto op, f32x16 (&cur)[2], f32x16 (&nxt)[2]) {
    constexpr int n = op;
    if constexpr (n < OPS_W) {
      constexpr int k = n / PER_PAIR, what = n % PER_PAIR;
      if constexpr (what < 4 && k < PAIRS) {
        constexpr int jc = k / 4, r = 8 * (jc & 1) + 2 * (k & 3) + (what & 1);
        if constexpr (what < 2)
          arg[what] = __builtin_fmaf(cur[jc >> 1][r], a.scale_log2, shift);
        else
          e[k & 1][what & 1] = __builtin_amdgcn_exp2f(arg[what & 1]);
      } else if constexpr (what >= 4 && k > 0) {
        constexpr int b = k - 1;
        if constexpr (what < 6) {
          sum[what - 4] += e[b & 1][what - 4];
        } else {
          p[b / 4][b & 3] = bf16x2_rne(e[b & 1][0], e[b & 1][1]);
        }
      }
    } else {
      constexpr int r = 2 * (n - OPS_W);
      const float x = nxt[r >> 4][r & 15], y = nxt[(r + 1) >> 4][(r + 1) & 15];
      top = r == 0 ? fmaxf(x, y) : fmaxf(fmaxf(top, x), y);
    }
  };
  constexpr int LEAD = D == 128 ? 8 : 4;  // fragments of operand A read ahead
  static_assert(F % LEAD == 0 && LEAD >= 2 * COPIES);  // (fragment n is always ring[n % LEAD])
  bf16x8_v ring[LEAD];

  if (ntiles > 0) {
    f32x16 sa[2], sb[2];
    tile_barrier();
    if constexpr (STAGED) {
      const uint32_t mine = staged(l32 * CH / 64) + l32 * CH % 64 * 16;
#pragma unroll
      for (int c = 0; c < DC; ++c) qf[c] = lds_row(mine + 16 * k_chunk<D>(l32, 2 * c + half));
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      fetch_k(1, odd ^ 1);
    }
    scores(sa, odd * 2 * TILE);
    hide(sa, 0);
    maxima(sa, top);
    raise(top);
    tile_barrier();  // (the first keys are read: their place takes the third tile's)
    fetch_k(2, odd);
    fetch_v(1, odd ^ 1);
    // Step t: scores of tile t + 1 (nxt) and, from those of tile t (cur), its weights and
    // their product with the values. Each MFMA is followed by its share of the vector work
    // and by the read of the fragment LEAD ahead; LEAD fragments before the end all reads of
    // the step are done and the workgroup meets: the step's tiles give way to those two
    // further, and the next step's fragments are read.
    auto step = [&](f32x16 (&cur)[2], f32x16 (&nxt)[2], int t, auto par) {
      constexpr uint32_t kbuf = (par ^ 1) * 2 * TILE, vbuf = par * 2 * TILE, next_k = par * 2 * TILE;
      i32x4 rk, rv;
      unroll<F>([&](auto slot) {
        constexpr int f = slot;  // a fragment a slot
        if constexpr (f == F - LEAD) {
          tile_barrier();
          __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (f < F1) {
          f32x16 z;
#pragma unroll
          for (int r = 0; r < 16; ++r) z[r] = 0.0f;
          nxt[f % 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[f % LEAD], qf[f / 2], f < 2 ? z : nxt[f % 2], 0, 0, 0);
        } else {
          constexpr int g = f - F1;
          o[g % DT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ring[f % LEAD], __builtin_bit_cast(bf16x8_v, p[g / DT]), o[g % DT], 0, 0, 0);
        }
        constexpr int ahead = f + LEAD;
        if constexpr (ahead < F1)
          ring[f % LEAD] = key_fragment(ahead, kbuf);
        else if constexpr (ahead < F)
          ring[f % LEAD] = value_fragment(ahead - F1, vbuf);
        else
          ring[f % LEAD] = key_fragment(ahead - F, next_k);
        constexpr int first = ops_before(f), last = ops_before(f + 1);
        // a copy a slot, from the barrier on
        constexpr int c = f - (F - LEAD);
        if constexpr (c == 0) rk = tile_rows(kbase, a.ldk, t + 3);
        if constexpr (c == 1) rv = tile_rows(vbase, a.ldv, t + 2);
        if constexpr (c >= 0 && c < COPIES) copy_k(rk, c, par ^ 1);
        if constexpr (c >= COPIES && c < 2 * COPIES) copy_v(rv, c - COPIES, par);
        unroll<last - first>([&](auto n) { vector_op(std::integral_constant<int, first + n>{}, cur, nxt); });
        __builtin_amdgcn_sched_barrier(0);
      });
      // (used here: the compiler would move sums and maxima behind the branches)
      asm volatile("" : "+v"(top), "+v"(sum[0]), "+v"(sum[1]));
      if (hide(nxt, t + 1)) maxima(nxt, top);
      raise(top);
    };
    if (odd) {
      sb[0] = sa[0];
      sb[1] = sa[1];
      unroll<LEAD>([&](auto f) { ring[f] = key_fragment(f, 0); });
      step(sb, sa, 0, std::integral_constant<int, 1>{});
    } else {
      unroll<LEAD>([&](auto f) { ring[f] = key_fragment(f, 2 * TILE); });
    }
    for (int t = odd; t < ntiles - 1; t += 2) {
      step(sa, sb, t, std::integral_constant<int, 0>{});
      step(sb, sa, t + 1, std::integral_constant<int, 1>{});
    }
    // the last tile's weights and product
    tile_barrier();
    unroll<OPS_W>([&](auto n) { vector_op(n, sa, sb); });
    unroll<F2>([&](auto f) {
      const bf16x8_v vf = value_fragment(f, 0);
      o[f % DT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, __builtin_bit_cast(bf16x8_v, p[f / DT]), o[f % DT], 0, 0, 0);
    });

    // An infinity or a NaN among the values of a tile that some rows see and others do not
    // reaches all of them, as 0 times it. Where a sum is not finite, once more, tile by tile:
    // such values are left out of the product and added to the rows that see them.
    bool spoilt = false;
    if (a.left >= 0 || a.right >= 0) {
      float zero = 0.0f;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) zero = __builtin_fmaf(0.0f, o[d][r], zero);
      spoilt = __syncthreads_or(zero != 0.0f);  // (NaN)
    }
    if (spoilt) {
      reset();
      for (int t = 0; t < ntiles; ++t) {
        fetch_k(t, 0);
        fetch_v(t, 0);
        tile_barrier();
        scores(sa, 0);
        hide(sa, t);
        maxima(sa, top);
        raise(top);
        unroll<OPS_W>([&](auto n) { vector_op(n, sa, sb); });
        unroll<F2>([&](auto f) {
          u32x4_v vf = __builtin_bit_cast(u32x4_v, value_fragment(f, 0));
#pragma unroll
          for (int h = 0; h < 4; ++h) vf[h] = finite_or_zero(vf[h]);
          o[f % DT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_v, vf), __builtin_bit_cast(bf16x8_v, p[f / DT]),
                                                              o[f % DT], 0, 0, 0);
        });
        const int key = tile_key(t);
        for (int r = 0; r < kKeys && key + r < nk; ++r) {
          const uint32_t at = lds0 + TILE + r * D * 2;
          const uint32_t mine = lds_word(at + 4 * (lane & (D / 2 - 1)));
          if (!__any(finite_or_zero(mine) != mine)) continue;
          const bool seen = (a.right < 0 || key + r <= (int64_t)pos + a.right) &&
                            (a.left < 0 || key + r >= pos - a.left || key + r < a.sinks);
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const int el = 32 * d + 2 * e + 4 * half;  // this lane's four elements
              const uint32_t from = at + 16 * v_chunk<D>(r, el >> 3) + 2 * (el & 7);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t v = lds_word(from + 4 * h), kept = finite_or_zero(v);
                if (seen && (v & 0xFFFFu) != (kept & 0xFFFFu)) o[d][e + 2 * h] += as_float(v << 16);
                if (seen && (v >> 16) != (kept >> 16)) o[d][e + 2 * h + 1] += as_float(v & 0xFFFF0000u);
              }
            }
        }
        read_barrier();
      }
    }
    l = sum[0] + sum[1];
  }

  if constexpr (NW != 4) read_barrier();  // (the last values are read: rows take their place)
  l = other_half_sum(l);
  if (a.splits > 1) {
    if (row >= w.rows) return;
    // unnormalised part: D sums, the maximum (in units of log2) and the sum of weights
    const int64_t at = ((int64_t)w.split * a.Mq + w.q0 + token) * (a.kv_heads * a.group) + w.hk * a.group + head;
    float* dst = a.part + at * D;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int r = 0; r < 16; r += 4)
        *reinterpret_cast<float4*>(dst + 32 * d + 2 * r + 4 * half) = make_float4(o[d][r], o[d][r + 1], o[d][r + 2], o[d][r + 3]);
    if (half == 0) {
      float* ml = a.part + (int64_t)a.splits * a.Mq * (a.kv_heads * a.group) * D + 2 * at;
      ml[0] = row_top(m, a.scale_log2);
      ml[1] = l;
    }
  } else {
    // through LDS, so that rows leave whole: 8 bytes a lane in, 16 bytes a lane out, chunks
    // permuted like those of K
    const float inv = row_inverse(row_top(m, a.scale_log2), l);
    const uint32_t mine = lds0 + (NW == 4 ? 2 * TILE : 0) + wave * 64 * D;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int r = 0; r < 16; r += 4)
        *reinterpret_cast<__attribute__((address_space(3))) u32x2_v*>(mine + l32 * D * 2 + 16 * k_chunk<D>(l32, 4 * d + r / 4) + 8 * half) =
            u32x2_v{bf16x2_rne(o[d][r] * inv, o[d][r + 1] * inv), bf16x2_rne(o[d][r + 2] * inv, o[d][r + 3] * inv)};
#pragma unroll
    for (int n = 0; n < CH / 2; ++n) {
      const int r = (n * 64 + lane) / CH, ch = lane % CH;
      const bf16x8_v y = lds_row(mine + r * D * 2 + 16 * k_chunk<D>(r, ch));
      const uint32_t off = __shfl(offset(a.ldo), r) / 2;
      if (w.row0 + wave * 32 + r < w.rows)
        __builtin_nontemporal_store(y, reinterpret_cast<bf16x8_v*>(a.out + base(a.ldo) + off + 8 * ch));
    }
  }
}

// Joins the parts of a row, weights 2^(m_s - max): D / 4 threads to a row and a quarter of
// its parts, the quarters joined in LDS.
constexpr int kJoin = 4;

template <int D>
__global__ __launch_bounds__(256) void attention_join_kernel(const AttnArgs a) {
  constexpr int LANES = D / 4, ROWS = 256 / LANES / kJoin;
  __shared__ __attribute__((aligned(16))) float so[ROWS][kJoin][D];
  __shared__ float sml[ROWS][kJoin][2];
  const int heads = a.kv_heads * a.group;
  const int end = a.starts_q != nullptr ? min(max(a.starts_q[a.sequences], 0), a.Mq) : a.Mq;
  const int begin = a.starts_q != nullptr ? min(max(a.starts_q[0], 0), a.Mq) : 0;
  const int local = threadIdx.x / (LANES * kJoin), which = threadIdx.x / LANES % kJoin, c = (threadIdx.x % LANES) * 4;
  const int64_t r = (int64_t)blockIdx.x * ROWS + local;
  const int64_t row = r / heads;
  const bool live = row >= begin && row < end;
  const int64_t total = (int64_t)a.Mq * heads;
  const float* ml = a.part + a.splits * total * D;
  float top = -__builtin_inff(), l = 0.0f;
  float4 o = make_float4(0, 0, 0, 0);
  auto add = [&](float pm, float pl, const float4& v) {
    const float now = fmaxf(top, pm);
    const float at = now == -__builtin_inff() ? 0.0f : now;
    const float f = __builtin_amdgcn_exp2f(top - at), w = __builtin_amdgcn_exp2f(pm - at);
    top = now;
    l = l * f + pl * w;
    o.x = o.x * f + v.x * w;
    o.y = o.y * f + v.y * w;
    o.z = o.z * f + v.z * w;
    o.w = o.w * f + v.w * w;
  };
  if (live)
#pragma unroll 8  // loads under way together: 21 parts of 2368 rows 5.2 us, by four 5.5
    for (int s = which; s < a.splits; s += kJoin) {
      const float2 p = *reinterpret_cast<const float2*>(ml + 2 * (s * total + r));
      add(p.x, p.y, *reinterpret_cast<const float4*>(a.part + (s * total + r) * D + c));
    }
  *reinterpret_cast<float4*>(&so[local][which][c]) = o;
  if (c == 0) {
    sml[local][which][0] = top;
    sml[local][which][1] = l;
  }
  __syncthreads();
  if (which != 0 || !live) return;
#pragma unroll
  for (int s = 1; s < kJoin; ++s) add(sml[local][s][0], sml[local][s][1], *reinterpret_cast<const float4*>(&so[local][s][c]));
  const float inv = row_inverse(top, l);
  *reinterpret_cast<uint2*>(a.out + row * a.ldo + (r - row * heads) * D + c) =
      make_uint2(bf16x2_rne(o.x * inv, o.y * inv), bf16x2_rne(o.z * inv, o.w * inv));
}

// Keys that a row sees, about: a sequence's, or its window.
static int64_t attention_keys(const mxq_attention_args& g) {
  const int64_t per = g.sequences > 0 ? g.Mk / g.sequences : 0;
  return g.left >= 0 && g.right >= 0 && g.left < per && g.right < per - g.left ? g.left + g.right + 1 : per;
}

// Workgroups of four waves and 128 rows, two on a CU, which fill each other's waits; of
// eight waves and 256 rows (a key tile is copied half as often) where heads are 128 long,
// a row sees some 6000 keys and there are rows for all CUs. 40 heads of 128, four waves
// against eight: 2048 x 2048 93 and 108 us, 4096 x 4096 304 and 318, 8192 x 8192 1173 and
// 1127, 32760 x 32760 18.6 and 18.0 ms; 8 + 40 heads, 16 x 32000 30 and 41 us. 64 heads of 64,
// 16384 x 16384: 4.39 and 4.59 ms (the exponentials bound it).
static int attention_waves(const mxq_attention_args& g) {
  return g.head_dim == 128 && attention_keys(g) >= 6144 && g.Mq * g.heads >= 256 * 256 ? 8 : 4;
}

static int64_t attention_slots(const mxq_attention_args& g) {
  return g.Mq * (g.heads / g.kv_heads) / (32 * attention_waves(g)) + g.sequences;
}

// Parts of the keys, so that few rows fill the chip: a workgroup for each CU, or two where
// one each would leave many CUs idle; two tiles a part at least; and no more than pays for
// writing and joining the parts (some 1.2 us for each MB of a part, against 0.8 us a tile).
// Keys in n parts, us: 16 x 8000, 40 + 8 heads of 128 n = 8, 16, 23 (taken), 48: 22.4, 17.1,
// 16.6, 20.4; 37 x 30011, 64 + 8 heads of 64 n = 10, 21 (taken), 32: 39.8, 37.3, 39.7;
// 100 x 4000, 40 + 40 of 128 n = 3, 6 (taken), 8, 16: 29.8, 25.5, 29.3, 36.4; 1000 x 1000,
// 16 + 8 of 128 n = 1 (taken), 2, 4: 18.1, 22.5, 25.2.
// The sequences' average length decides, and every sequence gets the same number: right for
// lengths that are alike (64 sequences of 4 x 2547, 40 + 8 heads of 128, 160 us), not for one
// long axis among many short ones, which one workgroup per key head and tile of rows then
// walks: 4 x 100000 alone 87 us, among 63 of 4 x 1000 1770 us.
static int attention_splits(const mxq_attention_args& g) {
  const int64_t items = attention_slots(g) * g.kv_heads;
  if (items == 0) return 1;
  int64_t s = 256 / items;
  if (512 / items > 2 * s) s = 512 / items;
  const int64_t tiles = (attention_keys(g) + kKeys - 1) / kKeys;
  if (s > tiles / 2) s = tiles / 2;
  if (s > 64) s = 64;
  const int64_t part = g.Mq * g.heads * (g.head_dim + 2) * 4;
  while (s > 1 && s * s * part > tiles * 1500000) --s;
  return s < 2 ? 1 : (int)s;
}

size_t attention_workspace(const mxq_attention_args& g) {
  const int splits = attention_splits(g);
  return splits < 2 ? 0 : (size_t)splits * g.Mq * g.heads * (g.head_dim + 2) * 4;
}

bool attention_fits(const mxq_attention_args& g) {
  return g.Mq * (g.heads / g.kv_heads) < (int64_t(1) << 31) - 256 &&
         (attention_slots(g) * g.kv_heads * attention_splits(g) + 8) * 64 * attention_waves(g) < (int64_t(1) << 32);
}

template <int D, int NW>
static hipError_t launch(const AttnArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((attention_kernel<D, NW>), dim3((unsigned)((a.items + 7) / 8 * 8)), dim3(64 * NW), 4 * kKeys * D * 2, s, a);
  if (a.splits > 1) {
    const int64_t rows = (int64_t)a.Mq * a.kv_heads * a.group, per = 256 / (D / 4) / kJoin;
    hipLaunchKernelGGL((attention_join_kernel<D>), dim3((unsigned)((rows + per - 1) / per)), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

hipError_t launch_attention(const mxq_attention_args& g, void* workspace, hipStream_t s) {
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
  // (a limit that no position reaches is none)
  a.left = g.left < 0 || g.left >= g.Mk ? -1 : (int)g.left;
  a.right = g.right < 0 || g.right >= g.Mq ? -1 : (int)g.right;
  a.sinks = (int)(g.sinks < g.Mk ? g.sinks : g.Mk);
  a.kv_heads = g.kv_heads; a.group = g.heads / g.kv_heads;
  a.slots = (int)attention_slots(g);
  a.splits = attention_splits(g);
  a.items = a.slots * a.kv_heads * a.splits;
  a.by_group = divider(a.group);
  a.by_slots = divider(a.slots);
  a.by_splits = divider(a.splits);
  a.scale_log2 = g.scale * 1.4426950408889634f;
  // Scores up to a factor 2^3 above the running maximum leave it where it is: raising it costs
  // a pass over the sums, and the fp32 sums have room for that and more. A row's largest weight
  // is exact in bf16 only where it is 1, so more slack costs accuracy where few keys carry the
  // row. Factors 2^0, 2^3, 2^8: 32760 x 32760 18.0, 17.5, 17.3 ms with a relative error of
  // .0022, .0024, .0025; 65520 queries of two sequences against 741 keys 700, 693, 678 us
  // with .0019, .0022, .0025.
  // (finite, for scales near 0: -infinity of a row that has seen nothing and an infinite slack
  // would be NaN, which no score exceeds)
  a.slack = fminf(3.0f / a.scale_log2, 3.4e38f);
  if (g.head_dim == 64) return launch<64, 4>(a, s);
  return attention_waves(g) == 8 ? launch<128, 8>(a, s) : launch<128, 4>(a, s);
}

}  // namespace mxq
