/*
 * mxq_attention.h - C ABI of libmxq, the attention half of a transformer
 * block: what a block computes between its stacked q/k/v projection
 * (mxq_gemm) and its output projection (mxq_quantize_act, mxq_gemm_residual).
 *
 *   mxq_page_plan        pages, slots and positions of a step's new tokens in a
 *                        paged key-value cache, from the requests' lengths
 *   mxq_rotary_qkv       RMS norm of q and k, rotary positions of one or several
 *                        axes, k and v into the cache
 *   mxq_attention        ragged sequences of tokens, grouped heads, sliding
 *                        windows and sinks
 *   mxq_attention_paged  one new token per sequence against a paged cache
 *
 * Status codes and the conventions of every entry point (pointers, streams,
 * validation before anything is enqueued, empty problems, alignment) are those
 * of mxq.h. No call allocates or synchronizes, every call can be captured into
 * a graph, calls may overlap on one device (each with a workspace of its own),
 * and results do not depend on the schedule (no atomics). int32 vectors need 4-
 * byte alignment, float64 ones 8, all others 16.
 *
 * What a call reads on the device (lengths, starts, tables, slots, positions,
 * axes) cannot be checked by the host: the kernels bound every index by the
 * sizes of the call, so that wrong values give wrong results and never an
 * access outside the buffers.
 *
 * MXQ_CHECK_FINITE: mxq_rotary_qkv scans qkv and the norm weights before
 * anything is written, and q and k after it; the attention calls scan the rows
 * of q, k and v that belong to sequences, and the same rows of the output. A
 * cache is not scanned: its free pages may hold anything. The scans synchronize
 * the stream and cannot be captured.
 */
#ifndef MXQ_ATTENTION_H
#define MXQ_ATTENTION_H

#include "mxq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most requests of mxq_page_plan and sequences of mxq_attention_paged (their
 * running sums stay in one workgroup's memory). */
#define MXQ_MAX_REQUESTS 4096

/* Formats of a key-value cache. MXQ_KV_MXFP8: OCP MX blocks of 32 elements along
 * a head, E4M3 elements and one E8M0 scale 2^(floor(log2 amax) - 8), rounded to
 * nearest even and saturating at 448 (as the MXFP4 of mxq.h with wider elements).
 * A NaN stays one (code 0x7F or 0xFF) and an infinity reads as one, but the finite
 * values of their block are lost to its scale. */
enum { MXQ_KV_BF16 = 0, MXQ_KV_MXFP8 = 1 };

/* RMS norms of q and k: none, over all heads of a row, or per head. */
enum { MXQ_ROTARY_NORM_NONE = 0, MXQ_ROTARY_NORM_ROW = 1, MXQ_ROTARY_NORM_HEAD = 2 };

/*
 * A paged key-value cache.
 *   k, v       device, [pages][kv_heads][page_size][head_dim]: bf16, or E4M3 codes
 *   k_scales,
 *   v_scales   device uint8 [pages][kv_heads][page_size][head_dim / 32], null for
 *              bf16
 *   page_size  a power of two, 16 to 1024; pages * page_size < 2^31
 *   head_dim   64 or 128
 * Slot s of the cache is token s % page_size of page s / page_size.
 */
typedef struct mxq_kv_cache {
  void* k;
  void* v;
  void* k_scales;
  void* v_scales;
  int64_t pages, page_size;
  int32_t kv_heads, head_dim, format;
} mxq_kv_cache;

/*
 * mxq_page_plan: request b has cached[b] tokens in the cache and gets added[b]
 * more. With P = page_size, W = width and pages(n) = min(ceil(n / P), W) it needs
 * pages(cached + added) - pages(cached) new pages, taken from free_pages in the
 * order of the requests, and
 *   block_table[b][pages(cached) + j] = its j-th new page, -1 when the list is
 *                                       used up (other entries stay)
 *   starts[b]    = added[0] + .. + added[b - 1]   (starts[requests]: all of them)
 *   lengths[b]   = cached[b] + added[b]
 *   positions[t] = cached[b] + t - starts[b] for the tokens t of request b
 *   slots[t]     = page of that position * P + position % P, -1 where the table
 *                  has no page for it
 *   taken[0], taken[1] = pages taken from the list, new tokens without a page
 * Entries of slots and positions behind the last token are -1 and 0; tokens past
 * `tokens` are not listed.
 *   cached, added  device int32 [requests], below 2^30, their sum over all requests
 *                  below 2^31 (negative ones count as 0)
 *   block_table    device int32 [requests][width] (in and out)
 *   free_pages     device int32 [n_free]
 *   slots, positions, starts, lengths, taken   device int32 [tokens], [tokens],
 *                  [requests + 1], [requests], [2] (outputs, apart from each
 *                  other and the inputs)
 */
int mxq_page_plan(const int32_t* cached, const int32_t* added, int32_t* block_table, const int32_t* free_pages,
                  int64_t requests, int64_t width, int64_t n_free, int64_t page_size, int64_t tokens, int32_t* slots,
                  int32_t* positions, int32_t* starts, int32_t* lengths, int32_t* taken, hipStream_t stream);

/*
 * mxq_rotary_qkv: row m of qkv holds heads of q, kv_heads of k and kv_heads of v,
 * head_dim elements each. In fp32, for the heads of q and k:
 *   n = x / sqrt(mean x^2 + eps) * weight      (norm; mean over the row's heads
 *                                               or over the head; n = x without)
 *   pair p of a head, (a, b) = (n[2p], n[2p + 1]) interleaved, (n[p], n[p + pairs])
 *   else, turned by the angle t = positions[axis[p]][m] * freqs[p]:
 *   (a cos t - b sin t, a sin t + b cos t)
 * and one rounding to bf16. Values whose squares sum past fp32's range (|x| about
 * 1e18) are not finite inputs of a norm: the row's q or k, or the head, is NaN,
 * which MXQ_CHECK_FINITE reports. The elements behind the 2 * pairs turned ones, and
 * pairs whose axis is not in 0 .. axes - 1, are only normed. The angle is formed
 * and reduced in 64 bits. v is only copied into the cache.
 *   qkv        device bf16 [M][ldx]
 *   positions  device int32 [axes][ld_pos]
 *   freqs      device float64 [pairs], radians per position; |t| below 2^40
 *   axis       device int32 [pairs], null for axis 0 throughout
 *   pairs      a multiple of 8, at most head_dim / 2; 0 for no rotation (positions,
 *              freqs and axis are then not read)
 *   q_weight, k_weight  device bf16 [heads * head_dim], [kv_heads * head_dim] (row
 *              norm) or [head_dim] (head norm), null for ones; null without a norm
 *   eps        at least 2^-126 and finite with a norm
 *   q          device bf16 [M][ldq] (output), null where heads is 0
 *   k          device bf16 [M][ldk] (output) or null
 *   cache      null for none; else k (after norm and rotation, of its bf16 values)
 *              and v go to slots[m], device int32 [M]; rows whose slot is outside
 *              the cache are not written. Two rows of one slot leave it undefined.
 * q may be the q part of qkv itself and k the k part (same address and stride);
 * else outputs may not overlap an input or each other. heads and kv_heads may be 0,
 * not both; (heads + 2 kv_heads) * head_dim at most 65536, head_dim 64 or 128.
 */
typedef struct mxq_rotary_args {
  const void* qkv;
  const int32_t* positions;
  const double* freqs;
  const int32_t* axis;
  const void* q_weight;
  const void* k_weight;
  void* q;
  void* k;
  const int32_t* slots;
  int64_t M, ldx, ldq, ldk, ld_pos;
  int32_t heads, kv_heads, head_dim, axes, pairs, interleaved, norm;
  float eps;
} mxq_rotary_args;
int mxq_rotary_qkv(const mxq_rotary_args* args, const mxq_kv_cache* cache, hipStream_t stream);

/*
 * mxq_attention: sequence b has the rows starts_q[b] .. starts_q[b + 1] - 1 of q
 * and out and starts_k[b] .. of k and v; its n_q queries are the last of its n_k
 * positions: query i is at p = n_k - n_q + i and sees the keys
 *   { j : 0 <= j < n_k, j <= p + right, j >= p - left or j < sinks }
 * (left, right < 0: unlimited; right = 0: causal). Query head h reads key head
 * h / (heads / kv_heads), and
 *   out_i = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q_i . k_j)
 * over the visible keys, in fp32 from fp32 scores; the w_j enter the product with
 * v as bf16 values (relative to the largest one of the keys seen so far), and out
 * is rounded to bf16 once. A row without visible keys is zeros, and so is one whose
 * scores are all -infinity. A row whose largest score (scale q . k) is past 7e8 in
 * magnitude, where fp32 holds no exponents any more, is NaN, and sums of weighted
 * values past fp32's range are infinities or NaN: MXQ_CHECK_FINITE reports all. Keys and
 * values at places that a query does not see may
 * hold anything. Rows of out behind the last sequence are left as they were.
 *   q, out     device bf16 [Mq][ldq], [Mq][ldo], heads * head_dim elements a row
 *   k, v       device bf16 [Mk][ldk], [Mk][ldv], kv_heads * head_dim elements a row
 *   starts_q, starts_k  device int32 [sequences + 1], not decreasing, or both null
 *              for one sequence of all rows
 *   scale      positive, below 2^127
 * out may not overlap an input or the workspace. head_dim 64 or 128; heads a multiple of kv_heads; Mq, Mk below 2^29, and
 * Mq * heads / kv_heads below 2^31 - 256.
 * The workspace (mxq_attention_workspace_bytes; 0: it may be null) joins the parts
 * of a long axis when there are few rows. It belongs to the call until its work is
 * done.
 */
typedef struct mxq_attention_args {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* starts_q;
  const int32_t* starts_k;
  void* out;
  int64_t sequences, Mq, Mk;
  int64_t ldq, ldk, ldv, ldo;
  int64_t left, right, sinks;
  int32_t heads, kv_heads, head_dim;
  float scale;
} mxq_attention_args;
int mxq_attention_workspace_bytes(const mxq_attention_args* args, size_t* bytes);
int mxq_attention(const mxq_attention_args* args, void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * mxq_attention_paged: one query per sequence, at position lengths[b] - 1, against
 * the lengths[b] tokens that the pages of block_table[b] hold in order:
 *   { j : 0 <= j < lengths[b], j >= lengths[b] - 1 - left or j < sinks }
 * as above otherwise. Keys on a page outside the cache (a table entry of -1) and
 * keys behind the table are not visible; a length of 0 gives zeros. MXFP8 keys and
 * values count as the bf16 numbers that they stand for.
 *   q, out       device bf16 [sequences][ldq], [sequences][ldo]
 *   block_table  device int32 [sequences][width]
 *   lengths      device int32 [sequences], at most 2^30
 *   scale        positive, below 2^127
 * out may not overlap an input, the cache or the workspace.
 * sequences * width * page_size below 2^34; heads a multiple of kv_heads.
 * The cache is split over workgroups by what the lengths say on the device; the
 * workspace (mxq_attention_paged_workspace_bytes) joins the parts.
 */
typedef struct mxq_paged_args {
  const void* q;
  const int32_t* block_table;
  const int32_t* lengths;
  void* out;
  int64_t sequences, width;
  int64_t ldq, ldo;
  int64_t left, sinks;
  int32_t heads;
  float scale;
} mxq_paged_args;
int mxq_attention_paged_workspace_bytes(const mxq_paged_args* args, const mxq_kv_cache* cache, size_t* bytes);
int mxq_attention_paged(const mxq_paged_args* args, const mxq_kv_cache* cache, void* workspace, size_t workspace_bytes,
                        hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_ATTENTION_H */
