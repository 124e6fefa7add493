// mxq_attention_api.cpp - the extern "C" boundary of the attention half of a
// block (declared in include/mxq_attention.h): validation on the host, before
// anything is enqueued, then dispatch to the gfx950 kernels.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <utility>

#include "mxq_attention.h"
#include "mxq_host.h"
#include "mxq_internal.h"

using namespace mxq;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxLd = int64_t(1) << 24;  // row strides, in elements
constexpr int kMaxHeads = 1024;

bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

int check_heads(int heads, int kv_heads) {
  if (heads <= 0 || kv_heads <= 0 || heads > kMaxHeads || heads % kv_heads != 0) return MXQ_ERR_SHAPE;
  return MXQ_OK;
}

bool head_dim_ok(int d) { return d == 64 || d == 128; }

bool page_size_ok(int64_t p) { return p >= 16 && p <= 1024 && (p & (p - 1)) == 0; }

// Everything about a cache but its addresses.
int check_cache_shape(const mxq_kv_cache& c) {
  if (c.format != MXQ_KV_BF16 && c.format != MXQ_KV_MXFP8) return MXQ_ERR_MODE;
  if (!head_dim_ok(c.head_dim) || c.kv_heads <= 0 || c.kv_heads > kMaxHeads || !page_size_ok(c.page_size)) return MXQ_ERR_SHAPE;
  if (c.pages <= 0 || c.pages > ((int64_t(1) << 31) - 1) / c.page_size) return MXQ_ERR_SHAPE;
  return MXQ_OK;
}

int check_cache_memory(const mxq_kv_cache& c) {
  if (c.k == nullptr || c.v == nullptr) return MXQ_ERR_NULL;
  if (c.format == MXQ_KV_MXFP8 && (c.k_scales == nullptr || c.v_scales == nullptr)) return MXQ_ERR_NULL;
  if (c.format == MXQ_KV_BF16 && (c.k_scales != nullptr || c.v_scales != nullptr)) return MXQ_ERR_MODE;
  for (const void* p : {c.k, c.v, c.k_scales, c.v_scales})
    if (!aligned16(p)) return MXQ_ERR_ALIGN;
  return MXQ_OK;
}

int check_ld(int64_t ld, int64_t width) {
  if (ld < width || ld > kMaxLd) return MXQ_ERR_SHAPE;
  return MXQ_OK;
}

bool positive(float v) { return v > 0.0f && isfinite(v); }
// (the kernels take scores in units of log2, scale / ln 2)
bool score_scale(float v) { return positive(v) && v < 0x1p127f; }

// MXQ_CHECK_FINITE on the rows of [rows][ld] that sequences own.
int owned_guard(const char* what, const void* x, const int32_t* starts, int64_t sequences, int64_t rows, int64_t cols, int64_t ld,
                hipStream_t stream) {
  if (!check_finite_enabled() || rows == 0) return MXQ_OK;
  int32_t ends[2] = {0, (int32_t)rows};
  if (starts != nullptr) {
    if (hipMemcpyAsync(&ends[0], starts, 4, hipMemcpyDeviceToHost, stream) != hipSuccess ||
        hipMemcpyAsync(&ends[1], starts + sequences, 4, hipMemcpyDeviceToHost, stream) != hipSuccess ||
        hipStreamSynchronize(stream) != hipSuccess)
      return MXQ_ERR_HIP;
  }
  const int64_t begin = ends[0] < 0 ? 0 : ends[0], end = ends[1] < rows ? ends[1] : rows;
  if (begin >= end) return MXQ_OK;
  return finite_guard(what, static_cast<const uint16_t*>(x) + begin * ld, end - begin, cols, ld, stream);
}

int check_attention(const mxq_attention_args* args) {
  if (args == nullptr) return MXQ_ERR_NULL;
  const mxq_attention_args& a = *args;
  int st = check_heads(a.heads, a.kv_heads);
  if (st != MXQ_OK) return st;
  if (!score_scale(a.scale)) return MXQ_ERR_MODE;
  if (!head_dim_ok(a.head_dim) || a.Mq < 0 || a.Mk < 0 || a.Mq >= kMaxRows / 2 || a.Mk >= kMaxRows / 2) return MXQ_ERR_SHAPE;
  if (a.sequences < 0 || a.sequences >= kMaxRows || a.sinks < 0) return MXQ_ERR_SHAPE;
  if ((a.starts_q == nullptr || a.starts_k == nullptr) && a.sequences != 1) return MXQ_ERR_SHAPE;
  const int64_t wq = (int64_t)a.heads * a.head_dim, wk = (int64_t)a.kv_heads * a.head_dim;
  for (const auto& [ld, width] : {std::pair{a.ldq, wq}, std::pair{a.ldo, wq}, std::pair{a.ldk, wk}, std::pair{a.ldv, wk}})
    if ((st = check_ld(ld, width)) != MXQ_OK) return st;
  if (!attention_fits(a)) return MXQ_ERR_SHAPE;
  return MXQ_OK;
}

int check_paged(const mxq_paged_args* args, const mxq_kv_cache* cache) {
  if (args == nullptr || cache == nullptr) return MXQ_ERR_NULL;
  const mxq_paged_args& a = *args;
  int st = check_cache_shape(*cache);
  if (st != MXQ_OK || (st = check_heads(a.heads, cache->kv_heads)) != MXQ_OK) return st;
  if (!score_scale(a.scale)) return MXQ_ERR_MODE;
  if (a.sequences < 0 || a.sequences > MXQ_MAX_REQUESTS || a.width <= 0 || a.width >= kMaxRows || a.sinks < 0) return MXQ_ERR_SHAPE;
  if (a.sequences * a.width >= (int64_t(1) << 34) / cache->page_size) return MXQ_ERR_SHAPE;
  const int64_t wq = (int64_t)a.heads * cache->head_dim;
  for (int64_t ld : {a.ldq, a.ldo})
    if ((st = check_ld(ld, wq)) != MXQ_OK) return st;
  return MXQ_OK;
}

}  // namespace

extern "C" {

int mxq_page_plan(const int32_t* cached, const int32_t* added, int32_t* block_table, const int32_t* free_pages,
                  int64_t requests, int64_t width, int64_t n_free, int64_t page_size, int64_t tokens, int32_t* slots,
                  int32_t* positions, int32_t* starts, int32_t* lengths, int32_t* taken, hipStream_t stream) {
  if (!page_size_ok(page_size)) return MXQ_ERR_SHAPE;
  if (requests < 0 || requests > MXQ_MAX_REQUESTS || width <= 0 || width >= kMaxRows || n_free < 0 || n_free >= kMaxDim ||
      tokens < 0 || tokens >= kMaxRows)
    return MXQ_ERR_SHAPE;
  if (starts == nullptr || taken == nullptr) return MXQ_ERR_NULL;
  if (requests > 0 && (cached == nullptr || added == nullptr || block_table == nullptr || lengths == nullptr)) return MXQ_ERR_NULL;
  if ((n_free > 0 && free_pages == nullptr) || (tokens > 0 && (slots == nullptr || positions == nullptr))) return MXQ_ERR_NULL;
  for (const void* p : {(const void*)cached, (const void*)added, (const void*)block_table, (const void*)free_pages,
                        (const void*)slots, (const void*)positions, (const void*)starts, (const void*)lengths, (const void*)taken})
    if (!aligned(p, 4)) return MXQ_ERR_ALIGN;
  if (log_enabled())
    fprintf(stderr, "[mxq] page_plan requests=%lld width=%lld page=%lld tokens=%lld\n", (long long)requests, (long long)width,
            (long long)page_size, (long long)tokens);
  return hip_status(launch_page_plan(cached, added, block_table, free_pages, requests, width, n_free, page_size, tokens, slots,
                                     positions, starts, lengths, taken, stream));
}

int mxq_rotary_qkv(const mxq_rotary_args* args, const mxq_kv_cache* cache, hipStream_t stream) {
  if (args == nullptr) return MXQ_ERR_NULL;
  const mxq_rotary_args& a = *args;
  int st;
  if (a.norm != MXQ_ROTARY_NORM_NONE && a.norm != MXQ_ROTARY_NORM_ROW && a.norm != MXQ_ROTARY_NORM_HEAD) return MXQ_ERR_MODE;
  // (the kernel's reciprocal square root takes normal numbers)
  if (a.norm != MXQ_ROTARY_NORM_NONE && !(a.eps >= 0x1p-126f && isfinite(a.eps))) return MXQ_ERR_MODE;
  if (a.norm == MXQ_ROTARY_NORM_NONE && (a.q_weight != nullptr || a.k_weight != nullptr)) return MXQ_ERR_MODE;
  if (a.interleaved != 0 && a.interleaved != 1) return MXQ_ERR_MODE;
  if (!head_dim_ok(a.head_dim) || a.heads < 0 || a.kv_heads < 0 || a.heads > kMaxHeads || a.kv_heads > kMaxHeads) return MXQ_ERR_SHAPE;
  if (a.heads == 0 && a.kv_heads == 0) return MXQ_ERR_SHAPE;
  const int64_t width = (a.heads + 2 * (int64_t)a.kv_heads) * a.head_dim;
  if (width > 65536 || a.M < 0 || a.M >= kMaxRows || (st = check_ld(a.ldx, width)) != MXQ_OK) return MXQ_ERR_SHAPE;
  if (a.pairs < 0 || a.pairs % 8 != 0 || a.pairs > a.head_dim / 2) return MXQ_ERR_SHAPE;
  if (a.pairs > 0 && (a.axes < 1 || a.ld_pos < a.M || a.ld_pos >= kMaxDim)) return MXQ_ERR_SHAPE;
  if (a.q != nullptr && (st = check_ld(a.ldq, (int64_t)a.heads * a.head_dim)) != MXQ_OK) return st;
  if (a.k != nullptr && (st = check_ld(a.ldk, (int64_t)a.kv_heads * a.head_dim)) != MXQ_OK) return st;
  if (cache != nullptr) {
    if ((st = check_cache_shape(*cache)) != MXQ_OK) return st;
    if (cache->kv_heads != a.kv_heads || cache->head_dim != a.head_dim) return MXQ_ERR_SHAPE;
  }
  if (a.M == 0) return MXQ_OK;
  if (a.qkv == nullptr || (a.heads > 0 && a.q == nullptr) || (a.kv_heads > 0 && a.k == nullptr && cache == nullptr)) return MXQ_ERR_NULL;
  if (a.pairs > 0 && (a.positions == nullptr || a.freqs == nullptr)) return MXQ_ERR_NULL;
  if ((cache != nullptr) != (a.slots != nullptr)) return MXQ_ERR_NULL;
  // outputs of heads that the row does not have
  if ((a.heads == 0 && a.q != nullptr) || (a.kv_heads == 0 && a.k != nullptr)) return MXQ_ERR_MODE;
  if (cache != nullptr && (st = check_cache_memory(*cache)) != MXQ_OK) return st;
  for (const void* p : {a.qkv, a.q_weight, a.k_weight, (const void*)a.q, (const void*)a.k})
    if (!aligned16(p)) return MXQ_ERR_ALIGN;
  if (!aligned(a.positions, 4) || !aligned(a.axis, 4) || !aligned(a.slots, 4) || !aligned(a.freqs, 8)) return MXQ_ERR_ALIGN;
  if (a.ldx % 8 != 0 || (a.q != nullptr && a.ldq % 8 != 0) || (a.k != nullptr && a.ldk % 8 != 0)) return MXQ_ERR_ALIGN;
  if (log_enabled())
    fprintf(stderr, "[mxq] rotary_qkv M=%lld heads=%d kv=%d d=%d norm=%d cache=%d\n", (long long)a.M, a.heads, a.kv_heads,
            a.head_dim, a.norm, cache == nullptr ? -1 : cache->format);
  if ((st = finite_guard("qkv", a.qkv, a.M, width, a.ldx, stream)) != MXQ_OK) return st;
  const struct { const char* what; const void* p; int heads; } weights[] = {{"q_weight", a.q_weight, a.heads},
                                                                           {"k_weight", a.k_weight, a.kv_heads}};
  for (const auto& w : weights) {
    const int64_t n = (int64_t)a.head_dim * (a.norm == MXQ_ROTARY_NORM_ROW ? w.heads : 1);
    if (w.p != nullptr && w.heads > 0 && (st = finite_guard(w.what, w.p, 1, n, n, stream)) != MXQ_OK) return st;
  }
  if ((st = hip_status(launch_rotary_qkv(a, cache, stream))) != MXQ_OK) return st;
  if (a.q != nullptr && (st = finite_guard("q", a.q, a.M, (int64_t)a.heads * a.head_dim, a.ldq, stream)) != MXQ_OK) return st;
  if (a.k != nullptr && (st = finite_guard("k", a.k, a.M, (int64_t)a.kv_heads * a.head_dim, a.ldk, stream)) != MXQ_OK) return st;
  return MXQ_OK;
}

int mxq_attention_workspace_bytes(const mxq_attention_args* args, size_t* bytes) {
  if (bytes == nullptr) return MXQ_ERR_NULL;
  const int st = check_attention(args);
  if (st != MXQ_OK) return st;
  *bytes = attention_workspace(*args);
  return MXQ_OK;
}

int mxq_attention(const mxq_attention_args* args, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int st = check_attention(args);
  if (st != MXQ_OK) return st;
  const mxq_attention_args& a = *args;
  if (a.Mq == 0 || a.sequences == 0) return MXQ_OK;
  if (a.q == nullptr || a.out == nullptr || (a.Mk > 0 && (a.k == nullptr || a.v == nullptr))) return MXQ_ERR_NULL;
  if ((a.starts_q == nullptr) != (a.starts_k == nullptr)) return MXQ_ERR_NULL;
  for (const void* p : {a.q, a.k, a.v, (const void*)a.out, (const void*)workspace})
    if (!aligned16(p)) return MXQ_ERR_ALIGN;
  if (!aligned(a.starts_q, 4) || !aligned(a.starts_k, 4)) return MXQ_ERR_ALIGN;
  if (a.ldq % 8 != 0 || a.ldk % 8 != 0 || a.ldv % 8 != 0 || a.ldo % 8 != 0) return MXQ_ERR_ALIGN;
  const size_t need = attention_workspace(a);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return MXQ_ERR_WORKSPACE;
  if (log_enabled())
    fprintf(stderr, "[mxq] attention sequences=%lld Mq=%lld Mk=%lld heads=%d kv=%d d=%d left=%lld right=%lld sinks=%lld\n",
            (long long)a.sequences, (long long)a.Mq, (long long)a.Mk, a.heads, a.kv_heads, a.head_dim, (long long)a.left,
            (long long)a.right, (long long)a.sinks);
  const int64_t wq = (int64_t)a.heads * a.head_dim, wk = (int64_t)a.kv_heads * a.head_dim;
  if ((st = owned_guard("q", a.q, a.starts_q, a.sequences, a.Mq, wq, a.ldq, stream)) != MXQ_OK) return st;
  if ((st = owned_guard("k", a.k, a.starts_k, a.sequences, a.Mk, wk, a.ldk, stream)) != MXQ_OK) return st;
  if ((st = owned_guard("v", a.v, a.starts_k, a.sequences, a.Mk, wk, a.ldv, stream)) != MXQ_OK) return st;
  if ((st = hip_status(launch_attention(a, workspace, stream))) != MXQ_OK) return st;
  return owned_guard("attention output", a.out, a.starts_q, a.sequences, a.Mq, wq, a.ldo, stream);
}

int mxq_attention_paged_workspace_bytes(const mxq_paged_args* args, const mxq_kv_cache* cache, size_t* bytes) {
  if (bytes == nullptr) return MXQ_ERR_NULL;
  const int st = check_paged(args, cache);
  if (st != MXQ_OK) return st;
  *bytes = paged_workspace(*args, *cache);
  return MXQ_OK;
}

int mxq_attention_paged(const mxq_paged_args* args, const mxq_kv_cache* cache, void* workspace, size_t workspace_bytes,
                        hipStream_t stream) {
  int st = check_paged(args, cache);
  if (st != MXQ_OK) return st;
  const mxq_paged_args& a = *args;
  if (a.sequences == 0) return MXQ_OK;
  if (a.q == nullptr || a.out == nullptr || a.block_table == nullptr || a.lengths == nullptr) return MXQ_ERR_NULL;
  if ((st = check_cache_memory(*cache)) != MXQ_OK) return st;
  if (!aligned16(a.q) || !aligned16(a.out) || !aligned16(workspace) || !aligned(a.block_table, 4) || !aligned(a.lengths, 4))
    return MXQ_ERR_ALIGN;
  if (a.ldq % 8 != 0 || a.ldo % 8 != 0) return MXQ_ERR_ALIGN;
  const size_t need = paged_workspace(a, *cache);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return MXQ_ERR_WORKSPACE;
  if (log_enabled())
    fprintf(stderr, "[mxq] attention_paged sequences=%lld width=%lld heads=%d kv=%d d=%d format=%d left=%lld sinks=%lld\n",
            (long long)a.sequences, (long long)a.width, a.heads, cache->kv_heads, cache->head_dim, cache->format,
            (long long)a.left, (long long)a.sinks);
  const int64_t wq = (int64_t)a.heads * cache->head_dim;
  if ((st = finite_guard("q", a.q, a.sequences, wq, a.ldq, stream)) != MXQ_OK) return st;
  if ((st = hip_status(launch_attention_paged(a, *cache, workspace, stream))) != MXQ_OK) return st;
  return finite_guard("attention output", a.out, a.sequences, wq, a.ldo, stream);
}

}  // extern "C"
