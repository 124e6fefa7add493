// mxq_pages.hip - pages, slots and positions of a step's new tokens
// (mxq_page_plan).
//
// One launch, no atomics and no wait between workgroups: every workgroup forms
// the two running sums over the requests (new tokens, new pages) in its LDS for
// itself, 8 bytes a request from the L2, and then places its own tokens. A
// token's request is found by bisection in LDS. A new page begins at a multiple
// of the page size that is not cached yet, so the token at that position writes
// the page into the block table: no other place of the table is written, and the
// one old entry that tokens read (a request's last page, where it is not full) is
// not. Of tokens that are not listed only the pages matter: those are gone through
// page by page (2 requests of 4 million tokens each, none listed, tables of 4: 7.0 ms
// token by token, 3.3 us so).
//
// Bound by latency: two dependent loads and the sums, about 8 bytes a token
// otherwise. A token a thread, so that the loads of a step of one token per
// request are all under way together: 64 requests with a token each 3.5 us (5.0 with
// four tokens a thread and a scan for each sum), 1000 requests with 200003 tokens 8.0
// us (10.1); called back to back 11 us each, the host's part.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq_attention.h"
#include "mxq_internal.h"

namespace mxq {

constexpr int kPlanThreads = 256;

struct PlanArgs {
  const int32_t* cached;
  const int32_t* added;
  int32_t* table;
  const int32_t* free_pages;
  int32_t* slots;
  int32_t* positions;
  int32_t* starts;
  int32_t* lengths;
  int32_t* taken;
  int64_t tokens, n_free, width;
  int requests, shift;
};

__device__ __forceinline__ int64_t plan_pages(int64_t n, int shift, int64_t width) {
  const int64_t p = (n + (int64_t(1) << shift) - 1) >> shift;
  return p < width ? p : width;
}

// Inclusive sums of two numbers over the workgroup, and their totals.
__device__ __forceinline__ void block_scan2(int& a, int& b, int (&waves)[kPlanThreads / 64][2], int& all_a, int& all_b) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int ua = __shfl_up(a, off), ub = __shfl_up(b, off);
    if (lane >= off) {
      a += ua;
      b += ub;
    }
  }
  if (lane == 63) {
    waves[wave][0] = a;
    waves[wave][1] = b;
  }
  __syncthreads();
  all_a = all_b = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    a += w < wave ? waves[w][0] : 0;
    b += w < wave ? waves[w][1] : 0;
    all_a += waves[w][0];
    all_b += waves[w][1];
  }
}

// The last of `count` requests whose running sum is at most x (sums[0] = 0).
__device__ __forceinline__ int last_request(const int* sums, int count, int64_t x) {
  int lo = 0, hi = count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ __launch_bounds__(kPlanThreads) void page_plan_kernel(const PlanArgs a) {
  // per request: first token (and the end), first new page, tokens in the cache
  extern __shared__ int sums[];
  __shared__ int waves[kPlanThreads / 64][2];
  int* const first = sums;
  int* const base = first + a.requests + 1;
  int* const cache = base + a.requests;
  const int tid = threadIdx.x;
  const int64_t page = int64_t(1) << a.shift;

  // a run of requests per thread
  const int per = (a.requests + kPlanThreads - 1) / kPlanThreads;
  const int r_begin = min(tid * per, a.requests), r_end = min(r_begin + per, a.requests);
  int tokens = 0, pages = 0;
  for (int r = r_begin; r < r_end; ++r) {
    const int c = max(a.cached[r], 0), n = max(a.added[r], 0);
    first[r] = n;
    cache[r] = c;
    tokens += n;
    pages += (int)(plan_pages((int64_t)c + n, a.shift, a.width) - plan_pages(c, a.shift, a.width));
  }
  int t = tokens, p = pages, all_tokens, all_pages;
  block_scan2(t, p, waves, all_tokens, all_pages);
  t -= tokens;
  p -= pages;
  for (int r = r_begin; r < r_end; ++r) {
    const int c = cache[r], n = first[r];
    first[r] = t;
    base[r] = p;
    t += n;
    p += (int)(plan_pages((int64_t)c + n, a.shift, a.width) - plan_pages(c, a.shift, a.width));
  }
  if (tid == 0) first[a.requests] = all_tokens;
  __syncthreads();

  const int64_t live = all_tokens, step = (int64_t)gridDim.x * kPlanThreads, begin = (int64_t)blockIdx.x * kPlanThreads + tid;
  auto free_page = [&](int64_t k) { return k >= 0 && k < a.n_free ? a.free_pages[k] : -1; };  // (k < 0: sums past 32 bits)
  for (int64_t at = begin; at < a.tokens; at += step) {
    int slot = -1, pos = 0;
    if (at < live) {
      const int r = last_request(first, a.requests, at);
      const int64_t c = cache[r], q = c + (at - first[r]), col = q >> a.shift, have = plan_pages(c, a.shift, a.width);
      pos = (int)q;
      if (col < a.width) {
        int id;
        if (col < have) {
          id = a.table[(int64_t)r * a.width + col];
        } else {
          id = free_page(base[r] + (col - have));
          if ((q & (page - 1)) == 0) a.table[(int64_t)r * a.width + col] = id;
        }
        if (id >= 0) slot = (int)(((int64_t)id << a.shift) + (q & (page - 1)));
      }
    }
    a.slots[at] = slot;
    a.positions[at] = pos;
  }
  if (live > a.tokens)  // new pages whose first token is not listed
    for (int64_t k = begin; k < all_pages; k += step) {
      const int r = last_request(base, a.requests, k);
      const int64_t c = cache[r], col = plan_pages(c, a.shift, a.width) + (k - base[r]);
      if (col < a.width && first[r] + ((col << a.shift) - c) >= a.tokens) a.table[(int64_t)r * a.width + col] = free_page(k);
    }

  if (blockIdx.x != 0) return;
  int unplaced = 0;
  for (int r = tid; r < a.requests; r += kPlanThreads) {
    const int64_t c = cache[r], n = first[r + 1] - first[r], have = plan_pages(c, a.shift, a.width);
    const int64_t need = plan_pages(c + n, a.shift, a.width) - have;
    a.starts[r] = first[r];
    a.lengths[r] = (int)(c + n);
    // tokens on an old page that the table lacks, and those behind the last page it gets
    const int64_t got = max((int64_t)0, min(need, a.n_free - base[r]));
    const int64_t old_end = min(c + n, have << a.shift), last = (have + got) << a.shift;
    if (old_end > c && a.table[(int64_t)r * a.width + have - 1] < 0) unplaced += (int)(old_end - c);
    unplaced += (int)max((int64_t)0, c + n - max(c, last));
  }
  __syncthreads();
  int none = 0, all = 0, zero = 0;
  block_scan2(unplaced, none, waves, all, zero);
  if (tid == 0) {
    a.starts[a.requests] = all_tokens;
    a.taken[0] = (int)min((int64_t)all_pages, a.n_free);
    a.taken[1] = all;
  }
}

hipError_t launch_page_plan(const int32_t* cached, const int32_t* added, int32_t* block_table, const int32_t* free_pages,
                            int64_t requests, int64_t width, int64_t n_free, int64_t page_size, int64_t tokens,
                            int32_t* slots, int32_t* positions, int32_t* starts, int32_t* lengths, int32_t* taken,
                            hipStream_t s) {
  const PlanArgs a{cached, added, block_table, free_pages, slots, positions, starts, lengths, taken, tokens, n_free, width,
                   (int)requests, __builtin_ctzll((unsigned long long)page_size)};
  const int64_t want = (tokens + kPlanThreads - 1) / kPlanThreads;
  const unsigned grid = (unsigned)(want < 1 ? 1 : want > 1024 ? 1024 : want);
  hipLaunchKernelGGL(page_plan_kernel, dim3(grid), dim3(kPlanThreads), (size_t)(3 * requests + 1) * 4, s, a);
  return hipGetLastError();
}

}  // namespace mxq
