// mxq_pages.hip - pages, slots and positions of a step's new tokens
// (mxq_page_plan).
//
// One launch, no atomics and no wait between workgroups: every workgroup forms
// the two running sums over the requests (new tokens, new pages) in its LDS for
// itself, 8 bytes a request from the L2, and then places its own tokens. A
// token's request is found by bisection in LDS; four consecutive tokens a thread
// share one search and their stores. A new page begins at a multiple of the page
// size that is not cached yet, so the token at that position writes the page
// into the block table: no other place of the table is written, and the one old
// entry that tokens read (a request's last page, where it is not full) is not.
//
// Bound by latency: three dependent loads and the sums, about 8 bytes a token
// otherwise.
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

// Inclusive sum over the workgroup; *total gets the last one.
__device__ __forceinline__ int block_scan(int v, int* waves, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int u = __shfl_up(v, off);
    if (lane >= off) v += u;
  }
  if (lane == 63) waves[wave] = v;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    before += w < wave ? waves[w] : 0;
    all += waves[w];
  }
  __syncthreads();
  *total = all;
  return v + before;
}

__global__ __launch_bounds__(kPlanThreads) void page_plan_kernel(const PlanArgs a) {
  extern __shared__ int sums[];  // starts [requests + 1], then first new page [requests]
  __shared__ int waves[kPlanThreads / 64];
  int* const first = sums;
  int* const base = sums + a.requests + 1;
  const int tid = threadIdx.x;
  const int64_t page = int64_t(1) << a.shift;

  int tokens_before = 0, pages_before = 0, unplaced = 0;
  for (int r0 = 0; r0 < a.requests; r0 += kPlanThreads) {
    const int r = r0 + tid;
    int c = 0, n = 0, have = 0, need = 0;
    if (r < a.requests) {
      c = max(a.cached[r], 0);
      n = max(a.added[r], 0);
      have = (int)plan_pages(c, a.shift, a.width);
      need = (int)(plan_pages((int64_t)c + n, a.shift, a.width) - have);
    }
    int all_tokens, all_pages;
    const int t = tokens_before + block_scan(n, waves, &all_tokens);
    const int p = pages_before + block_scan(need, waves, &all_pages);
    if (r < a.requests) {
      first[r + 1] = t;
      base[r] = p - need;
      if (blockIdx.x == 0) {
        a.starts[r + 1] = t;
        a.lengths[r] = c + n;
        // tokens on an old page that the table lacks, and those behind the last page it gets
        const int64_t got = max((int64_t)0, min((int64_t)need, a.n_free - (p - need)));
        const int64_t end = (have + got) << a.shift;
        const int64_t old_end = min((int64_t)c + n, (int64_t)have << a.shift);
        if (old_end > c && a.table[(int64_t)r * a.width + have - 1] < 0) unplaced += (int)(old_end - c);
        unplaced += (int)max((int64_t)0, (int64_t)c + n - max((int64_t)c, end));
      }
    }
    tokens_before += all_tokens;
    pages_before += all_pages;
  }
  if (tid == 0) first[0] = 0;
  if (blockIdx.x == 0) {
    int all;
    block_scan(unplaced, waves, &all);
    if (tid == 0) {
      a.starts[0] = 0;
      a.taken[0] = (int)min((int64_t)pages_before, a.n_free);
      a.taken[1] = all;
    }
  }
  __syncthreads();

  const int64_t live = tokens_before;
  const int64_t end = live > a.tokens ? live : a.tokens;
  for (int64_t t0 = 4 * ((int64_t)blockIdx.x * kPlanThreads + tid); t0 < end; t0 += 4 * (int64_t)gridDim.x * kPlanThreads) {
    int32_t slot[4], pos[4];
    int r = 0;
    if (t0 < live) {  // the last request that starts at or before t0
      int lo = 0, hi = a.requests;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= t0)
          lo = mid;
        else
          hi = mid;
      }
      r = lo;
    }
    int64_t c = -1, have = 0;
    int held = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = t0 + i;
      slot[i] = -1;
      pos[i] = 0;
      if (t >= live) continue;
      while (first[r + 1] <= t) {
        ++r;
        c = -1;
      }
      if (c < 0) {
        c = max(a.cached[r], 0);
        have = plan_pages(c, a.shift, a.width);
        held = (c & (page - 1)) != 0 && have > 0 ? a.table[(int64_t)r * a.width + have - 1] : -1;
      }
      const int64_t p = c + (t - first[r]);
      const int64_t col = p >> a.shift;
      pos[i] = (int32_t)p;
      if (col >= a.width) continue;
      int id = held;
      if (col >= have) {
        const int64_t k = base[r] + (col - have);
        id = k >= 0 && k < a.n_free ? a.free_pages[k] : -1;  // (k < 0: sums past 32 bits)
        if ((p & (page - 1)) == 0) a.table[(int64_t)r * a.width + col] = id;
      }
      if (id >= 0) slot[i] = (int32_t)(((int64_t)id << a.shift) + (p & (page - 1)));
    }
    if (t0 + 4 <= a.tokens && ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions)) & 15) == 0) {
      *reinterpret_cast<int4*>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t0 + i < a.tokens) {
          a.slots[t0 + i] = slot[i];
          a.positions[t0 + i] = pos[i];
        }
    }
  }
}

hipError_t launch_page_plan(const int32_t* cached, const int32_t* added, int32_t* block_table, const int32_t* free_pages,
                            int64_t requests, int64_t width, int64_t n_free, int64_t page_size, int64_t tokens,
                            int32_t* slots, int32_t* positions, int32_t* starts, int32_t* lengths, int32_t* taken,
                            hipStream_t s) {
  const PlanArgs a{cached, added, block_table, free_pages, slots, positions, starts, lengths, taken, tokens, n_free, width,
                   (int)requests, __builtin_ctzll((unsigned long long)page_size)};
  const int64_t per_wg = 4 * kPlanThreads;
  const int64_t want = (tokens + per_wg - 1) / per_wg;
  const unsigned grid = (unsigned)(want < 1 ? 1 : want > 1024 ? 1024 : want);
  hipLaunchKernelGGL(page_plan_kernel, dim3(grid), dim3(kPlanThreads), (size_t)(2 * requests + 1) * 4, s, a);
  return hipGetLastError();
}

}  // namespace mxq
