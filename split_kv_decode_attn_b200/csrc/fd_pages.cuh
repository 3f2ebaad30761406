// fd_pages.cuh — page bookkeeping of a paged KV cache on the device: pages,
// slots and positions for the new tokens of a batch (fd_alloc_pages) and the
// way back of finished requests' pages (fd_release_pages).
//
// Both are one exclusive sum over the requests followed by an expansion of
// each request into its tokens (or pages).  The sum is short (at most 65,535
// requests of 4 bytes each, in L2), so every CTA repeats it, 1,024 requests
// per pass, and expands only its own range of the output: one launch, no
// waiting between CTAs, and no atomics, so the result is a function of the
// inputs alone.  What bounds them is latency: 3.0-3.1 us a launch from graph
// replays for 16 requests, 4.1 for 1,024 (two sums of 10 exchanges each and three
// barriers per pass) and 5.9 for 250,000 tokens of 200 prompts (3 MB written).
// Inputs are read through L2, where the kernel before left them.
#pragma once

#include <cstdint>

#include "fd_ptx.cuh"

namespace fd {

constexpr int kPageThreads = 1024;   // requests per pass, and threads per CTA

struct PageArgs {
  int B, log2_block_size, max_blocks, num_pages;
  int max_items;               // capacity of the expansion: tokens, or pages
  int items_per_cta;
  const int32_t* seqlens;      // [B]
  const int32_t* new_lens;     // [B]                (alloc)
  const uint8_t* done;         // [B]                (release)
  int32_t* free_pages;         // [num_pages]
  const int32_t* free_count;   // [1]
  int32_t* block_table;        // [B, max_blocks]
  int32_t* seqlens_out;        // [B]
  int32_t* cu_new;             // [B + 1]            (alloc)
  int64_t* slots;              // [max_items]        (alloc)
  int32_t* positions;          // [max_items] or null (alloc)
  int32_t* free_count_out;     // [1]
  bool write_items;            // expand into tokens or pages (and write cu_new)
  bool write_state;            // write seqlens_out and free_count_out
};

// min(x + y, cap) for x, y <= cap < 2^31: associative, so that it can be
// scanned, and exact below the cap.
__device__ __forceinline__ uint32_t sat_add(uint32_t x, uint32_t y, uint32_t cap) {
  const uint32_t s = x + y;
  return s < cap ? s : cap;
}

// Inclusive saturating sum over the CTA's threads.  scratch: 32 words.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t cap, uint32_t* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v = sat_add(v, u, cap);
  }
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  if (warp == 0) {
    uint32_t w = scratch[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w = sat_add(w, u, cap);
    }
    scratch[lane] = w;
  }
  __syncthreads();
  const uint32_t r = warp > 0 ? sat_add(scratch[warp - 1], v, cap) : v;
  __syncthreads();   // scratch is free again
  return r;
}

// Last index b of s[0 .. n] (ascending, s[0] <= k < s[n]) with s[b] <= k.
__device__ __forceinline__ int segment_of(const uint32_t* s, int n, uint32_t k) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s[mid] <= k)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int clamp_len(int n, long long cap) {
  return n < 0 ? 0 : (n > cap ? static_cast<int>(cap) : n);
}

// Pages for the new tokens.  Request b holds n tokens and gets a new ones
// (those beyond max_items in all are not listed); it needs the pages
// ceil(n / bs) .. ceil((n + a) / bs) - 1 of its table row.  Page number k over
// the batch, in request order, is free_pages[F - 1 - k] of the F free ones; a
// request that the pool or its table row cannot serve in full keeps what it
// got.  Token t lies in slot table[b][t / bs] * bs + t % bs.
__global__ void __launch_bounds__(kPageThreads) fd_alloc_pages_kernel(const PageArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  __shared__ uint32_t scratch[32];
  __shared__ uint32_t s_cu[kPageThreads + 1];   // first token of each request of the pass
  __shared__ int s_n[kPageThreads];             // tokens held
  __shared__ int s_end[kPageThreads];           // tokens held afterwards
  __shared__ uint32_t s_page[kPageThreads];     // number of the request's first new page

  const int lbs = a.log2_block_size, bs = 1 << lbs;
  const long long room = min(static_cast<long long>(a.max_blocks) << lbs, 0x7fffffffll);
  const uint32_t T = static_cast<uint32_t>(a.max_items);
  const uint32_t F = static_cast<uint32_t>(clamp_len(__ldcg(a.free_count), a.num_pages));
  const bool first = blockIdx.x == 0;
  const uint32_t lo = min(static_cast<uint32_t>(blockIdx.x) * a.items_per_cta, T);
  const uint32_t hi = min(lo + static_cast<uint32_t>(a.items_per_cta), T);
  uint32_t tokens = 0, pages = 0;   // of the passes so far

  for (int b0 = 0; b0 < a.B; b0 += kPageThreads) {
    // Only the first CTA needs the sums behind its own tokens.
    if (!first && tokens >= hi) break;
    const int b = b0 + threadIdx.x;
    const bool live = b < a.B;
    const int n = live ? clamp_len(__ldcg(a.seqlens + b), room) : 0;
    const int want = live ? clamp_len(__ldcg(a.new_lens + b), T) : 0;
    const uint32_t cu1 = sat_add(tokens, block_scan(want, T, scratch), T);
    __syncthreads();
    if (threadIdx.x == 0) s_cu[0] = tokens;
    s_cu[threadIdx.x + 1] = cu1;
    __syncthreads();
    const uint32_t cu0 = s_cu[threadIdx.x];
    const long long e = min(static_cast<long long>(n) + (cu1 - cu0), room);
    const int p0 = static_cast<int>((static_cast<long long>(n) + bs - 1) >> lbs);
    const uint32_t need = static_cast<uint32_t>((e + bs - 1) >> lbs) - p0;
    const uint32_t page1 = pages + block_scan(need, 0x7fffffffu, scratch);
    const uint32_t page0 = page1 - need;
    const uint32_t granted = min(F - min(page0, F), need);
    const int end = static_cast<int>(min(e, static_cast<long long>(p0 + granted) << lbs));
    s_n[threadIdx.x] = n;
    s_end[threadIdx.x] = end;
    s_page[threadIdx.x] = page0;
    if (threadIdx.x == kPageThreads - 1) scratch[0] = page1;
    __syncthreads();
    const uint32_t begin = tokens;
    tokens = s_cu[kPageThreads];
    pages = scratch[0];
    if (first && live) {
      if (a.write_items) {
        if (b == 0) a.cu_new[0] = 0;
        a.cu_new[b + 1] = static_cast<int32_t>(cu1);
      }
      if (a.write_state) a.seqlens_out[b] = end;
    }
    if (a.write_items) {
      const uint32_t stop = min(hi, tokens);
      for (uint32_t k = max(lo, begin) + threadIdx.x; k < stop; k += kPageThreads) {
        const int r = segment_of(s_cu, kPageThreads, k);
        const long long t = static_cast<long long>(s_n[r]) + (k - s_cu[r]);
        int64_t slot = -1;
        if (t < s_end[r]) {
          const int j = static_cast<int>(t >> lbs);
          const int held = static_cast<int>((static_cast<long long>(s_n[r]) + bs - 1) >> lbs);
          int32_t* entry = a.block_table + static_cast<size_t>(b0 + r) * a.max_blocks + j;
          int page;
          if (j < held) {
            page = __ldcg(entry);
          } else {
            page = __ldcg(a.free_pages + (F - 1 - (s_page[r] + (j - held))));
            if ((t & (bs - 1)) == 0) *entry = page;
          }
          if (page >= 0) slot = (static_cast<int64_t>(page) << lbs) + (t & (bs - 1));
        }
        a.slots[k] = slot;
        if (a.positions) a.positions[k] = static_cast<int32_t>(t);
      }
    }
    __syncthreads();   // the next pass rewrites the shared arrays
  }
  if (a.write_items)   // places behind the last token: no slot
    for (uint32_t k = max(lo, tokens) + threadIdx.x; k < hi; k += kPageThreads) {
      a.slots[k] = -1;
      if (a.positions) a.positions[k] = 0;
    }
  if (first && a.write_state && threadIdx.x == 0)
    *a.free_count_out = static_cast<int32_t>(F - min(F, pages));
}

// Pages of finished requests go on top of the free ones, in request order:
// page number k over the batch becomes free_pages[F + k] (pages that do not
// fit num_pages are dropped).  A finished request holds no token afterwards.
__global__ void __launch_bounds__(kPageThreads) fd_release_pages_kernel(const PageArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  __shared__ uint32_t scratch[32];
  __shared__ uint32_t s_cu[kPageThreads + 1];   // number of each request's first page

  const int lbs = a.log2_block_size, bs = 1 << lbs;
  const long long room = min(static_cast<long long>(a.max_blocks) << lbs, 0x7fffffffll);
  const uint32_t F = static_cast<uint32_t>(clamp_len(__ldcg(a.free_count), a.num_pages));
  const uint32_t cap = static_cast<uint32_t>(a.num_pages) - F;
  const bool first = blockIdx.x == 0;
  const uint32_t lo = min(static_cast<uint32_t>(blockIdx.x) * a.items_per_cta, cap);
  const uint32_t hi = min(lo + static_cast<uint32_t>(a.items_per_cta), cap);
  uint32_t pages = 0;

  for (int b0 = 0; b0 < a.B; b0 += kPageThreads) {
    if (!first && pages >= hi) break;
    const int b = b0 + threadIdx.x;
    const bool live = b < a.B;
    const int n = live ? clamp_len(__ldcg(a.seqlens + b), room) : 0;
    const bool gone = live && __ldcg(a.done + b) != 0;
    const uint32_t held = gone ? static_cast<uint32_t>((static_cast<long long>(n) + bs - 1) >> lbs) : 0;
    const uint32_t cu1 = sat_add(pages, block_scan(min(held, cap), cap, scratch), cap);
    if (threadIdx.x == 0) s_cu[0] = pages;
    s_cu[threadIdx.x + 1] = cu1;
    __syncthreads();
    const uint32_t begin = pages;
    pages = s_cu[kPageThreads];
    if (first && live && a.write_state) a.seqlens_out[b] = gone ? 0 : n;
    if (a.write_items) {
      const uint32_t stop = min(hi, pages);
      for (uint32_t k = max(lo, begin) + threadIdx.x; k < stop; k += kPageThreads) {
        const int r = segment_of(s_cu, kPageThreads, k);
        a.free_pages[F + k] = __ldcg(a.block_table + static_cast<size_t>(b0 + r) * a.max_blocks + (k - s_cu[r]));
      }
    }
    __syncthreads();
  }
  if (first && a.write_state && threadIdx.x == 0)
    *a.free_count_out = static_cast<int32_t>(F + pages);
}

}  // namespace fd
