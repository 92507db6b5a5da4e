// pa_evict.h -- what pa_cache_accept and pa_cache_evict share: where a position's
// row lies, and the list of pages that a shorter length leaves free (not part of
// the public C ABI).
#pragma once

#include "pa_internal.h"

namespace pa {

constexpr int kMaxHeadBytes = 16384;  // of one KV head's row: 1024 pieces of 16 bytes

// Division of 0 <= n < 2^31 by d >= 1, the same for a whole call, by a high product
// (Granlund and Montgomery, "Division by invariant integers using multiplication",
// 1994): with s = ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1,
//   floor(n / d) = (floor(n m / 2^32) + n) >> s,
// whose sum stays below 2^32 for these n.  These kernels run once over little data,
// so they are as fast as their code comes in: a few instructions for a division's many.
struct FastDiv {
  unsigned mul, shift;
};
inline FastDiv fast_div(unsigned d) {
  unsigned s = 0;
  while ((1ull << s) < d) ++s;
  return FastDiv{(unsigned)(((1ull << 32) * ((1ull << s) - d)) / d + 1), s};
}
__device__ inline int divide(int n, FastDiv d) {
  return (int)((__umulhi((unsigned)n, d.mul) + (unsigned)n) >> d.shift);
}

struct FreeList {
  int32_t *pages, *count;  // both null: not wanted
  int capacity;
};

// Index of KV head h's row in slot `slot` of a page.
__device__ inline long long row_at(int page, int slot, int h, int Hk, int bs, int hnd) {
  return hnd ? ((long long)page * Hk + h) * bs + slot : ((long long)page * bs + slot) * Hk + h;
}
// Byte offset of KV head h's row at position pos; -1 where the page id is bad.
__device__ inline long long row_offset(const int32_t *bt, int pos, int h, int Hk, int bs, FastDiv by_bs,
                                       int num_blocks, int hnd, int head_bytes) {
  const int lp = divide(pos, by_bs), slot = pos - lp * bs, page = bt[lp];
  if (page < 0 || page >= num_blocks) return -1;
  return row_at(page, slot, h, Hk, bs, hnd) * head_bytes;
}

// 16 bytes from global to shared memory, past L1.
__device__ inline void copy16(uint4 *dst, const uint8_t *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// One block (all THREADS threads of it): lens(s, before, after) for every request,
// once, and the pages from ceil(after / bs) to ceil(before / bs) of each listed in
// request order.
template <int THREADS, typename Lens>
__device__ inline void list_free_pages(const FreeList &list, const int32_t *block_table,
                                       int max_blocks_per_seq, int bs, int num_blocks, int num_seqs,
                                       unsigned int *status, Lens lens) {
  __shared__ long long scratch[33];
  __shared__ long long s_end[THREADS];
  __shared__ int s_n[THREADS], s_page[THREADS];
  const int tid = threadIdx.x;
  long long sum = 0;
  unsigned flags = 0;
  for (int base = 0; base < num_seqs; base += THREADS) {
    const int s = base + tid, in = min(THREADS, num_seqs - base);
    int from = 0, n = 0;
    if (s < num_seqs) {
      int before, after;
      lens(s, before, after);
      if (after < before && after >= 0) {
        from = (int)(((unsigned)after + bs - 1) / bs);
        n = (int)(((unsigned)before + bs - 1) / bs) - from;
      }
    }
    if (!list.count) continue;
    long long tot;
    s_end[tid] = block_inclusive_scan(n, scratch, &tot);
    s_n[tid] = n;
    s_page[tid] = from;
    __syncthreads();
    // an entry a thread, all of their loads on their way at once
    for (long long e = tid; e < min(tot, list.capacity - sum); e += THREADS) {
      int lo = 0, hi = in - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s_end[mid] > e) hi = mid; else lo = mid + 1;
      }
      const int i = (int)(e - (s_end[lo] - s_n[lo]));
      int page = block_table[(size_t)(base + lo) * max_blocks_per_seq + s_page[lo] + i];
      if (page < 0 || page >= num_blocks) {
        page = -1;
        flags |= PA_DEV_BAD_BLOCK;
      }
      list.pages[sum + e] = page;
    }
    sum += tot;
    __syncthreads();  // the shared arrays are read
  }
  if (list.count && tid == 0) {
    *list.count = (int)min(sum, (long long)list.capacity);
    if (sum > list.capacity) flags |= PA_DEV_OVERFLOW;
  }
  if (flags) atomicOr(status, flags);
}

}  // namespace pa
