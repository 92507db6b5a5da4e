// pa_evict.h -- what pa_cache_accept and pa_cache_evict share: where a position's
// row lies, and the list of pages that a shorter length leaves free (not part of
// the public C ABI).
#pragma once

#include "pa_internal.h"

namespace pa {

constexpr int kMaxHeadBytes = 16384;  // of one KV head's row: 1024 pieces of 16 bytes

// Division of 0 <= n < 2^31 by d >= 1, the same for a whole call: one high product
// instead of the twenty instructions of a division (these kernels run once over
// little data, so they are as fast as their code comes in).
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

// Byte offset of KV head h's row at position pos; -1 where the page id is bad.
__device__ inline long long row_offset(const int32_t *bt, int pos, int h, int Hk, int bs, FastDiv by_bs,
                                       int num_blocks, int hnd, int head_bytes) {
  const int lp = divide(pos, by_bs), slot = pos - lp * bs, page = __ldg(bt + lp);
  if (page < 0 || page >= num_blocks) return -1;
  const long long row = hnd ? ((long long)page * Hk + h) * bs + slot : ((long long)page * bs + slot) * Hk + h;
  return row * head_bytes;
}

// Whether path[0 .. n) rises strictly within [0, q_len).  A whole warp calls.
__device__ inline bool path_ok(const int32_t *path, int n, int q_len, int lane) {
  bool ok = true;
  for (int i = lane; i < n; i += 32) {
    const int x = __ldg(path + i), last = i > 0 ? __ldg(path + i - 1) : -1;
    ok &= x > last && x < q_len;
  }
  return __all_sync(0xffffffffu, ok);
}

// One block (all THREADS threads of it): lens(s, before, after) for every request,
// once, and the pages from ceil(after / bs) to ceil(before / bs) of each listed in
// request order.
template <int THREADS, typename Lens>
__device__ inline void list_free_pages(const FreeList &list, const int32_t *block_table,
                                       int max_blocks_per_seq, int bs, int num_blocks, int num_seqs,
                                       unsigned int *status, Lens lens) {
  __shared__ long long scratch[33];
  __shared__ int s_first[THREADS], s_n[THREADS], s_page[THREADS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long sum = 0;
  unsigned flags = 0;
  for (int base = 0; base < num_seqs; base += THREADS) {
    const int s = base + tid;
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
    const long long at = block_inclusive_scan(n, scratch, &tot) + sum - n;
    // (counts fit 32 bits where they fit the list; beyond it nothing is written)
    s_first[tid] = (int)min(at, 0x7fffffffll);
    s_n[tid] = n;
    s_page[tid] = from;
    __syncthreads();
    for (int k = warp; k < min(THREADS, num_seqs - base); k += THREADS / 32) {
      const int32_t *bt = block_table + (size_t)(base + k) * max_blocks_per_seq;
      for (int i = lane; i < s_n[k]; i += 32) {
        int page = __ldg(bt + s_page[k] + i);
        if (page < 0 || page >= num_blocks) {
          page = -1;
          flags |= PA_DEV_BAD_BLOCK;
        }
        const long long to = (long long)s_first[k] + i;
        if (to < list.capacity) list.pages[to] = page;
        else flags |= PA_DEV_OVERFLOW;
      }
    }
    sum += tot;
    __syncthreads();  // the shared arrays are read
  }
  if (list.count && tid == 0) *list.count = (int)min(sum, (long long)list.capacity);
  if (flags) atomicOr(status, flags);
}

}  // namespace pa
