// pa_evict.cu -- pa_cache_evict: a cache held to a budget.  Request s of length
// L > B = keep_lens[s] keeps, KV head by KV head, its first f positions, its last r
// and the B - f - r of largest accumulated weight among the others (ties: the
// lowest position; NaN below everything).  The kept rows move to positions 0 ..
// B - 1 in order, in place, and their weights with them.
//
// Two launches.  select: a block for each (request, KV head) finds the weight of
// rank B - f - r by three passes of radix counting (11, 11 and 10 bits of an order-
// preserving integer), then lists the kept positions in order.  move: position i
// of the list goes to i <= list[i]; runs of B positions (chunks) are handed out in
// order, and a block may write over positions only when the blocks whose rows lie
// there have read them.
#include <algorithm>

#include "pa_evict.h"

namespace pa {
namespace {

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr int kSelectThreads = 512;
constexpr int kBits = 11, kBins = 1 << kBits;
constexpr int kMoveThreads = 256;
constexpr int kMovePieces = 4;  // 16-byte pieces of K, and of V, that a thread holds
constexpr int kChunkPieces = kMoveThreads * kMovePieces;

struct EvictHeader {
  unsigned ticket;  // next chunk to hand out
  unsigned chunks;  // of all requests
};

struct EvictArgs {
  uint8_t *k_cache, *v_cache;
  const float *weights;
  float *weights_out;
  const int32_t *block_table, *seq_lens, *keep_lens;
  int32_t *seq_lens_out;
  FreeList free;
  int num_first, num_recent;
  int num_seqs, num_kv_heads, head_bytes, block_size, max_blocks_per_seq, num_blocks, max_seq_len, hnd;
  int chunk_rows;   // positions of a chunk
  int max_chunks;   // of one (request, KV head)
  unsigned int *status;
  EvictHeader *head;
  unsigned *chunk_end;  // [num_seqs] inclusive sum of the requests' chunks
  unsigned *ready;      // [num_seqs * num_kv_heads][max_chunks] 1: the chunk's rows are read
  int32_t *kept;        // [num_seqs * num_kv_heads][max_seq_len]
};

// The request's length behind the eviction; bad metadata: its length, nothing moves.
__device__ inline int evicted_len(const EvictArgs &a, int s, int &len, unsigned &flags) {
  len = a.seq_lens[s];
  const int keep = a.keep_lens[s];
  if (len < 0 || len > a.max_seq_len || len > (long long)a.max_blocks_per_seq * a.block_size || keep < 0) {
    flags |= PA_DEV_BAD_SEQLEN;
    return len;
  }
  return min(len, keep);
}

// An integer that orders as the weight does; NaN is the lowest.
__device__ inline uint32_t order_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);  // (-0 as 0)
  if (w != w) return 0;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// ---------------------------------------------------------------------------
// select
// ---------------------------------------------------------------------------

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ long long scratch[33];
  __shared__ unsigned s_hist[kBins];
  __shared__ unsigned s_prefix, s_rank;
  const int tid = threadIdx.x, Hk = a.num_kv_heads, bs = a.block_size;
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x == a.num_seqs * Hk) {
    // -- the last block: chunks, new lengths, the pages that are free again
    long long sum = 0;
    for (int base = 0; base < a.num_seqs; base += kSelectThreads) {
      const int s = base + tid;
      long long n = 0, tot;
      if (s < a.num_seqs) {
        int len;
        unsigned flags = 0;
        const int after = evicted_len(a, s, len, flags);
        if (flags) atomicOr(a.status, flags);
        if (after < len) n = (long long)Hk * ((after + a.chunk_rows - 1) / a.chunk_rows);
        a.seq_lens_out[s] = after;
      }
      const long long end = block_inclusive_scan(n, scratch, &tot) + sum;
      if (s < a.num_seqs) a.chunk_end[s] = (unsigned)end;
      sum += tot;
    }
    if (tid == 0) *a.head = EvictHeader{0, (unsigned)sum};
    auto lens = [&](int s, int &before, int &after) {
      unsigned flags = 0;
      after = evicted_len(a, s, before, flags);
    };
    if (a.free.count)
      list_free_pages<kSelectThreads>(a.free, a.block_table, a.max_blocks_per_seq, bs, a.num_blocks,
                                      a.num_seqs, a.status, lens);
    return;
  }

  const int s = blockIdx.x / Hk, h = blockIdx.x - s * Hk;
  int len;
  unsigned flags = 0;
  const int after = evicted_len(a, s, len, flags);
  if (flags) return;  // (the last block reports it)
  const int32_t *bt = a.block_table + (size_t)s * a.max_blocks_per_seq;
  auto slot_of = [&](int pos) -> long long {  // of a weight; -1: a bad page
    const int lp = (unsigned)pos / (unsigned)bs, page = __ldg(bt + lp);
    if (page < 0 || page >= a.num_blocks) {
      flags |= PA_DEV_BAD_BLOCK;
      return -1;
    }
    return ((long long)page * Hk + h) * bs + (pos - lp * bs);
  };
  if (after == len) {
    if (a.weights_out != a.weights) {
      for (int pos = tid; pos < len; pos += kSelectThreads) {
        const long long at = slot_of(pos);
        if (at >= 0) a.weights_out[at] = a.weights[at];
      }
      if (flags) atomicOr(a.status, flags);
    }
    return;
  }
  const int first = min(a.num_first, after), recent = min(a.num_recent, after - first);
  const int need = after - first - recent, lo = first, hi = len - recent;  // candidates [lo, hi)
  for (int c = tid; c < (after + a.chunk_rows - 1) / a.chunk_rows; c += kSelectThreads)
    a.ready[(size_t)blockIdx.x * a.max_chunks + c] = 0;

  // -- the candidate of rank `need` from the top: `prefix` its leading bits
  unsigned prefix = 0, rank = need;
  if (need > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1 << 10 : kBins;
      for (int b = tid; b < kBins; b += kSelectThreads) s_hist[b] = 0;
      __syncthreads();
      const unsigned above = pass == 0 ? 0u : ~0u << (pass == 1 ? 21 : 10);
#pragma unroll 4
      for (int pos = lo + tid; pos < hi; pos += kSelectThreads) {
        const long long at = slot_of(pos);
        const uint32_t key = at < 0 ? 0u : order_of(a.weights[at]);
        if ((key & above) == prefix) atomicAdd(&s_hist[(key >> shift) & (bins - 1)], 1u);
      }
      __syncthreads();
      // bins from the top: thread t takes the t-th group of kBins / kSelectThreads
      constexpr int PER = kBins / kSelectThreads;
      long long n = 0, tot;
      const int top = kBins - 1 - tid * PER;
#pragma unroll
      for (int i = 0; i < PER; ++i) n += s_hist[top - i];
      const long long end = block_inclusive_scan(n, scratch, &tot);
      unsigned before = (unsigned)(end - n);
      if (before < rank && rank <= (unsigned)end) {  // one thread
        int b = top;
        while (before + s_hist[b] < rank) before += s_hist[b--];
        s_prefix = prefix | (unsigned)b << shift;
        s_rank = rank - before;
      }
      __syncthreads();
      prefix = s_prefix;
      rank = s_rank;
    }
  }
  // -- the kept positions in order: the first `rank` of those that equal the threshold
  int32_t *kept = a.kept + (size_t)blockIdx.x * a.max_seq_len;
  long long done = 0;  // kept positions so far in the low half, equal ones in the high half
  constexpr int PER = 4;
  for (int base = 0; base < len; base += kSelectThreads * PER) {
    float w[PER];
    bool there[PER];  // (not on a bad page)
    int state[PER];   // 0 no, 1 kept, 2 equal to the threshold
    long long n = 0, tot;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int pos = base + tid * PER + i;
      state[i] = 0;
      w[i] = 0.f;
      there[i] = false;
      if (pos >= len) continue;
      const long long at = slot_of(pos);
      there[i] = at >= 0;
      if (there[i]) w[i] = a.weights[at];
      const uint32_t key = at < 0 ? 0u : order_of(w[i]);
      state[i] = pos < lo || pos >= hi ? 1 : need == 0 ? 0 : key > prefix ? 1 : key == prefix ? 2 : 0;
      n += state[i] == 1 ? 1ll : state[i] == 2 ? 1ll << 32 : 0ll;
    }
    long long at = block_inclusive_scan(n, scratch, &tot) + done - n;
    // (every weight of this step is read: the scan is a barrier)
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const unsigned equal = (unsigned)(at >> 32);
      const bool keep = state[i] == 1 || (state[i] == 2 && equal < rank);
      if (keep) {
        const int dst = (int)((unsigned)at + min(equal, rank));
        kept[dst] = base + tid * PER + i;
        const long long to = slot_of(dst);
        if (to >= 0 && there[i]) a.weights_out[to] = w[i];
      }
      at += state[i] == 1 ? 1ll : state[i] == 2 ? 1ll << 32 : 0ll;
    }
    done += tot;
  }
  if (flags) atomicOr(a.status, flags);
}

// ---------------------------------------------------------------------------
// move
// ---------------------------------------------------------------------------

__device__ inline unsigned load_acquire(const unsigned *p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
  __shared__ unsigned s_ticket;
  const int tid = threadIdx.x, Hk = a.num_kv_heads, bs = a.block_size, ppr = a.head_bytes / 16;
  pdl_trigger();
  pdl_wait();
  const unsigned chunks = a.head->chunks;
  for (;;) {
    __syncthreads();  // s_ticket is read
    if (tid == 0) s_ticket = atomicAdd(&a.head->ticket, 1u);
    __syncthreads();
    const unsigned t = s_ticket;
    if (t >= chunks) return;
    int lo = 0, hi = a.num_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (a.chunk_end[mid] > t) hi = mid; else lo = mid + 1;
    }
    const int s = lo, len = a.seq_lens[s], after = min(len, a.keep_lens[s]);
    const int nc = (after + a.chunk_rows - 1) / a.chunk_rows;
    const int local = (int)(t - (a.chunk_end[s] - (unsigned)(Hk * nc))), h = local / nc, c = local - h * nc;
    const int32_t *bt = a.block_table + (size_t)s * a.max_blocks_per_seq;
    const int32_t *kept = a.kept + ((size_t)s * Hk + h) * a.max_seq_len;
    unsigned *ready = a.ready + ((size_t)s * Hk + h) * a.max_chunks;
    const int i0 = c * a.chunk_rows, rows = min(a.chunk_rows, after - i0);
    // -- this chunk's rows
    uint4 k[kMovePieces], v[kMovePieces];
    long long to[kMovePieces];
    unsigned flags = 0;
#pragma unroll
    for (int u = 0; u < kMovePieces; ++u) {
      const int e = u * kMoveThreads + tid, row = e / ppr, piece = e - row * ppr;
      to[u] = -1;
      if (row >= rows) continue;
      const int dst = i0 + row, src = __ldg(kept + dst);
      if (src == dst) continue;
      const long long from = row_offset(bt, src, h, Hk, bs, a.num_blocks, a.hnd, a.head_bytes);
      const long long into = row_offset(bt, dst, h, Hk, bs, a.num_blocks, a.hnd, a.head_bytes);
      if (from < 0 || into < 0) {
        flags |= PA_DEV_BAD_BLOCK;
        continue;
      }
      to[u] = into + piece * 16;
      k[u] = __ldcg(reinterpret_cast<const uint4 *>(a.k_cache + from + piece * 16));
      v[u] = __ldcg(reinterpret_cast<const uint4 *>(a.v_cache + from + piece * 16));
    }
    // (the barrier's operand needs every loaded value: the rows are read when it opens)
    unsigned seen = 0;
#pragma unroll
    for (int u = 0; u < kMovePieces; ++u)
      if (to[u] >= 0) seen ^= k[u].x ^ v[u].x;
    __syncthreads_or(seen);
    if (tid == 0) {
      __threadfence();
      atomicExch(ready + c, 1u);
    }
    // -- the chunks whose rows lie where this one writes: those that hold the kept
    // positions of [i0, i0 + rows), from the first one's chunk on; they were handed
    // out before this one, and mark their rows read without waiting for anything
    int from = 0, until = after;  // the first kept position that is not below i0
    while (from < until) {
      const int mid = (from + until) >> 1;
      if (__ldg(kept + mid) < i0) from = mid + 1; else until = mid;
    }
    bool late = false;
    for (int w = from / a.chunk_rows + tid; w < c; w += kMoveThreads) {
      if (load_acquire(ready + w)) continue;
      const uint64_t t0 = global_timer_ns();
      for (uint32_t i = 1; !load_acquire(ready + w); ++i) {
        if ((i & 63u) == 0 && global_timer_ns() - t0 > kWaitLimitNs) {
          late = true;
          break;
        }
      }
      if (late) break;
    }
    if (late) flags |= PA_DEV_TIMEOUT;
    if (!__syncthreads_or(late)) {
#pragma unroll
      for (int u = 0; u < kMovePieces; ++u) {
        if (to[u] < 0) continue;
        *reinterpret_cast<uint4 *>(a.k_cache + to[u]) = k[u];
        *reinterpret_cast<uint4 *>(a.v_cache + to[u]) = v[u];
      }
    }
    if (flags) atomicOr(a.status, flags);
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct EvictLayout {
  size_t head, chunk_end, ready, kept, total;
  int chunk_rows, max_chunks;
  bool ok;
};

EvictLayout evict_layout(int head_bytes, int num_seqs, int num_kv_heads, int max_seq_len) {
  EvictLayout l{};
  const long long S = std::max(num_seqs, 1), units = S * num_kv_heads, msl = std::max(max_seq_len, 1);
  l.chunk_rows = std::max(1, kChunkPieces / std::max(head_bytes / 16, 1));
  l.max_chunks = (int)ceil_div_ll(msl, l.chunk_rows);
  l.ok = units < (1ll << 30) && units * l.max_chunks < (1ll << 31);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  l.head = take(sizeof(EvictHeader));
  l.chunk_end = take(S * sizeof(unsigned));
  l.ready = take((size_t)units * l.max_chunks * sizeof(unsigned));
  l.kept = take((size_t)units * msl * sizeof(int32_t));
  l.total = off;
  return l;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

size_t pa_cache_evict_workspace_bytes(pa_dtype dtype, int num_seqs, int num_kv_heads, int head_dim,
                                      int max_seq_len) {
  const int es = dtype == PA_F32 ? 4 : 2;
  if (num_seqs < 0 || num_kv_heads <= 0 || head_dim <= 0 || max_seq_len < 0 ||
      (long long)head_dim * es > kMaxHeadBytes)
    return 0;
  const EvictLayout l = evict_layout(head_dim * es, num_seqs, num_kv_heads, max_seq_len);
  return l.ok ? l.total : 0;
}

pa_status pa_cache_evict(void *k_cache, void *v_cache, const float *weights, float *weights_out,
                         const int32_t *block_table, const int32_t *seq_lens,
                         const int32_t *keep_lens, int32_t *seq_lens_out, int32_t *freed_pages,
                         int32_t *num_freed, int num_first, int num_recent, int num_kv_heads,
                         int head_dim, int block_size, void *stream, pa_dtype dtype, int num_seqs,
                         int max_blocks_per_seq, int num_blocks, int freed_capacity,
                         int max_seq_len, pa_kv_layout kv_layout, void *workspace,
                         size_t workspace_bytes) {
  if (num_seqs < 0 || num_first < 0 || num_recent < 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      block_size <= 0 || max_blocks_per_seq < 0 || num_blocks < 0 || freed_capacity < 0 ||
      max_seq_len < 0 || (dtype != PA_F32 && dtype != PA_BF16) ||
      (kv_layout != PA_KV_NHD && kv_layout != PA_KV_HND))
    return PA_ERR_INVALID_ARG;
  if ((num_freed == nullptr) != (freed_pages == nullptr) || (!freed_pages && freed_capacity > 0))
    return PA_ERR_INVALID_ARG;
  const int es = dtype == PA_F32 ? 4 : 2;
  if ((long long)head_dim * es % 16 != 0 || (long long)head_dim * es > kMaxHeadBytes)
    return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0 && !num_freed) return PA_OK;
  if (num_seqs > 0 && (!k_cache || !v_cache || !weights || !weights_out || !block_table ||
                       !seq_lens || !keep_lens || !seq_lens_out || max_blocks_per_seq == 0 ||
                       num_blocks == 0))
    return PA_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(weights, 4) ||
      !aligned(weights_out, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(keep_lens, 4) || !aligned(seq_lens_out, 4) || !aligned(freed_pages, 4) ||
      !aligned(num_freed, 4) || seq_lens_out == seq_lens || seq_lens_out == keep_lens)
    return PA_ERR_INVALID_ARG;
  const EvictLayout lay = evict_layout(head_dim * es, num_seqs, num_kv_heads, max_seq_len);
  if (!lay.ok) return PA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < lay.total) return PA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return PA_ERR_INVALID_ARG;
  EvictArgs a{};
  void *lib_ws = nullptr;
  int num_sms = 0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const pa_status s = device_resources(st, 0, &lib_ws, &a.status, &num_sms);
  if (s != PA_OK) return s;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  a.k_cache = static_cast<uint8_t *>(k_cache);
  a.v_cache = static_cast<uint8_t *>(v_cache);
  a.weights = weights;
  a.weights_out = weights_out;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.keep_lens = keep_lens;
  a.seq_lens_out = seq_lens_out;
  a.free = FreeList{freed_pages, num_freed, freed_capacity};
  a.num_first = num_first;
  a.num_recent = num_recent;
  a.num_seqs = num_seqs;
  a.num_kv_heads = num_kv_heads;
  a.head_bytes = head_dim * es;
  a.block_size = block_size;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.max_seq_len = max_seq_len;
  a.hnd = kv_layout == PA_KV_HND;
  a.chunk_rows = lay.chunk_rows;
  a.max_chunks = lay.max_chunks;
  a.head = reinterpret_cast<EvictHeader *>(ws + lay.head);
  a.chunk_end = reinterpret_cast<unsigned *>(ws + lay.chunk_end);
  a.ready = reinterpret_cast<unsigned *>(ws + lay.ready);
  a.kept = reinterpret_cast<int32_t *>(ws + lay.kept);
  if (launch_dependent(evict_select_kernel, dim3((unsigned)(num_seqs * num_kv_heads + 1)),
                       dim3(kSelectThreads), 0, st, a) != cudaSuccess)
    return PA_ERR_CUDA;
  if (num_seqs == 0) return PA_OK;
  const long long most = (long long)num_seqs * num_kv_heads * lay.max_chunks;
  const long long blocks = std::min<long long>(most, 8ll * num_sms);
  return launch_dependent(evict_move_kernel, dim3((unsigned)blocks), dim3(kMoveThreads), 0, st, a) ==
                 cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

}  // extern "C"
