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

constexpr int kMaxEvictLen = 1 << 30;  // positions some steps behind the end count in 32 bits
constexpr int kSelectThreads = 1024;
constexpr int kBits = 11, kBins = 1 << kBits;
constexpr int kMoveThreads = 256;
constexpr int kMoveSeqs = 256;  // requests whose chunks and lengths a block keeps at hand
constexpr int kMovePieces = 4;  // 16-byte pieces of K, and of V, that a thread copies
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
  FastDiv by_bs, by_ppr, by_rows;
  unsigned int *status;
  EvictHeader *head;
  unsigned *chunk_end;  // [num_seqs] inclusive sum of the requests' chunks
  unsigned *ready;      // [num_seqs * num_kv_heads][max_chunks] 1: the chunk's rows are read
  int32_t *kept;        // [num_seqs * num_kv_heads][max_seq_len] positions, in order,
  float *kept_w;        // and their weights
  int32_t *below;       // [num_seqs * num_kv_heads][max_chunks] kept positions below the chunk's first one
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

constexpr uint32_t kZeroKey = 0x80000000u;  // of 0 and of -0
// The weight of a key, bit for bit, unless it is 0 (a NaN) or kZeroKey.
__device__ inline float weight_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// ---------------------------------------------------------------------------
// select
// ---------------------------------------------------------------------------
// A cluster of C blocks for each (request, KV head), each with its share of the
// positions, whose weights it reads once, as keys in shared memory.  Three passes
// over them count the keys' leading bits, a fourth lists what is kept; counts are summed
// over the cluster through distributed shared memory.  Bound by latency: the pages, the
// weights, a barrier or two between the steps of a pass.  16 requests of up to 8192
// positions, 8 KV heads: 14 us; 4 of up to 131072 in clusters of 16 blocks 22 (a
// call 36, 42 in clusters of 8; what digits the keys have changes it by 3).

constexpr int kMostCluster = 16;

struct SelectShared {
  alignas(16) unsigned hist[kBins];
  unsigned count[2 * kMostCluster];  // of each block's share: kept for sure, then equal to the threshold
  unsigned prefix, rank;
  unsigned slice[kMostCluster];
  unsigned warp_sum[2][32];
  long long scratch[33];
};

__device__ inline unsigned load_cluster(const unsigned *p, unsigned rank) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_map(smem_u32(p), rank)) : "memory");
  return v;
}
__device__ inline void store_cluster(unsigned *p, unsigned rank, unsigned v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_map(smem_u32(p), rank)), "r"(v) : "memory");
}

// Inclusive sum over the block's threads, one barrier; `turn` alternates between
// calls (the sums of the call before may still be read).
__device__ inline unsigned select_scan(SelectShared &sh, unsigned v, int turn, unsigned &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) sh.warp_sum[turn & 1][warp] = v;
  __syncthreads();
  static_assert(kSelectThreads == 1024, "a warp's sum for each lane");
  const unsigned y = sh.warp_sum[turn & 1][lane];
  total = __reduce_add_sync(0xffffffffu, y);
  return v + __reduce_add_sync(0xffffffffu, lane < warp ? y : 0u);
}

// The weight of one position (NaN on a bad page), where it is not in shared memory.
__device__ __noinline__ float read_weight(const EvictArgs &a, const int32_t *bt, int h, int pos) {
  const int lp = divide(pos, a.by_bs), page = bt[lp];
  if (page < 0 || page >= a.num_blocks) {
    atomicOr(a.status, PA_DEV_BAD_BLOCK);
    return __int_as_float(0x7fc00000);
  }
  return a.weights[((long long)page * a.num_kv_heads + h) * a.block_size + (pos - lp * a.block_size)];
}

// cached: keys that the dynamic shared memory holds (the others are made again)
__global__ void __launch_bounds__(kSelectThreads, 1) evict_select_kernel(const __grid_constant__ EvictArgs a, int C, int cached) {
  extern __shared__ uint32_t s_key[];
  __shared__ SelectShared sh;
  const int tid = threadIdx.x, Hk = a.num_kv_heads, bs = a.block_size;
  const int unit = blockIdx.x / C, part = blockIdx.x - unit * C;
  pdl_trigger();
  pdl_wait();
  if (unit == a.num_seqs * Hk) {
    if (part) return;
    // -- the last cluster: chunks, new lengths, the pages that are free again
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
      const long long end = block_inclusive_scan(n, sh.scratch, &tot) + sum;
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

  const int s = unit / Hk, h = unit - s * Hk;
  int len;
  unsigned flags = 0;
  const int after = evicted_len(a, s, len, flags);
  if (flags) return;  // (the last cluster reports it; the same for the whole cluster)
  const int32_t *bt = a.block_table + (size_t)s * a.max_blocks_per_seq;
  auto slot_of = [&](int pos) -> long long {  // of a weight; -1: a bad page
    const int lp = divide(pos, a.by_bs), page = bt[lp];
    if (page < 0 || page >= a.num_blocks) {
      flags |= PA_DEV_BAD_BLOCK;
      return -1;
    }
    return ((long long)page * Hk + h) * bs + (pos - lp * bs);
  };
  if (after == len) {
    if (a.weights_out != a.weights) {
      for (int pos = part * kSelectThreads + tid; pos < len; pos += C * kSelectThreads) {
        const long long at = slot_of(pos);
        if (at >= 0) a.weights_out[at] = a.weights[at];
      }
      if (flags) atomicOr(a.status, flags);
    }
    return;
  }
  // The cluster's blocks are all there before any of them reaches into another's shared
  // memory, whether or not there is something to count; the weights are read meanwhile.
  if (C > 1) cluster_arrive_all();
  const int first = min(a.num_first, after), recent = min(a.num_recent, after - first);
  const int need = after - first - recent, lo = first, hi = len - recent;  // candidates [lo, hi)
  for (int c = part * kSelectThreads + tid; c < (after + a.chunk_rows - 1) / a.chunk_rows; c += C * kSelectThreads)
    a.ready[(size_t)unit * a.max_chunks + c] = 0;
  const int share = (len + C - 1) / C, p0 = min(part * share, len), p1 = min(p0 + share, len);
  // (a position on a bad page counts as NaN)
  auto read = [&](int pos) { return read_weight(a, bt, h, pos); };
  const int c1 = min(p1, p0 + cached);  // positions below it are in shared memory
  for (int b = tid; b < kBins; b += kSelectThreads) sh.hist[b] = 0;
  {
    // two latencies for several of them: the pages, then the weights
    constexpr int U = 8;
    for (int base = p0 + tid; base < c1; base += U * kSelectThreads) {
      int page[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int pos = base + u * kSelectThreads;
        page[u] = pos < c1 ? bt[divide(pos, a.by_bs)] : 0;
      }
      float w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int pos = base + u * kSelectThreads;
        const bool ok = page[u] >= 0 && page[u] < a.num_blocks;
        w[u] = __int_as_float(0x7fc00000);
        if (!ok) flags |= PA_DEV_BAD_BLOCK;
        else if (pos < c1)
          w[u] = a.weights[((long long)page[u] * Hk + h) * bs + (pos - divide(pos, a.by_bs) * bs)];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int pos = base + u * kSelectThreads;
        if (pos < c1) s_key[pos - p0] = order_of(w[u]);
      }
    }
    __syncthreads();
  }
  if (C > 1) cluster_wait_all();
  auto key_of = [&](int pos) { return pos < c1 ? s_key[pos - p0] : order_of(read(pos)); };

  // -- the candidate of rank `need` from the top: `prefix` its leading bits
  // (once a bin is kept as a whole the passes end: prefix is then below all of it, and
  // no equal ones are wanted)
  unsigned prefix = 0, rank = need;
#pragma unroll 1
  for (int pass = 0; rank > 0 && pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1 << 10 : kBins;
    const unsigned above = pass == 0 ? 0u : ~0u << (pass == 1 ? 21 : 10);
    auto count = [&](uint32_t key) {
      if ((key & above) == prefix) atomicAdd(&sh.hist[(key >> shift) & (bins - 1)], 1u);
    };
    int pos = max(p0, lo) + tid;
#pragma unroll 4
    for (; pos < min(c1, hi); pos += kSelectThreads) count(s_key[pos - p0]);
    for (; pos < min(p1, hi); pos += kSelectThreads) count(order_of(read(pos)));
    if (C > 1) cluster_sync_all();
    else __syncthreads();
    // bins from the top: thread t takes the t-th pair
    static_assert(kBins == 2 * kSelectThreads, "two bins a thread");
    const int low = kBins - 2 - tid * 2;
    const uint2 own = *reinterpret_cast<const uint2 *>(&sh.hist[low]);
    unsigned tot;
    if (C > 1) {
      // block k sums its slice of the bins over the cluster; the slices' sums, given
      // to all, say in whose slice the rank lies, and that block finds the bin
      const int width = kBins / C, s0 = kBins - (part + 1) * width;  // slices from the top too
      unsigned n = 0, v[kMostCluster];
      const int mine = s0 + width - 1 - tid;  // thread t: the t-th bin from the slice's top
      if (tid < width) {
#pragma unroll
        for (int k = 0; k < kMostCluster; ++k) v[k] = k < C ? load_cluster(&sh.hist[mine], k) : 0u;
#pragma unroll
        for (int k = 0; k < kMostCluster; ++k) n += v[k];
      }
      const unsigned end = select_scan(sh, n, pass, tot);
      if (tid < C) store_cluster(&sh.slice[part], tid, tot);
      cluster_sync_all();
      unsigned before = end - n;
      for (int k = 0; k < part; ++k) before += sh.slice[k];
      if (tid < width && before < rank && rank <= before + n) {  // one thread of the cluster
        const unsigned bin = prefix | (unsigned)mine << shift;
        const bool whole = n == rank - before && bin != 0;
        for (int k = 0; k < C; ++k) {
          store_cluster(&sh.prefix, k, bin - whole);
          store_cluster(&sh.rank, k, whole ? 0u : rank - before);
        }
      }
      cluster_sync_all();
    } else {
      const unsigned n = own.x + own.y, end = select_scan(sh, n, pass, tot), before = end - n;
      if (before < rank && rank <= end) {  // one thread
        const bool high = before + own.y >= rank;
        const unsigned bin = prefix | (unsigned)(low + high) << shift;
        const unsigned left = high ? rank - before : rank - before - own.y;
        const bool whole = left == (high ? own.y : own.x) && bin != 0;
        sh.prefix = bin - whole;
        sh.rank = whole ? 0u : left;
      }
      __syncthreads();
    }
    prefix = sh.prefix;
    rank = sh.rank;
    sh.hist[low] = sh.hist[low + 1] = 0;
    __syncthreads();
  }
  auto state_of = [&](int pos, uint32_t key) {  // 0 no, 1 kept, 2 equal to the threshold
    return pos < lo || pos >= hi ? 1 : need == 0 ? 0 : key > prefix ? 1 : key == prefix ? 2 : 0;
  };
  // -- how many of either kind lie before each warp's stretch of the share
  const int lane = tid & 31, warp = tid >> 5;
  const int stretch = (p1 - p0 + kSelectThreads - 1) / kSelectThreads * 32;
  const int w0 = min(p0 + warp * stretch, p1), w1 = min(w0 + stretch, p1);
  unsigned sure = 0, equal = 0;
#pragma unroll 4
  for (int pos = w0 + lane; pos < w1; pos += 32) {
    const int st = state_of(pos, key_of(pos));
    sure += st == 1;
    equal += st == 2;
  }
  sure = __reduce_add_sync(0xffffffffu, sure);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) {
    sh.warp_sum[0][warp] = sure;
    sh.warp_sum[1][warp] = equal;
  }
  __syncthreads();
  const unsigned ws = sh.warp_sum[0][lane], we = sh.warp_sum[1][lane];
  unsigned sure_before = __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0u);
  unsigned equal_before = __reduce_add_sync(0xffffffffu, lane < warp ? we : 0u);
  if (C > 1) {
    if (warp == 0) {
      const unsigned ts = __reduce_add_sync(0xffffffffu, ws), te = __reduce_add_sync(0xffffffffu, we);
      if (lane < C) {
        store_cluster(&sh.count[part], lane, ts);
        store_cluster(&sh.count[kMostCluster + part], lane, te);
      }
    }
    cluster_sync_all();
    for (int k = 0; k < part; ++k) {
      sure_before += sh.count[k];
      equal_before += sh.count[kMostCluster + k];
    }
  }
  // -- the kept positions in order: the first `rank` of those that equal the threshold
  int32_t *kept = a.kept + (size_t)unit * a.max_seq_len;
  float *kept_w = a.kept_w + (size_t)unit * a.max_seq_len;
  int32_t *below = a.below + (size_t)unit * a.max_chunks;
  const unsigned under = (1u << lane) - 1;
  for (int base = w0; base < w1; base += 32) {
    const int pos = base + lane;
    const uint32_t key = pos < w1 ? key_of(pos) : 0u;
    const int st = pos < w1 ? state_of(pos, key) : 0;
    const unsigned b1 = __ballot_sync(0xffffffffu, st == 1), b2 = __ballot_sync(0xffffffffu, st == 2);
    const unsigned eq = equal_before + __popc(b2 & under);
    const int dst = (int)(sure_before + __popc(b1 & under) + min(eq, rank));  // kept ones below pos
    if (pos < w1 && pos < after) {
      const int c = divide(pos, a.by_rows);
      if (c * a.chunk_rows == pos) below[c] = dst;
    }
    if (st == 1 || (st == 2 && eq < rank)) {
      kept[dst] = pos;
      kept_w[dst] = key == 0u || key == kZeroKey ? read(pos) : weight_of(key);
    }
    sure_before += __popc(b1);
    equal_before += __popc(b2);
  }
  if (flags) atomicOr(a.status, flags);
}

// ---------------------------------------------------------------------------
// move
// ---------------------------------------------------------------------------
// A chunk is 16 KB of K and as much of V: read into shared memory, marked read, then
// written when the chunks whose rows lie there are marked.  Six blocks an SM, so that
// the reads of some run beside the writes of others.  Bound by HBM and by the chain of
// a chunk (ticket, list, page, row, flags): 16 requests cut to 2048 positions, 8 KV heads
// of 128, 238 MB read and written in 51 us, 4.7 TB/s, 70 % of the measured copy rate.

__device__ inline unsigned load_acquire(const unsigned *p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__global__ void __launch_bounds__(kMoveThreads, 6) evict_move_kernel(const EvictArgs a) {
  __shared__ uint4 s_k[kChunkPieces], s_v[kChunkPieces];
  __shared__ unsigned s_ticket, s_end[kMoveSeqs];
  __shared__ int s_after[kMoveSeqs];
  const int tid = threadIdx.x, Hk = a.num_kv_heads, bs = a.block_size, ppr = a.head_bytes / 16;
  pdl_trigger();
  pdl_wait();
  const unsigned chunks = a.head->chunks;
  // (in shared memory: an acquire empties L1, and these loads follow one another)
  const bool few = a.num_seqs <= kMoveSeqs;
  for (int s = tid; few && s < a.num_seqs; s += kMoveThreads) {
    s_end[s] = a.chunk_end[s];
    s_after[s] = min(a.seq_lens[s], a.keep_lens[s]);
  }
  auto end_of = [&](int s) { return few ? s_end[s] : a.chunk_end[s]; };
  for (;;) {
    __syncthreads();  // s_ticket and the rows of the chunk before are read
    if (tid == 0) s_ticket = atomicAdd(&a.head->ticket, 1u);
    __syncthreads();
    const unsigned t = s_ticket;
    if (t >= chunks) return;
    int lo = 0, hi = a.num_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (end_of(mid) > t) hi = mid; else lo = mid + 1;
    }
    const int s = lo, after = few ? s_after[s] : min(a.seq_lens[s], a.keep_lens[s]);
    const int nc = divide(after + a.chunk_rows - 1, a.by_rows);
    const int local = (int)(t - (end_of(s) - (unsigned)(Hk * nc))), h = local / nc, c = local - h * nc;
    const int unit = s * Hk + h;
    const int32_t *bt = a.block_table + (size_t)s * a.max_blocks_per_seq;
    const int32_t *kept = a.kept + (size_t)unit * a.max_seq_len;
    unsigned *ready = a.ready + (size_t)unit * a.max_chunks;
    const int i0 = c * a.chunk_rows, rows = min(a.chunk_rows, after - i0);
    const int below = a.below[(size_t)unit * a.max_chunks + c];
    // -- this chunk's rows into shared memory
    unsigned flags = 0;
    long long into[kMovePieces];  // -1: not moved
#pragma unroll
    for (int u = 0; u < kMovePieces; ++u) {
      const int e = u * kMoveThreads + tid, row = divide(e, a.by_ppr), piece = e - row * ppr;
      into[u] = -1;
      if (row >= rows) continue;
      const int src = kept[i0 + row];
      if (src == i0 + row) continue;
      const long long from = row_offset(bt, src, h, Hk, bs, a.by_bs, a.num_blocks, a.hnd, a.head_bytes),
                      to = row_offset(bt, i0 + row, h, Hk, bs, a.by_bs, a.num_blocks, a.hnd, a.head_bytes);
      if (from < 0 || to < 0) {
        flags |= PA_DEV_BAD_BLOCK;
        continue;
      }
      copy16(s_k + e, a.k_cache + from + piece * 16);
      copy16(s_v + e, a.v_cache + from + piece * 16);
      into[u] = to + piece * 16;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      atomicExch(ready + c, 1u);
    }
    // -- meanwhile its weights (select has read them all)
    for (int i = i0 + tid; i < i0 + rows; i += kMoveThreads) {
      const int from = kept[i], page = bt[divide(from, a.by_bs)],
                lp = divide(i, a.by_bs), dst = bt[lp];
      if (page >= 0 && page < a.num_blocks && dst >= 0 && dst < a.num_blocks)
        a.weights_out[((long long)dst * Hk + h) * bs + (i - lp * bs)] = a.kept_w[(size_t)unit * a.max_seq_len + i];
    }
    // -- the chunks whose rows lie where this one writes: those that hold the kept
    // positions from i0 on, from the first one's chunk on; they were handed out
    // before this one, and mark their rows read without waiting for anything
    bool late = false;
    for (int w = divide(below, a.by_rows) + tid; w < c; w += kMoveThreads) {
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
        if (into[u] < 0) continue;
        *reinterpret_cast<uint4 *>(a.k_cache + into[u]) = s_k[u * kMoveThreads + tid];
        *reinterpret_cast<uint4 *>(a.v_cache + into[u]) = s_v[u * kMoveThreads + tid];
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
  size_t head, chunk_end, ready, kept, kept_w, below, total;
  int chunk_rows, max_chunks;
  bool ok;
};

EvictLayout evict_layout(int head_bytes, int num_seqs, int num_kv_heads, int max_seq_len) {
  EvictLayout l{};
  const long long S = std::max(num_seqs, 1), units = S * num_kv_heads, msl = std::max(max_seq_len, 1);
  l.chunk_rows = std::max(1, kChunkPieces / std::max(head_bytes / 16, 1));
  l.max_chunks = (int)ceil_div_ll(msl, l.chunk_rows);
  l.ok = units < (1ll << 30) && units * l.max_chunks < (1ll << 31) && msl <= kMaxEvictLen;
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
  l.kept_w = take((size_t)units * msl * sizeof(float));
  l.below = take((size_t)units * l.max_chunks * sizeof(int32_t));
  l.total = off;
  return l;
}

cudaError_t launch_select(const EvictArgs &a, int num_sms, cudaStream_t st) {
  const long long units = (long long)a.num_seqs * a.num_kv_heads;
  // Blocks of a cluster: while the grid leaves SMs and a share has work for its
  // threads.
  int C = 1;
  while (C < kMostCluster && units * C * 2 <= num_sms && a.max_seq_len / (2 * C) >= kSelectThreads) C *= 2;
  const long long share = ceil_div_ll(std::max(a.max_seq_len, 1), C);
  // (keys beyond 192 KB are read from memory in every pass, one behind the other: 16
  // requests of up to 131072 positions, 8 KV heads, take 727 us a call, 287 of them the
  // bytes; 16 of up to 65536 323 and 144)
  const int cached = (int)std::min<long long>(share, 48 * 1024);
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  if (dev >= 64 || !(done.load(std::memory_order_acquire) & 1ull << dev)) {  // (16 is beyond the portable 8)
    const cudaError_t n =
        cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (n != cudaSuccess) return n;
  }
  const cudaError_t e = set_smem_attrs_once(evict_select_kernel, 48 * 1024 * 4, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((units + 1) * C));
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = (size_t)cached * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel, a, C, cached);
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
      !aligned(num_freed, 4))
    return PA_ERR_INVALID_ARG;
  const EvictLayout lay = evict_layout(head_dim * es, num_seqs, num_kv_heads, max_seq_len);
  if (!lay.ok) return PA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < lay.total) return PA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return PA_ERR_INVALID_ARG;
  const MemRange from(weights, (long long)num_blocks * num_kv_heads, block_size * 4ll),
      to(weights_out, (long long)num_blocks * num_kv_heads, block_size * 4ll);
  if (any_overlap({{seq_lens_out, num_seqs, 4}, {freed_pages, freed_capacity, 4}, {num_freed, 1, 4}},
                  {{block_table, (long long)num_seqs * max_blocks_per_seq, 4},
                   {seq_lens, num_seqs, 4},
                   {keep_lens, num_seqs, 4}}) ||
      (weights != weights_out && from.meets(to)))
    return PA_ERR_INVALID_ARG;
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
  a.by_bs = fast_div(block_size);
  a.by_ppr = fast_div(a.head_bytes / 16);
  a.by_rows = fast_div(lay.chunk_rows);
  a.chunk_rows = lay.chunk_rows;
  a.max_chunks = lay.max_chunks;
  a.head = reinterpret_cast<EvictHeader *>(ws + lay.head);
  a.chunk_end = reinterpret_cast<unsigned *>(ws + lay.chunk_end);
  a.ready = reinterpret_cast<unsigned *>(ws + lay.ready);
  a.kept = reinterpret_cast<int32_t *>(ws + lay.kept);
  a.kept_w = reinterpret_cast<float *>(ws + lay.kept_w);
  a.below = reinterpret_cast<int32_t *>(ws + lay.below);
  if (launch_select(a, num_sms, st) != cudaSuccess) return PA_ERR_CUDA;
  if (num_seqs == 0) return PA_OK;
  const long long most = (long long)num_seqs * num_kv_heads * lay.max_chunks;
  const long long blocks = std::min<long long>(most, 8ll * num_sms);
  return launch_dependent(evict_move_kernel, dim3((unsigned)blocks), dim3(kMoveThreads), 0, st, a) ==
                 cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

}  // extern "C"
