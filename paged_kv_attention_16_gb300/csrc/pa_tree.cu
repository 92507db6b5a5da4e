// pa_tree.cu -- drafted trees of tokens: the masks and positions of their nodes
// (pa_tree_masks), and what follows the verification: the accepted path's rows
// moved down to the positions behind the cached ones (pa_cache_accept).
#include <algorithm>

#include "pa_evict.h"

namespace pa {
namespace {

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// ---------------------------------------------------------------------------
// pa_tree_masks
// ---------------------------------------------------------------------------
// Token i of a request has parent p(i) < i among the request's new tokens, or -1.
// Its mask is its own bit and those on the chain p(i), p(p(i)), ... to the root, its
// depth their number.  Chains are followed by doubling: with m(i) the bits of i and
// its next 2^k - 1 ancestors and u(i) the ancestor behind those,
//   m(i) |= m(u(i)),  u(i) = u(u(i)),
// so a chain of 250 takes 8 steps instead of 250 loads one behind the other.  A
// request of up to 32 tokens is a warp's (shuffles), one of up to kMaskTokens a
// block's (shared memory); beyond that a thread walks its token's chain, which only
// goes down, and writes its row's words from the top one to the bottom one.
// Bound by latency (lengths, parents, the steps): 64 trees of up to 16 tokens 2.8 us in
// a graph, 256 of up to 250 9.0 (27 with a chain a thread for all of them).  Beyond
// kMaskTokens the chain's loads follow one another: 64 trees of 512 tokens, each under a
// random one before it, 7.5 us, as one chain 87; of 1000 tokens 17 and 284.
constexpr int kMaskThreads = 256, kMaskTokens = 256, kMaskWords = kMaskTokens / 64;

struct MaskArgs {
  const int32_t *parents, *qsl, *seq_lens;
  unsigned long long *mask;
  int32_t *positions;
  int num_seqs, num_tokens, words, per_block;  // requests of a block
  unsigned int *status;
};

// What u(i) ends at: the root, or a parent that is none.
constexpr int kRoot = -1, kBadParent = -2;

__device__ inline int parent_of(const MaskArgs &a, int q0, int i) {
  const int up = a.parents[q0 + i];
  return up >= i || up < -1 ? kBadParent : up;
}

__global__ void __launch_bounds__(kMaskThreads) tree_masks_kernel(const MaskArgs a) {
  __shared__ unsigned long long s_mask[2][kMaskTokens][kMaskWords];
  __shared__ int s_up[2][kMaskTokens];
  const int S = a.num_seqs, T = a.num_tokens, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();  // (the next kernel's blocks come in behind these: 256 trees one call
               // after the other 8.2 us, 14.1 with a trigger here)
  int bad = 0;
  for (int s = tid; s < S; s += kMaskThreads) {
    const int q0 = a.qsl[s], q1 = a.qsl[s + 1];
    if (q1 < q0 || (s == 0 && q0 != 0) || (s == S - 1 && q1 > T)) bad = 1;
  }
  bad = __syncthreads_or(bad);
  if (bad && blockIdx.x == 0 && tid == 0) atomicOr(a.status, PA_DEV_BAD_QSL);
  // -- rows that belong to no request, or all of them
  const long long n = bad || S == 0 ? 0 : a.qsl[S];
  for (long long e = n * a.words + blockIdx.x * kMaskThreads + tid; e < (long long)T * a.words;
       e += (long long)gridDim.x * kMaskThreads)
    a.mask[e] = 0;
  if (a.positions)
    for (long long t = n + blockIdx.x * kMaskThreads + tid; t < T; t += (long long)gridDim.x * kMaskThreads)
      a.positions[t] = 0;
  if (bad) return;

  for (int base = blockIdx.x * a.per_block; base < S; base += gridDim.x * a.per_block) {
    for (int k = 0; k < min(a.per_block, S - base); ++k) {
      const int s = base + k, q0 = a.qsl[s], q_len = a.qsl[s + 1] - q0;
      if (q_len == 0 || (q_len <= 32 && k % (kMaskThreads / 32) != warp)) continue;
      const int len = a.seq_lens ? a.seq_lens[s] : q_len;
      unsigned flags = len < 0 ? PA_DEV_BAD_SEQLEN : q_len > len || q_len > 64ll * a.words ? PA_DEV_BAD_QLEN : 0;
      unsigned long long *rows = a.mask + (size_t)q0 * a.words;
      auto finish = [&](int i, bool good, int ancestors) {
        if (a.positions) a.positions[q0 + i] = good ? len - q_len + ancestors : 0;
      };
      if (flags) {  // (the same for all that are here)
        const int from = q_len <= 32 ? lane : tid, step = q_len <= 32 ? 32 : kMaskThreads;
        for (long long e = from; e < (long long)q_len * a.words; e += step) rows[e] = 0;
        for (int i = from; i < q_len; i += step) finish(i, false, 0);
      } else if (q_len <= 32) {
        const int i = lane;
        unsigned m = i < q_len ? 1u << i : 0u;
        int up = i < q_len ? parent_of(a, q0, i) : kRoot;
        if (up == kBadParent) flags = PA_DEV_BAD_TREE;
        while (__any_sync(0xffffffffu, up >= 0)) {
          const unsigned more = __shfl_sync(0xffffffffu, m, max(up, 0));
          const int above = __shfl_sync(0xffffffffu, up, max(up, 0));
          if (up >= 0) {
            m |= more;
            up = above;
          }
        }
        if (i < q_len) {
          const bool good = up == kRoot;
          rows[(size_t)i * a.words] = good ? m : 0u;
          for (int w = 1; w < a.words; ++w) rows[(size_t)i * a.words + w] = 0;
          finish(i, good, __popc(m) - 1);
        }
      } else if (q_len <= kMaskTokens) {
        const int W = (q_len + 63) >> 6;
        __syncthreads();  // the request before is read
        for (int i = tid; i < q_len; i += kMaskThreads) {
          const int up = parent_of(a, q0, i);
          if (up == kBadParent) flags = PA_DEV_BAD_TREE;
          s_up[0][i] = up;
#pragma unroll
          for (int w = 0; w < kMaskWords; ++w) s_mask[0][i][w] = w == i >> 6 ? 1ull << (i & 63) : 0ull;
        }
        int cur = 0, more = 1;
        while (__syncthreads_or(more)) {
          more = 0;
          for (int i = tid; i < q_len; i += kMaskThreads) {
            const int up = s_up[cur][i], from = max(up, 0);
            const int above = up >= 0 ? s_up[cur][from] : up;
            s_up[cur ^ 1][i] = above;
            more |= above >= 0;
#pragma unroll
            for (int w = 0; w < kMaskWords; ++w)
              s_mask[cur ^ 1][i][w] = s_mask[cur][i][w] | (up >= 0 ? s_mask[cur][from][w] : 0ull);
          }
          cur ^= 1;
        }
        for (int i = tid; i < q_len; i += kMaskThreads) {
          const bool good = s_up[cur][i] == kRoot;
          int ancestors = -1;
          for (int w = 0; w < a.words; ++w) {
            const unsigned long long m = w < W ? s_mask[cur][i][w] : 0ull;
            ancestors += __popcll(m);
            rows[(size_t)i * a.words + w] = good ? m : 0ull;
          }
          finish(i, good, ancestors);
        }
      } else {
        for (int i = tid; i < q_len; i += kMaskThreads) {
          unsigned long long *row = rows + (size_t)i * a.words, bits = 0;
          int w = a.words - 1, depth = 0, node = i;  // w: the highest word not yet written
          for (;;) {
            for (; w > node >> 6; --w) {
              row[w] = bits;
              bits = 0;
            }
            bits |= 1ull << (node & 63);
            const int up = parent_of(a, q0, node);
            if (up < 0) {
              node = up;
              break;
            }
            node = up;
            ++depth;
          }
          const bool good = node == kRoot;
          if (good) {
            row[w--] = bits;
          } else {
            flags = PA_DEV_BAD_TREE;
            w = a.words - 1;  // the whole row again, as zeros
          }
          for (; w >= 0; --w) row[w] = 0;
          finish(i, good, depth);
        }
      }
      if (flags) atomicOr(a.status, flags);
    }
  }
}

// ---------------------------------------------------------------------------
// pa_cache_accept
// ---------------------------------------------------------------------------
// Row prefix + path[k] of every KV head goes to prefix + k <= prefix + path[k],
// in place.  A block takes one KV head of a request and walks its path upwards, some
// rows at a time, all of them read before the first is written; what a step writes
// lies below everything that later steps read.  500 paths of up to 200 rows of 256
// bytes, four KV heads, take 39 us: 181 MB read and written, 4.6 TB/s (a step's rows are
// awaited before they are written, and written before the next step's are asked for;
// 75 us with pages and rows loaded one behind the other).  The block of KV head 0 writes the new
// length; a second launch lists the pages from the lengths.  Where the paths are few
// and short in all (kListEntries) a block more of the first one lists them, looking
// through every path itself.  Two launches against one: 1 path of 8 4.2 and 2.7 us, 64 of
// 8 5.6 and 3.7, 256 of 8 7.8 and 7.5, 500 of 8 11.6 and 14.1, 128 of 32 7.2 and 7.2.
constexpr int kAcceptThreads = 128;
constexpr long long kListEntries = 2048;
constexpr int kAcceptPieces = 4;  // 16-byte pieces of K, and of V, that a thread copies at a time

struct AcceptArgs {
  uint8_t *k_cache, *v_cache;
  const int32_t *block_table, *seq_lens, *qsl, *path, *path_lens;
  int32_t *seq_lens_out;
  FreeList free;
  int num_seqs, max_path, num_kv_heads, head_bytes, block_size, max_blocks_per_seq,
      num_blocks, hnd;
  FastDiv by_bs, by_ppr;
  unsigned int *status;
};

// The request's new length; -1 where its metadata is bad (nothing moves then).
__device__ inline int accepted_len(const AcceptArgs &a, int s, int &prefix, int &n, unsigned &flags) {
  const int len = a.seq_lens[s], q0 = a.qsl[s], q_len = a.qsl[s + 1] - q0;
  n = a.path_lens[s];
  prefix = len - q_len;
  if (q_len < 0 || q0 < 0) flags |= PA_DEV_BAD_QSL;
  else if (len < 0 || len > (long long)a.max_blocks_per_seq * a.block_size) flags |= PA_DEV_BAD_SEQLEN;
  else if (q_len > len) flags |= PA_DEV_BAD_QLEN;
  else if (n < 0 || n > q_len || n > a.max_path) flags |= PA_DEV_BAD_TREE;
  else return prefix + n;
  return -1;
}

// Whether path[0 .. n) rises strictly within [0, q_len): of the entries from `from` on,
// every `step`-th.
__device__ inline bool path_rises(const int32_t *path, int n, int q_len, int from, int step) {
  bool ok = true;
#pragma unroll 8
  for (int i = from; i < n; i += step) {
    const int x = path[i], last = i > 0 ? path[i - 1] : -1;
    ok &= x > last && x < q_len;
  }
  return ok;
}

template <bool LIST>  // whether the block behind the movers lists the pages
__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(const AcceptArgs a, int movers) {
  __shared__ uint4 s_k[kAcceptThreads * kAcceptPieces], s_v[kAcceptThreads * kAcceptPieces];
  const int tid = threadIdx.x, bs = a.block_size, Hk = a.num_kv_heads, ppr = a.head_bytes / 16;  // pieces a row
  pdl_trigger();
  pdl_wait();
  if (LIST && (int)blockIdx.x == movers) {
    auto lens = [&](int s, int &before, int &after) {
      int prefix, n;
      unsigned flags = 0;  // (the others report them)
      before = a.seq_lens[s];
      after = accepted_len(a, s, prefix, n, flags);
      if (after < 0 || !path_rises(a.path + (size_t)s * a.max_path, n, before - prefix, 0, 1)) after = before;
    };
    list_free_pages<kAcceptThreads>(a.free, a.block_table, a.max_blocks_per_seq, bs, a.num_blocks,
                                    a.num_seqs, a.status, lens);
    return;
  }
  unsigned bad = 0;
  for (long long item = blockIdx.x; item < (long long)a.num_seqs * Hk; item += movers) {
    const int s = (int)(item / Hk), h = (int)(item - (long long)s * Hk);
    int prefix, n;
    unsigned flags = 0;
    const int32_t *path = a.path + (size_t)s * a.max_path;
    int after = accepted_len(a, s, prefix, n, flags);  // (the same for all threads)
    if (after >= 0 && !__syncthreads_and(path_rises(path, n, a.seq_lens[s] - prefix, tid, kAcceptThreads))) {
      flags = PA_DEV_BAD_TREE;
      after = -1;
    }
    if (h == 0 && tid == 0) {
      a.seq_lens_out[s] = after < 0 ? a.seq_lens[s] : after;
      if (flags) atomicOr(a.status, flags);
    }
    if (after < 0) continue;
    const int32_t *bt = a.block_table + (size_t)s * a.max_blocks_per_seq;
    const int total = n * ppr;
    for (int e0 = 0; e0 < total; e0 += kAcceptThreads * kAcceptPieces) {
      __syncthreads();  // the rows of the step before are written
      // (the pieces' path entries, pages and rows: three latencies for all of them)
      int row[kAcceptPieces], from[kAcceptPieces], page[kAcceptPieces];
#pragma unroll
      for (int u = 0; u < kAcceptPieces; ++u) {
        const int e = e0 + u * kAcceptThreads + tid;
        row[u] = divide(min(e, total - 1), a.by_ppr);
        from[u] = path[row[u]];
        if (e >= total) from[u] = row[u];  // (stays where it is)
      }
#pragma unroll
      for (int u = 0; u < kAcceptPieces; ++u) page[u] = bt[divide(prefix + from[u], a.by_bs)];
#pragma unroll
      for (int u = 0; u < kAcceptPieces; ++u) {
        if (from[u] == row[u]) continue;
        if (page[u] < 0 || page[u] >= a.num_blocks) {
          bad = PA_DEV_BAD_BLOCK;
          from[u] = row[u];
          continue;
        }
        const int i = u * kAcceptThreads + tid, pos = prefix + from[u], c = e0 + i - row[u] * ppr;
        const long long at = row_at(page[u], pos - divide(pos, a.by_bs) * bs, h, Hk, bs, a.hnd) * a.head_bytes + c * 16;
        copy16(s_k + i, a.k_cache + at);
        copy16(s_v + i, a.v_cache + at);
      }
#pragma unroll
      for (int u = 0; u < kAcceptPieces; ++u) page[u] = bt[divide(prefix + row[u], a.by_bs)];
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncthreads();  // all of the step's rows are read
#pragma unroll
      for (int u = 0; u < kAcceptPieces; ++u) {
        if (from[u] == row[u]) continue;
        if (page[u] < 0 || page[u] >= a.num_blocks) {
          bad = PA_DEV_BAD_BLOCK;
          continue;
        }
        const int i = u * kAcceptThreads + tid, pos = prefix + row[u], c = e0 + i - row[u] * ppr;
        const long long at = row_at(page[u], pos - divide(pos, a.by_bs) * bs, h, Hk, bs, a.hnd) * a.head_bytes + c * 16;
        *reinterpret_cast<uint4 *>(a.k_cache + at) = s_k[i];
        *reinterpret_cast<uint4 *>(a.v_cache + at) = s_v[i];
      }
    }
  }
  if (bad) atomicOr(a.status, bad);
}

// The pages behind the new lengths: one block.
constexpr int kFreeThreads = 512;
__global__ void __launch_bounds__(kFreeThreads) free_pages_kernel(const AcceptArgs a) {
  pdl_trigger();
  pdl_wait();
  auto lens = [&](int s, int &before, int &after) {
    before = a.seq_lens[s];
    after = a.seq_lens_out[s];
  };
  list_free_pages<kFreeThreads>(a.free, a.block_table, a.max_blocks_per_seq, a.block_size, a.num_blocks,
                                a.num_seqs, a.status, lens);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_tree_masks(const int32_t *parents, const int32_t *query_start_loc,
                                   const int32_t *seq_lens, uint64_t *tree_mask,
                                   int32_t *positions, void *stream, int num_seqs, int num_tokens,
                                   int mask_words) {
  if (num_seqs < 0 || num_tokens < 0 || mask_words <= 0) return PA_ERR_INVALID_ARG;
  if (num_tokens > 0 && (!tree_mask || !parents)) return PA_ERR_INVALID_ARG;
  if (num_seqs > 0 && !query_start_loc) return PA_ERR_INVALID_ARG;
  if (positions && num_seqs > 0 && !seq_lens) return PA_ERR_INVALID_ARG;
  if (!aligned(parents, 4) || !aligned(query_start_loc, 4) || !aligned(seq_lens, 4) ||
      !aligned(positions, 4) || !aligned(tree_mask, 8))
    return PA_ERR_INVALID_ARG;
  if (num_tokens == 0) return PA_OK;
  if (num_tokens > 1 << 30 || num_seqs > 1 << 30) return PA_ERR_UNSUPPORTED;
  if (any_overlap({{tree_mask, (long long)num_tokens * mask_words, 8}, {positions, num_tokens, 4}},
                  {{parents, num_tokens, 4}, {query_start_loc, num_seqs + 1ll, 4}, {seq_lens, num_seqs, 4}}))
    return PA_ERR_INVALID_ARG;
  MaskArgs a{};
  void *ws = nullptr;
  int num_sms = 0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const pa_status s = device_resources(st, 0, &ws, &a.status, &num_sms);
  if (s != PA_OK) return s;
  a.parents = parents;
  a.qsl = query_start_loc;
  a.seq_lens = seq_lens;
  a.mask = reinterpret_cast<unsigned long long *>(tree_mask);
  a.positions = positions;
  a.num_seqs = num_seqs;
  a.num_tokens = num_tokens;
  a.words = mask_words;
  // A block a request, or as many as it has warps where there are that many requests.
  a.per_block = (int)std::min<long long>(std::max<long long>(num_seqs / (4ll * num_sms), 1), kMaskThreads / 32);
  const long long blocks = std::min<long long>(std::max<long long>(ceil_div_ll(num_seqs, a.per_block), 1), 8ll * num_sms);
  return launch_dependent(tree_masks_kernel, dim3((unsigned)blocks), dim3(kMaskThreads), 0, st, a) ==
                 cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

extern "C" pa_status pa_cache_accept(void *k_cache, void *v_cache, const int32_t *block_table,
                                     const int32_t *seq_lens, const int32_t *query_start_loc,
                                     const int32_t *path, const int32_t *path_lens,
                                     int32_t *seq_lens_out, int32_t *freed_pages,
                                     int32_t *num_freed, int num_kv_heads, int head_dim,
                                     int block_size, void *stream, pa_dtype dtype, int num_seqs,
                                     int max_path, int max_blocks_per_seq, int num_blocks,
                                     int freed_capacity, pa_kv_layout kv_layout) {
  if (num_seqs < 0 || max_path < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
      max_blocks_per_seq < 0 || num_blocks < 0 || freed_capacity < 0 ||
      (dtype != PA_F32 && dtype != PA_BF16) || (kv_layout != PA_KV_NHD && kv_layout != PA_KV_HND))
    return PA_ERR_INVALID_ARG;
  if ((num_freed == nullptr) != (freed_pages == nullptr) || (!freed_pages && freed_capacity > 0))
    return PA_ERR_INVALID_ARG;
  const int es = dtype == PA_F32 ? 4 : 2;
  if ((long long)head_dim * es % 16 != 0 || (long long)head_dim * es > kMaxHeadBytes ||
      (long long)max_path * (head_dim * es / 16) > 1 << 30 ||  // pieces of a path, counted in 32 bits
      num_seqs > 1 << 30)
    return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0 && !num_freed) return PA_OK;
  if (num_seqs > 0 &&
      (!k_cache || !v_cache || !block_table || !seq_lens || !query_start_loc || !path_lens ||
       !seq_lens_out || (max_path > 0 && !path) || max_blocks_per_seq == 0 || num_blocks == 0))
    return PA_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(query_start_loc, 4) || !aligned(path, 4) ||
      !aligned(path_lens, 4) || !aligned(seq_lens_out, 4) || !aligned(freed_pages, 4) ||
      !aligned(num_freed, 4))
    return PA_ERR_INVALID_ARG;
  if (any_overlap({{seq_lens_out, num_seqs, 4}, {freed_pages, freed_capacity, 4}, {num_freed, 1, 4}},
                  {{block_table, (long long)num_seqs * max_blocks_per_seq, 4},
                   {seq_lens, num_seqs, 4},
                   {query_start_loc, num_seqs + 1ll, 4},
                   {path, (long long)num_seqs * max_path, 4},
                   {path_lens, num_seqs, 4}}))
    return PA_ERR_INVALID_ARG;
  AcceptArgs a{};
  void *ws = nullptr;
  int num_sms = 0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const pa_status s = device_resources(st, 0, &ws, &a.status, &num_sms);
  if (s != PA_OK) return s;
  a.k_cache = static_cast<uint8_t *>(k_cache);
  a.v_cache = static_cast<uint8_t *>(v_cache);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.qsl = query_start_loc;
  a.path = path;
  a.path_lens = path_lens;
  a.seq_lens_out = seq_lens_out;
  a.free = FreeList{freed_pages, num_freed, freed_capacity};
  a.num_seqs = num_seqs;
  a.max_path = max_path;
  a.num_kv_heads = num_kv_heads;
  a.head_bytes = head_dim * es;
  a.block_size = block_size;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.hnd = kv_layout == PA_KV_HND;
  a.by_bs = fast_div(block_size);
  a.by_ppr = fast_div(a.head_bytes / 16);
  const int movers = (int)std::min<long long>((long long)num_seqs * num_kv_heads, 16ll * num_sms);
  const bool list_here = num_freed && (long long)num_seqs * max_path <= kListEntries;
  if (movers + list_here > 0 &&
      launch_dependent(list_here ? accept_kernel<true> : accept_kernel<false>,
                       dim3((unsigned)(movers + list_here)), dim3(kAcceptThreads), 0, st, a, movers) != cudaSuccess)
    return PA_ERR_CUDA;
  if (num_freed && !list_here &&
      launch_dependent(free_pages_kernel, dim3(1), dim3(kFreeThreads), 0, st, a) != cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
}
