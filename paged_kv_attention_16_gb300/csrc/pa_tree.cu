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
// Its mask is its own bit and those on the chain p(i), p(p(i)), ... to the root,
// its depth the chain's length.  The chain only goes down, so a thread writes its
// row's words from the top one to the bottom one as it goes.
constexpr int kMaskThreads = 128;

struct MaskArgs {
  const int32_t *parents, *qsl, *seq_lens;
  unsigned long long *mask;
  int32_t *positions;
  int num_seqs, num_tokens, words;
  unsigned int *status;
};

__global__ void __launch_bounds__(kMaskThreads) tree_masks_kernel(const MaskArgs a) {
  const int S = a.num_seqs, T = a.num_tokens, tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  int bad = 0;
  for (int s = tid; s < S; s += kMaskThreads) {
    const int q0 = a.qsl[s], q1 = a.qsl[s + 1];
    if (q1 < q0 || (s == 0 && q0 != 0) || (s == S - 1 && q1 > T)) bad = 1;
  }
  bad = __syncthreads_or(bad);
  if (bad && blockIdx.x == 0 && tid == 0) atomicOr(a.status, PA_DEV_BAD_QSL);
  for (long long t64 = (long long)blockIdx.x * kMaskThreads + tid; t64 < T;
       t64 += (long long)gridDim.x * kMaskThreads) {
    const int t = (int)t64;
    unsigned long long *row = a.mask + (size_t)t * a.words;
    int w = a.words - 1, position = 0;  // the highest word not yet written
    unsigned flags = 0;
    if (!bad && S > 0 && t < a.qsl[S]) {
      int lo = 0, hi = S - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.qsl[mid] <= t) lo = mid; else hi = mid - 1;
      }
      const int q0 = a.qsl[lo], q_len = a.qsl[lo + 1] - q0, i = t - q0;
      const int len = a.seq_lens ? a.seq_lens[lo] : q_len;
      if (len < 0) flags |= PA_DEV_BAD_SEQLEN;
      else if (q_len > len || q_len > 64ll * a.words) flags |= PA_DEV_BAD_QLEN;
      if (!flags) {
        int depth = 0, node = i;
        unsigned long long bits = 0;
        for (;;) {
          for (; w > node >> 6; --w) {
            row[w] = bits;
            bits = 0;
          }
          bits |= 1ull << (node & 63);
          const int up = __ldg(a.parents + q0 + node);
          if (up < -1 || up >= node) flags = PA_DEV_BAD_TREE;
          if (flags || up < 0) break;
          node = up;
          ++depth;
        }
        if (flags) {
          w = a.words - 1;  // the whole row again, as zeros
        } else {
          row[w--] = bits;
          position = len - q_len + depth;
        }
      }
    }
    for (; w >= 0; --w) row[w] = 0;
    if (a.positions) a.positions[t] = position;
    if (flags) atomicOr(a.status, flags);
  }
}

// ---------------------------------------------------------------------------
// pa_cache_accept
// ---------------------------------------------------------------------------
// Row prefix + path[k] of every KV head goes to prefix + k <= prefix + path[k],
// in place.  A warp takes one KV head of a request and walks its path upwards,
// some rows at a time, all of them read before the first is written; what a step
// writes lies below everything that later steps read.  Block 0 lists the pages.
constexpr int kAcceptThreads = 256;
constexpr int kAcceptPieces = 4;  // 16-byte pieces of K, and of V, that a lane has in flight

struct AcceptArgs {
  uint8_t *k_cache, *v_cache;
  const int32_t *block_table, *seq_lens, *qsl, *path, *path_lens;
  int32_t *seq_lens_out;
  FreeList free;
  int num_seqs, num_tokens, max_path, num_kv_heads, head_bytes, block_size, max_blocks_per_seq,
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

__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(const AcceptArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_trigger();
  pdl_wait();
  const int warps = gridDim.x * (kAcceptThreads / 32);
  const int bs = a.block_size, Hk = a.num_kv_heads, ppr = a.head_bytes / 16;  // pieces a row
  for (long long item = blockIdx.x * (kAcceptThreads / 32) + warp; item < (long long)a.num_seqs * Hk;
       item += warps) {
    const int s = (int)(item / Hk), h = (int)(item - (long long)s * Hk);
    int prefix, n;
    unsigned flags = 0;
    if (accepted_len(a, s, prefix, n, flags) < 0) continue;  // (block 0 reports it)
    const int q_len = a.seq_lens[s] - prefix;
    const int32_t *path = a.path + (size_t)s * a.max_path;
    if (!path_ok(path, n, q_len, lane)) continue;
    const int32_t *bt = a.block_table + (size_t)s * a.max_blocks_per_seq;
    const int total = n * ppr;
    for (int e0 = 0; e0 < total; e0 += 32 * kAcceptPieces) {
      uint4 k[kAcceptPieces], v[kAcceptPieces];
      long long to[kAcceptPieces];
#pragma unroll
      for (int u = 0; u < kAcceptPieces; ++u) {
        const int e = e0 + u * 32 + lane;
        to[u] = -1;
        if (e >= total) continue;
        const int i = divide(e, a.by_ppr), c = e - i * ppr, from = __ldg(path + i);
        if (from == i) continue;
        const long long src = row_offset(bt, prefix + from, h, Hk, bs, a.by_bs, a.num_blocks, a.hnd, a.head_bytes);
        const long long dst = row_offset(bt, prefix + i, h, Hk, bs, a.by_bs, a.num_blocks, a.hnd, a.head_bytes);
        if (src < 0 || dst < 0) {
          flags |= PA_DEV_BAD_BLOCK;
          continue;
        }
        to[u] = dst + c * 16;
        k[u] = *reinterpret_cast<const uint4 *>(a.k_cache + src + c * 16);
        v[u] = *reinterpret_cast<const uint4 *>(a.v_cache + src + c * 16);
      }
      __syncwarp();  // all of the step's rows are read
#pragma unroll
      for (int u = 0; u < kAcceptPieces; ++u) {
        if (to[u] < 0) continue;
        *reinterpret_cast<uint4 *>(a.k_cache + to[u]) = k[u];
        *reinterpret_cast<uint4 *>(a.v_cache + to[u]) = v[u];
      }
    }
    if (flags) atomicOr(a.status, flags);
  }
  if (blockIdx.x != gridDim.x - 1) return;
  // the last block: new lengths and the pages that are free again
  auto lens = [&](int s, int &before, int &after) {
    int prefix, n;
    unsigned flags = 0;
    before = a.seq_lens[s];
    after = accepted_len(a, s, prefix, n, flags);
    if (after >= 0) {  // (one thread, the whole path)
      const int32_t *path = a.path + (size_t)s * a.max_path;
      int last = -1;
      for (int i = 0; i < n; ++i) {
        const int x = __ldg(path + i);
        if (x <= last || x >= before - prefix) {
          flags |= PA_DEV_BAD_TREE;
          break;
        }
        last = x;
      }
    }
    if (flags) {
      atomicOr(a.status, flags);
      after = before;
    }
    a.seq_lens_out[s] = after;
  };
  list_free_pages<kAcceptThreads>(a.free, a.block_table, a.max_blocks_per_seq, bs, a.num_blocks,
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
  const long long blocks = std::min<long long>(ceil_div_ll(num_tokens, kMaskThreads), 8ll * num_sms);
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
  if ((long long)head_dim * es % 16 != 0 || (long long)head_dim * es > kMaxHeadBytes)
    return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0 && !num_freed) return PA_OK;
  if (num_seqs > 0 &&
      (!k_cache || !v_cache || !block_table || !seq_lens || !query_start_loc || !path_lens ||
       !seq_lens_out || (max_path > 0 && !path) || max_blocks_per_seq == 0 || num_blocks == 0))
    return PA_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(query_start_loc, 4) || !aligned(path, 4) ||
      !aligned(path_lens, 4) || !aligned(seq_lens_out, 4) || !aligned(freed_pages, 4) ||
      !aligned(num_freed, 4) || seq_lens_out == seq_lens)
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
  const long long warps = (long long)num_seqs * num_kv_heads;
  const long long blocks = std::min<long long>(ceil_div_ll(warps, kAcceptThreads / 32) + 1, 8ll * num_sms);
  return launch_dependent(accept_kernel, dim3((unsigned)blocks), dim3(kAcceptThreads), 0, st, a) ==
                 cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}
