// pa_slots.cu -- a serving step's bookkeeping on the device: the block-table
// rows and the slot map of its new tokens (pa_block_tables), and the KV-cache
// write that goes by such a map (pa_cache_write_slots).
#include "pa_internal.h"

namespace pa {
namespace {

// ---------------------------------------------------------------------------
// pa_block_tables
// ---------------------------------------------------------------------------
// With L_s = seq_lens[s] and q_s new tokens among them, request s holds
// held = ceil((L_s - q_s) / bs) pages and needs need = ceil(L_s / bs) - held
// more; begin = the exclusive sum of need over the requests before it.  It is
// served when begin + need fits the free pages, and its page held + j is then
// free_pages[start + begin + j].  A token at position pos has the slot
// page(pos / bs) * bs + pos % bs.
//
// One launch, and no block waits for another: every block scans the lengths
// of all requests itself (from L2; 512 requests are one scan step) and keeps
// each request's first token, length and first free page in shared memory,
// then takes a share of the tokens (request by binary search).  The token at
// the start of a fresh page writes that page's table entry: pages held before
// are only read, fresh ones only written, so no entry is both.  What bounds it
// is the chain of its loads: the lengths, then the pages (calls in a graph: 64
// requests of one new token 2.7 us, 512 of up to 2048 9.9 us).
constexpr int kTablesThreads = 512;
constexpr int kTablesMaxSeqs = 16384;  // 12 bytes of shared memory a request
constexpr int kTokensPerThread = 4;    // tokens a thread takes at a time: each finds its page
                                       // behind the one before, the results are stored together
constexpr int kBadRequest = -1;        // in place of a free-page index: bad metadata,
constexpr int kUnserved = -2;          // or no pages left

struct TablesArgs {
  const int32_t *seq_lens, *qsl, *free_pages, *free_start;
  int32_t *free_end, *block_table, *positions;
  int64_t *slots;
  int num_seqs, num_tokens, block_size, max_blocks_per_seq, num_blocks, num_free;
  unsigned int *status;
};

__global__ void __launch_bounds__(kTablesThreads) block_tables_kernel(const TablesArgs a) {
  extern __shared__ int s_dyn[];
  constexpr int NW = kTablesThreads / 32;
  const int S = a.num_seqs, T = a.num_tokens, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int *s_qsl = s_dyn;            // [S + 1]
  int *s_len = s_qsl + S + 1;    // [S]
  int *s_first = s_len + S;      // [S] index of the request's first free page
  __shared__ int s_warp[2][NW];
  __shared__ int s_taken;
  const unsigned bs = a.block_size;
  const bool grow = a.free_start != nullptr;
  pdl_trigger();
  pdl_wait();
  if (tid == 0) s_taken = 0;
  const int start = grow ? *a.free_start : 0;

  // -- the pages each request lacks, their sum over the requests before it
  // (at most one a new token, so it fits 32 bits), and whether they are there
  int bad = 0, carry = 0, taken = 0, turn = 0;
  unsigned flags = 0;
  for (int base = 0; base < S; base += kTablesThreads, turn ^= 1) {
    const int s = base + tid;
    int need = 0;
    bool ok = false;
    if (s < S) {
      const int q0 = a.qsl[s], q1 = a.qsl[s + 1], len = a.seq_lens[s], q = q1 - q0;
      if (q1 < q0 || (s == 0 && q0 != 0) || (s == S - 1 && q1 > T)) bad = 1;
      s_qsl[s] = q0;
      s_len[s] = len;
      if (s == S - 1) s_qsl[S] = q1;
      const unsigned pages = ((unsigned)len + bs - 1) / bs;
      if (len < 0 || pages > (unsigned)a.max_blocks_per_seq) flags |= PA_DEV_BAD_SEQLEN;
      else if (q > len) flags |= PA_DEV_BAD_QLEN;
      else ok = true;
      if (ok && grow && q > 0) need = (int)(pages - ((unsigned)(len - q) + bs - 1) / bs);
    }
    int end = need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += v;
    }
    if (lane == 31) s_warp[turn][warp] = end;
    __syncthreads();
    int before = carry;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const int v = s_warp[turn][w];
      if (w < warp) before += v;
      carry += v;
    }
    end += before;
    if (s < S) {
      const bool served = need == 0 || (start >= 0 && end <= a.num_free - start);
      s_first[s] = !ok ? kBadRequest : !served ? kUnserved : need ? start + end - need : 0;
      if (ok && !served) flags |= PA_DEV_NO_PAGES;
      if (ok && served && need > 0) taken = end;
    }
  }
  if (taken && blockIdx.x == 0) atomicMax(&s_taken, taken);
  const bool qsl_bad = __syncthreads_or(bad) != 0;
  if (blockIdx.x == 0) {
    if (qsl_bad) flags = PA_DEV_BAD_QSL;
    if (flags) atomicOr(a.status, flags);
    if (grow && tid == 0) *a.free_end = start + (qsl_bad ? 0 : s_taken);
  }

  // -- the tokens
  const int n = S > 0 && !qsl_bad ? s_qsl[S] : 0;  // those that belong to a request
  constexpr int U = kTokensPerThread;
  const long long step = (long long)gridDim.x * kTablesThreads * U;
  for (long long t0 = (long long)blockIdx.x * kTablesThreads * U + tid; t0 < T; t0 += step) {
    int pos[U], page[U], fresh[U], entry_s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long t64 = t0 + u * kTablesThreads;
      const int t = (int)t64;
      pos[u] = 0;
      page[u] = -2;  // no slot
      fresh[u] = 0;
      if (t64 < n) {
        int lo = 0, hi = S - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (s_qsl[mid] <= t) lo = mid; else hi = mid - 1;
        }
        const int first = s_first[lo];
        entry_s[u] = lo;
        if (first != kBadRequest) {
          const int q0 = s_qsl[lo], prefix = s_len[lo] - (s_qsl[lo + 1] - q0);
          pos[u] = prefix + t - q0;
          if (first != kUnserved) {
            const unsigned j = (unsigned)pos[u] / bs, held = ((unsigned)prefix + bs - 1) / bs;
            fresh[u] = grow && j >= held;
            page[u] = fresh[u] ? __ldg(a.free_pages + first + (j - held))
                               : a.block_table[(size_t)lo * a.max_blocks_per_seq + j];
            if (page[u] < 0 || page[u] >= a.num_blocks) {
              page[u] = -1;
              atomicOr(a.status, PA_DEV_BAD_BLOCK);
            }
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long t = t0 + u * kTablesThreads;
      if (t >= T) break;
      const unsigned j = (unsigned)pos[u] / bs, off = pos[u] - j * bs;
      if (fresh[u] && off == 0) a.block_table[(size_t)entry_s[u] * a.max_blocks_per_seq + j] = page[u];
      a.slots[t] = page[u] < 0 ? -1 : (long long)page[u] * bs + off;
      if (a.positions) a.positions[t] = pos[u];
    }
  }
}

// ---------------------------------------------------------------------------
// pa_cache_write_slots
// ---------------------------------------------------------------------------
// A copy: 4 x the row bytes of a token move (K and V, read and written), so
// HBM bounds it.  One warp takes one token's K and V rows, 32 (or 16) bytes a
// lane at a time, two pieces of each row loaded before the first is stored.
// 32,730 tokens of 2 KB rows take 38 us (ncu, serialised): 7.1 TB/s where a plain
// copy reads and writes 6.8, part of the writes being in L2 still.  4099 tokens of
// 1 KB rows, of which a warp has one piece of each in flight, take 3.5 us a call in
// a graph.  A decode step's 64 tokens take 2.0, the latency of the slot, then of
// its rows.
constexpr int kWriteThreads = 256;

struct SlotWriteArgs {
  const uint8_t *k_new, *v_new;
  uint8_t *k_cache, *v_cache;
  const int64_t *slots;
  long long k_stride, v_stride;  // bytes from one token's row to the next
  long long num_slots;
  int num_tokens, row_bytes, head_bytes, block_size, num_kv_heads, hnd;
  unsigned int *status;
};

template <int VEC>
struct Piece {
  uint32_t w[VEC / 4];
};

template <int VEC>
__device__ inline Piece<VEC> load_piece(const uint8_t *src);
template <>
__device__ inline Piece<16> load_piece<16>(const uint8_t *src) {
  const uint4 v = *reinterpret_cast<const uint4 *>(src);
  return {{v.x, v.y, v.z, v.w}};
}
template <>
__device__ inline Piece<32> load_piece<32>(const uint8_t *src) {
  Piece<32> p;
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(p.w[0]), "=r"(p.w[1]), "=r"(p.w[2]), "=r"(p.w[3]), "=r"(p.w[4]), "=r"(p.w[5]),
                 "=r"(p.w[6]), "=r"(p.w[7])
               : "l"(src)
               : "memory");
  return p;
}
__device__ inline void store_piece(uint8_t *dst, const Piece<16> &p) {
  *reinterpret_cast<uint4 *>(dst) = make_uint4(p.w[0], p.w[1], p.w[2], p.w[3]);
}
__device__ inline void store_piece(uint8_t *dst, const Piece<32> &p) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(p.w[0]),
               "r"(p.w[1]), "r"(p.w[2]), "r"(p.w[3]), "r"(p.w[4]), "r"(p.w[5]), "r"(p.w[6]), "r"(p.w[7])
               : "memory");
}

template <int VEC>
__global__ void __launch_bounds__(kWriteThreads) slot_write_kernel(const SlotWriteArgs a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int nw = gridDim.x * (kWriteThreads / 32);
  for (long long t = blockIdx.x * (kWriteThreads / 32) + (threadIdx.x >> 5); t < a.num_tokens;
       t += nw) {
    const long long slot = __ldg(a.slots + t);
    if (slot < 0) continue;  // a padded token
    if (slot >= a.num_slots) {
      if (lane == 0) atomicOr(a.status, PA_DEV_BAD_BLOCK);
      continue;
    }
    const uint8_t *ks = a.k_new + t * a.k_stride, *vs = a.v_new + t * a.v_stride;
    long long page = 0;
    int off = 0;
    if (a.hnd) {
      page = slot <= 0xffffffffll ? (unsigned)slot / (unsigned)a.block_size : slot / a.block_size;
      off = (int)(slot - page * a.block_size);
    }
    auto dst_of = [&](int c) {  // where byte c of the row goes (a piece stays in its head)
      if (!a.hnd) return slot * a.row_bytes + c;
      const int h = c / a.head_bytes;
      return ((page * a.num_kv_heads + h) * a.block_size + off) * a.head_bytes + (c - h * a.head_bytes);
    };
    for (int c = lane * VEC; c < a.row_bytes; c += 64 * VEC) {
      const int c1 = c + 32 * VEC;
      const bool two = c1 < a.row_bytes;
      const Piece<VEC> k0 = load_piece<VEC>(ks + c), v0 = load_piece<VEC>(vs + c);
      Piece<VEC> k1, v1;
      if (two) {
        k1 = load_piece<VEC>(ks + c1);
        v1 = load_piece<VEC>(vs + c1);
      }
      const long long d0 = dst_of(c);
      store_piece(a.k_cache + d0, k0);
      store_piece(a.v_cache + d0, v0);
      if (two) {
        const long long d1 = dst_of(c1);
        store_piece(a.k_cache + d1, k1);
        store_piece(a.v_cache + d1, v1);
      }
    }
  }
}

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_block_tables(const int32_t *seq_lens, const int32_t *query_start_loc,
                                     const int32_t *free_pages, const int32_t *free_start,
                                     int32_t *free_end, int32_t *block_table,
                                     int64_t *slot_mapping, int32_t *positions, int block_size,
                                     void *stream, int num_seqs, int num_tokens,
                                     int max_blocks_per_seq, int num_blocks, int num_free) {
  if (num_seqs < 0 || num_tokens < 0 || block_size <= 0 || max_blocks_per_seq < 0 ||
      num_blocks < 0 || num_free < 0)
    return PA_ERR_INVALID_ARG;
  const bool grow = free_start != nullptr;
  if (grow ? (!free_end || free_end == free_start || (num_free > 0 && !free_pages))
           : (free_end || free_pages || num_free > 0))
    return PA_ERR_INVALID_ARG;
  if ((num_tokens > 0 && !slot_mapping) ||
      (num_seqs > 0 && (!seq_lens || !query_start_loc)) ||
      (num_seqs > 0 && num_tokens > 0 && (!block_table || max_blocks_per_seq == 0)))
    return PA_ERR_INVALID_ARG;
  if (!aligned(seq_lens, 4) || !aligned(query_start_loc, 4) || !aligned(free_pages, 4) ||
      !aligned(free_start, 4) || !aligned(free_end, 4) || !aligned(block_table, 4) ||
      !aligned(slot_mapping, 8) || !aligned(positions, 4))
    return PA_ERR_INVALID_ARG;
  if (num_seqs > kTablesMaxSeqs) return PA_ERR_UNSUPPORTED;
  if (num_tokens == 0 && !grow) return PA_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  void *ws = nullptr;
  TablesArgs a{};
  int num_sms = 0;
  const pa_status s = device_resources(st, 0, &ws, &a.status, &num_sms);
  if (s != PA_OK) return s;
  a.seq_lens = seq_lens;
  a.qsl = query_start_loc;
  a.free_pages = free_pages;
  a.free_start = free_start;
  a.free_end = free_end;
  a.block_table = block_table;
  a.positions = positions;
  a.slots = slot_mapping;
  a.num_seqs = num_seqs;
  a.num_tokens = num_tokens;
  a.block_size = block_size;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.num_free = num_free;
  static std::atomic<unsigned long long> done{0};
  constexpr int kMaxSmem = (3 * kTablesMaxSeqs + 1) * (int)sizeof(int);
  if (set_smem_attrs_once(block_tables_kernel, kMaxSmem, done) != cudaSuccess) return PA_ERR_CUDA;
  long long blocks = ceil_div_ll(num_tokens, kTablesThreads * kTokensPerThread);
  if (blocks < 1) blocks = 1;
  if (blocks > 2ll * num_sms) blocks = 2ll * num_sms;
  const size_t smem = (3 * (size_t)num_seqs + 1) * sizeof(int);
  return launch_dependent(block_tables_kernel, dim3((unsigned)blocks), dim3(kTablesThreads), smem,
                          st, a) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

extern "C" pa_status pa_cache_write_slots(const void *k_new, const void *v_new, void *k_cache,
                                          void *v_cache, const int64_t *slot_mapping,
                                          int num_kv_heads, int head_dim, int block_size,
                                          void *stream, pa_dtype dtype, int num_tokens,
                                          long long k_token_stride, long long v_token_stride,
                                          int num_blocks, pa_kv_layout kv_layout) {
  if (num_tokens < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks < 0 ||
      k_token_stride < 0 || v_token_stride < 0 || (dtype != PA_F32 && dtype != PA_BF16) ||
      (kv_layout != PA_KV_NHD && kv_layout != PA_KV_HND))
    return PA_ERR_INVALID_ARG;
  const int es = dtype == PA_F32 ? 4 : 2;
  if (((long long)head_dim * es) % 16 != 0 || (k_token_stride * es) % 16 != 0 ||
      (v_token_stride * es) % 16 != 0 || (long long)num_kv_heads * head_dim > (1 << 26))
    return PA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PA_OK;
  if (!k_new || !v_new || !k_cache || !v_cache || !slot_mapping || num_blocks == 0 ||
      !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(slot_mapping, 8))
    return PA_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  void *ws = nullptr;
  SlotWriteArgs a{};
  int num_sms = 0;
  const pa_status s = device_resources(st, 0, &ws, &a.status, &num_sms);
  if (s != PA_OK) return s;
  a.k_new = static_cast<const uint8_t *>(k_new);
  a.v_new = static_cast<const uint8_t *>(v_new);
  a.k_cache = static_cast<uint8_t *>(k_cache);
  a.v_cache = static_cast<uint8_t *>(v_cache);
  a.slots = slot_mapping;
  a.k_stride = k_token_stride * es;
  a.v_stride = v_token_stride * es;
  a.num_slots = (long long)num_blocks * block_size;
  a.num_tokens = num_tokens;
  a.row_bytes = num_kv_heads * head_dim * es;
  a.head_bytes = head_dim * es;
  a.block_size = block_size;
  a.num_kv_heads = num_kv_heads;
  a.hnd = kv_layout == PA_KV_HND;
  long long blocks = ceil_div_ll(num_tokens, kWriteThreads / 32);
  if (blocks > 8ll * num_sms) blocks = 8ll * num_sms;
  // 32-byte pieces where every row of both sides begins on 32 bytes
  const bool wide = a.head_bytes % 32 == 0 && a.k_stride % 32 == 0 && a.v_stride % 32 == 0 &&
                    aligned(k_new, 32) && aligned(v_new, 32) && aligned(k_cache, 32) &&
                    aligned(v_cache, 32);
  return launch_dependent(wide ? slot_write_kernel<32> : slot_write_kernel<16>,
                          dim3((unsigned)blocks), dim3(kWriteThreads), 0, st, a) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}
