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
// each request's first token and its first free page in shared memory, then
// takes a share of the tokens (request by binary search).  The token at the
// start of a fresh page writes that page's table entry: pages held before are
// only read, fresh ones only written, so no entry is both.  A plan kernel
// with a second launch would cost more than the repeated scan up to far
// larger batches than kTablesMaxSeqs.
constexpr int kTablesThreads = 512;
constexpr int kTablesMaxSeqs = 16384;  // 8 bytes of shared memory a request
constexpr int kTokensPerThread = 4;    // tokens a thread takes before the grid grows to the SMs
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
  int *s_qsl = s_dyn;                     // [S + 1]
  int *s_first = s_dyn + a.num_seqs + 1;  // [S] index of the request's first free page
  __shared__ long long scratch[33];
  __shared__ int s_taken;
  const int S = a.num_seqs, T = a.num_tokens, bs = a.block_size, tid = threadIdx.x;
  const bool grow = a.free_start != nullptr;
  pdl_trigger();
  pdl_wait();

  int bad = 0;
  for (int s = tid; s <= S && S > 0; s += kTablesThreads) {
    const int q = a.qsl[s];
    s_qsl[s] = q;
    if (s == 0 ? q != 0 : a.qsl[s - 1] > q) bad = 1;
    if (s == S && q > T) bad = 1;
  }
  if (tid == 0) s_taken = 0;
  const bool qsl_bad = __syncthreads_or(bad) != 0;
  const int start = grow ? *a.free_start : 0;
  const long long avail = grow && start >= 0 ? (long long)a.num_free - start : 0;

  unsigned flags = qsl_bad ? PA_DEV_BAD_QSL : 0u;
  long long carry = 0;
  int taken = 0;
  for (int base = 0; base < S && !qsl_bad; base += kTablesThreads) {
    const int s = base + tid;
    int need = 0;
    bool ok = false;
    if (s < S) {
      const int len = a.seq_lens[s], q = s_qsl[s + 1] - s_qsl[s];
      if (len < 0 || ceil_div_ll(len, bs) > a.max_blocks_per_seq) flags |= PA_DEV_BAD_SEQLEN;
      else if (q > len) flags |= PA_DEV_BAD_QLEN;
      else ok = true;
      if (ok)
        need = grow ? (int)(ceil_div_ll(len, bs) - ceil_div_ll(len - q, bs)) : 0;
    }
    long long tot;
    const long long end = block_inclusive_scan(need, scratch, &tot) + carry;
    carry += tot;
    if (s < S) {
      const bool served = need == 0 || end <= avail;
      s_first[s] = !ok ? kBadRequest : !served ? kUnserved : need ? start + (int)(end - need) : 0;
      if (ok && !served) flags |= PA_DEV_NO_PAGES;
      if (ok && served && need > 0) taken = (int)end;
    }
  }
  if (blockIdx.x == 0) {
    if (flags) atomicOr(a.status, flags);
    if (grow) {
      if (taken) atomicMax(&s_taken, taken);
      __syncthreads();
      if (tid == 0) *a.free_end = start + s_taken;
    }
  }
  __syncthreads();

  const int stride = gridDim.x * kTablesThreads;
  const int n = S > 0 && !qsl_bad ? s_qsl[S] : 0;  // tokens that belong to a request
  for (long long t64 = blockIdx.x * kTablesThreads + tid; t64 < T; t64 += stride) {
    const int t = (int)t64;
    long long slot = -1;
    int pos = 0;
    if (t < n) {
      int lo = 0, hi = S - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_qsl[mid] <= t) lo = mid; else hi = mid - 1;
      }
      const int s = lo, first = s_first[s];
      if (first != kBadRequest) {
        const int prefix = a.seq_lens[s] - (s_qsl[s + 1] - s_qsl[s]);
        pos = prefix + t - s_qsl[s];
        if (first != kUnserved) {
          const int j = pos / bs, off = pos - j * bs;
          int32_t *entry = a.block_table + (size_t)s * a.max_blocks_per_seq + j;
          const bool fresh = grow && (long long)j * bs >= prefix;
          const int held = fresh ? (int)ceil_div_ll(prefix, bs) : 0;
          const int page = fresh ? __ldg(a.free_pages + first + j - held) : *entry;
          const bool valid = page >= 0 && page < a.num_blocks;
          if (!valid) atomicOr(a.status, PA_DEV_BAD_BLOCK);
          if (fresh && off == 0) *entry = valid ? page : -1;
          if (valid) slot = (long long)page * bs + off;
        }
      }
    }
    a.slots[t] = slot;
    if (a.positions) a.positions[t] = pos;
  }
}

// ---------------------------------------------------------------------------
// pa_cache_write_slots
// ---------------------------------------------------------------------------
// A copy: 4 x the row bytes of a token move (K and V, read and written), so
// HBM bounds it.  One warp takes one token's K and V rows.
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
    const long long page = a.hnd ? slot / a.block_size : 0;
    const int off = (int)(a.hnd ? slot % a.block_size : 0);
    for (int c = lane * 16; c < a.row_bytes; c += 512) {
      long long dst = slot * a.row_bytes + c;
      if (a.hnd) {
        const int h = c / a.head_bytes;
        dst = ((page * a.num_kv_heads + h) * a.block_size + off) * a.head_bytes +
              (c - h * a.head_bytes);
      }
      const uint4 kv = *reinterpret_cast<const uint4 *>(ks + c);
      const uint4 vv = *reinterpret_cast<const uint4 *>(vs + c);
      *reinterpret_cast<uint4 *>(a.k_cache + dst) = kv;
      *reinterpret_cast<uint4 *>(a.v_cache + dst) = vv;
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
  constexpr int kMaxSmem = (2 * kTablesMaxSeqs + 1) * (int)sizeof(int);
  if (set_smem_attrs_once(block_tables_kernel, kMaxSmem, done) != cudaSuccess) return PA_ERR_CUDA;
  long long blocks = ceil_div_ll(num_tokens, kTablesThreads * kTokensPerThread);
  if (blocks < 1) blocks = 1;
  if (blocks > 2ll * num_sms) blocks = 2ll * num_sms;
  const size_t smem = (2 * (size_t)num_seqs + 1) * sizeof(int);
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
  return launch_dependent(slot_write_kernel, dim3((unsigned)blocks), dim3(kWriteThreads), 0, st,
                          a) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}
