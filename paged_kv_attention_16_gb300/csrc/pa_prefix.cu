// pa_prefix.cu -- attention for a batch whose requests share long prefixes
// (pa_forward_shared_prefix): argument checks, the planner, the fp32
// prefix kernel and the merge (pa_prefix_mma.cu holds the bf16 prefix kernel).
//
// Requests come in consecutive groups; the requests of group g see the same
// first P_g positions.  A row's softmax over [0, P_g) and its own positions is
// the log-sum-exp join of two parts:
//   prefix part   all rows of the group (its tokens x the G heads of a KV
//                 head) against [0, P_g): every key is visible to every row,
//                 so it is a dense product of many rows, and a tile of keys is
//                 read once for 256 rows instead of once for each request;
//   own part      each request's rows against its own positions, causal: the
//                 row and tile kernels of pa_forward, their splits starting
//                 at P_g, every split stored as a partial.
// The merge joins a row's partials of both parts, and its sink.
//
// Planner: the prefix part is cut into items (KV head, 256-row block, split).
// Splits are whole 128-position tiles of equal length, sized by a cost model
// over the whole grid (see plan_splits).  Items that read the same keys are
// neighbours, so that they run at the same time and share them through L2.
//
// Launches: plan, prefix part, rows, tiles (unless declared decode-only), merge.
// The rows and tiles need the plan alone: they start as the prefix part's blocks
// end (programmatic launches, see plan_wait), so the SMs that the prefix part
// leaves are theirs.
#include <algorithm>
#include <type_traits>

#include "pa_prefix.h"

namespace pa {
namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanCache = 1024;        // requests, and groups, planned from shared memory
constexpr int kMergeThreads = 256;
constexpr int kMergeCache = 1024;       // requests whose starts the merge keeps in shared memory
constexpr int kPrefetchGroups = 64;     // groups whose page lists the planner prefetches
constexpr int kModelGroups = 128;       // groups up to which the split model is evaluated
// The own part's decode rows are cut into about this many items a resident
// block of the row kernel, and kRowItemTarget in all at most (it bounds the
// partials).  2, 3, 4, 8 items: 90 requests at G = 16 take 38, 40, 42, 57 us of
// row kernel, 64 at G = 4 take 51.5, 51.4, 51.5, 55.
constexpr int kRowItems = 2;
constexpr int kRowItemTarget = 2560;
// Longer requests' rows (128-row tiles of the tile kernel): when they are fewer
// tiles than this, two blocks on each of 152 SMs (a constant, since the host
// bounds the partials by it), they are cut into about this many items
// of kTileMinSplit positions or more (17 requests of up to 15 tokens and 1368
// positions at G = 16: 70 -> 49 us; 9 of up to 236 and 751 at G = 1: 42 -> 34, 36
// with 256 positions).  More tiles stay whole: cutting them too costs 4 to 14 us of
// 111 for 24 requests of up to 512 tokens.
constexpr int kTileItems = 304;
constexpr int kTileMinSplit = 128;
// What an item costs beside its tiles (query loads, the first scores' and the
// last products' latency, storing and merging 256 partial rows), in tiles.  (1 to
// 4 measure alike, 5 and more slower on batches of many row blocks.)
constexpr int kItemOverhead = 3;

// ---------------------------------------------------------------------------
// planner: one block
// ---------------------------------------------------------------------------

// Tiles per split.  Each thread tries one number of splits of the longest
// prefix: its length L gives every group ceil(n_g / L) splits.  The prefix part
// is done after ceil(items / SMs) waves of L + kItemOverhead tiles; the SMs are
// done with it and with the own part, which takes the SMs that it leaves
// (`own` tiles of one SM), after (tiles + items kItemOverhead + own) / SMs; and
// what is left of the own part when the last prefix item ends should be a round
// of its items, own / (kRowItems SMs).  So a batch with much of its own gets few,
// long items, on some of the SMs: 64 requests behind 8192 positions 76 -> 67 us,
// 256 behind 32768 310 -> 288 us against the prefix part sized for itself.
__device__ inline int plan_splits(const PrefixParams &p, const int *s_n, const int *s_w, int nmax,
                                  unsigned long long tiles, unsigned long long own) {
  __shared__ unsigned long long s_cost[kPlanThreads / 32];
  const int NG = p.num_groups, tid = threadIdx.x;
  if (nmax <= 0) return 1;
  if (NG > kModelGroups) {
    // enough units to fill the SMs in most batches: about two items per SM
    const unsigned long long L = (tiles + 2 * p.num_sms - 1) / (2 * p.num_sms);
    return (int)(L < 1 ? 1 : L > (unsigned long long)nmax ? nmax : L);
  }
  const unsigned s = tid + 1, L = ((unsigned)nmax + s - 1) / s;
  unsigned long long cost = 0x3fffffffffffffull;
  if (s <= (unsigned)nmax) {
    unsigned long long items = 0;
    for (int g = 0; g < NG; ++g) items += (unsigned long long)s_w[g] * (((unsigned)s_n[g] + L - 1) / L);
    if (s == 1 || items <= (unsigned long long)p.item_cap) {
      const unsigned waves = ((unsigned)min(items, 0x7fffffffull) + p.num_sms - 1) / p.num_sms;
      cost = max((unsigned long long)waves * (L + kItemOverhead) * p.num_sms + own / kRowItems,
                 tiles + items * kItemOverhead + own);
    }
  }
  unsigned long long best = cost << 9 | tid;  // ties: the fewest splits
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) best = min(best, __shfl_xor_sync(0xffffffffu, best, o));
  if ((tid & 31) == 0) s_cost[tid >> 5] = best;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) best = min(best, s_cost[w]);
  const unsigned ns = (unsigned)(best & 511) + 1;
  return (int)(((unsigned)nmax + ns - 1) / ns);
}

// A chain of short steps: what it takes is the latency of each.  The metadata
// is read once, into shared memory, every step after that works from there
// (batches beyond kPlanCache read it again from L2), and the groups' items and
// the requests' lists share one scan.  4 to 64 requests take 4.6 us from the end
// of the kernel before it (metadata 0.6, checks 1.1, splits 1.1, lists 1.8), mostly
// its code's way into the instruction cache: each element is worked out once, and
// divisions are few and of 32 bits (5.5 us before).
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const PrefixParams p) {
  __shared__ long long scratch[4 * 33];
  __shared__ int s_qsl[kPlanCache + 1], s_len[kPlanCache], s_gsl[kPlanCache + 1], s_pre[kPlanCache];
  __shared__ int s_n[kModelGroups], s_w[kModelGroups];
  __shared__ int s_nmax;
  __shared__ unsigned s_units;
  __shared__ unsigned long long s_tiles, s_work, s_ext;
  const FwdParams &f = p.f;
  const int S = f.num_seqs, NG = p.num_groups, T = f.num_tokens, tid = threadIdx.x;
  const int Hk = f.num_kv_heads, G = f.num_heads / Hk, H = f.num_heads;
  const unsigned bs = f.block_size;
  const bool cached = S <= kPlanCache && NG <= kPlanCache;
  if (tid == 0) {
    s_nmax = 0;
    s_units = 0;
    s_tiles = s_work = s_ext = 0;
  }
  pdl_trigger();
  pdl_wait();
  if (cached) {
    for (int i = tid; i <= max(S, NG); i += kPlanThreads) {
      if (i <= S) s_qsl[i] = f.qsl[i];
      if (i < S) s_len[i] = f.seq_lens[i];
      if (i <= NG) s_gsl[i] = p.group_start[i];
      if (i < NG) s_pre[i] = p.prefix_lens[i];
    }
  }
  __syncthreads();
  auto qsl = [&](int s) { return cached ? s_qsl[s] : f.qsl[s]; };
  auto gsl = [&](int g) { return cached ? s_gsl[g] : p.group_start[g]; };

  // positions that a request may have: the caller's bound, and a block-table row's
  const int longest = (int)min((unsigned long long)f.max_seq_len, (unsigned long long)f.max_blocks_per_seq * bs);
  // a group's prefix, -1 when it is bad
  auto group_prefix = [&](int g) {
    const int P = cached ? s_pre[g] : p.prefix_lens[g];
    const bool ok = P >= 0 && P <= longest && P <= p.max_prefix_len && (unsigned)P % bs == 0;
    return ok ? P : -1;
  };
  unsigned flags = 0;
  auto group_of = [&](int g) {
    // (clamped: the starts may not have been found good yet)
    const int r0 = min(max(gsl(g), 0), S), r1 = min(max(gsl(g + 1), 0), S);
    const int q0 = qsl(r0), nq = qsl(r1) - q0;
    int P = group_prefix(g);
    if (P < 0) {
      if (r1 > r0) flags |= PA_DEV_BAD_SEQLEN;
      P = 0;
    }
    const int nrp = nq > 0 ? (int)(((long long)nq * G + kPrefixRows - 1) / kPrefixRows) : 0;
    return PrefixGroup{q0, nq, r0, P, nrp, 0, 0, 0};
  };
  auto tiles_of = [&](const PrefixGroup &g) {
    return g.q_len > 0 ? (int)(((unsigned)g.prefix + kPrefixTile - 1) / kPrefixTile) : 0;
  };
  auto classify = [&](int s, int &g, ReqInfo &r) {
    int lo = 0, hi = NG - 1;
    while (lo < hi) {  // the last group that starts at or before s
      const int mid = (lo + hi + 1) >> 1;
      if (gsl(mid) <= s) lo = mid; else hi = mid - 1;
    }
    g = lo;
    const int P = group_prefix(g);
    r.q_start = qsl(s);
    r.q_len = qsl(s + 1) - r.q_start;
    r.ctx = cached ? s_len[s] : f.seq_lens[s];
    r.kv_base = P < 0 ? 0 : P;
    const bool len_ok = r.ctx >= 0 && r.ctx <= longest;
    const bool q_ok = r.q_len <= r.ctx && (f.max_qlen <= 0 || r.q_len <= f.max_qlen);
    const bool own_ok = P >= 0 && r.ctx - r.q_len >= P;
    const bool valid = r.q_len > 0 && len_ok && q_ok && own_ok;
    r.flags = (r.q_len == 1 ? kDecode : kExtend) | (valid ? kFlagValid : 0) |
              (!f.tile_ok || r.q_len == 1 ? kFlagRowPath : 0);
    if (r.q_len != 0)
      flags |= (len_ok && own_ok ? 0u : PA_DEV_BAD_SEQLEN) | (q_ok ? 0u : PA_DEV_BAD_QLEN);
  };

  // -- the starts' checks; the groups' tiles; the decode rows' own work
  int bad = 0;
  if (tid == 0) bad = qsl(0) != 0 || qsl(S) > T || gsl(0) != 0 || gsl(NG) != S;
  // (this thread's first group and request stay in registers for the lists:
  // the planner's time is that of its code, so what runs once runs once)
  PrefixGroup gr0{};
  ReqInfo r0{};
  int group0 = 0;
  for (int g = tid; g < NG; g += kPlanThreads) {
    if (gsl(g + 1) < gsl(g)) bad = 1;
    const PrefixGroup gr = group_of(g);
    if (g == tid) gr0 = gr;
    const int n = tiles_of(gr);
    if (NG <= kModelGroups) {
      s_n[g] = n;
      s_w[g] = n > 0 ? Hk * gr.nrp : 0;
    }
    if (n > 0) {
      atomicMax(&s_nmax, n);
      atomicAdd(&s_tiles, (unsigned long long)n * Hk * gr.nrp);
    }
  }
  unsigned long long work = 0, ext = 0;  // positions of decode rows; 128 x 64 tiles of longer requests
  unsigned units = 0;                    // and their 128-row tiles, of a KV head
  for (int s = tid; s < S; s += kPlanThreads) {
    if (qsl(s + 1) < qsl(s)) bad = 1;
    int g;
    ReqInfo r{};
    classify(s, g, r);
    if (s == tid) r0 = r, group0 = g;
    if (r.flags & kFlagValid) {
      const unsigned len = r.ctx - r.kv_base;
      if (r.q_len == 1) work += len;
      else {
        const unsigned t = (unsigned)(((unsigned long long)r.q_len * G + kTileRows - 1) / kTileRows);
        units += t;
        ext += (unsigned long long)t * ((len + 63) / 64);
      }
    }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    work += __shfl_xor_sync(0xffffffffu, work, o);
    ext += __shfl_xor_sync(0xffffffffu, ext, o);
  }
  if ((tid & 31) == 0 && work) atomicAdd(&s_work, work);
  units = __reduce_add_sync(0xffffffffu, units);
  if ((tid & 31) == 0 && ext) {
    atomicAdd(&s_ext, ext);
    atomicAdd(&s_units, units);
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      atomicOr(f.status, PA_DEV_BAD_QSL);
      p.plan->n_items = 0;
      p.plan->all_bad = 1;
      for (int x = 0; x < kNumLists; ++x) f.plan->n[x] = 0;
      for (int x = 0; x < 8; ++x) f.plan->counter[x] = 0;
      f.plan->qsl_bad = 1;
    }
    return;
  }
  if (flags) atomicOr(f.status, flags);
  // the prefixes' page lists on their way to L2: the next kernel's first loads
  if (cached) {
    for (int g = tid >> 5; g < min(NG, kPrefetchGroups); g += kPlanThreads / 32) {
      const char *row = reinterpret_cast<const char *>(f.block_table + (size_t)s_gsl[g] * f.max_blocks_per_seq);
      // (pages have 16 positions or more; a prefix found bad is only held to the row)
      const unsigned pages = s_gsl[g + 1] > s_gsl[g] ? (unsigned)min(max(s_pre[g], 0), longest) / 16 : 0;
      const unsigned bytes = min(pages, (unsigned)f.max_blocks_per_seq) * 4;
      for (unsigned at = (tid & 31) * 128; at < bytes; at += 32 * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(row + at));
    }
  }
  // The own part's work in the prefix part's tiles, of 1.4 us of an SM at head_dim
  // 128 and 1.28 at 64: 128 positions of a decode row's KV head are 64 or 32 KB, at
  // an SM's share of the row kernel's 6.3 TB/s 1.57 or 0.79 us, so 18/16 or 10/16 of
  // a tile; a 128-row x 64-position tile of longer requests takes about 0.6 us, 7/16.
  // (Without the own part's weight 64 requests behind 8192 positions take 76 us, 67
  // with it; 256 behind 32768 310 and 288.)
  // (fp32: both parts run on CUDA cores, and the prefix part is sized alone)
  const unsigned long long own =
      f.dtype == PA_BF16 ? s_work * Hk / 128 * (f.head_dim == 128 ? 18 : 10) / 16 + s_ext * Hk * 7 / 16 : 0;
  const int L = plan_splits(p, s_n, s_w, s_nmax, s_tiles, own);
  // The own part's decode rows: about kRowItems items a resident block, down to
  // one 64-position stage of the row kernel.
  const unsigned target = min(kRowItems * max(f.row_ctas, 1), kRowItemTarget);
  // (in floats, whose rounding the bound on the partials has room for)
  const float Lw = fminf((float)s_work * Hk / target, (float)kRowMaxSplit);
  const int Ld = min(max(((int)Lw + 64) / 64 * 64, kFastMinSplit), kRowMaxSplit);
  // rows of longer requests: tiles (0: whole), or (fp32) row items of at most
  // about 4 splits
  const int Lt = s_units >= (unsigned)kTileItems / Hk
                     ? 0
                     : max((int)((float)s_ext * Hk / kTileItems) + 1, kTileMinSplit / 64) * 64;
  const int Lr = min(max(Ld, (f.max_seq_len / 4 + 16) / 16 * 16), kRowMaxSplit);

  // -- the groups' items, and the requests' lists: row items, tile items, partial rows
  long long sum[4] = {0, 0, 0, 0};
  for (int base = 0; base < max(S, NG); base += kPlanThreads) {
    const int i = base + tid;
    long long cnt[4] = {0, 0, 0, 0}, tot[4];
    PrefixGroup gr{};
    ReqInfo r{};
    int g = 0;
    if (base == 0) {
      gr = gr0;
      r = r0;
      g = group0;
    } else {
      if (i < NG) gr = group_of(i);
      if (i < S) classify(i, g, r);
    }
    if (i < NG) {
      const unsigned n = tiles_of(gr), ns = (n + L - 1) / (unsigned)L;
      // equal splits; as many as have tiles
      const unsigned len = ns > 0 ? (n + ns - 1) / ns : 1;
      gr.nsplit = (n + len - 1) / len;
      gr.split_len = len * kPrefixTile;
      cnt[0] = (long long)Hk * gr.nrp * gr.nsplit;
    }
    if (i < S) {
      const int own = r.ctx - r.kv_base;
      r.split_len = r.q_len == 1 ? Ld : (r.flags & kFlagRowPath) ? Lr : Lt > 0 ? Lt : max(own, 1);
      r.nsplit = max(((unsigned)max(own, 0) + r.split_len - 1) / (unsigned)r.split_len, 1u);
      if (r.flags & kFlagValid) {
        if (r.flags & kFlagRowPath) cnt[1] = (long long)Hk * r.q_len * r.nsplit;
        else cnt[2] = (long long)Hk * (((long long)r.q_len * G + kTileRows - 1) / kTileRows) * r.nsplit;
        cnt[3] = (long long)r.q_len * H * r.nsplit;
      }
    }
    const long long items = cnt[0], part = cnt[3];
    block_scan_multi<4>(cnt, scratch, tot);
    if (i < NG) {
      gr.item0 = (int)(cnt[0] + sum[0] - items);
      p.grp[i] = gr;
      p.grp_end[i] = (int)(cnt[0] + sum[0]);
    }
    if (i < S) {
      r.partial_base = cnt[3] + sum[3] - part;
      f.list_end[(size_t)kListRow * S + i] = cnt[1] + sum[1];
      f.list_end[(size_t)kListTile * S + i] = cnt[2] + sum[2];
      f.ord[i] = i;
      f.req[i] = r;
      p.req_grp[i] = g;
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) sum[x] += tot[x];
  }
  if (tid == 0) {
    const bool overflow = sum[3] > f.part_cap || sum[0] > p.item_cap;
    if (overflow) atomicOr(f.status, PA_DEV_OVERFLOW);
    p.plan->n_items = overflow ? 0 : (int)sum[0];
    p.plan->all_bad = overflow ? 1 : 0;
    for (int x = 0; x < kNumLists; ++x) f.plan->n[x] = 0;
    f.plan->n[kListRow] = overflow ? 0 : sum[1];
    f.plan->n[kListTile] = overflow ? 0 : sum[2];
    for (int x = 0; x < 8; ++x) f.plan->counter[x] = 0;
    f.plan->qsl_bad = overflow ? 1 : 0;
  }
}

// ---------------------------------------------------------------------------
// prefix part on CUDA cores (fp32)
// ---------------------------------------------------------------------------
// Eight threads share four rows (each every eighth 16-byte group of their
// head_dim values), 128 rows a pass; 32 keys and values at a time in shared
// memory, each load of them used for the four rows.  The scores of 8 keys are
// reduced over the eight threads so that each ends up with one key's (7
// shuffles a row), join the running maximum and sum there, and the weights are
// handed round again.  256 rows x 128 positions take 71 us of an SM at head_dim
// 128 (36 TFLOP/s over the GPU) and 47 at 64, against 143 and 80 with one row in
// four threads: what bounds it is the latency of the FMA chains and the shuffles
// with two warps a scheduler, all that four rows' registers leave room for.
constexpr int kSimtThreads = 256;
constexpr int kSimtKeys = 32;
constexpr int kSimtRows = 4;  // rows of a thread, 32 apart

template <int D>
struct SimtTile {  // two of them: one is loaded while the other is used
  float k[kSimtKeys][D], v[kSimtKeys][D];
};

// 16 bytes from global to shared memory, or zeros.
__device__ inline void copy16(float *dst, const float *src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(take ? 16 : 0)
               : "memory");
}

template <int D>
__global__ void __launch_bounds__(kSimtThreads, 1) prefix_simt_kernel(const PrefixParams p, int hnd) {
  constexpr int N = D / 8;  // values of a row that a thread holds
  extern __shared__ __align__(16) uint8_t s_raw[];
  SimtTile<D> *s_tile = reinterpret_cast<SimtTile<D> *>(s_raw);
  const FwdParams &f = p.f;
  const int tid = threadIdx.x, lane = tid & 31, c = tid & 7;
  const int G = f.num_heads / f.num_kv_heads, bs = f.block_size;
  const int Hk = f.num_kv_heads;
  pdl_wait();     // the plan
  pdl_trigger();  // the own part's kernels count on the plan being done
  const int n_items = p.plan->n_items;
  const PrefixGroup g0 = p.grp[0];
  const float *kc = static_cast<const float *>(p.k_cache);
  const float *vc = static_cast<const float *>(p.v_cache);
  for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
    const PrefixItem it = prefix_item(p, g0, item, G);
    const int32_t *bt = f.block_table + (size_t)it.req0 * f.max_blocks_per_seq;
    const int rows = min(kPrefixRows, (it.q_len - it.t0) * G);
    // (a pass of fewer rows than threads' rows holds one or two a thread)
    auto pass = [&](int row0, auto rows_c) {
      constexpr int R = decltype(rows_c)::value;
      float qv[R][N], o[R][N], m[R], l[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int row = min(row0 + r * 32 + (tid >> 3), rows - 1);
        const int tok = it.q_start + it.t0 + row / G, head = it.kvh * G + row % G;
        const float *q = static_cast<const float *>(f.q) + ((size_t)tok * f.num_heads + head) * D;
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          const float4 x = *reinterpret_cast<const float4 *>(q + i * 8 + c * 4);
          qv[r][i] = x.x * f.scale_log2;
          qv[r][i + 1] = x.y * f.scale_log2;
          qv[r][i + 2] = x.z * f.scale_log2;
          qv[r][i + 3] = x.w * f.scale_log2;
          o[r][i] = o[r][i + 1] = o[r][i + 2] = o[r][i + 3] = 0.f;
        }
      }
      int bad = 0;
      auto load = [&](SimtTile<D> &t, int lo) {
#pragma unroll 4
        for (int e = tid; e < kSimtKeys * (D / 4); e += kSimtThreads) {
          const int j = e / (D / 4), x = e % (D / 4) * 4, pos = lo + j;
          bool in = pos < it.kv_hi;
          size_t row = 0;
          if (in) {
            const int page = __ldg(bt + pos / bs), slot = pos % bs;
            if (page < 0 || page >= f.num_blocks) {
              bad = 1;
              in = false;
            } else {
              row = hnd ? ((size_t)page * Hk + it.kvh) * bs + slot : ((size_t)page * bs + slot) * Hk + it.kvh;
            }
          }
          copy16(&t.k[j][x], kc + row * D + x, in);
          copy16(&t.v[j][x], vc + row * D + x, in);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      int buf = 0;
      load(s_tile[0], it.kv_lo);
      for (int lo = it.kv_lo; lo < it.kv_hi; lo += kSimtKeys, buf ^= 1) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // the tile is there, and the other one has been read
        const SimtTile<D> &t = s_tile[buf];
        if (lo + kSimtKeys < it.kv_hi) load(s_tile[buf ^ 1], lo + kSimtKeys);
        for (int j0 = 0; j0 < kSimtKeys && lo + j0 < it.kv_hi; j0 += 8) {
          float w[R][8];  // the thread's shares of 8 scores, then its key's weight in [0]
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float4 k4[N / 4];
#pragma unroll
            for (int i = 0; i < N / 4; ++i)
              k4[i] = *reinterpret_cast<const float4 *>(&t.k[j0 + j][i * 32 + c * 4]);
#pragma unroll
            for (int r = 0; r < R; ++r) {
              float a0 = 0.f, a1 = 0.f, b0 = 0.f, b1 = 0.f;
#pragma unroll
              for (int i = 0; i < N / 4; ++i) {
                ffma2(a0, a1, qv[r][4 * i], qv[r][4 * i + 1], k4[i].x, k4[i].y);
                ffma2(b0, b1, qv[r][4 * i + 2], qv[r][4 * i + 3], k4[i].z, k4[i].w);
              }
              w[r][j] = (a0 + a1) + (b0 + b1);
            }
          }
          const bool seen = lo + j0 + c < it.kv_hi;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            // sum over the eight threads, half of the keys going to each half
#pragma unroll
            for (int h = 4; h >= 1; h >>= 1) {
#pragma unroll
              for (int j = 0; j < h; ++j) {
                const float keep = c & h ? w[r][j + h] : w[r][j], send = c & h ? w[r][j] : w[r][j + h];
                w[r][j] = keep + __shfl_xor_sync(0xffffffffu, send, h);
              }
            }
            const float sc = seen ? w[r][0] : -INFINITY;
            float mx = sc;
#pragma unroll
            for (int h = 4; h >= 1; h >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, h));
            if (mx > m[r]) {
              const float a = m[r] == -INFINITY ? 0.f : exp2f(m[r] - mx);
              l[r] *= a;
#pragma unroll
              for (int i = 0; i < N; ++i) o[r][i] *= a;
              m[r] = mx;
            }
            w[r][0] = exp2f(sc - (m[r] == -INFINITY ? 0.f : m[r]));
            l[r] += w[r][0];
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float4 v4[N / 4];
#pragma unroll
            for (int i = 0; i < N / 4; ++i)
              v4[i] = *reinterpret_cast<const float4 *>(&t.v[j0 + j][i * 32 + c * 4]);
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const float wj = __shfl_sync(0xffffffffu, w[r][0], (lane & 24) | j);
#pragma unroll
              for (int i = 0; i < N / 4; ++i) {
                ffma2(o[r][4 * i], o[r][4 * i + 1], v4[i].x, v4[i].y, wj, wj);
                ffma2(o[r][4 * i + 2], o[r][4 * i + 3], v4[i].z, v4[i].w, wj, wj);
              }
            }
          }
        }
      }
      bad = __syncthreads_or(bad);  // (and both tiles have been read)
      if (bad && tid == 0) atomicOr(f.status, PA_DEV_BAD_BLOCK);
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int h = 4; h >= 1; h >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], h);
        const int row = row0 + r * 32 + (tid >> 3);
        if (row < rows) {
          const long long prow = (long long)item * kPrefixRows + row;
          const float inv = l[r] > 0.f && !bad ? 1.f / l[r] : 0.f;
#pragma unroll
          for (int i = 0; i < N; i += 4)
            *reinterpret_cast<float4 *>(p.part_o + prow * D + i * 8 + c * 4) =
                make_float4(o[r][i] * inv, o[r][i + 1] * inv, o[r][i + 2] * inv, o[r][i + 3] * inv);
          if (c == 0)
            p.part_lse[prow] =
                bad ? __int_as_float(0x7fc00000) : l[r] > 0.f ? m[r] + log2f(l[r]) : -INFINITY;
        }
      }
    };
    for (int row0 = 0; row0 < rows; row0 += 32 * kSimtRows) {
      if (rows - row0 <= 32) pass(row0, std::integral_constant<int, 1>());
      else if (rows - row0 <= 64) pass(row0, std::integral_constant<int, 2>());
      else pass(row0, std::integral_constant<int, kSimtRows>());
    }
  }
}

// ---------------------------------------------------------------------------
// merge
// ---------------------------------------------------------------------------
// A row is one (token, query head); out = sum_i w_i O_i with
// w_i = 2^(lse_i - M) / (sum_j 2^(lse_j - M) + 2^(sink - M)) over the row's
// prefix partials, then its own.  Eight lanes hold a row's head_dim values and
// walk its partials with a running maximum, four at a time (their loads are
// independent); W such groups share a row's partials and meet in shared memory.
// Bound by the latency of a few dependent loads when rows are few (2048 rows of 7
// partials: 8 us alone), by reading the partials from L2 when they are many
// (38,700 rows of 256 bytes x 2 to 6: 16 us).
constexpr int kMergeGroups = kMergeThreads / 8;

template <typename T>
__device__ inline void store4(T *dst, float a, float b, float c, float d);
template <>
__device__ inline void store4<float>(float *dst, float a, float b, float c, float d) {
  *reinterpret_cast<float4 *>(dst) = make_float4(a, b, c, d);
}
template <>
__device__ inline void store4<__nv_bfloat16>(__nv_bfloat16 *dst, float a, float b, float c, float d) {
  // one rounding to nearest even, of the finished output
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b), y = __floats2bfloat162_rn(c, d);
  *reinterpret_cast<uint2 *>(dst) = make_uint2(*reinterpret_cast<const uint32_t *>(&x),
                                               *reinterpret_cast<const uint32_t *>(&y));
}

template <typename T, int D, int W>
__global__ void __launch_bounds__(kMergeThreads) prefix_merge_kernel(const PrefixParams p) {
  constexpr int V = D / 32;                   // float4 values a lane holds
  constexpr int ROWS = kMergeGroups / W;      // rows a block works on at a time
  constexpr int SPLIT = W > 1 ? W : 1;
  __shared__ int s_qsl[kMergeCache];
  __shared__ float4 s_o[W > 1 ? kMergeGroups : 1][W > 1 ? 8 * V : 1];
  __shared__ float s_m[kMergeGroups], s_l[kMergeGroups];
  const FwdParams &f = p.f;
  const int S = f.num_seqs, H = f.num_heads, G = H / f.num_kv_heads;
  const int tid = threadIdx.x, lane = tid & 7, grp = tid >> 3, part = grp % SPLIT;
  pdl_trigger();
  // The plan is done (see plan_wait): with few rows, everything up to the first
  // partials is read while the kernels that make them run (64 requests behind
  // 8192 positions 65 us, 67 without; 48 behind 131072 55, 57).  With many it
  // only costs (the loop over rows waits anew: merge of 98,000 rows 16.4 us, 14.2
  // without).
  if (W > 1) __threadfence();
  else pdl_wait();
  T *out = static_cast<T *>(f.out);
  const long long rows = (long long)f.num_tokens * H;
  const bool all_bad = p.plan->all_bad != 0;
  // a decode batch: token tok is most likely request tok's, no search
  const bool one = f.max_qlen == 1 && S == f.num_tokens;
  const bool cached = !one && S <= kMergeCache;
  if (cached) {
    for (int s = tid; s < S; s += kMergeThreads) s_qsl[s] = f.qsl[s];
    __syncthreads();
  }
  for (long long row0 = (long long)blockIdx.x * ROWS; row0 < rows; row0 += (long long)gridDim.x * ROWS) {
    const long long row = row0 + grp / SPLIT;
    float4 acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, l = 0.f;
    int h = 0, np = 0, n = 0;  // the row's prefix partials, and all of them
    bool mine = row < rows;    // (not a row behind the last request)
    long long pre0 = 0, own0 = 0, step = 0;
    if (row < rows && !all_bad) {
      const int tok = (int)(row / H);
      h = (int)(row % H);
      int lo = 0, hi = S - 1;
      if (one && f.req[tok].q_start == tok && f.req[tok].q_len == 1) lo = hi = tok;
      while (lo < hi) {  // the last request that starts at or before tok: its own
        const int mid = (lo + hi + 1) >> 1;
        if ((cached ? s_qsl[mid] : f.qsl[mid]) <= tok) lo = mid; else hi = mid - 1;
      }
      const ReqInfo r = f.req[lo];
      const PrefixGroup g = p.grp[p.num_groups == 1 ? 0 : p.req_grp[lo]];
      mine = tok - r.q_start < r.q_len;
      if (mine && (r.flags & kFlagValid)) {
        const int i = tok - r.q_start, pos = r.ctx - r.q_len + i;
        np = g.nsplit;
        n = np + (pos - r.kv_base) / r.split_len + 1;
        own0 = r.partial_base + ((long long)i * H + h) * r.nsplit - np;
        // row of the prefix part's blocks, and the step between its splits
        const int pr = (tok - g.q_start) * G + h % G;
        step = (long long)g.nrp * kPrefixRows;
        pre0 = (long long)(g.item0 + h / G * np * g.nrp + pr / kPrefixRows) * kPrefixRows + pr % kPrefixRows;
      }
    }
    if (W > 1) pdl_wait();  // the partials
    for (int e0 = part; e0 < n; e0 += 4 * SPLIT) {
      float lse[4];
      float4 x[4][V];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int e = e0 + u * SPLIT;
        const long long at = e < np ? pre0 + e * step : own0 + e;
        const float *src = (e < np ? p.part_o : f.part_o) + at * D + lane * 4;
        lse[u] = -INFINITY;
        if (e < n) {
          lse[u] = __ldcg((e < np ? p.part_lse : f.part_lse) + at);
#pragma unroll
          for (int v = 0; v < V; ++v) x[u][v] = __ldcg(reinterpret_cast<const float4 *>(src + v * 32));
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (e0 + u * SPLIT >= n) break;
        // (a bad split's NaN makes m NaN from here on; a split with no
        // weight adds 0 O, which keeps the NaN of a NaN input)
        const float top = lse[u] > m || isnan(lse[u]) ? lse[u] : m;
        const float a = m == -INFINITY ? 0.f : fast_exp2(m - top);
        const float w = lse[u] == -INFINITY ? 0.f : fast_exp2(lse[u] - top);
        m = top;
        l = fmaf(l, a, w);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          acc[v].x = fmaf(acc[v].x, a, w * x[u][v].x);
          acc[v].y = fmaf(acc[v].y, a, w * x[u][v].y);
          acc[v].z = fmaf(acc[v].z, a, w * x[u][v].z);
          acc[v].w = fmaf(acc[v].w, a, w * x[u][v].w);
        }
      }
    }
    if constexpr (W > 1) {
      // the row's groups: (m, l, O) to shared memory, joined by the first one
      __syncthreads();  // the rows before are read
      if (lane == 0) {
        s_m[grp] = m;
        s_l[grp] = l;
      }
#pragma unroll
      for (int v = 0; v < V; ++v) s_o[grp][v * 8 + lane] = acc[v];
      __syncthreads();
      if (part == 0) {
        float top = m;
#pragma unroll 4
        for (int k = 1; k < W; ++k) {
          const float v = s_m[grp + k];
          if (isnan(v) || v > top) top = v;
          if (isnan(top)) break;
        }
        const float a = m == -INFINITY ? 0.f : fast_exp2(m - top);
        l *= a;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          acc[v].x *= a;
          acc[v].y *= a;
          acc[v].z *= a;
          acc[v].w *= a;
        }
#pragma unroll 4
        for (int k = 1; k < W; ++k) {
          const float mk = s_m[grp + k], b = mk == -INFINITY ? 0.f : fast_exp2(mk - top);
          l = fmaf(s_l[grp + k], b, l);
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float4 o = s_o[grp + k][v * 8 + lane];
            acc[v].x = fmaf(o.x, b, acc[v].x);
            acc[v].y = fmaf(o.y, b, acc[v].y);
            acc[v].z = fmaf(o.z, b, acc[v].z);
            acc[v].w = fmaf(o.w, b, acc[v].w);
          }
        }
        m = top;
      }
    }
    if (mine && part == 0) {
      // the sink joins the denominator once, with no value; a row with no
      // weight is 0 O, one with a bad page zero
      float inv = 0.f;
      if (m != -INFINITY && !isnan(m)) {
        float k = 1.f;
        if (f.sinks) {
          const float sink2 = __ldg(f.sinks + h) * kLog2eF, top = fmaxf(m, sink2);
          k = fast_exp2(m - top);
          l = l * k + fast_exp2(sink2 - top);
        }
        inv = l > 0.f ? k / l : 0.f;
      }
      const bool zero = isnan(m);
      T *dst = out + row * D + lane * 4;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (zero) store4<T>(dst + v * 32, 0.f, 0.f, 0.f, 0.f);
        else store4<T>(dst + v * 32, acc[v].x * inv, acc[v].y * inv, acc[v].z * inv, acc[v].w * inv);
      }
    }
  }
}

template <typename T, int D>
cudaError_t launch_merge_d(const PrefixParams &p, cudaStream_t st) {
  // Groups a row: as many as the SMs hold at once (two blocks each): 2048 rows
  // take 64 us of a call with 4, 67 with 8; 5760 rows 66 with one, 70 with 4; 384
  // rows of 75 partials 52 with 16, 54 with 8, 78 with one.  And no more than a
  // row's partials fill, four at a time: 128 rows of 11 take 18.6 with 4, 19.3
  // with 16.
  const long long rows = (long long)p.f.num_tokens * p.f.num_heads, sms = p.num_sms;
  const long long most = ceil_div_ll(p.f.max_seq_len, kPrefixTile) + 4;
  const int fit = rows <= 4 * sms ? 16 : rows <= 8 * sms ? 8 : rows <= 16 * sms ? 4 : 1;
  const int W = std::min(fit, most <= 16 ? 4 : most <= 32 ? 8 : 16);
  auto kern = W == 16 ? prefix_merge_kernel<T, D, 16>
              : W == 8 ? prefix_merge_kernel<T, D, 8>
              : W == 4 ? prefix_merge_kernel<T, D, 4> : prefix_merge_kernel<T, D, 1>;
  const long long blocks = std::min(ceil_div_ll(rows * W, kMergeGroups), sms * 8);
  return launch_dependent(kern, dim3((unsigned)blocks), dim3(kMergeThreads), 0, st, p);
}

template <typename T>
cudaError_t launch_merge(const PrefixParams &p, cudaStream_t st) {
  return p.f.head_dim == 128 ? launch_merge_d<T, 128>(p, st) : launch_merge_d<T, 64>(p, st);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

constexpr long long kMaxItems = 1ll << 30;  // items are counted in ints

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct PrefixLayout {
  size_t plan, req, ord, list_end, pplan, grp, grp_end, req_grp, pre_o, pre_lse, own_o, own_lse,
      total;
  long long item_cap, part_cap;
};

// Host-side bounds of what the planner lays out, from the extents alone.
PrefixLayout prefix_layout(int dtype, int num_seqs, int num_groups, int num_tokens, int num_heads,
                           int num_kv_heads, int head_dim, int max_seq_len) {
  PrefixLayout l{};
  const long long S = num_seqs > 0 ? num_seqs : 1, NG = num_groups > 0 ? num_groups : 1;
  const long long T = num_tokens, H = num_heads, Hk = num_kv_heads, G = H / Hk;
  const long long msl = max_seq_len > 0 ? max_seq_len : 1;
  // one item per (KV head, 256-row block, group) unsplit, and what splitting
  // adds, but no more than one a tile
  const long long units = Hk * (ceil_div_ll(T * G, kPrefixRows) + NG);
  const long long splits = ceil_div_ll(msl, kPrefixTile);
  l.item_cap = units + (splits == 1 ? 0 : units >= kPrefixSplitItems ? kPrefixSplitItems
                                        : std::min((long long)kPrefixSplitItems, units * (splits - 1)));
  // own part: decode rows ceil(len / Ld) splits each, Ld sized to the item
  // target; longer rows one split and what kTileItems adds (tile kernel), or
  // about four (fp32)
  const long long dec = std::min(S, T);
  long long cap = H * dec * (1 + ceil_div_ll(msl, kRowMaxSplit)) + G * kRowItemTarget;
  long long per_row = 1;
  if (dtype == PA_F32) {
    long long lr = ceil_div_ll(ceil_div_ll(msl, 4), 16) * 16;
    lr = std::min(std::max(lr, (long long)kFastMinSplit), (long long)kRowMaxSplit);
    per_row = ceil_div_ll(msl, lr);
  } else {
    cap += std::min((long long)kTileItems * kTileRows, T * H * (ceil_div_ll(msl, kTileMinSplit) - 1));
  }
  cap += T * H * per_row;
  l.part_cap = cap;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  l.plan = take(sizeof(PlanHeader));
  l.req = take(S * sizeof(ReqInfo));
  l.ord = take(S * sizeof(int));
  l.list_end = take(S * kNumLists * sizeof(long long));
  l.pplan = take(sizeof(PrefixPlan));
  l.grp = take(NG * sizeof(PrefixGroup));
  l.grp_end = take(NG * sizeof(int));
  l.req_grp = take(S * sizeof(int));
  l.pre_o = take((size_t)l.item_cap * kPrefixRows * head_dim * sizeof(float));
  l.pre_lse = take((size_t)l.item_cap * kPrefixRows * sizeof(float));
  l.own_o = take((size_t)cap * head_dim * sizeof(float));
  l.own_lse = take((size_t)cap * sizeof(float));
  l.total = off;
  return l;
}

template <int D>
cudaError_t launch_simt_d(const PrefixParams &p, int hnd, int num_sms, cudaStream_t st) {
  constexpr int kSmem = 2 * (int)sizeof(SimtTile<D>);
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = set_smem_attrs_once(prefix_simt_kernel<D>, kSmem, done);
  if (e != cudaSuccess) return e;
  return launch_dependent(prefix_simt_kernel<D>, dim3(num_sms), dim3(kSimtThreads), kSmem, st, p, hnd);
}

cudaError_t launch_simt(const PrefixParams &p, int hnd, int num_sms, cudaStream_t st) {
  return p.f.head_dim == 128 ? launch_simt_d<128>(p, hnd, num_sms, st)
                             : launch_simt_d<64>(p, hnd, num_sms, st);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

size_t pa_forward_shared_prefix_workspace_bytes(pa_dtype dtype, int num_seqs, int num_groups,
                                                int num_tokens, int num_heads, int num_kv_heads,
                                                int head_dim, int max_seq_len) {
  if (num_seqs < 0 || num_groups < 0 || num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 ||
      num_heads % num_kv_heads || head_dim <= 0 || max_seq_len < 0 ||
      (long long)num_tokens * num_heads > (1ll << 40) / head_dim)
    return 0;
  const PrefixLayout lay = prefix_layout(dtype, num_seqs, num_groups, num_tokens, num_heads,
                                         num_kv_heads, head_dim, max_seq_len);
  return lay.item_cap > kMaxItems ? 0 : lay.total;
}

pa_status pa_forward_shared_prefix(
    const void *q, const void *k_cache, const void *v_cache, const int32_t *block_table,
    const int32_t *seq_lens, const int32_t *query_start_loc, const int32_t *group_start_loc,
    const int32_t *prefix_lens, int num_heads, int num_kv_heads, int head_dim, int block_size,
    float scale, void *out, void *stream, pa_dtype dtype, int num_seqs, int num_groups,
    int num_tokens, int max_blocks_per_seq, int num_blocks, int max_seq_len, int max_prefix_len,
    const pa_forward_options *options, void *workspace, size_t workspace_bytes) {
  FwdCall c{q, k_cache, v_cache, block_table, seq_lens, query_start_loc, num_heads,
            num_kv_heads, head_dim, block_size, scale, out, dtype, num_seqs, num_tokens,
            max_blocks_per_seq, num_blocks, max_seq_len, 0};
  if (num_groups < 0 || max_prefix_len < 0) return PA_ERR_INVALID_ARG;
  if (options) {
    if (options->sinks && (reinterpret_cast<uintptr_t>(options->sinks) & 3))
      return PA_ERR_INVALID_ARG;
    if ((options->kv_layout != PA_KV_NHD && options->kv_layout != PA_KV_HND) ||
        options->sliding_window < 0 || options->max_query_len < 0 ||
        (options->alibi_sqrt != 0 && options->alibi_sqrt != 1))
      return PA_ERR_INVALID_ARG;
    // every prefix key is visible to every row, whatever its position
    if (options->sliding_window || options->alibi_slopes) return PA_ERR_UNSUPPORTED;
    c.sinks = options->sinks;
    c.kv_layout = options->kv_layout;
    c.max_query_len = options->max_query_len;
  }
  pa_status s = fwd_check(c);
  if (s != PA_OK || num_tokens == 0) return s;
  if (num_groups == 0 || num_seqs == 0 || !group_start_loc || !prefix_lens)
    return PA_ERR_INVALID_ARG;
  for (const int32_t *x : {block_table, seq_lens, query_start_loc, group_start_loc, prefix_lens})
    if (reinterpret_cast<uintptr_t>(x) & 3) return PA_ERR_INVALID_ARG;
  const PrefixLayout lay = prefix_layout(dtype, num_seqs, num_groups, num_tokens, num_heads,
                                         num_kv_heads, head_dim, max_seq_len);
  if (lay.item_cap > kMaxItems) return PA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < lay.total) return PA_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return PA_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  PrefixParams p{};
  void *lib_ws = nullptr;
  int num_sms = 0;
  s = device_resources(st, 0, &lib_ws, &p.f.status, &num_sms);
  if (s != PA_OK) return s;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const int group = num_heads / num_kv_heads;
  FwdParams &f = p.f;
  f.q = q;
  f.out = out;
  f.block_table = block_table;
  f.seq_lens = seq_lens;
  f.qsl = query_start_loc;
  f.num_seqs = num_seqs;
  f.num_tokens = num_tokens;
  f.num_heads = num_heads;
  f.num_kv_heads = num_kv_heads;
  f.head_dim = head_dim;
  f.head_dim_qk = head_dim;
  f.block_size = block_size;
  f.max_blocks_per_seq = max_blocks_per_seq;
  f.num_blocks = num_blocks;
  f.max_seq_len = max_seq_len;
  f.scale = scale;
  f.scale_log2 = scale * kLog2eF;
  f.tile_ok = tile_kernel_supported(dtype, head_dim, group) ? 1 : 0;
  f.row_ctas = row_ctas_per_sm(dtype, head_dim, group) * num_sms;
  f.tile_ctas = 2 * num_sms;
  f.dtype = dtype;
  f.plan = reinterpret_cast<PlanHeader *>(ws + lay.plan);
  f.req = reinterpret_cast<ReqInfo *>(ws + lay.req);
  f.ord = reinterpret_cast<int *>(ws + lay.ord);
  f.list_end = reinterpret_cast<long long *>(ws + lay.list_end);
  f.part_o = reinterpret_cast<float *>(ws + lay.own_o);
  f.part_lse = reinterpret_cast<float *>(ws + lay.own_lse);
  f.part_cap = lay.part_cap;
  f.sinks = c.sinks;
  f.max_qlen = c.max_query_len;
  f.partial_only = 1;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.group_start = group_start_loc;
  p.prefix_lens = prefix_lens;
  p.num_groups = num_groups;
  p.max_prefix_len = max_prefix_len;
  p.num_sms = num_sms;
  p.plan = reinterpret_cast<PrefixPlan *>(ws + lay.pplan);
  p.grp = reinterpret_cast<PrefixGroup *>(ws + lay.grp);
  p.grp_end = reinterpret_cast<int *>(ws + lay.grp_end);
  p.req_grp = reinterpret_cast<int *>(ws + lay.req_grp);
  p.part_o = reinterpret_cast<float *>(ws + lay.pre_o);
  p.part_lse = reinterpret_cast<float *>(ws + lay.pre_lse);
  p.item_cap = lay.item_cap;

  int slot = prof_begin(PA_K_PLAN, st);
  cudaError_t err = launch_dependent(prefix_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, p);
  prof_end(slot, st);
  if (err != cudaSuccess) return PA_ERR_CUDA;
  slot = prof_begin(PA_K_PREFIX, st);
  err = dtype == PA_BF16 ? launch_prefix_mma(p, c.kv_layout, num_sms, st)
                         : launch_simt(p, c.kv_layout == PA_KV_HND, num_sms, st);
  prof_end(slot, st);
  if (err != cudaSuccess) return PA_ERR_CUDA;
  s = launch_rows_and_tiles(c, f, num_sms, st, true);
  if (s != PA_OK) return s;
  slot = prof_begin(PA_K_MERGE, st);
  err = dtype == PA_BF16 ? launch_merge<__nv_bfloat16>(p, st) : launch_merge<float>(p, st);
  prof_end(slot, st);
  return err == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
