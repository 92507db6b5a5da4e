// pa_span.cu -- attention of drafted trees (pa_forward_tree) and attention that
// adds up the weight every cached position gets (pa_forward_weights): argument
// checks, the planner, the fp32 kernel and the merge
// (pa_span_mma.cu holds the bf16 kernel).
//
// Both read a request's context once for all of its rows (a row: one new token
// x one query head of a KV head), in units of up to 256 rows cut into equal runs
// of 128-position tiles (pa_span.h).  For row r and visible positions j,
//   s_j = scale <q_r, k_j>,  out_r = sum_j e^(s_j) v_j / (sum_j e^(s_j) [+ e^sink]),
// where the new tokens' positions are visible by the bits of a mask (the
// ancestors of a drafted token) or causally.  pa_forward_weights also forms
//   W_j = sum_r e^(s_j) / (sum_i e^(s_i) [+ e^sink])
// over the rows of a KV head, which needs every row's whole sum first: the pass
// over the keys leaves each row's log-sum-exp and, for few rows, its scores; the
// kernels of pa_votes.cu then sum over the rows, position by position.
#include <algorithm>
#include <type_traits>

#include "pa_join.h"
#include "pa_span.h"

namespace pa {
namespace {

constexpr int kPlanThreads = 256;
constexpr int kMergeThreads = 256;
constexpr int kMergeGroups = kMergeThreads / 8;
constexpr int kMergeCache = 1024;  // requests whose starts the merge keeps in shared memory

// ---------------------------------------------------------------------------
// planner: one block
// ---------------------------------------------------------------------------

__global__ void __launch_bounds__(kPlanThreads) span_plan_kernel(const SpanParams p) {
  __shared__ long long scratch[4 * 33];
  const int S = p.f.num_seqs, tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  unsigned flags = 0;
  int bad = 0;
  long long sum[4] = {0, 0, 0, 0};
  for (int base = 0; base < S; base += kPlanThreads) {
    const int s = base + tid;
    SpanReq r{};
    long long cnt[4] = {0, 0, 0, 0}, own[4], tot[4];
    if (s < S) r = span_request(p, s, flags, bad, cnt);
#pragma unroll
    for (int x = 0; x < 4; ++x) own[x] = cnt[x];
    block_scan_multi<4>(cnt, scratch, tot);
    if (s < S) {
      const long long before[4] = {sum[0] + cnt[0] - own[0], sum[1] + cnt[1] - own[1], sum[2] + cnt[2] - own[2], 0};
      span_place(r, before);
      p.req[s] = r;
      p.vote_end[s] = (unsigned)(sum[3] + cnt[3]);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) sum[x] += tot[x];
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      atomicOr(p.f.status, PA_DEV_BAD_QSL);
      *p.plan = SpanPlan{0, 1, 0, 1};
    }
    return;
  }
  if (flags) atomicOr(p.f.status, flags);
  if (tid == 0) *p.plan = span_plan_of(p, sum);
}

// ---------------------------------------------------------------------------
// the pass over keys and values on CUDA cores (fp32)
// ---------------------------------------------------------------------------
// Eight threads share up to four rows (each every eighth 16-byte group of their
// head_dim values), 128 rows a pass; 64 keys and values at a time in shared
// memory, the next ones loaded meanwhile, each load of them used for the four
// rows.  The scores of 8 keys are reduced over the eight threads so that each ends
// up with one key's, join the running maximum and sum there, and the weights are
// handed round again.  Bound by the multiply-adds and the shuffles between them:
// 64 trees of up to 16 tokens, 32/8 heads of 128, up to 8192 positions: 3.06 ms, 17
// TFLOP/s.  Up to 16 rows are taken by 2, 4 or 8 sets of warps, each on its share of a
// tile's keys (64 decodes on those positions, 4 rows: 0.58 ms, 4.0 TB/s; with all warps
// on the same keys 2.76 ms).
constexpr int kSimtThreads = 256;
constexpr int kSimtKeys = 64;
constexpr int kSimtRows = 4;  // rows of a thread, 32 apart
constexpr uint32_t kHidden = 0x80000000u;  // -0, the weight of a hidden position

template <int D>
struct SpanTileBuf {
  float k[kSimtKeys][D], v[kSimtKeys][D];
};

// Four values from global to shared memory, or zeros.
__device__ inline void copy4(float *dst, const float *src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(take ? 16 : 0)
               : "memory");
}

template <int D, int MODE>
__global__ void __launch_bounds__(kSimtThreads, 1) span_simt_kernel(const SpanParams p) {
  constexpr int N = D / 8;  // values of a row that a thread holds
  constexpr bool VALUES = MODE != kSpanVotesOnly, CAUSAL = MODE != kSpanTree;
  extern __shared__ __align__(16) uint8_t s_raw[];
  SpanTileBuf<D> *s_tile = reinterpret_cast<SpanTileBuf<D> *>(s_raw);
  const FwdParams &f = p.f;
  const int tid = threadIdx.x, lane = tid & 31, c = tid & 7;
  const int Hk = f.num_kv_heads, G = f.num_heads / Hk, bs = f.block_size, lg = __ffs(G) - 1;
  pdl_wait();
  pdl_trigger();
  const SpanPlan plan = *p.plan;
  const float *kc = static_cast<const float *>(p.k_cache);
  const float *vc = static_cast<const float *>(p.v_cache);
  SpanCursor cur;
  cur.start(p, p.req, plan, blockIdx.x);
  SpanPiece it;
  while (cur.next(p, lg, CAUSAL, it)) {
    const int32_t *bt = f.block_table + (size_t)it.req * f.max_blocks_per_seq;
    const int rows = min(kSpanRows, (it.q_len - it.t0) * G), prefix = it.ctx - it.q_len;
    // (a pass of fewer rows than threads' rows holds one or two a thread)
    auto pass = [&](int row0, auto rows_c) {
      constexpr int R = decltype(rows_c)::value;
      // up to 16 rows: 2, 4 or 8 sets of warps take them, each its share of the keys
      const int left = rows - row0, sets = R > 1 || left > 16 ? 1 : left > 8 ? 2 : left > 4 ? 4 : 8;
      const int per = 32 / sets, set = (tid >> 3) / per, row1 = row0 + (tid >> 3) % per;
      float qv[R][N], o[R][VALUES ? N : 1], m[R], l[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int row = min(row1 + r * 32, rows - 1);
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
          if constexpr (VALUES) o[r][i] = o[r][i + 1] = o[r][i + 2] = o[r][i + 3] = 0.f;
        }
      }
      int bad = 0;
      auto load = [&](SpanTileBuf<D> &t, int lo) {
        // a run of 16 positions lies in one page
        constexpr int STEP = kSimtThreads / (D / 4);  // keys of one round of the threads
        const int x = tid % (D / 4) * 4;
        int page[kSimtKeys / 16];
#pragma unroll
        for (int run = 0; run < kSimtKeys / 16; ++run) {
          const int at = lo + run * 16;
          page[run] = at < it.kv_hi ? bt[at / bs] : -1;
          if (at < it.kv_hi && (page[run] < 0 || page[run] >= f.num_blocks)) {
            bad = 1;
            page[run] = -1;
          }
        }
#pragma unroll
        for (int run = 0; run < kSimtKeys / 16; ++run) {
          const int slot = (lo + run * 16) % bs;
          const size_t row = page[run] < 0 ? 0
                             : p.hnd       ? ((size_t)page[run] * Hk + it.kvh) * bs + slot
                                           : ((size_t)page[run] * bs + slot) * Hk + it.kvh;
#pragma unroll
          for (int i = tid / (D / 4); i < 16; i += STEP) {
            const int j = run * 16 + i;
            const bool in = page[run] >= 0 && lo + j < it.kv_hi;
            const size_t at = (in ? row + (size_t)i * (p.hnd ? 1 : Hk) : 0) * D + x;
            copy4(&t.k[j][x], kc + at, in);
            if constexpr (VALUES) copy4(&t.v[j][x], vc + at, in);
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      int buf = 0;
      load(s_tile[0], it.kv_lo);
      for (int lo = it.kv_lo; lo < it.kv_hi; lo += kSimtKeys, buf ^= 1) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // the tile is there, and the other one has been read
        const SpanTileBuf<D> &t = s_tile[buf];
        if (lo + kSimtKeys < it.kv_hi) load(s_tile[buf ^ 1], lo + kSimtKeys);
        for (int j0 = set * 8; j0 < kSimtKeys && lo + j0 < it.kv_hi; j0 += sets * 8) {
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
          const int pos = lo + j0 + c;  // this thread's key
          const bool in = pos < it.kv_hi;
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
            const int row = row1 + r * 32;
            const int tl = it.t0 + min(row, rows - 1) / G;
            bool seen = in;
            if (in && pos >= prefix) {
              const int n = pos - prefix;  // as a new token
              if constexpr (CAUSAL) seen = n <= tl;
              else seen = (p.mask[(size_t)(it.q_start + tl) * p.mask_words + (n >> 6)] >> (n & 63)) & 1;
            }
            const float sc = seen ? w[r][0] : -INFINITY;
            if constexpr (MODE != kSpanTree) {
              if (it.score0 >= 0 && in && row < rows)
                p.scores[it.score0 + (long long)row * it.ctx_pad + pos] = sc;
            }
            float mx = sc;
#pragma unroll
            for (int h = 4; h >= 1; h >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, h));
            if (mx > m[r]) {
              const float a = m[r] == -INFINITY ? 0.f : exp2f(m[r] - mx);
              l[r] *= a;
              if constexpr (VALUES) {
#pragma unroll
                for (int i = 0; i < N; ++i) o[r][i] *= a;
              }
              m[r] = mx;
            }
            w[r][0] = seen ? exp2f(sc - (m[r] == -INFINITY ? 0.f : m[r])) : __uint_as_float(kHidden);
            l[r] += w[r][0];
          }
          if constexpr (VALUES) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float4 v4[N / 4];
#pragma unroll
              for (int i = 0; i < N / 4; ++i)
                v4[i] = *reinterpret_cast<const float4 *>(&t.v[j0 + j][i * 32 + c * 4]);
#pragma unroll
              for (int r = 0; r < R; ++r) {
                const float wj = __shfl_sync(0xffffffffu, w[r][0], (lane & 24) | j);
                // (a hidden position's value may be anything, NaN too)
                if (__float_as_uint(wj) != kHidden) {
#pragma unroll
                  for (int i = 0; i < N / 4; ++i) {
                    ffma2(o[r][4 * i], o[r][4 * i + 1], v4[i].x, v4[i].y, wj, wj);
                    ffma2(o[r][4 * i + 2], o[r][4 * i + 3], v4[i].z, v4[i].w, wj, wj);
                  }
                }
              }
            }
          }
        }
      }
      bad = __syncthreads_or(bad);  // (and both tiles have been read)
      if (bad && tid == 0) atomicOr(f.status, PA_DEV_BAD_BLOCK);
      if (R == 1 && sets > 1) {  // the sets' sums meet in the tiles' place
        constexpr int LD = (VALUES ? N : 0) + 2;
        float *own = reinterpret_cast<float *>(s_raw) + tid * LD;
        own[0] = m[0];
        own[1] = l[0];
        if constexpr (VALUES) {
#pragma unroll
          for (int i = 0; i < N; ++i) own[2 + i] = o[0][i];
        }
        __syncthreads();
        for (int k = 1; set == 0 && k < sets; ++k) {
          const float *other = own + k * per * 8 * LD;
          const float top = fmaxf(m[0], other[0]);
          const float a = m[0] == top ? 1.f : exp2f(m[0] - top), b = other[0] == top ? 1.f : exp2f(other[0] - top);
          m[0] = top;
          l[0] = l[0] * a + other[1] * b;
          if constexpr (VALUES) {
#pragma unroll
            for (int i = 0; i < N; ++i) o[0][i] = o[0][i] * a + other[2 + i] * b;
          }
        }
        __syncthreads();  // (read, before the next pass's tiles)
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int h = 4; h >= 1; h >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], h);
        const int row = row1 + r * 32;
        if (row < rows && set == 0) {
          const long long at = span_row(p, it.slot, 0, row);
          if constexpr (VALUES) {
            const float inv = l[r] == 0.f || bad ? 0.f : 1.f / l[r];
#pragma unroll
            for (int i = 0; i < N; i += 4)
              *reinterpret_cast<float4 *>(p.part_o + at * D + i * 8 + c * 4) =
                  make_float4(o[r][i] * inv, o[r][i + 1] * inv, o[r][i + 2] * inv, o[r][i + 3] * inv);
          }
          if (c == 0)
            p.part_lse[at] = bad ? INFINITY : l[r] == 0.f ? -INFINITY : m[r] + log2f(l[r]);
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
// A row is one (token, query head).  Its partials are those of its unit's pieces:
//   L = log2(sum_i 2^(lse_i) [+ 2^sink]),  out = sum_i 2^(lse_i - L) O_i.
// Eight lanes hold a row's head_dim values and walk its partials four at a time;
// W such groups share a row's partials and meet in shared memory.  Rows of units that
// the pass has finished are passed over.  Bound by the reads of the partials, which are
// in L2, and with few rows by its latency (5 us by itself for one tree of 8 tokens).

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

// Where the partials of one row lie.
struct SpanRow {
  unsigned u0, len;     // its unit's laid-out work
  int c0, n;            // its first block, and the partials that there may be
  int w, ntile, blk_end, br;
  long long unit;
  bool pairs;
};

// Row of token i and head h of request r.  *done: of a unit in one piece, which the
// tensor-core kernel has finished.
__device__ inline SpanRow span_locate(const SpanParams &p, const SpanPlan &plan, const SpanReq &r, int i, int h,
                                      int lg, bool causal, bool *done) {
  SpanRow x;
  const int tq = kSpanRows >> lg, b = i / tq, kvh = h >> lg;
  const bool last = b == r.nblk - 1;
  x.br = ((i - b * tq) << lg) + (h & ((1 << lg) - 1));
  x.unit = (long long)r.unit0 + kvh * r.nblk + b;
  x.u0 = r.cost0 + (unsigned)kvh * r.kcost + (unsigned)b * r.ucost;
  x.len = last ? r.ulast : r.ucost;
  x.w = span_tile_cost(r, b, p.overhead);
  x.ntile = r.ntile;
  x.c0 = (int)(x.u0 / plan.run);
  x.blk_end = span_block_end(r, b * tq, tq, causal);
  x.n = (int)((x.u0 + x.len - 1) / plan.run) - x.c0 + 1;
  x.pairs = p.halves && (r.q_len - b * tq) << lg <= 128;
  *done = false;
  if (p.halves && (p.join || !x.pairs)) {
    for (int c = x.c0; c < x.c0 + x.n; ++c) {  // (pieces before it may have no tile)
      const int t1 = span_tile_at(p, r, min(x.u0 + x.len, (unsigned)(c + 1) * plan.run) - x.u0, x.w);
      if (t1 == r.ntile) *done = true;
      if (t1 > 0) break;
    }
  }
  if (x.pairs) x.n *= 2;
  return x;
}

// The e-th of them; -1: the piece has no tiles (its unit's overhead alone, or tiles
// behind the causal end), or no second one for the second half.
__device__ inline long long span_partial(const SpanParams &p, const SpanPlan &plan, const SpanRow &x, int e) {
  const int c = x.c0 + (x.pairs ? e >> 1 : e), half = x.pairs ? e & 1 : 0;
  const unsigned from = max(x.u0, (unsigned)c * plan.run) - x.u0,
                 to = min(x.u0 + x.len, (unsigned)(c + 1) * plan.run) - x.u0;
  const int t0 = min(max((int)from - p.overhead, 0) >> (x.w - 1), x.ntile),
            t1 = min(max((int)to - p.overhead, 0) >> (x.w - 1), x.ntile);
  if (min(t1 * kSpanTile, x.blk_end) <= (t0 + half) * kSpanTile) return -1;
  return span_row(p, x.unit + c, half, x.br);
}

// ---- the sums over rows of requests whose scores are kept (up to kSpanStoredRows
// rows): the scores are read once, four positions a thread.  OWN: each block works out
// the rows' log-sum-exps from their partials, so that this runs beside the merge;
// else the merge has left them.
constexpr int kKeptChunk = 4 * kMergeThreads;

template <bool OWN>
__device__ inline void votes_kept(const SpanParams &p, int block, int blocks, int chunks) {
  __shared__ float s_lse[kSpanStoredRows];
  const FwdParams &f = p.f;
  const int tid = threadIdx.x, Hk = f.num_kv_heads, lg = __ffs(f.num_heads / Hk) - 1, bs = f.block_size;
  pdl_wait();  // the plan, and what else the kernel before has left
  const SpanPlan plan = *p.plan;
  const int units = f.num_seqs * Hk;
  for (long long item = block; !plan.all_bad && item < (long long)chunks * units; item += blocks) {
    const int at = (int)(item / units) * kKeptChunk, sh = (int)(item - (long long)at / kKeptChunk * units);
    const int s = sh / Hk, kvh = sh - s * Hk, pos = at + tid * 4;
    const SpanReq r = p.req[s];
    if (r.nblk == 0 || r.score0 < 0 || at >= r.ctx) continue;  // (the same for all threads)
    const int R = r.q_len << lg, prefix = r.ctx - r.q_len;
    const bool mine = pos < r.ctx;
    const int page = mine ? f.block_table[(size_t)s * f.max_blocks_per_seq + pos / bs] : 0;
    const long long pad = (long long)r.ntile * kSpanTile;
    const float *src = p.scores + r.score0 + (long long)kvh * R * pad + pos;
    float4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (mine && i < R) x[i] = __ldcg(reinterpret_cast<const float4 *>(src + i * pad));
    __syncthreads();  // s_lse of the item before is read
    if (!OWN && tid < R)
      s_lse[tid] = __ldcg(p.row_lse + (size_t)(r.q_start + (tid >> lg)) * f.num_heads + (kvh << lg) +
                          (tid & ((1 << lg) - 1)));
    if (OWN && tid < R) {
      bool done;
      const int h = (kvh << lg) + (tid & ((1 << lg) - 1));
      const SpanRow row = span_locate(p, plan, r, tid >> lg, h, lg, true, &done);
      float m = -INFINITY, l = 0.f;
      if (done) {  // (the sink in it)
        m = __ldcg(p.row_lse + (size_t)(r.q_start + (tid >> lg)) * f.num_heads + h);
        l = 1.f;
      }
      for (int e = 0; e < row.n && !done; ++e) {
        const long long from = span_partial(p, plan, row, e);
        const float v = from < 0 ? -INFINITY : __ldcg(p.part_lse + from);
        if (v == -INFINITY) continue;
        const float top = join_top(m, v);
        l = l * (m == top ? 1.f : m == -INFINITY ? 0.f : fast_exp2(m - top)) + (v == top ? 1.f : fast_exp2(v - top));
        m = top;
      }
      if (f.sinks && !done && m != INFINITY && m != -INFINITY) {
        const float sink2 = __ldg(f.sinks + h) * kLog2eF, top = join_top(m, sink2);
        l = l * fast_exp2(m - top) + fast_exp2(sink2 - top);
        m = top;
      }
      s_lse[tid] = m == INFINITY || m == -INFINITY ? m : m + log2f(l);
    }
    __syncthreads();
    // (the last token sees all of the request's pages: a bad one leaves the weights)
    if (!mine || s_lse[R - 1] == INFINITY) continue;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < R) span_vote(x[i], s_lse[i], pos, prefix + (i >> lg), sum);
#pragma unroll 4
    for (int i = 4; i < R; ++i)
      span_vote(__ldcg(reinterpret_cast<const float4 *>(src + i * pad)), s_lse[i], pos, prefix + (i >> lg), sum);
    span_add_votes(p, r, page, kvh, pos, sum);
  }
}

// more: another kernel of the call follows.  (A next call's blocks would only take
// these ones' places: 64 decodes 223.7 us, 222.5 without.)
__global__ void __launch_bounds__(kMergeThreads) votes_kept_kernel(const SpanParams p, int chunks, int more) {
  if (more) pdl_trigger();
  votes_kept<false>(p, blockIdx.x, gridDim.x, chunks);
}

// merge_blocks: the blocks that merge; the others sum over rows.
template <typename T, int D, int W, int MODE>
__global__ void __launch_bounds__(kMergeThreads) span_merge_kernel(const SpanParams p, int merge_blocks, int chunks) {
  constexpr bool VALUES = MODE != kSpanVotesOnly, CAUSAL = MODE != kSpanTree;
  constexpr int V = VALUES ? D / 32 : 1;  // float4 values a lane holds
  constexpr int ROWS = kMergeGroups / W;  // rows a block works on at a time
  __shared__ float4 s_o[W > 1 ? kMergeGroups : 1][W > 1 ? 8 * V : 1];
  __shared__ float s_m[kMergeGroups], s_l[kMergeGroups];
  __shared__ int s_qsl[kMergeCache];
  const FwdParams &f = p.f;
  const int S = f.num_seqs, H = f.num_heads, lg = __ffs(H / f.num_kv_heads) - 1;
  const int tid = threadIdx.x, lane = tid & 7, grp = tid >> 3, part = grp % W;
  const long long rows = (long long)f.num_tokens * H;
  // (blocks of several steps keep their places to themselves: 12 wide trees 558 us, 555 so)
  if ((long long)merge_blocks * ROWS >= rows) pdl_trigger();
  if constexpr (MODE != kSpanTree) {
    if ((int)blockIdx.x >= merge_blocks) {
      votes_kept<true>(p, blockIdx.x - merge_blocks, gridDim.x - merge_blocks, chunks);
      return;
    }
  }
  // The plan too: where the span kernel makes it, it is a running kernel's until here.
  pdl_wait();
  T *out = static_cast<T *>(f.out);
  const SpanPlan plan = *p.plan;
  // a decode batch: token tok is most likely request tok's, no search
  const bool one = S == f.num_tokens && f.max_qlen == 1;
  const bool cached = !one && S <= kMergeCache;
  if (cached) {
    for (int s = tid; s < S; s += kMergeThreads) s_qsl[s] = f.qsl[s];
    __syncthreads();
  }
  for (long long row0 = (long long)blockIdx.x * ROWS; row0 < rows; row0 += (long long)merge_blocks * ROWS) {
    const long long row = row0 + grp / W;
    float4 acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, l = 0.f;
    int h = 0, n = 0;
    SpanRow at{};
    bool mine = row < rows;  // (not a row behind the last request)
    if (mine && !plan.all_bad) {
      const int tok = (int)(row / H);
      h = (int)(row - (long long)tok * H);
      int lo = 0, hi = S - 1;
      if (one && p.req[tok].q_start == tok && p.req[tok].q_len == 1) lo = hi = tok;
      while (lo < hi) {  // the last request that starts at or before tok: its own
        const int mid = (lo + hi + 1) >> 1;
        if ((cached ? s_qsl[mid] : f.qsl[mid]) <= tok) lo = mid; else hi = mid - 1;
      }
      const SpanReq r = p.req[lo];
      const int i = tok - r.q_start;
      mine = i < r.q_len;
      if (mine && r.nblk > 0) {
        bool done;
        at = span_locate(p, plan, r, i, h, lg, CAUSAL, &done);
        n = done ? 0 : at.n;
        if (done) mine = false;
      }
    }
    for (int e0 = part; e0 < n; e0 += 4 * W) {
      float lse[4];
      float4 x[4][V];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int e = e0 + u * W;
        lse[u] = -INFINITY;
        const long long from = e < n ? span_partial(p, plan, at, e) : -1;
        if (from < 0) continue;
        lse[u] = __ldcg(p.part_lse + from);
        if constexpr (VALUES) {
          const float *src = p.part_o + from * D + lane * 4;
#pragma unroll
          for (int v = 0; v < V; ++v) x[u][v] = __ldcg(reinterpret_cast<const float4 *>(src + v * 32));
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (lse[u] == -INFINITY) continue;  // no such partial, or one without a visible position
        const float top = join_top(m, lse[u]);
        // (equal infinities: a bad page, which m tells)
        const float a = m == -INFINITY || m == top ? (m == top ? 1.f : 0.f) : fast_exp2(m - top);
        const float wt = lse[u] == top ? 1.f : fast_exp2(lse[u] - top);
        m = top;
        l = fmaf(l, a, wt);
        if constexpr (VALUES) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            acc[v].x = fmaf(acc[v].x, a, wt * x[u][v].x);
            acc[v].y = fmaf(acc[v].y, a, wt * x[u][v].y);
            acc[v].z = fmaf(acc[v].z, a, wt * x[u][v].z);
            acc[v].w = fmaf(acc[v].w, a, wt * x[u][v].w);
          }
        }
      }
    }
    if constexpr (W > 1) {
      __syncthreads();  // the rows before are read
      if (lane == 0) {
        s_m[grp] = m;
        s_l[grp] = l;
      }
      if constexpr (VALUES) {
#pragma unroll
        for (int v = 0; v < V; ++v) s_o[grp][v * 8 + lane] = acc[v];
      }
      __syncthreads();
      if (part == 0) {
        float top = m;
        for (int k = 1; k < W; ++k) top = join_top(top, s_m[grp + k]);
        const float a = m == top ? 1.f : m == -INFINITY ? 0.f : fast_exp2(m - top);
        l *= a;
        if constexpr (VALUES) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            acc[v].x *= a;
            acc[v].y *= a;
            acc[v].z *= a;
            acc[v].w *= a;
          }
        }
        for (int k = 1; k < W; ++k) {
          const float mk = s_m[grp + k];
          if (mk == -INFINITY) continue;
          const float b = mk == top ? 1.f : fast_exp2(mk - top);
          l = fmaf(s_l[grp + k], b, l);
          if constexpr (VALUES) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
              const float4 o = s_o[grp + k][v * 8 + lane];
              acc[v].x = fmaf(o.x, b, acc[v].x);
              acc[v].y = fmaf(o.y, b, acc[v].y);
              acc[v].z = fmaf(o.z, b, acc[v].z);
              acc[v].w = fmaf(o.w, b, acc[v].w);
            }
          }
        }
        m = top;
      }
    }
    if (mine && part == 0) {
      // the sink joins the denominator once, with no value; a row that sees
      // nothing, or a bad page, is zero
      const bool bad = m == INFINITY, none = m == -INFINITY;
      if (!bad && !none && f.sinks) {
        const float sink2 = __ldg(f.sinks + h) * kLog2eF, top = join_top(m, sink2);
        const float k = fast_exp2(m - top);
        l = l * k + fast_exp2(sink2 - top);
        m = top;
        if constexpr (VALUES) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            acc[v].x *= k;
            acc[v].y *= k;
            acc[v].z *= k;
            acc[v].w *= k;
          }
        }
      }
      if (p.row_lse && lane == 0) p.row_lse[row] = bad || none ? m : m + log2f(l);
      if constexpr (VALUES) {
        const float inv = bad || none ? 0.f : 1.f / l;
        T *dst = out + row * D + lane * 4;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (bad || none) store4<T>(dst + v * 32, 0.f, 0.f, 0.f, 0.f);
          else store4<T>(dst + v * 32, acc[v].x * inv, acc[v].y * inv, acc[v].z * inv, acc[v].w * inv);
        }
      }
    }
  }
}

template <typename T, int D, int MODE>
cudaError_t launch_merge_d(const SpanParams &p, long long most, int most_rows, cudaStream_t st) {
  // Groups a row: as many as the SMs hold at once (two blocks each), and no more
  // than a row's partials fill, four at a time.
  const long long rows = (long long)p.f.num_tokens * p.f.num_heads, sms = p.num_sms;
  const int fit = rows <= 4 * sms ? 16 : rows <= 8 * sms ? 8 : rows <= 16 * sms ? 4 : 1;
  const int W = std::min(fit, most <= 4 ? 1 : most <= 16 ? 4 : most <= 32 ? 8 : 16);
  auto kern = W == 16 ? span_merge_kernel<T, D, 16, MODE>
              : W == 8 ? span_merge_kernel<T, D, 8, MODE>
              : W == 4 ? span_merge_kernel<T, D, 4, MODE> : span_merge_kernel<T, D, 1, MODE>;
  long long blocks = std::min(ceil_div_ll(rows * W, kMergeGroups), sms * 8);
  if (MODE == kSpanTree)
    return launch_dependent(kern, dim3((unsigned)blocks), dim3(kMergeThreads), 0, st, p, (int)blocks, 0);
  // The sums over rows of kept scores beside the merge where the two blocks an SM that
  // its registers leave hold them at once (4 decodes of up to 1000 positions 16.5 us,
  // 18.5 behind it); else behind it, eight blocks an SM (64 decodes of up to 8192
  // positions 223 us, 249 beside it).
  const long long chunks = ceil_div_ll(std::max(p.f.max_seq_len, 1), kKeptChunk);
  const long long items = chunks * p.f.num_seqs * p.f.num_kv_heads;
  if (items + blocks <= 2 * sms) {
    // (without an output the merge is for rows whose scores are not kept)
    if (MODE == kSpanVotesOnly && most_rows <= kSpanStoredRows) blocks = 0;
    return launch_dependent(kern, dim3((unsigned)(blocks + items)), dim3(kMergeThreads), 0, st, p, (int)blocks,
                            (int)chunks);
  }
  const cudaError_t e =
      launch_dependent(kern, dim3((unsigned)blocks), dim3(kMergeThreads), 0, st, p, (int)blocks, (int)chunks);
  if (e != cudaSuccess) return e;
  return launch_dependent(votes_kept_kernel, dim3((unsigned)std::min(items, 8 * sms)), dim3(kMergeThreads), 0, st,
                          p, (int)chunks, (int)(most_rows > kSpanStoredRows));
}

template <int D, int MODE>
cudaError_t launch_simt_d(const SpanParams &p, cudaStream_t st) {
  constexpr int kSmem = 2 * (int)sizeof(SpanTileBuf<D>);
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = set_smem_attrs_once(span_simt_kernel<D, MODE>, kSmem, done);
  if (e != cudaSuccess) return e;
  return launch_dependent(span_simt_kernel<D, MODE>, dim3(p.grid), dim3(kSimtThreads), kSmem, st, p);
}

template <int MODE>
cudaError_t launch_pass(const SpanParams &p, cudaStream_t st) {
  if (p.f.dtype == PA_BF16) return launch_span_mma(p, MODE, st);
  return p.f.head_dim == 128 ? launch_simt_d<128, MODE>(p, st) : launch_simt_d<64, MODE>(p, st);
}

template <int MODE>
cudaError_t launch_merge(const SpanParams &p, long long most, int most_rows, cudaStream_t st) {
  const bool bf16 = p.f.dtype == PA_BF16;
  if (p.f.head_dim == 128)
    return bf16 ? launch_merge_d<__nv_bfloat16, 128, MODE>(p, most, most_rows, st)
                : launch_merge_d<float, 128, MODE>(p, most, most_rows, st);
  return bf16 ? launch_merge_d<__nv_bfloat16, 64, MODE>(p, most, most_rows, st)
              : launch_merge_d<float, 64, MODE>(p, most, most_rows, st);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

constexpr int kMaxGrid = 160;  // blocks that the partials' bound allows for

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct SpanLayout {
  size_t plan, req, vote_end, part_o, part_lse, row_lse, scores, total;
  int slot_rows, one;
  bool ok;  // the extents are ones that the kernels count in 32 bits
};

// Host-side bounds of what the planner lays out, from the extents alone.
SpanLayout span_layout(int dtype, int num_seqs, int num_tokens, int num_heads, int num_kv_heads,
                       int head_dim, int max_seq_len, int max_query_len, bool votes, bool values) {
  SpanLayout l{};
  const long long S = num_seqs > 0 ? num_seqs : 1, T = num_tokens, H = num_heads, Hk = num_kv_heads,
                  G = H / Hk, msl = max_seq_len > 0 ? max_seq_len : 1;
  const long long most = max_query_len > 0 ? std::min<long long>(max_query_len, T) : T;  // new tokens
  const long long units =
      Hk * std::min(ceil_div_ll(T * G, kSpanRows) + S, S * ceil_div_ll(most * G, kSpanRows));
  const long long tiles = ceil_div_ll(msl, kSpanTile) * kSpanWide + kSpanOverhead;
  l.ok = units * tiles < (1ll << 31) - (1 << 20) && msl <= kSpanMaxLen;
  // two rows of partials for each row of a unit of up to 128
  l.one = most * G <= 128;
  l.slot_rows = l.one ? (int)(2 * ceil_div_ll(most * G, 4) * 4) : kSpanRows;
  const long long slots = units + kMaxGrid;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  l.plan = take(sizeof(SpanPlan));
  l.req = take(S * sizeof(SpanReq));
  l.vote_end = take(S * sizeof(unsigned));
  l.part_o = take(values ? (size_t)slots * l.slot_rows * head_dim * sizeof(float) : 0);
  l.part_lse = take((size_t)slots * l.slot_rows * sizeof(float));
  if (votes) {
    l.row_lse = take((size_t)T * H * sizeof(float));
    const long long kept = std::min(T * G, S * std::min<long long>(most * G, kSpanStoredRows));
    l.scores = take((size_t)(kept * Hk) * ceil_div_ll(msl, kSpanTile) * kSpanTile * sizeof(float));
  }
  l.total = off;
  (void)dtype;
  return l;
}

bool extents_ok(int num_seqs, int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                int max_seq_len, int max_query_len) {
  return num_seqs >= 0 && num_tokens >= 0 && num_heads > 0 && num_kv_heads > 0 &&
         num_heads % num_kv_heads == 0 && head_dim > 0 && max_seq_len >= 0 && max_query_len >= 0 &&
         (long long)num_tokens * num_heads <= (1ll << 40) / head_dim;
}

struct SpanCall {
  FwdCall c;
  const unsigned long long *mask = nullptr;
  int mask_words = 0;
  float *weights = nullptr;
  int accumulate = 0;
  void *stream = nullptr;
  void *workspace = nullptr;
  size_t workspace_bytes = 0;
};

// Options of both calls: sinks, layout and max_query_len.
pa_status take_options(const pa_forward_options *o, FwdCall *c) {
  if (!o) return PA_OK;
  if (o->sinks && (reinterpret_cast<uintptr_t>(o->sinks) & 3)) return PA_ERR_INVALID_ARG;
  if ((o->kv_layout != PA_KV_NHD && o->kv_layout != PA_KV_HND) || o->sliding_window < 0 ||
      o->max_query_len < 0 || (o->alibi_sqrt != 0 && o->alibi_sqrt != 1))
    return PA_ERR_INVALID_ARG;
  // a drafted token's position is its depth's, an evicted cache's not its slot's
  if (o->sliding_window || o->alibi_slopes) return PA_ERR_UNSUPPORTED;
  c->sinks = o->sinks;
  c->kv_layout = o->kv_layout;
  c->max_query_len = o->max_query_len;
  return PA_OK;
}

template <int MODE>
pa_status span_call(const SpanCall &sc) {
  const FwdCall &c = sc.c;
  constexpr bool votes = MODE != kSpanTree, values = MODE != kSpanVotesOnly;
  for (const int32_t *x : {c.block_table, c.seq_lens, c.qsl})
    if (reinterpret_cast<uintptr_t>(x) & 3) return PA_ERR_INVALID_ARG;
  const SpanLayout lay = span_layout(c.dtype, c.num_seqs, c.num_tokens, c.num_heads, c.num_kv_heads,
                                     c.head_dim, c.max_seq_len, c.max_query_len, votes, values);
  if (!lay.ok) return PA_ERR_UNSUPPORTED;
  if (!sc.workspace || sc.workspace_bytes < lay.total) return PA_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(sc.workspace) & 255) return PA_ERR_INVALID_ARG;
  // (queries are read again behind the first outputs' stores)
  const long long rows = (long long)c.num_tokens * c.num_heads, row_bytes = c.head_dim * (c.dtype == PA_F32 ? 4 : 2);
  if (any_overlap({{c.out, rows, row_bytes}}, {{c.q, rows, row_bytes}})) return PA_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(sc.stream);
  SpanParams p{};
  void *lib_ws = nullptr;
  int num_sms = 0;
  pa_status s = device_resources(st, 0, &lib_ws, &p.f.status, &num_sms);
  if (s != PA_OK) return s;
  uint8_t *ws = static_cast<uint8_t *>(sc.workspace);
  FwdParams &f = p.f;
  f.q = c.q;
  f.out = c.out;
  f.block_table = c.block_table;
  f.seq_lens = c.seq_lens;
  f.qsl = c.qsl;
  f.num_seqs = c.num_seqs;
  f.num_tokens = c.num_tokens;
  f.num_heads = c.num_heads;
  f.num_kv_heads = c.num_kv_heads;
  f.head_dim = c.head_dim;
  f.block_size = c.block_size;
  f.max_blocks_per_seq = c.max_blocks_per_seq;
  f.num_blocks = c.num_blocks;
  f.max_seq_len = c.max_seq_len;
  f.scale = c.scale;
  f.scale_log2 = c.scale * kLog2eF;
  f.dtype = c.dtype;
  f.sinks = c.sinks;
  f.max_qlen = c.max_query_len;
  p.k_cache = c.k_cache;
  p.v_cache = c.v_cache;
  p.hnd = c.kv_layout == PA_KV_HND;
  p.mask = sc.mask;
  p.mask_words = sc.mask_words;
  p.weights = sc.weights;
  p.accumulate = sc.accumulate;
  p.keep_scores = votes;
  p.num_sms = num_sms;
  p.grid = std::min(num_sms, kMaxGrid);
  p.halves = c.dtype == PA_BF16;
  p.one = lay.one;
  const long long units = (long long)c.num_kv_heads *
                          std::max<long long>(c.num_seqs, ceil_div_ll((long long)c.num_tokens * (c.num_heads / c.num_kv_heads), kSpanRows));
  p.overhead = units >= p.grid ? kSpanOverhead : 0;
  // Units of up to 128 rows finished in one row tile: where they are many, and have the
  // rows of trees (64 trees of 16 tokens, 4 heads each: 206 us, 200 so; the rows of
  // decode steps are few, 64 of them 222 us, 226 so, and the code that small calls wait
  // for grows: one tree 1.1 us more).
  p.join = p.halves && !votes && p.overhead > 0;
  p.slot_rows = lay.slot_rows;
  p.plan = reinterpret_cast<SpanPlan *>(ws + lay.plan);
  p.req = reinterpret_cast<SpanReq *>(ws + lay.req);
  p.vote_end = reinterpret_cast<unsigned *>(ws + lay.vote_end);
  p.part_o = reinterpret_cast<float *>(ws + lay.part_o);
  p.part_lse = reinterpret_cast<float *>(ws + lay.part_lse);
  p.row_lse = votes ? reinterpret_cast<float *>(ws + lay.row_lse) : nullptr;
  p.scores = votes ? reinterpret_cast<float *>(ws + lay.scores) : nullptr;

  // A launch less for few requests: one user's tree of 8 tokens 13.7 -> 12.9 us in a
  // graph, 23.4 -> 21.7 launched one by one.
  p.fused = c.dtype == PA_BF16 && c.num_seqs <= kSpanFusedSeqs;
  int slot;
  cudaError_t err = cudaSuccess;
  if (!p.fused) {
    slot = prof_begin(PA_K_PLAN, st);
    err = launch_dependent(span_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, p);
    prof_end(slot, st);
    if (err != cudaSuccess) return PA_ERR_CUDA;
  }
  slot = prof_begin(PA_K_SPAN, st);
  err = launch_pass<MODE>(p, st);
  prof_end(slot, st);
  if (err != cudaSuccess) return PA_ERR_CUDA;
  // partials that a row may have: two of each block that shares its unit
  const long long blocks = 2 * std::min<long long>(ceil_div_ll(c.max_seq_len, kSpanTile) + 1, p.grid);
  // rows of a KV head that one request may have
  const int most_rows = (int)std::min<long long>(
      (long long)(c.max_query_len > 0 ? std::min(c.max_query_len, c.num_tokens) : c.num_tokens) *
          (c.num_heads / c.num_kv_heads), 1 << 30);
  slot = prof_begin(PA_K_MERGE, st);
  err = launch_merge<MODE>(p, blocks, most_rows, st);
  prof_end(slot, st);
  if (err != cudaSuccess) return PA_ERR_CUDA;
  if (votes && most_rows > kSpanStoredRows) {
    slot = prof_begin(PA_K_VOTES, st);
    err = launch_votes(p, st);
    prof_end(slot, st);
    if (err != cudaSuccess) return PA_ERR_CUDA;
  }
  return PA_OK;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" {

size_t pa_forward_tree_workspace_bytes(pa_dtype dtype, int num_seqs, int num_tokens, int num_heads,
                                       int num_kv_heads, int head_dim, int max_seq_len,
                                       int max_query_len) {
  if (!extents_ok(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, max_seq_len, max_query_len))
    return 0;
  const SpanLayout l = span_layout(dtype, num_seqs, num_tokens, num_heads, num_kv_heads, head_dim,
                                   max_seq_len, max_query_len, false, true);
  return l.ok ? l.total : 0;
}

pa_status pa_forward_tree(const void *q, const void *k_cache, const void *v_cache,
                          const int32_t *block_table, const int32_t *seq_lens,
                          const int32_t *query_start_loc, const uint64_t *tree_mask, int num_heads,
                          int num_kv_heads, int head_dim, int block_size, float scale, void *out,
                          void *stream, pa_dtype dtype, int num_seqs, int num_tokens,
                          int mask_words, int max_blocks_per_seq, int num_blocks, int max_seq_len,
                          const pa_forward_options *options, void *workspace,
                          size_t workspace_bytes) {
  SpanCall sc;
  sc.c = FwdCall{q, k_cache, v_cache, block_table, seq_lens, query_start_loc, num_heads,
                 num_kv_heads, head_dim, block_size, scale, out, dtype, num_seqs, num_tokens,
                 max_blocks_per_seq, num_blocks, max_seq_len, 0};
  sc.stream = stream;
  if (mask_words < 0) return PA_ERR_INVALID_ARG;
  pa_status s = take_options(options, &sc.c);
  if (s != PA_OK) return s;
  s = fwd_check(sc.c);
  if (s != PA_OK || num_tokens == 0) return s;
  if (num_seqs == 0 || !tree_mask || mask_words == 0 || (reinterpret_cast<uintptr_t>(tree_mask) & 7))
    return PA_ERR_INVALID_ARG;
  sc.mask = reinterpret_cast<const unsigned long long *>(tree_mask);
  sc.mask_words = mask_words;
  sc.workspace = workspace;
  sc.workspace_bytes = workspace_bytes;
  return span_call<kSpanTree>(sc);
}

size_t pa_forward_weights_workspace_bytes(pa_dtype dtype, int num_seqs, int num_tokens,
                                          int num_heads, int num_kv_heads, int head_dim,
                                          int max_seq_len, int max_query_len) {
  if (!extents_ok(num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, max_seq_len, max_query_len))
    return 0;
  const SpanLayout l = span_layout(dtype, num_seqs, num_tokens, num_heads, num_kv_heads, head_dim,
                                   max_seq_len, max_query_len, true, true);
  return l.ok ? l.total : 0;
}

pa_status pa_forward_weights(const void *q, const void *k_cache, const void *v_cache,
                             const int32_t *block_table, const int32_t *seq_lens,
                             const int32_t *query_start_loc, int num_heads, int num_kv_heads,
                             int head_dim, int block_size, float scale, void *out, float *weights,
                             int accumulate, void *stream, pa_dtype dtype, int num_seqs,
                             int num_tokens, int max_blocks_per_seq, int num_blocks,
                             int max_seq_len, const pa_forward_options *options, void *workspace,
                             size_t workspace_bytes) {
  SpanCall sc;
  // (without an output the values are not read: the checks are those of the keys)
  sc.c = FwdCall{q, k_cache, out ? v_cache : k_cache, block_table, seq_lens, query_start_loc,
                 num_heads, num_kv_heads, head_dim, block_size, scale,
                 out ? out : const_cast<void *>(q), dtype, num_seqs, num_tokens,
                 max_blocks_per_seq, num_blocks, max_seq_len, 0};
  sc.stream = stream;
  if (accumulate != 0 && accumulate != 1) return PA_ERR_INVALID_ARG;
  pa_status s = take_options(options, &sc.c);
  if (s != PA_OK) return s;
  s = fwd_check(sc.c);
  if (s != PA_OK || num_tokens == 0) return s;
  if (num_seqs == 0 || !weights || (reinterpret_cast<uintptr_t>(weights) & 15)) return PA_ERR_INVALID_ARG;
  sc.c.out = out;
  sc.weights = weights;
  sc.accumulate = accumulate;
  sc.workspace = workspace;
  sc.workspace_bytes = workspace_bytes;
  return out ? span_call<kSpanVotes>(sc) : span_call<kSpanVotesOnly>(sc);
}

}  // extern "C"
