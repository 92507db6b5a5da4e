// pa_span.h -- what the kernels of pa_forward_tree and pa_forward_weights
// share: the work cut into spans of KV positions (not part of the public C ABI).
//
// A unit is one KV head of one request and up to kSpanRows of its rows (a row:
// one new token x one query head of the KV head) against the request's whole
// context, in tiles of kSpanTile positions.  All units' tiles are laid one after
// the other and cut into equal runs, one for each block of the grid, so every
// block gets the same work and a unit is split only where a run ends in it.  A
// block's share of a unit is a piece; its partial results go to slot
// unit + block, which is a piece's alone (each step from one piece to the next
// moves on by a unit, by a block, or by both).
#pragma once

#include "pa_internal.h"

namespace pa {

// Longest context taken: positions some tiles behind its end still count in 32 bits.
constexpr int kSpanMaxLen = 1 << 30;
constexpr int kSpanRows = 256;
constexpr int kSpanTile = 128;
// Work is laid out in half tiles: a tile of a unit of more than 128 rows, which keeps
// the tensor cores busy, is two (1.4 us of an SM at head_dim 128, 1.28 at 64); one of
// a unit of up to 128 rows is one where its keys come from L2, having been read for
// the request's other rows, or are half as wide (0.7 us), and two where they come
// from HBM at head_dim 128 (1.45 us).
constexpr int kSpanWide = 2;
__host__ __device__ inline int span_narrow(int nblk, int head_dim) {
  return nblk == 1 && head_dim == 128 ? 2 : 1;
}
// What a unit costs beside its tiles (queries, first scores, storing the results):
// 5 us of an SM, where there are units enough for every block; with fewer the tiles
// alone are cut, so that short contexts spread over the SMs.
constexpr int kSpanOverhead = 6;
// Requests with at most this many rows of a KV head have their scores kept for
// the sums over rows (pa_forward_weights); the others' are computed again.  A
// position's scores of 32 rows are 128 bytes written and read, its key in bf16
// 128 or 256 bytes read again and multiplied again.
constexpr int kSpanStoredRows = 32;

enum SpanMode : int {
  kSpanTree = 0,   // mask of the new tokens from bits
  kSpanVotes = 1,  // causal, scores kept, values too
  kSpanVotesOnly = 2,  // causal, scores kept, no values: the log-sum-exps alone
};

struct SpanReq {
  int q_start, q_len;  // its token rows
  int ctx;             // positions, the new tokens among them
  int nblk;            // blocks of kSpanRows rows of a KV head (0: bad, or nothing to do)
  int ntile;           // tiles of its context
  int unit0;           // first unit; unit = unit0 + kv head * nblk + block
  unsigned cost0;      // where its first unit begins in the laid-out work
  int kcost;           // laid-out work of a KV head: its blocks' one after the other,
  int ucost, ulast;    // a block's, and the last one's
  long long score0;    // first kept score, -1: not kept
};

// Laid-out work of a tile of block b of a request.
__device__ inline int span_tile_cost(const SpanReq &r, int b, int overhead) {
  return b < r.nblk - 1 || r.ulast - overhead > r.ntile ? kSpanWide : 1;
}

struct SpanPlan {
  unsigned total;  // laid-out work
  unsigned run;    // each block's share
  unsigned vote_tiles;  // (KV head, tile) of the requests whose scores are not kept
  int all_bad;     // bad query_start_loc: every row is zero
};

struct SpanParams {
  FwdParams f;
  const void *k_cache, *v_cache;
  int hnd;
  const unsigned long long *mask;  // [num_tokens][mask_words], or null
  int mask_words;
  float *weights;                  // [num_blocks][num_kv_heads][block_size], or null
  int accumulate;
  int keep_scores;
  int num_sms, grid;
  int halves, join;                // see span_row
  int one;                         // no unit has more than 128 rows
  int overhead;                    // kSpanOverhead, or 0
  int fused;                       // no planner: see span_plan_warp
  int slot_rows;
  SpanPlan *plan;
  SpanReq *req;          // [num_seqs]
  unsigned *vote_end;    // [num_seqs] inclusive sum of Hk * ntile where scores are not kept
  float *part_o;         // [slots * slot_rows][head_dim], normalised
  float *part_lse;       // base 2; +inf: a bad page in the piece's range
  float *row_lse;        // [num_tokens * num_heads], sinks included
  float *scores;         // kept scores, base 2: [kv head][row][ntile * kSpanTile] a request
};

// Where row r of a unit lies among the partials of slot `slot`.  The tensor-core
// kernel gives a unit of up to 128 rows to both of its row tiles, every other tile
// of positions each: x tells them apart (else x = 0).  It finishes units in one piece
// by itself: those of more than 128 rows, and (join) the others too.
__device__ inline long long span_row(const SpanParams &p, long long slot, int x, int r) {
  return slot * p.slot_rows + x * (p.slot_rows / 2) + r;
}

// Batches of up to this many requests (bf16) have no planner's launch: every block of
// the span kernel works the plan out for itself, a request a lane (and as many as its
// shared memory has room for).
constexpr int kSpanFusedSeqs = 20;

// Request s as its metadata say, without the sums over the requests before it; cnt:
// its units, laid-out work, kept scores and tiles of the KV heads that are summed up
// without them.
__device__ inline SpanReq span_request(const SpanParams &p, int s, unsigned &flags, int &bad,
                                       long long (&cnt)[4]) {
  const FwdParams &f = p.f;
  const int Hk = f.num_kv_heads, G = f.num_heads / Hk;
  const int longest =
      (int)min((unsigned long long)f.max_seq_len, (unsigned long long)f.max_blocks_per_seq * f.block_size);
  const int q0 = f.qsl[s], q1 = f.qsl[s + 1];
  if (q1 < q0 || (s == 0 && q0 != 0) || (s == f.num_seqs - 1 && q1 > f.num_tokens)) bad = 1;
  SpanReq r{};
  r.q_start = q0;
  r.q_len = q1 - q0;
  r.ctx = f.seq_lens[s];
  const bool len_ok = r.ctx >= 0 && r.ctx <= longest;
  const bool q_ok = r.q_len <= r.ctx && (f.max_qlen <= 0 || r.q_len <= f.max_qlen) &&
                    (!p.mask || r.q_len <= 64ll * p.mask_words);
  if (r.q_len != 0) flags |= (len_ok ? 0u : PA_DEV_BAD_SEQLEN) | (q_ok ? 0u : PA_DEV_BAD_QLEN);
  r.score0 = -1;
  cnt[0] = cnt[1] = cnt[2] = cnt[3] = 0;
  if (r.q_len > 0 && len_ok && q_ok) {
    const long long rows = (long long)r.q_len * G;
    r.nblk = (int)((rows + kSpanRows - 1) / kSpanRows);
    r.ntile = (r.ctx + kSpanTile - 1) / kSpanTile;
    const int wlast = rows - (r.nblk - 1ll) * kSpanRows > 128 ? kSpanWide : span_narrow(r.nblk, f.head_dim);
    r.ulast = r.ntile * wlast + p.overhead;
    r.ucost = r.nblk > 1 ? r.ntile * kSpanWide + p.overhead : r.ulast;
    r.kcost = (r.nblk - 1) * r.ucost + r.ulast;
    cnt[0] = (long long)Hk * r.nblk;
    cnt[1] = (long long)Hk * r.kcost;
    if (p.keep_scores && rows <= kSpanStoredRows) {
      cnt[2] = Hk * rows * r.ntile * kSpanTile;
      r.score0 = 0;
    } else if (p.keep_scores) {
      cnt[3] = (long long)Hk * r.ntile;
    }
  }
  return r;
}

// With the sums of cnt over the requests before it.
__device__ inline void span_place(SpanReq &r, const long long (&before)[4]) {
  r.unit0 = (int)before[0];
  r.cost0 = (unsigned)before[1];
  if (r.score0 >= 0) r.score0 = before[2];
}

// The plan over all requests' sums (the host has bounded the work by 2^31).
__device__ inline SpanPlan span_plan_of(const SpanParams &p, const long long (&sum)[4]) {
  const unsigned total = (unsigned)sum[1];
  return SpanPlan{total, max((total + p.grid - 1) / p.grid, (unsigned)kSpanWide), (unsigned)sum[3], 0};
}

struct alignas(16) SpanPiece {
  int q_start, q_len, ctx, req;  // the request's rows
  int kvh, t0;                   // KV head, first token of the row block
  int kv_lo, kv_hi;              // positions (kv_lo a multiple of kSpanTile)
  int ctx_pad;                   // the context in whole tiles
  int whole;                     // 1: all of the unit
  long long slot;
  long long score0;              // its kept scores: row r's position j at score0 + r * ctx_pad + j
};

// Positions that the rows of the block from token t0 on may see: all for bits,
// up to the block's last token's own position under a causal mask.
__device__ inline int span_block_end(const SpanReq &r, int t0, int tq, bool causal) {
  return causal ? r.ctx - r.q_len + min(t0 + tq, r.q_len) : r.ctx;
}
// The tile boundary at `cost` of a unit's laid-out work; w: of a tile, 1 or 2.
__device__ inline int span_tile_at(const SpanParams &p, const SpanReq &r, unsigned cost, int w) {
  return min(max((int)cost - p.overhead, 0) >> (w - 1), r.ntile);
}

// The pieces of block `cta`: the whole units of its run first, then the end of the
// unit that its run begins in, then the beginning of the one that it ends in.  So the
// blocks that share a KV head of a request all begin at its first position, and what
// one of them has brought from HBM the others find in L2 more often (12 trees of up to
// 250 tokens on up to 16384 positions, whose keys and values are 280 MB: 536 us in the
// order of the run, 527 so; 1.3 GB of 2.7 are then read from HBM).
struct SpanCursor {
  unsigned pos, end, u0;  // u0: where the unit begins
  int s, kvh, blk, cta;
  const SpanReq *req;     // [num_seqs]
  SpanReq r;
  bool put_off;           // the run's first piece is part of a unit
  unsigned first_pos, first_u0;
  int first_s, first_kvh, first_blk;

  __device__ unsigned unit_cost(const SpanReq &q, int b) const { return b == q.nblk - 1 ? q.ulast : q.ucost; }

  __device__ void step(const SpanParams &p) {  // to the next unit, where the run goes on
    u0 = pos;
    if (++blk < r.nblk) return;
    blk = 0;
    if (++kvh < p.f.num_kv_heads) return;
    kvh = 0;
    if (pos < end) {  // (then there is another request with work)
      do r = req[++s]; while (r.nblk == 0);
    }
  }

  __device__ void start(const SpanParams &p, const SpanReq *requests, const SpanPlan &plan, int block) {
    req = requests;
    cta = block;
    const unsigned long long at = (unsigned long long)block * plan.run;
    pos = (unsigned)min(at, (unsigned long long)plan.total);
    end = (unsigned)min(at + plan.run, (unsigned long long)plan.total);
    u0 = 0;
    s = kvh = blk = 0;
    put_off = false;
    if (pos >= end) return;
    int lo = 0, hi = p.f.num_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (req[mid].cost0 + (unsigned)(p.f.num_kv_heads * req[mid].kcost) > pos) hi = mid; else lo = mid + 1;
    }
    s = lo;
    r = req[s];
    unsigned rel = pos - r.cost0;
    kvh = (int)(rel / (unsigned)r.kcost);
    rel -= (unsigned)kvh * r.kcost;
    blk = (int)min(rel / (unsigned)r.ucost, (unsigned)(r.nblk - 1));
    u0 = r.cost0 + (unsigned)kvh * r.kcost + (unsigned)blk * r.ucost;
    const unsigned to = u0 + unit_cost(r, blk);
    if (pos > u0 && to < end) {
      put_off = true;
      first_pos = pos;
      first_u0 = u0;
      first_s = s;
      first_kvh = kvh;
      first_blk = blk;
      pos = to;
      step(p);
    }
  }

  // The piece [from, to) of a unit; whether it has positions.  lg: log2 of the query
  // heads of a KV head.
  __device__ bool make(const SpanParams &p, int lg, bool causal, const SpanReq &q, int req, int h, int b,
                       unsigned begin, unsigned from, unsigned to, SpanPiece &it) const {
    const int w = span_tile_cost(q, b, p.overhead);
    const int lo = span_tile_at(p, q, from - begin, w), hi = span_tile_at(p, q, to - begin, w);
    it.q_start = q.q_start;
    it.q_len = q.q_len;
    it.ctx = q.ctx;
    it.req = req;
    it.kvh = h;
    it.t0 = b * (kSpanRows >> lg);
    it.kv_lo = lo * kSpanTile;
    it.kv_hi = min(hi * kSpanTile, span_block_end(q, it.t0, kSpanRows >> lg, causal));
    it.ctx_pad = q.ntile * kSpanTile;
    it.whole = lo == 0 && hi == q.ntile;
    it.slot = (long long)q.unit0 + h * q.nblk + b + cta;
    it.score0 = q.score0 < 0 ? -1 : q.score0 + ((long long)h * q.q_len << lg) * it.ctx_pad;
    return it.kv_hi > it.kv_lo;
  }

  __device__ bool next(const SpanParams &p, int lg, bool causal, SpanPiece &it) {
    for (;;) {
      const unsigned n = pos < end ? unit_cost(r, blk) : 0;
      if (put_off && (pos >= end || u0 + n > end)) {  // no whole unit is left
        put_off = false;
        const SpanReq q = req[first_s];
        if (make(p, lg, causal, q, first_s, first_kvh, first_blk, first_u0, first_pos,
                 first_u0 + unit_cost(q, first_blk), it))
          return true;
        continue;
      }
      if (pos >= end) return false;
      const unsigned to = min(end, u0 + n);
      const bool has = make(p, lg, causal, r, s, kvh, blk, u0, pos, to, it);
      pos = to;
      if (to == u0 + n) step(p);
      if (has) return true;
    }
  }
};

// Bits of 64 positions from `at` on, as the new token in row `tok` of `mask` sees
// them: bit c stands for position at + c.  Cached positions (below `prefix`) are
// all seen; beyond ctx there is nothing.
__device__ inline unsigned long long span_bits(const unsigned long long *mask, int words, int tok,
                                               int at, int prefix, int ctx) {
  const unsigned long long *row = mask + (size_t)tok * words;
  const int n0 = at - prefix;  // as a new token
  unsigned long long bits;
  if (n0 <= -64) {
    bits = ~0ull;
  } else if (n0 < 0) {
    bits = (row[0] << -n0) | ((1ull << -n0) - 1);
  } else {
    const int w = n0 >> 6, sh = n0 & 63;
    bits = w < words ? row[w] >> sh : 0ull;
    if (sh && w + 1 < words) bits |= row[w + 1] << (64 - sh);
  }
  const int left = ctx - at;
  if (left < 64) bits &= left <= 0 ? 0ull : (1ull << left) - 1;
  return bits;
}

// The 64 positions from `at` on that the query at position `own` sees.
__device__ inline unsigned long long span_causal_bits(int at, int own) {
  const int n = own - at + 1;
  return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1;
}

// The pass over keys and values on the tensor cores (bf16; mode: a SpanMode).
cudaError_t launch_span_mma(const SpanParams &p, int mode, cudaStream_t stream);

// The weight of four scores of one row, of the positions from pos on; `own`: the row's
// token's.  A row that sees nothing (-inf) has none, and one that is not a number has
// none at the positions that it does not see (whose scores are -inf).
__device__ inline void span_vote(const float4 x, float lse, int pos, int own, float (&sum)[4]) {
  if (lse == -INFINITY) return;
  if (lse != lse) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (pos + c <= own) sum[c] += lse;
    return;
  }
  sum[0] += fast_exp2(x.x - lse);
  sum[1] += fast_exp2(x.y - lse);
  sum[2] += fast_exp2(x.z - lse);
  sum[3] += fast_exp2(x.w - lse);
}

// Adds `sum`, of the four positions from pos on, to their slots of `page`.  Positions
// of the new tokens start at their sum; positions from ctx on have no slot, nor has a
// page beyond the pool (its request is passed over; no access goes by that alone).
__device__ inline void span_add_votes(const SpanParams &p, const SpanReq &r, int page, int kvh, int pos,
                                      const float (&sum)[4]) {
  if (page < 0 || page >= p.f.num_blocks) return;
  const int bs = p.f.block_size;  // (bs % 16 == 0: one page)
  float *dst = p.weights + ((size_t)page * p.f.num_kv_heads + kvh) * bs + pos % bs;
  const int fresh = p.accumulate ? r.ctx - r.q_len : 0;
  if (pos + 4 <= r.ctx) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (pos < fresh) x = *reinterpret_cast<const float4 *>(dst);
    x.x = pos < fresh ? x.x + sum[0] : sum[0];
    x.y = pos + 1 < fresh ? x.y + sum[1] : sum[1];
    x.z = pos + 2 < fresh ? x.z + sum[2] : sum[2];
    x.w = pos + 3 < fresh ? x.w + sum[3] : sum[3];
    *reinterpret_cast<float4 *>(dst) = x;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (pos + i < r.ctx) dst[i] = (pos + i < fresh ? dst[i] : 0.f) + sum[i];
  }
}

// The sums over rows of requests whose scores were not kept, behind the rows'
// log-sum-exps: on CUDA cores (fp32) or, for launch_votes_mma, the tensor cores (bf16).
cudaError_t launch_votes(const SpanParams &p, cudaStream_t stream);
cudaError_t launch_votes_mma(const SpanParams &p, cudaStream_t stream);

}  // namespace pa
