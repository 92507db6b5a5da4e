// pa_span_mma.cu -- the pass over keys and values of pa_forward_tree and
// pa_forward_weights on the tensor cores (bf16).
//
// Mathematics: for a piece's rows (pa_span.h) and its positions [kv_lo, kv_hi),
//   S = Q K^T,  P = 2^(scale log2e S - ref),  l = sum P,  O = sum P V,
// tile by tile of 128 positions, one pass, with a reference ref for each row that
// moves (O and l rescaled) only when weights outgrow it.  Tiles that reach the new
// tokens are masked by select, 64 positions at a time from a word of bits.
//
// One CTA per SM (224 KB of shared memory, all 512 TMEM columns), 16 warps:
//   warps 0-3, 4-7  softmax of the two row tiles, thread = row (TMEM lane)
//   warps 8, 9      each issues one row tile's S = Q K^T (M = 128, N = 128) and
//                   O += P V (P from TMEM, N = head_dim)
//   warps 10-13     TMA: K boxes (10, 11) and V boxes (12, 13) into rings
//   warps 14, 15    the values of the new tokens (below)
// A piece of more than 128 rows is two row tiles on the same tiles of positions,
// whose products take turns.  A piece of up to 128 rows, as trees and decode steps
// mostly have, goes to both row tiles too: each takes every other tile of positions
// with sums of its own, so that two chains of S, softmax and P V run side by side.
//
// Values that a row does not see must not reach it, but 0 x NaN would: in tiles that
// reach hidden positions, warps 14 and 15 look at the values and zero the rows that
// are not finite; rows that see such a position get it back behind the piece, from
// memory (each_zeroed).
// A box that lies past the piece, or on a bad page, is loaded from a page beyond
// the pool, which TMA fills with zeros: every tile has the same byte count.
//
// What bounds it: units of up to 128 rows at head_dim 128 the stream of keys and
// values (64 trees of up to 16 tokens, 32/8 heads, up to 8192 positions: 188 to 192 us for
// 1.15 GB, 6.0 to 6.2 TB/s, 90 to 92 % of the measured copy rate); units of 256 rows the chain of a
// row tile's scores, softmax and value product, the two row tiles in turns (12 trees of
// up to 250 tokens, 64/4 heads, up to 16384 positions: 530 to 545 us, 1.2 PFLOP/s, a tile
// some 3100 clocks of which the products are 2200; the tensor pipe is busy 58 % of the
// time); one small tree the latencies from the plan to the partials (8 us).
#include "pa_span.h"
#include "pa_umma.cuh"

namespace pa {
namespace {

constexpr int kBN = kSpanTile;
// Half a tile's weights may sum to this much before the reference moves up to its
// maximum: far from overflow in bf16 and in the fp32 sums, so a row's reference
// is mostly its first tile's maximum, and no maximum is taken of the others.
constexpr float kMostSum = 1048576.f;
constexpr float kMostLead = 14.f;  // 64 weights of 2^14 sum to that much
constexpr int kThreads = 512;
constexpr int kIssueWarp = 8, kLoad0 = 10, kCheck0 = 14;
// launch registers 512 x 128; the softmax warpgroups take 176, the others keep 80
constexpr int kSoftmaxRegs = 176, kOtherRegs = 80;
constexpr int kPieces = 8;  // pieces that the first loading warp may be ahead
constexpr uint32_t kTmemCols = 512, kTmemO = 256;  // S of row tile x at 128 x, O at 256 + 128 x

// ONE: no piece has more than 128 rows; the second query tile's place holds values
template <int D, bool ONE>
struct Cfg {
  static constexpr int NH = D / 64;            // 128-byte chunks of a row
  static constexpr int Q_TILE = NH * 128 * 128;
  static constexpr int KV_BYTES = NH * kBN * 128;
  static constexpr int KST = D == 128 ? 3 : 5, VST = D == 128 ? (ONE ? 3 : 2) : 5;
  static constexpr int OFF_K = (ONE ? 1 : 2) * Q_TILE;
  static constexpr int OFF_V = OFF_K + KST * KV_BYTES;
  static constexpr int OFF_BAR = OFF_V + VST * KV_BYTES;
  // barriers
  static constexpr int Q_FULL = 0, Q_FREE = 1, S_FULL = 2, O_HALF = 4, O_DONE = 6, P_HALF = 8,
                       P_FULL = 10, O_FREE = 12, TURN = 14, END = 16, K_FULL = 17, V_FULL = K_FULL + KST,
                       K_FREE = V_FULL + VST, V_FREE = K_FREE + KST, V_OK = V_FREE + VST,
                       PAIR = V_OK + VST, PIECE = PAIR + 1, PIECE_FREE = PIECE + kPieces,
                       NBAR = PIECE_FREE + kPieces;
  static constexpr int OFF_PIECE = (OFF_BAR + NBAR * 8 + 15) & ~15;
  static constexpr int OFF_MISC = OFF_PIECE + kPieces * (int)sizeof(SpanPiece);
  static constexpr int OFF_PAIR = OFF_MISC + 144;     // references and sums of the second row tile
  static constexpr int OFF_REQ = OFF_PAIR + 128 * 8;  // requests, where this kernel plans
  static constexpr int SMEM = OFF_REQ + kSpanFusedSeqs * (int)sizeof(SpanReq);
  static constexpr uint32_t IDESC_S = umma_idesc_bf16(128, kBN, 0);
  static constexpr uint32_t IDESC_PV = umma_idesc_bf16(128, D, 1);
  static_assert(SMEM <= 232448, "shared memory of one CTA");
};

// The plan of up to kSpanFusedSeqs requests by one warp; req: theirs, for this block.
// `leave`: written to the workspace too, for the kernels behind this one.
__device__ inline SpanPlan span_plan_warp(const SpanParams &p, SpanReq *req, int lane, bool leave) {
  unsigned flags = 0;
  int bad = 0;
  SpanReq r{};
  long long cnt[4] = {0, 0, 0, 0}, end[4], sum[4];
  if (lane < p.f.num_seqs) r = span_request(p, lane, flags, bad, cnt);
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    end[x] = cnt[x];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, end[x], o);
      if (lane >= o) end[x] += y;
    }
    sum[x] = __shfl_sync(0xffffffffu, end[x], 31);
  }
  bad = __any_sync(0xffffffffu, bad);
  flags = bad ? PA_DEV_BAD_QSL : __reduce_or_sync(0xffffffffu, flags);
  const SpanPlan plan = bad ? SpanPlan{0, 1, 0, 1} : span_plan_of(p, sum);
  const long long before[4] = {end[0] - cnt[0], end[1] - cnt[1], end[2] - cnt[2], end[3] - cnt[3]};
  span_place(r, before);
  if (lane < p.f.num_seqs) {
    req[lane] = r;
    if (leave) {
      p.req[lane] = r;
      p.vote_end[lane] = (unsigned)end[3];
    }
  }
  if (leave && lane == 0) {
    *p.plan = plan;
    if (flags) atomicOr(p.f.status, flags);
  }
  __syncwarp();
  return plan;
}

// The first position that some row of the piece's block may not see.
template <bool CAUSAL>
__device__ inline int first_hidden(const SpanPiece &it) {
  return it.ctx - it.q_len + (CAUSAL ? it.t0 + 1 : 0);
}

__device__ inline bool not_finite(uint4 v) {  // of eight bf16 values, any
  const uint32_t x = (v.x & 0x7f807f80u) + 0x00800080u, y = (v.y & 0x7f807f80u) + 0x00800080u,
                 z = (v.z & 0x7f807f80u) + 0x00800080u, w = (v.w & 0x7f807f80u) + 0x00800080u;
  return ((x | y | z | w) & 0x80008000u) != 0;
}

// The positions whose values were zeroed and which one row sees: use(w, v), w the row's
// weight of the position, normalised by inv, v the values.  Rare and slow.
template <int D, bool CAUSAL, typename Use>
__device__ inline void each_zeroed(const SpanParams &p, const SpanPiece &it, int row, bool half, int x,
                                   float ref, float inv, Use use) {
  const FwdParams &f = p.f;
  const int Hk = f.num_kv_heads, G = f.num_heads / Hk, bs = f.block_size, prefix = it.ctx - it.q_len;
  const int tl = it.t0 + row / G, head = it.kvh * G + row % G;
  const __nv_bfloat16 *q =
      static_cast<const __nv_bfloat16 *>(f.q) + ((size_t)(it.q_start + tl) * f.num_heads + head) * D;
  const int32_t *bt = f.block_table + (size_t)it.req * f.max_blocks_per_seq;
  for (int pos = max(it.kv_lo, first_hidden<CAUSAL>(it)); pos < it.kv_hi; ++pos) {
    if (half && (((pos - it.kv_lo) / kBN) & 1) != x) continue;
    const int n = pos - prefix;
    if (n >= 0) {
      const bool seen = CAUSAL ? n <= tl
                               : (p.mask[(size_t)(it.q_start + tl) * p.mask_words + (n >> 6)] >> (n & 63)) & 1;
      if (!seen) continue;
    }
    const int page = bt[pos / bs], slot = pos % bs;
    const size_t at = (p.hnd ? ((size_t)page * Hk + it.kvh) * bs + slot : ((size_t)page * bs + slot) * Hk + it.kvh) * D;
    const uint4 *v = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.v_cache) + at);
    bool odd = false;
    for (int c = 0; c < D / 8; ++c) odd |= not_finite(v[c]);
    if (!odd) continue;
    const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(p.k_cache) + at;
    const __nv_bfloat16 *vv = static_cast<const __nv_bfloat16 *>(p.v_cache) + at;
    float s = 0.f;
    for (int d = 0; d < D; ++d) s = fmaf(__bfloat162float(q[d]), __bfloat162float(k[d]), s);
    use(fast_exp2(s * f.scale_log2 - ref) * inv, vv);
  }
}

// They are added to the row's partial.
template <int D, bool CAUSAL>
__device__ __noinline__ void fix_partial(const SpanParams &p, const SpanPiece it, int row, bool half,
                                         int x, float ref, float inv, float *out) {
  each_zeroed<D, CAUSAL>(p, it, row, half, x, ref, inv, [&](float w, const __nv_bfloat16 *v) {
    for (int d = 0; d < D; ++d) out[d] += w * __bfloat162float(v[d]);
  });
}

// They are added to a finished row that was left in its partial's place, `sum`, before it
// is rounded, once.
template <int D, bool CAUSAL>
__device__ __noinline__ void fix_finished(const SpanParams &p, const SpanPiece it, int row, float ref,
                                          float inv, float *sum, __nv_bfloat16 *out) {
  each_zeroed<D, CAUSAL>(p, it, row, false, 0, ref, inv, [&](float w, const __nv_bfloat16 *v) {
    for (int d = 0; d < D; ++d) sum[d] += w * __bfloat162float(v[d]);
  });
  for (int d = 0; d < D; ++d) out[d] = __float2bfloat16_rn(sum[d]);
}

// JOIN: units of up to 128 rows in one piece are finished here too, in one row tile.
template <int D, int MODE, bool ONE, bool JOIN>
__global__ void __launch_bounds__(kThreads, 1)
    span_mma_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ SpanParams p,
                    int box) {
  using C = Cfg<D, ONE>;
  constexpr bool VALUES = MODE != kSpanVotesOnly, CAUSAL = MODE != kSpanTree, VOTES = MODE != kSpanTree;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
  // piece k: s_fix[k % 16] is k + 1 when values of it were zeroed, s_bad[k % 16] when it
  // met a bad page (the warps that say so are at most 8 pieces ahead)
  volatile int *s_fix = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 8);  // [16]
  volatile int *s_bad = s_fix + 16;                                                // [16]
  const FwdParams &f = p.f;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = f.num_heads / f.num_kv_heads, TQ = 128 / G, bs = f.block_size, lg = __ffs(G) - 1;
  if (smem_u32(smem) & 1023) {  // the same for every thread: all leave together
    if (tid == 0) atomicOr(f.status, PA_DEV_INTERNAL);
    pdl_wait();  // (the plan's words are the call's before until then)
    if (p.fused && blockIdx.x == 0 && tid == 0) *p.plan = SpanPlan{0, 1, 0, 1};
    return;
  }
  if (tid == 0) {
    prefetch_tensor_map(&tm_q);
    prefetch_tensor_map(&tm_k);
    if (VALUES) prefetch_tensor_map(&tm_v);
  }
  // (a barrier a thread: one thread's loop over them takes a small call half a microsecond)
  if (tid < C::NBAR) {
    // P and O: the row tile's four warps; a ring stage: two loading warps, two
    // issuing ones, two that look at the values
    const int b = tid;
    const bool softmax = (b >= C::P_HALF && b < C::TURN) || b == C::PAIR, ring = b >= C::K_FULL;
    const int readers = VALUES ? 15 : 11;  // warps that read the pieces
    mbar_init(&bar[b], b >= C::PIECE_FREE ? readers : b >= C::PIECE ? 1 : softmax ? 4
                       : ring || b == C::Q_FREE || b == C::END ? 2 : 1);
    fence_mbar_init();
  }
  if (tid < 32) s_fix[tid] = 0;
  if (warp == kIssueWarp) tc_alloc(s_tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  bool dead = false;
  float2 *const s_pair = reinterpret_cast<float2 *>(smem + C::OFF_PAIR);
  SpanPiece *const s_piece = reinterpret_cast<SpanPiece *>(smem + C::OFF_PIECE);
  SpanPiece it;
  uint32_t pieces = 0;  // taken by this warp
  // The next piece, which the first loading warp has left; false behind the last one.
  auto next_piece = [&]() {
    const uint32_t at = pieces % kPieces;
    mbar_wait(&bar[C::PIECE + at], (pieces / kPieces) & 1, dead, f.status);
    it = s_piece[at];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[C::PIECE_FREE + at]);
    ++pieces;
    return it.kv_hi > 0 && !dead;
  };

  if (warp >= kIssueWarp) {
    reg_dec<kOtherRegs>();
    pdl_wait();  // the plan
    if (warp >= kCheck0) {
      // -------------------------------------------------- values of hidden positions
      if constexpr (VALUES) {
        const int t = tid - kCheck0 * 32;
        uint32_t vs = 0, vr = 0;
        for (int k = 0; next_piece(); ++k) {
          const int hidden = first_hidden<CAUSAL>(it);
          for (int lo = it.kv_lo; lo < it.kv_hi; lo += kBN) {
            mbar_wait(&bar[C::V_FULL + vs], vr & 1, dead, f.status);
            if (lo + kBN > hidden && !dead) {
              bool zeroed = false;
#pragma unroll 1
              for (int r = t; r < kBN; r += 64) {
                if (lo + r < hidden) continue;
                // row r of the box r / box, each box holding all chunks of its rows
                uint8_t *row = smem + C::OFF_V + vs * C::KV_BYTES + r * 128 + (C::NH - 1) * (r & ~(box - 1)) * 128;
                bool odd = false;
#pragma unroll
                for (int c = 0; c < C::NH; ++c)
#pragma unroll
                  for (int u = 0; u < 8; ++u)  // (each lane from its own unit on: no bank conflicts)
                    odd |= not_finite(*reinterpret_cast<const uint4 *>(row + c * box * 128 + ((u + lane) & 7) * 16));
                if (odd) {
                  for (int c = 0; c < C::NH; ++c)
                    for (int u = 0; u < 8; ++u)
                      *reinterpret_cast<uint4 *>(row + c * box * 128 + u * 16) = make_uint4(0, 0, 0, 0);
                  fence_proxy_async();
                  zeroed |= lo + r < it.kv_hi;  // (behind it nobody looks)
                }
              }
              if (zeroed) {
                s_fix[k & 15] = k + 1;
                __threadfence_block();
              }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[C::V_OK + vs]);
            if (++vs == C::VST) vs = 0, ++vr;
          }
        }
      }
    } else if (warp >= kLoad0) {
      // ------------------------------------------------------------- loads
      // Two warps for K and two for V, each half of a tile's boxes, one box a
      // lane: K one box per 64-wide chunk and run of `box` positions (the S
      // product needs a uniform row stride), V one box per run, all chunks.
      const bool is_v = warp >= kLoad0 + 2;
      const int half = (warp - kLoad0) & 1, runs = kBN / box;
      const int nbox = is_v ? runs : runs * C::NH;
      const int b0 = half * nbox / 2, nb = (half + 1) * nbox / 2 - b0;
      const int mine = b0 + lane;             // this lane's box
      const int run = mine % runs, chunk = mine / runs;
      const uint32_t bytes = (uint32_t)(nb * box * 128 * (is_v ? C::NH : 1));
      const uint32_t at = is_v ? run * C::NH * box * 128 : chunk * kBN * 128 + run * box * 128;
      const int stages = is_v ? C::VST : C::KST;
      uint64_t *full = &bar[is_v ? C::V_FULL : C::K_FULL], *free = &bar[is_v ? C::V_FREE : C::K_FREE];
      uint8_t *ring = smem + (is_v ? C::OFF_V : C::OFF_K) + at;
      uint32_t st = 0, round = 0, items = 0, queries = 0;
      // The first of them makes the block's pieces and leaves them to the others; one
      // without positions ends the list.
      SpanCursor cur;
      if (warp == kLoad0) {
        SpanReq *const s_req = reinterpret_cast<SpanReq *>(smem + C::OFF_REQ);
        if (p.fused) cur.start(p, s_req, span_plan_warp(p, s_req, lane, blockIdx.x == 0), blockIdx.x);
        else cur.start(p, p.req, *p.plan, blockIdx.x);
        pdl_trigger();
      }
      auto make_piece = [&]() {
        if (!cur.next(p, lg, CAUSAL, it)) it.kv_lo = it.kv_hi = 0;
        const uint32_t at = pieces % kPieces;
        if (pieces >= kPieces) mbar_wait(&bar[C::PIECE_FREE + at], (pieces / kPieces - 1) & 1, dead, f.status);
        if (lane == 0) {
          s_piece[at] = it;
          mbar_arrive(&bar[C::PIECE + at]);
        }
        __syncwarp();
        ++pieces;
        return it.kv_hi > 0 && !dead;
      };
      for (; (VALUES || !is_v) && !dead && (warp == kLoad0 ? make_piece() : next_piece()); ++items) {
        const int32_t *bt = f.block_table + (size_t)it.req * f.max_blocks_per_seq;
        auto page_of = [&](int pos) {
          int page = f.num_blocks;  // past the pool: zeros
          if (lane < nb && pos < it.kv_hi) {
            const int x = bt[pos / bs];
            if (x >= 0 && x < f.num_blocks) {
              page = x;
            } else {  // marks all of the piece's rows
              atomicOr(f.status, PA_DEV_BAD_BLOCK);
              s_bad[items & 15] = (int)items + 1;
              __threadfence_block();
            }
          }
          return page;
        };
        if (warp == kLoad0 && lane == 0) {
          const int tiles = !ONE && (it.q_len - it.t0) * G > 128 ? 2 : 1;
          if (items > 0) mbar_wait(&bar[C::Q_FREE], (items - 1) & 1, dead, f.status);
          if (!dead) {
            mbar_arrive_expect_tx(&bar[C::Q_FULL], tiles * C::Q_TILE);
            ++queries;
          }
          for (int x = 0; x < tiles && !dead; ++x)
            for (int h = 0; h < C::NH; ++h)
              tma_load_3d(smem + x * C::Q_TILE + h * 128 * 128, &tm_q, h * 64, it.kvh * G,
                          it.q_start + it.t0 + x * TQ, &bar[C::Q_FULL]);
        }
        int pos = it.kv_lo + run * box;
        int page = page_of(pos), next = page_of(pos + kBN);
        for (int lo = it.kv_lo; lo < it.kv_hi; lo += kBN) {
          const int after = page_of(pos + 2 * kBN);  // its latency passes during the wait
          if (lane == 0) {
            if (round > 0) mbar_wait(&free[st], (round - 1) & 1, dead, f.status);
            if (!dead) mbar_arrive_expect_tx(&full[st], bytes);
          }
          dead = __any_sync(0xffffffffu, dead);
          if (dead) break;  // timed out: the stage is not free
          if (lane < nb) {
            uint8_t *dst = ring + st * C::KV_BYTES;
            if (is_v) {
              tma_load_5d(dst, &tm_v, 0, pos % bs, 0, it.kvh, page, &full[st]);
              // with two stages of values (256 rows): the tile behind them to L2 meanwhile
              if (C::VST == 2 && after < f.num_blocks)
                tma_prefetch_5d(&tm_v, 0, (pos + 2 * kBN) % bs, 0, it.kvh, after);
            } else {
              tma_load_4d(dst, &tm_k, chunk * 64, it.kvh, pos % bs, page, &full[st]);
            }
          }
          __syncwarp();
          page = next;
          next = after;
          pos += kBN;
          if (++st == (uint32_t)stages) {
            st = 0;
            ++round;
          }
        }
      }
      // No copy may land after the CTA is gone, not even if its readers timed out.
      if (lane == 0) {
        bool late = false;
        for (uint32_t s = 0; s < (uint32_t)stages; ++s) {
          const uint32_t fills = round + (s < st);
          if (fills > 0) mbar_wait(&full[s], (fills - 1) & 1, late, f.status);
        }
        if (queries > 0) mbar_wait(&bar[C::Q_FULL], (queries - 1) & 1, late, f.status);
      }
    } else {
      // ------------------------------------------------------------- products
      // The warp of row tile x: the value product of its weights, and behind it
      // the scores of its next tile of positions.  With two row tiles the warps
      // take turns, two products a turn, so that each softmax has the other row
      // tile's products to run beside.  Both warps take every stage of the rings
      // and free it, by a commit or, where the tile is the other's, by an arrival.
      const int x = warp - kIssueWarp;
      const uint32_t sk = smem_u32(smem) + C::OFF_K, sv = smem_u32(smem) + C::OFF_V;
      const uint32_t tm_s = tmem + x * 128, tm_o = tmem + kTmemO + x * 128;
      uint32_t ks = 0, kr = 0, vs = 0, vr = 0;  // ring stage and round
      uint32_t items = 0, n = 0, mine = 0;      // pieces, own tiles, pieces with tiles here
      uint32_t turn = 0;
      auto take_turn = [&]() {
        if (x == 1 || turn > 0) mbar_wait(&bar[C::TURN + x], (turn - 1 + x) & 1, dead, f.status);
        ++turn;
      };
      auto pass_turn = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[C::TURN + (x ^ 1)]);
      };
      auto skip_k = [&]() {
        mbar_wait(&bar[C::K_FULL + ks], kr & 1, dead, f.status);
        if (lane == 0) mbar_arrive(&bar[C::K_FREE + ks]);
        if (++ks == C::KST) ks = 0, ++kr;
      };
      auto skip_v = [&]() {
        mbar_wait(&bar[C::V_OK + vs], vr & 1, dead, f.status);
        if (lane == 0) mbar_arrive(&bar[C::V_FREE + vs]);
        if (++vs == C::VST) vs = 0, ++vr;
      };
      while (next_piece()) {
        const bool two = !ONE && (it.q_len - it.t0) * G > 128;
        const int nt = (it.kv_hi - it.kv_lo + kBN - 1) / kBN;
        const int t0 = two ? 0 : x, dt = two ? 1 : 2;  // own tiles t0, t0 + dt, ..
        const uint32_t sq = smem_u32(smem) + (two ? x * C::Q_TILE : 0);
        auto scores = [&](uint32_t d) {
          const uint32_t a = desc_lo(sq, 16), b = desc_lo(sk + ks * C::KV_BYTES, 16);
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {  // 16 columns: 32 bytes, 4 to a chunk
            const uint32_t off = (kk / 4) * (128 * 128 / 16) + (kk % 4) * 2;
            mma_ss(d, a + off, b + off, C::IDESC_S, kk > 0);
          }
        };
        mbar_wait(&bar[C::Q_FULL], items & 1, dead, f.status);
        ++items;
        if (t0 >= nt) {  // a single tile, the other's
          skip_k();
          if constexpr (VALUES) {
            skip_v();
            // (nor does a row tile fall pieces behind: s_fix)
            mbar_wait(&bar[C::O_FREE + x], mine & 1, dead, f.status);
          }
          if (lane == 0) mbar_arrive(&bar[C::Q_FREE]);
          continue;
        }
        if constexpr (!VALUES) {
          // scores alone, into two buffers in turn: columns 128 x and 256 + 128 x
          for (int t = 0; t < nt; ++t) {
            if (!two && (t & 1) != x) {
              skip_k();
              continue;
            }
            mbar_wait(&bar[C::K_FULL + ks], kr & 1, dead, f.status);
            // the softmax has read the buffer's tile before (its dry round at first)
            if (n < 2) mbar_wait(&bar[C::O_FREE + x], 0, dead, f.status);
            else mbar_wait(&bar[(n & 1 ? C::P_FULL : C::P_HALF) + x], ((n >> 1) - 1) & 1, dead, f.status);
            scores(tm_s + (n & 1) * 256);
            commit(&bar[(n & 1 ? C::O_DONE : C::S_FULL) + x]);
            commit(&bar[C::K_FREE + ks]);
            if (t + dt >= nt) commit(&bar[C::Q_FREE]);
            if (++ks == C::KST) ks = 0, ++kr;
            ++n;
          }
          continue;
        }
        auto scores_done = [&](bool last) {  // last: of the piece, which is then done with Q
          commit(&bar[C::S_FULL + x]);
          commit(&bar[C::K_FREE + ks]);
          if (last) commit(&bar[C::Q_FREE]);
          if (++ks == C::KST) ks = 0, ++kr;
        };
        if (t0 == 1) skip_k();
        mbar_wait(&bar[C::K_FULL + ks], kr & 1, dead, f.status);
        // (the weights of the piece before have been read: O_DONE was awaited;
        // and the dry round is over)
        if (mine == 0) mbar_wait(&bar[C::O_FREE + x], 0, dead, f.status);
        if (two) take_turn();
        scores(tm_s);
        if (two) pass_turn();
        scores_done(t0 + dt >= nt);
        if (t0 == 1) skip_v();
        for (int t = t0; t < nt; t += dt, ++n) {
          const bool more = t + dt < nt;
          mbar_wait(&bar[C::V_OK + vs], vr & 1, dead, f.status);
          if (!two && t + 1 < nt) skip_k();
          if (more) mbar_wait(&bar[C::K_FULL + ks], kr & 1, dead, f.status);
          // O of the piece before has been stored (phase 0 is the dry round's)
          if (t == t0) mbar_wait(&bar[C::O_FREE + x], mine & 1, dead, f.status);
          // the leading offset steps to the next 64-wide chunk of the box
          const uint32_t b = desc_lo(sv + vs * C::KV_BYTES, box * 128);
          mbar_wait(&bar[C::P_HALF + x], n & 1, dead, f.status);
          if (two) take_turn();
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk) {  // 16 V rows
            if (kk == kBN / 32) {
              commit(&bar[C::O_HALF + x]);
              mbar_wait(&bar[C::P_FULL + x], n & 1, dead, f.status);
              tc_fence_after();
            }
            // row r of the box r / box, each box holding all chunks of its rows
            const uint32_t r = kk * 16, off = r * 8 + (C::NH - 1) * (r & ~(uint32_t)(box - 1)) * 8;
            mma_ts(tm_o, tm_s + kk * 8, b + off, C::IDESC_PV, t > t0 || kk > 0);
          }
          commit(&bar[C::O_DONE + x]);
          commit(&bar[C::V_FREE + vs]);
          if (++vs == C::VST) vs = 0, ++vr;
          // the scores go over the weights that the product reads
          mbar_wait(&bar[C::O_DONE + x], n & 1, dead, f.status);
          if (more) scores(tm_s);
          if (two) pass_turn();
          if (more) scores_done(t + 2 * dt >= nt);
          if (!two && t + 1 < nt) skip_v();
        }
        ++mine;
      }
      // nor may a product's commit
      bool late = false;
      commit(&bar[C::END]);
      mbar_wait(&bar[C::END], 0, late, f.status);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------------- softmax
    reg_inc<kSoftmaxRegs>();
    const int x = warp >> 2, r = tid & 127;  // row tile, row of it == TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tm_s0 = tmem + lane_off + x * 128, tm_o = tmem + lane_off + kTmemO + x * 128;
    const float c2 = f.scale_log2;
    // 2^(c s - ref) as one multiply-add needs c > 0 (the maximum is then c max s)
    const bool fold = c2 > 0.f;
    const float cs = fold ? c2 : 1.f;
    uint32_t n = 0, joined = 0;
    // The first round is dry: a tile of whatever TMEM holds, no barrier touched
    // and nothing stored, run before the plan is awaited.  It brings this
    // code into the instruction cache.
    int k = -1;  // piece
    it.q_start = it.q_len = it.req = it.kvh = it.t0 = it.kv_lo = it.ctx = it.ctx_pad = 0;
    it.kv_hi = kBN;
    it.slot = it.whole = 0;
    it.score0 = -1;
    for (;;) {
      const bool dry = k < 0;
      const int all = (it.q_len - it.t0) * G;
      const bool two = !ONE && all > 128;
      const int row0 = two ? x * 128 : 0, dt = two ? kBN : 2 * kBN;
      const int lo0 = it.kv_lo + (two || dry ? 0 : x * kBN);
      const int rows = dry ? 128 : min(128, all - row0);
      if (rows > 0 && lo0 < it.kv_hi) {
        const bool warp_active = (warp & 3) * 32 < rows;  // its other rows are padding
        const int prefix = it.ctx - it.q_len, seen = dry ? kBN : min(first_hidden<CAUSAL>(it), it.kv_hi);  // by all rows
        const int tl = min(it.t0 + (row0 + r) / G, it.q_len - 1);  // (padding rows: the last token's)
        float ref = 0.f, l = 0.f;  // the weights' reference exponent and their sum
        for (int lo = lo0; lo < it.kv_hi; lo += dt, n += !dry) {
          const uint32_t tm_s = tm_s0 + (VALUES ? 0 : (n & 1) * 256);
          uint64_t *const s_full = VALUES ? &bar[C::S_FULL + x] : &bar[(n & 1 ? C::O_DONE : C::S_FULL) + x];
          if (!dry) mbar_wait(s_full, VALUES ? n & 1 : (n >> 1) & 1, dead, f.status);
          tc_fence_after();
          if (warp_active) {
            uint32_t ua[2][32], ub[2][32], pw[32];
            // The 64 scores of columns c0 on, to be completed by take(): awaited,
            // scaled where the scale does not fold, hidden ones masked; kept for
            // the sums over rows where these are wanted.
            auto load = [&](uint32_t(&u)[2][32], int c0) {
              tc_ld32(tm_s + c0, u[0]);
              tc_ld32(tm_s + c0 + 32, u[1]);
            };
            auto take = [&](uint32_t(&u)[2][32], int c0, bool keep) {
              wait_ld(u[0], u[1]);
              if (!fold) {
#pragma unroll
                for (int c = 0; c < 64; ++c)
                  u[c / 32][c % 32] = __float_as_uint(__uint_as_float(u[c / 32][c % 32]) * c2);
              }
              if (__builtin_expect(lo + c0 + 64 > seen, 0)) {
                const unsigned long long bits =
                    CAUSAL ? span_causal_bits(lo + c0, prefix + tl)
                           : span_bits(p.mask, p.mask_words, it.q_start + tl, lo + c0, prefix, it.ctx);
#pragma unroll
                for (int c = 0; c < 64; ++c)
                  if (!((uint32_t)(bits >> (c & 32)) >> (c & 31) & 1)) u[c / 32][c % 32] = 0xff800000u;  // -inf
              }
              if constexpr (VOTES) {
                if (keep && it.score0 >= 0 && r < rows && !dry) {
                  float *dst = p.scores + it.score0 + (long long)r * it.ctx_pad + lo + c0;
#pragma unroll
                  for (int c = 0; c < 64; c += 8) store32(dst + c, u[c / 32], c % 32, cs);
                }
              }
            };
            // Their weights as bf16 pairs (the tensor core's operand); the sum,
            // of the weights before that rounding, stays fp32.
            auto weights = [&](const uint32_t(&u)[2][32]) {
              float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int w = 0; w < 32; ++w) {
                float a0 = -ref, a1 = -ref;
                ffma2(a0, a1, __uint_as_float(u[w / 16][2 * w % 32]),
                      __uint_as_float(u[w / 16][2 * w % 32 + 1]), cs, cs);
                const float p0 = fast_exp2(a0), p1 = fast_exp2(a1);
                ffma2(acc[2 * (w & 1)], acc[2 * (w & 1) + 1], p0, p1, 1.f, 1.f);
                if constexpr (VALUES) {
                  const __nv_bfloat162 h2 = __floats2bfloat162_rn(p0, p1);
                  pw[w] = *reinterpret_cast<const uint32_t *>(&h2);
                }
              }
              return (acc[0] + acc[1]) + (acc[2] + acc[3]);
            };
            // Half a tile's weights over columns 0 - 31 or 32 - 63, which are read.
            auto store = [&](int c0, float sum) {
              l += sum;
              if constexpr (VALUES) {
                tc_st16(tm_s + c0 / 2, *reinterpret_cast<const uint32_t(*)[16]>(pw));
                tc_st16(tm_s + c0 / 2 + 16, *reinterpret_cast<const uint32_t(*)[16]>(pw + 16));
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && !dry) mbar_arrive(&bar[(c0 ? C::P_FULL : C::P_HALF) + x]);
              }
            };
            // The maximum of columns [c0, 128), scaled.
            auto max_from = [&](int c0) {
              float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll 1
              for (; c0 < kBN; c0 += 64) {
                load(ua, c0);
                take(ua, c0, false);
#pragma unroll
                for (int c = 0; c < 64; c += 4) {
                  m0 = fmax3(m0, __uint_as_float(ua[c / 32][c % 32]), __uint_as_float(ua[c / 32][c % 32 + 1]));
                  m1 = fmax3(m1, __uint_as_float(ua[c / 32][c % 32 + 2]), __uint_as_float(ua[c / 32][c % 32 + 3]));
                }
              }
              return fmaxf(m0, m1) * cs;
            };
            // The first tile sets the references.  They stand until some row's
            // weights outgrow them (or all weights so far are zero, or a score is
            // not finite).
            const bool first = lo == lo0;
            if (first) {
              const float mx = max_from(0);
              ref = mx == -INFINITY ? 0.f : mx;
            }
            load(ua, 0);
            load(ub, 64);
            take(ua, 0, true);
            float sum = weights(ua);
            int done = 0;  // columns whose weights are stored
            bool redo = !first && (!(sum <= kMostSum) || l == 0.f);
            if (!__any_sync(0xffffffffu, redo)) {
              take(ub, 64, true);
              store(0, sum);
              done = 64;
              sum = weights(ub);
              redo = !first && (!(sum <= kMostSum) || l == 0.f);
              if (!__any_sync(0xffffffffu, redo)) {
                store(64, sum);
                done = kBN;
              }
            } else {
              wait_ld(ub[0], ub[1]);
            }
            if (done < kBN) {
              // The reference of a row that asked for it becomes the maximum of the
              // scores to come (unless they are all -inf); O and l follow.  So does
              // that of a row whose scores to come outgrow it: with another row's
              // first half rejected, nobody has looked at its second one yet.
              const float mx = max_from(done);
              float a = 1.f;
              if (mx != -INFINITY && (redo || mx - ref > kMostLead)) {
                if (l != 0.f) a = fast_exp2(ref - mx);
                l *= a;
                ref = mx;
              }
              if constexpr (VALUES) {
                // (these scores were issued after the last product on O was done;
                // that on this tile's first half is on its way)
                if (done > 0) {
                  mbar_wait(&bar[C::O_HALF + x], n & 1, dead, f.status);
                  tc_fence_after();
                }
#pragma unroll 1
                for (int o = 0; o < D; o += 16) {
                  uint32_t raw[16];
                  tc_ld16(tm_o + o, raw);
                  tc_wait_ld();
#pragma unroll
                  for (int i = 0; i < 16; ++i) raw[i] = __float_as_uint(__uint_as_float(raw[i]) * a);
                  tc_st16(tm_o + o, raw);
                }
                tc_wait_st();
              }
#pragma unroll 1
              for (; done < kBN; done += 64) {
                load(ua, done);
                take(ua, done, done > 0);
                store(done, weights(ua));
              }
            }
            if constexpr (!VALUES) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0 && !dry) mbar_arrive(&bar[(n & 1 ? C::P_FULL : C::P_HALF) + x]);
            }
          } else if (lane == 0 && !dry) {
            if constexpr (VALUES) {
              mbar_arrive(&bar[C::P_HALF + x]);
              mbar_arrive(&bar[C::P_FULL + x]);
            } else {
              mbar_arrive(&bar[(n & 1 ? C::P_FULL : C::P_HALF) + x]);
            }
          }
        }
        // ---- O / l and the log-sum-exp of the rows: finished ones where the piece is
        // the whole unit and one row tile has all of its positions, else partials
        if constexpr (VALUES) {
          if (!dry) mbar_wait(&bar[C::O_DONE + x], (n - 1) & 1, dead, f.status);
          tc_fence_after();
        }
        // Both row tiles' halves of a whole unit of up to 128 rows: the first one's threads
        // join them, the second one's O read from tensor memory (the same lanes).
        const bool joint = JOIN && !dry && !two && it.whole && it.kv_lo + kBN < it.kv_hi;
        if (joint && x == 1) {
          s_pair[r] = make_float2(ref, l);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar[C::PAIR]);
          // (s_pair is read when O is free again, and O written again only then)
          goto next;
        }
        float a0 = 1.f, a1 = 0.f;
        if (joint) {
          mbar_wait(&bar[C::PAIR], joined++ & 1, dead, f.status);
          tc_fence_after();
          const float2 other = s_pair[r];
          if (l == 0.f) {
            ref = other.x;
            l = other.y;
            a1 = 1.f;
          } else if (other.y != 0.f) {
            const float top = other.x > ref || other.x != other.x ? other.x : ref;
            a0 = ref == top ? 1.f : fast_exp2(ref - top);
            a1 = other.x == top ? 1.f : fast_exp2(other.x - top);
            l = l * a0 + other.y * a1;
            ref = top;
          }
        }
        const bool bad = !dry && s_bad[k & 15] == k + 1, none = l == 0.f;
        const long long prow = span_row(p, it.slot, x, r);
        float lse = bad ? INFINITY : none ? -INFINITY : ref + log2f(l), inv = bad || none ? 0.f : 1.f / l;
        const bool real = r < rows && !dry;
        if (it.whole && (JOIN || (!ONE && two))) {
          const int row = row0 + r, head = it.kvh * G + (row & (G - 1));
          const long long orow = (long long)(it.q_start + tl) * f.num_heads + head;
          if (f.sinks && !bad && !none && real) {
            const float sink2 = __ldg(f.sinks + head) * kLog2eF, top = lse != lse || lse > sink2 ? lse : sink2;
            const float all_lse = top + log2f(fast_exp2(lse - top) + fast_exp2(sink2 - top));
            inv *= fast_exp2(lse - all_lse);
            lse = all_lse;
          }
          if constexpr (VALUES) {
            if (warp_active) {
              __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(f.out) + orow * D;
              const float f0 = a0 * inv, f1 = a1 * inv;
              const bool later = real && s_fix[k & 15] == k + 1 && !bad && !none;  // fix_finished rounds it
#pragma unroll 1
              for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t raw[32], packed[16];
                __syncwarp();
                tc_ld32(tm_o + c0, raw);
                if (joint) {
                  uint32_t more[32];
                  tc_ld32(tm_o + 128 + c0, more);
                  wait_ld(raw, more);
#pragma unroll
                  for (int i = 0; i < 32; ++i)
                    raw[i] = __float_as_uint(fmaf(__uint_as_float(raw[i]), f0, __uint_as_float(more[i]) * f1));
                } else {
                  tc_wait_ld();
#pragma unroll
                  for (int i = 0; i < 32; ++i) raw[i] = __float_as_uint(__uint_as_float(raw[i]) * f0);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  // one rounding to nearest even, of the finished output
                  const __nv_bfloat162 h2 =
                      __floats2bfloat162_rn(__uint_as_float(raw[2 * i]), __uint_as_float(raw[2 * i + 1]));
                  packed[i] = bad || none ? 0u : *reinterpret_cast<const uint32_t *>(&h2);
                }
                if (later) {
#pragma unroll
                  for (int i = 0; i < 32; i += 8) store32(p.part_o + prow * D + c0 + i, raw, i, 1.f);
                } else if (real) {
#pragma unroll
                  for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<uint4 *>(dst + c0 + 2 * i) =
                        make_uint4(packed[i], packed[i + 1], packed[i + 2], packed[i + 3]);
                }
              }
              if (later) fix_finished<D, CAUSAL>(p, it, row, ref, inv, p.part_o + prow * D, dst);
            }
          }
          if (VOTES && real) p.row_lse[orow] = lse;
        } else {
          if constexpr (VALUES) {
            if (warp_active) {
#pragma unroll 1
              for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t raw[32];
                tc_ld32(tm_o + c0, raw);
                tc_wait_ld();
                if (real) {
#pragma unroll
                  for (int i = 0; i < 32; i += 8) store32(p.part_o + prow * D + c0 + i, raw, i, inv);
                }
              }
              if (real && s_fix[k & 15] == k + 1 && !bad && !none)
                fix_partial<D, CAUSAL>(p, it, row0 + r, !two, x, ref, inv, p.part_o + prow * D);
            }
          }
          if (real) p.part_lse[prow] = lse;
        }
        if (dry || VALUES) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bar[C::O_FREE + x]);
            if (joint) mbar_arrive(&bar[C::O_FREE + 1]);
          }
        }
      }
    next:
      if (dry) pdl_wait();  // the plan
      if (!next_piece()) break;
      ++k;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssueWarp) tc_dealloc(tmem, kTmemCols);
}

template <int D, int MODE, bool ONE, bool JOIN = false>
cudaError_t launch_d(const SpanParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
                     const CUtensorMap &tv, int box, cudaStream_t stream) {
  using C = Cfg<D, ONE>;
  auto kern = span_mma_kernel<D, MODE, ONE, JOIN>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = set_smem_attrs_once(kern, C::SMEM, done);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(p.grid), dim3(kThreads), C::SMEM, stream, tq, tk, tv, p, box);
}

template <int MODE>
cudaError_t launch_mode(const SpanParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
                        const CUtensorMap &tv, int box, cudaStream_t stream) {
  const bool one = p.one;
  if constexpr (MODE == kSpanTree) {
    if (p.join && p.f.head_dim == 128)
      return one ? launch_d<128, MODE, true, true>(p, tq, tk, tv, box, stream)
                 : launch_d<128, MODE, false, true>(p, tq, tk, tv, box, stream);
    if (p.join)
      return one ? launch_d<64, MODE, true, true>(p, tq, tk, tv, box, stream)
                 : launch_d<64, MODE, false, true>(p, tq, tk, tv, box, stream);
  }
  if (p.f.head_dim == 128)
    return one ? launch_d<128, MODE, true>(p, tq, tk, tv, box, stream)
               : launch_d<128, MODE, false>(p, tq, tk, tv, box, stream);
  return one ? launch_d<64, MODE, true>(p, tq, tk, tv, box, stream)
             : launch_d<64, MODE, false>(p, tq, tk, tv, box, stream);
}

}  // namespace

cudaError_t launch_span_mma(const SpanParams &p, int mode, cudaStream_t stream) {
  const FwdParams &f = p.f;
  const unsigned long long es = 2, D = f.head_dim, row = D * es, H = f.num_heads,
                           Hk = f.num_kv_heads, bs = f.block_size, NB = f.num_blocks;
  const unsigned long long G = H / Hk;
  // positions per copy box: a run that never crosses a page (tiles start at
  // multiples of 128)
  const int box = bs % 128 == 0 ? 128 : bs % 64 == 0 ? 64 : 16;
  const unsigned long long slot = p.hnd ? row : Hk * row, head = p.hnd ? bs * row : row;
  CUtensorMap tq, tk, tv;
  {
    const unsigned long long d[3] = {D, H, (unsigned long long)f.num_tokens}, s[2] = {row, H * row};
    const unsigned int b[3] = {64, (unsigned)G, (unsigned)(128 / G)};
    if (!encode_tiled(&tq, f.q, PA_BF16, 3, d, s, b, true)) return cudaErrorInvalidValue;
  }
  {
    const unsigned long long d[4] = {D, Hk, bs, NB}, s[3] = {head, slot, bs * Hk * row};
    const unsigned int b[4] = {64, 1, (unsigned)box, 1};
    if (!encode_tiled(&tk, p.k_cache, PA_BF16, 4, d, s, b, true)) return cudaErrorInvalidValue;
  }
  if (mode == kSpanVotesOnly) {
    tv = tk;  // not read
  } else {
    const unsigned long long d[5] = {64, bs, D / 64, Hk, NB}, s[4] = {slot, 128, head, bs * Hk * row};
    const unsigned int b[5] = {64, (unsigned)box, (unsigned)(D / 64), 1, 1};
    if (!encode_tiled(&tv, p.v_cache, PA_BF16, 5, d, s, b, true)) return cudaErrorInvalidValue;
  }
  return mode == kSpanTree    ? launch_mode<kSpanTree>(p, tq, tk, tv, box, stream)
         : mode == kSpanVotes ? launch_mode<kSpanVotes>(p, tq, tk, tv, box, stream)
                              : launch_mode<kSpanVotesOnly>(p, tq, tk, tv, box, stream);
}

}  // namespace pa
