// pa_prefix_mma.cu -- the prefix part of pa_forward_shared_prefix on the
// tensor cores (bf16).
//
// Mathematics: for an item's 256 rows (128 / G tokens x the G heads of one KV
// head, twice) and the positions [kv_lo, kv_hi) of its split,
//   S = Q K^T,  P = 2^(scale log2e S - ref),  l = sum P,  O = sum P V,
// tile by tile of 128 positions, one pass over K and V, with a reference ref for
// each row that moves (O and l rescaled) only when weights outgrow it.  Every
// position is visible to every row: no causal mask; only the last tile of a
// prefix may be short, its missing positions masked by select.
//
// One CTA per SM (224 KB of shared memory, all 512 TMEM columns), 16 warps:
//   warps 0-3, 4-7  softmax of the two 128-row tiles, thread = row (TMEM lane):
//                   P stored as bf16 over the tile's own S.  The sum of half a
//                   tile's weights tells whether the reference still holds: the
//                   maximum of the scores and its latency leave the loop
//   warps 8, 9      each issues one row tile's S = Q K^T (M = 128, N = 128) and
//                   O += P V (P from TMEM, N = head_dim), taking turns
//   warps 10-13     TMA: K boxes (10, 11) and V boxes (12, 13) into rings that
//                   both row tiles read
// What it takes: 1.4 to 1.45 us of an SM for 256 rows x 128 positions at head_dim
// 128 (92 % of the measured bf16 peak while it runs; products 1.32), 1.28 at 64
// (52 %: there the softmax, some 1400 clocks of two warps a scheduler, and the
// chain S, softmax, P V of each row tile bound it).  128 rows or fewer take 1.33
// with K and V in L2 and 1.53 from HBM, which is 6.5 TB/s over the SMs.  An item
// adds about 4 us: its first tile, and 2 us of storing 256 rows of partials.
// The turns keep the row tiles half a period apart: while one's softmax runs,
// the other's products do.  (Without them both row tiles' products went side by
// side, and so did their softmaxes while the tensor pipe idled.)  K and V are
// loaded once for 256 rows, so the loads stay below what HBM or L2 give as
// long as the products bound the tile; with few rows HBM does.
// A box that lies past the split, or on a bad page, is loaded from a page
// beyond the pool, which TMA fills with zeros: no NaN reaches a product, and
// every tile has the same byte count.
#include "pa_prefix.h"
#include "pa_umma.cuh"

namespace pa {
namespace {

constexpr int kBN = kPrefixTile;
// Half a tile's weights may sum to this much before the reference moves up to its
// maximum: far from overflow in bf16 and in the fp32 sums, so a row's reference
// is mostly its first tile's maximum, and no maximum is taken of the others.
constexpr float kMostSum = 1048576.f;
constexpr float kMostLead = 14.f;  // 64 weights of 2^14 sum to that much
constexpr int kThreads = 512;
constexpr int kIssueWarp = 8, kLoad0 = 10, kLoadEnd = 14;  // 14, 15 idle
// launch registers 512 x 128; the softmax warpgroups take 176, the others keep 80
constexpr int kSoftmaxRegs = 176, kOtherRegs = 80;
constexpr uint32_t kTmemCols = 512, kTmemO = 256;  // S of row tile x at 128 x, O at 256 + 128 x

template <int D>
struct Cfg {
  static constexpr int NH = D / 64;            // 128-byte chunks of a row
  static constexpr int Q_TILE = NH * 128 * 128;
  static constexpr int KV_BYTES = NH * kBN * 128;
  static constexpr int KST = D == 128 ? 3 : 5, VST = D == 128 ? 2 : 5;
  static constexpr int OFF_K = 2 * Q_TILE;
  static constexpr int OFF_V = OFF_K + KST * KV_BYTES;
  static constexpr int OFF_BAR = OFF_V + VST * KV_BYTES;
  // barriers
  static constexpr int Q_FULL = 0, Q_FREE = 1, S_FULL = 2, O_HALF = 4, O_DONE = 6, P_HALF = 8,
                       P_FULL = 10, O_FREE = 12, TURN = 14, END = 16, K_FULL = 17, V_FULL = K_FULL + KST, K_FREE = V_FULL + VST,
                       V_FREE = K_FREE + KST, NBAR = V_FREE + VST;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 32;
  static constexpr uint32_t IDESC_S = umma_idesc_bf16(128, kBN, 0);
  static constexpr uint32_t IDESC_PV = umma_idesc_bf16(128, D, 1);
  static_assert(SMEM <= 232448, "shared memory of one CTA");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_mma_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const PrefixParams p, int box) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
  int *s_bad = reinterpret_cast<int *>(smem + C::OFF_MISC + 8);  // [2]
  const FwdParams &f = p.f;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = f.num_heads / f.num_kv_heads, TQ = 128 / G, bs = f.block_size;
  if (smem_u32(smem) & 1023) {  // the same for every thread: all leave together
    if (tid == 0) atomicOr(f.status, PA_DEV_INTERNAL);
    pdl_wait();  // (the own part's kernels count on the plan being done)
    return;
  }
  if (tid == 0) {
    prefetch_tensor_map(&tm_q);
    prefetch_tensor_map(&tm_k);
    prefetch_tensor_map(&tm_v);
    for (int b = 0; b < C::NBAR; ++b) {
      // P and O: the row tile's four warps; a ring stage: two loading warps,
      // two issuing ones
      const bool softmax = b >= C::P_HALF && b < C::TURN, ring = b >= C::K_FULL;
      mbar_init(&bar[b], softmax ? 4 : ring || b == C::Q_FREE || b == C::END ? 2 : 1);
    }
    fence_mbar_init();
  }
  if (warp == kIssueWarp) tc_alloc(s_tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  bool dead = false;

  if (warp >= kIssueWarp) {
    reg_dec<kOtherRegs>();
    pdl_wait();     // the plan
    pdl_trigger();  // the own part's kernels count on it being done
    const int n_items = p.plan->n_items;
    const PrefixGroup g0 = p.grp[0];
    if (warp >= kLoad0 && warp < kLoadEnd) {
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
      for (int item = blockIdx.x; item < n_items && !dead; item += gridDim.x, ++items) {
        const PrefixItem it = prefix_item(p, g0, item, G);
        const int32_t *bt = f.block_table + (size_t)it.req0 * f.max_blocks_per_seq;
        auto page_of = [&](int pos) {
          int page = f.num_blocks;  // past the pool: zeros
          if (lane < nb && pos < it.kv_hi) {
            const int x = __ldg(bt + pos / bs);
            if (x >= 0 && x < f.num_blocks) page = x;
          }
          return page;
        };
        if (warp == kLoad0 && lane == 0) {
          const int tiles = (it.q_len - it.t0) * G > 128 ? 2 : 1;
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
        int page = page_of(pos);
        for (int lo = it.kv_lo; lo < it.kv_hi; lo += kBN) {
          const int next = page_of(pos + kBN);  // its latency passes during the wait
          if (lane == 0) {
            if (round > 0) mbar_wait(&free[st], (round - 1) & 1, dead, f.status);
            if (!dead) mbar_arrive_expect_tx(&full[st], bytes);
          }
          dead = __any_sync(0xffffffffu, dead);
          if (dead) break;  // timed out: the stage is not free
          if (lane < nb) {
            uint8_t *dst = ring + st * C::KV_BYTES;
            if (is_v) tma_load_5d(dst, &tm_v, 0, pos % bs, 0, it.kvh, page, &full[st]);
            else tma_load_4d(dst, &tm_k, chunk * 64, it.kvh, pos % bs, page, &full[st]);
          }
          __syncwarp();
          page = next;
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
    } else if (warp < kLoad0) {
      // ------------------------------------------------------------- products
      // The warp of row tile x: the value product of its weights, and behind it
      // the scores of the next tile of positions.  The two warps take turns,
      // two products a turn, so that each softmax has the other row tile's
      // products to run beside; a turn ends when its products are issued, so the
      // other's next ones queue up behind them.  Both warps take every stage of
      // the rings and free it, by a commit or, without rows, by an arrival.
      const int x = warp - kIssueWarp;
      const uint32_t sq = smem_u32(smem) + x * C::Q_TILE, sk = smem_u32(smem) + C::OFF_K,
                     sv = smem_u32(smem) + C::OFF_V;
      const uint32_t tm_s = tmem + x * 128, tm_o = tmem + kTmemO + x * 128;
      uint32_t ks = 0, kr = 0, vs = 0, vr = 0;  // ring stage and round
      uint32_t items = 0, n = 0, mine = 0;      // items, value products, items with rows here
      uint32_t turn = 0;
      auto take_turn = [&]() {
        if (x == 1 || turn > 0) mbar_wait(&bar[C::TURN + x], (turn - 1 + x) & 1, dead, f.status);
        ++turn;
      };
      auto pass_turn = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[C::TURN + (x ^ 1)]);
      };
      auto scores = [&]() {
        const uint32_t a = desc_lo(sq, 16), b = desc_lo(sk + ks * C::KV_BYTES, 16);
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {  // 16 columns: 32 bytes, 4 to a chunk
          const uint32_t off = (kk / 4) * (128 * 128 / 16) + (kk % 4) * 2;
          mma_ss(tm_s, a + off, b + off, C::IDESC_S, kk > 0);
        }
      };
      auto scores_done = [&](bool last) {  // last: of the item, which is then done with Q
        commit(&bar[C::S_FULL + x]);
        commit(&bar[C::K_FREE + ks]);
        if (last) commit(&bar[C::Q_FREE]);
        if (++ks == C::KST) ks = 0, ++kr;
      };
      for (int item = blockIdx.x; item < n_items; item += gridDim.x, ++items) {
        const PrefixItem it = prefix_item(p, g0, item, G);
        const int rows = (it.q_len - it.t0) * G;
        const bool two = rows > 128;
        mbar_wait(&bar[C::Q_FULL], items & 1, dead, f.status);
        if (x == 1 && !two) {
          for (int lo = it.kv_lo; lo < it.kv_hi; lo += kBN) {
            mbar_wait(&bar[C::K_FULL + ks], kr & 1, dead, f.status);
            mbar_wait(&bar[C::V_FULL + vs], vr & 1, dead, f.status);
            if (lane == 0) {
              mbar_arrive(&bar[C::K_FREE + ks]);
              mbar_arrive(&bar[C::V_FREE + vs]);
            }
            if (++ks == C::KST) ks = 0, ++kr;
            if (++vs == C::VST) vs = 0, ++vr;
          }
          if (lane == 0) mbar_arrive(&bar[C::Q_FREE]);
          continue;
        }
        mbar_wait(&bar[C::K_FULL + ks], kr & 1, dead, f.status);
        // (the weights of the item before have been read: O_DONE was awaited;
        // and the dry round is over)
        if (mine == 0) mbar_wait(&bar[C::O_FREE + x], 0, dead, f.status);
        if (two) take_turn();
        scores();
        if (two) pass_turn();
        scores_done(it.kv_lo + kBN >= it.kv_hi);
        for (int lo = it.kv_lo; lo < it.kv_hi; lo += kBN, ++n) {
          const bool more = lo + kBN < it.kv_hi;
          mbar_wait(&bar[C::V_FULL + vs], vr & 1, dead, f.status);
          if (more) mbar_wait(&bar[C::K_FULL + ks], kr & 1, dead, f.status);
          // O of the item before has been stored (phase 0 is the dry round's)
          if (lo == it.kv_lo) mbar_wait(&bar[C::O_FREE + x], mine & 1, dead, f.status);
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
            mma_ts(tm_o, tm_s + kk * 8, b + off, C::IDESC_PV, lo > it.kv_lo || kk > 0);
          }
          commit(&bar[C::O_DONE + x]);
          commit(&bar[C::V_FREE + vs]);
          if (++vs == C::VST) vs = 0, ++vr;
          // the scores go over the weights that the product reads
          mbar_wait(&bar[C::O_DONE + x], n & 1, dead, f.status);
          if (more) scores();
          if (two) pass_turn();
          if (more) scores_done(lo + 2 * kBN >= it.kv_hi);
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
    const uint32_t tm_s = tmem + lane_off + x * 128, tm_o = tmem + lane_off + kTmemO + x * 128;
    const float c2 = f.scale_log2;
    // 2^(c s - ref) as one multiply-add needs c > 0 (the maximum is then c max s)
    const bool fold = c2 > 0.f;
    const float cs = fold ? c2 : 1.f;
    uint32_t n = 0;
    // The first round is dry: a tile of whatever TMEM holds, no barrier touched
    // and nothing stored, run before the plan is awaited.  It brings this
    // code into the instruction cache, which costs the first tile 3 to 6 us
    // when a call's own keys have just swept L2.
    int n_items = 0;
    PrefixGroup g0{};
    for (int item = -1; item < n_items; item = item < 0 ? (int)blockIdx.x : item + (int)gridDim.x) {
      const bool dry = item < 0;
      PrefixItem it;
      if (dry) it.q_start = it.q_len = it.req0 = it.kvh = it.t0 = it.kv_lo = 0, it.kv_hi = kBN;
      else it = prefix_item(p, g0, item, G);
      const int rows = dry ? 128 : min(128, (it.q_len - it.t0) * G - x * 128);
      if (rows <= 0) continue;
      // a bad page in the split marks all of the item's rows
      if (!dry) {
        const int32_t *bt = f.block_table + (size_t)it.req0 * f.max_blocks_per_seq;
        int bad = 0;
        for (int lp = it.kv_lo / bs + r; lp <= (it.kv_hi - 1) / bs; lp += 128) {
          const int page = __ldg(bt + lp);
          if (page < 0 || page >= f.num_blocks) bad = 1;
        }
        if (bad) atomicOr(f.status, PA_DEV_BAD_BLOCK);
        if (r == 0) s_bad[x] = 0;
        named_sync(1 + x, 128);
        if (bad) atomicOr(&s_bad[x], 1);
        named_sync(1 + x, 128);
      }
      const bool item_bad = !dry && s_bad[x] != 0;
      const bool warp_active = (warp & 3) * 32 < rows;  // its other rows are padding
      float ref = 0.f, l = 0.f;  // the weights' reference exponent and their sum
      for (int lo = it.kv_lo; lo < it.kv_hi; lo += kBN, n += !dry) {
        if (!dry) mbar_wait(&bar[C::S_FULL + x], n & 1, dead, f.status);
        tc_fence_after();
        if (warp_active) {
          uint32_t ua[2][32], ub[2][32], pw[32];
          // The 64 scores of columns c0 on, to be completed by take(): awaited,
          // scaled where the scale does not fold, masked past the split.
          auto load = [&](uint32_t(&u)[2][32], int c0) {
            tc_ld32(tm_s + c0, u[0]);
            tc_ld32(tm_s + c0 + 32, u[1]);
          };
          auto take = [&](uint32_t(&u)[2][32], int c0) {
            wait_ld(u[0], u[1]);
            if (!fold) {
#pragma unroll
              for (int c = 0; c < 64; ++c)
                u[c / 32][c % 32] = __float_as_uint(__uint_as_float(u[c / 32][c % 32]) * c2);
            }
            if (lo + c0 + 64 > it.kv_hi) {
#pragma unroll
              for (int c = 0; c < 64; ++c)
                if (lo + c0 + c >= it.kv_hi) u[c / 32][c % 32] = 0xff800000u;  // -inf
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
              const __nv_bfloat162 h2 = __floats2bfloat162_rn(p0, p1);
              pw[w] = *reinterpret_cast<const uint32_t *>(&h2);
            }
            return (acc[0] + acc[1]) + (acc[2] + acc[3]);
          };
          // Half a tile's weights over columns 0 - 31 or 32 - 63, which are read.
          auto store = [&](int c0, float sum) {
            tc_st16(tm_s + c0 / 2, *reinterpret_cast<const uint32_t(*)[16]>(pw));
            tc_st16(tm_s + c0 / 2 + 16, *reinterpret_cast<const uint32_t(*)[16]>(pw + 16));
            l += sum;
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && !dry) mbar_arrive(&bar[(c0 ? C::P_FULL : C::P_HALF) + x]);
          };
          // The maximum of columns [c0, 128), scaled.
          auto max_from = [&](int c0) {
            float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll 1
            for (; c0 < kBN; c0 += 64) {
              load(ua, c0);
              take(ua, c0);
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
          const bool first = lo == it.kv_lo;
          if (first) {
            const float mx = max_from(0);
            ref = mx == -INFINITY ? 0.f : mx;
          }
          load(ua, 0);
          load(ub, 64);
          take(ua, 0);
          float sum = weights(ua);
          int done = 0;  // columns whose weights are stored
          bool redo = !first && (!(sum <= kMostSum) || l == 0.f);
          if (!__any_sync(0xffffffffu, redo)) {
            take(ub, 64);
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
#pragma unroll 1
            for (; done < kBN; done += 64) {
              load(ua, done);
              take(ua, done);
              store(done, weights(ua));
            }
          }
        } else if (lane == 0) {
          mbar_arrive(&bar[C::P_HALF + x]);
          mbar_arrive(&bar[C::P_FULL + x]);
        }
      }
      // ---- O / l and the log-sum-exp of the rows
      if (!dry) mbar_wait(&bar[C::O_DONE + x], (n - 1) & 1, dead, f.status);
      tc_fence_after();
      if (warp_active) {
        const float inv = l > 0.f && !item_bad ? 1.f / l : 0.f;
        const uint32_t keep = item_bad ? 0u : 0xffffffffu;
        const long long prow = (long long)item * kPrefixRows + x * 128 + r;
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t raw[32];
          tc_ld32(tm_o + c0, raw);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) raw[i] &= keep;
          if (r < rows && !dry) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) store32(p.part_o + prow * D + c0 + i, raw, i, inv);
          }
        }
        if (r < rows && !dry)
          p.part_lse[prow] = item_bad ? __int_as_float(0x7fc00000) : l > 0.f ? ref + log2f(l) : -INFINITY;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[C::O_FREE + x]);
      if (dry) {
        pdl_wait();  // the plan
        n_items = p.plan->n_items;
        g0 = p.grp[0];
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssueWarp) tc_dealloc(tmem, kTmemCols);
}

template <int D>
cudaError_t launch_d(const PrefixParams &p, const CUtensorMap &tq, const CUtensorMap &tk,
                     const CUtensorMap &tv, int box, int num_sms, cudaStream_t stream) {
  using C = Cfg<D>;
  auto kern = prefix_mma_kernel<D>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = set_smem_attrs_once(kern, C::SMEM, done);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(num_sms), dim3(kThreads), C::SMEM, stream, tq, tk, tv, p, box);
}

}  // namespace

cudaError_t launch_prefix_mma(const PrefixParams &p, int kv_layout, int num_sms,
                              cudaStream_t stream) {
  const FwdParams &f = p.f;
  const unsigned long long es = 2, D = f.head_dim, row = D * es, H = f.num_heads,
                           Hk = f.num_kv_heads, bs = f.block_size, NB = f.num_blocks;
  const unsigned long long G = H / Hk;
  // positions per copy box: a run that never crosses a page (tiles start at
  // multiples of 128)
  const int box = bs % 128 == 0 ? 128 : bs % 64 == 0 ? 64 : 16;
  const bool hnd = kv_layout == PA_KV_HND;
  const unsigned long long slot = hnd ? row : Hk * row, head = hnd ? bs * row : row;
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
  {
    const unsigned long long d[5] = {64, bs, D / 64, Hk, NB}, s[4] = {slot, 128, head, bs * Hk * row};
    const unsigned int b[5] = {64, (unsigned)box, (unsigned)(D / 64), 1, 1};
    if (!encode_tiled(&tv, p.v_cache, PA_BF16, 5, d, s, b, true)) return cudaErrorInvalidValue;
  }
  return D == 128 ? launch_d<128>(p, tq, tk, tv, box, num_sms, stream)
                  : launch_d<64>(p, tq, tk, tv, box, num_sms, stream);
}

}  // namespace pa
