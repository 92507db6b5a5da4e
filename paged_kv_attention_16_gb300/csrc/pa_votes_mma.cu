// pa_votes_mma.cu -- the sums over rows of pa_forward_weights on the tensor cores
// (bf16), for requests whose scores were not kept.
//
// Mathematics: for 128 positions j of a KV head and the request's rows r,
//   S^T = K Q^T,  W_j = sum_r 2^(scale log2e S_rj - L_r),
// L_r being the row's log-sum-exp from the pass before.  The scores are multiplied
// out again instead of being kept: a position of 256 rows would be 1 KB written
// and read, its key is 128 or 256 bytes.  Transposed, a position is a TMEM lane and
// its thread sums over the columns in registers: no reduction across threads, no
// atomics.
//
// Two CTAs per SM, each with two groups of 4 warps for the sums (thread = position),
// one issuing warp and one TMA warp.  A CTA walks a run of the (request, KV head, tile
// of 128 positions) list; a tile's keys stay while the rows pass in blocks of QR, whose
// scores go to two TMEM buffers in turn, a group of warps to each.  The groups' sums
// meet in shared memory.
//
// No unit is full; what a tile waits for is the chain between the roles (keys and rows,
// scores, sums): 16 requests of 64 tokens, 4 heads a KV head of 64, 16384 positions: 38
// to 40 us (268 million exponentials, the exponential unit at 38 %, 56 % of the issue
// slots, the tensor cores at 23 %, 71 MB from DRAM).  One group a CTA: 42 us, its scores fetched 32
// columns ahead; with two groups that prefetch costs registers and time (40).
#include "pa_span.h"
#include "pa_umma.cuh"

namespace pa {
namespace {

constexpr int kBN = kSpanTile;
constexpr int kThreads = 320;
constexpr int kIssueWarp = 8, kLoadWarp = 9;
constexpr int kLseRows = 512;  // rows whose log-sum-exps stay while a KV head's tiles pass

template <int D>
struct Cfg {
  static constexpr int NH = D / 64;
  static constexpr int QR = D == 128 ? 64 : 128;  // rows of a block
  static constexpr int K_BYTES = NH * kBN * 128, Q_BYTES = NH * QR * 128;
  static constexpr int KST = 2, QST = D == 128 ? 2 : 3, CTAS = 2;  // CTAs an SM
  static constexpr int OFF_Q = KST * K_BYTES;
  static constexpr int OFF_BAR = OFF_Q + QST * Q_BYTES;
  static constexpr int K_FULL = 0, K_FREE = K_FULL + KST, Q_FULL = K_FREE + KST, Q_FREE = Q_FULL + QST,
                       S_FULL = Q_FREE + QST, S_FREE = S_FULL + 2, END = S_FREE + 2, NBAR = END + 1;
  static constexpr int OFF_LSE = OFF_BAR + ((NBAR * 8 + 15) & ~15);
  static constexpr int OFF_SUM = OFF_LSE + kLseRows * 4;
  static constexpr int OFF_MISC = OFF_SUM + 2 * kBN * 4;
  static constexpr int SMEM = OFF_MISC + 16;
  static constexpr uint32_t COLS = 2 * QR;  // two buffers
  static constexpr uint32_t IDESC = umma_idesc_bf16(128, QR, 0);
};

struct VoteItem {
  SpanReq r;
  int s, kvh, at;     // at: the tile's first position
  int b0, nb;         // row blocks: those before b0 see none of the positions
};

// The items of this block, in order; every role walks them for itself.
struct VoteCursor {
  unsigned left;
  int s, kvh, tile;
  SpanReq r;
  bool skip;

  __device__ void take(const SpanParams &p) {
    r = p.req[s];
    skip = r.nblk > 0 && __ldcg(p.row_lse + (size_t)(r.q_start + r.q_len - 1) * p.f.num_heads) == INFINITY;
  }
  __device__ void start(const SpanParams &p) {
    const unsigned total = p.plan->vote_tiles;
    const unsigned pos = (unsigned)((unsigned long long)total * blockIdx.x / gridDim.x);
    left = (unsigned)((unsigned long long)total * (blockIdx.x + 1) / gridDim.x) - pos;
    s = kvh = tile = 0;
    if (left == 0) return;
    int lo = 0, hi = p.f.num_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (p.vote_end[mid] > pos) hi = mid; else lo = mid + 1;
    }
    s = lo;
    take(p);
    const int local = (int)(pos - (p.vote_end[s] - (unsigned)(p.f.num_kv_heads * r.ntile)));
    kvh = local / r.ntile;
    tile = local - kvh * r.ntile;
  }
  // lg: log2 of the heads of a KV head
  __device__ bool next(const SpanParams &p, int lg, int QR, VoteItem &it) {
    while (left > 0) {
      if (tile == r.ntile) {
        tile = 0;
        if (++kvh == p.f.num_kv_heads) {
          const unsigned last = p.vote_end[s];
          while (p.vote_end[++s] == last) {}  // (left > 0: there is one)
          take(p);
          kvh = 0;
        }
      }
      it.r = r;
      it.s = s;
      it.kvh = kvh;
      it.at = tile * kBN;
      it.nb = ((r.q_len << lg) + QR - 1) / QR;
      it.b0 = (max(0, it.at - (r.ctx - r.q_len)) << lg) / QR;
      --left;
      ++tile;
      if (!skip) return true;  // (a request with a bad page is left as it was)
    }
    return false;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, Cfg<D>::CTAS)
    votes_mma_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ SpanParams p, int box) {
  using C = Cfg<D>;
  constexpr int QR = C::QR;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
  float *s_lse = reinterpret_cast<float *>(smem + C::OFF_LSE);  // [kLseRows] or [2 groups][2][QR]
  float *s_sum = reinterpret_cast<float *>(smem + C::OFF_SUM);  // [2][kBN]
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
  const FwdParams &f = p.f;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = f.num_heads, G = H / f.num_kv_heads, bs = f.block_size, lg = __ffs(G) - 1;
  if (smem_u32(smem) & 1023) {  // the same for every thread: all leave together
    if (tid == 0) atomicOr(f.status, PA_DEV_INTERNAL);
    return;
  }
  if (tid == 0) {
    prefetch_tensor_map(&tm_q);
    prefetch_tensor_map(&tm_k);
  }
  if (tid < C::NBAR) {
    mbar_init(&bar[tid], tid >= C::S_FREE && tid < C::END ? 4 : 1);
    fence_mbar_init();
  }
  if (warp == kIssueWarp) tc_alloc(s_tmem, C::COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  bool dead = false;
  pdl_trigger();
  pdl_wait();
  VoteCursor cur;
  VoteItem it;
  cur.start(p);
  if (warp == kLoadWarp) {
    const int runs = kBN / box, run = lane % runs, chunk = lane / runs;
    const bool mine = lane < runs * C::NH;
    uint32_t ks = 0, kr = 0, qs = 0, qr = 0;
    while (!dead && cur.next(p, lg, QR, it)) {
      const int32_t *bt = f.block_table + (size_t)it.s * f.max_blocks_per_seq;
      const int pos = it.at + run * box;
      int page = mine && pos < it.r.ctx ? bt[pos / bs] : f.num_blocks;  // past the pool: zeros
      if (page < 0 || page > f.num_blocks) page = f.num_blocks;
      if (lane == 0) {
        if (kr > 0) mbar_wait(&bar[C::K_FREE + ks], (kr - 1) & 1, dead, f.status);
        if (!dead) mbar_arrive_expect_tx(&bar[C::K_FULL + ks], C::K_BYTES);
      }
      dead = __any_sync(0xffffffffu, dead);
      if (dead) break;
      if (mine)
        tma_load_4d(smem + ks * C::K_BYTES + chunk * kBN * 128 + run * box * 128, &tm_k, chunk * 64, it.kvh,
                    pos % bs, page, &bar[C::K_FULL + ks]);
      __syncwarp();
      if (++ks == C::KST) ks = 0, ++kr;
      if (lane == 0) {
        for (int b = it.b0; b < it.nb && !dead; ++b) {
          if (qr > 0) mbar_wait(&bar[C::Q_FREE + qs], (qr - 1) & 1, dead, f.status);
          if (dead) break;
          mbar_arrive_expect_tx(&bar[C::Q_FULL + qs], C::Q_BYTES);
          for (int h = 0; h < C::NH; ++h)
            tma_load_3d(smem + C::OFF_Q + qs * C::Q_BYTES + h * QR * 128, &tm_q, h * 64, it.kvh * G,
                        it.r.q_start + b * (QR / G), &bar[C::Q_FULL + qs]);
          if (++qs == C::QST) qs = 0, ++qr;
        }
      }
      dead = __any_sync(0xffffffffu, dead);
    }
    // No copy may land after the CTA is gone, not even if its readers timed out.
    if (lane == 0) {
      bool late = false;
      for (uint32_t s = 0; s < (uint32_t)C::KST; ++s) {
        const uint32_t fills = kr + (s < ks);
        if (fills > 0) mbar_wait(&bar[C::K_FULL + s], (fills - 1) & 1, late, f.status);
      }
      for (uint32_t s = 0; s < (uint32_t)C::QST; ++s) {
        const uint32_t fills = qr + (s < qs);
        if (fills > 0) mbar_wait(&bar[C::Q_FULL + s], (fills - 1) & 1, late, f.status);
      }
    }
    __syncwarp();
  } else if (warp == kIssueWarp) {
    const uint32_t sk = smem_u32(smem), sq = smem_u32(smem) + C::OFF_Q;
    uint32_t ks = 0, kr = 0, qs = 0, qr = 0, n = 0;
    while (cur.next(p, lg, QR, it)) {
      mbar_wait(&bar[C::K_FULL + ks], kr & 1, dead, f.status);
      for (int b = it.b0; b < it.nb; ++b, ++n) {
        mbar_wait(&bar[C::Q_FULL + qs], qr & 1, dead, f.status);
        if (n >= 2) mbar_wait(&bar[C::S_FREE + (n & 1)], ((n >> 1) - 1) & 1, dead, f.status);
        tc_fence_after();
        const uint32_t a = desc_lo(sk + ks * C::K_BYTES, 16), q = desc_lo(sq + qs * C::Q_BYTES, 16);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + (n & 1) * QR, a + (kk / 4) * (kBN * 128 / 16) + (kk % 4) * 2,
                 q + (kk / 4) * (QR * 128 / 16) + (kk % 4) * 2, C::IDESC, kk > 0);
        commit(&bar[C::S_FULL + (n & 1)]);
        commit(&bar[C::Q_FREE + qs]);
        if (++qs == C::QST) qs = 0, ++qr;
      }
      commit(&bar[C::K_FREE + ks]);
      if (++ks == C::KST) ks = 0, ++kr;
    }
    bool late = false;
    commit(&bar[C::END]);
    mbar_wait(&bar[C::END], 0, late, f.status);
    __syncwarp();
  } else {
    // Two groups of four warps, the one for buffer 0 and the one for buffer 1.
    const int grp = warp >> 2, th = tid & 127;
    const uint32_t tm = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float c2 = f.scale_log2;
    // rows behind the last one, and rows without weight, add nothing
    auto lse_of = [&](const VoteItem &v, int row) {
      if (row >= v.r.q_len << lg) return -INFINITY;
      const float l = __ldcg(p.row_lse + (size_t)(v.r.q_start + (row >> lg)) * H + v.kvh * G + (row & (G - 1)));
      return l == -INFINITY ? l : -l;
    };
    uint32_t n = 0, own = 0;
    int at_s = -1, at_kvh = -1;  // whose log-sum-exps are in shared memory, all of them
    for (uint32_t item = 0; cur.next(p, lg, QR, it); ++item) {
      const int pos = it.at + th, R = it.r.q_len << lg, prefix = it.r.ctx - it.r.q_len;
      const int first = max(0, pos - prefix) << lg;  // the first row that sees this position
      const bool few = it.nb * QR <= kLseRows;
      const int mine = it.b0 + ((n ^ grp) & 1);  // the group's first block
      float next = 0.f;
      if (!few) {
        if (mine < it.nb && th < QR) next = lse_of(it, mine * QR + th);
        if (at_s >= 0) named_sync(1, 256);  // those before are read
        at_s = -1;
      } else if (it.s != at_s || it.kvh != at_kvh) {
        named_sync(1, 256);
        for (int row = tid; row < it.nb * QR; row += 256) s_lse[row] = lse_of(it, row);
        named_sync(1, 256);
        at_s = it.s;
        at_kvh = it.kvh;
      }
      const bool store = (item & 1) == grp;  // the groups take turns
      const int page = store && pos < it.r.ctx ? f.block_table[(size_t)it.s * f.max_blocks_per_seq + pos / bs] : -1;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      const uint32_t behind = n + (it.nb - it.b0);
      n += mine - it.b0;
      for (int b = mine; b < it.nb; b += 2, n += 2) {
        const float *lse = s_lse + b * QR;
        if (!few) {  // (those of two blocks of the group ago were read before the barrier of the last)
          float *at = s_lse + (grp * 2 + (own++ & 1)) * QR;
          if (th < QR) at[th] = next;
          if (b + 2 < it.nb && th < QR) next = lse_of(it, (b + 2) * QR + th);
          named_sync(2 + grp, 128);
          lse = at;
        }
        mbar_wait(&bar[C::S_FULL + (n & 1)], (n >> 1) & 1, dead, f.status);
        tc_fence_after();
        const int all_see = max(0, it.at + kBN - 1 - prefix) << lg;  // rows from here on see the whole tile
        uint32_t x[32];
#pragma unroll
        for (int k = 0; k < QR / 32; ++k) {
          tc_ld32(tm + (n & 1) * QR + k * 32, x);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(x[i]));
          if (k + 1 == QR / 32) {  // the buffer is read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[C::S_FREE + (n & 1)]);
          }
          // (the same for all of the tile's threads: hidden positions, or rows behind the last)
          const int row0 = b * QR + k * 32;
          if (row0 >= R) continue;
          if (row0 >= all_see && row0 + 32 <= R) {
            const float4 *l4 = reinterpret_cast<const float4 *>(lse + k * 32);
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              float4 l = l4[c / 4];
              ffma2(l.x, l.y, __uint_as_float(x[c]), __uint_as_float(x[c + 1]), c2, c2);
              ffma2(l.z, l.w, __uint_as_float(x[c + 2]), __uint_as_float(x[c + 3]), c2, c2);
              ffma2(sum[0], sum[1], fast_exp2(l.x), fast_exp2(l.y), 1.f, 1.f);
              ffma2(sum[2], sum[3], fast_exp2(l.z), fast_exp2(l.w), 1.f, 1.f);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const int row = row0 + c;
              const float w = fast_exp2(fmaf(__uint_as_float(x[c]), c2, lse[k * 32 + c]));
              if (row >= first && row < R) sum[c & 3] += w;
            }
          }
        }
      }
      n = behind;
      // The other group's sum.  (A group that writes here for the next item but one has
      // stored the item between, behind the other's reading of this one.)
      float *add = s_sum + (item & 1) * kBN + th;
      const float w = (sum[0] + sum[1]) + (sum[2] + sum[3]);
      if (!store) {
        *add = w;
        named_arrive(4 + (item & 1), 256);
      } else {
        named_sync(4 + (item & 1), 256);
        if (page >= 0 && page < f.num_blocks) {
          float *dst = p.weights + ((size_t)page * f.num_kv_heads + it.kvh) * bs + pos % bs;
          const float all = *add + w;
          *dst = p.accumulate && pos < prefix ? *dst + all : all;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssueWarp) tc_dealloc(tmem, C::COLS);
}

template <int D>
cudaError_t launch_d(const SpanParams &p, cudaStream_t stream) {
  using C = Cfg<D>;
  const FwdParams &f = p.f;
  const unsigned long long row = D * 2, H = f.num_heads, Hk = f.num_kv_heads, bs = f.block_size,
                           NB = f.num_blocks, G = H / Hk;
  const int box = bs % 128 == 0 ? 128 : bs % 64 == 0 ? 64 : 16;
  const unsigned long long slot = p.hnd ? row : Hk * row, head = p.hnd ? bs * row : row;
  CUtensorMap tq, tk;
  {
    const unsigned long long d[3] = {D, H, (unsigned long long)f.num_tokens}, s[2] = {row, H * row};
    const unsigned int b[3] = {64, (unsigned)G, (unsigned)(C::QR / G)};
    if (!encode_tiled(&tq, f.q, PA_BF16, 3, d, s, b, true)) return cudaErrorInvalidValue;
  }
  {
    const unsigned long long d[4] = {D, Hk, bs, NB}, s[3] = {head, slot, bs * Hk * row};
    const unsigned int b[4] = {64, 1, (unsigned)box, 1};
    if (!encode_tiled(&tk, p.k_cache, PA_BF16, 4, d, s, b, true)) return cudaErrorInvalidValue;
  }
  auto kern = votes_mma_kernel<D>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = set_smem_attrs_once(kern, C::SMEM, done);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(C::CTAS * p.num_sms), dim3(kThreads), C::SMEM, stream, tq, tk, p, box);
}

}  // namespace

cudaError_t launch_votes_mma(const SpanParams &p, cudaStream_t stream) {
  return p.f.head_dim == 128 ? launch_d<128>(p, stream) : launch_d<64>(p, stream);
}

}  // namespace pa
