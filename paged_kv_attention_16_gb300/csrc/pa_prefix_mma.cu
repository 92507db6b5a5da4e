// pa_prefix_mma.cu -- the prefix part of pa_forward_shared_prefix on the
// tensor cores (bf16).
//
// Mathematics: for an item's 256 rows (128 / G tokens x the G heads of one KV
// head, twice) and the positions [kv_lo, kv_hi) of its split,
//   S = Q K^T,  m = running row maximum of scale S,  P = 2^(scale log2e S - m),
//   l = sum P,  O = sum P V,
// tile by tile of 128 positions, one pass over K and V.  Every position is
// visible to every row: no causal mask; only the last tile of a prefix may be
// short, its missing positions masked by select.
//
// One CTA per SM (224 KB of shared memory, all 512 TMEM columns), 16 warps:
//   warps 0-3, 4-7  softmax of the two 128-row tiles, thread = row (TMEM lane):
//                   S read once into 128 registers, lazy rescaling of O in
//                   TMEM (only when the maximum grows by more than 8, base 2),
//                   P as bf16 over the tile's own S
//   warps 8, 9      each issues one tile's products (one thread): S of tile j
//                   (M = 128, N = 128), then O += P V (P from TMEM)
//   warps 10-13     TMA: K boxes (10, 11) and V boxes (12, 13) into rings that
//                   both row tiles read
// While one row tile's softmax runs, the other's products do.  K and V are
// loaded once for 256 rows, so the loads stay below what HBM or L2 give as
// long as the products bound the tile; with few rows HBM does.
// A box that lies past the split, or on a bad page, is loaded from a page
// beyond the pool, which TMA fills with zeros: no NaN reaches a product, and
// every tile has the same byte count.
#include "pa_prefix.h"

namespace pa {
namespace {

constexpr int kBN = kPrefixTile;
constexpr float kTau = 8.0f;  // lazy-rescale headroom (base 2)
constexpr int kThreads = 512;
constexpr int kIssue0 = 8, kLoad0 = 10, kNumLoad = 4;  // issuing warps 8, 9; loading warps 10 .. 13
// launch registers 512 x 128; the softmax warpgroups take 200, the others keep 56
constexpr int kSoftmaxRegs = 200, kOtherRegs = 56;
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
  static constexpr int Q_FULL = 0, Q_FREE = 1, S_FULL = 2, P_FULL = 4, O_DONE = 6, O_FREE = 8,
                       K_FULL = 10, K_FREE = K_FULL + KST, V_FULL = K_FREE + KST,
                       V_FREE = V_FULL + VST, NBAR = V_FREE + VST;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 32;
  static constexpr uint32_t IDESC_S = umma_idesc_bf16(128, kBN, 0);
  static constexpr uint32_t IDESC_PV = umma_idesc_bf16(128, D, 1);
  static_assert(SMEM <= 232448, "shared memory of one CTA");
};

template <int N>
__device__ inline void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ inline void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 16 consecutive 32-bit TMEM columns of this thread's lane (warp-wide).
__device__ inline void tc_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

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
  pdl_trigger();
  if (smem_u32(smem) & 1023) {  // the same for every thread: all leave together
    if (tid == 0) atomicOr(f.status, PA_DEV_INTERNAL);
    return;
  }
  if (tid == 0) {
    prefetch_tensor_map(&tm_q);
    prefetch_tensor_map(&tm_k);
    prefetch_tensor_map(&tm_v);
    for (int b = 0; b < C::NBAR; ++b) {
      int n = 1;
      if (b == C::Q_FREE || (b >= C::K_FULL)) n = 2;  // two issuers / two loading warps
      if ((b >= C::P_FULL && b < C::P_FULL + 2) || (b >= C::O_FREE && b < C::O_FREE + 2)) n = 4;
      mbar_init(&bar[b], n);
    }
    fence_mbar_init();
  }
  if (warp == kIssue0) tc_alloc(s_tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  pdl_wait();  // the plan
  const long long n_items = p.plan->n_items;
  bool dead = false;

  if (warp >= kIssue0) {
    reg_dec<kOtherRegs>();
    if (warp >= kLoad0 && warp < kLoad0 + kNumLoad) {
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
      uint32_t st = 0, round = 0, items = 0;
      for (long long item = blockIdx.x; item < n_items; item += gridDim.x, ++items) {
        const PrefixItem it = prefix_item(p, item, G);
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
          mbar_arrive_expect_tx(&bar[C::Q_FULL], tiles * C::Q_TILE);
          for (int x = 0; x < tiles; ++x)
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
            mbar_arrive_expect_tx(&full[st], bytes);
          }
          __syncwarp();
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
    } else if (warp < kLoad0 && lane == 0) {
      // ------------------------------------------------------------- products
      const int x = warp - kIssue0;  // row tile
      const uint32_t sq = smem_u32(smem) + x * C::Q_TILE, sk = smem_u32(smem) + C::OFF_K,
                     sv = smem_u32(smem) + C::OFF_V;
      const uint32_t tm_s = tmem + x * 128, tm_o = tmem + kTmemO + x * 128;
      uint32_t ks = 0, kr = 0, vs = 0, vr = 0;  // ring stage and round
      uint32_t n = 0, items = 0, mine = 0;      // this tile's S products; items; items with rows here
      for (long long item = blockIdx.x; item < n_items; item += gridDim.x, ++items) {
        const PrefixItem it = prefix_item(p, item, G);
        const bool active = (it.q_len - it.t0) * G > x * 128;
        mbar_wait(&bar[C::Q_FULL], items & 1, dead, f.status);
        for (int lo = it.kv_lo; lo < it.kv_hi; lo += kBN) {
          mbar_wait(&bar[C::K_FULL + ks], kr & 1, dead, f.status);
          if (active) {
            // the S buffer holds P until the product that reads it is done
            if (n > 0) mbar_wait(&bar[C::O_DONE + x], (n - 1) & 1, dead, f.status);
            tc_fence_after();
            const uint32_t kb = sk + ks * C::KV_BYTES;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const int h = kk / 4, sub = kk % 4;
              tc_mma_bf16(tm_s, umma_desc_sw128(sq + h * 128 * 128 + sub * 32, 16, 1024),
                          umma_desc_sw128(kb + h * kBN * 128 + sub * 32, 16, 1024), C::IDESC_S,
                          kk > 0);
            }
            tc_commit(&bar[C::S_FULL + x]);
            tc_commit(&bar[C::K_FREE + ks]);
          } else {
            mbar_arrive(&bar[C::K_FREE + ks]);
          }
          if (++ks == C::KST) ks = 0, ++kr;
          if (active) mbar_wait(&bar[C::P_FULL + x], n & 1, dead, f.status);
          mbar_wait(&bar[C::V_FULL + vs], vr & 1, dead, f.status);
          if (active) {
            if (lo == it.kv_lo && mine > 0)
              mbar_wait(&bar[C::O_FREE + x], (mine - 1) & 1, dead, f.status);
            tc_fence_after();
            const uint32_t vb = sv + vs * C::KV_BYTES;
#pragma unroll
            for (int kk = 0; kk < kBN / 16; ++kk) {
              // 16 V rows; the leading offset steps to the next 64-wide chunk
              const int r = kk * 16;
              const uint32_t a = vb + (r / box) * C::NH * box * 128 + (r % box) * 128;
              tc_mma_bf16_ts(tm_o, tm_s + kk * 8, umma_desc_sw128(a, box * 128, 1024), C::IDESC_PV,
                             lo > it.kv_lo || kk > 0);
            }
            tc_commit(&bar[C::O_DONE + x]);
            tc_commit(&bar[C::V_FREE + vs]);
            ++n;
          } else {
            mbar_arrive(&bar[C::V_FREE + vs]);
          }
          if (++vs == C::VST) vs = 0, ++vr;
        }
        if (active) {
          tc_commit(&bar[C::Q_FREE]);
          ++mine;
        } else {
          mbar_arrive(&bar[C::Q_FREE]);
        }
      }
      // no commit of this thread may land after the CTA is gone
      if (items > 0) mbar_wait(&bar[C::Q_FREE], (items - 1) & 1, dead, f.status);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------------- softmax
    reg_inc<kSoftmaxRegs>();
    const int x = warp >> 2, r = tid & 127;  // row tile, row of it == TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tm_s = tmem + lane_off + x * 128, tm_o = tmem + lane_off + kTmemO + x * 128;
    const float c2 = f.scale_log2;
    // 2^(c s - m) as one multiply-add needs c > 0 (the maximum is then c max s)
    const bool fold = c2 > 0.f;
    uint32_t n = 0;
    for (long long item = blockIdx.x; item < n_items; item += gridDim.x) {
      const PrefixItem it = prefix_item(p, item, G);
      const int rows = min(128, (it.q_len - it.t0) * G - x * 128);
      if (rows <= 0) continue;
      // a bad page in the split marks all of the item's rows
      {
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
      const bool item_bad = s_bad[x] != 0;
      const bool warp_active = (warp & 3) * 32 < rows;  // its other rows are padding
      float m = -INFINITY, l = 0.f;
      for (int lo = it.kv_lo; lo < it.kv_hi; lo += kBN, ++n) {
        mbar_wait(&bar[C::S_FULL + x], n & 1, dead, f.status);
        tc_fence_after();
        if (warp_active) {
          float s[kBN];
#pragma unroll
          for (int c0 = 0; c0 < kBN; c0 += 32)
            tc_ld32(tm_s + c0, *reinterpret_cast<uint32_t(*)[32]>(s + c0));
          tc_wait_ld();
          if (!fold) {
#pragma unroll
            for (int c = 0; c < kBN; ++c) s[c] *= c2;
          }
          if (lo + kBN > it.kv_hi) {
#pragma unroll
            for (int c = 0; c < kBN; ++c) s[c] = lo + c < it.kv_hi ? s[c] : -INFINITY;
          }
          float mxa[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) mxa[c] = s[c];
#pragma unroll
          for (int c = 8; c < kBN; c += 2)
            mxa[(c >> 1) & 7] = fmax3(mxa[(c >> 1) & 7], s[c], s[c + 1]);
          float mx = fmax3(fmax3(mxa[0], mxa[1], mxa[2]), fmax3(mxa[3], mxa[4], mxa[5]),
                           fmaxf(mxa[6], mxa[7]));
          if (fold && mx != -INFINITY) mx *= c2;
          float alpha = 1.f;
          bool rescale = false;
          if (mx > m + kTau) {
            alpha = fast_exp2(m - mx);
            l *= alpha;
            m = mx;
            rescale = lo > it.kv_lo;
          }
          if (__any_sync(0xffffffffu, rescale)) {
            // (S of this tile was issued after the last product on O was done)
            const float a = rescale ? alpha : 1.f;
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += 16) {
              uint32_t raw[16];
              tc_ld16(tm_o + c0, raw);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) raw[i] = __float_as_uint(__uint_as_float(raw[i]) * a);
              tc_st16(tm_o + c0, raw);
            }
            tc_wait_st();
          }
          const float mu = m == -INFINITY ? 0.f : m;
          const float cs = fold ? c2 : 1.f;
          float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c0 = 0; c0 < kBN; c0 += 32) {
            uint32_t pw[16];
#pragma unroll
            for (int w = 0; w < 16; ++w) {
              float a0 = -mu, a1 = -mu;
              ffma2(a0, a1, s[c0 + 2 * w], s[c0 + 2 * w + 1], cs, cs);
              const float p0 = fast_exp2(a0), p1 = fast_exp2(a1);
              ffma2(sum[2 * (w & 3)], sum[2 * (w & 3) + 1], p0, p1, 1.f, 1.f);
              // weights to bf16 for the tensor core; their sum stays fp32
              const __nv_bfloat162 h2 = __floats2bfloat162_rn(p0, p1);
              pw[w] = *reinterpret_cast<const uint32_t *>(&h2);
            }
            tc_st16(tm_s + c0 / 2, pw);
          }
          tc_wait_st();
          l += ((sum[0] + sum[1]) + (sum[2] + sum[3])) + ((sum[4] + sum[5]) + (sum[6] + sum[7]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[C::P_FULL + x]);
      }
      // ---- O / l and the log-sum-exp of the rows
      mbar_wait(&bar[C::O_DONE + x], (n - 1) & 1, dead, f.status);
      tc_fence_after();
      if (warp_active) {
        const float inv = l > 0.f && !item_bad ? 1.f / l : 0.f;
        const uint32_t keep = item_bad ? 0u : 0xffffffffu;
        const long long prow = item * kPrefixRows + x * 128 + r;
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t raw[32];
          tc_ld32(tm_o + c0, raw);
          tc_wait_ld();
          if (r < rows) {
            float4 *dst = reinterpret_cast<float4 *>(p.part_o + prow * D + c0);
#pragma unroll
            for (int v = 0; v < 8; ++v)
              dst[v] = make_float4(__uint_as_float(raw[4 * v] & keep) * inv,
                                   __uint_as_float(raw[4 * v + 1] & keep) * inv,
                                   __uint_as_float(raw[4 * v + 2] & keep) * inv,
                                   __uint_as_float(raw[4 * v + 3] & keep) * inv);
          }
        }
        if (r < rows)
          p.part_lse[prow] = item_bad ? __int_as_float(0x7fc00000) : l > 0.f ? m + log2f(l) : -INFINITY;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[C::O_FREE + x]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssue0) tc_dealloc(tmem, kTmemCols);
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
