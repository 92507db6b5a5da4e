// pa_votes.cu -- the sums over rows of pa_forward_weights: with L_r the
// log-sum-exp of row r (its sink included) and s_rj its score of position j,
//   W[kv head][slot of j] (+)= sum_r 2^(s_rj - L_r)
// over the rows of the KV head, position by position, each written by one thread
// in a fixed order of rows: no atomics, the same bits every time.
#include <algorithm>

#include "pa_span.h"

namespace pa {
namespace {

constexpr int kVoteThreads = 256;

// The weight of one score; a row that sees nothing (L = -inf) has none.
__device__ inline float vote(float score, float lse) {
  return lse == -INFINITY ? 0.f : fast_exp2(score - lse);
}

// Whether the request's last row met a bad page: it sees all of them.
__device__ inline bool request_bad(const SpanParams &p, const SpanReq &r) {
  return __ldcg(p.row_lse + (size_t)(r.q_start + r.q_len - 1) * p.f.num_heads) == INFINITY;
}

// fp32: 64 positions x 64 rows a step, a thread 4 positions x 4 rows; a block's keys
// stay in shared memory while all rows pass.  Bound by the multiply-adds and the shared
// memory that feeds them: 16 windows of 64 tokens, 16/4 heads of 64, up to 16384
// positions: 0.81 ms, 16 TFLOP/s (two rows a thread and neighbouring positions, whose
// keys met in one bank: 1.79).
constexpr int kPos = 64, kRows = 64, kOwn = kRows / 16;  // kOwn: rows of a thread, 16 apart

__device__ inline float4 load4f(const float *src) { return *reinterpret_cast<const float4 *>(src); }

template <int D>
__global__ void __launch_bounds__(kVoteThreads) votes_simt_kernel(const SpanParams p, int chunks) {
  extern __shared__ __align__(16) float s_dyn[];
  constexpr int LD = D + 4;
  float *s_k = s_dyn, *s_q = s_dyn + kPos * LD;
  __shared__ float s_lse[kRows], s_sum[kVoteThreads / 16][kPos];
  const FwdParams &f = p.f;
  const int tid = threadIdx.x, H = f.num_heads, Hk = f.num_kv_heads, G = H / Hk, bs = f.block_size;
  const int tx = tid & 15, ty = tid >> 4;  // positions tx, tx + 16, .. (no two in a bank), rows ty, ty + 16, ..
  pdl_trigger();
  pdl_wait();
  if (p.plan->all_bad) return;
  const long long n = (long long)chunks * f.num_seqs * Hk;
  for (long long item = blockIdx.x; item < n; item += gridDim.x) {
    const int sh = (int)(item % ((long long)f.num_seqs * Hk)), s = sh / Hk, kvh = sh % Hk;
    const int at = (int)(item / ((long long)f.num_seqs * Hk)) * kPos;
    const SpanReq r = p.req[s];
    if (r.nblk == 0 || r.score0 >= 0 || at >= r.ctx) continue;
    if (request_bad(p, r)) continue;
    const int32_t *bt = f.block_table + (size_t)s * f.max_blocks_per_seq;
    const int R = r.q_len * G, prefix = r.ctx - r.q_len;
    __syncthreads();
    for (int e = tid; e < kPos * (D / 4); e += kVoteThreads) {
      const int j = e / (D / 4), x = e % (D / 4) * 4, pos = at + j;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      const int page = pos < r.ctx ? bt[pos / bs] : -1, slot = pos % bs;
      if (page >= 0 && page < f.num_blocks) {
        const size_t row = p.hnd ? ((size_t)page * Hk + kvh) * bs + slot : ((size_t)page * bs + slot) * Hk + kvh;
        v = load4f(static_cast<const float *>(p.k_cache) + row * D + x);
      }
      *reinterpret_cast<float4 *>(&s_k[j * LD + x]) = v;
    }
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    // rows that see none of these positions are left out
    const int first = max(0, at - prefix) * G;
    for (int r0 = first / kRows * kRows; r0 < R; r0 += kRows) {
      __syncthreads();
      for (int e = tid; e < kRows * (D / 4); e += kVoteThreads) {
        const int i = e / (D / 4), x = e % (D / 4) * 4, row = min(r0 + i, R - 1);
        const size_t at_q = ((size_t)(r.q_start + row / G) * H + kvh * G + row % G) * D + x;
        float4 v = load4f(static_cast<const float *>(f.q) + at_q);
        v.x *= f.scale_log2;
        v.y *= f.scale_log2;
        v.z *= f.scale_log2;
        v.w *= f.scale_log2;
        *reinterpret_cast<float4 *>(&s_q[i * LD + x]) = v;
      }
      if (tid < kRows) {
        const int row = r0 + tid;
        s_lse[tid] = row < R ? __ldcg(p.row_lse + (size_t)(r.q_start + row / G) * H + kvh * G + row % G)
                             : -INFINITY;
      }
      __syncthreads();
      float even[kOwn][4] = {}, odd[kOwn][4] = {};  // sums over even and odd columns
#pragma unroll 2
      for (int x = 0; x < D; x += 4) {
        float4 a[kOwn], b[4];
#pragma unroll
        for (int i = 0; i < kOwn; ++i) a[i] = *reinterpret_cast<const float4 *>(&s_q[(ty + 16 * i) * LD + x]);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4 *>(&s_k[(tx + 16 * j) * LD + x]);
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            ffma2(even[i][j], odd[i][j], a[i].x, a[i].y, b[j].x, b[j].y);
            ffma2(even[i][j], odd[i][j], a[i].z, a[i].w, b[j].z, b[j].w);
          }
      }
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int row = r0 + ty + 16 * i, own = prefix + min(row, R - 1) / G;
        const float l = s_lse[ty + 16 * i];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (at + tx + 16 * j <= own) sum[j] += vote(even[i][j] + odd[i][j], l);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) s_sum[ty][tx + 16 * j] = sum[j];
    __syncthreads();
    if (tid < kPos / 4 && at + tid * 4 < r.ctx) {
      float tot[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float x = 0.f;
        for (int y = 0; y < kVoteThreads / 16; ++y) x += s_sum[y][tid * 4 + j];
        tot[j] = x;
      }
      span_add_votes(p, r, bt[(at + tid * 4) / bs], kvh, at + tid * 4, tot);
    }
  }
}

template <int D>
cudaError_t launch_simt(const SpanParams &p, cudaStream_t st) {
  constexpr int kSmem = (kPos + kRows) * (D + 4) * (int)sizeof(float);
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = set_smem_attrs_once(votes_simt_kernel<D>, kSmem, done);
  if (e != cudaSuccess) return e;
  const long long chunks = ceil_div_ll(std::max(p.f.max_seq_len, 1), kPos);
  const long long n = chunks * p.f.num_seqs * p.f.num_kv_heads;
  return launch_dependent(votes_simt_kernel<D>, dim3((unsigned)std::min<long long>(n, 3ll * p.num_sms)),
                          dim3(kVoteThreads), kSmem, st, p, (int)chunks);
}

}  // namespace

cudaError_t launch_votes(const SpanParams &p, cudaStream_t stream) {
  if (p.f.dtype == PA_BF16) return launch_votes_mma(p, stream);
  return p.f.head_dim == 128 ? launch_simt<128>(p, stream) : launch_simt<64>(p, stream);
}

}  // namespace pa
