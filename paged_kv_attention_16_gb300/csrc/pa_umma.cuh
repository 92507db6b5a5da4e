// pa_umma.cuh -- what the tcgen05 kernels of one issuing warp a row tile share
// (pa_prefix_mma.cu, pa_span_mma.cu, pa_votes_mma.cu): register shares, tensor-
// memory loads, descriptors and products issued by converged warps.
#pragma once

#include "pa_common.cuh"

namespace pa {

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

// tcgen05.wait::ld, which the uses of these registers stay behind.
__device__ inline void wait_ld(uint32_t (&a)[32], uint32_t (&b)[32]) {
  tc_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(a[i]), "+r"(b[i]));
}

// 32 bytes in one store.
__device__ inline void store32(float *dst, const uint32_t (&v)[32], int at, float scale) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(v[at + i]) * scale;
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(x[0]),
               "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
               : "memory");
}

// Matrix descriptors of 128-byte-swizzled tiles by their two words: the high
// one (8-row groups 1024 bytes apart) is the same for every operand here, the
// low one is the address and the leading offset, both in 16-byte units.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ inline uint32_t desc_lo(uint32_t saddr, uint32_t leading) {
  return ((saddr >> 4) & 0x3FFFu) | (leading >> 4) << 16;
}

// The products and commits are run by a whole warp, one lane of it issuing
// (always the same one).  Run by one lane in a branch of its own, an issue
// held the thread for 85 clocks (A from shared memory) or 120 (from tensor
// memory); run by a converged warp it takes 35 to 45.

// tmem_d (+)= A B^T, A and B from shared memory.
__device__ inline void mma_ss(uint32_t tmem_d, uint32_t alo, uint32_t blo, uint32_t idesc,
                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(alo), "r"(blo), "r"(idesc), "r"(accumulate), "r"(kDescHi)
      : "memory");
}

// tmem_d (+)= A B, A (bf16 pairs) from tensor memory.
__device__ inline void mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint32_t blo, uint32_t idesc,
                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "r"(blo), "r"(idesc), "r"(accumulate), "r"(kDescHi)
      : "memory");
}

// Arrive on `bar` when every product issued so far by the electing lane is done.
__device__ inline void commit(uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}

}  // namespace pa
