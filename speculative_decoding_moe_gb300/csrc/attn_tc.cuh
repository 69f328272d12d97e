// attn_tc.cuh -- what the attention kernels on the fifth-generation tensor cores
// share: descriptors and MMAs issued by an elected lane, tensor-memory loads and
// stores of a thread's row, and p = 2^(c s - z) of its scores, two at a time.
#pragma once

#include "tc05.cuh"
#include "tree_common.cuh"

namespace dfv {
namespace {

// shared-memory descriptor of a V tile as the B operand with its N dimension
// (the head's elements) contiguous: 128-byte swizzled rows of 64 elements, one
// row per key; stride byte offset 1024 between groups of 8 keys, leading byte
// offset 16 KB between blocks of 64 elements
__device__ __forceinline__ uint64_t sdesc_mn128(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3fffu);
  d |= (uint64_t)(16384u >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

// kind::f16 instruction descriptor: fp32 accumulator, both operands bf16 or
// both fp16, B with N contiguous when b_mn
template <bool F16>
__device__ __forceinline__ uint32_t idesc_16(int N, bool b_mn) {
  return (1u << 4) | (F16 ? 0u : (1u << 7) | (1u << 10)) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(128 >> 4) << 24);
}

// The MMA warp runs in step and an elected lane issues: descriptors are computed
// in uniform registers.  (Issued under `if (lane == 0)`, or under a predicate that
// does not come from elect.sync, every operand was moved there first, about as
// long as the MMA itself takes.)
// D[tmem] (+)= A[smem] * B[smem]^T
__device__ __forceinline__ void tc_mma_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Scores of a block: D[tmem] = A B^T over D elements, in blocks of 64: A's AROWS rows, B's
// 128 rows each.  One elected lane for all of it: an elect.sync an MMA took about as
// long as the MMA.
template <int D, int AROWS>
__device__ __forceinline__ void tc_scores(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc) {
  if (D == 128)
    asm volatile(
      "{\n .reg .pred no, yes, q;\n .reg .b64 a, b;\n setp.ne.b32 no, %3, %3;\n setp.eq.b32 yes, %3, %3;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, no;\n"
      " add.s64 a, %1, 2;\n add.s64 b, %2, 2;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, yes;\n"
      " add.s64 a, %1, 4;\n add.s64 b, %2, 4;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, yes;\n"
      " add.s64 a, %1, 6;\n add.s64 b, %2, 6;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, yes;\n"
      " add.s64 a, %1, %4;\n add.s64 b, %2, 1024;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, yes;\n"
      " add.s64 a, %1, %5;\n add.s64 b, %2, 1026;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, yes;\n"
      " add.s64 a, %1, %6;\n add.s64 b, %2, 1028;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, yes;\n"
      " add.s64 a, %1, %7;\n add.s64 b, %2, 1030;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, yes;\n"
      "}"
      ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "n"(AROWS * 8), "n"(AROWS * 8 + 2), "n"(AROWS * 8 + 4), "n"(AROWS * 8 + 6)
      : "memory");
  else
    asm volatile(
      "{\n .reg .pred no, yes, q;\n .reg .b64 a, b;\n setp.ne.b32 no, %3, %3;\n setp.eq.b32 yes, %3, %3;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, no;\n"
      " add.s64 a, %1, 2;\n add.s64 b, %2, 2;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, yes;\n"
      " add.s64 a, %1, 4;\n add.s64 b, %2, 4;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, yes;\n"
      " add.s64 a, %1, 6;\n add.s64 b, %2, 6;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, yes;\n"
      "}"
      ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc)
      : "memory");
}
// D[tmem] (+)= A[tmem] B over KEYS = 64 or 128 keys: A 8 columns further and B 16 rows of 128
// bytes further an MMA
template <int KEYS>
__device__ __forceinline__ void tc_values(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  if (KEYS == 128)
    asm volatile(
      "{\n .reg .pred p, yes, q;\n .reg .b64 b;\n .reg .b32 a;\n setp.ne.b32 p, %4, 0;\n setp.eq.b32 yes, %3, %3;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
      " add.s64 b, %2, 128;\n add.u32 a, %1, 8;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, yes;\n"
      " add.s64 b, %2, 256;\n add.u32 a, %1, 16;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, yes;\n"
      " add.s64 b, %2, 384;\n add.u32 a, %1, 24;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, yes;\n"
      " add.s64 b, %2, 512;\n add.u32 a, %1, 32;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, yes;\n"
      " add.s64 b, %2, 640;\n add.u32 a, %1, 40;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, yes;\n"
      " add.s64 b, %2, 768;\n add.u32 a, %1, 48;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, yes;\n"
      " add.s64 b, %2, 896;\n add.u32 a, %1, 56;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, yes;\n"
      "}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
  else
    asm volatile(
      "{\n .reg .pred p, yes, q;\n .reg .b64 b;\n .reg .b32 a;\n setp.ne.b32 p, %4, 0;\n setp.eq.b32 yes, %3, %3;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
      " add.s64 b, %2, 128;\n add.u32 a, %1, 8;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, yes;\n"
      " add.s64 b, %2, 256;\n add.u32 a, %1, 16;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, yes;\n"
      " add.s64 b, %2, 384;\n add.u32 a, %1, 24;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, yes;\n"
      "}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tc_commit_elect(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar)
      : "memory");
}

#define DFV_R8(r, b) "=f"(r[b]), "=f"(r[b + 1]), "=f"(r[b + 2]), "=f"(r[b + 3]), "=f"(r[b + 4]), "=f"(r[b + 5]), \
                     "=f"(r[b + 6]), "=f"(r[b + 7])
#define DFV_I8(r, b) "r"(r[b]), "r"(r[b + 1]), "r"(r[b + 2]), "r"(r[b + 3]), "r"(r[b + 4]), "r"(r[b + 5]), \
                     "r"(r[b + 6]), "r"(r[b + 7])

// 32 columns of the thread's lane; the caller waits
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : DFV_R8(r, 0), DFV_R8(r, 8), DFV_R8(r, 16), DFV_R8(r, 24)
      : "r"(addr));
}
// 16 columns, the caller waits
__device__ __forceinline__ void tmem_ld16_async(uint32_t addr, float *r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : DFV_R8(r, 0), DFV_R8(r, 8)
               : "r"(addr));
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), DFV_I8(r, 0) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      DFV_I8(r, 0), DFV_I8(r, 8)
      : "memory");
}
// Waits for every load of the thread; r passes through, so that no use of it can
// move above the wait.
#define DFV_P8(r, b) "+f"(r[b]), "+f"(r[b + 1]), "+f"(r[b + 2]), "+f"(r[b + 3]), "+f"(r[b + 4]), "+f"(r[b + 5]), \
                     "+f"(r[b + 6]), "+f"(r[b + 7])
__device__ __forceinline__ void tmem_wait_ld32(float *r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : DFV_P8(r, 0), DFV_P8(r, 8), DFV_P8(r, 16), DFV_P8(r, 24)::"memory");
}
__device__ __forceinline__ void tmem_wait_ld16(float *r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : DFV_P8(r, 0), DFV_P8(r, 8)::"memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void sts128(uint32_t addr, const uint4 &v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// (a, b) * (c, c) + (d, d) and sums, two at a time
__device__ __forceinline__ float2 fma2(float2 a, float c, float d) {
  float2 r;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %4};\n mov.b64 z, {%5, %5};\n"
      " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float max32(const float *s, float m) {
#pragma unroll
  for (int q = 0; q < 32; q += 2) m = fmaxf(m, fmaxf(s[q], s[q + 1]));
  return m;
}
__device__ __forceinline__ float max16(const float *s, float m) {
#pragma unroll
  for (int q = 0; q < 16; q += 2) m = fmaxf(m, fmaxf(s[q], s[q + 1]));
  return m;
}
// p of 16 scores less `from` as fp16 pairs, and their sum
__device__ __forceinline__ void exp16(const float *s, float from, float c, float z, uint32_t *x, float2 &l) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float2 y = fma2(add2(make_float2(s[2 * e], s[2 * e + 1]), make_float2(-from, -from)), c, -z);
    y.x = ex2(y.x);
    y.y = ex2(y.y);
    l = add2(l, y);
    x[e] = pack2<true>(y.x, y.y);
  }
}
// p of 32 scores as 16-bit pairs, and their sum
template <bool F16>
__device__ __forceinline__ void exp32(const float *s, float c, float z, uint32_t *x, float2 &l) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float2 y = fma2(make_float2(s[2 * e], s[2 * e + 1]), c, -z);
    y.x = ex2(y.x);
    y.y = ex2(y.y);
    l = add2(l, y);
    x[e] = pack2<F16>(y.x, y.y);
  }
}

// Scores of a tile whose first key is node j0 (below 0: committed): what the row
// does not see becomes -inf, in place.  A short loop: it runs once per sequence, and
// unrolled its instructions took longer to fetch than to execute.
__device__ __forceinline__ void mask_tile(uint32_t t_s, int j0, uint64_t mask) {
#pragma unroll 1
  for (int q = 0; q < 128; q += 16) {
    const int j = j0 + q;  // node of the first of 16 keys
    if (j + 16 <= 0) continue;
    uint32_t sees;
    if (j >= 0)
      sees = j < 64 ? (uint32_t)(mask >> j) : 0u;
    else
      sees = (uint32_t)(mask << -j) | ((1u << -j) - 1u);
    float s[16];
    tmem_ld16(t_s + q, s);
    uint32_t x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = sees >> e & 1u ? __float_as_uint(s[e]) : 0xff800000u;
    tmem_st16(t_s + q, x);
  }
  tmem_wait_st();
}

}  // namespace
}  // namespace dfv
