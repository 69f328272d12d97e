// tree_attn_tc.cu -- tree attention with many rows per kv head, on the
// fifth-generation tensor cores.
//
// A CTA takes 128 rows (SINGLE) or 256 rows (DUAL) of one kv head and streams
// the keys in tiles of 128: S = Q K^T into tensor memory, a warpgroup turns S
// into P = 2^(c S - M) (one row per thread, so the maximum and the sum need no
// shuffles) and writes P over S, and O += P V accumulates in tensor memory with
// P as the tensor-memory operand.  Two warpgroups keep the tensor core busy
// while the other is in its exponentials:
//   SINGLE  they take the even and the odd key tiles of the same rows, each with
//           its own (M, l, O); the two states are joined at the end
//   DUAL    they take 128 rows each and every key tile; a tile is fetched once
//           for 256 rows
// M is only raised, and O only rescaled, when a row's maximum grew by more than
// 2^8: p then stays below 2^8 (fp16: 2^14 with its offset), the sums are exact
// in the same M, and almost every tile needs one pass over its scores and no read
// or write of O.
//
// What binds: with one 128-row tile the reading of the cache (32 sequences x 16
// nodes x 8 heads over up to 8191 keys: 90 us, 4.6 TB/s with 8 us before the first
// product and ranges that end 10 us apart); with two the tensor core's shared
// memory, which the first product reads at its full rate for both operands while
// the copies write it (8 sequences x 64 nodes over up to 32749 keys: 196 us as a call
// among others, 1.07 PFLOP/s; 179 to 181 replayed from a graph, of which the products
// without exponentials alone take 165).
//
// Warps 0-3 and 4-7 are the two warpgroups, warps 8 and 10 stream K and V tiles
// with TMA into one ring in the order the MMAs use them (half of each tile's boxes
// each), warp 9 issues the MMAs.
// Tensor memory: S0 S1 O0 O1 of 128 columns each; P (16-bit pairs) over S.
#include <cstdio>

#include "tc05.cuh"
#include "tree_attn.cuh"

namespace dfv {
namespace {

constexpr int kTKeys = 128;
constexpr int kTThreads = 352;
constexpr int kProducers = 2;

template <int D, bool DUAL>
struct TcShape {
  static constexpr uint32_t kTile = kTKeys * D * 2;            // one K or V tile
  static constexpr int kSlots = D == 64 ? 8 : DUAL ? 5 : 6;
  static constexpr int kOver = DUAL ? 5 : 2;                   // tiles' worth of time that a pair costs at least
  static constexpr uint32_t kQ = (DUAL ? 2 : 1) * 128 * D * 2;
  static constexpr size_t kSmem = 1024 + kQ + (size_t)kSlots * kTile;
};

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
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

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
// does not see becomes -inf, in place.  A short loop, as is clean_row: they run
// once per sequence, and unrolled their instructions took longer to fetch than
// to execute.
__device__ __forceinline__ void mask_tile(uint32_t t_s, int j0, uint64_t mask) {
#pragma unroll 1
  for (int q = 0; q < kTKeys; q += 16) {
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

// Key row `row` of a V tile in shared memory: zeroed past the last node (j >= n);
// a node's values that are not finite become zero and set *bad.
template <bool F16, int D>
__device__ __forceinline__ void clean_row(unsigned char *tile, int row, int j, int n, int *bad) {
  if (j < 0) return;
  constexpr uint32_t kExp = F16 ? 0x7c00u : 0x7f80u;
#pragma unroll 1
  for (int c = 0; c < D / 8; ++c) {  // chunk order turned by the row: no bank conflicts, and any order will do
    uint4 *at = reinterpret_cast<uint4 *>(tile + (c >> 3) * 16384 + row * 128 + (((c ^ row) & 7) << 4));
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    bool hit = j >= n;
    if (!hit) {
      v = *at;
      uint32_t *w = &v.x;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if ((w[e] & kExp) == kExp) { w[e] &= 0xffff0000u; hit = true; }
        if ((w[e] & (kExp << 16)) == (kExp << 16)) { w[e] &= 0x0000ffffu; hit = true; }
      }
      if (hit) *bad = 1;
    }
    if (hit) *at = v;
  }
}

template <bool F16, int D, bool DUAL>
__global__ void __launch_bounds__(kTThreads, 1) tree_attn_tc_kernel(const __grid_constant__ AttnLaunch L) {
  using S = TcShape<D, DUAL>;
  constexpr int LA = DUAL ? 1 : 2;  // K tiles ahead of the V tile in the ring
  constexpr float kBias = F16 ? 6.f : 0.f;
  constexpr int kHalves = D / 64;
  extern __shared__ __align__(16) unsigned char sm_raw[];
  unsigned char *sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) unsigned long long s_full[S::kSlots], s_empty[S::kSlots], s_sfull[2], s_pready[2], s_odone[2],
      s_qready, s_drain;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ SchedStart s_start;
  __shared__ long long s_scan[kTThreads / 32];
  __shared__ int s_bad;
  const TreeAttnParams &p = L.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned char *s_q = sm, *s_ring = sm + S::kQ;
  const uint32_t q_addr = smem_u32(s_q), ring = smem_u32(s_ring);
  if (tid == 0) {
    s_abort = 0;
    s_bad = 0;
    for (int s = 0; s < S::kSlots; ++s) {
      mbar_init(smem_u32(&s_full[s]), kProducers);
      mbar_init(smem_u32(&s_empty[s]), 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(smem_u32(&s_sfull[w]), 1);
      mbar_init(smem_u32(&s_pready[w]), 128);
      mbar_init(smem_u32(&s_odone[w]), 1);
    }
    mbar_init(smem_u32(&s_qready), 256);
    mbar_init(smem_u32(&s_drain), 1);
    mbar_init_fence();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&s_tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  pdl_wait();
  pdl_trigger();  // the join may now read the call's inputs
  sched_start<kTThreads, kTKeys, S::kOver>(L, blockIdx.x, s_scan, &s_start);  // syncs the CTA
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int row0 = (int)(blockIdx.x % L.n_rt) * L.rows;  // first row of this CTA
  SegWalk<kTKeys, S::kOver> wk(L, s_start);

  if (warp == 8 || warp == 10) {
    // ---------------------------------------------------------------- producer
    const int me = (warp - 8) / 2;
    int st = 0, ph = 0, issued = 0;
    bool ok = true;
    const int shift = p.c.page_shift, boxes = shift >= 7 ? 1 : kTKeys >> shift, rows = kTKeys / boxes;
    while (ok && wk.next()) {
      if (row0 >= wk.v.n * p.G) continue;
      const int pages = wk.v.s < 0 ? 0 : (wk.total + (1 << shift) - 1) >> shift, n = wk.t1 - wk.t0;
      const int32_t *table = p.c.table + (size_t)(wk.v.s < 0 ? 0 : wk.v.s) * p.c.max_pages;
      auto page = [&](int j) {  // this lane's page of the segment's tile j, or -1 when there is none
        const int at = (((wk.t0 + j) * kTKeys) >> shift) + lane;
        return j < n && lane < boxes && at < pages ? checked_page(p.c, table[at]) : -1;
      };
      auto load = [&](const CUtensorMap *map, int j, int pg) {
        ok = ok && __all_sync(0xffffffffu,
                              mbar_wait_fast(smem_u32(&s_empty[st]), ph ^ 1, p.err, DFV_DEVERR_SLOT_WAIT, &s_abort));
        if (!ok) return;
        const uint32_t fb = smem_u32(&s_full[st]), dst = ring + (uint32_t)st * S::kTile;
        const int nb = __popc(__ballot_sync(0xffffffffu, pg >= 0));
        // this warp's boxes: one half of the head (D = 128), or every other page
        const int b0 = kHalves > 1 ? 0 : me, step = kHalves > 1 ? 1 : kProducers, hf = kHalves > 1 ? me : 0;
        const int mine = (nb - b0 + step - 1) / step;
        if (lane == 0) {
          if (mine > 0)
            mbar_expect_tx(fb, (uint32_t)mine * rows * 128);
          else
            mbar_arrive(fb);
        }
        __syncwarp();
        const int tok = ((wk.t0 + j) * kTKeys) & ((1 << shift) - 1);  // 0 unless a page holds several tiles
#pragma unroll 2
        for (int b = b0; b < nb; b += step)
          tma_kv(dst + (uint32_t)(hf * 16384 + b * rows * 128), map, hf * 64, tok, wk.h, __shfl_sync(0xffffffffu, pg, b),
                 L.swap, fb);
        ++issued;
        if (++st == S::kSlots) { st = 0; ph ^= 1; }
      };
      // pages of tiles j .. j + LA, and one more fetched ahead
      int pg[LA + 2];
#pragma unroll
      for (int k = 0; k < LA + 2; ++k) pg[k] = page(k);
#pragma unroll
      for (int k = 0; k < LA; ++k)
        if (k < n) load(&L.tm_k, k, pg[k]);
      for (int j = 0; j < n && ok; ++j) {
        load(&L.tm_v, j, pg[0]);
        if (j + LA < n) load(&L.tm_k, j + LA, pg[LA]);
#pragma unroll
        for (int k = 0; k < LA + 1; ++k) pg[k] = pg[k + 1];
        pg[LA + 1] = page(j + LA + 2);
      }
    }
    // no copy may land after the CTA exits: wait for the last fill of every slot
    volatile int never = 0;
    for (int j = issued - S::kSlots < 0 ? 0 : issued - S::kSlots; j < issued; ++j)
      if (!mbar_wait(smem_u32(&s_full[j % S::kSlots]), (j / S::kSlots) & 1, p.err, DFV_DEVERR_DRAIN_WAIT, &never)) break;
  } else if (warp == 9) {
    // ---------------------------------------------------------------- MMA issue
    {
      int st = 0, ph = 0, seg = 0;
      unsigned np[2] = {0u, 0u};  // tiles of each warpgroup whose P was awaited
      bool ok = true;
      const uint32_t iq = idesc_16<F16>(kTKeys, false), iv = idesc_16<F16>(D, true);
      auto full = [&]() {
        ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_full[st]), ph, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
        tc_fence_after();
      };
      auto done = [&]() {  // the slot is free once the MMAs issued so far have read it
        tc_commit_elect(smem_u32(&s_empty[st]));
        if (++st == S::kSlots) { st = 0; ph ^= 1; }
      };
      auto qk = [&](int w) {
        const uint32_t kb = ring + (uint32_t)st * S::kTile, qb = q_addr + (DUAL ? (uint32_t)w * 128u * D * 2u : 0u);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          tc_mma_ss(tmem + (uint32_t)w * 128u, sdesc_k128(qb + (ks >> 2) * 16384) + (uint64_t)(2 * (ks & 3)),
                 sdesc_k128(kb + (ks >> 2) * 16384) + (uint64_t)(2 * (ks & 3)), iq, ks > 0 ? 1u : 0u);
        tc_commit_elect(smem_u32(&s_sfull[w]));
      };
      auto pv = [&](int w, bool first, bool last) {
        const uint32_t vb = ring + (uint32_t)st * S::kTile;
        ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_pready[w]), np[w] & 1u, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
        if (!ok) return;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < kTKeys / 16; ++ks)
          tc_mma_ts(tmem + 256u + (uint32_t)w * 128u, tmem + (uint32_t)w * 128u + (uint32_t)ks * 8u,
                    sdesc_mn128(vb + (uint32_t)ks * 2048u), iv, (first && ks == 0) ? 0u : 1u);
        ++np[w];
        if (last) tc_commit_elect(smem_u32(&s_odone[w]));
      };
      while (ok && wk.next()) {
        if (row0 >= wk.v.n * p.G) continue;
        const int n = wk.t1 - wk.t0;
        ok = __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_qready), seg & 1, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
        ++seg;
        tc_fence_after();
        if (DUAL) {
          full();
          if (!ok) break;
          qk(0);
          qk(1);
          done();
          for (int j = 0; j < n && ok; ++j) {
            // V_j, then K_j+1; each warpgroup's next scores right after its own product
            full();
            if (!ok) break;
            pv(0, j == 0, j == n - 1);
            if (!ok) break;
            if (j + 1 < n) {
              int kst = st + 1, kph = ph;
              if (kst == S::kSlots) { kst = 0; kph ^= 1; }
              const int sv = st, pv_ = ph;
              st = kst; ph = kph;
              full();
              if (!ok) break;
              qk(0);
              st = sv; ph = pv_;
            }
            pv(1, j == 0, j == n - 1);
            if (!ok) break;
            done();  // V_j
            if (j + 1 < n) {
              qk(1);
              done();  // K_j+1
            }
          }
        } else {
          for (int k = 0; k < LA && k < n && ok; ++k) {
            full();
            if (!ok) break;
            qk(k);
            done();
          }
          for (int j = 0; j < n && ok; ++j) {
            full();
            if (!ok) break;
            pv(j & 1, j < 2, j + 2 >= n);
            if (!ok) break;
            done();
            if (j + LA < n) {
              full();
              if (!ok) break;
              qk(j & 1);
              done();
            }
          }
        }
      }
      // every MMA issued has completed before tensor memory is released
      tc_commit_elect(smem_u32(&s_drain));
      volatile int never = 0;
      mbar_wait(smem_u32(&s_drain), 0u, p.err, DFV_DEVERR_DRAIN_WAIT, &never);
    }
  } else {
    // ---------------------------------------------------------------- softmax and output
    const int w = warp >> 2, wt = tid & 127;  // warpgroup, and its thread = row of the tile
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_s = lane_base + (uint32_t)w * 128u, t_o = lane_base + 256u + (uint32_t)w * 128u;
    const float c = p.scale_log2;
    unsigned nt = 0;     // tiles this warpgroup has taken
    unsigned outs = 0;   // segments it has put out
    unsigned items = 0;  // ring items of the segments before
    bool ok = true;
    // after a wait gives up the loops still run to the end without touching
    // tensor memory, so the warpgroups meet at every barrier
    while (wk.next()) {
      const int R = wk.v.n * p.G;
      if (row0 >= R) continue;  // never the CTA that tells of the pair: its rows are the first
      const int n = wk.t1 - wk.t0;
      // rows into the swizzled layout; past R zero
      {
        constexpr int kCh = D / 8, kStep = 256 / kCh;  // 16-byte chunks of a row; rows apart
        constexpr int kIter = (DUAL ? 256 : 128) / kStep, kBatch = kIter < 8 ? kIter : 8;
        const int ch = tid % kCh;
        const char *qh = p.q + 2 * (wk.v.row0 * p.q_row + (long long)wk.h * p.G * p.q_head + ch * 8);
        uint4 x[kBatch];
#pragma unroll
        for (int k0 = 0; k0 < kIter; k0 += kBatch) {
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int r = row0 + tid / kCh + (k0 + k) * kStep, i = node_of(L, r);
            x[k] = make_uint4(0u, 0u, 0u, 0u);
            if (r < R) x[k] = *reinterpret_cast<const uint4 *>(qh + 2 * (i * p.q_row + (r - i * p.G) * p.q_head));
          }
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int rr = tid / kCh + (k0 + k) * kStep;
            *reinterpret_cast<uint4 *>(s_q + (rr >> 7) * (128 * D * 2) + (ch >> 3) * 16384 + (rr & 127) * 128 +
                                       (((ch & 7) ^ (rr & 7)) << 4)) = x[k];
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(smem_u32(&s_qready));

      const int r = row0 + (DUAL ? w * 128 : 0) + wt;  // this thread's row
      uint64_t mask = 0;
      if (r < R) mask = wk.mask_of(r);
      float m = -INFINITY, l = 0.f;
      bool started = false;
      for (int j = DUAL ? 0 : w; j < n; j += DUAL ? 1 : 2) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_sfull[w]), nt & 1u, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
        ++nt;
        if (!ok) continue;
        tc_fence_after();
        const int k0 = (wk.t0 + j) * kTKeys, j0 = k0 - wk.v.len;  // node number of the tile's first key
        const bool special = j0 + kTKeys > 0;  // tree nodes or keys past the end in the tile
        if (special) mask_tile(t_s, j0, mask);
        if (special && (!DUAL || w == 0)) {
          // this tile's V before it is multiplied
          const unsigned it = items + (unsigned)(j + (j + LA < n ? j + LA : n));
          ok = __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_full[it % S::kSlots]), (it / S::kSlots) & 1u, p.err,
                                                      DFV_DEVERR_STAGE_WAIT, &s_abort));
          if (!ok) continue;
          clean_row<F16, D>(s_ring + (size_t)(it % S::kSlots) * S::kTile, wt, j0 + wt, wk.nodes, &s_bad);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        // One pass with the M so far: p and the new maximum together, a quarter
        // of the scores read while the one before is used.  Only when some row's
        // maximum grew too far is O rescaled and the pass made again (the first
        // tile's always is).
        uint32_t x[64];
        float2 l2;
        for (;;) {
          const float z = (m == -INFINITY ? 0.f : m * c) - kBias;
          float s0[32], s1[32], mx = m;
          l2 = make_float2(0.f, 0.f);
          tmem_ld32(t_s, s0);
          tmem_wait_ld32(s0);
          tmem_ld32(t_s + 32, s1);
          mx = max32(s0, mx);
          exp32<F16>(s0, c, z, x, l2);
          tmem_wait_ld32(s1);
          tmem_ld32(t_s + 64, s0);
          mx = max32(s1, mx);
          exp32<F16>(s1, c, z, x + 16, l2);
          tmem_wait_ld32(s0);
          tmem_ld32(t_s + 96, s1);
          mx = max32(s0, mx);
          exp32<F16>(s0, c, z, x + 32, l2);
          tmem_wait_ld32(s1);
          mx = max32(s1, mx);
          exp32<F16>(s1, c, z, x + 48, l2);
          if (!__any_sync(0xffffffffu, (mx - m) * c > 8.f)) break;
          if (started) {
            // the last product into O is complete: it was issued before these
            // scores, and their barrier follows all that was issued before it
            const float f = m == -INFINITY ? 0.f : ex2((m - mx) * c);
            l *= f;
#pragma unroll 1
            for (int q = 0; q < D; q += 16) {
              float o[16];
              tmem_ld16(t_o + q, o);
              uint32_t y[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(o[e] * f);
              tmem_st16(t_o + q, y);
            }
          }
          m = mx;
        }
        started = true;
        l += l2.x + l2.y;
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_st16(t_s + 16 * q, x + 16 * q);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(smem_u32(&s_pready[w]));
      }
      items += 2u * (unsigned)n;
      // ---- output: the last product of this warpgroup, then (SINGLE) both states
      if (DUAL || w < n) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_odone[w]), outs & 1u, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
        ++outs;
      }
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      const int rr = DUAL ? w * 128 + wt : wt;
      float M = m, lsum = l, f0 = 1.f, f1 = 1.f;
      // all scores are done when either warpgroup's last product is: Q's place is free
      float2 *ml = reinterpret_cast<float2 *>(s_q);
      if (!DUAL && started) ml[w * 128 + wt] = make_float2(m, l);
      // SINGLE: each warpgroup waited for its own products and reads both outputs, so
      // what it learned about tensor memory goes through the barrier
      tc_fence_before();
      bar_sync_n(1, 256);  // the states, s_bad, and Q's place
      tc_fence_after();
      if (!DUAL) {
        const float2 a = ml[wt];
        const float2 b = n > 1 ? ml[128 + wt] : make_float2(-INFINITY, 0.f);
        M = fmaxf(a.x, b.x);
        // a state without keys adds its zeros (or NaN of a NaN query)
        f0 = a.x == -INFINITY ? 1.f : ex2((a.x - M) * c);
        f1 = b.x == -INFINITY ? 1.f : ex2((b.x - M) * c);
        lsum = a.y * f0 + b.y * f1;
      }
      const int bad = s_bad;
      const float z = (M == -INFINITY ? 0.f : M * c) - kBias;
      const int c0 = DUAL ? 0 : w * (D / 2), c1 = DUAL ? D : c0 + D / 2;
      const bool whole = wk.whole();
      const int slot = wk.slot(blockIdx.x), i = node_of(L, r), head = wk.h * p.G + r - i * p.G;
      const size_t row = wk.v.row0 + i;
      const float inv = lsum == 0.f ? 0.f : 1.f / lsum;  // NaN stays NaN
      char *out = p.o + 2 * (row * p.o_row + head * p.o_head);
      float4 *part = reinterpret_cast<float4 *>(L.part_o) + (size_t)slot * (D / 4) * L.rows + rr;
#pragma unroll 1
      for (int q = c0; q < c1 && ok; q += 32) {
        float o[32];
        tmem_ld32(lane_base + 256u + (DUAL ? (uint32_t)w * 128u : 0u) + q, o);
        if (!DUAL && n > 1) {
          float o1[32];
          tmem_ld32(lane_base + 384u + q, o1);
          tmem_wait_ld32(o);
          tmem_wait_ld32(o1);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = o[e] * f0 + o1[e] * f1;
        } else {
          tmem_wait_ld32(o);
        }
        if (r >= R) continue;
        if (whole) {
          uint32_t x[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = pack2<F16>(o[2 * e] * inv, o[2 * e + 1] * inv);
          uint4 *to = reinterpret_cast<uint4 *>(out + 2 * q);
#pragma unroll
          for (int e = 0; e < 4; ++e) to[e] = make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        } else {
          float4 *to = part + (size_t)(q / 4) * L.rows;
#pragma unroll
          for (int e = 0; e < 8; ++e) to[(size_t)e * L.rows] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      if (r < R && ok && c0 == 0) {
        if (whole) {
          if (p.lse) p.lse[row * p.H + head] = lsum == 0.f ? -INFINITY : (z + log2f(lsum)) * 0.69314718055994531f;
        } else {
          L.part_ml[(size_t)slot * L.rows + rr] = make_float2(M == -INFINITY ? -INFINITY : z, lsum);
        }
      }
      if (whole && bad && r < R && ok) add_unseen<F16>(p, wk.v, i, wk.h, out, c0, c1);
      if (tid == 0) {
        if (!whole) L.part_bad[slot] = bad;
        wk.tell(s_start, blockIdx.x);
      }
      tc_fence_before();
      bar_sync_n(1, 256);  // O, Q's place and s_bad are read
      if (tid == 0) s_bad = 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

template <bool F16, int D, bool DUAL>
cudaError_t launch_one(const AttnLaunch &L, cudaStream_t s) {
  auto kern = tree_attn_tc_kernel<F16, D, DUAL>;
  const size_t smem = TcShape<D, DUAL>::kSmem;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kern, smem, done);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, dim3(L.n_groups * L.n_rt), dim3(kTThreads), smem, s, L);
}

}  // namespace

cudaError_t launch_attn_tc(const AttnLaunch &L, cudaStream_t s) {
  const bool dual = L.rows == 256;
  if (L.p.c.D == 128) {
    if (L.p.c.f16) return dual ? launch_one<true, 128, true>(L, s) : launch_one<true, 128, false>(L, s);
    return dual ? launch_one<false, 128, true>(L, s) : launch_one<false, 128, false>(L, s);
  }
  if (L.p.c.f16) return dual ? launch_one<true, 64, true>(L, s) : launch_one<true, 64, false>(L, s);
  return dual ? launch_one<false, 64, true>(L, s) : launch_one<false, 64, false>(L, s);
}

}  // namespace dfv
