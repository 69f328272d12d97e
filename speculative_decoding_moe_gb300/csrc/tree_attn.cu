// tree_attn.cu -- attention of drafted tree nodes over the paged cache.
//
// Mathematics.  For row (node i, query head of kv head h) and the keys it sees,
// o = sum_j p_j v_j / sum_j p_j with p_j = 2^(c q.k_j - M), c = scale log2(e),
// for any M: M is the running maximum of c q.k_j, so one pass over the keys
// needs only (M, l = sum p, O = sum p v) as state.  Two states over disjoint
// keys join exactly: with M = max(M1, M2) both l and O are weighted by
// 2^(Mi - M).  fp16 caches use M - 6 instead (p up to 64), which keeps small p
// out of fp16's subnormals.
//
// Precision.  Scores, M, l and O are fp32.  p alone is rounded to the cache's 16-bit
// type before it multiplies the values: both operands of a product have one type, and
// p in 32 bits would take the values widened to tf32 (half the rate, twice the bytes
// of a tile) or a second product of what the rounding left.  l sums p before its
// rounding.  An output's error is then a half step of the type for its own rounding
// and, weighted by p |v|, at most another for p: with normal values the outputs'
// error in the 2-norm is 0.0020 to 0.0023 on bf16 caches, where their own rounding
// alone makes 0.0017 (fp16: 0.00028 and 0.00021).
//
// Work split.  The nodes x query heads of one kv head are the rows of one tile,
// so keys and values are read once for all of them.  All (sequence, kv head)
// pairs' key tiles form one line of units that is cut into equal ranges, one
// per CTA (or per group of CTAs when the rows need several): short and long
// sequences, few and many of them, load the SMs alike.  A range that ends
// inside a pair leaves its state (M, l, O) in the workspace, and a second launch
// joins the states in range order (no atomics: the same bits every time).
// The cut depends on the lengths only on the device, so a captured call may be
// replayed after they change.
//
// Kernels, by rows per kv head:
//   up to 16   mma.sync m16n8k16: bound by reading the cache (one token over
//              131071 keys, 8 kv heads of 64: 53 us, 5.0 TB/s; 6.1 TB/s between
//              the first tile and the last)
//   above      tcgen05 on 128-row tiles, scores and outputs in tensor memory
//              (two 16-row tiles of mma.sync took 110 us where it takes 79:
//              32 x 4 nodes of 8 heads over 8191 keys)
// Caches in e4m3 codes have kernels of their own for both (tree_attn_codes.cu,
// tree_attn_codes_tc.cu): the work split and the join are these.
#include <cstdio>
#include <cstring>

#include <cudaTypedefs.h>

#include "tc05.cuh"
#include "tree_attn.cuh"

namespace dfv {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn(char *why, size_t why_len);

namespace {

// ---------------------------------------------------------------- mma.sync kernel
// A CTA is two producer warps (keys and values) and eight consumer warps.  A tile
// is 64 keys, 16 for each of four warps; two groups of four warps take every other
// tile, which hides the chain from one tile's scores to its product.  Each group
// has stages of its own: a parity wait is only sound for a warp that sees every
// phase of a barrier.
constexpr int kKt = 64;
constexpr int kRows = 16;
constexpr int kProd = 2, kCons = 8, kGroups = 2, kMmaThreads = 32 * (kProd + kCons);
template <int D>
struct MmaShape {
  static constexpr uint32_t kTile = kKt * D * 2;           // one K or V tile
  static constexpr int kStages = D == 64 ? 10 : 4;         // of K and V: 160 and 128 KB in flight
  static constexpr int kPer = kStages / kGroups;           // stages of a group
  static constexpr int kPitch = D + 4;                     // floats of a row of a warp's state
  static constexpr int kOver = D == 64 ? 6 : 3;            // tiles' worth of time that a pair costs at least
  static constexpr size_t kState = (size_t)kRows * kPitch * 4;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * 2 * kTile + kCons * kState;
};

// Keys of a tile sit in rows of 128 bytes (64 elements), one block of rows per
// 64 elements of the head, 16-byte chunks XOR row % 8 (128-byte TMA swizzle).
__device__ __forceinline__ uint32_t tile_addr(uint32_t base, int half, int row, int chunk) {
  return base + (uint32_t)(half * kKt * 128 + row * 128) + (uint32_t)((chunk ^ (row & 7)) << 4);
}

template <bool F16>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    mma_f16(c, a[0], a[1], a[2], a[3], b0, b1);
  else
    mma_bf16(c, a[0], a[1], a[2], a[3], b0, b1);
}

template <bool F16, int D>
__global__ void __launch_bounds__(kMmaThreads, 1) tree_attn_mma_kernel(const __grid_constant__ AttnLaunch L) {
  using S = MmaShape<D>;
  constexpr int kStages = S::kStages, kHalves = D / 64;
  constexpr uint32_t kTileBytes = S::kTile;
  extern __shared__ __align__(16) unsigned char sm_raw[];
  unsigned char *sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) unsigned long long s_full[kStages], s_empty[kStages];
  __shared__ volatile int s_abort;
  __shared__ SchedStart s_start;
  __shared__ long long s_scan[kMmaThreads / 32];
  __shared__ float2 s_ml[kCons][kRows];
  __shared__ int s_bad[2];  // of a segment, in turn
  const TreeAttnParams &p = L.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = smem_u32(sm);
  unsigned char *s_state = sm + (size_t)kStages * 2 * kTileBytes;  // [warp][row][kPitch] fp32
  if (tid == 0) {
    s_abort = 0;
    s_bad[0] = s_bad[1] = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&s_full[s]), kProd);
      mbar_init(smem_u32(&s_empty[s]), 4);
    }
    mbar_init_fence();
  }
  pdl_wait();
  pdl_trigger();  // the join may now read the call's inputs
  sched_start<kMmaThreads, kKt, S::kOver>(L, blockIdx.x, s_scan, &s_start);  // syncs the CTA
  const int row0 = (int)(blockIdx.x % L.n_rt) * kRows;  // first row of this CTA

  if (warp < kProd) {
    // ---------------------------------------------------------------- producers: warp 0 keys, warp 1 values
    const CUtensorMap *map = warp == 0 ? &L.tm_k : &L.tm_v;
    int issued[kGroups] = {};  // tiles of each group
    bool ok = true;
    SegWalk<kKt, S::kOver> wk(L, s_start);
    const int shift = p.c.page_shift, boxes = shift >= 6 ? 1 : kKt >> shift, rows = kKt / boxes;
    while (ok && wk.next()) {
      const int pages = wk.v.s < 0 ? 0 : (wk.total + (1 << shift) - 1) >> shift;
      const int32_t *table = p.c.table + (size_t)(wk.v.s < 0 ? 0 : wk.v.s) * p.c.max_pages;
      auto page = [&](int t) {  // this lane's page of tile t, or -1 when there is none
        const int at = ((t * kKt) >> shift) + lane;
        return lane < boxes && at < pages ? checked_page(p.c, table[at]) : -1;
      };
      int pg = page(wk.t0);
      for (int t = wk.t0; t < wk.t1; ++t) {
        const int pgn = t + 1 < wk.t1 ? page(t + 1) : -1;  // the next tile's ids are fetched a tile ahead
        const int g = (t - wk.t0) & 1, turn = issued[g];
        const int st = g * S::kPer + turn % S::kPer, ph = (turn / S::kPer) & 1;
        ok = __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_empty[st]), ph ^ 1, p.err, DFV_DEVERR_SLOT_WAIT, &s_abort));
        if (!ok) break;
        const uint32_t fb = smem_u32(&s_full[st]), dst = ring + (uint32_t)(2 * st + warp) * kTileBytes;
        const int nb = __popc(__ballot_sync(0xffffffffu, pg >= 0));
        if (lane == 0) {
          if (nb)
            mbar_expect_tx(fb, (uint32_t)nb * rows * D * 2);
          else
            mbar_arrive(fb);
        }
        __syncwarp();
        const int tok = (t * kKt) & ((1 << shift) - 1);  // 0 unless a page holds several tiles
#pragma unroll 2
        for (int b = 0; b < nb; ++b) {
          const int pb = __shfl_sync(0xffffffffu, pg, b);
#pragma unroll
          for (int hf = 0; hf < kHalves; ++hf)
            tma_kv(dst + (uint32_t)(hf * kKt * 128 + b * rows * 128), map, hf * 64, tok, wk.h, pb, L.swap, fb);
        }
        ++issued[g];
        pg = pgn;
      }
    }
    // no copy may land after the CTA exits: wait for the last fill of every stage
    volatile int never = 0;
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
      for (int j = issued[g] - S::kPer < 0 ? 0 : issued[g] - S::kPer; j < issued[g]; ++j)
        if (!mbar_wait(smem_u32(&s_full[g * S::kPer + j % S::kPer]), (j / S::kPer) & 1, p.err, DFV_DEVERR_DRAIN_WAIT, &never))
          break;
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int cw = (warp - kProd) & 3, group = (warp - kProd) >> 2, gr = lane >> 2, qc = lane & 3;
  const float c = p.scale_log2;
  int st = group * S::kPer, ph = 0, turn = 0;
  bool ok = true;
  SegWalk<kKt, S::kOver> wk(L, s_start);
  while (wk.next()) {
    const int R = wk.v.n * p.G;
    // row r = node * G + head of the group; rows past R are zero and see nothing
    uint32_t q[D / 16][4];
    uint64_t mask[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int r = row0 + hh * 8 + gr, i = node_of(L, r), g = r - i * p.G;
      mask[hh] = 0;
      const uint32_t *qp = nullptr;
      if (r < R) {
        mask[hh] = wk.mask_of(r);
        qp = reinterpret_cast<const uint32_t *>(p.q + 2 * ((wk.v.row0 + i) * p.q_row + (wk.h * p.G + g) * p.q_head));
      }
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        q[ks][hh] = qp ? qp[ks * 8 + qc] : 0u;
        q[ks][2 + hh] = qp ? qp[ks * 8 + 4 + qc] : 0u;
      }
    }
    float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    bool bad = false;
    for (int t = wk.t0 + group; t < wk.t1; t += kGroups) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_full[st]), ph, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
      if (!ok) break;
      const uint32_t kb = ring + (uint32_t)st * 2 * kTileBytes, vb = kb + kTileBytes;
      const int k0 = t * kKt + cw * 16;  // this warp's 16 keys
      if (k0 < wk.total) {
        float s[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
        {
          const int row = cw * 16 + ((lane >> 4) << 3) + (lane & 7), ch = (lane >> 3) & 1;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t b[4];
            ldsm4(b, tile_addr(kb, ks >> 2, row, (ks & 3) * 2 + ch));
            mma16<F16>(s[0], q[ks], b[0], b[1]);
            mma16<F16>(s[1], q[ks], b[2], b[3]);
          }
        }
        const bool special = k0 + 16 > wk.v.len;  // tree nodes or keys past the end among the 16
        if (special) {
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = k0 + nt * 8 + 2 * qc + (e & 1) - wk.v.len;  // below 0: committed
              if (j >= 0 && (j >= wk.nodes || !((mask[e >> 1] >> j) & 1))) s[nt][e] = -INFINITY;
            }
        }
        float mn[2];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float x = fmaxf(fmaxf(s[0][2 * hh], s[0][2 * hh + 1]), fmaxf(s[1][2 * hh], s[1][2 * hh + 1]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          mn[hh] = fmaxf(m[hh], x);
        }
        if (__any_sync(0xffffffffu, mn[0] > m[0] || mn[1] > m[1])) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            // f = 0 without keys so far: nothing is summed yet
            const float f = m[hh] == -INFINITY ? 0.f : ex2((m[hh] - mn[hh]) * c);
            m[hh] = mn[hh];
            l[hh] *= f;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              o[n][2 * hh] *= f;
              o[n][2 * hh + 1] *= f;
            }
          }
        }
        uint32_t a[4];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const float z = base_of<F16>(m[hh], c);
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const float x = ex2(fmaf(s[nt][2 * hh], c, -z)), y = ex2(fmaf(s[nt][2 * hh + 1], c, -z));
            l[hh] += x + y;
            a[nt * 2 + hh] = pack2<F16>(x, y);
          }
        }
        {
          const int row = cw * 16 + (((lane >> 3) & 1) << 3) + (lane & 7), cc = lane >> 4;
#pragma unroll
          for (int d2 = 0; d2 < D / 16; ++d2) {  // 16 elements of the head at a time
            uint32_t b[4];
            ldsm4t(b, tile_addr(vb, d2 >> 2, row, (d2 & 3) * 2 + cc));
            if (special) {
              // keys past the end count as zero; what is not finite in a node's
              // value is taken out here and given to the rows that see it at the end
#pragma unroll
              for (int e = 0; e < 4; ++e)
                b[e] = clean_pair<F16>(b[e], k0 + (e & 1) * 8 + 2 * qc - wk.v.len, wk.nodes, &bad);
            }
            mma16<F16>(o[2 * d2], a, b[0], b[1]);
            mma16<F16>(o[2 * d2 + 1], a, b[2], b[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s_empty[st]));
      if (++st == (group + 1) * S::kPer) { st = group * S::kPer; ph ^= 1; }
    }
    // ---- the warps' states, side by side
    {
      const int w = warp - kProd;
      float *mine = reinterpret_cast<float *>(s_state + w * S::kState);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int r = hh * 8 + gr;
        float x = l[hh];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (qc == 0) s_ml[w][r] = make_float2(m[hh], x);
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
          *reinterpret_cast<float2 *>(mine + r * S::kPitch + n * 8 + 2 * qc) = make_float2(o[n][2 * hh], o[n][2 * hh + 1]);
      }
    }
    if (bad) s_bad[turn] = 1;
    bar_sync_n(1, 32 * kCons);
    const int isbad = s_bad[turn], ct = tid - 32 * kProd;
    const bool whole = wk.whole();
    const int slot = wk.slot(blockIdx.x);
    // ---- the state of the whole segment: output, or partial state
#pragma unroll 1
    for (int u = ct; u < kRows * (D / 8); u += 32 * kCons) {
      const int r = u % kRows, e = u / kRows;
      float M = -INFINITY, lsum = 0.f, x[8];
#pragma unroll
      for (int w = 0; w < kCons; ++w) M = fmaxf(M, s_ml[w][r].x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.f;
#pragma unroll
      for (int w = 0; w < kCons; ++w) {
        const float2 ml = s_ml[w][r];
        // a warp without keys for the row adds its zeros (or NaN of a NaN query)
        const float f = ml.x == -INFINITY ? 1.f : ex2((ml.x - M) * c);
        lsum = fmaf(ml.y, f, lsum);
        const float4 *from = reinterpret_cast<const float4 *>(s_state + w * S::kState) + (r * S::kPitch + e * 8) / 4;
        const float4 a = from[0], b = from[1];
        x[0] = fmaf(a.x, f, x[0]); x[1] = fmaf(a.y, f, x[1]); x[2] = fmaf(a.z, f, x[2]); x[3] = fmaf(a.w, f, x[3]);
        x[4] = fmaf(b.x, f, x[4]); x[5] = fmaf(b.y, f, x[5]); x[6] = fmaf(b.z, f, x[6]); x[7] = fmaf(b.w, f, x[7]);
      }
      const float z = base_of<F16>(M, c);
      if (whole) {
        if (row0 + r < R) store_out<F16>(L, wk.v, row0 + r, wk.h, e, x, z, lsum, isbad);
      } else {
        float4 *to = reinterpret_cast<float4 *>(L.part_o) + ((size_t)slot * (D / 4) + 2 * e) * L.rows + r;
        to[0] = make_float4(x[0], x[1], x[2], x[3]);
        to[L.rows] = make_float4(x[4], x[5], x[6], x[7]);
        if (e == 0) {
          L.part_ml[(size_t)slot * L.rows + r] = make_float2(M == -INFINITY ? -INFINITY : z, lsum);
          if (r == 0) L.part_bad[slot] = isbad;
        }
      }
    }
    if (ct == 0) wk.tell(s_start, blockIdx.x);
    // the next segment's flag: last read before this segment's first barrier, set
    // again after its last one.  (Its own flag cleared after the last barrier could
    // take back what a warp of the other group, a segment ahead, had set.)
    if (ct == 0) s_bad[turn ^ 1] = 0;
    bar_sync_n(1, 32 * kCons);  // the states' places are free
    turn ^= 1;
  }
}

// ---------------------------------------------------------------- join
// Rows of pairs whose units were cut: the states of their ranges, in order.
// Pairs done by one range were stored by it.  A CTA takes eight rows and CH
// blocks of 16 head elements; its eight warps are those blocks times a split of
// the states.  Many rows of few states: all blocks, no split; few rows of many
// states: one block and eight parts, because then the latency of reading the
// states one after the other is what counts.  A lane holds four elements of a
// row, so that a warp's 16-byte reads cover eight rows side by side (the order
// the states are stored in: the kernels' threads hold a row each).
constexpr int kJoinWarps = 8;
constexpr int kJoinRows = 8;
constexpr int kJoinStates = (kAttnCtas + 31) / 32;

template <bool F16, int D, int CH>
__global__ void __launch_bounds__(32 * kJoinWarps, CH == 1 ? 3 : 6) tree_attn_join_kernel(const __grid_constant__ AttnLaunch L) {
  constexpr int kBlocks = D / 16, kSplit = kJoinWarps / CH, kAhead = CH == 1 ? 8 : 4;  // states of a warp in flight
  __shared__ float s_w[kAttnCtas][kJoinRows], s_max[kJoinWarps][kJoinRows], s_l[kJoinWarps][kJoinRows];
  __shared__ float4 s_x[kSplit > 1 ? kJoinWarps : 1][32];
  pdl_trigger();
  const TreeAttnParams &p = L.p;
  const int b = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r0 = (int)blockIdx.z / (kBlocks / CH) * kJoinRows, r8 = lane & 7, cg = lane >> 3, r = r0 + r8;
  // the first launch releases this one after its own wait: the call's inputs are final
  const SeqView v = seq_view(p.c, p.t, b);
  const int R = v.n * p.G;
  pdl_wait();  // by every CTA: what follows this launch may rely on the first one's end
  if (r0 >= R) return;
  const int2 pair = __ldcg(&L.pairs[b * p.c.Hkv + h]);
  const int g0 = pair.x, n = pair.y;
  if (n < 2) return;
  const int rt = r0 / L.rows, rr = r - rt * L.rows;
  // state k is range g0 + k's; the pair goes on after the first and began before the others
  auto slot = [&](int k) { return (size_t)(2 * ((g0 + k) * L.n_rt + rt) + (k == 0)); };
  // ---- the first sums of p v, on their way while the weights are found
  const int part = warp % kSplit, c4 = ((int)blockIdx.z % (kBlocks / CH) * CH + warp / kSplit) * 4 + cg;
  const float4 *base = reinterpret_cast<const float4 *>(L.part_o) + (size_t)c4 * L.rows + rr;
  const size_t pitch = (size_t)(D / 4) * L.rows;
  float4 y[kAhead];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (k0 + i * kSplit < n && r < R) y[i] = __ldcg(base + slot(k0 + i * kSplit) * pitch);
  };
  fetch(part);
  // ---- weights of the states, and the sum
  float2 ml[kJoinStates];
  int bad = 0;
  float M = -INFINITY, l = 0.f;
#pragma unroll
  for (int q = 0; q < kJoinStates; ++q) {
    const int k = warp * 4 + cg + 32 * q;
    ml[q] = make_float2(-INFINITY, 0.f);
    if (k < n && r < R) {
      ml[q] = __ldcg(&L.part_ml[slot(k) * L.rows + rr]);
      bad |= __ldcg(&L.part_bad[slot(k)]);
    }
    M = fmaxf(M, ml[q].x);
  }
  M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 8));
  M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
  if (cg == 0) s_max[warp][r8] = M;
  bad = __syncthreads_or(bad);
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, s_max[w][r8]);
#pragma unroll
  for (int q = 0; q < kJoinStates; ++q) {
    const int k = warp * 4 + cg + 32 * q;
    const float w = ml[q].x == -INFINITY ? 1.f : ex2(ml[q].x - M);  // a state without keys holds zeros (or NaN of a NaN query)
    l += ml[q].y * w;
    if (k < n) s_w[k][r8] = w;
  }
  l += __shfl_xor_sync(0xffffffffu, l, 8);
  l += __shfl_xor_sync(0xffffffffu, l, 16);
  if (cg == 0) s_l[warp][r8] = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) l += s_l[w][r8];
  // ---- sums of p v
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r < R) {
    for (int k0 = part; k0 < n; k0 += kAhead * kSplit) {
      if (k0 != part) fetch(k0);
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (k0 + i * kSplit < n) {
          const float f = s_w[k0 + i * kSplit][r8];
          x.x = fmaf(y[i].x, f, x.x);
          x.y = fmaf(y[i].y, f, x.y);
          x.z = fmaf(y[i].z, f, x.z);
          x.w = fmaf(y[i].w, f, x.w);
        }
    }
  }
  if (kSplit > 1) {
    s_x[warp % kJoinWarps][lane] = x;
    __syncthreads();
    if (part) return;
#pragma unroll
    for (int k = 1; k < kSplit; ++k) {
      const float4 y = s_x[(warp + k) % kJoinWarps][lane];
      x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
    }
  }
  if (r >= R) return;
  const int i = node_of(L, r), head = h * p.G + r - i * p.G;
  const size_t row = v.row0 + i;
  const float inv = l == 0.f ? 0.f : 1.f / l;  // NaN stays NaN
  char *out = p.o + 2 * (row * p.o_row + head * p.o_head);
  *reinterpret_cast<uint2 *>(out + 8 * c4) = make_uint2(pack2<F16>(x.x * inv, x.y * inv), pack2<F16>(x.z * inv, x.w * inv));
  if (bad) add_unseen<F16>(p, v, i, h, out, 4 * c4, 4 * c4 + 4);
  if (p.lse && c4 == 0)
    p.lse[row * p.H + head] = l == 0.f ? -INFINITY : (M == -INFINITY ? l : (M + log2f(l)) * 0.69314718055994531f);
}

bool encode_kv(CUtensorMap *map, const CacheParams &c, const char *base, int layer, int rows, int swap, char *why,
               size_t why_len) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn(why, why_len);
  if (!fn) return false;
  // a dimension of one entry has no stride of its own
  const cuuint64_t one = 16;
  const cuuint64_t tok[2] = {(cuuint64_t)1 << c.page_shift, (cuuint64_t)c.st << c.esh};
  const cuuint64_t head[2] = {(cuuint64_t)c.Hkv, c.Hkv > 1 ? (cuuint64_t)c.sh << c.esh : one};
  const cuuint64_t page[2] = {(cuuint64_t)c.n_pages, c.n_pages > 1 ? (cuuint64_t)c.sp << c.esh : one};
  const cuuint64_t *a = swap ? head : tok, *b = swap ? tok : head;
  const cuuint64_t dims[4] = {(cuuint64_t)c.D, a[0], b[0], page[0]};
  const cuuint64_t strides[3] = {a[1], b[1], page[1]};
  // 64 elements of 16 bits, or the whole head of codes: rows of 128 bytes, or of 64
  const bool codes = c.esh == 0;
  const cuuint32_t box[4] = {codes ? (cuuint32_t)c.D : 64u, swap ? 1u : (cuuint32_t)rows, swap ? (cuuint32_t)rows : 1u, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : c.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                        const_cast<char *>(base + (layer * c.sl << c.esh)), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, codes && c.D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    snprintf(why, why_len, "tensor map of the cache refused (%d)", (int)r);
    return false;
  }
  return true;
}

template <bool F16, int D>
cudaError_t launch_mma(const AttnLaunch &L, cudaStream_t s) {
  auto kern = tree_attn_mma_kernel<F16, D>;
  const size_t smem = MmaShape<D>::kSmem;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kern, smem, done);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, dim3(L.n_groups * L.n_rt), dim3(kMmaThreads), smem, s, L);
}

template <bool F16, int D>
cudaError_t launch_typed(AttnLaunch &L, cudaStream_t s) {
  const int R = L.p.t.max_nodes * L.p.G;
  const bool codes = L.p.c.esh == 0;
  cudaError_t e = L.rows >= 128 ? (codes ? launch_attn_codes_tc(L, s) : launch_attn_tc(L, s))
                                : (codes ? launch_attn_codes(L, s) : launch_mma<F16, D>(L, s));
  if (e != cudaSuccess) return e;
  const int blocks = (R + kJoinRows - 1) / kJoinRows;
  // CTAs of eight rows fill the SMs from about 4000 rows on
  if ((long long)L.p.t.n_seqs * L.p.c.Hkv * R < 4096)
    return launch_chained(tree_attn_join_kernel<F16, D, 1>, dim3(L.p.t.n_seqs, L.p.c.Hkv, blocks * (D / 16)),
                          dim3(32 * kJoinWarps), 0, s, L);
  return launch_chained(tree_attn_join_kernel<F16, D, D / 16>, dim3(L.p.t.n_seqs, L.p.c.Hkv, blocks),
                        dim3(32 * kJoinWarps), 0, s, L);
}

}  // namespace

AttnPlan tree_attn_plan(int max_nodes, int G) {
  AttnPlan a = {};
  const int R = max_nodes * G;
  a.rows = R <= kRows ? kRows : R <= 128 ? 128 : 256;
  a.n_rt = (R + a.rows - 1) / a.rows;
  a.n_groups = kAttnCtas / a.n_rt < 1 ? 1 : kAttnCtas / a.n_rt;
  return a;
}

size_t tree_attn_ws(const AttnPlan &a, int n_seqs, int Hkv, int D) {
  return attn_sections(nullptr, a, n_seqs, Hkv, D, nullptr);
}

cudaError_t launch_tree_attn(const TreeAttnParams &p, const AttnPlan &a, void *ws, cudaStream_t s, char *why,
                             size_t why_len) {
  static thread_local AttnLaunch L;
  L.p = p;
  L.rows = a.rows;
  L.n_rt = a.n_rt;
  L.n_groups = a.n_groups;
  L.inv_g = (65536u + p.G - 1) / p.G;
  attn_sections(&L, a, p.t.n_seqs, p.c.Hkv, p.c.D, ws);
  const int tile = L.rows >= 128 ? 128 : p.c.esh == 0 ? attn_codes_tile(p.c.D) : kKt, page = 1 << p.c.page_shift, rows = page < tile ? page : tile;
  L.swap = p.c.Hkv > 1 && p.c.sh < p.c.st;
  if (!encode_kv(&L.tm_k, p.c, p.c.k, p.layer, rows, L.swap, why, why_len) ||
      !encode_kv(&L.tm_v, p.c, p.c.v, p.layer, rows, L.swap, why, why_len))
    return cudaErrorInvalidValue;
  if (p.c.D == 128) return p.c.f16 ? launch_typed<true, 128>(L, s) : launch_typed<false, 128>(L, s);
  return p.c.f16 ? launch_typed<true, 64>(L, s) : launch_typed<false, 64>(L, s);
}

}  // namespace dfv
