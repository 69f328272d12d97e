// tree_attn_codes.cu -- tree attention over a cache in e4m3 codes, up to 16 rows per
// kv head (mma.sync): half the bytes of a cache in 16 bits.
//
// Mathematics.  Key j is K_j 2^a_j and value j is V_j 2^b_j, K and V being codes and
// a, b the powers of the token and head.  Codes are exact in fp16, so both products
// take them as they are: with x_j = c 2^a_j (q . K_j) in units of log2,
//   o = sum_j 2^(x_j + b_j - M) V_j / sum_j 2^(x_j - M)
// for any M.  M is the running maximum of x_j + b_j, so that the weights
// 2^(x_j + b_j - M) of the second product lie in (0, 1] whatever the powers are, and
// the sum takes them times 2^-b_j.  States of disjoint keys join as in tree_attn.cu.
//
// Precision.  A row of q becomes fp16 times the power of two that puts its largest
// element into [1, 2): bf16 elements down to 2^-17 of it stay exact, smaller ones
// round at 2^-25 of it.  The weights are rounded to fp16 (11 bits, times 2^6 so
// that small ones stay out of its subnormals).  Scores, M, sums and outputs are fp32.
//
// A tile is 16 KB of codes, keys and values: 64 keys of 128 elements or 128 of 64.
// Two producer warps stream the codes with TMA and bring the tile's powers (a byte
// per token and head) along with plain loads, a tile ahead; eight consumer warps in
// two groups take every other tile, in stages of their own.  ldmatrix moves pairs of
// codes: a thread gets four neighbouring codes of a key, two of which are one operand
// register once widened, so the head's elements of both operands are taken in the
// order 4i, 4i+1 | 4i+2, 4i+3.  Of values it gets two neighbouring codes of two
// keys, which a byte permutation sorts into a pair of keys for the even and one for
// the odd element: outputs come as four neighbouring elements.
#include "tc05.cuh"
#include "tree_attn.cuh"

namespace dfv {
namespace {

constexpr int kRows = 16;
constexpr int kProd = 2, kCons = 8, kGroups = 2, kThreads = 32 * (kProd + kCons);
constexpr float kBias = 6.f;

template <int D>
struct CodeShape {
  static constexpr int kKt = 8192 / D;            // keys of a tile
  static constexpr int kStep = kKt / 64;          // 16-key steps of a warp in a tile
  static constexpr uint32_t kTile = kKt * D;      // bytes of one K or V tile
  static constexpr int kStages = 8;               // of K and V: 128 KB in flight
  static constexpr int kPer = kStages / kGroups;  // stages of a group
  static constexpr int kPitch = D + 4;            // floats of a row of a warp's state
  static constexpr int kOver = 6;                 // tiles' worth of time that a pair costs at least
  static constexpr size_t kState = (size_t)kRows * kPitch * 4;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * 2 * (kTile + kKt) + kCons * kState;
};

// Keys of a tile sit in rows of D bytes; 16-byte chunks are XORed with the row's place
// among 1024 (D = 128) or 512 bytes (128- and 64-byte TMA swizzle).
template <int D>
__device__ __forceinline__ uint32_t code_addr(uint32_t base, int row, int chunk) {
  return base + (uint32_t)(row * D) + (uint32_t)((D == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3)) << 4);
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) tree_attn_codes_kernel(const __grid_constant__ AttnLaunch L) {
  using S = CodeShape<D>;
  constexpr int kStages = S::kStages, kKt = S::kKt, kStep = S::kStep;
  extern __shared__ __align__(16) unsigned char sm_raw[];
  unsigned char *sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) unsigned long long s_full[kStages], s_empty[kStages];
  __shared__ volatile int s_abort;
  __shared__ SchedStart s_start;
  __shared__ long long s_scan[kThreads / 32];
  __shared__ float2 s_ml[kCons][kRows];
  __shared__ int s_bad[2];  // of a segment, in turn
  const TreeAttnParams &p = L.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = smem_u32(sm), powers = ring + kStages * 2 * S::kTile;  // [stage][keys, values][kKt]
  unsigned char *s_state = sm + (size_t)kStages * 2 * (S::kTile + kKt);        // [warp][row][kPitch] fp32
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
  sched_start<kThreads, kKt, S::kOver>(L, blockIdx.x, s_scan, &s_start);  // syncs the CTA

  if (warp < kProd) {
    // ---------------------------------------------------------------- producers: warp 0 keys, warp 1 values
    const CUtensorMap *map = warp == 0 ? &L.tm_k : &L.tm_v;
    const uint8_t *exps = warp == 0 ? p.c.ke : p.c.ve;
    int issued[kGroups] = {};  // tiles of each group
    bool ok = true;
    SegWalk<kKt, S::kOver> wk(L, s_start);
    const int shift = p.c.page_shift, boxes = (1 << shift) >= kKt ? 1 : kKt >> shift, rows = kKt / boxes;
    while (ok && wk.next()) {
      const int pages = wk.v.s < 0 ? 0 : (wk.total + (1 << shift) - 1) >> shift;
      const int32_t *table = p.c.table + (size_t)(wk.v.s < 0 ? 0 : wk.v.s) * p.c.max_pages;
      auto page = [&](int t) {  // this lane's page of tile t, or -1 when there is none
        const int at = ((t * kKt) >> shift) + lane;
        return lane < boxes && at < pages ? checked_page(p.c, table[at]) : -1;
      };
      auto power = [&](int t, int pg) {  // powers of this lane's four keys of tile t
        const int mine = __shfl_sync(0xffffffffu, pg, boxes == 1 ? 0 : (4 * lane) >> shift & 31);
        if (4 * lane >= kKt || mine < 0) return 0x7f7f7f7fu;
        return *reinterpret_cast<const uint32_t *>(exps + exp_off(p.c, p.layer, mine, wk.h, (t * kKt + 4 * lane) & ((1 << shift) - 1)));
      };
      int pg = page(wk.t0);
      int pgn = wk.t0 + 1 < wk.t1 ? page(wk.t0 + 1) : -1;
      uint32_t pw = power(wk.t0, pg);
      for (int t = wk.t0; t < wk.t1; ++t) {
        // a tile ahead: the next one's powers; two ahead: page ids
        const uint32_t pwn = power(t + 1, pgn);
        const int pgnn = t + 2 < wk.t1 ? page(t + 2) : -1;
        const int g = (t - wk.t0) & 1, turn = issued[g];
        const int st = g * S::kPer + turn % S::kPer, ph = (turn / S::kPer) & 1;
        ok = __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_empty[st]), ph ^ 1, p.err, DFV_DEVERR_SLOT_WAIT, &s_abort));
        if (!ok) break;
        const uint32_t fb = smem_u32(&s_full[st]), dst = ring + (uint32_t)(2 * st + warp) * S::kTile;
        const int nb = __popc(__ballot_sync(0xffffffffu, pg >= 0));
        if (4 * lane < kKt)
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(powers + (uint32_t)((2 * st + warp) * kKt + 4 * lane)), "r"(pw) : "memory");
        __syncwarp();
        if (lane == 0) {
          if (nb)
            mbar_expect_tx(fb, (uint32_t)nb * rows * D);
          else
            mbar_arrive(fb);
        }
        __syncwarp();
        const int tok = (t * kKt) & ((1 << shift) - 1);  // 0 unless a page holds several tiles
#pragma unroll 2
        for (int b = 0; b < nb; ++b)
          tma_kv(dst + (uint32_t)(b * rows * D), map, 0, tok, wk.h, __shfl_sync(0xffffffffu, pg, b), L.swap, fb);
        ++issued[g];
        pg = pgn;
        pgn = pgnn;
        pw = pwn;
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
  int st = group * S::kPer, ph = 0, turn = 0;
  bool ok = true;
  SegWalk<kKt, S::kOver> wk(L, s_start);
  while (wk.next()) {
    const int R = wk.v.n * p.G;
    // row r = node * G + head of the group; rows past R are zero and see nothing
    uint32_t q[D / 16][4];
    uint64_t mask[2];
    float crow[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int r = hh * 8 + gr, i = node_of(L, r), g = r - i * p.G;
      mask[hh] = 0;
      const uint2 *qp = nullptr;
      if (r < R) {
        mask[hh] = wk.mask_of(r);
        qp = reinterpret_cast<const uint2 *>(p.q + 2 * ((wk.v.row0 + i) * p.q_row + (wk.h * p.G + g) * p.q_head));
      }
      float top = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint2 x = qp ? qp[ks * 4 + qc] : make_uint2(0u, 0u);
        q[ks][hh] = x.x;
        q[ks][2 + hh] = x.y;
        top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16_lo(x.x)), fabsf(bf16_hi(x.x))), fmaxf(fabsf(bf16_lo(x.y)), fabsf(bf16_hi(x.y)))));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // times 2^(127 - exponent), the largest two exponents the same (up to 8 is fine)
      const int f = max(1, 254 - (int)(__float_as_uint(top) >> 23));
      const float up = exp_value((uint32_t)f);
      crow[hh] = p.scale_log2 * exp_value((uint32_t)(254 - f));
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int e = hh; e < 4; e += 2) q[ks][e] = pack2<true>(bf16_lo(q[ks][e]) * up, bf16_hi(q[ks][e]) * up);
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
      const uint32_t kb = ring + (uint32_t)st * 2 * S::kTile, vb = kb + S::kTile, pk = powers + (uint32_t)st * 2 * kKt, pv = pk + kKt;
      const int w0 = cw * 16 * kStep, k0 = t * kKt + w0;  // this warp's first key in the tile, in the sequence
      if (k0 < wk.total) {
        float s[2 * kStep][4];
#pragma unroll
        for (int nt = 0; nt < 2 * kStep; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
          const int row = w0 + 16 * u + ((lane >> 4) << 3) + (lane & 7), ch = (lane >> 3) & 1;
#pragma unroll
          for (int c = 0; c < D / 16; c += 2) {
            uint32_t b[4];
            ldsm4(b, code_addr<D>(kb, row, c + ch));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              mma_f16(s[2 * u], q[c + h][0], q[c + h][1], q[c + h][2], q[c + h][3], codes_f16(b[h]), codes_f16_hi(b[h]));
              mma_f16(s[2 * u + 1], q[c + h][0], q[c + h][1], q[c + h][2], q[c + h][3], codes_f16(b[2 + h]), codes_f16_hi(b[2 + h]));
            }
          }
        }
        const bool special = k0 + 16 * kStep > wk.v.len;  // tree nodes or keys past the end among them
        // x + b in place of the scores, and 2^-b
        float back[2 * kStep][2];
#pragma unroll
        for (int nt = 0; nt < 2 * kStep; ++nt) {
          const uint32_t at = (uint32_t)(w0 + 8 * nt + 2 * qc), ka = lds_u16(pk + at), va = lds_u16(pv + at);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float a = exp_value(ka >> (8 * e) & 255u);
            const uint32_t vb8 = min(va >> (8 * e) & 255u, 253u);  // whatever a masked place holds, 2^-b is finite
            const float bpow = (float)((int)vb8 - 127);
            back[nt][e] = exp_value(254u - vb8);
            s[nt][e] = fmaf(s[nt][e], a * crow[0], bpow);
            s[nt][2 + e] = fmaf(s[nt][2 + e], a * crow[1], bpow);
          }
        }
        if (special) {
#pragma unroll
          for (int nt = 0; nt < 2 * kStep; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = k0 + nt * 8 + 2 * qc + (e & 1) - wk.v.len;  // below 0: committed
              if (j >= 0 && (j >= wk.nodes || !((mask[e >> 1] >> j) & 1))) s[nt][e] = -INFINITY;
            }
        }
        float mn[2];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float x = fmaxf(s[0][2 * hh], s[0][2 * hh + 1]);
#pragma unroll
          for (int nt = 1; nt < 2 * kStep; ++nt) x = fmaxf(x, fmaxf(s[nt][2 * hh], s[nt][2 * hh + 1]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          mn[hh] = fmaxf(m[hh], x);
        }
        if (__any_sync(0xffffffffu, mn[0] > m[0] || mn[1] > m[1])) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            // f = 0 without keys so far: nothing is summed yet
            const float f = m[hh] == -INFINITY ? 0.f : ex2(m[hh] - mn[hh]);
            m[hh] = mn[hh];
            l[hh] *= f;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              o[n][2 * hh] *= f;
              o[n][2 * hh + 1] *= f;
            }
          }
        }
        uint32_t a[kStep][4];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const float z = (m[hh] == -INFINITY ? 0.f : m[hh]) - kBias;
#pragma unroll
          for (int nt = 0; nt < 2 * kStep; ++nt) {
            const float x = ex2(s[nt][2 * hh] - z), y = ex2(s[nt][2 * hh + 1] - z);
            l[hh] = fmaf(x, back[nt][0], fmaf(y, back[nt][1], l[hh]));
            a[nt >> 1][(nt & 1) * 2 + hh] = pack2<true>(x, y);
          }
        }
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
          const int row = w0 + 16 * u + (((lane >> 3) & 1) << 3) + (lane & 7), cc = lane >> 4;
#pragma unroll
          for (int c = 0; c < D / 16; c += 2) {
            uint32_t b[4];
            ldsm4t(b, code_addr<D>(vb, row, c + cc));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t lo = __byte_perm(b[2 * h], 0u, 0x3120), hi = __byte_perm(b[2 * h + 1], 0u, 0x3120);
              uint32_t e0 = codes_f16(lo), e1 = codes_f16(hi), d0 = codes_f16_hi(lo), d1 = codes_f16_hi(hi);
              if (special) {
                // keys past the end count as zero; NaN in a node's value is taken out
                // here and given to the rows that see it at the end
                const int j = k0 + 16 * u + 2 * qc - wk.v.len;
                e0 = clean_pair<true>(e0, j, wk.nodes, &bad);
                d0 = clean_pair<true>(d0, j, wk.nodes, &bad);
                e1 = clean_pair<true>(e1, j + 8, wk.nodes, &bad);
                d1 = clean_pair<true>(d1, j + 8, wk.nodes, &bad);
              }
              mma_f16(o[2 * (c + h)], a[u][0], a[u][1], a[u][2], a[u][3], e0, e1);
              mma_f16(o[2 * (c + h) + 1], a[u][0], a[u][1], a[u][2], a[u][3], d0, d1);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s_empty[st]));
      if (++st == (group + 1) * S::kPer) { st = group * S::kPer; ph ^= 1; }
    }
    // ---- the warps' states, side by side; a thread's outputs are four neighbours of
    // every 16 elements
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
        for (int c = 0; c < D / 16; ++c)
          *reinterpret_cast<float4 *>(mine + r * S::kPitch + c * 16 + 4 * qc) =
              make_float4(o[2 * c][2 * hh], o[2 * c + 1][2 * hh], o[2 * c][2 * hh + 1], o[2 * c + 1][2 * hh + 1]);
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
        const float f = ml.x == -INFINITY ? 1.f : ex2(ml.x - M);
        lsum = fmaf(ml.y, f, lsum);
        const float4 *from = reinterpret_cast<const float4 *>(s_state + w * S::kState) + (r * S::kPitch + e * 8) / 4;
        const float4 a = from[0], b = from[1];
        x[0] = fmaf(a.x, f, x[0]); x[1] = fmaf(a.y, f, x[1]); x[2] = fmaf(a.z, f, x[2]); x[3] = fmaf(a.w, f, x[3]);
        x[4] = fmaf(b.x, f, x[4]); x[5] = fmaf(b.y, f, x[5]); x[6] = fmaf(b.z, f, x[6]); x[7] = fmaf(b.w, f, x[7]);
      }
      const float z = (M == -INFINITY ? 0.f : M) - kBias;
      if (whole) {
        if (r < R) store_out<false>(L, wk.v, r, wk.h, e, x, z, lsum, isbad);
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
    // again after its last one
    if (ct == 0) s_bad[turn ^ 1] = 0;
    bar_sync_n(1, 32 * kCons);  // the states' places are free
    turn ^= 1;
  }
}

template <int D>
cudaError_t launch_one(const AttnLaunch &L, cudaStream_t s) {
  auto kern = tree_attn_codes_kernel<D>;
  const size_t smem = CodeShape<D>::kSmem;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kern, smem, done);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, dim3(L.n_groups * L.n_rt), dim3(kThreads), smem, s, L);
}

}  // namespace

int attn_codes_tile(int D) { return D == 128 ? CodeShape<128>::kKt : CodeShape<64>::kKt; }
cudaError_t launch_attn_codes(const AttnLaunch &L, cudaStream_t s) {
  return L.p.c.D == 128 ? launch_one<128>(L, s) : launch_one<64>(L, s);
}

}  // namespace dfv
