// tree_attn_codes.cu -- tree attention over a cache in e4m3 codes, up to 16 rows per
// kv head (mma.sync): half the bytes of a cache in 16 bits.
//
// Mathematics.  Key j is K_j 2^a_j and value j is V_j 2^b_j, K and V being codes and
// a, b the powers of the token and head.  Codes are exact in fp16, so both products
// take them as they are: with x_j = c 2^a_j (q . K_j) in units of log2,
//   o = sum_j 2^(x_j + b_j - M) V_j / sum_j 2^(x_j - M)
// for any M.  M follows the maximum of x_j + b_j, so that the weights
// 2^(x_j + b_j - M) of the second product fit fp16 whatever the powers are, and the
// sum takes them times 2^-b_j.  A row's M is only raised, and O only rescaled, when some
// x_j + b_j of the row is more than 8 above it.  States of disjoint keys join as in
// tree_attn.cu.
//
// Precision.  A row of q becomes fp16 times the power of two that puts its largest
// element into [1, 2): bf16 elements down to 2^-17 of it stay exact, smaller ones
// round at 2^-25 of it.  The weights are rounded to fp16 (11 bits, times 2^6 so
// that small ones stay out of its subnormals).  Scores, M, sums and outputs are fp32.  The
// sum is relative to the largest x + b: where values' powers are 2^110 and more apart, keys
// of less than 2^-20 of the weight of others can drop out of it.
//
// Next to reading the cache, issuing binds: each code is widened once, in registers,
// and every instruction per code counts.  So keys and the head's elements are the M side of
// the products (S^T = K Q^T, O^T = V^T P^T) and the rows are their N side of 8 or 16:
// a token of a model with up to 8 query heads per kv head takes half the products
// and half the exponentials that 16 rows on the M side would.  ldmatrix moves pairs
// of codes: of a key a thread gets four neighbouring codes, two of which are one
// operand register once widened, so the head's elements of both operands are taken
// in the order 4i, 4i+1 | 4i+2, 4i+3.  Of values it gets two neighbouring codes of
// two keys, which a byte permutation sorts into one register for the even and one
// for the odd element.  P^T is turned with movmatrix.
//
// A stage is a tile of keys and values: 64 keys of 128 elements or 128 of 64.  Four
// producer warps stream the codes with TMA and the tile's powers (a byte per token
// and head) with four-byte asynchronous copies that count on the same barrier; eight
// consumer warps in groups take tiles in turn, in stages of their own.
//
// Measured: one token over 131071 keys of 8 x 64 elements 31 us, 64 tokens over up to
// 8191 keys of 4 x 128 81 us (5.1 TB/s with start and join; without the consumers'
// work 77, without the loads 67).  Steps on the way, of the second: 16 rows on the M
// side with powers loaded through registers 154 us; asynchronous copies 146; rows on
// the N side and a rarely raised M 135; page ids 32 at a time, and several sums of a
// score 110; four producers in place of two 81 (one issues a box in about 100 ns).
#include "tc05.cuh"
#include "tree_attn.cuh"

namespace dfv {
namespace {

constexpr int kProd = 4, kCons = 8, kThreads = 32 * (kProd + kCons);

template <int D, int NT>  // NT blocks of 8 rows
struct CodeShape {
  static constexpr int kRows = 8 * NT;
  static constexpr int kKt = 8192 / D;              // keys of a tile
  static constexpr int kStep = 2;                   // 16-key steps of a warp in a tile
  static constexpr int kWarps = kKt / 16 / kStep;   // of a tile
  static constexpr int kGroups = kCons / kWarps;
  static constexpr uint32_t kTile = kKt * D;        // bytes of one K or V tile
  static constexpr int kStages = 8;                 // of K and V: 128 KB in flight
  static constexpr int kPer = kStages / kGroups;    // stages of a group
  static constexpr int kPitch = D + 4;              // floats of a row of a warp's state
  static constexpr int kOver = 8;                   // tiles' worth of time that a pair costs at least
  static constexpr size_t kState = (size_t)kRows * kPitch * 4;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * 2 * (kTile + kKt) + kCons * kState;
};

// Keys of a tile sit in rows of D bytes; 16-byte chunks are XORed with the row's place
// among 1024 (D = 128) or 512 bytes (128- and 64-byte TMA swizzle).
template <int D>
__device__ __forceinline__ uint32_t code_addr(uint32_t base, int row, int chunk) {
  return base + (uint32_t)(row * D) + (uint32_t)((D == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3)) << 4);
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t turn8(uint32_t x) {  // an 8 x 8 matrix of 16-bit elements, transposed
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Value rows w0 .. w0 + N of a tile, the first of which is node j0 (below 0: committed):
// codes zeroed past the last node, with powers of 1; NaN in a node's codes becomes
// zero and is told of.  Each warp cleans what it alone reads.
template <int D, int N>
__device__ __noinline__ bool clean_codes(uint32_t vb, uint32_t pv, int w0, int j0, int nodes) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
#pragma unroll 1
  for (int u = lane; u < N * (D / 16); u += 32) {
    const int row = u / (D / 16), c = u % (D / 16), j = j0 + row;
    if (j < 0) continue;
    const uint32_t at = code_addr<D>(vb, w0 + row, c);
    uint32_t x[4];
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // a byte of 0x7f but for its sign: NaN
      uint32_t nan = ((x[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
      bad = bad || (nan && j < nodes);
      nan = (nan >> 7) * 255u;
      x[e] = j < nodes ? x[e] & ~nan : 0u;
    }
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
    if (c == 0 && j >= nodes) asm volatile("st.shared.u8 [%0], %1;" ::"r"(pv + (uint32_t)(w0 + row)), "r"(127u) : "memory");
  }
  // before a copy takes the stage again
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  return bad;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1) tree_attn_codes_kernel(const __grid_constant__ AttnLaunch L) {
  using S = CodeShape<D, NT>;
  static_assert(S::kGroups % 2 == 0 && kProd == 4, "a stage is filled by one pair of producers: they see all its phases");
  constexpr int kStages = S::kStages, kKt = S::kKt, kStep = S::kStep, kGroups = S::kGroups, kRows = S::kRows;
  extern __shared__ __align__(16) unsigned char sm_raw[];
  unsigned char *sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) unsigned long long s_full[kStages], s_empty[kStages];
  __shared__ volatile int s_abort;
  __shared__ SchedStart s_start;
  __shared__ long long s_scan[kThreads / 32];
  __shared__ float2 s_ml[kCons][16];
  __shared__ int s_bad[2];  // of a segment, in turn
  const TreeAttnParams &p = L.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = smem_u32(sm), powers = ring + kStages * 2 * S::kTile;  // [stage][keys, values][kKt]
  unsigned char *s_state = sm + (size_t)kStages * 2 * (S::kTile + kKt);        // [warp][row][kPitch] fp32
  if (tid == 0) {
    s_abort = 0;
    s_bad[0] = s_bad[1] = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&s_full[s]), 2 * 33);  // keys' and values' producer: its codes, and its lanes' powers
      mbar_init(smem_u32(&s_empty[s]), S::kWarps);
    }
    mbar_init_fence();
  }
  pdl_wait();
  pdl_trigger();  // the join may now read the call's inputs
  sched_start<kThreads, kKt, S::kOver>(L, blockIdx.x, s_scan, &s_start);  // syncs the CTA

  if (warp < kProd) {
    // ---------------------------------------------------------------- producers: even warps keys, odd ones values, of
    // every other tile
    const int side = warp & 1, me = warp >> 1;
    const CUtensorMap *map = side == 0 ? &L.tm_k : &L.tm_v;
    const uint8_t *exps = side == 0 ? p.c.ke : p.c.ve;
    int issued[kGroups] = {};  // tiles of each group in the segments before
    bool ok = true;
    SegWalk<kKt, S::kOver> wk(L, s_start);
    const int shift = p.c.page_shift, boxes = (1 << shift) >= kKt ? 1 : kKt >> shift, rows = kKt / boxes;
    while (ok && wk.next()) {
      const int pages = wk.v.s < 0 ? 0 : (wk.total + (1 << shift) - 1) >> shift;
      const int32_t *table = p.c.table + (size_t)(wk.v.s < 0 ? 0 : wk.v.s) * p.c.max_pages;
      // page ids a warp's worth at a time, the next ones on their way: one load per 32
      // pages, whose latency a tile would not cover
      auto ids = [&](int first) { return first + lane < pages ? table[first + lane] : 0; };
      int base = (((wk.t0 + me) * kKt) >> shift) & ~31;
      int cur = ids(base), ahead = ids(base + 32);
      if (base + lane < pages) cur = checked_page(p.c, cur);
      for (int t = wk.t0 + me; t < wk.t1; t += kProd / 2) {
        const int first = (t * kKt) >> shift;  // a tile's pages are within one such lot: their number divides 32
        if (first >= base + 32) {  // two tiles have 32 pages at most
          base += 32;
          cur = base + lane < pages ? checked_page(p.c, ahead) : 0;
          ahead = ids(base + 32);
        }
        const int g = (t - wk.t0) % kGroups;
        int turn = (t - wk.t0) / kGroups;
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
          if (i == g) turn += issued[i];
        const int st = g * S::kPer + turn % S::kPer, ph = (turn / S::kPer) & 1;
        ok = __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_empty[st]), ph ^ 1, p.err, DFV_DEVERR_SLOT_WAIT, &s_abort));
        if (!ok) break;
        const uint32_t fb = smem_u32(&s_full[st]), dst = ring + (uint32_t)(2 * st + side) * S::kTile;
        const int nb = min(boxes, pages - first), at = first & 31;
        if (lane == 0) {
          if (nb > 0)
            mbar_expect_tx(fb, (uint32_t)nb * rows * D);
          else
            mbar_arrive(fb);
        }
        __syncwarp();
        const int tok = (t * kKt) & ((1 << shift) - 1);  // 0 unless a page holds several tiles
        // this lane's four keys' powers (without a page they are not looked at)
        const int my = boxes == 1 ? 0 : (4 * lane) >> shift, mine = __shfl_sync(0xffffffffu, cur, (at + my) & 31);
        if (4 * lane < kKt && my < nb)
          cp_async4(powers + (uint32_t)((2 * st + side) * kKt + 4 * lane),
                    exps + exp_off(p.c, p.layer, mine, wk.h, (t * kKt + 4 * lane) & ((1 << shift) - 1)));
        cp_async_arrive(fb);
#pragma unroll 2
        for (int b = 0; b < nb; ++b)
          tma_kv(dst + (uint32_t)(b * rows * D), map, 0, tok, wk.h, __shfl_sync(0xffffffffu, cur, at + b), L.swap, fb);
      }
#pragma unroll
      for (int i = 0; i < kGroups; ++i) issued[i] += (wk.t1 - wk.t0 - i + kGroups - 1) / kGroups;
    }
    // no copy may land after the CTA exits: wait for the last fill of every stage (after
    // a wait gave up fewer were made, and these waits give up too)
    volatile int never = 0;
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
      for (int j = g % 2 != me ? issued[g] : issued[g] - S::kPer < 0 ? 0 : issued[g] - S::kPer; j < issued[g]; ++j)
        if (!mbar_wait(smem_u32(&s_full[g * S::kPer + j % S::kPer]), (j / S::kPer) & 1, p.err, DFV_DEVERR_DRAIN_WAIT, &never))
          break;
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int cw = (warp - kProd) % S::kWarps, group = (warp - kProd) / S::kWarps, gr = lane >> 2, qc = lane & 3;
  int st = group * S::kPer, ph = 0, turn = 0;
  bool ok = true;
  SegWalk<kKt, S::kOver> wk(L, s_start);
  while (wk.next()) {
    const int R = wk.v.n * p.G;
    // row r = node * G + head of the group; rows past R are zero and see nothing.  As an
    // operand a thread has row 8 n + gr, of the scores rows 8 n + 2 qc and the next.
    uint32_t q[NT][D / 16][2];
    uint64_t mask[NT][2];
    float crow[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = 8 * n + gr, i = node_of(L, r), g = r - i * p.G;
      const uint2 *qp = r < R ? reinterpret_cast<const uint2 *>(p.q + 2 * ((wk.v.row0 + i) * p.q_row + (wk.h * p.G + g) * p.q_head)) : nullptr;
      float top = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint2 x = qp ? qp[ks * 4 + qc] : make_uint2(0u, 0u);
        q[n][ks][0] = x.x;
        q[n][ks][1] = x.y;
        top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16_lo(x.x)), fabsf(bf16_hi(x.x))), fmaxf(fabsf(bf16_lo(x.y)), fabsf(bf16_hi(x.y)))));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // times 2^(127 - exponent), the largest two exponents the same (up to 8 is fine)
      const int f = max(1, 254 - (int)(__float_as_uint(top) >> 23));
      const float up = exp_value((uint32_t)f), down = p.scale_log2 * exp_value((uint32_t)(254 - f));
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e) q[n][ks][e] = pack2<true>(bf16_lo(q[n][ks][e]) * up, bf16_hi(q[n][ks][e]) * up);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int s = 8 * n + 2 * qc + e;
        crow[n][e] = __shfl_sync(0xffffffffu, down, 4 * (2 * qc + e));
        mask[n][e] = s < R ? wk.mask_of(s) : 0;
      }
    }
    float o[NT][D / 16][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][c][e] = 0.f;
    }
    bool bad = false;
    for (int t = wk.t0 + group; t < wk.t1; t += kGroups) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_full[st]), ph, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
      if (!ok) break;
      const uint32_t kb = ring + (uint32_t)st * 2 * S::kTile, vb = kb + S::kTile, pk = powers + (uint32_t)st * 2 * kKt, pv = pk + kKt;
      const int w0 = cw * 16 * kStep, k0 = t * kKt + w0;  // this warp's first key in the tile, in the sequence
      if (k0 < wk.total) {
        const bool special = k0 + 16 * kStep > wk.v.len;  // tree nodes or keys past the end among them
        if (special) bad |= clean_codes<D, 16 * kStep>(vb, pv, w0, k0 - wk.v.len, wk.nodes);
        // ---- scores of key 16 u + gr + 8 e / 2 against row 8 n + 2 qc + e % 2
        // (several sums at a time: a product waits for the one before it into the same)
        float s[kStep][NT][4], s1[kStep][NT][4];
#pragma unroll
        for (int u = 0; u < kStep; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[u][n][e] = s1[u][n][e] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; c += 2) {
          uint32_t b[kStep][4];
#pragma unroll
          for (int u = 0; u < kStep; ++u) ldsm4(b[u], code_addr<D>(kb, w0 + 16 * u + (lane & 15), c + (lane >> 4)));
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int u = 0; u < kStep; ++u) {
              const uint32_t *x = b[u] + 2 * h;
              const uint32_t a0 = codes_f16(x[0]), a1 = codes_f16(x[1]), a2 = codes_f16_hi(x[0]), a3 = codes_f16_hi(x[1]);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_f16(h ? s1[u][n] : s[u][n], a0, a1, a2, a3, q[n][c + h][0], q[n][c + h][1]);
            }
        }
#pragma unroll
        for (int u = 0; u < kStep; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[u][n][e] += s1[u][n][e];
        // ---- x + b in their place; 2^-b
        float back[kStep][2];
#pragma unroll
        for (int u = 0; u < kStep; ++u)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t at = (uint32_t)(w0 + 16 * u + 8 * e + gr), pb = lds_u8(pv + at);
            const float a = exp_value(lds_u8(pk + at)), b = __uint_as_float(0x4b000000u | pb) - 8388735.f;  // pb - 127
            back[u][e] = exp_value(254u - pb);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              s[u][n][2 * e] = fmaf(s[u][n][2 * e], a * crow[n][0], b);
              s[u][n][2 * e + 1] = fmaf(s[u][n][2 * e + 1], a * crow[n][1], b);
            }
          }
        if (special) {
#pragma unroll
          for (int u = 0; u < kStep; ++u)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int j = k0 + 16 * u + 8 * (e >> 1) + gr - wk.v.len;  // below 0: committed
                if (j >= 0 && (j >= wk.nodes || !((mask[n][e & 1] >> j) & 1))) s[u][n][e] = -INFINITY;
              }
        }
        bool grew = false;
        float top[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(s[0][n][e], s[0][n][2 + e]);
#pragma unroll
            for (int u = 1; u < kStep; ++u) x = fmaxf(x, fmaxf(s[u][n][e], s[u][n][2 + e]));
            top[n][e] = x;
            grew = grew || x - 8.f > m[n][e];
          }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = fmaxf(m[n][e], top[n][e]);
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
              // a row's M follows what the row sees, not its neighbours; f = 0 without keys so
              // far: nothing is summed yet
              const bool rise = x - 8.f > m[n][e];
              const float f = !rise ? 1.f : m[n][e] == -INFINITY ? 0.f : ex2(m[n][e] - x);
              if (rise) m[n][e] = x;
              l[n][e] *= f;
#pragma unroll
              for (int c = 0; c < D / 16; ++c) {
                o[n][c][e] *= f;
                o[n][c][2 + e] *= f;
              }
            }
        }
        uint32_t pt[kStep][NT][2];  // P^T of keys 16 u + 8 i + 2 qc, + 1 and row 8 n + gr
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float z0 = base_of<true>(m[n][0], 1.f), z1 = base_of<true>(m[n][1], 1.f);
#pragma unroll
          for (int u = 0; u < kStep; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float x = ex2(s[u][n][2 * i] - z0), y = ex2(s[u][n][2 * i + 1] - z1);
              l[n][0] = fmaf(x, back[u][i], l[n][0]);
              l[n][1] = fmaf(y, back[u][i], l[n][1]);
              pt[u][n][i] = turn8(pack2<true>(x, y));
            }
        }
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
          const int row = w0 + 16 * u + (lane & 15), ch = lane >> 4;
#pragma unroll
          for (int c = 0; c < D / 16; c += 2) {
            uint32_t b[4];
            ldsm4t(b, code_addr<D>(vb, row, c + ch));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t lo = __byte_perm(b[2 * h], 0u, 0x3120), hi = __byte_perm(b[2 * h + 1], 0u, 0x3120);
              const uint32_t a0 = codes_f16(lo), a1 = codes_f16_hi(lo), a2 = codes_f16(hi), a3 = codes_f16_hi(hi);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_f16(o[n][c + h], a0, a1, a2, a3, pt[u][n][0], pt[u][n][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s_empty[st]));
      if (++st == (group + 1) * S::kPer) { st = group * S::kPer; ph ^= 1; }
    }
    // ---- the warps' states, side by side: a thread has elements 16 c + 2 gr and the next
    {
      const int w = warp - kProd;
      float *mine = reinterpret_cast<float *>(s_state + w * S::kState);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * n + 2 * qc + e;
          float x = l[n][e];
          x += __shfl_xor_sync(0xffffffffu, x, 4);
          x += __shfl_xor_sync(0xffffffffu, x, 8);
          x += __shfl_xor_sync(0xffffffffu, x, 16);
          if (gr == 0) s_ml[w][r] = make_float2(m[n][e], x);
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
            *reinterpret_cast<float2 *>(mine + r * S::kPitch + c * 16 + 2 * gr) = make_float2(o[n][c][e], o[n][c][2 + e]);
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
      const float z = base_of<true>(M, 1.f);
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

template <int D, int NT>
cudaError_t launch_one(const AttnLaunch &L, cudaStream_t s) {
  auto kern = tree_attn_codes_kernel<D, NT>;
  const size_t smem = CodeShape<D, NT>::kSmem;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kern, smem, done);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, dim3(L.n_groups * L.n_rt), dim3(kThreads), smem, s, L);
}

}  // namespace

int attn_codes_tile(int D) { return D == 128 ? CodeShape<128, 1>::kKt : CodeShape<64, 1>::kKt; }
cudaError_t launch_attn_codes(const AttnLaunch &L, cudaStream_t s) {
  const bool few = L.p.t.max_nodes * L.p.G <= 8;
  if (L.p.c.D == 128) return few ? launch_one<128, 1>(L, s) : launch_one<128, 2>(L, s);
  return few ? launch_one<64, 1>(L, s) : launch_one<64, 2>(L, s);
}

}  // namespace dfv
