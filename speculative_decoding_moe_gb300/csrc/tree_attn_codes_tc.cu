// tree_attn_codes_tc.cu -- tree attention over a cache in e4m3 codes with many rows
// per kv head, on the fifth-generation tensor cores.
//
// As in tree_attn_tc.cu a CTA takes 128 rows (SINGLE) or 256 rows (DUAL) of one kv
// head and streams the keys in tiles of 128.  DUAL: a warpgroup takes 128 rows.
// SINGLE: a warpgroup takes the first or the second 64 keys of every tile, with its own
// (M, l, O); scores take turns in two places, so that the next tile's are ready while
// one is in its exponentials; the two states are joined at the end.  Between the copies
// and the products, four warps widen the codes of K and four those of V into fp16 in
// shared memory, a key row a thread, each in rings of their own.
//
// Mathematics.  Key j is K_j 2^a_j, value j is V_j 2^b_j.  With A and B the largest a
// and b of a tile of 128 keys, the products take K_j 2^(a_j - A) and V_j 2^(b_j - B) in
// fp16, exact for tokens within 2^15 of the tile's largest power.  A and B are then
// constants of the tile: scores are x_j = c 2^A s_j, the weights 2^(x_j + B - M), and
// the sum takes a tile's weights times 2^-B.  M follows the maximum of x_j + B; it is
// raised, and O rescaled, when some x_j + B is more than 8 above it.  Precision of q and
// of the weights as in tree_attn_codes.cu.
//
// A tile has no such constants where its powers are further apart (a beyond 2^15, b
// beyond 2^8: M would follow a value that has no weight, and the weights of others would
// round among fp16's subnormals), or where there are nodes in it: what a row does not see may
// be of any size and must not touch the row.  Its products take the codes as they are,
// and a key's powers come in behind the mask, x_j = c 2^a_j s_j and weights
// 2^(x_j + b_j - M), as in tree_attn_codes.cu.  A row's M is raised by what the row sees
// alone, though the warp's other rows then take part in the rescaling of O.
//
// A tile's maximum is found in one pass over its scores, 16 at a time, and p in another:
// with 20 warps a thread has 96 registers.
//
// What binds: shared memory, then the chain from a tile's copy to its product.  Per tile
// of 128 keys of 128 elements the codes are written (256 clocks at 128 bytes), read and
// written as fp16 (768), and read by the products (768 a row tile), beside 1024 clocks
// of products a row tile.  Measured: 32 x 16 nodes of 8 heads over up to 8191 keys 88.5 us,
// 32 x 32 nodes 141, and 118 and 203 where every tile's keys take their own powers.  Before
// nodes did, and rows were raised alone, they were 84 (2000 clocks of the 2600 a tile took
// were shared memory's) and 134.  Steps on the way there, of the first: unrolled widening
// 157 us (a third of the warps' time went to waiting for instructions), short loops and
// powers by asynchronous copies 102, the products' waits together and eight widening warps
// 97, both warpgroups on every tile and rings of K and V apart 93, producers apart 85.
//
// Warps 0-3 and 4-7 are the two warpgroups, warp 8 issues the MMAs, warps 9 and 10
// stream codes of K with TMA, warp 11 those of V, warps 12-15 widen K and 16-19 V.
// Tensor memory: S0 S1 O0 O1 of 128 columns each; P (16-bit pairs) over S.
#include <cstdio>

#include "attn_tc.cuh"
#include "tree_attn.cuh"

namespace dfv {
namespace {

constexpr int kKeys = 128;
constexpr int kThreads = 640;
constexpr int kWiden = 4;  // warps that widen K, and that widen V

constexpr float kBias = 6.f;
constexpr int kApartK = 15, kApartV = 8;  // how far a tile's powers may be apart for constants of the tile
static_assert(kApartK <= 15 && kApartV <= 15, "half_power");
constexpr int kFlags = 8;
constexpr int kTells = 16;  // tiles whose powers are kept: more than are between their widening and their scores

template <int D, bool DUAL>
struct CodeTcShape {
  static constexpr uint32_t kCodes = kKeys * D;      // a K or V tile in codes
  static constexpr uint32_t kTile = kKeys * D * 2;   // and in fp16
  static constexpr int kK = D == 64 ? 2 : 1, kV = D == 64 ? 3 : 2;  // fp16 tiles of K, and of V behind them
  static constexpr int kCK = D == 64 ? 4 : DUAL ? 1 : 3, kCV = D == 64 ? 4 : 2;  // tiles of codes
  static constexpr int kSlots = kK + kV, kCSlots = kCK + kCV;
  static_assert(kFlags >= kV + 2 && kFlags >= kK + 3, "flags of segments under way");
  static constexpr int kOver = DUAL ? 5 : 3;         // tiles' worth of time that a pair costs at least
  static constexpr uint32_t kQ = (DUAL ? 2 : 1) * 128 * D * 2;
  static constexpr size_t kSmem = 1024 + kQ + (size_t)kSlots * kTile + (size_t)kCSlots * kCodes;
};

// Codes of 16 elements (a 16-byte chunk) as fp16 times m
__device__ __forceinline__ void widen16(const uint4 &x, __half2 m, uint4 &lo, uint4 &hi) {
  const uint32_t *w = &x.x;
  uint32_t y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = codes_f16(w[i]);
    y[2 * i + 1] = codes_f16_hi(w[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2 z = __hmul2(*reinterpret_cast<const __half2 *>(&y[i]), m);
    y[i] = *reinterpret_cast<const uint32_t *>(&z);
  }
  lo = make_uint4(y[0], y[1], y[2], y[3]);
  hi = make_uint4(y[4], y[5], y[6], y[7]);
}

// 2^-d in fp16, d from 0 to 15 (kApartK; the last is a subnormal)
__device__ __forceinline__ __half2 half_power(int d) {
  const uint32_t b = d <= 14 ? (uint32_t)(15 - d) << 10 : 1u << 9;
  const uint32_t two = b | b << 16;
  return *reinterpret_cast<const __half2 *>(&two);
}

// Where a row's chunk of 16 codes is in its swizzled tile.
template <int D>
__device__ __forceinline__ uint32_t place(int row, int c) {
  return (uint32_t)(D == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3));
}

// A key's codes in shared memory: zeroed where it is no node, else its NaN become zero;
// whether there were any.
template <int D>
__device__ __noinline__ bool clean_key(uint32_t row, bool node) {
  bool nan = false;
#pragma unroll 1
  for (int c = 0; c < D / 16; ++c) {
    uint4 x = lds128(row + 16u * c);
    uint32_t *w = &x.x;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t z = ((w[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
      nan = nan || z;
      w[e] = node ? w[e] & ~((z >> 7) * 255u) : 0u;
    }
    sts128(row + 16u * c, x);
  }
  return nan && node;
}

// A tile whose keys have factors of their own: x + b of the scores of the keys that the row sees,
// in place, and their maximum; M and O as they grow; then p and the sum of p 2^-b.  (m, l) before
// and after; j0: node number of the first key (below 0: committed); bar: the product into O before,
// 0 where it is done.  Out of line: calls took 1 to 3 % longer with it among the other tiles' code.
template <int D, int KEYS>
__device__ __noinline__ float2 own_tile(uint32_t t_s, uint32_t t_o, bool started, int j0, uint64_t mask, float crow, uint32_t own, uint32_t back, float m, float l,
                                        uint32_t bar, unsigned phase, unsigned *err, volatile int *abort) {
  float top = -INFINITY;
#pragma unroll 1
  for (int q = 0; q < KEYS; q += 16) {
    const int j = j0 + q;  // node of the first of 16 keys (below 0: committed)
    const uint32_t sees = j >= 0 ? (j < 64 ? (uint32_t)(mask >> j) : 0u) : j > -16 ? (uint32_t)(mask << -j) | ((1u << -j) - 1u) : ~0u;
    float s[16];
    uint32_t x[16];
    tmem_ld16(t_s + q, s);
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const uint4 k = lds128(own + 8u * (q + e));  // 2^a and b of two keys
      s[e] = sees >> e & 1u ? fmaf(s[e], crow * __uint_as_float(k.x), __uint_as_float(k.y)) : -INFINITY;
      s[e + 1] = sees >> e & 2u ? fmaf(s[e + 1], crow * __uint_as_float(k.z), __uint_as_float(k.w)) : -INFINITY;
      x[e] = __float_as_uint(s[e]);
      x[e + 1] = __float_as_uint(s[e + 1]);
    }
    top = max16(s, top);
    tmem_st16(t_s + q, x);
  }
  tmem_wait_st();
  const float mx = top - 8.f > m ? top : m;  // a row's M follows what the row sees, not its neighbours
  if (__any_sync(0xffffffffu, mx > m)) {
    const float f = m == -INFINITY ? 0.f : ex2(m - mx);
    l *= f;
    if (bar && started) {  // the product into O before
      mbar_wait_fast(bar, phase, err, DFV_DEVERR_STAGE_WAIT, abort);
      __syncwarp();
      tc_fence_after();
    }
#pragma unroll 1
    for (int q = 0; q < D && started; q += 16) {
      float o[16];
      tmem_ld16(t_o + q, o);
      uint32_t y[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(o[e] * f);
      tmem_st16(t_o + q, y);
    }
    m = mx;
  }
  const float from = m == -INFINITY ? 0.f : m;
  float l0 = 0.f, l1 = 0.f;
#pragma unroll 1
  for (int q = 0; q < KEYS; q += 16) {
    float s[16];
    uint32_t x[8];
    tmem_ld16(t_s + q, s);
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      const uint4 k = lds128(back + 4u * (q + e));
      const float p0 = ex2((s[e] - from) + kBias), p1 = ex2((s[e + 1] - from) + kBias);
      const float p2 = ex2((s[e + 2] - from) + kBias), p3 = ex2((s[e + 3] - from) + kBias);
      l0 = fmaf(p2, __uint_as_float(k.z), fmaf(p0, __uint_as_float(k.x), l0));
      l1 = fmaf(p3, __uint_as_float(k.w), fmaf(p1, __uint_as_float(k.y), l1));
      x[e / 2] = pack2<true>(p0, p1);
      x[e / 2 + 1] = pack2<true>(p2, p3);
    }
    tmem_st8(t_s + q / 2, x);  // over x + b that have been read
  }
  return make_float2(m, l + (l0 + l1));
}

template <int D, bool DUAL>
__global__ void __launch_bounds__(kThreads, 1) tree_attn_codes_tc_kernel(const __grid_constant__ AttnLaunch L) {
  using S = CodeTcShape<D, DUAL>;
  extern __shared__ __align__(16) unsigned char sm_raw[];
  unsigned char *sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) unsigned long long s_full[S::kSlots], s_empty[S::kSlots], s_cfull[S::kCSlots], s_cempty[S::kCSlots],
      s_sfull[2], s_pready[2][2], s_pvdone[2], s_odone[2], s_qready, s_drain;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ SchedStart s_start;
  __shared__ long long s_scan[kThreads / 32];
  // Of a segment, in turn: NaN was left out.  V is cleaned before its slot is waited for, so with short segments
  // kV + 1 of them may be cleaned before one is put out and its flag cleared.
  __shared__ volatile int s_bad[kFlags];
  __shared__ volatile int2 s_tell[kTells];  // A and B of a tile; A = -1: its keys' own powers are in s_own and s_back
  __shared__ __align__(16) float2 s_own[8][kKeys];  // 2^a and b
  __shared__ __align__(16) float s_back[8][kKeys];  // 2^-b
  __shared__ uint8_t s_below[8][kKeys];  // how far a key's b is below B, of tiles whose V is to come
  __shared__ __align__(8) unsigned long long s_told[8];  // (K is widened up to four tiles before V) s_below and s_tell of a tile are there
  __shared__ __align__(16) unsigned char s_power[S::kCK * 2 * kKeys];  // with K: a and b of the tile's keys
  __shared__ float s_crow[256];        // c times the power that a row of q was divided by
  const TreeAttnParams &p = L.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned char *s_q = sm, *s_ring = sm + S::kQ, *s_codes = s_ring + (size_t)S::kSlots * S::kTile;
  const uint32_t q_addr = smem_u32(s_q), ring = smem_u32(s_ring), codes = smem_u32(s_codes);
  if (tid == 0) {
    s_abort = 0;
    for (int s = 0; s < kFlags; ++s) s_bad[s] = 0;
    for (int s = 0; s < S::kSlots; ++s) {
      mbar_init(smem_u32(&s_full[s]), kWiden);
      mbar_init(smem_u32(&s_empty[s]), 1);
    }
    for (int s = 0; s < S::kCSlots; ++s) {
      mbar_init(smem_u32(&s_cfull[s]), s < S::kCK ? 2 + 64 : 1);  // producers; with K, the powers' lanes
      mbar_init(smem_u32(&s_cempty[s]), kWiden);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(smem_u32(&s_sfull[w]), 1);
      mbar_init(smem_u32(&s_pready[w][0]), 128);
      mbar_init(smem_u32(&s_pready[w][1]), 128);
      mbar_init(smem_u32(&s_pvdone[w]), 1);
      mbar_init(smem_u32(&s_odone[w]), 1);
    }
    for (int s = 0; s < 8; ++s) mbar_init(smem_u32(&s_told[s]), kWiden);
    mbar_init(smem_u32(&s_qready), 256);
    mbar_init(smem_u32(&s_drain), 1);
    mbar_init_fence();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(&s_tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  pdl_wait();
  pdl_trigger();  // the join may now read the call's inputs
  sched_start<kThreads, kKeys, S::kOver>(L, blockIdx.x, s_scan, &s_start);  // syncs the CTA
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int row0 = (int)(blockIdx.x % L.n_rt) * L.rows;  // first row of this CTA
  SegWalk<kKeys, S::kOver> wk(L, s_start);

  if (warp >= 9 && warp < 12) {
    // ---------------------------------------------------------------- producers: every other box of K each, or V
    const bool isk = warp < 11;
    const int me = isk ? warp - 9 : 0, many = isk ? 2 : 1, c0 = isk ? 0 : S::kCK, cn = isk ? S::kCK : S::kCV;
    const CUtensorMap *map = isk ? &L.tm_k : &L.tm_v;
    int st = 0, ph = 0, issued = 0;
    bool ok = true;
    const int shift = p.c.page_shift, boxes = shift >= 7 ? 1 : kKeys >> shift, rows = kKeys / boxes;
    while (ok && wk.next()) {
      if (row0 >= wk.v.n * p.G) continue;
      const int pages = wk.v.s < 0 ? 0 : (wk.total + (1 << shift) - 1) >> shift;
      const int32_t *table = p.c.table + (size_t)(wk.v.s < 0 ? 0 : wk.v.s) * p.c.max_pages;
      // page ids a warp's worth at a time, the next ones on their way
      auto ids = [&](int first) { return first + lane < pages ? table[first + lane] : 0; };
      int base = ((wk.t0 * kKeys) >> shift) & ~31;
      int cur = ids(base), ahead = ids(base + 32);
      if (base + lane < pages) cur = checked_page(p.c, cur);
      for (int t = wk.t0; t < wk.t1; ++t) {
        const int first = (t * kKeys) >> shift;  // a tile's pages are within one such lot: their number divides 32
        if (first >= base + 32) {
          base += 32;
          cur = base + lane < pages ? checked_page(p.c, ahead) : 0;
          ahead = ids(base + 32);
        }
        ok = __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_cempty[c0 + st]), ph ^ 1, p.err, DFV_DEVERR_SLOT_WAIT, &s_abort));
        if (!ok) break;
        const uint32_t fb = smem_u32(&s_cfull[c0 + st]), dst = codes + (uint32_t)(c0 + st) * S::kCodes;
        const int nb = min(boxes, pages - first), at = first & 31, mine = nb > me ? (nb - me + many - 1) / many : 0;
        if (lane == 0) {
          if (mine > 0)
            mbar_expect_tx(fb, (uint32_t)mine * rows * D);
          else
            mbar_arrive(fb);
        }
        __syncwarp();
        const int tok = (t * kKeys) & ((1 << shift) - 1);  // 0 unless a page holds several tiles
        if (isk) {  // with K: this lane's four keys' a (the first producer) or b
          const int my = boxes == 1 ? 0 : (4 * lane) >> shift, page = __shfl_sync(0xffffffffu, cur, (at + my) & 31);
          if (my < nb)
            cp_async4(smem_u32(s_power + (st * 2 + me) * kKeys + 4 * lane),
                      (me == 0 ? p.c.ke : p.c.ve) + exp_off(p.c, p.layer, page, wk.h, (t * kKeys + 4 * lane) & ((1 << shift) - 1)));
          cp_async_arrive(fb);
        }
        for (int b = me; b < nb; b += many)
          tma_kv(dst + (uint32_t)(b * rows * D), map, 0, tok, wk.h, __shfl_sync(0xffffffffu, cur, at + b), L.swap, fb);
        ++issued;
        if (++st == cn) { st = 0; ph ^= 1; }
      }
    }
    // no copy may land after the CTA exits: wait for the last fill of every slot
    volatile int never = 0;
    for (int j = issued - cn < 0 ? 0 : issued - cn; j < issued; ++j)
      if (!mbar_wait(smem_u32(&s_cfull[c0 + j % cn]), (j / cn) & 1, p.err, DFV_DEVERR_DRAIN_WAIT, &never)) break;
  } else if (warp >= 12) {
    // ---------------------------------------------------------------- widening: a key row a thread
    // (Short loops: with the chunks of two tiles unrolled the warps waited for instructions
    // a third of their time.)
    const bool isv = warp >= 16;
    const int kt = (tid - 384) & 127, c0 = isv ? S::kCK : 0, cn = isv ? S::kCV : S::kCK, f0 = isv ? S::kK : 0, fn = isv ? S::kV : S::kK;
    int st = 0, ph = 0, cst = 0, cph = 0;
    unsigned tile = 0, seg = 0;
    bool ok = true;
    while (ok && wk.next()) {
      if (row0 >= wk.v.n * p.G) continue;
#pragma unroll 1
      for (int t = wk.t0; t < wk.t1 && ok; ++t, ++tile) {
        ok = __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_cfull[c0 + cst]), cph, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
        if (!ok) break;
        const uint32_t from = codes + (uint32_t)(c0 + cst) * S::kCodes + (uint32_t)(kt * D);
        int below;
        if (!isv) {
          // the powers of the tile: their largest, and how far this key's are below
          const unsigned char *pw = s_power + cst * 2 * kKeys;
          const int valid = wk.total - t * kKeys - 4 * lane;  // of this lane's four keys
          const uint32_t keep = valid >= 4 ? ~0u : valid <= 0 ? 0u : (1u << (8 * valid)) - 1u;
          const uint32_t w1 = *reinterpret_cast<const uint32_t *>(pw + 4 * lane), w2 = *reinterpret_cast<const uint32_t *>(pw + kKeys + 4 * lane);
          uint32_t m = w1 & keep, m2 = w2 & keep, n = w1 | ~keep, n2 = w2 | ~keep;
          m = __vmaxu4(m, m >> 16);
          m2 = __vmaxu4(m2, m2 >> 16);
          n = __vminu4(n, n >> 16);
          n2 = __vminu4(n2, n2 >> 16);
          const int a = __reduce_max_sync(0xffffffffu, max(m & 255u, m >> 8 & 255u));
          const int b = __reduce_max_sync(0xffffffffu, max(m2 & 255u, m2 >> 8 & 255u));
          const int low = min(n & 255u, n >> 8 & 255u), low2 = min(n2 & 255u, n2 >> 8 & 255u);  // of this lane's
          // factors of their own: nodes among them, or far apart
          const bool own = __any_sync(0xffffffffu, (t + 1) * kKeys > wk.v.len || a - low > kApartK || b - low2 > kApartV), is = t * kKeys + kt < wk.total;
          below = own ? 0 : max(0, a - pw[kt]);
          s_below[tile & 7][kt] = (uint8_t)(own ? 0 : max(0, b - pw[kKeys + kt]));
          if (own) {
            const int pa = is ? max((int)pw[kt], 1) : 127, pb = is ? min(max((int)pw[kKeys + kt], 1), 253) : 127;
            s_own[tile & 7][kt] = make_float2(exp_value((uint32_t)pa), (float)(pb - 127));
            s_back[tile & 7][kt] = exp_value((uint32_t)(254 - pb));
          }
          if (kt == 0) {
            s_tell[tile % kTells].x = own ? -1 : a;
            s_tell[tile % kTells].y = b;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s_told[tile & 7]));
        } else {
          const int jn = t * kKeys + kt - wk.v.len;  // this key's node
          if (jn >= 0 && clean_key<D>(from, jn < wk.nodes)) s_bad[seg % kFlags] = 1;
          ok = __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_told[tile & 7]), (tile >> 3) & 1u, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
          if (!ok) break;
          below = s_below[tile & 7][kt];
        }
        const __half2 m = half_power(below);
        ok = __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_empty[f0 + st]), ph ^ 1, p.err, DFV_DEVERR_SLOT_WAIT, &s_abort));
        if (!ok) break;
        const uint32_t to = ring + (uint32_t)(f0 + st) * S::kTile + (uint32_t)(kt * 128);
#pragma unroll 1
        for (int q = 0; q < D / 16; q += 4) {  // 64 elements
          uint4 x[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) x[c] = lds128(from + 16u * place<D>(kt, q + c));
          const uint32_t half = to + (uint32_t)(q >> 2) * 16384u;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint4 lo, hi;
            widen16(x[c], m, lo, hi);
            sts128(half + (((2 * c) ^ (kt & 7)) << 4), lo);
            sts128(half + (((2 * c + 1) ^ (kt & 7)) << 4), hi);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&s_full[f0 + st]));
          mbar_arrive(smem_u32(&s_cempty[c0 + cst]));
        }
        if (++st == fn) { st = 0; ph ^= 1; }
        if (++cst == cn) { cst = 0; cph ^= 1; }
      }
      ++seg;
    }
  } else if (warp == 8) {
    // ---------------------------------------------------------------- MMA issue
    int kst = 0, kph = 0, vst = 0, vph = 0, seg = 0;  // slots of K and V, and their phases
    bool ok = true;
    const uint32_t iq = idesc_16<true>(kKeys, false), iv = idesc_16<true>(D, true);
    auto wait = [&](unsigned long long &bar, unsigned phase) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&bar), phase, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
    };
    // A step's waits come together: P on `a` (and `b`), V, and the next K.  Each costs about
    // as long as the tensor core's queue lasts.
    auto ready = [&](unsigned long long &a, unsigned long long *b, unsigned phase, bool v, bool k) {
      bool r = mbar_try_wait(smem_u32(&a), phase);
      if (b) r = mbar_try_wait(smem_u32(b), phase) && r;
      if (v) r = mbar_try_wait(smem_u32(&s_full[S::kK + vst]), vph) && r;
      if (k) r = mbar_try_wait(smem_u32(&s_full[kst]), kph) && r;
      if (!__all_sync(0xffffffffu, r)) {
        if (v) wait(s_full[S::kK + vst], vph);
        if (k) wait(s_full[kst], kph);
        wait(a, phase);
        if (b) wait(*b, phase);
      }
      tc_fence_after();
    };
    // a slot is free once the MMAs issued so far have read it
    auto done_k = [&]() {
      tc_commit_elect(smem_u32(&s_empty[kst]));
      if (++kst == S::kK) { kst = 0; kph ^= 1; }
    };
    auto done_v = [&]() {
      tc_commit_elect(smem_u32(&s_empty[S::kK + vst]));
      if (++vst == S::kV) { vst = 0; vph ^= 1; }
    };
    // place of scores `to`, and DUAL warpgroup `to`'s rows
    auto qk = [&](int to) {
      tc_scores<D, 128>(tmem + (uint32_t)to * 128u, sdesc_k128(q_addr + (DUAL ? (uint32_t)to * 128u * D * 2u : 0u)), sdesc_k128(ring + (uint32_t)kst * S::kTile), iq);
      tc_commit_elect(smem_u32(&s_sfull[to]));
    };
    int place = 0, turn = 0;  // SINGLE: of the next product's P, and its barriers' phase; DUAL: the phase
    while (ok && wk.next()) {
      if (row0 >= wk.v.n * p.G) continue;
      const int n = wk.t1 - wk.t0;
      wait(s_qready, seg & 1);
      ++seg;
      wait(s_full[kst], kph);
      tc_fence_after();
      if (!ok) break;
      if (DUAL) {
        auto pv = [&](int w, bool first, bool last) {
          tc_values<128>(tmem + 256u + (uint32_t)w * 128u, tmem + (uint32_t)w * 128u, sdesc_mn128(ring + (uint32_t)(S::kK + vst) * S::kTile), iv, first ? 0u : 1u);
          if (last) tc_commit_elect(smem_u32(&s_odone[w]));
        };
        qk(0);
        qk(1);
        done_k();
        for (int j = 0; j < n; ++j) {
          // each warpgroup's next scores right after its own product
          const bool more = j + 1 < n;
          ready(s_pready[0][0], nullptr, turn, true, more);
          if (!ok) break;
          pv(0, j == 0, !more);
          if (more) qk(0);
          ready(s_pready[1][0], nullptr, turn, false, false);
          if (!ok) break;
          pv(1, j == 0, !more);
          done_v();
          if (more) {
            qk(1);
            done_k();
          }
          turn ^= 1;
        }
      } else {
        qk(place);
        done_k();
        if (n > 1) {
          wait(s_full[kst], kph);
          tc_fence_after();
          if (!ok) break;
          qk(place ^ 1);
          done_k();
        }
        for (int j = 0; j < n; ++j) {
          // each warpgroup's 64 keys of V_j into its own O, then the scores of K_j+2
          ready(s_pready[0][place], &s_pready[1][place], turn, true, j + 2 < n);
          if (!ok) break;
          const uint32_t from = tmem + (uint32_t)place * 128u;
          const uint64_t vd = sdesc_mn128(ring + (uint32_t)(S::kK + vst) * S::kTile);
          tc_values<64>(tmem + 256u, from, vd, iv, j ? 1u : 0u);
          tc_values<64>(tmem + 384u, from + 64u, vd + 512u, iv, j ? 1u : 0u);
          tc_commit_elect(smem_u32(&s_pvdone[place]));
          if (j + 1 == n) {
            tc_commit_elect(smem_u32(&s_odone[0]));
            tc_commit_elect(smem_u32(&s_odone[1]));
          }
          done_v();
          if (j + 2 < n) {
            qk(place);
            done_k();
          }
          turn ^= place;
          place ^= 1;
        }
      }
    }
    // every MMA issued has completed before tensor memory is released
    tc_commit_elect(smem_u32(&s_drain));
    volatile int never = 0;
    mbar_wait(smem_u32(&s_drain), 0u, p.err, DFV_DEVERR_DRAIN_WAIT, &never);
  } else {
    // ---------------------------------------------------------------- softmax and output
    const int w = warp >> 2, wt = tid & 127;  // warpgroup, and its thread = row of the tile
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_o = lane_base + 256u + (uint32_t)w * 128u;
    constexpr int kMine = DUAL ? kKeys : kKeys / 2;  // keys of a tile that the warpgroup takes
    unsigned nt = 0;     // tiles this warpgroup has taken
    unsigned outs = 0;   // segments it has put out
    unsigned tiles = 0, seg = 0;  // of the segments before
    bool ok = true;
    // after a wait gives up the loops still run to the end without touching
    // tensor memory, so the warpgroups meet at every barrier
    while (wk.next()) {
      const int R = wk.v.n * p.G;
      if (row0 >= R) continue;  // never the CTA that tells of the pair: its rows are the first
      const int n = wk.t1 - wk.t0;
      // rows into the swizzled layout as fp16, each divided by a power of two; past R zero
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
            uint32_t *v = &x[k].x;
            float top = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(bf16_lo(v[e])), fabsf(bf16_hi(v[e]))));
#pragma unroll
            for (int o = 1; o < kCh; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            // times 2^(127 - exponent), the ends of the range the same
            const int f = min(253, max(1, 254 - (int)(__float_as_uint(top) >> 23)));
            const float up = exp_value((uint32_t)f);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = pack2<true>(bf16_lo(v[e]) * up, bf16_hi(v[e]) * up);
            if (ch == 0) s_crow[rr] = p.scale_log2 * exp_value((uint32_t)(254 - f));
            *reinterpret_cast<uint4 *>(s_q + (rr >> 7) * (128 * D * 2) + (ch >> 3) * 16384 + (rr & 127) * 128 +
                                       (((ch & 7) ^ (rr & 7)) << 4)) = x[k];
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(smem_u32(&s_qready));
      bar_sync_n(1, 256);  // s_crow

      const int rr = DUAL ? w * 128 + wt : wt, r = row0 + rr;  // this thread's row
      const float crow = s_crow[rr];
      uint64_t mask = 0;
      if (r < R) mask = wk.mask_of(r);
      float m = -INFINITY, l = 0.f;
      bool started = false;
      for (int j = 0; j < n; ++j) {
        const unsigned T = nt++, place = T & 1;
        const uint32_t t_s = lane_base + (DUAL ? (uint32_t)w * 128u : place * 128u + (uint32_t)w * 64u);
        if (DUAL)
          ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_sfull[w]), T & 1u, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
        else
          ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_sfull[place]), (T >> 1) & 1u, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
        if (!ok) continue;
        tc_fence_after();
        const int j0 = (wk.t0 + j) * kKeys + (DUAL ? 0 : 64 * w) - wk.v.len;  // node number of the first key
        const unsigned tell = (tiles + (unsigned)j) % kTells;
        const int ea = s_tell[tell].x;
        if (ea < 0) {
          const int at = DUAL ? 0 : 64 * w;
          const float2 ml = own_tile<D, kMine>(t_s, t_o, started, j0, mask, crow, smem_u32(&s_own[tell & 7][at]), smem_u32(&s_back[tell & 7][at]), m, l,
                                               DUAL ? 0u : smem_u32(&s_pvdone[place ^ 1]), ((T - 1) >> 1) & 1u, p.err, &s_abort);
          m = ml.x;
          l = ml.y;
          ok = __all_sync(0xffffffffu, s_abort == 0);
        } else {
          // in (0, infinity)
          const float c = fminf(fmaxf(crow * exp_value((uint32_t)ea), 0x1p-120f), 0x1p120f);
          const int eb = min(max(s_tell[tell].y, 1), 253);
          const float B = (float)(eb - 127), back = exp_value((uint32_t)(254 - eb));
          float high = -INFINITY;
          {
            float s0[16], s1[16];
            tmem_ld16_async(t_s, s0);
#pragma unroll 1
            for (int q = 0; q < kMine; q += 32) {
              tmem_wait_ld16(s0);
              tmem_ld16_async(t_s + q + 16, s1);
              high = max16(s0, high);
              tmem_wait_ld16(s1);
              tmem_ld16_async(t_s + (q + 32) % kMine, s0);  // (the last one is the first again)
              high = max16(s1, high);
            }
            tmem_wait_ld16(s0);
          }
          const float top = fmaf(high, c, B);
          if (__any_sync(0xffffffffu, top - 8.f > m)) {
            // the product into O before: DUAL's was issued before these scores, and their
            // barrier follows all that was issued before it
            if (!DUAL && started) {
              ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_pvdone[place ^ 1]), ((T - 1) >> 1) & 1u, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
              tc_fence_after();
            }
            // a row's M follows what the row sees, not its neighbours
            const float mx = top - 8.f > m ? top : m, f = m == -INFINITY ? 0.f : ex2(m - mx);
            l *= f;
            if (started && ok) {
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
          {
            // x + B - M by differences from the tile's maximum: whatever the scores' size, the
            // exponents are 8 at most and right next to it
            const float from = high == -INFINITY ? 0.f : high, z = (high == -INFINITY ? 0.f : m - top) - kBias;
            float2 l2 = make_float2(0.f, 0.f);
            float s0[16], s1[16];
            uint32_t x[8];
            tmem_ld16_async(t_s, s0);
#pragma unroll 1
            for (int q = 0; q < kMine; q += 32) {
              tmem_wait_ld16(s0);
              tmem_ld16_async(t_s + q + 16, s1);
              exp16(s0, from, c, z, x, l2);
              tmem_wait_ld16(s1);
              if (q + 32 < kMine) tmem_ld16_async(t_s + q + 32, s0);
              tmem_st8(t_s + q / 2, x);  // over scores that have been read
              exp16(s1, from, c, z, x, l2);
              tmem_st8(t_s + q / 2 + 8, x);
            }
            l = fmaf(l2.x + l2.y, back, l);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(smem_u32(&s_pready[w][DUAL ? 0 : place]));
        started = true;
      }
      tiles += (unsigned)n;
      // ---- output: the last product of this warpgroup, then (SINGLE) both states
      ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_odone[w]), outs & 1u, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
      ++outs;
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      float M = m, lsum = l, f0 = 1.f, f1 = 1.f;
      // all scores are done when either warpgroup's last product is: Q's place is free
      float2 *ml = reinterpret_cast<float2 *>(s_q);
      if (!DUAL) ml[w * 128 + wt] = make_float2(m, l);
      // SINGLE: each warpgroup waited for its own products and reads both outputs, so
      // what it learned about tensor memory goes through the barrier
      tc_fence_before();
      bar_sync_n(1, 256);  // the states, and Q's place
      tc_fence_after();
      if (!DUAL) {
        const float2 a = ml[wt];
        const float2 b = ml[128 + wt];
        M = fmaxf(a.x, b.x);
        // a state without keys adds its zeros (or NaN of a NaN query)
        f0 = a.x == -INFINITY ? 1.f : ex2(a.x - M);
        f1 = b.x == -INFINITY ? 1.f : ex2(b.x - M);
        lsum = a.y * f0 + b.y * f1;
      }
      const int bad = s_bad[seg % kFlags];
      const float z = (M == -INFINITY ? 0.f : M) - kBias;
      const int c0 = DUAL ? 0 : w * (D / 2), c1 = DUAL ? D : c0 + D / 2;
      const bool whole = wk.whole();
      const int slot = wk.slot(blockIdx.x), i = node_of(L, r), head = wk.h * p.G + r - i * p.G;
      const size_t row = wk.v.row0 + i;
      const float inv = lsum == 0.f ? 0.f : 1.f / lsum;  // NaN stays NaN
      char *out = p.o + 2 * (row * p.o_row + head * p.o_head);
      float4 *part = reinterpret_cast<float4 *>(L.part_o) + (size_t)slot * (D / 4) * L.rows + rr;
#pragma unroll 1
      for (int q = c0; q < c1 && ok; q += 16) {
        float o[16];
        tmem_ld16_async(lane_base + 256u + (DUAL ? (uint32_t)w * 128u : 0u) + q, o);
        if (!DUAL) {
          float o1[16];
          tmem_ld16_async(lane_base + 384u + q, o1);
          tmem_wait_ld16(o);
          tmem_wait_ld16(o1);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = o[e] * f0 + o1[e] * f1;
        } else {
          tmem_wait_ld16(o);
        }
        if (r >= R) continue;
        if (whole) {
          uint32_t x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = pack2<false>(o[2 * e] * inv, o[2 * e + 1] * inv);
          uint4 *to = reinterpret_cast<uint4 *>(out + 2 * q);
          to[0] = make_uint4(x[0], x[1], x[2], x[3]);
          to[1] = make_uint4(x[4], x[5], x[6], x[7]);
        } else {
          float4 *to = part + (size_t)(q / 4) * L.rows;
#pragma unroll
          for (int e = 0; e < 4; ++e) to[(size_t)e * L.rows] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      if (r < R && ok && c0 == 0) {
        if (whole) {
          if (p.lse) p.lse[row * p.H + head] = lsum == 0.f ? -INFINITY : (z + log2f(lsum)) * 0.69314718055994531f;
        } else {
          L.part_ml[(size_t)slot * L.rows + rr] = make_float2(M == -INFINITY ? -INFINITY : z, lsum);
        }
      }
      if (whole && bad && r < R && ok) add_unseen<false>(p, wk.v, i, wk.h, out, c0, c1);
      if (tid == 0) {
        if (!whole) L.part_bad[slot] = bad;
        wk.tell(s_start, blockIdx.x);
      }
      tc_fence_before();
      bar_sync_n(1, 256);  // O, Q's place and s_bad are read
      if (tid == 0) s_bad[seg % kFlags] = 0;
      ++seg;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

template <int D, bool DUAL>
cudaError_t launch_one(const AttnLaunch &L, cudaStream_t s) {
  auto kern = tree_attn_codes_tc_kernel<D, DUAL>;
  const size_t smem = CodeTcShape<D, DUAL>::kSmem;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kern, smem, done);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, dim3(L.n_groups * L.n_rt), dim3(kThreads), smem, s, L);
}

}  // namespace

cudaError_t launch_attn_codes_tc(const AttnLaunch &L, cudaStream_t s) {
  const bool dual = L.rows == 256;
  if (L.p.c.D == 128) return dual ? launch_one<128, true>(L, s) : launch_one<128, false>(L, s);
  return dual ? launch_one<64, true>(L, s) : launch_one<64, false>(L, s);
}

}  // namespace dfv
