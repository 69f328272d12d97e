// prompt_attn.cu -- causal attention of packed prompts on the fifth-generation
// tensor cores.
//
// Mathematics as in tree_attn.cu: o = sum_j p_j v_j / sum_j p_j with p_j =
// 2^(c q.k_j - M) for any M, c = scale log2(e); the state (M, l, O) of some keys, and
// states over disjoint keys join exactly.
//
// Rows.  The query heads of a kv head share its keys, so row r of a (sequence, kv
// head) is position r / G, head r % G of the group, and a tile is 256 rows: 32
// positions of 8 heads.  The keys that a tile needs end with its last position, so
// little is computed above the diagonal, and the causal mask is one limit per
// row.  A CTA streams the tile's keys in blocks of 128: two warpgroups take 128
// rows each, S = Q K^T goes to tensor memory, a thread turns its row of S into P
// over S, and O += P V accumulates in tensor memory.  P is given to the products in
// halves of 64 keys, so that a product starts while the second half is in its
// exponentials.  M is only raised, and O only rescaled, when a row's maximum grew by
// more than 2^8; before the second half of a block that waits for the first half's
// product.
//
// Work split.  All tiles' blocks form one line, (sequence, kv head, tile) after
// (sequence, kv head, tile), with some blocks' worth for what a tile costs however
// few its keys; the line is cut into one range per SM.  A tile that a range cuts
// leaves states that a second launch joins in range order (no atomics: the same
// bits every time).  Where no tile is long the ranges end at tiles instead, and
// there is no second launch.  How many blocks the tiles before tile i have follows
// from a closed form, since the lengths are only known on the device.
//
// Masked places.  Scores beyond a row's limit are selected away.  V rows past the
// sequence's end (the next sequence's) are zeroed in shared memory before the
// product; values that are not finite, in rows that not all of the tile's rows
// see, are taken out and given back to the rows that see them at the end.
//
// Warps 0-3 and 4-7 are the two warpgroups, warps 8 and 10 stream K and V blocks
// with TMA into one ring in the order the MMAs use them (half of the head, or half
// of the keys, each), warp 9 issues the MMAs.
// Tensor memory: S0 S1 O0 O1 of 128 columns each; P (16-bit pairs) over S.
#include <cstdio>

#include <cudaTypedefs.h>

#include "attn_tc.cuh"

namespace dfv {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn(char *why, size_t why_len);

namespace {

constexpr int kKeys = 128;   // of a block
constexpr int kTile = 256;   // rows of a tile
constexpr int kThreads = 352;
constexpr int kOver = 5;     // blocks' worth of time that a tile costs at least
constexpr int kWholeKeys = 1024;  // tiles are cut where a sequence may have more keys

template <int D>
struct PromptShape {
  static constexpr uint32_t kBlock = kKeys * D * 2;  // one K or V block
  static constexpr int kSlots = D == 64 ? 8 : 5;
  static constexpr uint32_t kQ = kTile * D * 2;
  static constexpr size_t kSmem = 1024 + kQ + (size_t)kSlots * kBlock;
};

struct PromptLaunch {
  CUtensorMap tm_k, tm_v;  // {head_dim, head, row}, head and row in stride order
  PromptParams p;
  int swap_k, swap_v;      // row before head
  int whole;               // ranges end at tiles
  uint32_t inv_g;          // ceil(2^16 / G)
  int4 *cut;               // [kAttnCtas] sequence, head, tile that begins in the range and goes on, ranges it is in (0: none)
  float2 *part_ml;         // [2 kAttnCtas][kTile] (M, l) of partial states
  float *part_o;           // [2 kAttnCtas][D / 4][kTile][4] their sums of p v
  int *part_bad;           // [2 kAttnCtas] a value that is not finite was left out
};

size_t sections(PromptLaunch *L, int D, void *ws) {
  constexpr size_t slots = 2 * (size_t)kAttnCtas;
  size_t off = kWsScratch;
  auto take = [&](size_t n) {
    void *q = ws ? (void *)((char *)ws + off) : nullptr;
    off += align256(n);
    return q;
  };
  int4 *cut = (int4 *)take(kAttnCtas * sizeof(int4));
  int *bad = (int *)take(slots * 4);
  float2 *ml = (float2 *)take(slots * kTile * 8);
  float *o = (float *)take(slots * kTile * D * 4);
  if (L) {
    L->cut = cut;
    L->part_bad = bad;
    L->part_ml = ml;
    L->part_o = o;
  }
  return off;
}

// ---------------------------------------------------------------- the work line
struct PromptSeq {
  int row0, n, key0, nk;  // rows of q and of k; n = 0 where there is nothing to do
};
__device__ __forceinline__ PromptSeq prompt_seq(const PromptParams &p, int b) {
  const int r0 = p.row_off[b], r1 = p.row_off[b + 1], k0 = p.key_off[b], k1 = p.key_off[b + 1];
  PromptSeq s = {r0, r1 - r0, k0, k1 - k0};
  if (r0 < 0 || r1 < r0 || r1 > p.n_rows || s.n > p.max_rows || k0 < 0 || k1 < k0 || k1 > p.n_keys || s.nk > p.max_keys) {
    flag_err(p.kverr, DFV_KVERR_LEN);
    s.n = s.nk = 0;
    s.row0 = s.key0 = 0;
  }
  return s;
}
__device__ __forceinline__ int tiles_of(const PromptParams &p, const PromptSeq &s) { return (s.n * p.G + kTile - 1) / kTile; }

// Keys that position i of a sequence sees.
__device__ __forceinline__ int limit_of(const PromptSeq &s, int i) { return min(s.nk, max(0, s.nk - s.n + i + 1)); }

// Blocks of tile t: at least one (its outputs have to be written).
__device__ __forceinline__ int blocks_of(const PromptParams &p, const PromptSeq &s, int t) {
  const int last = min(s.n - 1, (kTile * t + kTile - 1) / p.G);
  return max(1, (limit_of(s, last) + kKeys - 1) / kKeys);
}

// Blocks of the tiles before tile i <= last tile of the sequence.  Tile t that is
// not the last ends with position (256 t + 255) / G, so its blocks are
//   max(1, floor((2 t + B) / G)),  B = floor((255 + G (128 + nk - n)) / 128);
// the floors are counted in runs of G tiles, over which they grow by 2.
__device__ __forceinline__ long long blocks_before(const PromptParams &p, const PromptSeq &s, int i) {
  const int G = p.G, B = (int)((255 + (long long)G * (kKeys + s.nk - s.n)) >> 7);
  const int i1 = B >= G ? 0 : (G - B + 1) / 2;  // the first tile with a block by the formula
  if (i <= i1) return i;
  const int c = 2 * i1 + B, w = i - i1, a = w / G, r = w - a * G;
  int all = 0, part = 0;
  for (int u = 0; u < G; ++u) {
    const int f = (2 * u + c) / G;
    all += f;
    if (u < r) part += f;
  }
  return i1 + (long long)a * all + (long long)G * a * (a - 1) + part + 2ll * a * r;
}

__device__ __forceinline__ long long head_units(const PromptParams &p, const PromptSeq &s) {
  const int m = tiles_of(p, s);
  return m == 0 ? 0 : (long long)kOver * m + blocks_before(p, s, m - 1) + blocks_of(p, s, m - 1);
}

struct PromptStart {
  long long u0, u1, base;  // the range, and the first unit of sequence b
  long long U;             // units
  int b, G;                // ranges in use
};
__device__ __forceinline__ long long range_start(int g, long long U, int G) { return g * U / G; }
__device__ __forceinline__ int range_of(long long u, long long U, int G) { return (int)(((u + 1) * G - 1) / U); }

// The range of CTA `g` and the sequence it starts in; all threads of the CTA call it.
__device__ __forceinline__ void prompt_start(const PromptLaunch &L, int g, long long *s_scan, PromptStart *out) {
  const PromptParams &p = L.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = p.n_seqs;
  const int per = (n + kThreads - 1) / kThreads, b0 = min(n, tid * per), b1 = min(n, b0 + per);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) sum += p.Hkv * head_units(p, prompt_seq(p, b));
  long long run = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += a;
  }
  if (lane == 31) s_scan[warp] = run;
  if (tid == 0) {
    out->u0 = out->u1 = out->base = 0;
    out->b = 0;
  }
  __syncthreads();
  long long U = 0, at = run - sum;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) at += s_scan[w];
    U += s_scan[w];
  }
  const int G = U >= kAttnCtas ? kAttnCtas : U > 0 ? (int)U : 1;
  const long long u0 = range_start(g, U, G), u1 = g < G ? range_start(g + 1, U, G) : u0;
  if (u0 < u1 && at <= u0 && u0 < at + sum) {
    long long base = at;
    for (int b = b0; b < b1; ++b) {
      const long long c = per == 1 ? sum : p.Hkv * head_units(p, prompt_seq(p, b));
      if (base <= u0 && u0 < base + c) {
        out->u0 = u0;
        out->u1 = u1;
        out->base = base;
        out->b = b;
      }
      base += c;
    }
  }
  if (tid == 0) {
    out->U = U;
    out->G = G;
  }
  __syncthreads();
}

// Segments of a range: blocks [t0, t1) of one tile.
struct PromptWalk {
  const PromptLaunch &L;
  const long long end;
  long long u;       // units of the line so far
  long long last;    // last unit of the tile
  int b, h, t, m;    // sequence, kv head, tile, tiles of a head
  int t0, t1, T;     // blocks of the segment, of the tile
  int p0;            // units of the next tile that lie before the range
  bool first;
  PromptSeq s;
  __device__ __forceinline__ PromptWalk(const PromptLaunch &l, const PromptStart &st) : L(l), end(st.u1), u(st.u0), b(st.b), h(0), t(-1), m(0), p0(0), first(true) {
    if (u >= end) return;
    s = prompt_seq(L.p, b);
    m = tiles_of(L.p, s);
    const long long per = head_units(L.p, s);
    long long w = u - st.base;
    h = (int)(w / per);
    w -= h * per;
    // the last tile that begins at or before unit w of the head
    int lo = 0, hi = m;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((long long)kOver * mid + blocks_before(L.p, s, mid) <= w)
        lo = mid;
      else
        hi = mid;
    }
    t = lo;
    p0 = (int)(w - ((long long)kOver * t + blocks_before(L.p, s, t)));
    if (L.whole && p0) {  // it belongs to the range before
      u += kOver + blocks_of(L.p, s, t) - p0;
      p0 = 0;
      ++t;
    }
  }
  __device__ __forceinline__ bool next() {
    for (;;) {
      if (!first) ++t;
      first = false;
      if (u >= end) return false;
      while (t >= m) {
        t = 0;
        if (++h >= L.p.Hkv || m == 0) {
          h = 0;
          ++b;
          s = prompt_seq(L.p, b);
          m = tiles_of(L.p, s);
        }
      }
      T = blocks_of(L.p, s, t);
      const int units = kOver + T, p1 = L.whole ? units : (int)min((long long)units, p0 + (end - u));
      last = u - p0 + units - 1;
      t0 = max(0, p0 - kOver);
      t1 = max(0, p1 - kOver);
      u += p1 - p0;
      p0 = 0;
      if (t0 < t1) return true;
    }
  }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == T; }
  // Partial states of a range: of a tile that began before it, and of one that goes
  // on after it.
  __device__ __forceinline__ int slot(int g) const { return 2 * g + (t0 == 0); }
};

// ---------------------------------------------------------------- pieces
// A block's box, issued by an elected lane of a warp in step.
__device__ __forceinline__ void tma_block(uint32_t dst, const CUtensorMap *map, int x, int h, int row, int swap, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(swap ? row : h), "r"(swap ? h : row), "r"(bar)
      : "memory");
}

// Scores of a block of which the row sees the first `sees` keys: the others become
// -inf, in place.
__device__ __forceinline__ void mask_block(uint32_t t_s, int sees) {
#pragma unroll 1
  for (int q = 0; q < kKeys; q += 16) {
    if (__all_sync(0xffffffffu, q + 16 <= sees)) continue;
    float s[16];
    tmem_ld16(t_s + q, s);
    uint32_t x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = q + e < sees ? __float_as_uint(s[e]) : 0xff800000u;
    tmem_st16(t_s + q, x);
  }
  tmem_wait_st();
}

// Key row `row` of a V block in shared memory: zeroed where `past`; else its values
// that are not finite become zero and set *bad.
template <bool F16, int D>
__device__ __forceinline__ void clean_key(unsigned char *block, int row, bool past, int *bad) {
  constexpr uint32_t kExp = F16 ? 0x7c00u : 0x7f80u;
#pragma unroll 1
  for (int c = 0; c < D / 8; ++c) {  // chunk order turned by the row: no bank conflicts
    uint4 *at = reinterpret_cast<uint4 *>(block + (c >> 3) * 16384 + row * 128 + (((c ^ row) & 7) << 4));
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    bool hit = past;
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

// What clean_key took out of the values of keys [from, to), added to elements c0 .. c1
// of a stored output (rare: a value next to the diagonal is not finite).
template <bool F16>
__device__ __noinline__ void add_taken(const PromptParams &p, const PromptSeq &s, int h, int from, int to, char *out, int c0, int c1) {
  uint32_t *w = reinterpret_cast<uint32_t *>(out);
#pragma unroll 1
  for (int d = c0; d < c1; d += 2) {
    float2 x = unpack2<F16>(w[d / 2]);
#pragma unroll 1
    for (int j = from; j < to; ++j) {
      const float2 y = unpack2<F16>(*reinterpret_cast<const uint32_t *>(p.v + 2 * ((s.key0 + (long long)j) * p.v_row + h * p.v_head + d)));
      if (!isfinite(y.x)) x.x += y.x;
      if (!isfinite(y.y)) x.y += y.y;
    }
    w[d / 2] = pack2<F16>(x.x, x.y);
  }
}

// Position within the tile's first row's group and head of row rr of a tile: the
// quotient of a number below 1024 + 256 by G <= 16.
__device__ __forceinline__ int over_g(const PromptLaunch &L, int r) { return (int)(((uint32_t)r * L.inv_g) >> 16); }

template <bool F16, int D>
__global__ void __launch_bounds__(kThreads, 1) prompt_attn_kernel(const __grid_constant__ PromptLaunch L) {
  using S = PromptShape<D>;
  constexpr float kBias = F16 ? 6.f : 0.f;
  extern __shared__ __align__(16) unsigned char sm_raw[];
  unsigned char *sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) unsigned long long s_full[S::kSlots], s_empty[S::kSlots], s_sfull[2], s_pready[2][2], s_half[2],
      s_odone[2], s_qready, s_drain;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ PromptStart s_start;
  __shared__ long long s_scan[kThreads / 32];
  __shared__ int s_bad;
  const PromptParams &p = L.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned char *s_q = sm, *s_ring = sm + S::kQ;
  const uint32_t q_addr = smem_u32(s_q), ring = smem_u32(s_ring);
  if (tid == 0) {
    s_abort = 0;
    s_bad = 0;
    for (int s = 0; s < S::kSlots; ++s) {
      mbar_init(smem_u32(&s_full[s]), 2);
      mbar_init(smem_u32(&s_empty[s]), 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(smem_u32(&s_sfull[w]), 1);
      mbar_init(smem_u32(&s_pready[w][0]), 128);
      mbar_init(smem_u32(&s_pready[w][1]), 128);
      mbar_init(smem_u32(&s_half[w]), 1);
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
  prompt_start(L, blockIdx.x, s_scan, &s_start);  // syncs the CTA
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  PromptWalk wk(L, s_start);

  if (warp == 8 || warp == 10) {
    // ---------------------------------------------------------------- producers
    const int me = (warp - 8) / 2;
    int st = 0, ph = 0, issued = 0;
    bool ok = true;
    while (ok && wk.next()) {
      auto load = [&](const CUtensorMap *map, int swap, int t) {
        ok = ok && __all_sync(0xffffffffu,
                              mbar_wait_fast(smem_u32(&s_empty[st]), ph ^ 1, p.err, DFV_DEVERR_SLOT_WAIT, &s_abort));
        if (!ok) return;
        // this warp's box: 64 elements of 128 keys (D = 128), or all 64 of half the keys
        const uint32_t fb = smem_u32(&s_full[st]), dst = ring + (uint32_t)st * S::kBlock + (uint32_t)me * (S::kBlock / 2);
        if (lane == 0) mbar_expect_tx(fb, S::kBlock / 2);
        __syncwarp();
        tma_block(dst, map, D == 128 ? 64 * me : 0, wk.h, wk.s.key0 + t * kKeys + (D == 128 ? 0 : 64 * me), swap, fb);
        ++issued;
        if (++st == S::kSlots) { st = 0; ph ^= 1; }
      };
      load(&L.tm_k, L.swap_k, wk.t0);
      for (int t = wk.t0; t < wk.t1 && ok; ++t) {
        load(&L.tm_v, L.swap_v, t);
        if (t + 1 < wk.t1) load(&L.tm_k, L.swap_k, t + 1);
      }
    }
    // no copy may land after the CTA exits: wait for the last fill of every slot
    volatile int never = 0;
    for (int j = issued - S::kSlots < 0 ? 0 : issued - S::kSlots; j < issued; ++j)
      if (!mbar_wait(smem_u32(&s_full[j % S::kSlots]), (j / S::kSlots) & 1, p.err, DFV_DEVERR_DRAIN_WAIT, &never)) break;
  } else if (warp == 9) {
    // ---------------------------------------------------------------- MMA issue
    int st = 0, ph = 0, seg = 0;
    unsigned np[2] = {0u, 0u};  // blocks of each warpgroup whose P was awaited
    bool ok = true;
    const uint32_t iq = idesc_16<F16>(kKeys, false), iv = idesc_16<F16>(D, true);
    auto full = [&]() {
      ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_full[st]), ph, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
      tc_fence_after();
    };
    auto done = [&]() {  // the slot is free once the MMAs issued so far have read it
      tc_commit_elect(smem_u32(&s_empty[st]));
      if (++st == S::kSlots) { st = 0; ph ^= 1; }
    };
    auto qk = [&](int w) {
      const uint32_t kb = ring + (uint32_t)st * S::kBlock, qb = q_addr + (uint32_t)w * 128u * D * 2u;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        tc_mma_ss(tmem + (uint32_t)w * 128u, sdesc_k128(qb + (ks >> 2) * 16384) + (uint64_t)(2 * (ks & 3)),
                  sdesc_k128(kb + (ks >> 2) * 16384) + (uint64_t)(2 * (ks & 3)), iq, ks > 0 ? 1u : 0u);
      tc_commit_elect(smem_u32(&s_sfull[w]));
    };
    auto pv = [&](int w, bool first, bool last) {
      const uint32_t vb = ring + (uint32_t)st * S::kBlock;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_pready[w][hf]), np[w] & 1u, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
        if (!ok) return;
        tc_fence_after();
#pragma unroll
        for (int ks = 4 * hf; ks < 4 * hf + 4; ++ks)
          tc_mma_ts(tmem + 256u + (uint32_t)w * 128u, tmem + (uint32_t)w * 128u + (uint32_t)ks * 8u,
                    sdesc_mn128(vb + (uint32_t)ks * 2048u), iv, (first && ks == 0) ? 0u : 1u);
        if (hf == 0) tc_commit_elect(smem_u32(&s_half[w]));
      }
      ++np[w];
      if (last) tc_commit_elect(smem_u32(&s_odone[w]));
    };
    while (ok && wk.next()) {
      const int n = wk.t1 - wk.t0;
      ok = __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_qready), seg & 1, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
      ++seg;
      tc_fence_after();
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
          const int sv = st, pv_ = ph;
          if (++st == S::kSlots) { st = 0; ph ^= 1; }
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
    }
    // every MMA issued has completed before tensor memory is released
    tc_commit_elect(smem_u32(&s_drain));
    volatile int never = 0;
    mbar_wait(smem_u32(&s_drain), 0u, p.err, DFV_DEVERR_DRAIN_WAIT, &never);
  } else {
    // ---------------------------------------------------------------- softmax and output
    const int w = warp >> 2, wt = tid & 127;  // warpgroup, and its thread = row of the tile
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_s = lane_base + (uint32_t)w * 128u, t_o = lane_base + 256u + (uint32_t)w * 128u;
    const float c = p.scale_log2;
    unsigned nt = 0;     // blocks this warpgroup has taken
    unsigned outs = 0;   // segments it has put out
    unsigned items = 0;  // ring items of the segments before
    bool ok = true, told = false;
    // after a wait gives up the loops still run to the end without touching
    // tensor memory, so the warpgroups meet at every barrier
    while (wk.next()) {
      const int R = wk.s.n * p.G, n = wk.t1 - wk.t0, r0 = wk.t * kTile;
      const int i0 = r0 / p.G, rest = r0 - i0 * p.G;  // position and head of the tile's first row
      // rows into the swizzled layout; past R zero
      {
        constexpr int kCh = D / 8, kStep = 256 / kCh;  // 16-byte chunks of a row; rows apart
        constexpr int kIter = kTile / kStep, kBatch = kIter < 8 ? kIter : 8;
        const int ch = tid % kCh;
        const char *qh = p.q + 2 * ((wk.s.row0 + (long long)i0) * p.q_row + (long long)wk.h * p.G * p.q_head + ch * 8);
        uint4 x[kBatch];
#pragma unroll
        for (int k0 = 0; k0 < kIter; k0 += kBatch) {
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int rr = tid / kCh + (k0 + k) * kStep, i = over_g(L, rest + rr), g = rest + rr - i * p.G;
            x[k] = make_uint4(0u, 0u, 0u, 0u);
            if (r0 + rr < R) x[k] = *reinterpret_cast<const uint4 *>(qh + 2 * (i * p.q_row + g * p.q_head));
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

      const int rr = w * 128 + wt, r = r0 + rr;  // this thread's row
      const int pi = over_g(L, rest + rr), i = i0 + pi, head = wk.h * p.G + rest + rr - pi * p.G;
      const int lim = r < R ? limit_of(wk.s, i) : wk.s.nk, lim0 = limit_of(wk.s, i0);  // keys that this row, and every row, sees
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_sfull[w]), nt & 1u, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
        ++nt;
        if (!ok) continue;
        tc_fence_after();
        const int k0 = (wk.t0 + j) * kKeys;
        if (k0 + kKeys > lim0) {
          mask_block(t_s, lim - k0);
          if (w == 0) {
            // this block's V before it is multiplied
            const unsigned it = items + 2u * (unsigned)j + 1u;
            ok = __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_full[it % S::kSlots]), (it / S::kSlots) & 1u, p.err,
                                                        DFV_DEVERR_STAGE_WAIT, &s_abort));
            if (!ok) continue;
            if (k0 + wt >= lim0) clean_key<F16, D>(s_ring + (size_t)(it % S::kSlots) * S::kBlock, wt, k0 + wt >= wk.s.nk, &s_bad);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
        }
        if (j == 0) {  // a maximum to begin with
          float s0[32], s1[32];
          tmem_ld32(t_s, s0);
          tmem_ld32(t_s + 32, s1);
          tmem_wait_ld32(s0);
          tmem_wait_ld32(s1);
          m = max32(s1, max32(s0, m));
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          // One pass with the M so far: p and the new maximum together.  Only when
          // some row's maximum grew too far is O rescaled and the pass made again.
          uint32_t x[32];
          float2 l2;
          for (;;) {
            // (rounded up: the largest p stays within its bound however large the scores are)
            const float z = (m == -INFINITY ? 0.f : __fmul_ru(m, c)) - kBias;
            float s0[32], s1[32], mx = m;
            l2 = make_float2(0.f, 0.f);
            tmem_ld32(t_s + 64 * hf, s0);
            tmem_wait_ld32(s0);
            tmem_ld32(t_s + 64 * hf + 32, s1);
            mx = max32(s0, mx);
            exp32<F16>(s0, c, z, x, l2);
            tmem_wait_ld32(s1);
            mx = max32(s1, mx);
            exp32<F16>(s1, c, z, x + 16, l2);
            if (!__any_sync(0xffffffffu, (mx - m) * c > 8.f)) break;
            // products into O before these scores: those of the blocks before were
            // complete when the scores were; the first half's own is waited for
            if (hf == 1) {
              ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_half[w]), (nt - 1u) & 1u, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
              tc_fence_after();
            }
            const float f = m == -INFINITY ? 0.f : ex2((m - mx) * c);
            l *= f;
            if (ok && (j > 0 || hf == 1)) {
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
          l += l2.x + l2.y;
          tmem_st16(t_s + 32 * hf, x);
          tmem_st16(t_s + 32 * hf + 16, x + 16);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(smem_u32(&s_pready[w][hf]));
        }
      }
      items += 2u * (unsigned)n;
      // ---- output: the last product of this warpgroup
      ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_odone[w]), outs & 1u, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
      ++outs;
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      bar_sync_n(1, 256);  // s_bad, and Q's place
      const int bad = s_bad;
      const float z = (m == -INFINITY ? 0.f : __fmul_ru(m, c)) - kBias;
      const bool whole = wk.whole();
      const int slot = wk.slot(blockIdx.x);
      const size_t row = wk.s.row0 + (size_t)i;
      const float inv = l == 0.f ? 0.f : 1.f / l;  // NaN stays NaN
      char *out = p.o + 2 * ((long long)row * p.o_row + head * p.o_head);
      float4 *part = reinterpret_cast<float4 *>(L.part_o) + (size_t)slot * (D / 4) * kTile + rr;
#pragma unroll 1
      for (int q = 0; q < D && ok; q += 32) {
        float o[32];
        tmem_ld32(t_o + q, o);
        tmem_wait_ld32(o);
        if (r >= R) continue;
        if (whole) {
          uint32_t x[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = pack2<F16>(o[2 * e] * inv, o[2 * e + 1] * inv);
          uint4 *to = reinterpret_cast<uint4 *>(out + 2 * q);
#pragma unroll
          for (int e = 0; e < 4; ++e) to[e] = make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        } else {
          float4 *to = part + (size_t)(q / 4) * kTile;
#pragma unroll
          for (int e = 0; e < 8; ++e) to[(size_t)e * kTile] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      if (r < R && ok) {
        if (whole) {
          if (p.lse) p.lse[row * p.H + head] = l == 0.f ? -INFINITY : (z + log2f(l)) * 0.69314718055994531f;
          if (bad) add_taken<F16>(p, wk.s, wk.h, lim0, lim, out, 0, D);
        } else {
          L.part_ml[(size_t)slot * kTile + rr] = make_float2(m == -INFINITY ? -INFINITY : z, l);
        }
      }
      if (tid == 0 && !whole) {
        L.part_bad[slot] = bad;
        if (wk.t0 == 0) {
          L.cut[blockIdx.x] = make_int4(wk.b, wk.h, wk.t, range_of(wk.last, s_start.U, s_start.G) - (int)blockIdx.x + 1);
          told = true;
        }
      }
      tc_fence_before();
      bar_sync_n(1, 256);  // O, Q's place and s_bad are read
      if (tid == 0) s_bad = 0;
    }
    if (tid == 0 && !told) L.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- join
// A CTA joins 32 rows of the tile that begins in a range and goes on behind it: a
// lane per row, a warp per D / 8 elements of the head.
constexpr int kJoinWarps = 8, kJoinRows = 32;

template <bool F16, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) prompt_join_kernel(const __grid_constant__ PromptLaunch L) {
  constexpr int kPer = D / 4 / kJoinWarps;  // float4 of a thread
  const PromptParams &p = L.p;
  const int g0 = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rr = blockIdx.y * kJoinRows + lane;
  pdl_trigger();
  pdl_wait();
  const int4 cut = __ldcg(&L.cut[g0]);
  const int n = cut.w;
  if (n < 2) return;
  const PromptSeq s = prompt_seq(p, cut.x);
  const int r = cut.z * kTile + rr;
  if (r >= s.n * p.G) return;
  // state k is range g0 + k's; the tile goes on after the first and began before the others
  auto slot = [&](int k) { return (size_t)(2 * (g0 + k) + (k == 0)); };
  float M = -INFINITY;
  for (int k = 0; k < n; ++k) M = fmaxf(M, __ldcg(&L.part_ml[slot(k) * kTile + rr]).x);
  float4 x[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) x[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  int bad = 0;
#pragma unroll 2
  for (int k = 0; k < n; ++k) {
    const float2 ml = __ldcg(&L.part_ml[slot(k) * kTile + rr]);
    bad |= __ldcg(&L.part_bad[slot(k)]);
    const float f = ml.x == -INFINITY ? 1.f : ex2(ml.x - M);  // a state without keys holds zeros (or NaN of a NaN query)
    l = fmaf(ml.y, f, l);
    const float4 *from = reinterpret_cast<const float4 *>(L.part_o) + (slot(k) * (D / 4) + warp * kPer) * kTile + rr;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const float4 y = __ldcg(from + (size_t)e * kTile);
      x[e].x = fmaf(y.x, f, x[e].x);
      x[e].y = fmaf(y.y, f, x[e].y);
      x[e].z = fmaf(y.z, f, x[e].z);
      x[e].w = fmaf(y.w, f, x[e].w);
    }
  }
  const int i = r / p.G, head = cut.y * p.G + r - i * p.G;
  const size_t row = s.row0 + (size_t)i;
  const float inv = l == 0.f ? 0.f : 1.f / l;  // NaN stays NaN
  char *out = p.o + 2 * ((long long)row * p.o_row + head * p.o_head);
#pragma unroll
  for (int e = 0; e < kPer; ++e)
    reinterpret_cast<uint2 *>(out)[warp * kPer + e] = make_uint2(pack2<F16>(x[e].x * inv, x[e].y * inv), pack2<F16>(x[e].z * inv, x[e].w * inv));
  if (bad) add_taken<F16>(p, s, cut.y, limit_of(s, cut.z * kTile / p.G), limit_of(s, i), out, 4 * warp * kPer, 4 * (warp + 1) * kPer);
  if (p.lse && warp == 0) p.lse[row * p.H + head] = l == 0.f ? -INFINITY : (M == -INFINITY ? l : (M + log2f(l)) * 0.69314718055994531f);
}

bool encode_rows(CUtensorMap *map, const PromptParams &p, const char *base, long long row, long long head, int box_rows,
                 int *swap, char *why, size_t why_len) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn(why, why_len);
  if (!fn) return false;
  *swap = p.Hkv > 1 && p.n_keys > 1 && row < head;
  // a dimension of one entry has no stride of its own
  const cuuint64_t one = 16;
  const cuuint64_t r[2] = {(cuuint64_t)p.n_keys, p.n_keys > 1 ? (cuuint64_t)row * 2 : one};
  const cuuint64_t h[2] = {(cuuint64_t)p.Hkv, p.Hkv > 1 ? (cuuint64_t)head * 2 : one};
  const cuuint64_t *a = *swap ? r : h, *b = *swap ? h : r;
  const cuuint64_t dims[3] = {(cuuint64_t)p.D, a[0], b[0]};
  const cuuint64_t strides[2] = {a[1], b[1]};
  const cuuint32_t box[3] = {64, *swap ? (cuuint32_t)box_rows : 1u, *swap ? 1u : (cuuint32_t)box_rows};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult e = fn(map, p.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                        const_cast<char *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (e != CUDA_SUCCESS) {
    snprintf(why, why_len, "tensor map of the keys or values refused (%d)", (int)e);
    return false;
  }
  return true;
}

template <bool F16, int D>
cudaError_t launch_typed(const PromptLaunch &L, cudaStream_t s) {
  auto kern = prompt_attn_kernel<F16, D>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kern, PromptShape<D>::kSmem, done);
  if (e != cudaSuccess) return e;
  e = launch_chained(kern, dim3(kAttnCtas), dim3(kThreads), PromptShape<D>::kSmem, s, L);
  if (e != cudaSuccess || L.whole) return e;
  return launch_chained(prompt_join_kernel<F16, D>, dim3(kAttnCtas, kTile / kJoinRows), dim3(32 * kJoinWarps), 0, s, L);
}

}  // namespace

size_t prompt_attn_ws(int D) { return sections(nullptr, D, nullptr); }

cudaError_t launch_prompt_attn(const PromptParams &p, void *ws, cudaStream_t s, char *why, size_t why_len) {
  static thread_local PromptLaunch L;
  L.p = p;
  L.inv_g = (65536u + p.G - 1) / p.G;
  L.whole = p.max_keys <= kWholeKeys;
  sections(&L, p.D, ws);
  const int box = p.D == 128 ? kKeys : kKeys / 2;
  if (!encode_rows(&L.tm_k, p, p.k, p.k_row, p.k_head, box, &L.swap_k, why, why_len) ||
      !encode_rows(&L.tm_v, p, p.v, p.v_row, p.v_head, box, &L.swap_v, why, why_len))
    return cudaErrorInvalidValue;
  if (p.D == 128) return p.f16 ? launch_typed<true, 128>(L, s) : launch_typed<false, 128>(L, s);
  return p.f16 ? launch_typed<true, 64>(L, s) : launch_typed<false, 64>(L, s);
}

}  // namespace dfv
