// prompt_attn.cu -- causal attention of packed prompts on the fifth-generation
// tensor cores.
//
// Mathematics as in tree_attn.cu: o = sum_j p_j v_j / sum_j p_j with p_j =
// 2^(c q.k_j - M) for any M, c = scale log2(e); the state (M, l, O) of some keys, and
// states over disjoint keys join exactly.
//
// Rows.  The query heads of a kv head share its keys.  A tile is P consecutive
// positions (256 / G, a multiple of 8) of the G heads of a kv head: row g P + i.  The
// keys that a tile needs end with its last position, so little is computed above the
// diagonal, and the causal mask is one limit per row.  A CTA streams the tile's keys
// in blocks of 128: two warpgroups take 128 rows each, S = Q K^T goes to tensor
// memory, a thread turns its row of S into P over S, and O += P V accumulates in
// tensor memory.  One pass over the scores computes p with the M so far; M is only
// raised, and O only rescaled, when a row's maximum grew by more than 2^8, and the
// pass is then made again; rows of the warp whose maxima did not keep theirs, so that
// a key that a row does not see leaves the row's bits alone (with scores six times as
// far apart as products of normal q and k, 4 x 2039 rows took 145 us when they were raised
// together, and take 153).
//
// Precision.  As in tree_attn.cu: scores, M, l and O are fp32, and p alone is rounded
// to the inputs' type for the second product, since both its operands have one type (p in
// 32 bits would take tf32 values, at half the rate and twice the bytes, or a second
// product).  With normal values the outputs' error in the 2-norm is 0.0019 to 0.0023 for
// bf16, where 32-bit p and the outputs' own rounding make 0.0015 to 0.0017 (fp16:
// 0.0003 and 0.0002).
//
// Scores take turns in NB places of 128 columns: two with heads of 128, one a
// warpgroup; three with heads of 64, where the outputs leave room, so that a warpgroup's
// next scores are ready while it is still in its exponentials.  The products follow the
// warpgroups' places in turn, PV_i then QK_(i + NB) in one step: the tensor core's queue
// is a few MMAs deep, and each wait of the warp that fills it, ready or not, takes
// about as long as they do, so a step's waits come first and together (apart, before
// each product, they took a third of the time).  A tile's queries are copied, and
// its first scores made, while the warpgroups put out the tile before.
//
// Work split.  All tiles' blocks form one line, (sequence, kv head, tile) after
// (sequence, kv head, tile), with some blocks' worth for what a tile costs however
// few its keys; the line is cut into one range per SM.  A tile that a range cuts
// leaves states that a second launch joins in range order (no atomics: the same
// bits every time).  Where no tile is long the ranges end at tiles instead, and
// there is no second launch; with no more tiles than SMs each has one.  How many blocks the tiles before tile i have follows
// from a closed form, since the lengths are only known on the device.
//
// Masked places.  Scores beyond a row's limit are selected away.  V rows past the
// sequence's end (the next sequence's) are zeroed in shared memory before the
// product; values that are not finite, in rows that not all of the tile's rows
// see, are taken out and given back to the rows that see them at the end.
//
// Warps 0-3 and 4-7 are the two warpgroups, warps 8 and 10 stream K and V blocks
// with TMA into a ring each in the order the MMAs use them (half of the head, or half
// of the keys, each), warp 9 issues the MMAs, warp 11 copies Q and cleans V.
// Tensor memory: NB places of scores, P (16-bit pairs) over them, then O0 O1.
//
// What binds.  With heads of 128 the tensor core: a block takes 2048 clocks of
// products and 2700 in all (16381 tokens without the softmax's arithmetic 1174 us).  With
// heads of 64 a block takes 2050 clocks, 1600 without that arithmetic where its products
// should take 1024: those of 64 columns may take longer than half of 128 columns' time,
// or wait for shared memory, of which a block reads 96 KB (768 clocks) while TMA writes
// 32; the two were not told apart.  Measured (GB300, device time): 16381 tokens of 32 heads
// of 128 over 4 kv heads 1385 us, 1.59 PFLOP/s of 1.88 (ten in a row 1455 each, under the
// power limit); 16 prompts of 1020 to 2039 tokens 312 us (1.04 PFLOP/s: a tile's start and
// output cost it 6500 clocks beside 2700 a block); 2 x 1021 tokens behind 30011 with heads
// of 64 421 to 446 us.  Not kept: P handed on in halves (1384 -> 1459 us), the maximum in a
// pass of its own (1504 -> 1527; heads of 64 458 -> 508).
#include <cstdio>

#include <cudaTypedefs.h>

#include "attn_tc.cuh"

namespace dfv {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn(char *why, size_t why_len);

namespace {

constexpr int kKeys = 128;   // of a block
constexpr int kTile = 256;   // rows of a tile
constexpr int kThreads = 384;
constexpr int kOver = 3;     // blocks' worth of time that a tile costs at least
// Tiles are whole where no sequence has more keys (without a second launch; whole and cut, prompts
// of equal length: 16 of 600 tokens 77 and 90 us, one of 1200 22 and 31, one of 2039 53 and 50),
// and where there are many: each saves about two thirds of a block's time by not being cut, and
// ranges end up to half the longest tile apart (16 prompts of 2039 459 and 479, 64 of 3000 3650 and
// 3690; 8 of 4096 810 and 806, 4 of 8192 1510 and 1453).
constexpr int kWholeKeys = 1536;
enum PromptMode { kCut, kWhole, kOne };  // ranges cut tiles, end at tiles, are tiles

template <int D>
struct PromptShape {
  static constexpr uint32_t kBlock = kKeys * D * 2;  // one K or V block
  static constexpr int kK = D == 64 ? 4 : 3, kV = D == 64 ? 4 : 2;  // blocks of K, and of V behind them
  static constexpr int kSlots = kK + kV;
  static constexpr uint32_t kQ = kTile * D * 2;
  static constexpr int kNB = D == 64 ? 3 : 2;        // places of scores
  static constexpr uint32_t kO = 128 * kNB;          // tensor-memory column of O0
  static constexpr size_t kSmem = 1024 + kQ + (size_t)kSlots * kBlock;
};

struct PromptLaunch {
  CUtensorMap tm_q, tm_k, tm_v;  // {head_dim, row, head}
  PromptParams p;
  int pos;                 // positions of a tile
  int run, rise;           // so many tiles further, tiles have so many blocks more
  uint32_t inv_pos;        // ceil(2^16 / pos)
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
__device__ __forceinline__ int tiles_of(const PromptLaunch &L, const PromptSeq &s) { return (s.n + L.pos - 1) / L.pos; }

// Keys that position i of a sequence sees.
__device__ __forceinline__ int limit_of(const PromptSeq &s, int i) { return min(s.nk, max(0, s.nk - s.n + i + 1)); }

// Blocks of tile t: at least one (its outputs have to be written).
__device__ __forceinline__ int blocks_of(const PromptLaunch &L, const PromptSeq &s, int t) {
  return max(1, (limit_of(s, min(s.n, (t + 1) * L.pos) - 1) + kKeys - 1) / kKeys);
}

// Blocks of the tiles before tile i <= last tile of the sequence.  Tile t that is not
// the last has max(1, floor((P t + C) / 128)) of them, C = P + 127 + nk - n; the
// floors are counted in runs of 128 / gcd(P, 128) tiles, over which they grow by
// P / gcd(P, 128).
__device__ __forceinline__ long long blocks_before(const PromptLaunch &L, const PromptSeq &s, int i) {
  const int P = L.pos, C = P + kKeys - 1 + s.nk - s.n;
  const int i1 = C >= kKeys ? 0 : (kKeys - C + P - 1) / P;  // the first tile with a block by the formula
  if (i <= i1) return i;
  const int c = P * i1 + C, w = i - i1, a = w / L.run, r = w - a * L.run;
  int all = 0, part = 0;
  for (int u = 0; u < L.run; ++u) {
    const int f = (P * u + c) / kKeys;
    all += f;
    if (u < r) part += f;
  }
  return i1 + (long long)a * all + (long long)L.rise * L.run * ((long long)a * (a - 1) / 2) + part + (long long)L.rise * a * r;
}

__device__ __forceinline__ long long head_units(const PromptLaunch &L, const PromptSeq &s) {
  const int m = tiles_of(L, s);
  return m == 0 ? 0 : (long long)kOver * m + blocks_before(L, s, m - 1) + blocks_of(L, s, m - 1);
}

// The start of a kernel is a chain of reads and divisions that nothing overlaps: what it
// finds out is kept for all warps, and divisions are of 32 bits where the numbers are
// (one prompt of 137 tokens 12.4 -> 11.0 us).
struct PromptStart {
  long long u0, u1, base;  // the range, and the first unit of sequence b
  long long U;             // units
  long long per;           // units of a head of b
  int b, G;                // ranges in use
  PromptSeq s;             // b
  int h, t;                // where a CTA has one tile: its head, and its number
};
__device__ __forceinline__ long long range_start(int g, long long U, int G) {
  return U < 1 << 24 ? (uint32_t)g * (uint32_t)U / (uint32_t)G : g * U / G;  // (G <= 152)
}
__device__ __forceinline__ int range_of(long long u, long long U, int G) { return (int)(((u + 1) * G - 1) / U); }

// The range of CTA `g` and the sequence it starts in; all threads of the CTA call it.  (Where
// ranges are tiles no units are counted.)
template <int MODE>
__device__ __forceinline__ void prompt_start(const PromptLaunch &L, int g, long long *s_scan, PromptStart *out) {
  const PromptParams &p = L.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = p.n_seqs;
  const int per = (n + kThreads - 1) / kThreads, b0 = min(n, tid * per), b1 = min(n, b0 + per);
  long long sum = 0, units = 0;
  PromptSeq s = {0, 0, 0, 0};
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    s = prompt_seq(p, b);
    units = MODE == kOne ? tiles_of(L, s) : head_units(L, s);
    sum += p.Hkv * units;
  }
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
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const long long x = s_scan[w];
    if (w < warp) at += x;
    U += x;
  }
  const int G = U >= kAttnCtas ? kAttnCtas : U > 0 ? (int)U : 1;
  const long long u0 = MODE == kOne ? g : range_start(g, U, G), u1 = MODE == kOne ? min((long long)g + 1, max(U, (long long)g)) : g < G ? range_start(g + 1, U, G) : u0;
  if (u0 < u1 && at <= u0 && u0 < at + sum) {
    long long base = at;
    int b = b0;
#pragma unroll 1
    while (per > 1) {  // the one of this thread's that has u0
      s = prompt_seq(p, b);
      units = MODE == kOne ? tiles_of(L, s) : head_units(L, s);
      if (u0 < base + p.Hkv * units) break;
      base += p.Hkv * units;
      ++b;
    }
    out->u0 = u0;
    out->u1 = u1;
    out->base = base;
    out->per = units;
    out->b = b;
    out->s = s;
    if (MODE == kOne) {
      const int w = (int)(u0 - base);
      out->h = w / (int)units;
      out->t = w - out->h * (int)units;
    }
  }
  if (tid == 0) {
    out->U = U;
    out->G = G;
  }
  __syncthreads();
}

// Segments of a range: blocks [t0, t1) of one tile.
template <int MODE>
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
    s = st.s;
    if (MODE == kOne) {
      h = st.h;
      t = st.t;
      return;
    }
    m = tiles_of(L, s);
    long long w = u - st.base;
    h = (w | st.per) >> 31 ? (int)(w / st.per) : (int)((uint32_t)w / (uint32_t)st.per);
    w -= h * st.per;
    // the last tile that begins at or before unit w of the head: 32 places at a time, which
    // a warp's lanes try together (the first one fits)
    int lo = 0, hi = m;
    long long at = 0;
#pragma unroll 1
    while (lo + 1 < hi) {
      const int gap = (hi - lo + 31) >> 5, i = lo + gap * (int)(threadIdx.x & 31);
      const long long begins = i < hi ? (long long)kOver * i + blocks_before(L, s, i) : 0;
      const int last = 31 - __clz(__ballot_sync(0xffffffffu, i < hi && begins <= w));
      at = __shfl_sync(0xffffffffu, begins, last);
      lo += gap * last;
      hi = min(hi, lo + gap);
    }
    t = lo;
    p0 = (int)(w - at);
    if (MODE == kWhole && p0) {  // it belongs to the range before
      u += kOver + blocks_of(L, s, t) - p0;
      p0 = 0;
      ++t;
    }
  }
  __device__ __forceinline__ bool next() {
    if (MODE == kOne) {
      if (u >= end) return false;
      ++u;
      T = blocks_of(L, s, t);
      t0 = 0;
      t1 = T;
      return true;
    }
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
          m = tiles_of(L, s);
        }
      }
      T = blocks_of(L, s, t);
      const int units = kOver + T, p1 = MODE != kCut ? units : (int)min((long long)units, p0 + (end - u));
      last = u - p0 + units - 1;
      t0 = max(0, p0 - kOver);
      t1 = max(0, p1 - kOver);
      u += p1 - p0;
      p0 = 0;
      if (t0 < t1) return true;
    }
  }
  __device__ __forceinline__ bool whole() const { return MODE != kCut || (t0 == 0 && t1 == T); }
  // Partial states of a range: of a tile that began before it, and of one that goes
  // on after it.
  __device__ __forceinline__ int slot(int g) const { return 2 * g + (t0 == 0); }
};

// ---------------------------------------------------------------- pieces
// A block's box, issued by an elected lane of a warp in step.
__device__ __forceinline__ void tma_block(uint32_t dst, const CUtensorMap *map, int x, int row, int h, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(row), "r"(h), "r"(bar)
      : "memory");
}

// Keys of a block that the products take, 16 at a time: those that the tile's last row
// sees, of the first block 16 at least (its product writes O).
__device__ __forceinline__ int steps_of(const PromptLaunch &L, const PromptSeq &s, int t, int j) {
  const int seen = limit_of(s, min(s.n, (t + 1) * L.pos) - 1) - j * kKeys;
  return min(kKeys / 16, max(1, (seen + 15) >> 4));
}

// Scores of the first `n` keys of a block of which the row sees the first `sees`: the
// others become -inf, in place.
__device__ __forceinline__ void mask_block(uint32_t t_s, int sees, int n) {
#pragma unroll 1
  for (int q = 0; q < n; q += 16) {
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

// Rows [from, to) of a V block in shared memory, by one warp: zeroed from `past` on;
// values that are not finite before that become zero and are told of.
template <bool F16, int D>
__device__ __forceinline__ bool clean_block(uint32_t block, int from, int past, int to) {
  // a 16-bit half whose exponent is all ones carries into its sign
  constexpr uint32_t kExp = F16 ? 0x7c007c00u : 0x7f807f80u, kOne = F16 ? 0x04000400u : 0x00800080u;
  constexpr int kCh = D / 8;  // 16-byte chunks of a row
  const int lane = threadIdx.x & 31;
  auto place = [&](int u) {
    const int row = u / kCh, c = u % kCh;
    return block + (uint32_t)((c >> 3) * 16384 + row * 128 + (((c ^ row) & 7) << 4));
  };
  for (int u = max(from, past) * kCh + lane; u < to * kCh; u += 32) sts128(place(u), make_uint4(0u, 0u, 0u, 0u));
  bool hit = false;
  const int end = min(past, to) * kCh;
  for (int u0 = from * kCh + lane; u0 < end; u0 += 128) {
    uint4 v[4];
    uint32_t any = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (u0 + 32 * i < end) v[i] = lds128(place(u0 + 32 * i));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t *w = &v[i].x;
#pragma unroll
      for (int e = 0; e < 4; ++e) any |= (w[e] & kExp) + kOne;
    }
    if (any & 0x80008000u) {  // rare
      hit = true;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t *w = &v[i].x;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t z = ((w[e] & kExp) + kOne) & 0x80008000u;
          w[e] &= ~((z >> 15) * 0xffffu);
        }
        if (u0 + 32 * i < end) sts128(place(u0 + 32 * i), v[i]);
      }
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  return __any_sync(0xffffffffu, hit);
}

// What clean_block took out of the values of keys [from, to), added to elements c0 .. c1
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

// Head of row r < 256 of a tile (its product's error stays below one part in 2^16 / P).
__device__ __forceinline__ int head_of(const PromptLaunch &L, int r) { return (int)(((uint32_t)r * L.inv_pos) >> 16); }

// A row's 32 elements of a lane become rows' 16-byte quarters among four lanes: lane q of
// four then stores quarter q of each of the four rows, 64 bytes of a row side by side.
__device__ __forceinline__ void turn_quads(uint4 (&x)[4]) {
  const int q = threadIdx.x & 3;
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {  // swap the parts that differ in bit d of (row, quarter)
    const bool up = q & d;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & d) continue;
      uint4 &lo = x[i], &hi = x[i | d];
      uint4 give = up ? lo : hi, got;
      got.x = __shfl_xor_sync(0xffffffffu, give.x, d);
      got.y = __shfl_xor_sync(0xffffffffu, give.y, d);
      got.z = __shfl_xor_sync(0xffffffffu, give.z, d);
      got.w = __shfl_xor_sync(0xffffffffu, give.w, d);
      if (up)
        lo = got;
      else
        hi = got;
    }
  }
}

// (A kernel for each way to end the ranges: without what only cut tiles need, and where
// there are no more tiles than CTAs without the units, it is smaller and starts sooner.  One
// prompt of 137 tokens 10.8 -> 8.3 us.)
template <bool F16, int D, int MODE>
__global__ void __launch_bounds__(kThreads, 1) prompt_attn_kernel(const __grid_constant__ PromptLaunch L) {
  using S = PromptShape<D>;
  constexpr int NB = S::kNB, LA = NB - 1;  // K blocks ahead of the V block in the ring
  extern __shared__ __align__(16) unsigned char sm_raw[];
  unsigned char *sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) unsigned long long s_full[S::kSlots], s_empty[S::kSlots], s_odone[2], s_qfull, s_qfree, s_drain;
  // By warpgroup and the block's parity: with three places of scores a warpgroup and the
  // MMA warp can be one block apart, and a wait by parity must not find two phases done.
  __shared__ __align__(8) unsigned long long s_sfull[2][2], s_pready[2][2];
  // V may be cleaned once it is there, and is clean.  (Not seeing all phases of the ring's
  // barriers, the cleaning warp cannot tell a phase to come from the one before: it asks
  // about a block only when the MMA warp has had the one before in its slot, which it has
  // a block ahead.)
  __shared__ __align__(8) unsigned long long s_dirty, s_clean;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ PromptStart s_start;
  __shared__ long long s_scan[kThreads / 32];
  __shared__ volatile int s_bad[4];  // of a segment, in turn: a value that is not finite was left out
  const PromptParams &p = L.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t q_addr = smem_u32(sm), ring = q_addr + S::kQ;
  if (tid == 0) {
    s_abort = 0;
    for (int s = 0; s < 4; ++s) s_bad[s] = 0;
    for (int s = 0; s < S::kSlots; ++s) {
      mbar_init(smem_u32(&s_full[s]), 2);
      mbar_init(smem_u32(&s_empty[s]), 1);
    }
    for (int w = 0; w < 2; ++w) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_u32(&s_sfull[w][b]), 1);
        mbar_init(smem_u32(&s_pready[w][b]), 128);
      }
      mbar_init(smem_u32(&s_odone[w]), 1);
    }
    mbar_init(smem_u32(&s_qfull), 1);
    mbar_init(smem_u32(&s_qfree), 1);
    mbar_init(smem_u32(&s_dirty), 1);
    mbar_init(smem_u32(&s_clean), 1);
    mbar_init(smem_u32(&s_drain), 1);
    mbar_init_fence();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&s_tmem), 512);
    tmem_relinquish();
  }
  if (warp == 11 && lane < 3) {
    const CUtensorMap *map = lane == 0 ? &L.tm_q : lane == 1 ? &L.tm_k : &L.tm_v;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
  }
  // rows of Q that no copy writes
  for (int u = p.G * L.pos * (D / 8) + tid; u < kTile * (D / 8); u += kThreads)
    sts128(q_addr + (uint32_t)((u % (D / 8) >> 3) * 32768 + u / (D / 8) * 128 + (u & 7) * 16), make_uint4(0u, 0u, 0u, 0u));
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  tc_fence_before();
  pdl_wait();
  pdl_trigger();  // the join may now read the call's inputs
  prompt_start<MODE>(L, blockIdx.x, s_scan, &s_start);  // syncs the CTA
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  PromptWalk<MODE> wk(L, s_start);

  if (warp == 8 || warp == 10) {
    // ---------------------------------------------------------------- producers
    const int me = (warp - 8) / 2;
    unsigned nk = 0, nv = 0;  // blocks of K and V so far
    bool ok = true;
    auto load = [&](const CUtensorMap *map, const PromptWalk<MODE> &wk, int t, int slot, unsigned phase) {
      ok = ok && __all_sync(0xffffffffu,
                            mbar_wait_fast(smem_u32(&s_empty[slot]), (phase & 1u) ^ 1u, p.err, DFV_DEVERR_SLOT_WAIT, &s_abort));
      if (!ok) return;
      // this warp's box: 64 elements of 128 keys (D = 128), or all 64 of half the keys
      const uint32_t fb = smem_u32(&s_full[slot]), dst = ring + (uint32_t)slot * S::kBlock + (uint32_t)me * (S::kBlock / 2);
      if (lane == 0) mbar_expect_tx(fb, S::kBlock / 2);
      __syncwarp();
      tma_block(dst, map, D == 128 ? 64 * me : 0, wk.s.key0 + t * kKeys + (D == 128 ? 0 : 64 * me), wk.h, fb);
    };
    while (ok && wk.next()) {
      for (int t = wk.t0 - LA; t < wk.t1 && ok; ++t) {  // in the order of their first uses
        if (t >= wk.t0) {
          load(&L.tm_v, wk, t, S::kK + (int)(nv % S::kV), nv / S::kV);
          ++nv;
        }
        if (ok && t + LA < wk.t1) {
          load(&L.tm_k, wk, t + LA, (int)(nk % S::kK), nk / S::kK);
          ++nk;
        }
      }
    }
    // no copy may land after the CTA exits: wait for the last fill of every slot (after a
    // wait gave up the last one was not made, and this wait gives up too)
    volatile int never = 0;
    for (unsigned j = nk > S::kK ? nk - S::kK : 0; j < nk; ++j)
      if (!mbar_wait(smem_u32(&s_full[j % S::kK]), (j / S::kK) & 1, p.err, DFV_DEVERR_DRAIN_WAIT, &never)) break;
    for (unsigned j = nv > S::kV ? nv - S::kV : 0; j < nv; ++j)
      if (!mbar_wait(smem_u32(&s_full[S::kK + j % S::kV]), (j / S::kV) & 1, p.err, DFV_DEVERR_DRAIN_WAIT, &never)) break;
  } else if (warp == 11) {
    // ---------------------------------------------------------------- Q, and V next to the diagonal
    unsigned seg = 0, blocks = 0, cleaned = 0;  // segments; blocks of those before; blocks cleaned
    bool ok = true;
    while (ok && wk.next()) {
      const int n = wk.t1 - wk.t0, i0 = wk.t * L.pos, lim0 = limit_of(wk.s, i0);
      // the scores of the segment before are made: its Q has been read
      if (seg) ok = __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_qfree), (seg - 1) & 1u, p.err, DFV_DEVERR_SLOT_WAIT, &s_abort));
      if (!ok) break;
      if (lane == 0) {
        mbar_expect_tx(smem_u32(&s_qfull), (uint32_t)(p.G * L.pos * D * 2));
        s_bad[seg & 3] = 0;  // of four segments before: long put out
      }
      __syncwarp();
#pragma unroll
      for (int hf = 0; hf < D / 64; ++hf)
        tma_block(q_addr + (uint32_t)hf * (S::kQ / (D / 64)), &L.tm_q, 64 * hf, wk.s.row0 + i0, wk.h * p.G, smem_u32(&s_qfull));
      // blocks that some row does not see the end of
      for (int j = max(0, lim0 / kKeys - wk.t0); j < n && ok; ++j) {
        const unsigned nv = blocks + (unsigned)j, slot = S::kK + nv % S::kV;
        ok = __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_dirty), cleaned & 1u, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
        ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_full[slot]), (nv / S::kV) & 1u, p.err,
                                                          DFV_DEVERR_STAGE_WAIT, &s_abort));
        if (!ok) break;
        const int k0 = (wk.t0 + j) * kKeys;
        if (clean_block<F16, D>(ring + slot * S::kBlock, max(0, lim0 - k0), max(0, wk.s.nk - k0), 16 * steps_of(L, wk.s, wk.t, wk.t0 + j)))
          s_bad[seg & 3] = 1;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s_clean));
        ++cleaned;
      }
      blocks += (unsigned)n;
      ++seg;
    }
    volatile int never = 0;
    if (seg) mbar_wait(smem_u32(&s_qfull), (seg - 1) & 1u, p.err, DFV_DEVERR_DRAIN_WAIT, &never);
  } else if (warp == 9) {
    // ---------------------------------------------------------------- MMA issue
    // (Counters that only ever step on: what the descriptors and addresses come from stays
    // in uniform registers.  Taken from a segment's lengths they made the issue of an MMA
    // take longer than the MMA: 1972 us for 1504 with 16381 tokens.)
    unsigned seg = 0, cleaned = 0;           // segments; blocks cleaned
    unsigned kst = 0, kph = 0, vst = 0, vph = 0;  // slots of K and V and their phases
    unsigned kpl = 0, vpl = 0;               // places of scores: of the next QK, of the next PV
    unsigned kb = 0, vb = 0;                 // blocks of QK and of PV
    bool ok = true;
    const uint32_t iq = idesc_16<F16>(kKeys, false), iv = idesc_16<F16>(D, true);
    auto wait = [&](unsigned long long &bar, unsigned phase) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&bar), phase, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
    };
    // what PV of warpgroup w waits for, and QK of warpgroup wq (-1: none) behind it
    auto ready = [&](int w, int wq) {
      bool r = mbar_try_wait(smem_u32(&s_pready[w][vb & 1]), (vb >> 1) & 1u);
      if (w == 0) r = mbar_try_wait(smem_u32(&s_full[S::kK + vst]), vph) && r;
      if (wq == 0) r = mbar_try_wait(smem_u32(&s_full[kst]), kph) && r;
      if (!__all_sync(0xffffffffu, r)) {
        if (w == 0) wait(s_full[S::kK + vst], vph);
        if (wq == 0) wait(s_full[kst], kph);
        wait(s_pready[w][vb & 1], (vb >> 1) & 1u);
      }
      tc_fence_after();
    };
    // scores of the next block of warpgroup w, each block's for both in turn
    auto qk = [&](int w, bool last) {
      const uint32_t kaddr = ring + kst * S::kBlock, qb = q_addr + (uint32_t)w * 16384u, to = tmem + 128u * (NB == 2 ? (uint32_t)w : kpl);
      tc_scores<D, kTile>(to, sdesc_k128(qb), sdesc_k128(kaddr), iq);
      tc_commit_elect(smem_u32(&s_sfull[w][kb & 1]));
      if (++kpl == NB) kpl = 0;
      if (w) {  // the slot is free once both have read it, and the segment's Q
        tc_commit_elect(smem_u32(&s_empty[kst]));
        if (last) tc_commit_elect(smem_u32(&s_qfree));
        if (++kst == S::kK) { kst = 0; kph ^= 1; }
        ++kb;
      }
    };
    auto pv = [&](int w, bool first, bool last, int steps) {
      const uint32_t vaddr = ring + (S::kK + vst) * S::kBlock, from = tmem + 128u * (NB == 2 ? (uint32_t)w : vpl), to = tmem + S::kO + (uint32_t)(w * D);
      if (steps == kKeys / 16) {
        tc_values<128>(to, from, sdesc_mn128(vaddr), iv, first ? 0u : 1u);
      } else {  // keys that no row of the tile sees, 16 at a time, take part in no product
#pragma unroll 1
        for (int ks = 0; ks < steps; ++ks)
          tc_mma_ts(to, from + (uint32_t)(8 * ks), sdesc_mn128(vaddr + (uint32_t)ks * 2048u), iv, (first && ks == 0) ? 0u : 1u);
      }
      if (last) tc_commit_elect(smem_u32(&s_odone[w]));
      if (++vpl == NB) vpl = 0;
      if (w) {
        tc_commit_elect(smem_u32(&s_empty[S::kK + vst]));
        if (++vst == S::kV) { vst = 0; vph ^= 1; }
        ++vb;
      }
    };
    while (ok && wk.next()) {
      const int n = wk.t1 - wk.t0, j0 = limit_of(wk.s, wk.t * L.pos) / kKeys - wk.t0;  // blocks from j0 on are cleaned
      wait(s_qfull, seg & 1u);
      ++seg;
      wait(s_full[kst], kph);
      tc_fence_after();
      if (!ok) break;
      qk(0, false);
      qk(1, n == 1);
      if (NB == 3 && n > 1) {
        wait(s_full[kst], kph);
        tc_fence_after();
        if (!ok) break;
        qk(0, false);
      }
      if (j0 <= 0 && lane == 0) mbar_arrive(smem_u32(&s_dirty));
      for (int j = 0; j < n; ++j) {  // the next scores right after a product freed their place
        const bool more = j + 1 < n, more2 = j + NB - 1 < n;
        int steps = kKeys / 16;
        if (j >= j0) {
          steps = steps_of(L, wk.s, wk.t, wk.t0 + j);
          wait(s_clean, cleaned & 1u);
          ++cleaned;
        }
        if (j + 1 >= j0 && more && ok && lane == 0) mbar_arrive(smem_u32(&s_dirty));
        ready(0, NB == 2 && more ? 0 : -1);
        if (!ok) break;
        pv(0, j == 0, j == n - 1, steps);
        if (more) qk(NB == 2 ? 0 : 1, j + 2 == n);
        ready(1, NB == 3 && more2 ? 0 : -1);
        if (!ok) break;
        pv(1, j == 0, j == n - 1, steps);
        if (more2) qk(NB == 2 ? 1 : 0, j + 2 == n);
      }
    }
    // every MMA issued has completed before tensor memory is released
    tc_commit_elect(smem_u32(&s_drain));
    volatile int never = 0;
    mbar_wait(smem_u32(&s_drain), 0u, p.err, DFV_DEVERR_DRAIN_WAIT, &never);
  } else {
    // ---------------------------------------------------------------- softmax and output
    const int w = warp >> 2, rr = tid & 255;  // warpgroup, and the thread's row of the tile
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_o = lane_base + S::kO + (uint32_t)(w * D);
    const float c = p.scale_log2;
    unsigned nt = 0;              // blocks this warpgroup has taken
    unsigned seg = 0, turn = (unsigned)w;  // segments it has put out; its place of scores
    const int g = head_of(L, rr), pi = rr - g * L.pos;
    bool ok = true, told = false;
    // after a wait gives up the loops still run to the end without touching
    // tensor memory
    while (wk.next()) {
      const int n = wk.t1 - wk.t0, i0 = wk.t * L.pos, i = i0 + pi, head = wk.h * p.G + g;
      const bool mine = g < p.G && i < wk.s.n;
      const int lim = mine ? limit_of(wk.s, i) : wk.s.nk, lim0 = limit_of(wk.s, i0);  // keys that this row, and every row, sees
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_sfull[w][nt & 1]), (nt >> 1) & 1u, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
        const unsigned b = nt++;
        const uint32_t t_s = lane_base + 128u * turn;
        turn = (turn + 2u) % NB;
        if (!ok) continue;
        tc_fence_after();
        // keys that no row of the tile sees take part in no product: neither do their 64
        bool both = true;
        if ((wk.t0 + j + 1) * kKeys > lim0) {
          both = steps_of(L, wk.s, wk.t, wk.t0 + j) > 4;
          mask_block(t_s, lim - (wk.t0 + j) * kKeys, both ? 128 : 64);
        }
        if (j == 0) {  // a maximum to begin with
          float s0[32], s1[32];
          tmem_ld32(t_s, s0);
          tmem_ld32(t_s + 32, s1);
          tmem_wait_ld32(s0);
          tmem_wait_ld32(s1);
          m = max32(s1, max32(s0, m));
        }
        // One pass with the M so far: p and the new maximum together, a quarter of the
        // scores read while the one before is used.
        uint32_t x[64];
        float2 l2;
        for (;;) {
          // (rounded up: the largest p stays within its bound however large the scores are)
          const float z = F16 ? base_of<true>(m, c) : m == -INFINITY ? 0.f : __fmul_ru(m, c);
          float s0[32], s1[32], mx = m;
          l2 = make_float2(0.f, 0.f);
          tmem_ld32(t_s, s0);
          tmem_wait_ld32(s0);
          tmem_ld32(t_s + 32, s1);
          mx = max32(s0, mx);
          exp32<F16>(s0, c, z, x, l2);
          tmem_wait_ld32(s1);
          if (both) tmem_ld32(t_s + 64, s0);
          mx = max32(s1, mx);
          exp32<F16>(s1, c, z, x + 16, l2);
          if (both) {
            tmem_wait_ld32(s0);
            tmem_ld32(t_s + 96, s1);
            mx = max32(s0, mx);
            exp32<F16>(s0, c, z, x + 32, l2);
            tmem_wait_ld32(s1);
            mx = max32(s1, mx);
            exp32<F16>(s1, c, z, x + 48, l2);
          }
          const bool grew = (mx - m) * c > 8.f;
          if (!__any_sync(0xffffffffu, grew)) break;
          if (!grew) mx = m;  // a row's M follows what the row sees, not its neighbours
          const float f = m == -INFINITY ? 0.f : ex2((m - mx) * c);
          l *= f;
          if (j > 0) {
            // the product of the block before: with two places it was issued before these
            // scores; with three its block of V is free once both have it
            if (NB == 3) {
              const unsigned last = b - 1;
              ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_empty[S::kK + last % S::kV]), (last / S::kV) & 1u, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
              tc_fence_after();
            }
            if (ok) {
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
          }
          m = mx;
        }
        l += l2.x + l2.y;
        tmem_st16(t_s, x);
        tmem_st16(t_s + 16, x + 16);
        if (both) {
          tmem_st16(t_s + 32, x + 32);
          tmem_st16(t_s + 48, x + 48);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(smem_u32(&s_pready[w][b & 1]));
      }
      // ---- output: after the last product of this warpgroup.  Its next product into O needs
      // its next P, which comes after these loads.
      ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(smem_u32(&s_odone[w]), seg & 1u, p.err, DFV_DEVERR_STAGE_WAIT, &s_abort));
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      const int bad = s_bad[seg & 3];
      const float z = F16 ? base_of<true>(m, c) : m == -INFINITY ? 0.f : __fmul_ru(m, c);
      const bool whole = wk.whole();
      const int slot = wk.slot(blockIdx.x);
      const size_t row = wk.s.row0 + (size_t)i;
      const float inv = l == 0.f ? 0.f : 1.f / l;  // NaN stays NaN
      char *out = p.o + 2 * ((long long)row * p.o_row + head * p.o_head);
      char *rows[4];  // of the four lanes
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const unsigned long long r = __shfl_sync(0xffffffffu, mine ? (unsigned long long)out : 0ull, (lane & 28) + e);
        rows[e] = (char *)r;
      }
      float4 *part = reinterpret_cast<float4 *>(L.part_o) + (size_t)slot * (D / 4) * kTile + rr;
#pragma unroll 1
      for (int q = 0; q < D && ok; q += 32) {
        float o[32];
        tmem_ld32(t_o + q, o);
        tmem_wait_ld32(o);
        if (whole) {
          uint4 x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[e] = make_uint4(pack2<F16>(o[8 * e] * inv, o[8 * e + 1] * inv), pack2<F16>(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                              pack2<F16>(o[8 * e + 4] * inv, o[8 * e + 5] * inv), pack2<F16>(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
          turn_quads(x);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (rows[e]) *reinterpret_cast<uint4 *>(rows[e] + 2 * q + 16 * (lane & 3)) = x[e];
        } else if (mine) {
          float4 *to = part + (size_t)(q / 4) * kTile;
#pragma unroll
          for (int e = 0; e < 8; ++e) to[(size_t)e * kTile] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      tc_fence_before();
      if (mine && ok) {
        if (whole) {
          if (p.lse) p.lse[row * p.H + head] = l == 0.f ? -INFINITY : (z + log2f(l)) * 0.69314718055994531f;
        } else {
          L.part_ml[(size_t)slot * kTile + rr] = make_float2(m == -INFINITY ? -INFINITY : z, l);
        }
      }
      if (whole && bad && ok) {
        __syncwarp();  // the row's pieces were stored by four lanes
        if (mine) add_taken<F16>(p, wk.s, wk.h, lim0, lim, out, 0, D);
      }
      if (MODE == kCut && tid == 0 && !whole) {
        L.part_bad[slot] = bad;
        if (wk.t0 == 0) {
          L.cut[blockIdx.x] = make_int4(wk.b, wk.h, wk.t, range_of(wk.last, s_start.U, s_start.G) - (int)blockIdx.x + 1);
          told = true;
        }
      }
      ++seg;
    }
    if (MODE == kCut && tid == 0 && !told) L.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- join
// A CTA joins 32 rows of the tile that begins in a range and goes on behind it: a
// lane per row, a warp per D / 8 elements of the head.  One pass in range order, four
// states' loads at once: with few rows over many keys a tile is in dozens of ranges (3 x 2
// rows behind 29412 keys 47 us in two passes, 32; sixteen warps and eight states 35, and 5
// more than these where tiles are in two ranges).
constexpr int kJoinWarps = 8, kJoinRows = 32, kJoinAhead = 4;

template <bool F16, int D>
__global__ void __launch_bounds__(32 * kJoinWarps, 2) prompt_join_kernel(const __grid_constant__ PromptLaunch L) {
  constexpr int kPer = D / 4 / kJoinWarps;  // float4 of a thread
  const PromptParams &p = L.p;
  const int g0 = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rr = blockIdx.y * kJoinRows + lane;
  pdl_trigger();
  pdl_wait();
  const int4 cut = __ldcg(&L.cut[g0]);
  const int n = cut.w;
  if (n < 2) return;
  const PromptSeq s = prompt_seq(p, cut.x);
  const int g = head_of(L, rr), i = cut.z * L.pos + rr - g * L.pos, head = cut.y * p.G + g;
  if (g >= p.G || i >= s.n) return;
  // state k is range g0 + k's; the tile goes on after the first and began before the others
  auto slot = [&](int k) { return (size_t)(2 * (g0 + k) + (k == 0)); };
  float4 x[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) x[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, l = 0.f;
  int bad = 0;
#pragma unroll 1
  for (int k0 = 0; k0 < n; k0 += kJoinAhead) {
    float2 ml[kJoinAhead];
    float4 y[kJoinAhead][kPer];
#pragma unroll
    for (int u = 0; u < kJoinAhead; ++u) {
      ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < kPer; ++e) y[u][e] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k0 + u < n) {
        const size_t at = slot(k0 + u);
        ml[u] = __ldcg(&L.part_ml[at * kTile + rr]);
        bad |= __ldcg(&L.part_bad[at]);
        const float4 *from = reinterpret_cast<const float4 *>(L.part_o) + (at * (D / 4) + warp * kPer) * kTile + rr;
#pragma unroll
        for (int e = 0; e < kPer; ++e) y[u][e] = __ldcg(from + (size_t)e * kTile);
      }
    }
    float top = M;
#pragma unroll
    for (int u = 0; u < kJoinAhead; ++u) top = fmaxf(top, ml[u].x);
    // a state without keys holds zeros (or NaN of a NaN query)
    auto weight = [&](float m) { return m == -INFINITY ? 1.f : ex2(m - top); };
    auto join = [&](float f, float with, float4 *z, float m) {  // this so far times `with`, and a state times f
      l = fmaf(m, f, l * with);
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        x[e].x = fmaf(z[e].x, f, x[e].x * with);
        x[e].y = fmaf(z[e].y, f, x[e].y * with);
        x[e].z = fmaf(z[e].z, f, x[e].z * with);
        x[e].w = fmaf(z[e].w, f, x[e].w * with);
      }
    };
#pragma unroll
    for (int u = 0; u < kJoinAhead; ++u) join(weight(ml[u].x), u == 0 ? weight(M) : 1.f, y[u], ml[u].y);
    M = top;
  }
  const size_t row = s.row0 + (size_t)i;
  const float inv = l == 0.f ? 0.f : 1.f / l;  // NaN stays NaN
  char *out = p.o + 2 * ((long long)row * p.o_row + head * p.o_head);
#pragma unroll
  for (int e = 0; e < kPer; ++e)
    reinterpret_cast<uint2 *>(out)[warp * kPer + e] = make_uint2(pack2<F16>(x[e].x * inv, x[e].y * inv), pack2<F16>(x[e].z * inv, x[e].w * inv));
  if (bad) add_taken<F16>(p, s, cut.y, limit_of(s, cut.z * L.pos), limit_of(s, i), out, 4 * warp * kPer, 4 * (warp + 1) * kPer);
  if (p.lse && warp == 0) p.lse[row * p.H + head] = l == 0.f ? -INFINITY : (M == -INFINITY ? l : (M + log2f(l)) * 0.69314718055994531f);
}

bool encode_rows(CUtensorMap *map, const PromptParams &p, const char *base, int n, int heads, long long row, long long head,
                 int box_rows, int box_heads, char *why, size_t why_len) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn(why, why_len);
  if (!fn) return false;
  // a dimension of one entry has no stride of its own
  const cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)n, (cuuint64_t)heads};
  const cuuint64_t strides[2] = {n > 1 ? (cuuint64_t)row * 2 : 16, heads > 1 ? (cuuint64_t)head * 2 : 16};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_heads};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult e = fn(map, p.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                        const_cast<char *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (e != CUDA_SUCCESS) {
    snprintf(why, why_len, "tensor map of the queries, keys or values refused (%d)", (int)e);
    return false;
  }
  return true;
}

template <bool F16, int D, int MODE>
cudaError_t launch_kernel(const PromptLaunch &L, int ctas, cudaStream_t s) {
  auto kern = prompt_attn_kernel<F16, D, MODE>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kern, PromptShape<D>::kSmem, done);
  if (e != cudaSuccess) return e;
  return launch_chained(kern, dim3(ctas), dim3(kThreads), PromptShape<D>::kSmem, s, L);
}

template <bool F16, int D>
cudaError_t launch_typed(const PromptLaunch &L, cudaStream_t s) {
  // at most so many tiles (a sequence's last one may be short)
  const long long tiles = (long long)L.p.Hkv * (L.p.n_rows / L.pos + L.p.n_seqs);
  const long long longest = kOver + (L.p.max_keys + kKeys - 1) / kKeys;
  if (L.p.max_keys <= kWholeKeys || 4 * tiles >= 3 * kAttnCtas * longest) {
    if (tiles <= kAttnCtas) return launch_kernel<F16, D, kOne>(L, (int)tiles, s);
    return launch_kernel<F16, D, kWhole>(L, kAttnCtas, s);
  }
  const cudaError_t e = launch_kernel<F16, D, kCut>(L, kAttnCtas, s);
  if (e != cudaSuccess) return e;
  return launch_chained(prompt_join_kernel<F16, D>, dim3(kAttnCtas, kTile / kJoinRows), dim3(32 * kJoinWarps), 0, s, L);
}

}  // namespace

size_t prompt_attn_ws(int D) { return sections(nullptr, D, nullptr); }

cudaError_t launch_prompt_attn(const PromptParams &p, void *ws, cudaStream_t s, char *why, size_t why_len) {
  static thread_local PromptLaunch L;
  L.p = p;
  // positions of a tile: a multiple of 8, so that each head's rows begin on a 1024-byte
  // boundary of the swizzled tile
  L.pos = kTile / p.G & ~7;
  int gcd = 8;
  while (gcd < kKeys && L.pos % (2 * gcd) == 0) gcd *= 2;
  L.run = kKeys / gcd;
  L.rise = L.pos / gcd;
  L.inv_pos = (65536u + L.pos - 1) / L.pos;
  sections(&L, p.D, ws);
  const int box = p.D == 128 ? kKeys : kKeys / 2;
  if (!encode_rows(&L.tm_q, p, p.q, p.n_rows, p.H, p.q_row, p.q_head, L.pos, p.G, why, why_len) ||
      !encode_rows(&L.tm_k, p, p.k, p.n_keys, p.Hkv, p.k_row, p.k_head, box, 1, why, why_len) ||
      !encode_rows(&L.tm_v, p, p.v, p.n_keys, p.Hkv, p.v_row, p.v_head, box, 1, why, why_len))
    return cudaErrorInvalidValue;
  if (p.D == 128) return p.f16 ? launch_typed<true, 128>(L, s) : launch_typed<false, 128>(L, s);
  return p.f16 ? launch_typed<true, 64>(L, s) : launch_typed<false, 64>(L, s);
}

}  // namespace dfv
