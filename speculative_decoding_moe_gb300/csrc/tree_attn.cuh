// tree_attn.cuh -- what the attention kernels share: the cut of the work line
// into ranges, the walk over a range's segments, and how states and outputs
// are stored.
#pragma once

#include "tree_common.cuh"

namespace dfv {

struct AttnLaunch {
  CUtensorMap tm_k, tm_v;  // one layer's pages: {head_dim, token, head, page}, token and head in stride order
  TreeAttnParams p;
  int rows;      // rows (nodes x heads of a kv head) per CTA
  int n_rt;      // CTAs per range, for further rows
  int n_groups;  // ranges
  int swap;      // head before token in the tensor maps
  uint32_t inv_g;  // ceil(2^16 / G)
  int2 *pairs;        // [n_seqs][kv heads] of each pair: first range, ranges
  float2 *part_ml;    // [2 CTAs][rows] (M, l) of partial states
  float *part_o;      // [2 CTAs][D / 4][rows][4] their sums of p v
  int *part_bad;      // [2 CTAs] a tree value that is not finite was left out
};

cudaError_t launch_attn_tc(const AttnLaunch &L, cudaStream_t s);  // tree_attn_tc.cu: rows 128 or 256

// Sections of the attention workspace; returns its size.  Places for the states of
// kAttnCtas CTAs whatever the plan (n_groups * n_rt of them run, a few less where n_rt
// does not divide): a workspace for large trees is then enough for smaller ones.
inline size_t attn_sections(AttnLaunch *L, const AttnPlan &a, int n_seqs, int Hkv, int D, void *ws) {
  const size_t slots = 2 * (size_t)kAttnCtas;
  size_t off = kWsScratch;
  auto take = [&](size_t n) {
    void *q = ws ? (void *)((char *)ws + off) : nullptr;
    off += (n + 255) & ~(size_t)255;
    return q;
  };
  int2 *pairs = (int2 *)take((size_t)n_seqs * Hkv * 8);
  int *bad = (int *)take(slots * 4);
  float2 *ml = (float2 *)take(slots * a.rows * 8);
  float *o = (float *)take(slots * a.rows * D * 4);
  if (L) {
    L->pairs = pairs;
    L->part_bad = bad;
    L->part_ml = ml;
    L->part_o = o;
  }
  return off;
}

// Node of row r: r / G for r < 1024 + 256 and G <= 16 (the product's error stays
// below one part in 2^16 / G).
__device__ __forceinline__ int node_of(const AttnLaunch &L, int r) { return (int)(((uint32_t)r * L.inv_g) >> 16); }

// ---------------------------------------------------------------- the work line
// Sequence b's units are its kv heads' pairs one after the other: V units for
// what a pair costs however long it is (queries, the first scores, the output;
// without them the ranges of many short pieces ended last), then its key tiles.
// A pair without keys has one tile (its outputs have to be written), a sequence
// without rows no unit.  Range g of G over U units is [g U / G, (g + 1) U / G);
// there are no more ranges than units.
struct SchedStart {
  long long u0, u1, base;  // the range, and the first unit of sequence b
  long long U;             // units, and ranges in use
  int b, G;
};

// Ranges in use.
__device__ __forceinline__ int ranges_of(long long U, int n_groups) {
  return U >= n_groups ? n_groups : U > 0 ? (int)U : 1;
}
// (32-bit divisions while the products fit: a 64-bit one takes a few hundred cycles)
__device__ __forceinline__ long long group_start(int g, long long U, int G) {
  return U < (1 << 24) ? (long long)((uint32_t)g * (uint32_t)U / (uint32_t)G) : g * U / G;
}
__device__ __forceinline__ int group_of(long long u, long long U, int G) {
  return U < (1 << 24) ? (int)((((uint32_t)u + 1u) * (uint32_t)G - 1u) / (uint32_t)U) : (int)(((u + 1) * G - 1) / U);
}

template <int KT, int V>
__device__ __forceinline__ long long seq_units(const AttnLaunch &L, int b) {
  const SeqView v = seq_view(L.p.c, L.p.t, b);
  if (v.n == 0) return 0;
  const int total = v.s < 0 ? 0 : v.len + v.n;
  return (long long)L.p.c.Hkv * (V + (total > 0 ? (total + KT - 1) / KT : 1));
}

// The range of CTA `block` and the sequence it starts in.  All NT threads of
// the CTA call it; s_scan holds NT / 32 values.
template <int NT, int KT, int V>
__device__ __forceinline__ void sched_start(const AttnLaunch &L, int block, long long *s_scan, SchedStart *out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = L.p.t.n_seqs;
  const int per = (n + NT - 1) / NT, b0 = min(n, tid * per), b1 = min(n, b0 + per);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) sum += seq_units<KT, V>(L, b);
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
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) at += s_scan[w];
    U += s_scan[w];
  }
  const int g = block / L.n_rt, G = ranges_of(U, L.n_groups);
  const long long u0 = group_start(g, U, G), u1 = g < G ? group_start(g + 1, U, G) : u0;
  if (u0 < u1 && at <= u0 && u0 < at + sum) {
    long long base = at;
    for (int b = b0; b < b1; ++b) {
      const long long c = per == 1 ? sum : seq_units<KT, V>(L, b);
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

// Segments of a range: tiles [t0, t1) of one (sequence, kv head).
template <int KT, int V>
struct SegWalk {
  const AttnLaunch &L;
  const long long end;
  long long u, base;
  int b, h, t0, t1, T, total;
  int nodes;  // of the sequence in the cache: none where the cache side is unusable
  long long last;  // last unit of the pair
  SeqView v;
  __device__ __forceinline__ SegWalk(const AttnLaunch &l, const SchedStart &s)
      : L(l), end(s.u1), u(s.u0), base(s.base), b(s.b) {}
  __device__ __forceinline__ bool next() {
    while (u < end) {
      v = seq_view(L.p.c, L.p.t, b);
      nodes = v.s < 0 ? 0 : v.n;
      total = v.len + nodes;
      T = v.n == 0 ? 0 : total > 0 ? (total + KT - 1) / KT : 1;
      const int pair = T + V;  // units
      const long long w = u - base, units = v.n == 0 ? 0 : (long long)L.p.c.Hkv * pair;
      if (w < units) {
        h = (units >> 31) ? (int)(w / pair) : (int)((uint32_t)w / (uint32_t)pair);
        const int p0 = (int)(w - (long long)h * pair), p1 = (int)min((long long)pair, p0 + (end - u));
        last = u - p0 + pair - 1;
        u += p1 - p0;
        t0 = max(0, p0 - V);
        t1 = max(0, p1 - V);
        if (t0 < t1) return true;
        continue;  // the range ends before the pair's first tile
      }
      base += units;
      ++b;
    }
    return false;
  }
  // The nodes that row r sees.
  __device__ __forceinline__ uint64_t mask_of(int r) const {
    if (nodes == 0) return 0;
    return row_mask(L.p.t, v.row0, node_of(L, r)) & (nodes >= 64 ? ~0ull : (1ull << nodes) - 1ull);
  }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == T; }
  // For the join: one thread of the range that holds the pair's first tile tells
  // which ranges share it.
  __device__ __forceinline__ void tell(const SchedStart &s, int block) const {
    if (t0 || block % L.n_rt) return;
    const int g = block / L.n_rt;
    L.pairs[b * L.p.c.Hkv + h] = make_int2(g, whole() ? 1 : group_of(last, s.U, s.G) - g + 1);
  }
  // Partial states of a range: of a pair that began before it, and of one that
  // goes on after it.
  __device__ __forceinline__ int slot(int block) const { return 2 * block + (t0 == 0); }
};

// ---------------------------------------------------------------- pieces
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A page id as read from the table; one out of range is read as page 0.
__device__ __forceinline__ int checked_page(const CacheParams &c, int pg) {
  if ((unsigned)pg < (unsigned)c.n_pages) return pg;
  flag_err(c.err, DFV_KVERR_PAGE);
  return 0;
}

// One page's box of a tile, issued by an elected lane of a warp in step.  (With a
// lane per page the compiler issued the lanes' copies one after the other, each
// after moving its operands to uniform registers: 16-token pages were bound by
// that.)
__device__ __forceinline__ void tma_kv(uint32_t dst, const CUtensorMap *map, int x, int tok, int h, int pg, int swap,
                                       uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];\n}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(swap ? h : tok), "r"(swap ? tok : h), "r"(pg), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// Values of keys j (low half) and j + 1, j counted from the tree's first node:
// zero past the last node; a node's value that is not finite becomes zero and
// sets *bad.
template <bool F16>
__device__ __forceinline__ uint32_t clean_pair(uint32_t v, int j, int n, bool *bad) {
  constexpr uint32_t kExp = F16 ? 0x7c00u : 0x7f80u;
  if (j >= n) v &= 0xffff0000u;
  if (j + 1 >= n) v &= 0x0000ffffu;
  if (j >= 0 && (v & kExp) == kExp) {
    v &= 0xffff0000u;
    *bad = true;
  }
  if (j + 1 >= 0 && (v & (kExp << 16)) == (kExp << 16)) {
    v &= 0x0000ffffu;
    *bad = true;
  }
  return v;
}

// What clean_pair took out of element d of the values that node i sees.
template <bool F16>
__device__ __noinline__ float unseen(const TreeAttnParams &p, const SeqView &v, int i, int h, int d) {
  if (v.s < 0) return 0.f;
  const uint64_t mask = row_mask(p.t, v.row0, i);
  float x = 0.f;
  for (int j = 0; j < v.n; ++j) {
    if (!((mask >> j) & 1)) continue;
    const int pos = v.len + j;
    const int pg = checked_page(p.c, p.c.table[(size_t)v.s * p.c.max_pages + (pos >> p.c.page_shift)]);
    const long long off = kv_off(p.c, p.layer, pg, h, pos & ((1 << p.c.page_shift) - 1)) + d;
    const uint32_t w = reinterpret_cast<const uint16_t *>(p.c.v)[off];
    const float y = unpack2<F16>(w).x;
    if (!isfinite(y)) x += y;
  }
  return x;
}

// unseen() added to elements c0 .. c1 of a stored output (rare: a value in the
// tree is not finite).
template <bool F16>
__device__ __noinline__ void add_unseen(const TreeAttnParams &p, const SeqView &v, int i, int h, char *out, int c0,
                                        int c1) {
  uint32_t *w = reinterpret_cast<uint32_t *>(out);
#pragma unroll 1
  for (int d = c0; d < c1; d += 2) {
    float2 x = unpack2<F16>(w[d / 2]);
    x.x += unseen<F16>(p, v, i, h, d);
    x.y += unseen<F16>(p, v, i, h, d + 1);
    w[d / 2] = pack2<F16>(x.x, x.y);
  }
}

// Output piece e (8 elements) of row r: x / l, and lse = (z + log2 l) ln 2.
template <bool F16>
__device__ __forceinline__ void store_out(const AttnLaunch &L, const SeqView &v, int r, int h, int e, const float *x,
                                          float z, float l, int bad) {
  const TreeAttnParams &p = L.p;
  const int i = node_of(L, r), head = h * p.G + r - i * p.G;
  const size_t row = v.row0 + i;
  const float inv = l == 0.f ? 0.f : 1.f / l;  // NaN stays NaN
  char *out = p.o + 2 * (row * p.o_row + head * p.o_head);
  *reinterpret_cast<uint4 *>(out + 16 * e) =
      make_uint4(pack2<F16>(x[0] * inv, x[1] * inv), pack2<F16>(x[2] * inv, x[3] * inv),
                 pack2<F16>(x[4] * inv, x[5] * inv), pack2<F16>(x[6] * inv, x[7] * inv));
  if (bad) add_unseen<F16>(p, v, i, h, out, 8 * e, 8 * e + 8);
  if (e == 0 && p.lse) p.lse[row * p.H + head] = l == 0.f ? -INFINITY : (z + log2f(l)) * 0.69314718055994531f;
}

}  // namespace dfv
