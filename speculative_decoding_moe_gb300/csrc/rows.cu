// rows.cu -- rows into the paged cache and back: norms of queries and keys for
// each head, rotary positions and the append in one launch, for any number of
// rows and for caches in 16 bits or in e4m3 codes; and cached tokens as packed
// rows.
//
// Mathematics.  n(x) = x / sqrt(mean(x^2) + eps) * gain over a head, then each pair
// turned by the angle position * f_i.  The angle is kept as a 64-bit fraction of a
// turn: position * turns in wrapping integers is exact, and its upper 32 bits,
// read as signed, go to sincospi.  Codes: e is the smallest integer with
// max |y| <= 448 * 2^e, found from the bits of the maximum (448 = 1.75 * 2^8), so
// that y * 2^-e is exact and the code's rounding (to nearest, ties to even) is
// the only one after fp32.  A power of two loses nothing against a scale of 24 bits
// but range: e4m3 is a floating format, and its steps are relative.
//
// Both kernels are bound by memory: a row is read and written once.  A head is 16
// elements a lane, in two 16-byte pieces of which one lane holds both sides of
// its pairs (half layout: pieces half a rotation apart), so that the sums and
// maxima over a head are shuffles within D / 16 lanes.  Append: a warp takes a row (or
// a share of one, while there are few), finds the sines and cosines once for all its
// heads, and walks the heads one at a time in a short loop with the next three on
// their way by asynchronous copies into places of its lanes' own.
//
// Measured (GB300, device time): 8 prompts of up to 2039 rows of 32 + 2 x 4 heads of
// 128, normed and turned, 46 us, 5.6 TB/s; into codes and back, 4 x 1021 rows of 32 + 2 x
// 8 heads of 64 and the 17402 tokens of each, 47 us, 5.1 TB/s; one row 3 us.  Steps of
// the first: four items loaded to registers at once, heads of several rows in turn 59
// (fewer at once 94 to 103; fetching the unrolled items' instructions took longer than
// what more loads at once gained); a warp a row, four items at once 62 to 66; by
// asynchronous copies, four items a turn 58, two 50, one 48, without a division a head 46.
#include <cfloat>

#include "tree_common.cuh"

namespace dfv {
namespace {

constexpr int kRowThreads = 256;
constexpr int kMaxRowsCta = 8;  // append: rows of a CTA, a warp each
constexpr int kAhead = 3, kPlaces = 4;  // append: items of a lane on their way, and places for them
constexpr int kReadRows = 32;     // read: rows of a CTA
constexpr int kReadAhead = 4;

struct AppendLaunch {
  RopeParams p;
  int rows;     // log2 of a CTA's
  int by_seq;   // rows are counted as (sequence, row of it) with max_nodes each
  int lanes;    // log2 of the lanes of a head
  float inv_d;  // 1 / head_dim
};
struct ReadLaunch {
  CacheReadParams p;
  int rows, lanes;
};

// log2 of the lanes that hold a head of D elements, 16 each
int head_lanes(int D) {
  int l = 0;
  while ((16 << l) < D) ++l;
  return l;
}

// a's code in the low byte, b's above it; what is not finite must be NaN by now
__device__ __forceinline__ uint32_t codes_of(float a, float b) {
  uint32_t r;
  asm("{\n .reg .b16 x;\n cvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n cvt.u32.u16 %0, x;\n}" : "=r"(r) : "f"(a), "f"(b));
  return r;
}
// e of a maximum that is finite
__device__ __forceinline__ int exponent_of(float top) {
  const uint32_t b = __float_as_uint(top);
  const int e = (int)(b >> 23) - 135 + ((b & 0x7fffffu) > 0x600000u);
  return e < -100 ? -100 : e;  // 120 at most: the largest finite value
}

// Pieces of 8 elements that lane `lid` holds of a head of 2 n pieces.
__device__ __forceinline__ int2 pieces_of(int lid, int n, int r16, bool halves) {
  if (!halves) return make_int2(lid, lid + n);
  if (lid < r16) return make_int2(lid, lid + r16);
  return make_int2(lid + r16, lid + n);  // behind the turned ones: 2 r16 + (lid - r16), and n - r16 further
}

// two at a time
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

template <bool F16>
__device__ __forceinline__ void widen(const uint4 &a, float2 *x) {
  const uint32_t *w = &a.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = unpack2<F16>(w[i]);
}
template <bool F16>
__device__ __forceinline__ uint4 narrow(const float2 *x) {
  return make_uint4(pack2<F16>(x[0].x, x[0].y), pack2<F16>(x[1].x, x[1].y), pack2<F16>(x[2].x, x[2].y), pack2<F16>(x[3].x, x[3].y));
}

__device__ __forceinline__ void copy16(uint32_t to, const char *from, bool have) {  // zeros if not
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(have ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t from) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(from) : "memory");
  return v;
}

// NORM: some gain is given.  INTER: pairs are neighbours.
template <bool F16, bool CODES, bool NORM, bool INTER>
__global__ void __launch_bounds__(kRowThreads, 3) append_kernel(const __grid_constant__ AppendLaunch L) {
  __shared__ __align__(16) float s_cos[kMaxRowsCta][128], s_sin[kMaxRowsCta][128];
  __shared__ int s_row[kMaxRowsCta], s_page[kMaxRowsCta], s_tok[kMaxRowsCta];
  const RopeParams &p = L.p;
  const CacheParams &c = p.c;
  const int tid = threadIdx.x, rows = 1 << L.rows, first = blockIdx.x << L.rows, HK = p.H + c.Hkv, NH = HK + c.Hkv;
  // The CTA's threads are split among its rows; a row's groups of lanes take its heads in
  // turn, queries first, then keys, then values.
  const int lid = tid & ((1 << L.lanes) - 1), group = tid >> L.lanes, share = 8 - L.lanes - L.rows;  // log2 of a row's groups
  const int j = group >> share, head0 = group & ((1 << share) - 1), step = 1 << share;
  const int n16 = c.D / 16, r16 = p.rot / 16;
  const bool on = lid < n16;
  // pieces of a turned head, and of one that is copied
  const int2 at_turned = pieces_of(lid, n16, r16, !INTER), at_plain = make_int2(lid, lid + n16);
  pdl_trigger();
  pdl_wait();

  // Items on their way to this lane, in two pieces each, in places of its own.
  extern __shared__ __align__(16) unsigned char sm_x[];
  const uint32_t mine = smem_u32(sm_x) + 16u * tid;
  auto place = [&](int at, int piece) { return mine + (uint32_t)((2 * at + piece) * 16 * kRowThreads); };
  auto load = [&](int to, int row, int h) {
    if (on && h < NH) {
      const bool have = (unsigned)row < (unsigned)p.t.n_rows;
      const char *src = h < p.H ? p.q + 2 * (row * p.q_row + h * p.q_head)
                                : h < HK ? p.k + 2 * (row * p.k_row + (h - p.H) * p.k_head) : p.v + 2 * (row * p.v_row + (h - HK) * p.v_head);
      const int2 at = h < HK ? at_turned : at_plain;
      if (!have) src = p.q;
      copy16(place(to, 0), src + 16 * at.x, have);
      copy16(place(to, 1), src + 16 * at.y, have);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto load_first = [&](int row) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(i, row, head0 + i * step);
  };
  if (!L.by_seq) load_first(first + j);

  // ---- whose rows, and where they go (one warp: a chain of reads)
  if (tid < rows) {
    const int v = first + tid;
    int row = -1, pg = -1, tok = 0, b = -1;
    if (L.by_seq) {
      b = v / p.t.max_nodes;
      if (b >= p.t.n_seqs) b = -1;
    } else if (v < p.t.n_rows) {
      b = owner_of(p.t, v);
    }
    if (b >= 0) {
      const SeqView s = seq_view(c, p.t, b);
      const int i = L.by_seq ? v - b * p.t.max_nodes : v - s.row0;
      if (i >= 0 && i < s.n) {
        row = s.row0 + i;
        if (s.s >= 0) {
          pg = page_of(c, s.s, s.len + i);
          tok = (s.len + i) & ((1 << c.page_shift) - 1);
        }
      }
    }
    s_row[tid] = row;
    s_page[tid] = pg;
    s_tok[tid] = tok;
  }
  if (L.by_seq) {
    __syncthreads();
    load_first(s_row[j]);
  }
  // ---- sines and cosines, once for all heads (the other warps)
  for (int u = tid - 32; u < (p.rot / 2) << L.rows && tid >= 32; u += kRowThreads - 32) {
    const int r = u / (p.rot / 2), i = u - r * (p.rot / 2), row = L.by_seq ? s_row[r] : first + r;
    if ((unsigned)row >= (unsigned)p.t.n_rows) continue;
    const uint64_t turn = (uint64_t)(long long)p.positions[row] * p.turns[i];
    float sn, cs;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn, &cs);
    s_cos[r][i] = cs * p.scale;
    s_sin[r][i] = sn * p.scale;
  }
  __syncthreads();
  const int row = s_row[j], pg = s_page[j], tok = s_tok[j];
  // this lane's eight pairs: of its first piece's elements (half layout), or of both pieces
  float2 cs[4], sn[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int at = INTER ? 2 * ((e < 2 ? at_turned.x : at_turned.y) * 2 + (e & 1)) : 8 * lid + 2 * e;
    cs[e] = make_float2(1.f, 1.f);
    sn[e] = make_float2(0.f, 0.f);
    if (2 * at < p.rot) {
      cs[e] = *reinterpret_cast<const float2 *>(&s_cos[j][at]);
      sn[e] = *reinterpret_cast<const float2 *>(&s_sin[j][at]);
    }
  }
  float2 g[8];  // the gain of this lane's elements: queries' first, then keys'
  auto gains = [&](const char *from) {
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = make_float2(1.f, 1.f);
    if (from && on) {
      widen<F16>(__ldg(reinterpret_cast<const uint4 *>(from) + at_turned.x), g);
      widen<F16>(__ldg(reinterpret_cast<const uint4 *>(from) + at_turned.y), g + 4);
    }
  };
  bool of_q = head0 < p.H;
  if (NORM) gains(of_q ? p.q_gain : p.k_gain);

  int at_x = 0;
#pragma unroll 1
  for (int h0 = 0; h0 < NH; h0 += step) {  // the same for all threads
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    const int h = h0 + head0;
    const bool have = h < NH && on && row >= 0, isq = h < p.H, turned = h < HK;
    const int2 at = turned ? at_turned : at_plain;
    uint4 x0 = make_uint4(0u, 0u, 0u, 0u), x1 = x0;
    if (on && h < NH) {
      x0 = lds128(place(at_x, 0));
      x1 = lds128(place(at_x, 1));
    }
    load((at_x + kAhead) % kPlaces, row, h + kAhead * step);  // where the item before was
    at_x = (at_x + 1) % kPlaces;
    if (!CODES && !turned) {  // values as they are
      if (have && pg >= 0) {
        uint4 *to = reinterpret_cast<uint4 *>(c.v + 2 * kv_off(c, p.layer, pg, h - HK, tok));
        to[at.x] = x0;
        to[at.y] = x1;
      }
      if (!NORM || h0 >= HK) continue;  // (with norms the warp's other heads sum over shuffles)
    }
    float2 a[4], b[4];
    widen<F16>(x0, a);
    widen<F16>(x1, b);
    if (NORM) {
      if (of_q && !isq) {
        of_q = false;
        gains(p.k_gain);
      }
      float2 s2 = mul2(a[0], a[0]), s3 = mul2(b[0], b[0]);
#pragma unroll
      for (int e = 1; e < 4; ++e) {
        s2 = fma2(a[e], a[e], s2);
        s3 = fma2(b[e], b[e], s3);
      }
      float ss = (s2.x + s2.y) + (s3.x + s3.y);
      for (int o = 1 << L.lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (turned && (isq ? p.q_gain : p.k_gain)) {
        const float2 inv = both(rsqrtf(fmaf(ss, L.inv_d, p.eps)));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a[e] = mul2(mul2(a[e], inv), g[e]);
          b[e] = mul2(mul2(b[e], inv), g[4 + e]);
        }
      }
    }
    if (turned) {
      if (INTER) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float2 &y = e < 4 ? a[e] : b[e - 4];
          const float2 c2 = cs[e / 2], s2 = sn[e / 2];
          if ((e < 4 ? at.x : at.y) < 2 * r16) y = fma2(make_float2(-y.y, y.x), both(e & 1 ? s2.y : s2.x), mul2(y, both(e & 1 ? c2.y : c2.x)));
        }
      } else if (lid < r16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 a0 = a[e];
          a[e] = fma2(make_float2(-b[e].x, -b[e].y), sn[e], mul2(a0, cs[e]));
          b[e] = fma2(a0, sn[e], mul2(b[e], cs[e]));
        }
      }
    }
    auto put = [&](char *to_row) {
      uint4 *to = reinterpret_cast<uint4 *>(to_row);
      to[at.x] = narrow<F16>(a);
      to[at.y] = narrow<F16>(b);
    };
    if (CODES && have && turned) {  // rows as they are, whatever becomes of them in codes
      if (isq) put(p.o + 2 * (row * p.o_row + h * p.o_head));
      if (!isq && p.ko) put(p.ko + 2 * (row * p.ko_row + (h - p.H) * p.ko_head));
    }
    float top = 0.f;
    if (CODES) {  // of the finite elements; the others become NaN
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float2 *y = q ? b : a;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!(fabsf(y[e].x) <= FLT_MAX)) y[e].x = NAN;
          if (!(fabsf(y[e].y) <= FLT_MAX)) y[e].y = NAN;
          top = fmaxf(top, fmaxf(fabsf(y[e].x), fabsf(y[e].y)));  // fmaxf passes NaN over
        }
      }
      for (int o = 1 << L.lanes >> 1; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    if (!have) continue;
    if (isq) {
      if (!CODES) put(p.o + 2 * (row * p.o_row + h * p.o_head));
      continue;
    }
    if (!CODES && turned && p.ko) put(p.ko + 2 * (row * p.ko_row + (h - p.H) * p.ko_head));
    if (pg < 0) continue;
    if (CODES) {
      const int kh = turned ? h - p.H : h - HK;
      const int e = exponent_of(top);
      const float f = exp_value((uint32_t)(127 - e));
      uint2 *to = reinterpret_cast<uint2 *>((turned ? c.k : c.v) + kv_off(c, p.layer, pg, kh, tok));
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float2 *y = q ? b : a;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], both(f));
        to[q ? at.y : at.x] = make_uint2(codes_of(y[0].x, y[0].y) | codes_of(y[1].x, y[1].y) << 16,
                                         codes_of(y[2].x, y[2].y) | codes_of(y[3].x, y[3].y) << 16);
      }
      if (lid == 0) (turned ? c.ke : c.ve)[exp_off(c, p.layer, pg, kh, tok)] = (uint8_t)(e + 127);
    } else if (turned) {
      uint4 *to = reinterpret_cast<uint4 *>(c.k + 2 * kv_off(c, p.layer, pg, h - p.H, tok));
      to[at.x] = narrow<F16>(a);
      to[at.y] = narrow<F16>(b);
    }
  }
}

// ---------------------------------------------------------------- read
template <bool CODES>
__global__ void __launch_bounds__(kRowThreads) read_kernel(const __grid_constant__ ReadLaunch L) {
  __shared__ int s_page[kReadRows], s_tok[kReadRows];
  const CacheReadParams &p = L.p;
  const CacheParams &c = p.c;
  const int tid = threadIdx.x, first = blockIdx.x * L.rows;
  const int lid = tid & ((1 << L.lanes) - 1), group = tid >> L.lanes, groups = kRowThreads >> L.lanes, n16 = c.D / 16;
  pdl_trigger();
  pdl_wait();
  if (tid < L.rows) {
    const int r = first + tid;
    int pg = -2, tok = 0;  // -2: nobody's row, -1: zeros
    if (r < p.t.n_rows) {
      const int b = owner_of(p.t, r);
      const int r0 = p.t.row_off[b], r1 = p.t.row_off[b + 1], s = p.t.seq ? p.t.seq[b] : b, i = r - r0;
      if (r0 < 0 || r1 > p.t.n_rows || r1 - r0 > p.t.max_nodes) {
        flag_err(c.err, DFV_KVERR_LEN);
      } else if (i >= 0 && r < r1) {
        pg = -1;
        tok = i & ((1 << c.page_shift) - 1);
        if ((unsigned)s >= (unsigned)c.max_seqs)
          flag_err(c.err, DFV_KVERR_SEQ);
        else if ((long long)i >= ((long long)c.max_pages << c.page_shift))
          flag_err(c.err, DFV_KVERR_LEN);
        else
          pg = page_of(c, s, i);
      }
    }
    s_page[tid] = pg;
    s_tok[tid] = tok;
  }
  __syncthreads();
  if (lid >= n16) return;
  // Items: side (keys, values) and head w of the CTA's row j; a lane's next one is
  // `groups` further
  const int sides = (p.k ? 1 : 0) + (p.v ? 1 : 0), per = sides * c.Hkv, items = L.rows * per;
  const int dj = groups / per, dw = groups - dj * per;
  int lj = group / per, lw = group - lj * per, cj = lj, cw = lw;
  for (int done = group; done < items; done += kReadAhead * groups) {
    uint4 x[kReadAhead][2];
    uint32_t e[kReadAhead];
#pragma unroll
    for (int u = 0; u < kReadAhead; ++u) {
      x[u][0] = x[u][1] = make_uint4(0u, 0u, 0u, 0u);
      e[u] = 127u;
      const int pg = lj < L.rows ? s_page[lj] : -1;
      if (pg >= 0) {
        const bool isk = p.k && lw < c.Hkv;
        const int h = lw < c.Hkv ? lw : lw - c.Hkv;
        const char *src = (isk ? c.k : c.v) + (kv_off(c, p.layer, pg, h, s_tok[lj]) << c.esh);
        if (CODES) {
          const uint2 a = reinterpret_cast<const uint2 *>(src)[lid], b = reinterpret_cast<const uint2 *>(src)[lid + n16];
          x[u][0] = make_uint4(a.x, a.y, b.x, b.y);
          e[u] = (isk ? c.ke : c.ve)[exp_off(c, p.layer, pg, h, s_tok[lj])];
        } else {
          x[u][0] = reinterpret_cast<const uint4 *>(src)[lid];
          x[u][1] = reinterpret_cast<const uint4 *>(src)[lid + n16];
        }
      }
      lj += dj;
      lw += dw;
      if (lw >= per) { lw -= per; ++lj; }
    }
#pragma unroll
    for (int u = 0; u < kReadAhead; ++u) {
      const int j = cj, w = cw;
      cj += dj;
      cw += dw;
      if (cw >= per) { cw -= per; ++cj; }
      if (j >= L.rows || s_page[j] == -2) continue;
      const bool isk = p.k && w < c.Hkv;
      const int h = w < c.Hkv ? w : w - c.Hkv;
      const long long row = first + j;
      uint4 *to = reinterpret_cast<uint4 *>(isk ? p.k + 2 * (row * p.k_row + h * p.k_head) : p.v + 2 * (row * p.v_row + h * p.v_head));
      if (CODES) {
        const float f = exp_value(e[u]);
        const uint32_t *codes = &x[u][0].x;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float2 y[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            y[2 * i] = mul2(unpack2<true>(codes_f16(codes[2 * q + i])), both(f));
            y[2 * i + 1] = mul2(unpack2<true>(codes_f16_hi(codes[2 * q + i])), both(f));
          }
          to[lid + q * n16] = narrow<false>(y);
        }
      } else {
        to[lid] = x[u][0];
        to[lid + n16] = x[u][1];
      }
    }
  }
}

template <bool F16, bool CODES>
cudaError_t append_typed(const AppendLaunch &L, cudaStream_t s) {
  const long long rows = L.by_seq ? (long long)L.p.t.n_seqs * L.p.t.max_nodes : L.p.t.n_rows;
  const dim3 grid((unsigned)((rows + (1 << L.rows) - 1) >> L.rows)), block(kRowThreads);
  constexpr size_t smem = kPlaces * 2 * 16 * kRowThreads;
  if (L.p.q_gain || L.p.k_gain)
    return L.p.inter ? launch_chained(append_kernel<F16, CODES, true, true>, grid, block, smem, s, L)
                     : launch_chained(append_kernel<F16, CODES, true, false>, grid, block, smem, s, L);
  return L.p.inter ? launch_chained(append_kernel<F16, CODES, false, true>, grid, block, smem, s, L)
                   : launch_chained(append_kernel<F16, CODES, false, false>, grid, block, smem, s, L);
}

}  // namespace

cudaError_t launch_norm_rope_append(const RopeParams &p, cudaStream_t s) {
  static thread_local AppendLaunch L;
  L.p = p;
  L.by_seq = p.by_seq;
  L.lanes = head_lanes(p.c.D);
  L.inv_d = 1.f / (float)p.c.D;
  // a warp a row; more of them while the CTAs, three an SM, run at once all the same (125
  // rows: eight warps a row 4.3 us, one 8.7; 807 rows: eight in two waves 8.4, four in one
  // 5.9, two 8.0)
  const long long n = L.by_seq ? (long long)p.t.n_seqs * p.t.max_nodes : p.t.n_rows;
  L.rows = 0;
  while (L.rows < 3 && n >> L.rows > 3 * kAttnCtas) ++L.rows;
  if (p.c.esh == 0) return append_typed<false, true>(L, s);
  return p.c.f16 ? append_typed<true, false>(L, s) : append_typed<false, false>(L, s);
}

cudaError_t launch_cache_read(const CacheReadParams &p, cudaStream_t s) {
  static thread_local ReadLaunch L;
  L.p = p;
  L.lanes = head_lanes(p.c.D);
  const int sides = (p.k ? 1 : 0) + (p.v ? 1 : 0), fit = 2 * kReadAhead * (kRowThreads >> L.lanes) / (sides * p.c.Hkv);
  L.rows = fit < 1 ? 1 : fit > kReadRows ? kReadRows : fit;
  const dim3 grid((unsigned)((p.t.n_rows + L.rows - 1) / L.rows));
  return p.c.esh == 0 ? launch_chained(read_kernel<true>, grid, dim3(kRowThreads), 0, s, L)
                      : launch_chained(read_kernel<false>, grid, dim3(kRowThreads), 0, s, L);
}

}  // namespace dfv
