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
// maxima over a head are shuffles within D / 16 lanes.  A CTA takes a few rows,
// whose sines and cosines it finds once for all heads, while its first pieces are
// on their way.
//
// Measured (GB300, device time): 8 prompts of up to 2039 rows of 32 + 2 x 4 heads of
// 128, normed and turned, 59 us, 4.4 TB/s (with 4 CTAs an SM at 64 registers 72; two
// pieces ahead instead of four 94 to 103); into codes and back, 4 x 1021 rows of 32 + 2
// x 8 heads of 64 and the 17402 tokens of each, 49 us, 4.9 TB/s; one row 3 us.
#include <cfloat>

#include "tree_common.cuh"

namespace dfv {
namespace {

constexpr int kRowThreads = 256;
constexpr int kMaxRowsCta = 8;    // append: rows of a CTA
constexpr int kAppendAhead = 4;   // items of a lane that are loaded at once
constexpr int kReadRows = 32;     // read: rows of a CTA
constexpr int kReadAhead = 4;

struct AppendLaunch {
  RopeParams p;
  int rows;     // of a CTA
  int by_seq;   // rows are counted as (sequence, row of it) with max_nodes each
  int lanes;    // log2 of the lanes of a head
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

// NORM: some gain is given.  INTER: pairs are neighbours.
template <bool F16, bool CODES, bool NORM, bool INTER>
__global__ void __launch_bounds__(kRowThreads, 3) append_kernel(const __grid_constant__ AppendLaunch L) {
  __shared__ __align__(16) float2 s_cos[kMaxRowsCta][64], s_sin[kMaxRowsCta][64];  // of two pairs each
  __shared__ int s_row[kMaxRowsCta], s_page[kMaxRowsCta], s_tok[kMaxRowsCta];
  const RopeParams &p = L.p;
  const CacheParams &c = p.c;
  const int tid = threadIdx.x, first = blockIdx.x * L.rows, HK = p.H + c.Hkv, NH = HK + c.Hkv, items = L.rows * NH;
  const int lid = tid & ((1 << L.lanes) - 1), group = tid >> L.lanes, groups = kRowThreads >> L.lanes;
  const int n16 = c.D / 16, r16 = p.rot / 16;
  const bool on = lid < n16;
  // pieces of a turned head, and of one that is copied
  const int2 at_turned = pieces_of(lid, n16, r16, !INTER), at_plain = make_int2(lid, lid + n16);
  pdl_trigger();
  pdl_wait();

  // Items: head h of the CTA's row j, queries first, then keys, then values.  A lane's
  // next item is `groups` further.
  const int dj = groups / NH, dh = groups - dj * NH;
  int lj = group / NH, lh = group - lj * NH;  // the next one to load
  int cj = lj, ch = lh;                       // the next one to work on
  uint4 x[kAppendAhead][2];
  auto load = [&]() {
#pragma unroll
    for (int u = 0; u < kAppendAhead; ++u) {
      x[u][0] = x[u][1] = make_uint4(0u, 0u, 0u, 0u);
      const int row = lj >= L.rows ? -1 : L.by_seq ? s_row[lj] : first + lj;
      if (on && (unsigned)row < (unsigned)p.t.n_rows) {
        const char *src = lh < p.H ? p.q + 2 * (row * p.q_row + lh * p.q_head)
                                   : lh < HK ? p.k + 2 * (row * p.k_row + (lh - p.H) * p.k_head) : p.v + 2 * (row * p.v_row + (lh - HK) * p.v_head);
        const int2 at = lh < HK ? at_turned : at_plain;
        x[u][0] = reinterpret_cast<const uint4 *>(src)[at.x];
        x[u][1] = reinterpret_cast<const uint4 *>(src)[at.y];
      }
      lj += dj;
      lh += dh;
      if (lh >= NH) { lh -= NH; ++lj; }
    }
  };
  if (!L.by_seq) load();

  // ---- whose rows, and where they go (one warp: a chain of reads)
  if (tid < L.rows) {
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
    load();
  }
  // ---- sines and cosines, once for all heads (the other warps)
  for (int u = tid - 32; u < L.rows * (p.rot / 2) && tid >= 32; u += kRowThreads - 32) {
    const int j = u / (p.rot / 2), i = u - j * (p.rot / 2), row = L.by_seq ? s_row[j] : first + j;
    if ((unsigned)row >= (unsigned)p.t.n_rows) continue;
    const uint64_t turn = (uint64_t)(long long)p.positions[row] * p.turns[i];
    float sn, cs;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn, &cs);
    reinterpret_cast<float *>(s_cos[j])[i] = cs * p.scale;
    reinterpret_cast<float *>(s_sin[j])[i] = sn * p.scale;
  }
  __syncthreads();

  for (int done = 0; done < items; done += kAppendAhead * groups) {
    if (done) load();
#pragma unroll
    for (int u = 0; u < kAppendAhead; ++u) {
      if (done + u * groups >= items) break;  // the same for all threads
      const int j = cj < L.rows ? cj : 0, h = ch;
      const bool have = cj < L.rows && on;
      cj += dj;
      ch += dh;
      if (ch >= NH) { ch -= NH; ++cj; }
      const int row = s_row[j], pg = s_page[j];
      const bool isq = h < p.H, turned = h < HK;
      const int2 at = turned ? at_turned : at_plain;
      if (!CODES && !turned) {  // values as they are
        if (have && pg >= 0) {
          uint4 *to = reinterpret_cast<uint4 *>(c.v + 2 * kv_off(c, p.layer, pg, h - HK, s_tok[j]));
          to[at.x] = x[u][0];
          to[at.y] = x[u][1];
        }
        if (!NORM) continue;  // (with norms the warp's other heads sum over shuffles)
      }
      float2 a[4], b[4];
      widen<F16>(x[u][0], a);
      widen<F16>(x[u][1], b);
      if (NORM) {
        float2 s2 = mul2(a[0], a[0]);
        s2 = fma2(b[0], b[0], s2);
#pragma unroll
        for (int e = 1; e < 4; ++e) s2 = fma2(b[e], b[e], fma2(a[e], a[e], s2));
        float ss = s2.x + s2.y;
        for (int o = 1 << L.lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const char *gain = isq ? p.q_gain : p.k_gain;
        if (turned && gain && on) {
          const float2 inv = both(rsqrtf(ss / (float)c.D + p.eps));
          float2 g[4];
          widen<F16>(__ldg(reinterpret_cast<const uint4 *>(gain) + at.x), g);
#pragma unroll
          for (int e = 0; e < 4; ++e) a[e] = mul2(mul2(a[e], inv), g[e]);
          widen<F16>(__ldg(reinterpret_cast<const uint4 *>(gain) + at.y), g);
#pragma unroll
          for (int e = 0; e < 4; ++e) b[e] = mul2(mul2(b[e], inv), g[e]);
        }
      }
      if (turned && on) {
        if (INTER) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int piece = q ? at.y : at.x;
            float2 *y = q ? b : a;
            if (piece < 2 * r16) {
              const float4 cs = *reinterpret_cast<const float4 *>(&s_cos[j][2 * piece]), sn = *reinterpret_cast<const float4 *>(&s_sin[j][2 * piece]);
              const float *cp = &cs.x, *sp = &sn.x;
#pragma unroll
              for (int e = 0; e < 4; ++e) y[e] = fma2(make_float2(-y[e].y, y[e].x), both(sp[e]), mul2(y[e], both(cp[e])));
            }
          }
        } else if (lid < r16) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 cs = s_cos[j][4 * lid + e], sn = s_sin[j][4 * lid + e], a0 = a[e];
            a[e] = fma2(make_float2(-b[e].x, -b[e].y), sn, mul2(a0, cs));
            b[e] = fma2(a0, sn, mul2(b[e], cs));
          }
        }
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
      if (!have || row < 0) continue;
      if (isq) {
        uint4 *to = reinterpret_cast<uint4 *>(p.o + 2 * (row * p.o_row + h * p.o_head));
        to[at.x] = narrow<F16>(a);
        to[at.y] = narrow<F16>(b);
        continue;
      }
      if (turned && p.ko) {
        uint4 *to = reinterpret_cast<uint4 *>(p.ko + 2 * (row * p.ko_row + (h - p.H) * p.ko_head));
        to[at.x] = narrow<F16>(a);
        to[at.y] = narrow<F16>(b);
      }
      if (pg < 0) continue;
      if (CODES) {
        const int kh = turned ? h - p.H : h - HK;
        const int e = exponent_of(top);
        const float f = exp_value((uint32_t)(127 - e));
        uint2 *to = reinterpret_cast<uint2 *>((turned ? c.k : c.v) + kv_off(c, p.layer, pg, kh, s_tok[j]));
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float2 *y = q ? b : a;
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], both(f));
          to[q ? at.y : at.x] = make_uint2(codes_of(y[0].x, y[0].y) | codes_of(y[1].x, y[1].y) << 16,
                                           codes_of(y[2].x, y[2].y) | codes_of(y[3].x, y[3].y) << 16);
        }
        if (lid == 0) (turned ? c.ke : c.ve)[exp_off(c, p.layer, pg, kh, s_tok[j])] = (uint8_t)(e + 127);
      } else if (turned) {
        uint4 *to = reinterpret_cast<uint4 *>(c.k + 2 * kv_off(c, p.layer, pg, h - p.H, s_tok[j]));
        to[at.x] = narrow<F16>(a);
        to[at.y] = narrow<F16>(b);
      }
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
  const dim3 grid((unsigned)((rows + L.rows - 1) / L.rows)), block(kRowThreads);
  if (L.p.q_gain || L.p.k_gain)
    return L.p.inter ? launch_chained(append_kernel<F16, CODES, true, true>, grid, block, 0, s, L)
                     : launch_chained(append_kernel<F16, CODES, true, false>, grid, block, 0, s, L);
  return L.p.inter ? launch_chained(append_kernel<F16, CODES, false, true>, grid, block, 0, s, L)
                   : launch_chained(append_kernel<F16, CODES, false, false>, grid, block, 0, s, L);
}

}  // namespace

cudaError_t launch_norm_rope_append(const RopeParams &p, cudaStream_t s) {
  static thread_local AppendLaunch L;
  L.p = p;
  L.by_seq = p.by_seq;
  L.lanes = head_lanes(p.c.D);
  // rows for two rounds of a CTA's loads, one row while there are fewer CTAs than SMs hold
  const int fit = 2 * kAppendAhead * (kRowThreads >> L.lanes) / (p.H + 2 * p.c.Hkv);
  L.rows = p.t.n_rows <= 4 * kAttnCtas || fit < 1 ? 1 : fit > kMaxRowsCta ? kMaxRowsCta : fit;
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
