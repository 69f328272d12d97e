// logits.cu -- penalties for repeated tokens, biases and grammar masks on the
// logits of drafted nodes, with the argmax of each row in the same pass.
//
// Bound by issue before memory: every logit is read and written once, with some 26
// instructions a column with every rule and 16 without, 60 % of the issue slots
// taken.  Measured on the device: 32 trees of up to 16 nodes (390 rows) of 151936
// bf16 with every rule and 4093 tokens of history 73 us (3.6 TB/s), without rules
// 47 us (5.1 TB/s); one row 6.3 us.  A CTA owns a slice of
// kSlice vocabulary columns of one sequence, eight columns per thread, and
// walks rows of the sequence: the thread's bias and its knowledge of which
// columns repeat stay in registers over the rows, several rows' loads are in
// flight at once, and no barrier separates rows.
//
// The columns that penalties can touch are few (the history and the tree's
// tokens).  The CTA counts the history's tokens of its slice in shared memory
// (integer atomics: their order does not matter) and lists the columns met.  The
// dense walk leaves those columns' logits as they are and out of the argmax;
// afterwards warps apply all steps to the listed columns, where the row's own
// path adds to the counts.  (Applying the steps in the dense walk took
// twice the instructions: some lane of a warp nearly always meets a token.)
#include <algorithm>

#include "tree_common.cuh"

namespace dfv {
namespace {

constexpr int kLogitThreads = 512;
constexpr int kCols = 8;                              // columns of a thread
constexpr int kSlice = kLogitThreads * kCols;
static_assert(kSlice == kLogitSlice, "the host's limit on V counts these slices");
constexpr int kEarly = 2;                             // quads of history tokens of a thread loaded first
constexpr int kAhead = 4;                             // listed columns of a lane in flight
constexpr uint32_t kPromptBit = 0x80000000u;          // the token is in the prompt
constexpr uint32_t kTreeBit = 0x40000000u;            // some drafted node holds the token:
constexpr int kNodeShift = 24;                        // the first such node, in 6 bits
constexpr uint32_t kCountMask = (1u << kNodeShift) - 1u;  // how often the history generated it

// Eight columns of a row: consecutive ones of a 16-byte aligned row (VEC), or
// one in kLogitThreads each, so that a warp's 2- or 4-byte accesses are
// consecutive whatever the row's alignment.
template <bool VEC>
__device__ __forceinline__ int column(int j) {
  return VEC ? (int)threadIdx.x * kCols + j : (int)threadIdx.x + j * kLogitThreads;
}

// A row's columns of the thread, as loaded: packed pairs of bf16, or fp32.  Masks
// over them have all bits of a column set or none.
template <bool F32>
struct Raw {
  static constexpr int kWords = F32 ? kCols : kCols / 2;
  static constexpr uint32_t kNegInf = F32 ? 0xff800000u : 0xff80ff80u;
  uint32_t w[kWords];
  __device__ __forceinline__ float at(int j) const {
    if (F32) return __uint_as_float(w[j % kWords]);
    return j & 1 ? bf16_hi(w[j / 2 % kWords]) : bf16_lo(w[j / 2 % kWords]);
  }
  // a column whose number is not known when compiling, without local memory
  __device__ __forceinline__ float pick(int j) const {
    uint32_t v = 0u;
#pragma unroll
    for (int q = 0; q < kWords; ++q)
      if (q == (F32 ? j : j >> 1)) v = w[q];
    return __uint_as_float(F32 ? v : j & 1 ? v & 0xffff0000u : v << 16);
  }
  __device__ __forceinline__ void put(int j, uint32_t f) {  // f: fp32 bits of a value of the type
#pragma unroll
    for (int q = 0; q < kWords; ++q)
      if (q == (F32 ? j : j >> 1)) w[q] = F32 ? f : __byte_perm(w[q], f, j & 1 ? 0x7610 : 0x3276);
  }
  // the largest column: fp32, or one of a pair
  __device__ __forceinline__ uint32_t largest() const {
    if (F32) {
      float m = at(0);
#pragma unroll
      for (int j = 1; j < kCols; ++j) m = fmaxf(m, at(j));
      return __float_as_uint(m);
    }
    __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162 *>(&w[0]);
#pragma unroll
    for (int q = 1; q < kWords; ++q) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162 *>(&w[q]));
    return *reinterpret_cast<const uint32_t *>(&m);
  }
  static __device__ __forceinline__ float value(uint32_t m) {
    return F32 ? __uint_as_float(m) : fmaxf(bf16_lo(m), bf16_hi(m));
  }
  // whether largest() may beat a row's `floor`, held in the same form
  static __device__ __forceinline__ bool reaches(uint32_t m, uint32_t floor) {
    if (F32) return !(__uint_as_float(m) < __uint_as_float(floor));
    return !__hblt2(*reinterpret_cast<const __nv_bfloat162 *>(&m), *reinterpret_cast<const __nv_bfloat162 *>(&floor));
  }
  static __device__ __forceinline__ uint32_t floor_of(uint32_t key) {
    const uint32_t f = key == 0u ? 0xff800000u : key & 0x80000000u ? key ^ 0x80000000u : ~key;
    return F32 ? f : __byte_perm(f, 0u, 0x3232);
  }
};

// Bit j of `bits` as a mask over column j.
template <bool F32>
__device__ __forceinline__ void spread(uint32_t bits, uint32_t (&m)[Raw<F32>::kWords]) {
  if (F32) {
#pragma unroll
    for (int j = 0; j < kCols; ++j) m[j % Raw<F32>::kWords] = (uint32_t)((int)(bits << (31 - j)) >> 31);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // four bits to the top bits of four bytes, then each byte's sign twice
      const uint32_t t = ((bits >> (4 * h) & 0xfu) * 0x10204080u) & 0x80808080u;
      asm("prmt.b32 %0, %1, 0, 0x9988;" : "=r"(m[2 * h % Raw<F32>::kWords]) : "r"(t));
      asm("prmt.b32 %0, %1, 0, 0xbbaa;" : "=r"(m[(2 * h + 1) % Raw<F32>::kWords]) : "r"(t));
    }
  }
}

// The same for pairs from a table of four bits' masks: few instructions count more
// here than two shared-memory reads.
__device__ __forceinline__ void spread_pairs(const uint2 *table, uint32_t bits, uint32_t (&m)[4]) {
  const uint2 a = table[bits & 15u], b = table[bits >> 4];
  m[0] = a.x; m[1] = a.y; m[2] = b.x; m[3] = b.y;
}

// What is in flight of a row: its columns, one 16-bit column a register where
// they are loaded one by one, and the mask bits.  Loading waits for nothing that
// it loads and has no branch on a column; ready() puts the pieces together when
// the row's turn comes.
template <bool F32, bool VEC>
struct Fetched {
  static constexpr int kWords = VEC || F32 ? Raw<F32>::kWords : kCols;
  uint32_t w[kWords], bits;

  // row and allowed start at the thread's columns (VEC) or at the slice
  __device__ __forceinline__ void load(const char *row, const uint8_t *allowed, int left) {
    const int tid = threadIdx.x;
    if (VEC) {
      if (column<VEC>(0) < left) {  // left is a multiple of kCols
#pragma unroll
        for (int q = 0; q < kWords; q += 4) {
          const uint4 a = ldg_stream(row + 4 * q);
          w[q] = a.x; w[q + 1] = a.y; w[q + 2] = a.z; w[q + 3] = a.w;
        }
        bits = allowed ? (uint32_t)__ldg(allowed) : 0xffu;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
        const int c = min(column<VEC>(j), left - 1);
        w[j % kWords] = F32 ? reinterpret_cast<const uint32_t *>(row)[c] : (uint32_t)reinterpret_cast<const uint16_t *>(row)[c];
      }
      // a warp's columns j are one word: lane j holds it
      bits = allowed ? __ldg(reinterpret_cast<const uint32_t *>(allowed) + min((column<VEC>(0) >> 5) + kLogitThreads / 32 * (tid & 7), (left - 1) >> 5)) : 0xffffffffu;
    }
  }
  __device__ __forceinline__ uint32_t ready(Raw<F32> &x) const {
    if (VEC || F32) {
#pragma unroll
      for (int j = 0; j < Raw<F32>::kWords; ++j) x.w[j] = w[j % kWords];
    } else {
#pragma unroll
      for (int j = 0; j < Raw<F32>::kWords; ++j) x.w[j] = w[2 * j % kWords] | w[(2 * j + 1) % kWords] << 16;
    }
    if (VEC) return bits;
    uint32_t ok = 0u;
#pragma unroll
    for (int j = 0; j < kCols; ++j) ok |= (__shfl_sync(0xffffffffu, bits, j) >> (threadIdx.x & 31) & 1u) << j;
    return ok;
  }
};

template <bool F32, bool VEC>
__device__ __forceinline__ void store_row(char *row, int left, const Raw<F32> &x) {  // row: as Fetched::load
  if (VEC) {
    if (column<VEC>(0) < left) {
#pragma unroll
      for (int q = 0; q < Raw<F32>::kWords; q += 4)
        *reinterpret_cast<uint4 *>(row + 4 * q) = make_uint4(x.w[q], x.w[q + 1], x.w[q + 2], x.w[q + 3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
      const int c = column<VEC>(j);
      if (c < left) {
        if (F32)
          reinterpret_cast<uint32_t *>(row)[c] = x.w[j % Raw<F32>::kWords];
        else
          reinterpret_cast<uint16_t *>(row)[c] = (uint16_t)(x.w[j / 2 % Raw<F32>::kWords] >> (j & 1 ? 16 : 0));
      }
    }
  }
}

// Two sums, each rounded to nearest.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long x, y;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(y));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(x));
  return a;
}

__device__ __forceinline__ float round_bf16(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }

// The largest of a warp's values (the lowest column among equals) into *key;
// col() is only asked of lanes that hold it.  A lane without a value above -inf
// passes best = -inf.  (Leaving every thread's best in shared memory and asking
// the row's winner alone took more for its barriers than it saved.)
template <class Col>
__device__ __forceinline__ void warp_argmax(unsigned long long *key, float best, Col col) {
  const uint32_t k = best == -INFINITY ? 0u : float_key(best);
  const uint32_t m = __reduce_max_sync(0xffffffffu, k);
  // Most warps are below what their row has already: the rest is for the others.
  if (m == 0u || m < reinterpret_cast<volatile uint32_t *>(key)[1]) return;
  uint32_t c = 0xffffffffu;
  if (k == m) c = (uint32_t)col();
  c = __reduce_min_sync(0xffffffffu, c);
  if ((threadIdx.x & 31) == 0) atomicMax(key, ((unsigned long long)m << 32) | (0xffffffffu - c));
}

// ONE: one row a CTA, and more CTAs than run at once.  The walk takes every step
// itself where a column is met, which is less work than the list, a barrier and
// reading the columns again (32 single rows with 4093 tokens of history 29 -> 26 us,
// with 200 tokens 25 -> 20).  Where all CTAs run at once the lanes that meet many
// columns, one after the other, decide: one row 8 -> 10 us.
template <bool F32, bool VEC, bool ONE>
__global__ void __launch_bounds__(kLogitThreads, 2) logits_kernel(const LogitsParams p) {
  __shared__ __align__(16) uint32_t s_cnt[kSlice];
  __shared__ uint16_t s_list[kSlice];
  __shared__ unsigned long long s_key[DFV_MAX_TREE];
  __shared__ int s_tok[DFV_MAX_TREE];                  // drafted tokens, from the slice's start
  __shared__ uint64_t s_same[DFV_MAX_TREE];            // nodes with the token of this (first) one
  __shared__ uint64_t s_mask[DFV_MAX_TREE];            // the rows' own paths
  __shared__ uint32_t s_floor[DFV_MAX_TREE];           // a row's best so far, or less: skips most of the argmax
  __shared__ uint2 s_table[16];
  __shared__ float s_rep, s_freq, s_pres;
  __shared__ int s_n;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x;
  const int v0 = blockIdx.y * kSlice, left = min(kSlice, p.V - v0);  // columns of the slice
  // what needs no other load first is on its way together: a chain of loads is
  // most of a short call's time
  const int r0 = __ldg(p.t.row_off + b), r1 = __ldg(p.t.row_off + b + 1), n = r1 - r0;
  const int32_t *h = p.r.hist ? p.r.hist + b * p.r.hist_row : nullptr;
  // four tokens a load from the first 16-byte boundary on, the first ones before
  // the history's length is known
  const int head = h ? (int)((16u - ((uint32_t)(uintptr_t)h & 15u)) & 15u) / 4 : 0;
  const int4 *h4 = reinterpret_cast<const int4 *>(h + head);
  int4 early[kEarly];
  int said = 0, prompt = 0;
  if (h) {
    said = __ldg(p.r.hist_len + b);
    if (p.r.prompt_len) prompt = __ldg(p.r.prompt_len + b);
#pragma unroll
    for (int e = 0; e < kEarly; ++e) {
      early[e] = make_int4(-1, -1, -1, -1);
      if (head + 4 * (tid + e * kLogitThreads) + 4 <= p.r.hist_row) early[e] = __ldg(h4 + tid + e * kLogitThreads);
    }
  }
  if (r0 < 0 || r1 > p.t.n_rows || n > p.t.max_nodes || n <= (int)blockIdx.z) return;
  const bool pen = p.r.repetition || p.r.frequency || p.r.presence;
  const float *bias = p.r.bias ? p.r.bias + b * p.r.bias_row + v0 : nullptr;
  constexpr int kBytes = F32 ? 4 : 2;
  constexpr int kRowsAhead = F32 || !VEC || ONE ? 2 : 4;  // rows whose logits are in flight: 8 or 16 registers
  // a row starts from what the slices that are done have found
  if (tid < n) {
    s_key[tid] = p.argmax && gridDim.y > 1 ? __ldcg(&p.state[r0 + tid].key) : 0ull;
    s_floor[tid] = Raw<F32>::floor_of((uint32_t)(s_key[tid] >> 32));
  }
  if (tid >= 64 && tid < 80) {
    auto pair = [&](int k) { return (tid >> k & 1 ? 0xffffu : 0u) | (tid >> k & 2 ? 0xffff0000u : 0u); };
    s_table[tid - 64] = make_uint2(pair(0), pair(2));
  }

  // rows i0, i0 + gridDim.z, ... of the sequence, and their masks: the first ones
  // are on their way while the history is counted
  uint32_t inside = 0u;
  if (VEC) {
    inside = column<VEC>(0) < left ? 0xffu : 0u;
  } else {
#pragma unroll
    for (int j = 0; j < kCols; ++j) inside |= (column<VEC>(j) < left ? 1u : 0u) << j;
  }
  Fetched<F32, VEC> ahead[kRowsAhead];
  // addresses move from row to row: a 64-bit product for each cost a third of the walk
  const int own = VEC ? column<VEC>(0) : 0;
  const long long x_step = kBytes * p.row * (int)gridDim.z, out_step = kBytes * p.out_row * (int)gridDim.z,
                  allowed_step = 4 * p.r.allowed_row * (int)gridDim.z;
  const char *x_at = p.x + kBytes * ((r0 + (int)blockIdx.z) * p.row + v0 + own);
  const uint8_t *allowed_at = nullptr;
  if (p.r.allowed)
    allowed_at = reinterpret_cast<const uint8_t *>(p.r.allowed + (r0 + (int)blockIdx.z) * p.r.allowed_row + v0 / 32) + own / 8;
  auto fetch = [&](int q, int i) {  // in the rows' order
    if (i >= n) return;
    ahead[q].load(x_at, allowed_at, left);
    x_at += x_step;
    if (allowed_at) allowed_at += allowed_step;
  };
#pragma unroll
  for (int q = 0; q < kRowsAhead; ++q) fetch(q, blockIdx.z + q * gridDim.z);

  // steps 1-5 of dfv_logits_process on a column that penalties may touch, every
  // product, quotient and difference rounded on its own (no contraction)
  auto steps = [&](float y, uint32_t w, uint64_t mask, float add, bool ok, float rep, float freq, float pres) {
    uint32_t cnt = w & kCountMask;
    if (w & kTreeBit) cnt += __popcll(s_same[w >> kNodeShift & 63u] & mask);
    if (p.r.repetition && (cnt || (w & kPromptBit))) y = y > 0.f ? __fdiv_rn(y, rep) : __fmul_rn(y, rep);
    if (p.r.frequency) y = __fsub_rn(y, __fmul_rn(freq, (float)cnt));
    if (p.r.presence && cnt) y = __fsub_rn(y, pres);
    if (bias) y = __fadd_rn(y, add);
    if (!ok) y = -INFINITY;
    return F32 ? y : round_bf16(y);
  };
  const int rows = (n - (int)blockIdx.z + (int)gridDim.z - 1) / (int)gridDim.z;  // of this CTA

  // ---- the thread's columns
  float bv[kCols];
  uint32_t listed = 0u, touched = 0u;  // bit j: penalties may touch column j; listed: their steps come after the walk
  if (VEC && ((uint32_t)(uintptr_t)bias & 15u) == 0u) {
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f), *from = reinterpret_cast<const float4 *>(bias) + 2 * tid;
    const bool some = bias && inside;
    const float4 a = some ? from[0] : none, b = some ? from[1] : none;
    bv[0] = a.x; bv[1] = a.y; bv[2] = a.z; bv[3] = a.w; bv[4] = b.x; bv[5] = b.y; bv[6] = b.z; bv[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < kCols; ++j) bv[j] = bias && column<VEC>(j) < left ? bias[column<VEC>(j)] : 0.f;
  }
  if (pen) {
    for (int i = tid; i < kSlice / 4; i += kLogitThreads) reinterpret_cast<uint4 *>(s_cnt)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) s_n = 0;
    if (tid < n) {
      s_tok[tid] = p.tokens[r0 + tid] - v0;
      s_mask[tid] = row_mask(p.t, r0, tid);
    }
    if (tid == 64) s_rep = p.r.repetition ? p.r.repetition[b] : 1.f;
    if (tid == 65) s_freq = p.r.frequency ? p.r.frequency[b] : 0.f;
    if (tid == 66) s_pres = p.r.presence ? p.r.presence[b] : 0.f;
    __syncthreads();
    if (h) {
      const int len = (int)min((long long)said, (long long)p.r.hist_row);
      auto count = [&](int token, int i) {
        const unsigned c = (unsigned)token - (unsigned)v0;
        if (c < (unsigned)left) {
          if (i < prompt)
            atomicOr(&s_cnt[c], kPromptBit);
          else
            atomicAdd(&s_cnt[c], 1u);
        }
      };
      const int quads = max(len - head, 0) / 4, rest = head + 4 * quads;
      auto count4 = [&](const int4 &t, int i) {
        count(t.x, head + 4 * i);
        count(t.y, head + 4 * i + 1);
        count(t.z, head + 4 * i + 2);
        count(t.w, head + 4 * i + 3);
      };
#pragma unroll
      for (int e = 0; e < kEarly; ++e)
        if (tid + e * kLogitThreads < quads) count4(early[e], tid + e * kLogitThreads);
#pragma unroll 2
      for (int i = tid + kEarly * kLogitThreads; i < quads; i += kLogitThreads) count4(__ldg(h4 + i), i);
      if (tid < min(head, len)) count(h[tid], tid);
      if (tid >= 32 && tid - 32 < len - rest) count(h[rest + tid - 32], rest + tid - 32);
    }
    if (tid < n && (unsigned)s_tok[tid] < (unsigned)left) {
      uint64_t same = 0ull;
      for (int j = 0; j < n; ++j) same |= (uint64_t)(s_tok[j] == s_tok[tid]) << j;
      s_same[tid] = same;
      if (__ffsll((long long)same) - 1 == tid) atomicOr(&s_cnt[s_tok[tid]], kTreeBit | (uint32_t)tid << kNodeShift);
    }
    __syncthreads();
    if (VEC) {
      const uint4 *from = reinterpret_cast<const uint4 *>(s_cnt) + 2 * tid;
      const uint4 a = from[0], b = from[1];
      const uint32_t w[kCols] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < kCols; ++j) listed |= (w[j] ? 1u : 0u) << j;
    } else {
#pragma unroll
      for (int j = 0; j < kCols; ++j)
        if (s_cnt[column<VEC>(j)]) listed |= 1u << j;
    }
    if (ONE) {
      touched = listed;
      listed = 0u;
    } else {
      int at = 0;
      const int mine = __popc(listed);
      int run = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += a;
      }
      if (lane == 31) at = atomicAdd(&s_n, run);
      at = __shfl_sync(0xffffffffu, at, 31) + run - mine;
#pragma unroll
      for (int j = 0; j < kCols; ++j)
        if (listed >> j & 1u) s_list[at++] = (uint16_t)column<VEC>(j);
    }
  } else {
    __syncthreads();  // s_key
  }

  // ---- all rows, dense: bias and mask
  uint32_t keep[Raw<F32>::kWords];
  spread<F32>(listed, keep);
  // bias and mask of a row; afterwards x is what is stored, y what may win
  auto bias_of = [&](int j) {
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < kCols; ++q)
      if (q == j) v = bv[q];
    return v;
  };
  auto apply = [&](Raw<F32> &x, uint32_t ok, Raw<F32> &y) {
    if (bias) {
#pragma unroll
      for (int j = 0; j < kCols; j += 2) {
        const float2 z = add2(make_float2(x.at(j), x.at(j + 1)), make_float2(bv[j], bv[j + 1]));
        if (F32) {
          y.w[j % Raw<F32>::kWords] = __float_as_uint(z.x);
          y.w[(j + 1) % Raw<F32>::kWords] = __float_as_uint(z.y);
        } else {
          y.w[j / 2 % Raw<F32>::kWords] = pack2<false>(z.x, z.y);
        }
      }
    } else {
      y = x;
    }
    // not allowed: -inf; listed: stored as they came, out of the argmax
    uint32_t may[Raw<F32>::kWords];
    if constexpr (F32)
      spread<F32>(ok & ~listed, may);
    else
      spread_pairs(s_table, ok & ~listed, may);
#pragma unroll
    for (int j = 0; j < Raw<F32>::kWords; ++j) {
      y.w[j] = (y.w[j] & may[j]) | (Raw<F32>::kNegInf & ~may[j]);
      x.w[j] = (y.w[j] & ~keep[j]) | (x.w[j] & keep[j]);
    }
  };
  char *out_at = p.out + kBytes * ((r0 + (int)blockIdx.z) * p.out_row + v0 + own);
  for (int i0 = blockIdx.z; i0 < n; i0 += kRowsAhead * gridDim.z) {
#pragma unroll
    for (int q = 0; q < kRowsAhead; ++q) {
      const int i = i0 + q * gridDim.z;
      if (i >= n) break;
      Raw<F32> x, y;
      const uint32_t ok = ahead[q].ready(x) & inside;  // past the slice's end nothing may win
      if (ONE) {
        const Raw<F32> from = x;
        apply(x, ok, y);
        for (uint32_t c = touched; c; c &= c - 1u) {
          const int j = __ffs((int)c) - 1;
          y.put(j, __float_as_uint(steps(from.pick(j), s_cnt[column<VEC>(j)], s_mask[i], bias_of(j), ok >> j & 1u, s_rep,
                                         s_freq, s_pres)));
        }
        x = y;  // nothing is listed
      } else {
        apply(x, ok, y);
      }
      if (p.out) store_row<F32, VEC>(out_at, left, x);
      out_at += out_step;
      fetch(q, i + kRowsAhead * gridDim.z);
      if (p.argmax) {
        const uint32_t top = y.largest();
        if (__any_sync(0xffffffffu, Raw<F32>::reaches(top, *static_cast<volatile uint32_t *>(&s_floor[i])))) {
          const float best = Raw<F32>::value(top);
          warp_argmax(&s_key[i], best, [&]() {
            int bj = 0;
#pragma unroll
            for (int j = kCols - 1; j >= 0; --j)
              if (y.at(j) == best) bj = j;
            return v0 + column<VEC>(bj);
          });
          // never above the row's best: any of the values stored here is one of its logits
          if (lane == 0) s_floor[i] = Raw<F32>::floor_of(reinterpret_cast<volatile uint32_t *>(&s_key[i])[1]);
        }
      }
    }
  }

  // ---- the listed columns: every step
  if (pen && !ONE) {
    __syncthreads();  // the dense walk's stores come first
    const int m = s_n;
    const float rep = s_rep, freq = s_freq, pres = s_pres;
    // a warp takes a row, or several a row with fewer rows than warps; kAhead
    // columns of a lane are in flight
    constexpr int kW = kLogitThreads / 32;
    const int share = rows >= kW ? 1 : kW / rows;
    for (int u = warp; u < rows * share; u += kW) {
      const int i = blockIdx.z + (u / share) * gridDim.z, part = u % share;
      const char *from = p.x + kBytes * ((r0 + i) * p.row + v0);
      char *to = p.out + kBytes * ((r0 + i) * p.out_row + v0);
      const uint32_t *words = p.r.allowed ? p.r.allowed + (r0 + i) * p.r.allowed_row + v0 / 32 : nullptr;
      const uint64_t mask = s_mask[i];
      float best = -INFINITY;
      int bc = 0x7fffffff;
      for (int k0 = part * 32 * kAhead + lane; k0 < m; k0 += share * 32 * kAhead) {
        // past the list's end the last column again: loads without a branch, none
        // of them used before all are issued
        int c[kAhead];
        uint32_t raw[kAhead], word[kAhead];
        float add[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
          c[q] = s_list[min(k0 + 32 * q, m - 1)];
          raw[q] = F32 ? *reinterpret_cast<const uint32_t *>(from + 4 * c[q])
                       : (uint32_t)*reinterpret_cast<const uint16_t *>(from + 2 * c[q]);
          add[q] = bias ? bias[c[q]] : 0.f;
          word[q] = words ? words[c[q] >> 5] : 0xffffffffu;
        }
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
          if (k0 + 32 * q >= m) continue;
          const float y = steps(__uint_as_float(F32 ? raw[q] : raw[q] << 16), s_cnt[c[q]], mask, add[q],
                                word[q] >> (c[q] & 31) & 1u, rep, freq, pres);
          if (p.out) {
            if (F32)
              *reinterpret_cast<float *>(to + 4 * c[q]) = y;
            else
              *reinterpret_cast<uint16_t *>(to + 2 * c[q]) = f32_to_bf16_bits(y);
          }
          if (y > best || (y == best && c[q] < bc)) {  // the list is in no order
            best = y;
            bc = c[q];
          }
        }
      }
      if (p.argmax) warp_argmax(&s_key[i], best, [&]() { return v0 + bc; });
    }
  }

  // ---- join the slices of each row: the last one to arrive writes the token
  if (!p.argmax) return;
  __syncthreads();
  const int i = blockIdx.z + tid * gridDim.z;
  if (tid < DFV_MAX_TREE && i < n) {
    const int row = r0 + i;
    unsigned long long k = s_key[i];
    if (gridDim.y > 1) {
      LogitRow &state = p.state[row];
      if (k) atomicMax(&state.key, k);
      __threadfence();
      if (atomicAdd(&state.ticket, 1u) != gridDim.y - 1) return;
      __threadfence();
      k = atomicExch(&state.key, 0ull);
      state.ticket = 0u;
    }
    p.argmax[row] = k ? (int32_t)(0xffffffffu - (unsigned)(k & 0xffffffffull)) : 0;  // nothing above -inf: column 0
  }
}

template <bool F32, bool VEC>
cudaError_t launch_rows(const LogitsParams &p, bool one, dim3 grid, cudaStream_t s) {
  return one ? launch_chained(logits_kernel<F32, VEC, true>, grid, dim3(kLogitThreads), 0, s, p)
             : launch_chained(logits_kernel<F32, VEC, false>, grid, dim3(kLogitThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_logits(const LogitsParams &p, cudaStream_t s) {
  const int slices = (p.V + kSlice - 1) / kSlice;
  // Rows of a sequence share a CTA's counts.  They are spread over as many CTAs as
  // run at once, which ends soonest with few rows (16 nodes of one sequence: 12 us
  // so, 17 with half as many CTAs again); over twice as many where that leaves more
  // than eight rows each, so that one CTA's counting overlaps another's rows (4 x 64
  // nodes: 56 us so, 61 in one round).
  const int resident = 2 * kAttnCtas, ctas = (int)std::min((long long)slices * p.t.n_seqs, 4ll * resident);
  int z = resident / ctas;
  if (z < 1 || p.t.max_nodes > 8 * z) z = 2 * resident / ctas;
  z = z < 1 ? 1 : z > p.t.max_nodes ? p.t.max_nodes : z;
  // the first slices first: in most vocabularies the low ids are the frequent
  // tokens, so those CTAs have the longest lists
  const dim3 grid(p.t.n_seqs, slices, z);
  const int esz = p.f32 ? 4 : 2;
  const bool vec = p.V % kCols == 0 && ((uintptr_t)p.x | (uintptr_t)p.out) % 16 == 0 && p.row * esz % 16 == 0 &&
                   (!p.out || p.out_row * esz % 16 == 0);
  const bool one = p.t.max_nodes <= z && (long long)slices * p.t.n_seqs * z > resident;
  if (p.f32) return vec ? launch_rows<true, true>(p, one, grid, s) : launch_rows<true, false>(p, one, grid, s);
  return vec ? launch_rows<false, true>(p, one, grid, s) : launch_rows<false, false>(p, one, grid, s);
}

}  // namespace dfv
