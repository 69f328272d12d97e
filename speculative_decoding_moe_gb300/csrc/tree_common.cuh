// tree_common.cuh -- parameter blocks and device helpers shared by the
// tree-verify kernels: the paged cache, the drafted trees of a call, and the
// checks on device-side data (lengths, row offsets, page ids) that the host
// cannot see.  Every one of those checks turns bad data into an error bit and a
// skipped access.
#pragma once

#include <atomic>

#include "dfv_internal.cuh"

namespace dfv {

struct CacheParams {
  char *k, *v;
  long long sl, sp, sh, st;  // strides in elements: layer, page, head, token
  int n_layers, n_pages, page_shift, Hkv, D, f16;
  int max_seqs, max_pages;
  int32_t *table, *lens, *refs;
  uint32_t *err;
  int esh;            // log2 of an element's bytes: 1, or 0 for e4m3 codes
  uint8_t *ke, *ve;   // e4m3: exponent bytes [layer][page][head][token of the page]
};

// Drafted trees, or (max_nodes = max_rows, no mask) a batch of rows.
struct TreeParams {
  int n_seqs, n_rows, max_nodes;
  const int32_t *seq, *row_off;
  const uint64_t *mask;  // null: chain
};

struct RopeParams {
  CacheParams c;
  TreeParams t;
  int layer, H, rot, inter;
  float scale;
  const uint64_t *turns;
  const char *q, *k, *v;
  char *o;
  long long q_row, q_head, k_row, k_head, v_row, v_head, o_row, o_head;
  const int32_t *positions;
  // norm_rope_append only
  const char *q_gain, *k_gain;  // null: no norm
  float eps;
  int by_seq;  // row_off may be in any order
  char *ko;    // turned keys as rows, or null
  long long ko_row, ko_head;
};

struct CacheReadParams {
  CacheParams c;
  TreeParams t;
  int layer;
  char *k, *v;
  long long k_row, k_head, v_row, v_head;
};

struct PromptParams {
  int n_seqs, n_rows, max_rows, n_keys, max_keys;
  const int32_t *row_off, *key_off;
  int H, Hkv, G, D, f16;
  float scale_log2;  // scale * log2(e)
  const char *q;
  char *o;
  long long q_row, q_head, o_row, o_head;
  const char *k, *v;
  long long k_row, k_head, v_row, v_head;
  float *lse;
  uint32_t *kverr;  // the caller's error bits, or null
  unsigned *err;    // workspace error word (bounded waits)
};

struct TreeAttnParams {
  CacheParams c;
  TreeParams t;
  int layer, H, G;   // query heads, query heads per kv head
  float scale_log2;  // scale * log2(e)
  const char *q;
  char *o;
  long long q_row, q_head, o_row, o_head;
  float *lse;
  unsigned *err;  // workspace error word (bounded waits)
};

// A row's running maximum and how many slices are done, zero between calls.
struct LogitRow {
  unsigned long long key;
  unsigned ticket, unused;
};

// Every tree-verify call's workspace begins alike: the error word, then all counters
// that have to be zero between calls, at offsets that depend on no size.  What a call
// may leave behind lies after them, so one workspace serves calls of every kind.
constexpr size_t kWsErr = 256;
constexpr size_t kWsTickets = 512;                                          // commit: [DFV_MAX_TREE_SEQS] unsigned
constexpr size_t kWsRows = kWsTickets + DFV_MAX_TREE_SEQS * 4;              // logits: [rows] LogitRow
constexpr size_t kWsScratch = kWsRows + (size_t)DFV_MAX_TREE * DFV_MAX_TREE_SEQS * sizeof(LogitRow);
static_assert(kWsRows % 256 == 0 && kWsScratch % 256 == 0, "sections are 256-byte aligned");

// Columns of a CTA of the logit rules; a launch has at most 65535 such slices.
constexpr int kLogitSlice = 4096;
constexpr int kMaxVocab = 65535 * kLogitSlice;

struct LogitsParams {
  TreeParams t;
  dfv_logit_rules r;
  const char *x;
  char *out;
  long long row, out_row;
  int V, f32;
  const int32_t *tokens;
  int32_t *argmax;
  LogitRow *state;  // [n_rows]
};

struct AcceptTreeParams {
  TreeParams t;
  const int32_t *tokens, *target;
  int32_t *path, *tau;
  long long path_row;
};

struct CommitParams {
  CacheParams c;
  TreeParams t;
  const int32_t *path, *tau;
  long long path_row;
  int32_t *new_lens;
  unsigned *ticket;
};

struct PagesParams {
  CacheParams c;
  const int32_t *a, *b;  // reserve: seqs, n_new; fork: src, dst; copy: src, dst; free: seqs
  int n;
  int32_t *got;     // [n_pages] pages handed out
  int32_t *plan;    // fork: [n][4] source length, last source page, its copy, state
};

__device__ __forceinline__ void flag_err(uint32_t *err, uint32_t bit) {
  if (err) atomicOr(err, bit);
}

// Sequence b of a call: its rows [row0, row0 + n) and its cache sequence s with
// len committed tokens; s = -1 when the cache side is unusable (flagged).
struct SeqView {
  int row0, n, s, len;
};
__device__ __forceinline__ SeqView seq_view(const CacheParams &c, const TreeParams &t, int b) {
  // the loads first: one round trip when the sequences are not given by index
  const int s = t.seq ? t.seq[b] : b;
  const bool known = (unsigned)s < (unsigned)c.max_seqs;
  const int len = known ? c.lens[s] : 0, r0 = t.row_off[b], r1 = t.row_off[b + 1];
  SeqView v;
  v.row0 = r0;
  v.n = r1 - r0;
  v.s = s;
  v.len = len;
  if (r0 < 0 || r1 > t.n_rows || r1 < r0 || v.n > t.max_nodes) {
    flag_err(c.err, DFV_KVERR_LEN);
    v.n = 0;
    v.row0 = 0;
  }
  if (!known) {
    flag_err(c.err, DFV_KVERR_SEQ);
    v.s = -1;
  } else if (len < 0 || (long long)len + v.n > ((long long)c.max_pages << c.page_shift)) {
    flag_err(c.err, DFV_KVERR_LEN);
    v.s = -1;
    v.len = 0;
  }
  return v;
}

// Page of token `pos` of cache sequence s, or -1 (flagged) when there is none.
__device__ __forceinline__ int page_of(const CacheParams &c, int s, int pos) {
  const int pg = c.table[(size_t)s * c.max_pages + (pos >> c.page_shift)];
  if ((unsigned)pg >= (unsigned)c.n_pages) {
    flag_err(c.err, DFV_KVERR_PAGE);
    return -1;
  }
  return pg;
}

// Element offset of row `row` of page pg, head h, layer l.
__device__ __forceinline__ long long kv_off(const CacheParams &c, int l, int pg, int h, int row) {
  return l * c.sl + pg * c.sp + h * c.sh + row * c.st;
}

// Byte of token `row` of page pg, head h, layer l in the exponents of a cache in codes.
__device__ __forceinline__ size_t exp_off(const CacheParams &c, int l, int pg, int h, int row) {
  return ((((size_t)l * c.n_pages + pg) * c.Hkv + h) << c.page_shift) + row;
}

// 2^e of an exponent byte e + 127.
__device__ __forceinline__ float exp_value(uint32_t byte) { return __uint_as_float(byte << 23); }

// Two codes (low byte first) as an fp16 pair: exact, NaN stays NaN.
__device__ __forceinline__ uint32_t codes_f16(uint32_t two) {
  uint32_t r;
  asm("{\n .reg .b16 x, y;\n mov.b32 {x, y}, %1;\n cvt.rn.f16x2.e4m3x2 %0, x;\n}" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t codes_f16_hi(uint32_t two) {
  uint32_t r;
  asm("{\n .reg .b16 x, y;\n mov.b32 {x, y}, %1;\n cvt.rn.f16x2.e4m3x2 %0, y;\n}" : "=r"(r) : "r"(two));
  return r;
}

// The sequence that owns packed row r, or -1: the last one whose rows begin at or before it.
__device__ __forceinline__ int owner_of(const TreeParams &t, int r) {
  int lo = 0, hi = t.n_seqs;  // row_off[lo] <= r < row_off[hi], the ends taken for granted
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.row_off[mid] <= r)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ uint64_t row_mask(const TreeParams &t, int row0, int i) {
  return t.mask ? t.mask[row0 + i] : (i >= 63 ? ~0ull : (2ull << i) - 1ull);
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What p = 2^(x - z) takes for a maximum m of scores whose x is c times as large: c m, for fp16 less
// 6, rounded up there: scores beyond 2^25 are steps of 4 and more apart, and rounded down z
// would let p past fp16's largest value.
template <bool F16>
__device__ __forceinline__ float base_of(float m, float c) {
  if (m == -INFINITY) return F16 ? -6.f : 0.f;
  return F16 ? __fadd_ru(__fmul_ru(m, c), -6.f) : m * c;
}

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if (F16) return __half22float2(*reinterpret_cast<const __half2 *>(&v));
  return make_float2(bf16_lo(v), bf16_hi(v));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

cudaError_t launch_rope_append(const RopeParams &p, cudaStream_t s);
cudaError_t launch_norm_rope_append(const RopeParams &p, cudaStream_t s);
cudaError_t launch_cache_read(const CacheReadParams &p, cudaStream_t s);
size_t prompt_attn_ws(int D);
cudaError_t launch_prompt_attn(const PromptParams &p, void *ws, cudaStream_t s, char *why, size_t why_len);
// Rows per CTA, CTAs per range and ranges of an attention call.
constexpr int kAttnCtas = 152;  // one per SM of GB300
struct AttnPlan {
  int rows, n_rt, n_groups;
};
AttnPlan tree_attn_plan(int max_nodes, int G);
size_t tree_attn_ws(const AttnPlan &a, int n_seqs, int Hkv, int D);
cudaError_t launch_tree_attn(const TreeAttnParams &p, const AttnPlan &a, void *ws, cudaStream_t s, char *why,
                             size_t why_len);
cudaError_t launch_logits(const LogitsParams &p, cudaStream_t s);
cudaError_t launch_accept_tree(const AcceptTreeParams &p, cudaStream_t s);
cudaError_t launch_commit(const CommitParams &p, cudaStream_t s);
cudaError_t launch_copy_pages(const PagesParams &p, cudaStream_t s);
cudaError_t launch_reserve(const PagesParams &p, cudaStream_t s);
cudaError_t launch_fork(const PagesParams &p, cudaStream_t s);
cudaError_t launch_free(const PagesParams &p, cudaStream_t s);

// status reporting of api.cu (thread-local detail text)
int api_fail(int status, const char *fmt, ...);

// ---- checks that the entry points share (tree_api.cu)
inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline bool words(const void *p) { return aligned(p, 4); }  // NULL too
inline bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0 && s <= ((int64_t)1 << 40); }
int launched(cudaError_t e, const char *where);
int check_cache(const dfv_kv_cache *c);
int check_ws(const void *ws, size_t have, size_t need);
int check_rope(const dfv_kv_cache *cache, int layer, int n_heads, int rot_dim, int interleaved, float scale,
               const RopeParams &p);
CacheParams cache_params(const dfv_kv_cache *c);

// Raises a kernel's limit of dynamic shared memory, once per device (the call took
// 0.5 us of an attention call's 4.4).
template <class Kern>
cudaError_t allow_smem(Kern kern, size_t smem, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if (e != cudaSuccess || (done.load(std::memory_order_relaxed) & bit)) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <class Kern, class Par>
cudaError_t launch_chained(Kern kern, dim3 grid, dim3 block, size_t smem, cudaStream_t s, const Par &p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace dfv
