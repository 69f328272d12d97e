// tree_api.cu -- the tree-verify part of the C ABI: argument validation and
// workspace layout.  Everything is checked on the host before any launch.
#include <cmath>
#include <cstdio>

#include "tree_common.cuh"

namespace {

using dfv::api_fail;

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

int launched(cudaError_t e, const char *where) {
  if (e == cudaSuccess) return DFV_OK;
  return api_fail(DFV_ERR_CUDA, "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool words(const void *p) { return aligned(p, 4); }  // NULL too
bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0 && s <= ((int64_t)1 << 40); }

int check_cache(const dfv_kv_cache *c) {
  if (!c) return api_fail(DFV_ERR_INVALID_ARG, "cache is NULL");
  if (c->n_layers < 1 || c->n_pages < 1 || c->n_kv_heads < 1 || c->max_seqs < 1 || c->max_pages < 1 || c->head_dim < 1)
    return api_fail(DFV_ERR_INVALID_ARG, "non-positive cache size");
  if (c->dtype != DFV_BF16 && c->dtype != DFV_F16) return api_fail(DFV_ERR_UNSUPPORTED, "cache dtype %d", c->dtype);
  if (c->page_size < 8 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
    return api_fail(DFV_ERR_UNSUPPORTED, "page_size %d: a power of two in 8..256 is needed", c->page_size);
  if (c->head_dim % 16 || c->head_dim > 256)
    return api_fail(DFV_ERR_UNSUPPORTED, "head_dim %d: a multiple of 16 up to 256 is needed", c->head_dim);
  if (c->n_kv_heads > 1024 || c->n_layers > 65535)
    return api_fail(DFV_ERR_UNSUPPORTED, "%d kv heads, %d layers (at most 1024 and 65535)", c->n_kv_heads, c->n_layers);
  if ((int64_t)c->max_pages * c->page_size > 0x7fff0000)
    return api_fail(DFV_ERR_UNSUPPORTED, "max_pages * page_size exceeds 2^31 - 2^16 tokens");
  if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16))
    return api_fail(DFV_ERR_INVALID_ARG, "cache k/v NULL or not 16-byte aligned");
  if (!stride_ok(c->stride_layer) || !stride_ok(c->stride_page) || !stride_ok(c->stride_head) ||
      !stride_ok(c->stride_token))
    return api_fail(DFV_ERR_INVALID_ARG, "cache strides must be non-negative multiples of 8 elements");
  if (c->stride_token < c->head_dim)
    return api_fail(DFV_ERR_INVALID_ARG, "stride_token %lld below head_dim", (long long)c->stride_token);
  if (!c->page_table || !c->lens || !words(c->page_table) || !words(c->lens) || !words(c->refs) || !words(c->err))
    return api_fail(DFV_ERR_INVALID_ARG, "page_table/lens NULL, or page_table/lens/refs/err not 4-byte aligned");
  return DFV_OK;
}

int check_tree(const dfv_tree_batch *t) {
  if (!t) return api_fail(DFV_ERR_INVALID_ARG, "tree is NULL");
  if (t->n_seqs < 1 || t->n_seqs > DFV_MAX_TREE_SEQS)
    return api_fail(DFV_ERR_INVALID_ARG, "n_seqs %d outside 1..%d", t->n_seqs, DFV_MAX_TREE_SEQS);
  if (t->max_nodes < 1 || t->max_nodes > DFV_MAX_TREE)
    return api_fail(DFV_ERR_INVALID_ARG, "max_nodes %d outside 1..%d", t->max_nodes, DFV_MAX_TREE);
  if (t->n_rows < 1 || t->n_rows > DFV_MAX_TREE * DFV_MAX_TREE_SEQS)
    return api_fail(DFV_ERR_INVALID_ARG, "n_rows %d outside 1..%d", t->n_rows, DFV_MAX_TREE * DFV_MAX_TREE_SEQS);
  if (!t->row_off || !words(t->row_off) || !words(t->seq))
    return api_fail(DFV_ERR_INVALID_ARG, "row_off NULL, or row_off/seq not 4-byte aligned");
  if (t->mask && !aligned(t->mask, 8)) return api_fail(DFV_ERR_INVALID_ARG, "mask not 8-byte aligned");
  return DFV_OK;
}

int check_ws(const void *ws, size_t have, size_t need) {
  if (!ws || !aligned(ws, 256)) return api_fail(DFV_ERR_WORKSPACE, "workspace NULL or not 256-byte aligned");
  if (have < need) return api_fail(DFV_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", have, need);
  return DFV_OK;
}

dfv::CacheParams cache_params(const dfv_kv_cache *c) {
  dfv::CacheParams p = {};
  p.k = (char *)c->k;
  p.v = (char *)c->v;
  p.sl = c->stride_layer;
  p.sp = c->stride_page;
  p.sh = c->stride_head;
  p.st = c->stride_token;
  p.n_layers = c->n_layers;
  p.n_pages = c->n_pages;
  p.page_shift = 0;
  while ((1 << p.page_shift) < c->page_size) ++p.page_shift;
  p.Hkv = c->n_kv_heads;
  p.D = c->head_dim;
  p.f16 = c->dtype == DFV_F16;
  p.max_seqs = c->max_seqs;
  p.max_pages = c->max_pages;
  p.table = c->page_table;
  p.lens = c->lens;
  p.refs = c->refs;
  p.err = c->err;
  return p;
}

dfv::TreeParams tree_params(const dfv_tree_batch *t) {
  dfv::TreeParams p = {};
  p.n_seqs = t->n_seqs;
  p.n_rows = t->n_rows;
  p.max_nodes = t->max_nodes;
  p.seq = t->seq;
  p.row_off = t->row_off;
  p.mask = t->mask;
  return p;
}

// the page calls' workspace: tickets, then fork plan and pages handed out
struct PageWs {
  unsigned *ticket;
  int32_t *plan, *got;
  size_t bytes;
};
PageWs page_ws(const dfv_kv_cache *c, void *base) {
  PageWs w = {};
  w.ticket = base ? (unsigned *)((char *)base + dfv::kWsTickets) : nullptr;
  size_t off = dfv::kWsScratch;
  auto take = [&](size_t n) {
    void *p = base ? (void *)((char *)base + off) : nullptr;
    off += align256(n);
    return p;
  };
  w.plan = (int32_t *)take(DFV_MAX_TREE_SEQS * 16);
  w.got = (int32_t *)take((size_t)c->n_pages * 4);
  w.bytes = off;
  return w;
}

int check_list(const dfv_kv_cache *c, const int32_t *a, const int32_t *b, int n, bool refs) {
  int st = check_cache(c);
  if (st) return st;
  if (n < 1 || n > DFV_MAX_TREE_SEQS) return api_fail(DFV_ERR_INVALID_ARG, "n %d outside 1..%d", n, DFV_MAX_TREE_SEQS);
  if (!a || !b || !words(a) || !words(b)) return api_fail(DFV_ERR_INVALID_ARG, "index list NULL or not 4-byte aligned");
  if (refs && !c->refs) return api_fail(DFV_ERR_INVALID_ARG, "the cache has no refs");
  return DFV_OK;
}

}  // namespace

extern "C" {

int dfv_rope_table(int rot_dim, double theta, int scaling, double factor, double original, double low, double high,
                   uint64_t *turns) {
  if (rot_dim < 16 || rot_dim % 16 || rot_dim > 256)
    return api_fail(DFV_ERR_UNSUPPORTED, "rot_dim %d: a multiple of 16 up to 256 is needed", rot_dim);
  if (!(theta > 1.0) || !std::isfinite(theta)) return api_fail(DFV_ERR_INVALID_ARG, "theta must be above 1");
  if (scaling < DFV_ROPE_NONE || scaling > DFV_ROPE_BANDS)
    return api_fail(DFV_ERR_UNSUPPORTED, "rotary scaling %d", scaling);
  if (scaling != DFV_ROPE_NONE && !(factor >= 1.0 && std::isfinite(factor)))
    return api_fail(DFV_ERR_INVALID_ARG, "factor must be at least 1");
  if (scaling == DFV_ROPE_BANDS &&
      !(original >= 1.0 && std::isfinite(original) && low >= 0.0 && high > low && std::isfinite(high)))
    return api_fail(DFV_ERR_INVALID_ARG, "bands need original >= 1 and 0 <= low < high");
  if (!turns) return api_fail(DFV_ERR_INVALID_ARG, "turns NULL");
  const double r = rot_dim, two_pi = 6.283185307179586476925286766559;
  const double base = scaling == DFV_ROPE_NTK ? theta * std::pow(factor, r / (r - 2.0)) : theta;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / r);
    if (scaling == DFV_ROPE_LINEAR) f /= factor;
    if (scaling == DFV_ROPE_BANDS) {
      double g = (original * f / two_pi - low) / (high - low);
      g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
      f = (1.0 - g) * f / factor + g * f;
    }
    turns[i] = (uint64_t)std::nearbyint(std::ldexp(f / two_pi, 64));  // f <= 1: below 2^64 / 2 pi
  }
  return DFV_OK;
}

int dfv_rope_append(const dfv_kv_cache *cache, int layer, const dfv_tree_batch *tree, int n_heads, int rot_dim,
                    int interleaved, float scale, const uint64_t *turns, const void *q, int64_t q_row, int64_t q_head,
                    const void *k, int64_t k_row, int64_t k_head, const void *v, int64_t v_row, int64_t v_head,
                    const int32_t *positions, void *q_out, int64_t o_row, int64_t o_head, void *stream) {
  int st = check_cache(cache);
  if (st) return st;
  if ((st = check_tree(tree))) return st;
  if (layer < 0 || layer >= cache->n_layers)
    return api_fail(DFV_ERR_INVALID_ARG, "layer %d outside 0..%d", layer, cache->n_layers - 1);
  if (n_heads < 1 || n_heads > 16384) return api_fail(DFV_ERR_INVALID_ARG, "n_heads %d outside 1..16384", n_heads);
  if (rot_dim < 16 || rot_dim % 16 || rot_dim > cache->head_dim)
    return api_fail(DFV_ERR_UNSUPPORTED, "rot_dim %d: a multiple of 16 up to head_dim %d is needed", rot_dim,
                    cache->head_dim);
  if (interleaved != 0 && interleaved != 1) return api_fail(DFV_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if (!std::isfinite(scale)) return api_fail(DFV_ERR_INVALID_ARG, "scale must be finite");
  if (!turns || !aligned(turns, 8) || !positions || !words(positions))
    return api_fail(DFV_ERR_INVALID_ARG, "turns/positions NULL, or not 8- and 4-byte aligned");
  if (!q || !k || !v || !q_out || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16))
    return api_fail(DFV_ERR_INVALID_ARG, "q/k/v/q_out NULL or not 16-byte aligned");
  if (!stride_ok(q_row) || !stride_ok(q_head) || !stride_ok(k_row) || !stride_ok(k_head) || !stride_ok(v_row) ||
      !stride_ok(v_head) || !stride_ok(o_row) || !stride_ok(o_head))
    return api_fail(DFV_ERR_INVALID_ARG, "row and head strides must be non-negative multiples of 8 elements");
  if (q == q_out && (q_row != o_row || q_head != o_head))
    return api_fail(DFV_ERR_INVALID_ARG, "q_out is q: the strides must be the same");
  dfv::RopeParams p = {};
  p.c = cache_params(cache);
  p.t = tree_params(tree);
  p.layer = layer;
  p.H = n_heads;
  p.rot = rot_dim;
  p.inter = interleaved;
  p.scale = scale;
  p.turns = turns;
  p.q = (const char *)q;
  p.k = (const char *)k;
  p.v = (const char *)v;
  p.o = (char *)q_out;
  p.q_row = q_row;
  p.q_head = q_head;
  p.k_row = k_row;
  p.k_head = k_head;
  p.v_row = v_row;
  p.v_head = v_head;
  p.o_row = o_row;
  p.o_head = o_head;
  p.positions = positions;
  return launched(dfv::launch_rope_append(p, (cudaStream_t)stream), "rotary append launch");
}

static int check_attn_shape(const dfv_kv_cache *cache, const dfv_tree_batch *tree, int n_heads) {
  int st = check_cache(cache);
  if (st) return st;
  if ((st = check_tree(tree))) return st;
  if (cache->head_dim != 64 && cache->head_dim != 128)
    return api_fail(DFV_ERR_UNSUPPORTED, "attention takes head_dim 64 or 128, not %d", cache->head_dim);
  if (n_heads < 1 || n_heads % cache->n_kv_heads)
    return api_fail(DFV_ERR_INVALID_ARG, "n_heads %d is no multiple of %d kv heads", n_heads, cache->n_kv_heads);
  if (n_heads / cache->n_kv_heads > 16)
    return api_fail(DFV_ERR_UNSUPPORTED, "%d query heads per kv head (at most 16)", n_heads / cache->n_kv_heads);
  return DFV_OK;
}

size_t dfv_tree_attention_workspace_size(const dfv_kv_cache *cache, const dfv_tree_batch *tree, int n_heads) {
  if (check_attn_shape(cache, tree, n_heads)) return 0;
  const dfv::AttnPlan a = dfv::tree_attn_plan(tree->max_nodes, n_heads / cache->n_kv_heads);
  return dfv::tree_attn_ws(a, tree->n_seqs, cache->n_kv_heads, cache->head_dim);
}

int dfv_tree_attention(const dfv_kv_cache *cache, int layer, const dfv_tree_batch *tree, int n_heads, float scale,
                       const void *q, int64_t q_row, int64_t q_head, void *out, int64_t o_row, int64_t o_head,
                       float *opt_lse, void *ws, size_t ws_bytes, void *stream) {
  int st = check_attn_shape(cache, tree, n_heads);
  if (st) return st;
  if (layer < 0 || layer >= cache->n_layers)
    return api_fail(DFV_ERR_INVALID_ARG, "layer %d outside 0..%d", layer, cache->n_layers - 1);
  if (!(scale > 0.f) || !std::isfinite(scale)) return api_fail(DFV_ERR_INVALID_ARG, "scale must be positive");
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16))
    return api_fail(DFV_ERR_INVALID_ARG, "q/out NULL or not 16-byte aligned");
  if (q == out) return api_fail(DFV_ERR_INVALID_ARG, "out must not be q");
  if (!words(opt_lse)) return api_fail(DFV_ERR_INVALID_ARG, "lse not 4-byte aligned");
  if (!stride_ok(q_row) || !stride_ok(q_head) || !stride_ok(o_row) || !stride_ok(o_head))
    return api_fail(DFV_ERR_INVALID_ARG, "row and head strides must be non-negative multiples of 8 elements");
  if ((st = check_ws(ws, ws_bytes, dfv_tree_attention_workspace_size(cache, tree, n_heads)))) return st;
  dfv::TreeAttnParams p = {};
  p.c = cache_params(cache);
  p.t = tree_params(tree);
  p.layer = layer;
  p.H = n_heads;
  p.G = n_heads / cache->n_kv_heads;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.q = (const char *)q;
  p.o = (char *)out;
  p.q_row = q_row;
  p.q_head = q_head;
  p.o_row = o_row;
  p.o_head = o_head;
  p.lse = opt_lse;
  p.err = (unsigned *)((char *)ws + dfv::kWsErr);
  char why[256] = {0};
  const cudaError_t e = dfv::launch_tree_attn(p, dfv::tree_attn_plan(tree->max_nodes, p.G), ws, (cudaStream_t)stream,
                                              why, sizeof why);
  if (e != cudaSuccess && why[0]) return api_fail(DFV_ERR_CUDA, "tree attention: %s", why);
  return launched(e, "tree attention launch");
}

size_t dfv_logits_workspace_size(int n_rows_max) {
  if (n_rows_max < 1 || n_rows_max > DFV_MAX_TREE * DFV_MAX_TREE_SEQS) return 0;
  return dfv::kWsRows + align256((size_t)n_rows_max * sizeof(dfv::LogitRow));
}

int dfv_logits_process(const void *logits, int64_t row, int dtype, int V, const dfv_tree_batch *tree,
                       const int32_t *tokens, const dfv_logit_rules *rules, void *out, int64_t out_row,
                       int32_t *argmax, void *ws, size_t ws_bytes, void *stream) {
  int st = check_tree(tree);
  if (st) return st;
  if (dtype != DFV_BF16 && dtype != DFV_F32) return api_fail(DFV_ERR_UNSUPPORTED, "logits dtype %d", dtype);
  if (V < 1 || V > dfv::kMaxVocab) return api_fail(DFV_ERR_INVALID_ARG, "V=%d outside 1..%d", V, dfv::kMaxVocab);
  const size_t esz = dtype == DFV_F32 ? 4 : 2;
  if (!logits || !aligned(logits, esz) || !aligned(out, esz))
    return api_fail(DFV_ERR_INVALID_ARG, "logits NULL, or logits/out not aligned to their type");
  if (!out && !argmax) return api_fail(DFV_ERR_INVALID_ARG, "neither out nor argmax is given");
  if (row < V || (out && out_row < V)) return api_fail(DFV_ERR_INVALID_ARG, "row stride below V");
  if (out == logits && out_row != row) return api_fail(DFV_ERR_INVALID_ARG, "out is logits: the strides must be the same");
  if (!rules) return api_fail(DFV_ERR_INVALID_ARG, "rules is NULL");
  if (!words(tokens) || !words(argmax) || !words(rules->hist) || !words(rules->hist_len) || !words(rules->prompt_len) ||
      !words(rules->repetition) || !words(rules->frequency) || !words(rules->presence) || !words(rules->bias) ||
      !words(rules->allowed))
    return api_fail(DFV_ERR_INVALID_ARG, "tokens, argmax and the rules' arrays must be 4-byte aligned");
  const bool pen = rules->repetition || rules->frequency || rules->presence;
  if (pen && !tokens) return api_fail(DFV_ERR_INVALID_ARG, "penalties need the drafted tokens");
  if (rules->hist && (!rules->hist_len || rules->hist_row < 0))
    return api_fail(DFV_ERR_INVALID_ARG, "hist needs hist_len and a non-negative hist_row");
  if (pen && rules->hist && rules->hist_row >= (1 << 24))
    return api_fail(DFV_ERR_UNSUPPORTED, "hist_row %lld: at most 2^24 - 1 tokens of history", (long long)rules->hist_row);
  if (rules->bias && rules->bias_row != 0 && rules->bias_row < V)
    return api_fail(DFV_ERR_INVALID_ARG, "bias_row must be 0 or at least V");
  if (rules->allowed && rules->allowed_row != 0 && rules->allowed_row < (V + 31) / 32)
    return api_fail(DFV_ERR_INVALID_ARG, "allowed_row must be 0 or at least V / 32 words");
  if ((st = check_ws(ws, ws_bytes, dfv_logits_workspace_size(tree->n_rows)))) return st;
  dfv::LogitsParams p = {};
  p.t = tree_params(tree);
  p.r = *rules;
  if (!pen) p.r.hist = p.r.hist_len = p.r.prompt_len = nullptr;  // only penalties read the history
  p.x = (const char *)logits;
  p.out = (char *)out;
  p.row = row;
  p.out_row = out_row;
  p.V = V;
  p.f32 = dtype == DFV_F32;
  p.tokens = tokens;
  p.argmax = argmax;
  p.state = (dfv::LogitRow *)((char *)ws + dfv::kWsRows);
  return launched(dfv::launch_logits(p, (cudaStream_t)stream), "logit rules launch");
}

int dfv_accept_tree(const dfv_tree_batch *tree, const int32_t *tokens, const int32_t *target, int32_t *path,
                    int64_t path_row, int32_t *tau, void *stream) {
  int st = check_tree(tree);
  if (st) return st;
  if (!tokens || !target || !path || !tau || !words(tokens) || !words(target) || !words(path) || !words(tau))
    return api_fail(DFV_ERR_INVALID_ARG, "tokens/target/path/tau NULL or not 4-byte aligned");
  if (path_row < tree->max_nodes) return api_fail(DFV_ERR_INVALID_ARG, "path_row below max_nodes");
  dfv::AcceptTreeParams p = {};
  p.t = tree_params(tree);
  p.tokens = tokens;
  p.target = target;
  p.path = path;
  p.path_row = path_row;
  p.tau = tau;
  return launched(dfv::launch_accept_tree(p, (cudaStream_t)stream), "tree acceptance launch");
}

size_t dfv_cache_workspace_size(const dfv_kv_cache *cache) {
  if (check_cache(cache)) return 0;
  return page_ws(cache, nullptr).bytes;
}

int dfv_cache_commit(const dfv_kv_cache *cache, const dfv_tree_batch *tree, const int32_t *path, int64_t path_row,
                     const int32_t *tau, int32_t *new_lens, void *ws, size_t ws_bytes, void *stream) {
  int st = check_cache(cache);
  if (st) return st;
  if ((st = check_tree(tree))) return st;
  if (!path || !tau || !new_lens || !words(path) || !words(tau) || !words(new_lens))
    return api_fail(DFV_ERR_INVALID_ARG, "path/tau/new_lens NULL or not 4-byte aligned");
  if (path_row < tree->max_nodes) return api_fail(DFV_ERR_INVALID_ARG, "path_row below max_nodes");
  if ((st = check_ws(ws, ws_bytes, page_ws(cache, nullptr).bytes))) return st;
  dfv::CommitParams p = {};
  p.c = cache_params(cache);
  p.t = tree_params(tree);
  p.path = path;
  p.path_row = path_row;
  p.tau = tau;
  p.new_lens = new_lens;
  p.ticket = page_ws(cache, ws).ticket;
  return launched(dfv::launch_commit(p, (cudaStream_t)stream), "cache commit launch");
}

int dfv_cache_copy_pages(const dfv_kv_cache *cache, const int32_t *src, const int32_t *dst, int n, void *stream) {
  int st = check_cache(cache);
  if (st) return st;
  if (n < 1 || n > (1 << 20)) return api_fail(DFV_ERR_INVALID_ARG, "n %d outside 1..2^20", n);
  if (!src || !dst || !words(src) || !words(dst))
    return api_fail(DFV_ERR_INVALID_ARG, "index list NULL or not 4-byte aligned");
  dfv::PagesParams p = {};
  p.c = cache_params(cache);
  p.a = src;
  p.b = dst;
  p.n = n;
  return launched(dfv::launch_copy_pages(p, (cudaStream_t)stream), "page copy launch");
}

int dfv_pages_reserve(const dfv_kv_cache *cache, const int32_t *seqs, const int32_t *n_new, int n, void *ws,
                      size_t ws_bytes, void *stream) {
  int st = check_list(cache, seqs, n_new, n, true);
  if (st) return st;
  // missing entries are summed in 32 bits, and n_new may ask for all of them
  if ((int64_t)n * cache->max_pages > INT32_MAX)
    return api_fail(DFV_ERR_UNSUPPORTED, "%d sequences of %d table entries: at most 2^31 - 1 in all", n, cache->max_pages);
  if ((st = check_ws(ws, ws_bytes, page_ws(cache, nullptr).bytes))) return st;
  const PageWs w = page_ws(cache, ws);
  dfv::PagesParams p = {};
  p.c = cache_params(cache);
  p.a = seqs;
  p.b = n_new;
  p.n = n;
  p.got = w.got;
  return launched(dfv::launch_reserve(p, (cudaStream_t)stream), "page reservation launch");
}

int dfv_pages_fork(const dfv_kv_cache *cache, const int32_t *src, const int32_t *dst, int n, void *ws,
                   size_t ws_bytes, void *stream) {
  int st = check_list(cache, src, dst, n, true);
  if (st) return st;
  if ((st = check_ws(ws, ws_bytes, page_ws(cache, nullptr).bytes))) return st;
  const PageWs w = page_ws(cache, ws);
  dfv::PagesParams p = {};
  p.c = cache_params(cache);
  p.a = src;
  p.b = dst;
  p.n = n;
  p.got = w.got;
  p.plan = w.plan;
  return launched(dfv::launch_fork(p, (cudaStream_t)stream), "fork launch");
}

int dfv_pages_free(const dfv_kv_cache *cache, const int32_t *seqs, int n, void *stream) {
  int st = check_list(cache, seqs, seqs, n, true);
  if (st) return st;
  dfv::PagesParams p = {};
  p.c = cache_params(cache);
  p.a = seqs;
  p.n = n;
  return launched(dfv::launch_free(p, (cudaStream_t)stream), "page release launch");
}

}  // extern "C"
