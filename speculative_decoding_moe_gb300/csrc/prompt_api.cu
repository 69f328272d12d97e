// prompt_api.cu -- the prompt part of the C ABI: argument validation.
// Everything is checked on the host before any launch.
#include <cmath>

#include "tree_common.cuh"

namespace {

using namespace dfv;

int check_rows(const dfv_row_batch *r, const char *what) {
  if (!r) return api_fail(DFV_ERR_INVALID_ARG, "%s is NULL", what);
  if (r->n_seqs < 1 || r->n_seqs > DFV_MAX_TREE_SEQS)
    return api_fail(DFV_ERR_INVALID_ARG, "%s: n_seqs %d outside 1..%d", what, r->n_seqs, DFV_MAX_TREE_SEQS);
  if (r->n_rows < 1 || r->n_rows > DFV_MAX_ROWS)
    return api_fail(DFV_ERR_INVALID_ARG, "%s: n_rows %d outside 1..%d", what, r->n_rows, DFV_MAX_ROWS);
  if (r->max_rows < 1 || r->max_rows > DFV_MAX_ROWS)
    return api_fail(DFV_ERR_INVALID_ARG, "%s: max_rows %d outside 1..%d", what, r->max_rows, DFV_MAX_ROWS);
  if (!r->row_off || !words(r->row_off) || !words(r->seq))
    return api_fail(DFV_ERR_INVALID_ARG, "%s: row_off NULL, or row_off/seq not 4-byte aligned", what);
  return DFV_OK;
}

TreeParams row_params(const dfv_row_batch *r) {
  TreeParams p = {};
  p.n_seqs = r->n_seqs;
  p.n_rows = r->n_rows;
  p.max_nodes = r->max_rows;
  p.seq = r->seq;
  p.row_off = r->row_off;
  return p;
}

// Rows or heads of an output that certainly share elements.
bool overlap(int rows, int heads, int head_dim, int64_t row, int64_t head) {
  return (rows > 1 && row < head_dim) || (heads > 1 && head < head_dim) || (rows > 1 && heads > 1 && row == head);
}

int check_prompt(const dfv_row_batch *rows, int n_heads, int n_kv_heads, int head_dim) {
  const int st = check_rows(rows, "rows");
  if (st) return st;
  if (head_dim != 64 && head_dim != 128)
    return api_fail(DFV_ERR_UNSUPPORTED, "attention takes head_dim 64 or 128, not %d", head_dim);
  if (n_kv_heads < 1 || n_kv_heads > 1024 || n_heads < 1 || n_heads % n_kv_heads)
    return api_fail(DFV_ERR_INVALID_ARG, "n_heads %d is no multiple of %d kv heads (1..1024)", n_heads, n_kv_heads);
  if (n_heads / n_kv_heads > 16)
    return api_fail(DFV_ERR_UNSUPPORTED, "%d query heads per kv head (at most 16)", n_heads / n_kv_heads);
  return DFV_OK;
}

}  // namespace

extern "C" {

int dfv_norm_rope_append(const dfv_kv_cache *cache, int layer, const dfv_row_batch *rows, int n_heads,
                         const void *q_gain, const void *k_gain, float eps, int rot_dim, int interleaved, float scale,
                         const uint64_t *turns, const void *q, int64_t q_row, int64_t q_head, const void *k,
                         int64_t k_row, int64_t k_head, const void *v, int64_t v_row, int64_t v_head,
                         const int32_t *positions, void *q_out, int64_t o_row, int64_t o_head, void *k_out,
                         int64_t ko_row, int64_t ko_head, void *stream) {
  int st = check_cache(cache);
  if (st) return st;
  if ((st = check_rows(rows, "rows"))) return st;
  if (!aligned(q_gain, 16) || !aligned(k_gain, 16)) return api_fail(DFV_ERR_INVALID_ARG, "gains not 16-byte aligned");
  if ((q_gain || k_gain) && !(eps >= 0.f && std::isfinite(eps)))
    return api_fail(DFV_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (!aligned(k_out, 16) || (k_out && (!stride_ok(ko_row) || !stride_ok(ko_head))))
    return api_fail(DFV_ERR_INVALID_ARG, "k_out not 16-byte aligned, or its strides no non-negative multiples of 8 elements");
  if (k_out && k_out == k && (ko_row != k_row || ko_head != k_head))
    return api_fail(DFV_ERR_INVALID_ARG, "k_out is k: the strides must be the same");
  if (k_out && (k_out == q || k_out == v || k_out == q_out))
    return api_fail(DFV_ERR_INVALID_ARG, "k_out must not be q, v or q_out");
  RopeParams p = {};
  p.c = cache_params(cache);
  p.t = row_params(rows);
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
  p.q_gain = (const char *)q_gain;
  p.k_gain = (const char *)k_gain;
  p.eps = eps;
  p.ko = (char *)k_out;
  p.ko_row = ko_row;
  p.ko_head = ko_head;
  if ((st = check_rope(cache, layer, n_heads, rot_dim, interleaved, scale, p))) return st;
  if (overlap(rows->n_rows, n_heads, cache->head_dim, o_row, o_head) ||
      (k_out && overlap(rows->n_rows, cache->n_kv_heads, cache->head_dim, ko_row, ko_head)))
    return api_fail(DFV_ERR_INVALID_ARG, "rows or heads of q_out or k_out overlap");
  return launched(launch_norm_rope_append(p, (cudaStream_t)stream), "norm and rotary append launch");
}

int dfv_cache_read(const dfv_kv_cache *cache, int layer, const dfv_row_batch *rows, void *k_out, int64_t k_row,
                   int64_t k_head, void *v_out, int64_t v_row, int64_t v_head, void *stream) {
  int st = check_cache(cache);
  if (st) return st;
  if ((st = check_rows(rows, "rows"))) return st;
  if (layer < 0 || layer >= cache->n_layers)
    return api_fail(DFV_ERR_INVALID_ARG, "layer %d outside 0..%d", layer, cache->n_layers - 1);
  if ((!k_out && !v_out) || !aligned(k_out, 16) || !aligned(v_out, 16))
    return api_fail(DFV_ERR_INVALID_ARG, "neither k_out nor v_out is given, or one is not 16-byte aligned");
  if (!stride_ok(k_row) || !stride_ok(k_head) || !stride_ok(v_row) || !stride_ok(v_head))
    return api_fail(DFV_ERR_INVALID_ARG, "row and head strides must be non-negative multiples of 8 elements");
  if ((k_out && overlap(rows->n_rows, cache->n_kv_heads, cache->head_dim, k_row, k_head)) ||
      (v_out && overlap(rows->n_rows, cache->n_kv_heads, cache->head_dim, v_row, v_head)))
    return api_fail(DFV_ERR_INVALID_ARG, "rows or heads of k_out or v_out overlap");
  if (k_out == v_out) return api_fail(DFV_ERR_INVALID_ARG, "k_out must not be v_out");
  CacheReadParams p = {};
  p.c = cache_params(cache);
  p.t = row_params(rows);
  p.layer = layer;
  p.k = (char *)k_out;
  p.v = (char *)v_out;
  p.k_row = k_row;
  p.k_head = k_head;
  p.v_row = v_row;
  p.v_head = v_head;
  return launched(launch_cache_read(p, (cudaStream_t)stream), "cache read launch");
}

size_t dfv_prompt_attention_workspace_size(const dfv_row_batch *rows, int n_heads, int n_kv_heads, int head_dim) {
  if (check_prompt(rows, n_heads, n_kv_heads, head_dim)) return 0;
  return prompt_attn_ws(head_dim);
}

int dfv_prompt_attention(int dtype, const dfv_row_batch *rows, const dfv_row_batch *keys, int n_heads, int n_kv_heads,
                         int head_dim, float scale, const void *q, int64_t q_row, int64_t q_head, const void *k,
                         int64_t k_row, int64_t k_head, const void *v, int64_t v_row, int64_t v_head, void *out,
                         int64_t o_row, int64_t o_head, float *opt_lse, uint32_t *opt_err, void *ws, size_t ws_bytes,
                         void *stream) {
  if (dtype != DFV_BF16 && dtype != DFV_F16) return api_fail(DFV_ERR_UNSUPPORTED, "attention dtype %d", dtype);
  int st = check_prompt(rows, n_heads, n_kv_heads, head_dim);
  if (st) return st;
  if (!keys) keys = rows;
  if ((st = check_rows(keys, "keys"))) return st;
  if (keys->n_seqs != rows->n_seqs)
    return api_fail(DFV_ERR_INVALID_ARG, "keys of %d sequences, rows of %d", keys->n_seqs, rows->n_seqs);
  if (!(scale > 0.f) || !std::isfinite(scale)) return api_fail(DFV_ERR_INVALID_ARG, "scale must be positive");
  if (!q || !k || !v || !out || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16))
    return api_fail(DFV_ERR_INVALID_ARG, "q/k/v/out NULL or not 16-byte aligned");
  if (out == q || out == k || out == v) return api_fail(DFV_ERR_INVALID_ARG, "out must not be q, k or v");
  if (!words(opt_lse) || !words(opt_err)) return api_fail(DFV_ERR_INVALID_ARG, "lse/err not 4-byte aligned");
  const int64_t most = (int64_t)1 << 36;  // what a tensor map's strides hold
  for (const int64_t s : {q_row, q_head, k_row, k_head, v_row, v_head, o_row, o_head})
    if (!stride_ok(s) || s >= most)
      return api_fail(DFV_ERR_INVALID_ARG, "row and head strides must be non-negative multiples of 8 elements below 2^36");
  if ((keys->n_rows > 1 && (k_row == 0 || v_row == 0)) || (n_kv_heads > 1 && (k_head == 0 || v_head == 0)))
    return api_fail(DFV_ERR_UNSUPPORTED, "k and v with a stride of 0");
  if ((rows->n_rows > 1 && q_row == 0) || (n_heads > 1 && q_head == 0))
    return api_fail(DFV_ERR_UNSUPPORTED, "q with a stride of 0");
  if (overlap(rows->n_rows, n_heads, head_dim, o_row, o_head))
    return api_fail(DFV_ERR_INVALID_ARG, "rows or heads of out overlap");
  if ((st = check_ws(ws, ws_bytes, prompt_attn_ws(head_dim)))) return st;
  PromptParams p = {};
  p.n_seqs = rows->n_seqs;
  p.n_rows = rows->n_rows;
  p.max_rows = rows->max_rows;
  p.n_keys = keys->n_rows;
  p.max_keys = keys->max_rows;
  p.row_off = rows->row_off;
  p.key_off = keys->row_off;
  p.H = n_heads;
  p.Hkv = n_kv_heads;
  p.G = n_heads / n_kv_heads;
  p.D = head_dim;
  p.f16 = dtype == DFV_F16;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.q = (const char *)q;
  p.o = (char *)out;
  p.q_row = q_row;
  p.q_head = q_head;
  p.o_row = o_row;
  p.o_head = o_head;
  p.k = (const char *)k;
  p.v = (const char *)v;
  p.k_row = k_row;
  p.k_head = k_head;
  p.v_row = v_row;
  p.v_head = v_head;
  p.lse = opt_lse;
  p.kverr = opt_err;
  p.err = (unsigned *)((char *)ws + kWsErr);
  char why[256] = {0};
  const cudaError_t e = launch_prompt_attn(p, ws, (cudaStream_t)stream, why, sizeof why);
  if (e != cudaSuccess && why[0]) return api_fail(DFV_ERR_CUDA, "prompt attention: %s", why);
  return launched(e, "prompt attention launch");
}

}  // extern "C"
