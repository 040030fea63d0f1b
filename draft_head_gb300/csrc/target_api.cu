// C ABI of the target's side of a cycle: argument checks and dispatch of
// domino_qk_norm_rope, domino_block_attention and domino_sample, of their forms for
// a cache in pages and of domino_token_logprobs. Declarations and the meaning of
// every argument: domino.h.
#include <math.h>

#include "common.cuh"
#include "pages.cuh"

namespace domino {

namespace {

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

domino_status check_ws(void* ws, size_t ws_bytes, size_t need) {
  if (!ws || ((uintptr_t)ws & 255u) || ws_bytes < need) return DOMINO_ERR_WORKSPACE;
  return DOMINO_OK;
}

inline domino_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return DOMINO_OK;
  if (e == cudaErrorInvalidConfiguration) return DOMINO_ERR_UNSUPPORTED;
  return DOMINO_ERR_CUDA;
}

// A row or head stride: whole 16-byte units, not negative.
inline bool stride_ok(int64_t s, int dtype) { return s >= 0 && (s & (dtype == DOMINO_BF16 ? 7 : 3)) == 0; }

domino_status check_cache(const domino_kv_cache* c) {
  if (!c) return DOMINO_ERR_INVALID_ARG;
  if (c->dtype != DOMINO_F32 && c->dtype != DOMINO_BF16) return DOMINO_ERR_INVALID_ARG;
  if (c->batch < 0 || c->n_kv_heads <= 0 || c->head_dim <= 0 || c->capacity <= 0) return DOMINO_ERR_INVALID_ARG;
  if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return DOMINO_ERR_INVALID_ARG;
  if (!stride_ok(c->request_stride, c->dtype) || !stride_ok(c->head_stride, c->dtype) ||
      !stride_ok(c->slot_stride, c->dtype))
    return DOMINO_ERR_INVALID_ARG;
  if (c->head_dim > 256 || (c->head_dim & 7) || c->batch > 65535 || c->n_kv_heads > 1024)
    return DOMINO_ERR_UNSUPPORTED;
  return DOMINO_OK;
}

domino_status check_block(const domino_kv_cache* c, const domino_block* b, int n_q_heads, bool device) {
  if (!b || n_q_heads < 0) return DOMINO_ERR_INVALID_ARG;
  if (b->tokens < 0 || b->max_q < 0 || b->max_ctx < 0) return DOMINO_ERR_INVALID_ARG;
  if ((int64_t)b->max_q * c->batch < b->tokens) return DOMINO_ERR_INVALID_ARG;
  if (device && b->tokens > 0) {
    if (!b->ctx_len) return DOMINO_ERR_INVALID_ARG;
    if (!b->q_start && (int64_t)b->max_q * c->batch != b->tokens) return DOMINO_ERR_INVALID_ARG;
  }
  if (n_q_heads % c->n_kv_heads) return DOMINO_ERR_INVALID_ARG;
  if (n_q_heads > 8192) return DOMINO_ERR_UNSUPPORTED;
  return DOMINO_OK;
}

RowsArgs rows_of(const domino_kv_cache* c, const domino_block* b) {
  return RowsArgs{c->batch, b->tokens, b->max_q, b->max_ctx, c->capacity, b->q_start, b->ctx_len, b->positions};
}

AttnArgs attn_args(const domino_kv_cache* c, const domino_block* b, int n_q_heads) {
  AttnArgs a = {};
  a.rows = rows_of(c, b);
  a.dtype = c->dtype; a.hq = n_q_heads; a.hkv = c->n_kv_heads; a.D = c->head_dim;
  a.k = c->k; a.v = c->v;
  a.rs = c->request_stride; a.hs = c->head_stride; a.ss = c->slot_stride;
  return a;
}

// The checks and arguments of norm and rotation; nothing is filled in for a block without rows.
domino_status norm_rope_args(const domino_kv_cache* cache, const domino_block* block, int n_q_heads, const void* q, int64_t q_stride,
                             const void* k, int64_t k_stride, const void* v, int64_t v_stride, const void* q_weight,
                             const void* k_weight, float eps, const float* rope, int max_pos, int rot_dim, int interleaved,
                             void* q_out, void* ws, size_t ws_bytes, NormRopeArgs* args) {
  domino_status st = check_block(cache, block, n_q_heads, true);
  if (st != DOMINO_OK) return st;
  if (!(eps >= 0.0f) || !isfinite(eps)) return DOMINO_ERR_INVALID_ARG;
  if (rot_dim < 0 || (rot_dim & 1) || rot_dim > cache->head_dim || max_pos < 0) return DOMINO_ERR_INVALID_ARG;
  if (rot_dim > 0 && (!rope || !aligned16(rope))) return DOMINO_ERR_INVALID_ARG;
  if (block->tokens == 0) return DOMINO_OK;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return DOMINO_ERR_INVALID_ARG;
  if (n_q_heads > 0 && (!q || !q_out || !aligned16(q) || !aligned16(q_out))) return DOMINO_ERR_INVALID_ARG;
  if (!stride_ok(q_stride, cache->dtype) || !stride_ok(k_stride, cache->dtype) || !stride_ok(v_stride, cache->dtype))
    return DOMINO_ERR_INVALID_ARG;
  if ((q_weight && !aligned16(q_weight)) || (k_weight && !aligned16(k_weight))) return DOMINO_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, 256)) != DOMINO_OK) return st;
  NormRopeArgs& a = *args;
  a = NormRopeArgs{};
  a.norm = 1;
  a.rows = rows_of(cache, block);
  a.dtype = cache->dtype; a.hq = n_q_heads; a.hkv = cache->n_kv_heads; a.D = cache->head_dim;
  a.rot = rot_dim; a.interleaved = interleaved != 0; a.max_pos = max_pos;
  a.q = q; a.k = k; a.v = v;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.q_weight = q_weight; a.k_weight = k_weight;
  a.eps = eps; a.rope = rope;
  a.q_out = q_out; a.k_cache = cache->k; a.v_cache = cache->v;
  a.rs = cache->request_stride; a.hs = cache->head_stride; a.ss = cache->slot_stride;
  a.ctl = (Ctl*)ws;
  return DOMINO_OK;
}

// What a cache in pages is to the checks of a block's rows: its batch, heads and type of rows, and as many slots as a row of
// the table has places for.
domino_status check_pages(const domino_paged_cache* c, domino_kv_cache* rows) {
  if (!c) return DOMINO_ERR_INVALID_ARG;
  const bool e4m3 = c->dtype == DOMINO_E4M3;
  if (c->dtype != DOMINO_F32 && c->dtype != DOMINO_BF16 && !e4m3) return DOMINO_ERR_INVALID_ARG;
  if (c->batch < 0 || c->n_kv_heads <= 0 || c->head_dim <= 0 || c->n_pages <= 0 || c->page_size <= 0 || c->max_pages <= 0)
    return DOMINO_ERR_INVALID_ARG;
  if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return DOMINO_ERR_INVALID_ARG;
  const int64_t st[3] = {c->page_stride, c->head_stride, c->slot_stride};
  for (int64_t s : st)
    if (e4m3 ? s < 0 || (s & 15) : !stride_ok(s, c->dtype)) return DOMINO_ERR_INVALID_ARG;
  if ((c->batch > 0 && !c->page_table) || ((uintptr_t)c->page_table & 3u) || (c->batch > 1 && c->table_stride < c->max_pages)) return DOMINO_ERR_INVALID_ARG;
  if (e4m3 && (!c->k_scale || !c->v_scale || !aligned16(c->k_scale) || !aligned16(c->v_scale))) return DOMINO_ERR_INVALID_ARG;
  if (c->head_dim > 256 || (c->head_dim & (e4m3 ? 15 : 7)) || c->batch > 65535 || c->n_kv_heads > 1024) return DOMINO_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 4096 || (c->page_size & (c->page_size - 1))) return DOMINO_ERR_UNSUPPORTED;
  const int64_t capacity = (int64_t)c->max_pages * c->page_size;
  *rows = domino_kv_cache{e4m3 ? DOMINO_BF16 : c->dtype, c->batch, c->n_kv_heads, c->head_dim,
                          (int32_t)(capacity < 0x7fffff00 ? capacity : 0x7fffff00), c->k, c->v, 0, c->head_stride, c->slot_stride};
  return DOMINO_OK;
}

PagesArgs pages_of(const domino_paged_cache* c) {
  int shift = 0;
  while ((1 << shift) < c->page_size) ++shift;
  return PagesArgs{c->page_table, c->table_stride, c->page_stride, c->n_pages, shift, c->k_scale, c->v_scale};
}

size_t attention_ws_bytes(const AttnArgs& a) { return 256 + ((attn_ws_bytes(a) + 255) & ~(size_t)255); }

domino_status attention(AttnArgs a, const void* q, float scale, int mask_mode, const uint8_t* mask, int window, int sinks, void* out,
                        float* lse, void* ws, size_t ws_bytes, void* stream) {
  if (a.hq == 0 || !(scale >= 0.0f) || !isfinite(scale) || window < 0 || sinks < 0) return DOMINO_ERR_INVALID_ARG;
  if (mask_mode != DOMINO_MASK_CAUSAL && mask_mode != DOMINO_MASK_FULL && mask_mode != DOMINO_MASK_TREE)
    return DOMINO_ERR_INVALID_ARG;
  if (a.rows.tokens == 0) return DOMINO_OK;
  if (mask_mode == DOMINO_MASK_TREE && !mask) return DOMINO_ERR_INVALID_ARG;
  if (!q || !out || !aligned16(q) || !aligned16(out)) return DOMINO_ERR_INVALID_ARG;
  const domino_status st = check_ws(ws, ws_bytes, attention_ws_bytes(a));
  if (st != DOMINO_OK) return st;
  a.q = q; a.scale = scale; a.mode = mask_mode; a.mask = mask; a.window = window; a.sinks = sinks;
  a.out = out; a.lse = lse;
  a.ctl = (Ctl*)ws;
  a.scratch = (uint8_t*)ws + 256;
  return cuda_status(launch_attention(a, (cudaStream_t)stream));
}

AttnArgs paged_attn_args(const domino_paged_cache* c, const domino_kv_cache* rows, const domino_block* b, int n_q_heads) {
  AttnArgs a = attn_args(rows, b, n_q_heads);
  a.cache = c->dtype == DOMINO_E4M3 ? kPagedE4m3 : kPaged;
  a.pages = pages_of(c);
  return a;
}

}  // namespace
}  // namespace domino

using namespace domino;

extern "C" {

domino_status domino_qk_norm_rope(const domino_kv_cache* cache, const domino_block* block, int n_q_heads,
                                  const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                  const void* v, int64_t v_stride, const void* q_weight,
                                  const void* k_weight, float eps, const float* rope, int max_pos, int rot_dim,
                                  int interleaved, void* q_out, void* ws, size_t ws_bytes, void* stream) {
  domino_status st = check_cache(cache);
  if (st != DOMINO_OK) return st;
  NormRopeArgs a;
  if ((st = norm_rope_args(cache, block, n_q_heads, q, q_stride, k, k_stride, v, v_stride, q_weight, k_weight, eps, rope, max_pos,
                           rot_dim, interleaved, q_out, ws, ws_bytes, &a)) != DOMINO_OK)
    return st;
  if (block->tokens == 0) return DOMINO_OK;
  return cuda_status(launch_norm_rope(a, (cudaStream_t)stream));
}

size_t domino_block_attention_workspace_bytes(const domino_kv_cache* cache, const domino_block* block,
                                              int n_q_heads) {
  if (check_cache(cache) != DOMINO_OK || check_block(cache, block, n_q_heads, false) != DOMINO_OK) return 0;
  return attention_ws_bytes(attn_args(cache, block, n_q_heads));
}

domino_status domino_block_attention(const domino_kv_cache* cache, const domino_block* block, int n_q_heads,
                                     const void* q, float scale, int mask_mode, const uint8_t* mask, int window,
                                     int sinks, void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  domino_status st = check_cache(cache);
  if (st != DOMINO_OK) return st;
  if ((st = check_block(cache, block, n_q_heads, true)) != DOMINO_OK) return st;
  return attention(attn_args(cache, block, n_q_heads), q, scale, mask_mode, mask, window, sinks, out, lse, ws, ws_bytes, stream);
}

domino_status domino_sample(int dtype, const void* logits, int64_t logits_stride, int rows, int V,
                            const float* temperature, const int32_t* top_k, const float* top_p,
                            const float* min_p, const float* gumbel, int64_t gumbel_stride, int32_t* tokens,
                            float* logprob, void* ws, size_t ws_bytes, void* stream) {
  if (dtype != DOMINO_F32 && dtype != DOMINO_BF16) return DOMINO_ERR_INVALID_ARG;
  if (rows < 0 || V <= 0) return DOMINO_ERR_INVALID_ARG;
  if (rows == 0) return DOMINO_OK;
  if (!logits || !tokens || (!gumbel && !temperature)) return DOMINO_ERR_INVALID_ARG;
  if (((uintptr_t)logits & (dtype == DOMINO_BF16 ? 1u : 3u)) || ((uintptr_t)gumbel & 3u)) return DOMINO_ERR_INVALID_ARG;
  if (rows > 1 && (logits_stride < V || (gumbel && gumbel_stride < V))) return DOMINO_ERR_INVALID_ARG;
  domino_status st = check_ws(ws, ws_bytes, 256);
  if (st != DOMINO_OK) return st;
  SampleArgs a;
  a.dtype = dtype; a.rows = rows; a.V = V;
  a.logits = logits; a.ls = logits_stride;
  a.temperature = temperature; a.top_k = top_k; a.top_p = top_p; a.min_p = min_p;
  a.gumbel = gumbel; a.gs = gumbel_stride;
  a.tokens = tokens; a.logprob = logprob;
  a.ctl = (Ctl*)ws;
  return cuda_status(launch_sample(a, (cudaStream_t)stream));
}

domino_status domino_paged_append(const domino_paged_cache* cache, const domino_block* block, int n_q_heads,
                                  const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                  const void* v, int64_t v_stride, int norm, const void* q_weight,
                                  const void* k_weight, float eps, const float* rope, int max_pos, int rot_dim,
                                  int interleaved, void* q_out, void* ws, size_t ws_bytes, void* stream) {
  domino_kv_cache rows;
  domino_status st = check_pages(cache, &rows);
  if (st != DOMINO_OK) return st;
  if (!norm && (q_weight || k_weight)) return DOMINO_ERR_INVALID_ARG;
  NormRopeArgs a;
  if ((st = norm_rope_args(&rows, block, n_q_heads, q, q_stride, k, k_stride, v, v_stride, q_weight, k_weight, eps, rope, max_pos,
                           rot_dim, interleaved, q_out, ws, ws_bytes, &a)) != DOMINO_OK)
    return st;
  if (block->tokens == 0) return DOMINO_OK;
  a.norm = norm != 0;
  a.e4m3 = cache->dtype == DOMINO_E4M3;
  a.pages = pages_of(cache);
  return cuda_status(launch_paged_append(a, (cudaStream_t)stream));
}

domino_status domino_paged_read(const domino_paged_cache* cache, const int32_t* first, const int32_t* count, int max_count,
                                const domino_kv_cache* out, void* ws, size_t ws_bytes, void* stream) {
  domino_kv_cache rows;
  domino_status st = check_pages(cache, &rows);
  if (st != DOMINO_OK) return st;
  if ((st = check_cache(out)) != DOMINO_OK) return st;
  if (out->dtype != rows.dtype || out->batch != cache->batch || out->n_kv_heads != cache->n_kv_heads ||
      out->head_dim != cache->head_dim || max_count < 0 || max_count > out->capacity)
    return DOMINO_ERR_INVALID_ARG;
  if (cache->batch == 0 || max_count == 0) return DOMINO_OK;
  if (!count) return DOMINO_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, 256)) != DOMINO_OK) return st;
  PagedReadArgs a;
  a.dtype = rows.dtype; a.e4m3 = cache->dtype == DOMINO_E4M3;
  a.batch = cache->batch; a.hkv = cache->n_kv_heads; a.D = cache->head_dim;
  a.capacity = rows.capacity; a.max_count = max_count;
  a.first = first; a.count = count;
  a.k = cache->k; a.v = cache->v; a.hs = cache->head_stride; a.ss = cache->slot_stride;
  a.pages = pages_of(cache);
  a.k_out = out->k; a.v_out = out->v; a.out_capacity = out->capacity;
  a.out_rs = out->request_stride; a.out_hs = out->head_stride; a.out_ss = out->slot_stride;
  a.ctl = (Ctl*)ws;
  return cuda_status(launch_paged_read(a, (cudaStream_t)stream));
}

size_t domino_paged_attention_workspace_bytes(const domino_paged_cache* cache, const domino_block* block, int n_q_heads) {
  domino_kv_cache rows;
  if (check_pages(cache, &rows) != DOMINO_OK || check_block(&rows, block, n_q_heads, false) != DOMINO_OK) return 0;
  return attention_ws_bytes(paged_attn_args(cache, &rows, block, n_q_heads));
}

domino_status domino_paged_attention(const domino_paged_cache* cache, const domino_block* block, int n_q_heads,
                                     const void* q, float scale, int mask_mode, const uint8_t* mask, int window,
                                     int sinks, void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  domino_kv_cache rows;
  domino_status st = check_pages(cache, &rows);
  if (st != DOMINO_OK) return st;
  if ((st = check_block(&rows, block, n_q_heads, true)) != DOMINO_OK) return st;
  return attention(paged_attn_args(cache, &rows, block, n_q_heads), q, scale, mask_mode, mask, window, sinks, out, lse, ws, ws_bytes,
                   stream);
}

domino_status domino_token_logprobs(int dtype, const void* logits, int64_t logits_stride, int rows, int V,
                                    const int32_t* tokens, const float* temperature, int top_n, float* logprob,
                                    int32_t* rank, float* entropy, float* lse, int32_t* top_ids, float* top_logprob,
                                    void* ws, size_t ws_bytes, void* stream) {
  if (dtype != DOMINO_F32 && dtype != DOMINO_BF16) return DOMINO_ERR_INVALID_ARG;
  if (rows < 0 || V <= 0 || top_n < 0) return DOMINO_ERR_INVALID_ARG;
  if (top_n > 32) return DOMINO_ERR_UNSUPPORTED;
  if (rows == 0) return DOMINO_OK;
  if (!logits || ((uintptr_t)logits & (dtype == DOMINO_BF16 ? 1u : 3u)) || (rows > 1 && logits_stride < V)) return DOMINO_ERR_INVALID_ARG;
  const domino_status st = check_ws(ws, ws_bytes, 256);
  if (st != DOMINO_OK) return st;
  ScoreArgs a;
  a.dtype = dtype; a.rows = rows; a.V = V; a.top_n = top_ids || top_logprob ? top_n : 0;
  a.logits = logits; a.ls = logits_stride;
  a.tokens = tokens; a.temperature = temperature;
  a.logprob = logprob; a.rank = rank; a.entropy = entropy; a.lse = lse;
  a.top_ids = top_ids; a.top_logprob = top_logprob;
  a.ctl = (Ctl*)ws;
  return cuda_status(launch_score(a, (cudaStream_t)stream));
}

}  // extern "C"
