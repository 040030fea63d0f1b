// C ABI of the target's side of a cycle: argument checks and dispatch of
// domino_qk_norm_rope, domino_block_attention and domino_sample. Declarations
// and the meaning of every argument: domino.h.
#include <math.h>

#include "common.cuh"

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
  if ((st = check_block(cache, block, n_q_heads, true)) != DOMINO_OK) return st;
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
  NormRopeArgs a;
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
  return cuda_status(launch_norm_rope(a, (cudaStream_t)stream));
}

size_t domino_block_attention_workspace_bytes(const domino_kv_cache* cache, const domino_block* block,
                                              int n_q_heads) {
  if (check_cache(cache) != DOMINO_OK || check_block(cache, block, n_q_heads, false) != DOMINO_OK) return 0;
  return 256 + ((attn_ws_bytes(attn_args(cache, block, n_q_heads)) + 255) & ~(size_t)255);
}

domino_status domino_block_attention(const domino_kv_cache* cache, const domino_block* block, int n_q_heads,
                                     const void* q, float scale, int mask_mode, const uint8_t* mask, int window,
                                     int sinks, void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  domino_status st = check_cache(cache);
  if (st != DOMINO_OK) return st;
  if ((st = check_block(cache, block, n_q_heads, true)) != DOMINO_OK) return st;
  if (n_q_heads == 0 || !(scale >= 0.0f) || !isfinite(scale) || window < 0 || sinks < 0) return DOMINO_ERR_INVALID_ARG;
  if (mask_mode != DOMINO_MASK_CAUSAL && mask_mode != DOMINO_MASK_FULL && mask_mode != DOMINO_MASK_TREE)
    return DOMINO_ERR_INVALID_ARG;
  if (block->tokens == 0) return DOMINO_OK;
  if (mask_mode == DOMINO_MASK_TREE && !mask) return DOMINO_ERR_INVALID_ARG;
  if (!q || !out || !aligned16(q) || !aligned16(out)) return DOMINO_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, domino_block_attention_workspace_bytes(cache, block, n_q_heads))) != DOMINO_OK)
    return st;
  AttnArgs a = attn_args(cache, block, n_q_heads);
  a.q = q; a.scale = scale; a.mode = mask_mode; a.mask = mask; a.window = window; a.sinks = sinks;
  a.out = out; a.lse = lse;
  a.ctl = (Ctl*)ws;
  a.scratch = (uint8_t*)ws + 256;
  return cuda_status(launch_attention(a, (cudaStream_t)stream));
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

}  // extern "C"
