// C ABI entry points of the paged-cache calls and of the head norms with the
// position rotation: argument validation and dispatch.
#include <cmath>

#include "paged.h"

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool dtype_ok(int t) { return t == TQ_F32 || t == TQ_BF16; }

size_t elem(int t) { return t == TQ_BF16 ? 2 : 4; }

// Checks shared by the paged calls; fills the device view.
int paged_view(const char *who, const tq_codec *c, const tq_cache *cache, const tq_paged_batch *b, int N,
               PagedView *v) {
  const std::string w(who);
  if (!c) return tq_fail(TQ_ERR_INVALID_ARG, w + ": NULL codec");
  if (c->d > 128) return tq_fail(TQ_ERR_UNSUPPORTED, w + ": paged calls support d = 64 and 128");
  if (!cache || !cache->kcode || !cache->kscale || !cache->vcode || !cache->vnorm)
    return tq_fail(TQ_ERR_INVALID_ARG, w + ": every cache plane is required");
  if (cache->B <= 0 || cache->Hkv <= 0)
    return tq_fail(TQ_ERR_INVALID_ARG, w + ": cache needs B (pages) and Hkv > 0");
  if (cache->Hkv > 65535 || static_cast<int64_t>(N) * cache->Hkv > INT32_MAX)
    return tq_fail(TQ_ERR_INVALID_ARG, w + ": at most 65535 KV heads and 2^31 - 1 rows (tokens x KV heads) a call");
  const int64_t P = cache->rows_cap;
  if (P < 32 || (P & (P - 1)) || P > (1 << 20))
    return tq_fail(TQ_ERR_INVALID_ARG, w + ": the page size (rows_cap) must be a power of two, 32 to 2^20");
  if (!aligned(cache->kcode, 16) || !aligned(cache->kscale, 16) || !aligned(cache->vcode, 16) ||
      !aligned(cache->vnorm, 16))
    return tq_fail(TQ_ERR_ALIGNMENT, w + ": every cache plane needs 16-byte alignment");
  if (!b) return tq_fail(TQ_ERR_INVALID_ARG, w + ": NULL batch");
  if (N < 0 || b->num_seqs < 0 || b->max_new < 0 || b->max_seq_len < 0 || b->max_pages < 0)
    return tq_fail(TQ_ERR_INVALID_ARG, w + ": negative size");
  if (N > (1 << 24) || b->num_seqs > 65535)
    return tq_fail(TQ_ERR_INVALID_ARG, w + ": at most 2^24 tokens and 65535 sequences a call");
  if (b->max_seq_len > (1 << 30) || b->max_seq_len > b->max_pages * P)
    return tq_fail(TQ_ERR_INVALID_ARG, w + ": max_seq_len exceeds max_pages pages (or 2^30)");
  if (N > 0 && b->num_seqs > 0) {
    if (!b->q_start || !b->seq_lens || (b->max_pages > 0 && !b->page_table))
      return tq_fail(TQ_ERR_INVALID_ARG, w + ": NULL page_table, q_start or seq_lens");
    if (b->table_stride < b->max_pages)
      return tq_fail(TQ_ERR_INVALID_ARG, w + ": table_stride smaller than max_pages");
    if (!aligned(b->page_table, 4) || !aligned(b->q_start, 4) || !aligned(b->seq_lens, 4))
      return tq_fail(TQ_ERR_ALIGNMENT, w + ": page_table, q_start and seq_lens need 4-byte alignment");
  }
  v->table = b->page_table;
  v->q_start = b->q_start;
  v->seq_lens = b->seq_lens;
  v->table_stride = b->table_stride;
  v->num_seqs = b->num_seqs;
  v->max_pages = b->max_pages;
  v->max_new = std::min(b->max_new, N);
  v->max_len = b->max_seq_len;
  v->N = N;
  v->num_pages = cache->B;
  v->page_shift = 0;
  while ((int64_t{1} << v->page_shift) < P) ++v->page_shift;
  return TQ_OK;
}

bool empty(const PagedView &v) { return v.N == 0 || v.num_seqs == 0 || v.max_new == 0; }

int check_rope(const char *who, const float *rc, const float *rs, int rope_len, int need) {
  const std::string w(who);
  if ((rc == nullptr) != (rs == nullptr))
    return tq_fail(TQ_ERR_INVALID_ARG, w + ": rope_cos and rope_sin go together");
  if (rc && rope_len < need)
    return tq_fail(TQ_ERR_INVALID_ARG, w + ": the rope table has fewer rows than the positions need");
  if (!aligned(rc, 4) || !aligned(rs, 4)) return tq_fail(TQ_ERR_ALIGNMENT, w + ": rope table alignment");
  return TQ_OK;
}

int check_heads(const char *name, const tq_heads *h, int N, int dtype, int w_dtype) {
  const std::string w = std::string("qk_norm_rope: ") + name;
  if (h->heads < 0) return tq_fail(TQ_ERR_INVALID_ARG, w + ": negative head count");
  if (h->heads == 0 || N == 0) return TQ_OK;
  if (!h->x || !h->y) return tq_fail(TQ_ERR_INVALID_ARG, w + ": NULL input or output");
  if (!aligned(h->x, elem(dtype)) || !aligned(h->y, elem(dtype)) || !aligned(h->weight, elem(w_dtype)))
    return tq_fail(TQ_ERR_ALIGNMENT, w + ": not aligned to the element size");
  return TQ_OK;
}

}  // namespace

extern "C" {

int tq_qk_norm_rope(const tq_heads *q, const tq_heads *k, int dtype, int weight_dtype, int d, int num_tokens,
                    float eps, const int32_t *positions, const float *rope_cos, const float *rope_sin,
                    int rope_len, void *stream) {
  if (!q && !k) return tq_fail(TQ_ERR_INVALID_ARG, "qk_norm_rope: queries or keys are required");
  if (d != 64 && d != 128) return tq_fail(TQ_ERR_UNSUPPORTED, "qk_norm_rope: d must be 64 or 128");
  if (!dtype_ok(dtype) || !dtype_ok(weight_dtype)) return tq_fail(TQ_ERR_INVALID_ARG, "qk_norm_rope: dtype");
  if (num_tokens < 0 || num_tokens > (1 << 24))
    return tq_fail(TQ_ERR_INVALID_ARG, "qk_norm_rope: num_tokens outside 0..2^24");
  if (!(eps >= 0.f) || !std::isfinite(eps))
    return tq_fail(TQ_ERR_INVALID_ARG, "qk_norm_rope: eps must be finite and >= 0");
  int64_t heads = 0;
  if (q) {
    if (int e = check_heads("queries", q, num_tokens, dtype, weight_dtype)) return e;
    heads += q->heads;
  }
  if (k) {
    if (int e = check_heads("keys", k, num_tokens, dtype, weight_dtype)) return e;
    heads += k->heads;
  }
  if (heads > 4096) return tq_fail(TQ_ERR_INVALID_ARG, "qk_norm_rope: at most 4096 heads");
  if (int e = check_rope("qk_norm_rope", rope_cos, rope_sin, rope_len, 1)) return e;
  if (num_tokens == 0 || heads == 0) return TQ_OK;
  if (rope_cos && !positions)
    return tq_fail(TQ_ERR_INVALID_ARG, "qk_norm_rope: the rotation needs positions");
  if (!aligned(positions, 4)) return tq_fail(TQ_ERR_ALIGNMENT, "qk_norm_rope: positions alignment");
  return launch_norm_rope(q, k, dtype, weight_dtype, d, num_tokens, eps, positions, rope_cos, rope_sin,
                          rope_len, static_cast<cudaStream_t>(stream));
}

int tq_paged_quantize_kv(const tq_codec *c, const void *k, const void *v, int dtype, int num_tokens,
                         int64_t stride_t, int64_t stride_h, const float *rope_cos, const float *rope_sin,
                         int rope_len, const tq_cache *cache, const tq_paged_batch *batch, uint32_t *status,
                         void *stream) {
  PagedView view;
  if (int e = paged_view("paged_quantize", c, cache, batch, num_tokens, &view)) return e;
  if (!dtype_ok(dtype)) return tq_fail(TQ_ERR_INVALID_ARG, "paged_quantize: dtype");
  if (int e = check_rope("paged_quantize", rope_cos, rope_sin, rope_len, view.max_len)) return e;
  if (empty(view) || view.max_len == 0) return TQ_OK;
  if (!k || !v) return tq_fail(TQ_ERR_INVALID_ARG, "paged_quantize: NULL k or v");
  if (!aligned(k, elem(dtype)) || !aligned(v, elem(dtype)) || !aligned(status, 4))
    return tq_fail(TQ_ERR_ALIGNMENT, "paged_quantize: k/v/status not aligned to their element size");
  return launch_paged_quantize(c, view, k, v, dtype, stride_t, stride_h, rope_cos, rope_sin, cache, status,
                               static_cast<cudaStream_t>(stream));
}

int tq_paged_dequantize(const tq_codec *c, const tq_cache *cache, const tq_paged_batch *batch, int num_tokens,
                        void *k_out, void *v_out, int out_dtype, void *stream) {
  PagedView view;
  if (int e = paged_view("paged_dequantize", c, cache, batch, num_tokens, &view)) return e;
  if (!dtype_ok(out_dtype)) return tq_fail(TQ_ERR_INVALID_ARG, "paged_dequantize: dtype");
  if (!k_out && !v_out && num_tokens > 0)
    return tq_fail(TQ_ERR_INVALID_ARG, "paged_dequantize: NULL outputs");
  if (!aligned(k_out, 16) || !aligned(v_out, 16))
    return tq_fail(TQ_ERR_ALIGNMENT, "paged_dequantize: outputs need 16-byte alignment");
  if (empty(view)) return TQ_OK;
  return launch_paged_dequant(c, view, cache, k_out, v_out, out_dtype, static_cast<cudaStream_t>(stream));
}

int tq_paged_attention_workspace(const tq_codec *c, const tq_paged_batch *batch, int num_tokens, int Hq,
                                 int Hkv, size_t *bytes) {
  if (!c || !batch || !bytes || num_tokens < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || batch->num_seqs < 0 ||
      batch->max_new < 0 || batch->max_seq_len < 0)
    return tq_fail(TQ_ERR_INVALID_ARG, "paged_attention workspace: bad arguments");
  if (c->d > 128) return tq_fail(TQ_ERR_UNSUPPORTED, "paged_attention workspace: d must be 64 or 128");
  if (num_tokens > (1 << 24) || Hq > 65535 || static_cast<int64_t>(num_tokens) * Hq > INT32_MAX ||
      batch->num_seqs > 65535 || batch->max_seq_len > (1 << 30))
    return tq_fail(TQ_ERR_INVALID_ARG, "paged_attention workspace: beyond the limits of a call");
  *bytes = paged_attn_workspace_bytes(c, num_tokens, batch->num_seqs, std::min(batch->max_new, num_tokens),
                                      batch->max_seq_len, Hq, Hkv);
  return TQ_OK;
}

int tq_paged_attention(const tq_codec *c, const void *q, int dtype, int num_tokens, int Hq, int64_t stride_t,
                       int64_t stride_h, const tq_cache *cache, const tq_paged_batch *batch, float scale,
                       const float *rope_cos, const float *rope_sin, int rope_len, void *workspace,
                       size_t ws_bytes, void *out, int out_dtype, void *stream) {
  PagedView view;
  if (int e = paged_view("paged_attention", c, cache, batch, num_tokens, &view)) return e;
  if (!dtype_ok(dtype) || !dtype_ok(out_dtype)) return tq_fail(TQ_ERR_INVALID_ARG, "paged_attention: dtype");
  if (Hq <= 0 || Hq % cache->Hkv || Hq > 65535)
    return tq_fail(TQ_ERR_INVALID_ARG, "paged_attention: Hq must be a multiple of Hkv, at most 65535");
  if (static_cast<int64_t>(num_tokens) * Hq > INT32_MAX)
    return tq_fail(TQ_ERR_INVALID_ARG, "paged_attention: at most 2^31 - 1 rows (tokens x query heads) a call");
  if (!std::isfinite(scale)) return tq_fail(TQ_ERR_INVALID_ARG, "paged_attention: scale not finite");
  if (int e = check_rope("paged_attention", rope_cos, rope_sin, rope_len, view.max_len)) return e;
  if (empty(view)) return TQ_OK;
  if (!q || !out) return tq_fail(TQ_ERR_INVALID_ARG, "paged_attention: NULL q or out");
  if (!aligned(q, elem(dtype)) || !aligned(out, 16))
    return tq_fail(TQ_ERR_ALIGNMENT, "paged_attention: q needs its element's, out 16-byte alignment");
  const size_t need = paged_attn_workspace_bytes(c, num_tokens, view.num_seqs, view.max_new, view.max_len, Hq,
                                                 cache->Hkv);
  if (need > 0 && (!workspace || ws_bytes < need))
    return tq_fail(TQ_ERR_WORKSPACE, "paged_attention: workspace smaller than tq_paged_attention_workspace()");
  if (!aligned(workspace, 16)) return tq_fail(TQ_ERR_ALIGNMENT, "paged_attention: workspace alignment");
  return launch_paged_attention(c, view, q, dtype, stride_t, stride_h, Hq, cache, scale, rope_cos, rope_sin,
                                workspace, out, out_dtype, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
