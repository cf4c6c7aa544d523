// Launchers of the paged-cache kernels and of the head norms.
#pragma once

#include "paged.cuh"

int launch_norm_rope(const tq_heads *q, const tq_heads *k, int dtype, int w_dtype, int d, int N, float eps,
                     const int32_t *pos, const float *rc, const float *rs, int rope_len, cudaStream_t stream);
int launch_paged_quantize(const tq_codec *c, const PagedView &p, const void *k, const void *v, int dtype,
                          int64_t st, int64_t sh, const float *rc, const float *rs, const tq_cache *cache,
                          uint32_t *status, cudaStream_t stream);
int launch_paged_dequant(const tq_codec *c, const PagedView &p, const tq_cache *cache, void *k_out,
                         void *v_out, int out_dtype, cudaStream_t stream);
size_t paged_attn_workspace_bytes(const tq_codec *c, int N, int num_seqs, int max_new, int max_len, int Hq,
                                  int Hkv);
int launch_paged_attention(const tq_codec *c, const PagedView &p, const void *q, int dtype, int64_t st,
                           int64_t sh, int Hq, const tq_cache *cache, float scale, const float *rc,
                           const float *rs, void *ws, void *out, int out_dtype, cudaStream_t stream);
