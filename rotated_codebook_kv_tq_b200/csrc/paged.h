// Launchers of the paged-cache kernels and of the head norms.
#pragma once

#include <algorithm>

#include "paged.cuh"

// An answer row (coordinate lane + 32 k of the rotated sum in x[k], the sum of
// weights l): out = Pi^T x / l, zeros where nothing was seen.  scratch: d
// floats of this warp's shared memory (dense rotations only).
template <int D>
__device__ __forceinline__ void paged_store_row(float (&x)[D / 32], float l, const TqBooks &bk, float *scratch,
                                                void *out, int out_dtype, int64_t row, int lane) {
  constexpr int NPL = D / 32;
  float f = l == 0.f ? 0.f : 1.0f / l;
  if (bk.pi != nullptr) {
    __syncwarp();
    tq_warp_dense<NPL>(x, bk.pi, scratch, lane);
  } else {
    tq_warp_wht<NPL>(x, lane);
    tq_apply_signs<NPL>(x, bk.dneg, lane);
    f *= 1.0f / sqrtf(static_cast<float>(D));
  }
#pragma unroll
  for (int k = 0; k < NPL; ++k) {
    const int64_t o = row * D + lane + 32 * k;
    if (out_dtype == TQ_BF16)
      static_cast<__nv_bfloat16 *>(out)[o] = __float2bfloat16_rn(x[k] * f);
    else
      static_cast<float *>(out)[o] = x[k] * f;
  }
}

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
// Few query rows a KV head (paged_decode.cu).
size_t paged_decode_workspace_bytes(const tq_codec *c, int N, int num_seqs, int max_new, int max_len, int Hq,
                                    int Hkv);
int launch_paged_decode(const tq_codec *c, const PagedView &p, const void *q, int dtype, int64_t st, int64_t sh,
                        int Hq, const tq_cache *cache, float scale, const float *rc, const float *rs, void *ws,
                        void *out, int out_dtype, cudaStream_t stream);
// Many query rows a KV head (paged_prefill.cu); at most 128 query heads a KV head.
size_t paged_prefill_workspace_bytes(const tq_codec *c, int N, int num_seqs, int max_len, int Hq, int Hkv);
int launch_paged_prefill(const tq_codec *c, const PagedView &p, const void *q, int dtype, int64_t st, int64_t sh,
                         int Hq, const tq_cache *cache, float scale, const float *rc, const float *rs, void *ws,
                         void *out, int out_dtype, cudaStream_t stream);
