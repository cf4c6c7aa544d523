// RMS norm of every query and key head, then the rotate-half position
// rotation, in one pass:
//   y = x w / sqrt(mean(x^2) + eps),
//   out_i = y_i cos - y_{i+d/2} sin,  out_{i+d/2} = y_{i+d/2} cos + y_i sin.
// ("TurboESM ...", section 2.A: the rotation comes before Pi; the norm before
// the rotation.)
#include "paged.h"

namespace {

struct NormRopeArgs {
  const void *x[2];        // queries, keys
  void *y[2];
  const void *w[2];        // [d] or null (ones)
  int64_t st[2], sh[2];    // input strides (elements) of a token, a head
  int64_t yt[2], yh[2];
  int H[2];
  int N;
  int dtype, w_dtype;
  float eps;
  const int32_t *pos;
  const float *rc, *rs;
  int rope_len;
};

// One warp per (token, head); coordinate lane + 32 k in register k.
template <int D>
__global__ void __launch_bounds__(256) norm_rope_kernel(NormRopeArgs a) {
  constexpr int NPL = D / 32, HALF = NPL / 2;
  const int lane = threadIdx.x & 31;
  const int heads = a.H[0] + a.H[1];
  const int64_t it = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (it >= static_cast<int64_t>(a.N) * heads) return;
  const int64_t t = it / heads;
  int h = static_cast<int>(it % heads);
  const int which = h >= a.H[0];
  if (which) h -= a.H[0];
  float x[NPL], ss = 0.f;
#pragma unroll
  for (int k = 0; k < NPL; ++k) {
    x[k] = tq_load_elem(a.x[which], t * a.st[which] + h * a.sh[which] + lane + 32 * k, a.dtype);
    ss += x[k] * x[k];
  }
  const float f = rsqrtf(tq_warp_sum(ss) * (1.0f / D) + a.eps);
#pragma unroll
  for (int k = 0; k < NPL; ++k) {
    x[k] *= f;
    if (a.w[which] != nullptr) x[k] *= tq_load_elem(a.w[which], lane + 32 * k, a.w_dtype);
  }
  if (a.rc != nullptr) {
    const int64_t p = min(max(a.pos[t], 0), a.rope_len - 1);
#pragma unroll
    for (int k = 0; k < HALF; ++k) {
      const float c = a.rc[p * (D / 2) + lane + 32 * k], s = a.rs[p * (D / 2) + lane + 32 * k];
      const float u = x[k], v = x[k + HALF];
      x[k] = u * c - v * s;
      x[k + HALF] = v * c + u * s;
    }
  }
#pragma unroll
  for (int k = 0; k < NPL; ++k) {
    const int64_t o = t * a.yt[which] + h * a.yh[which] + lane + 32 * k;
    if (a.dtype == TQ_BF16)
      static_cast<__nv_bfloat16 *>(a.y[which])[o] = __float2bfloat16_rn(x[k]);
    else
      static_cast<float *>(a.y[which])[o] = x[k];
  }
}

}  // namespace

int launch_norm_rope(const tq_heads *q, const tq_heads *k, int dtype, int w_dtype, int d, int N,
                     float eps, const int32_t *pos, const float *rc, const float *rs, int rope_len,
                     cudaStream_t stream) {
  NormRopeArgs a = {};
  const tq_heads *hs[2] = {q, k};
  for (int i = 0; i < 2; ++i) {
    if (hs[i] == nullptr) continue;
    a.x[i] = hs[i]->x;
    a.y[i] = hs[i]->y;
    a.w[i] = hs[i]->weight;
    a.st[i] = hs[i]->x_stride_t;
    a.sh[i] = hs[i]->x_stride_h;
    a.yt[i] = hs[i]->y_stride_t;
    a.yh[i] = hs[i]->y_stride_h;
    a.H[i] = hs[i]->heads;
  }
  a.N = N;
  a.dtype = dtype;
  a.w_dtype = w_dtype;
  a.eps = eps;
  a.pos = pos;
  a.rc = rc;
  a.rs = rs;
  a.rope_len = rope_len;
  const int64_t rows = static_cast<int64_t>(N) * (a.H[0] + a.H[1]);
  const unsigned grid = static_cast<unsigned>((rows + 7) / 8);
  if (d == 64)
    norm_rope_kernel<64><<<grid, 256, 0, stream>>>(a);
  else
    norm_rope_kernel<128><<<grid, 256, 0, stream>>>(a);
  tq_count_launch(1);
  return tq_check_launch("norm_rope_kernel");
}
