// Rows of a paged compressed cache read back as vectors ("FibQuant ...",
// section 2.3, decoder; keys add the QJL term):
//   keys   nu Pi^T (c_k[idx] + sqrt(pi/2)/d rho S^T (2 sigma - 1))
//   values nu Pi^T c_v[idx]
#include "paged.h"

namespace {

struct PagedDequantArgs {
  PagedView p;
  int Hkv;
  const uint8_t *kcode;
  const uint16_t *kscale;
  const uint32_t *vcode;
  const uint16_t *vnorm;
  void *k_out, *v_out;     // [N][Hkv][d], either may be null
  int out_dtype;
  float qjl_coef;
  const uint16_t *S;
  TqBooks books;
};

// One warp per (token, KV head).
template <int D>
__global__ void __launch_bounds__(256) paged_dequant_kernel(PagedDequantArgs a) {
  constexpr int NPL = D / 32;
  __shared__ float dsc[8][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t it = static_cast<int64_t>(blockIdx.x) * 8 + warp;
  const int tok = static_cast<int>(it / a.Hkv), h = static_cast<int>(it % a.Hkv);
  if (tok >= a.p.N) return;
  const int s = paged_find_seq(a.p, tok, 1, 0);
  const SeqSpan sp = paged_span(a.p, s);
  const int i = tok - sp.row0, pos = sp.len - sp.n + i;
  if (i < 0 || i >= sp.n) return;
  const int page = pos >= 0 ? paged_page(a.p, s, pos) : -1;
  const int P = 1 << a.p.page_shift;
  const int64_t row = (static_cast<int64_t>(page) * a.Hkv + h) * P + (pos & (P - 1));
  const int mbk = a.books.mse_bits_k, planes = mbk + a.books.qjl;
  for (int which = 0; which < 2; ++which) {
    void *out = which ? a.v_out : a.k_out;
    if (out == nullptr) continue;
    float y[NPL], nu = 0.f;
#pragma unroll
    for (int k = 0; k < NPL; ++k) y[k] = 0.f;
    if (page >= 0 && which == 0) {
      const uint32_t *krow = reinterpret_cast<const uint32_t *>(a.kcode + row * planes * (D / 8));
      const uint32_t sc = reinterpret_cast<const uint32_t *>(a.kscale)[row];
      nu = tq_half_to_f32(static_cast<uint16_t>(sc & 0xffffu));
      if (a.books.qjl) {
        for (int j = 0; j < D; ++j) {
          const bool pos_sign = (krow[mbk * NPL + (j >> 5)] >> (j & 31)) & 1;
#pragma unroll
          for (int k = 0; k < NPL; ++k) {
            const float sv = tq_bf16_to_f32(a.S[j * D + lane + 32 * k]);
            y[k] += pos_sign ? sv : -sv;
          }
        }
      }
      const float f = a.qjl_coef * tq_half_to_f32(static_cast<uint16_t>(sc >> 16));
#pragma unroll
      for (int k = 0; k < NPL; ++k) {
        int idx = 0;
        for (int p = 0; p < mbk; ++p) idx |= ((krow[p * NPL + k] >> lane) & 1) << p;
        y[k] = fmaf(f, y[k], a.books.ck[idx]);
      }
    } else if (page >= 0) {
      const uint32_t *vg = a.vcode + (row >> 5) * a.books.bits_v * D;
      nu = tq_half_to_f32(a.vnorm[row]);
#pragma unroll
      for (int k = 0; k < NPL; ++k) {
        int idx = 0;
        for (int p = 0; p < a.books.bits_v; ++p) idx |= ((vg[p * D + lane + 32 * k] >> (pos & 31)) & 1) << p;
        y[k] = a.books.cv[idx];
      }
    }
    if (a.books.pi != nullptr) {
      tq_warp_dense<NPL>(y, a.books.pi, dsc[warp], lane);
    } else {
      tq_warp_wht<NPL>(y, lane);
      tq_apply_signs<NPL>(y, a.books.dneg, lane);
      nu *= 1.0f / sqrtf(static_cast<float>(D));
    }
#pragma unroll
    for (int k = 0; k < NPL; ++k) {
      const int64_t o = it * D + lane + 32 * k;
      if (a.out_dtype == TQ_BF16)
        static_cast<__nv_bfloat16 *>(out)[o] = __float2bfloat16_rn(y[k] * nu);
      else
        static_cast<float *>(out)[o] = y[k] * nu;
    }
  }
}

}  // namespace

int launch_paged_dequant(const tq_codec *c, const PagedView &p, const tq_cache *cache, void *k_out,
                         void *v_out, int out_dtype, cudaStream_t stream) {
  PagedDequantArgs a;
  a.p = p;
  a.Hkv = cache->Hkv;
  a.kcode = cache->kcode;
  a.kscale = cache->kscale;
  a.vcode = cache->vcode;
  a.vnorm = cache->vnorm;
  a.k_out = k_out;
  a.v_out = v_out;
  a.out_dtype = out_dtype;
  a.qjl_coef = c->qjl_k ? sqrtf(static_cast<float>(M_PI) / 2.0f) / c->d : 0.f;
  a.S = c->S_dev;
  a.books = c->books;
  const int64_t rows = static_cast<int64_t>(p.N) * cache->Hkv;
  const unsigned grid = static_cast<unsigned>((rows + 7) / 8);
  if (c->d == 64)
    paged_dequant_kernel<64><<<grid, 256, 0, stream>>>(a);
  else
    paged_dequant_kernel<128><<<grid, 256, 0, stream>>>(a);
  tq_count_launch(1);
  return tq_check_launch("paged_dequant_kernel");
}
