// Attention of new tokens over a paged compressed cache: query i of a
// sequence (position pos_i) attends to cached tokens j <= pos_i,
//   l_ij = scale nu_j (<q'_i, c_k[idx_j]> + sqrt(pi/2)/d rho_j <S q'_i, 2 sigma_j - 1>),
//   q'_i = Pi RoPE(q_i, pos_i),  out_i = Pi^T sum_j softmax(l_i)_j nu^v_j c_v[idx^v_j]
// ("TurboESM ...", sections 2.A and 2.E; "Google presenta TurboQuant ...",
// "Eliminacion del sesgo").
#include <math_constants.h>

#include "paged.h"

namespace {

struct PagedAttnArgs {
  PagedView p;
  const void *q;           // [N][Hq][d] with strides st, sh
  int dtype;
  int64_t st, sh;
  int Hq, Hkv;
  const uint8_t *kcode;
  const uint16_t *kscale;
  const uint32_t *vcode;
  const uint16_t *vnorm;
  float scale, qjl_coef;
  const float *rc, *rs;
  void *out;               // [N][Hq][d]
  int out_dtype;
  const uint16_t *ST;
  TqBooks books;
};

// One block per (new token, query head): 128 keys at a time, a thread per key
// for the logits, a thread per coordinate for the values.
template <int D>
__global__ void __launch_bounds__(128) paged_attn_kernel(PagedAttnArgs a) {
  constexpr int NPL = D / 32;
  __shared__ float q1[D], q2[D], pw[128], red[4], cks[16], cvs[16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tok = blockIdx.x, h = blockIdx.y, kvh = h / (a.Hq / a.Hkv);
  if (tid < 16) {
    cks[tid] = a.books.ck[tid];
    cvs[tid] = a.books.cv[tid];
  }
  const int s = paged_find_seq(a.p, tok, 1, 0);
  const SeqSpan sp = paged_span(a.p, s);
  const int i = tok - sp.row0, pos = sp.len - sp.n + i;
  if (i < 0 || i >= sp.n) return;
  if (warp == 0) {
    float x[NPL];
#pragma unroll
    for (int k = 0; k < NPL; ++k)
      x[k] = tq_load_elem(a.q, tok * a.st + h * a.sh + lane + 32 * k, a.dtype);
    if (a.rc != nullptr && pos >= 0) {
#pragma unroll
      for (int k = 0; k < NPL / 2; ++k) {
        const float c = a.rc[static_cast<int64_t>(pos) * (D / 2) + lane + 32 * k];
        const float sn = a.rs[static_cast<int64_t>(pos) * (D / 2) + lane + 32 * k];
        const float u = x[k], v = x[k + NPL / 2];
        x[k] = u * c - v * sn;
        x[k + NPL / 2] = v * c + u * sn;
      }
    }
    if (a.books.pi != nullptr) {
      tq_warp_dense<NPL>(x, a.books.pi_t, q1, lane);
    } else {
      tq_apply_signs<NPL>(x, a.books.dneg, lane);
      tq_warp_wht<NPL>(x, lane);
#pragma unroll
      for (int k = 0; k < NPL; ++k) x[k] *= 1.0f / sqrtf(static_cast<float>(D));
    }
#pragma unroll
    for (int k = 0; k < NPL; ++k) q1[lane + 32 * k] = x[k];
  }
  __syncthreads();
  if (tid < D) {
    float z = 0.f;
    if (a.books.qjl)
      for (int j = 0; j < D; ++j) z = fmaf(tq_bf16_to_f32(a.ST[j * D + tid]), q1[j], z);
    q2[tid] = z;
  }
  __syncthreads();
  const int mbk = a.books.mse_bits_k, planes = mbk + a.books.qjl, nbv = a.books.bits_v;
  const int P = 1 << a.p.page_shift;
  float m = -CUDART_INF_F, l = 0.f, acc = 0.f;
  for (int j0 = 0; j0 <= pos; j0 += 128) {
    const int j = j0 + tid;
    float lg = -CUDART_INF_F;
    const int page = j <= pos ? paged_page(a.p, s, j) : -1;
    if (page >= 0) {
      const int64_t row = (static_cast<int64_t>(page) * a.Hkv + kvh) * P + (j & (P - 1));
      const uint32_t *kr = reinterpret_cast<const uint32_t *>(a.kcode + row * planes * (D / 8));
      const uint32_t sc = reinterpret_cast<const uint32_t *>(a.kscale)[row];
      float z1 = 0.f, z2 = 0.f;
      for (int k = 0; k < NPL; ++k) {
        uint32_t w[5];
        for (int p = 0; p < 5; ++p) w[p] = p < planes ? kr[p * NPL + k] : 0u;
        for (int e = 0; e < 32; ++e) {
          int idx = 0;
          uint32_t sg = 0u;
          for (int p = 0; p < 5; ++p) {
            if (p < mbk) idx |= ((w[p] >> e) & 1) << p;
            else if (p == mbk) sg = (w[p] >> e) & 1;
          }
          z1 = fmaf(q1[32 * k + e], cks[idx], z1);
          z2 += sg ? q2[32 * k + e] : -q2[32 * k + e];
        }
      }
      lg = a.scale * tq_half_to_f32(sc & 0xffff) * (z1 + a.qjl_coef * tq_half_to_f32(sc >> 16) * z2);
    }
    const float wm = tq_warp_max(lg);
    if (lane == 0) red[warp] = wm;
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float base = mn == -CUDART_INF_F ? 0.f : mn;
    const float corr = __expf(m - base);
    pw[tid] = __expf(lg - base);
    __syncthreads();
    l *= corr;
    acc *= corr;
    m = mn;
    for (int e = 0; e < 128; ++e) l += pw[e];
    if (tid < D) {
      for (int g = 0; g < 128 && j0 + g <= pos; g += 32) {
        const int pg = paged_page(a.p, s, j0 + g);
        if (pg < 0) continue;
        const int64_t row = (static_cast<int64_t>(pg) * a.Hkv + kvh) * P + ((j0 + g) & (P - 1));
        const uint32_t *vg = a.vcode + (row >> 5) * nbv * D;
        uint32_t w[4];
        for (int p = 0; p < 4; ++p) w[p] = p < nbv ? vg[p * D + tid] : 0u;
        for (int e = 0; e < 32; ++e) {
          int idx = 0;
          for (int p = 0; p < 4; ++p) idx |= ((w[p] >> e) & 1) << p;
          if (pw[g + e] != 0.f) acc = fmaf(pw[g + e] * tq_half_to_f32(a.vnorm[row + e]), cvs[idx], acc);
        }
      }
    }
    __syncthreads();
  }
  // out = Pi^T acc / l; a token that sees nothing gets zeros
  if (tid < D) q1[tid] = l > 0.f ? acc / l : 0.f;
  __syncthreads();
  if (warp == 0) {
    float x[NPL];
#pragma unroll
    for (int k = 0; k < NPL; ++k) x[k] = q1[lane + 32 * k];
    float f = 1.f;
    if (a.books.pi != nullptr) {
      tq_warp_dense<NPL>(x, a.books.pi, q2, lane);
    } else {
      tq_warp_wht<NPL>(x, lane);
      tq_apply_signs<NPL>(x, a.books.dneg, lane);
      f = 1.0f / sqrtf(static_cast<float>(D));
    }
#pragma unroll
    for (int k = 0; k < NPL; ++k) {
      const int64_t o = (static_cast<int64_t>(tok) * a.Hq + h) * D + lane + 32 * k;
      if (a.out_dtype == TQ_BF16)
        static_cast<__nv_bfloat16 *>(a.out)[o] = __float2bfloat16_rn(x[k] * f);
      else
        static_cast<float *>(a.out)[o] = x[k] * f;
    }
  }
}

bool few_rows(int max_new, int Hq, int Hkv) { return static_cast<int64_t>(max_new) * (Hq / Hkv) <= 64; }

}  // namespace

size_t paged_attn_workspace_bytes(const tq_codec *c, int N, int num_seqs, int max_new, int max_len, int Hq,
                                  int Hkv) {
  if (N == 0 || num_seqs == 0 || max_new == 0) return 16;
  return few_rows(max_new, Hq, Hkv)
             ? paged_decode_workspace_bytes(c, N, num_seqs, max_new, max_len, Hq, Hkv)
             : 16;
}

int launch_paged_attention(const tq_codec *c, const PagedView &p, const void *q, int dtype, int64_t st,
                           int64_t sh, int Hq, const tq_cache *cache, float scale, const float *rc,
                           const float *rs, void *ws, void *out, int out_dtype, cudaStream_t stream) {
  if (few_rows(p.max_new, Hq, cache->Hkv))
    return launch_paged_decode(c, p, q, dtype, st, sh, Hq, cache, scale, rc, rs, ws, out, out_dtype, stream);
  PagedAttnArgs a;
  a.p = p;
  a.q = q;
  a.dtype = dtype;
  a.st = st;
  a.sh = sh;
  a.Hq = Hq;
  a.Hkv = cache->Hkv;
  a.kcode = cache->kcode;
  a.kscale = cache->kscale;
  a.vcode = cache->vcode;
  a.vnorm = cache->vnorm;
  a.scale = scale;
  a.qjl_coef = c->qjl_k ? sqrtf(static_cast<float>(M_PI) / 2.0f) / c->d : 0.f;
  a.rc = rc;
  a.rs = rs;
  a.out = out;
  a.out_dtype = out_dtype;
  a.ST = c->ST_dev;
  a.books = c->books;
  const dim3 grid(p.N, Hq);
  if (c->d == 64)
    paged_attn_kernel<64><<<grid, 128, 0, stream>>>(a);
  else
    paged_attn_kernel<128><<<grid, 128, 0, stream>>>(a);
  tq_count_launch(1);
  return tq_check_launch("paged_attn_kernel");
}
