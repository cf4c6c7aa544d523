// Append of new tokens' keys and values to a paged compressed cache.
//
// Same row computation as quantize.cu ("TurboESM ...", section 2.A: RoPE, then
// the rotation; "FibQuant ...", section 2.3; "Google presenta TurboQuant ...",
// "Eliminacion del sesgo"), with the codes of exact arithmetic: a coordinate's
// code does not depend on the batch a token arrives in.
#include "paged.h"

namespace {

struct PagedQuantArgs {
  PagedView p;
  const void *k, *v;
  int dtype;
  int Hkv;
  int64_t st, sh;
  const float *rc, *rs;
  uint8_t *kcode;
  uint16_t *kscale;
  uint32_t *vcode;
  uint16_t *vnorm;
  uint32_t *status;
  const uint16_t *S;
  TqBooks books;
};

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(TQ_FULL, v, o);
  return v;
}

// nu and u = Pi x / nu of a warp-held row (coordinate lane + 32 k), in 64
// bits; a row with a non-finite element or an fp16-overflowing norm becomes
// the zero row.  scratch: d doubles of this warp.
template <int NPL>
__device__ __forceinline__ double unit_f64(double (&x)[NPL], const TqBooks &bk, double *scratch,
                                           int lane, bool &bad) {
  constexpr int D = NPL * 32;
  bool finite = true;
  double ss = 0.0;
#pragma unroll
  for (int k = 0; k < NPL; ++k) {
    finite &= isfinite(x[k]);
    ss += x[k] * x[k];
  }
  bad = __any_sync(TQ_FULL, !finite);
  double nu = sqrt(warp_sum_f64(ss));
  if (!bad && isinf(__half2float(__double2half(nu)))) bad = true;
  if (bad) nu = 0.0;
  const double inv = nu > 0.0 ? 1.0 / nu : 0.0;
#pragma unroll
  for (int k = 0; k < NPL; ++k) x[k] = inv > 0.0 ? x[k] : 0.0;
  if (bk.pi != nullptr) {
#pragma unroll
    for (int k = 0; k < NPL; ++k) scratch[lane + 32 * k] = x[k];
    __syncwarp();
    double acc[NPL];
#pragma unroll
    for (int k = 0; k < NPL; ++k) acc[k] = 0.0;
    for (int j = 0; j < D; ++j)
#pragma unroll
      for (int k = 0; k < NPL; ++k)
        acc[k] = fma(static_cast<double>(bk.pi_t[j * D + lane + 32 * k]), scratch[j], acc[k]);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < NPL; ++k) x[k] = acc[k] * inv;
    return nu;
  }
#pragma unroll
  for (int k = 0; k < NPL; ++k) x[k] = (bk.dneg[k] >> lane) & 1u ? -x[k] : x[k];
#pragma unroll
  for (int s = 1; s < 32; s <<= 1)
#pragma unroll
    for (int k = 0; k < NPL; ++k) {
      const double o = __shfl_xor_sync(TQ_FULL, x[k], s);
      x[k] = lane & s ? o - x[k] : x[k] + o;
    }
#pragma unroll
  for (int s = 1; s < NPL; s <<= 1)
#pragma unroll
    for (int k = 0; k < NPL; ++k)
      if (!(k & s)) {
        const double a = x[k], b = x[k + s];
        x[k] = a + b;
        x[k + s] = a - b;
      }
  const double f = inv / sqrt(static_cast<double>(D));
#pragma unroll
  for (int k = 0; k < NPL; ++k) x[k] *= f;
  return nu;
}

__device__ __forceinline__ int code_f64(double u, const float *t) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < TQ_MAX_LEVELS - 1; ++i) n += u >= static_cast<double>(t[i]);
  return n;
}

// One warp per (new token, KV head).
template <int D>
__global__ void __launch_bounds__(128) paged_quantize_kernel(PagedQuantArgs a) {
  constexpr int NPL = D / 32;
  __shared__ double buf[4][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t it = static_cast<int64_t>(blockIdx.x) * 4 + warp;
  const int tok = static_cast<int>(it / a.Hkv), h = static_cast<int>(it % a.Hkv);
  if (tok >= a.p.N) return;
  const int s = paged_find_seq(a.p, tok, 1, 0);
  const SeqSpan sp = paged_span(a.p, s);
  const int i = tok - sp.row0, pos = sp.len - sp.n + i;
  if (i < 0 || i >= sp.n || pos < 0) return;
  const int page = paged_page(a.p, s, pos);
  if (page < 0) {
    if (lane == 0 && a.status) atomicAdd(a.status, 2u);
    return;
  }
  const int P = 1 << a.p.page_shift;
  const int64_t row = (static_cast<int64_t>(page) * a.Hkv + h) * P + (pos & (P - 1));
  const int mbk = a.books.mse_bits_k, planes = mbk + a.books.qjl;
  const int64_t off = tok * a.st + h * a.sh;
  double x[NPL];
  bool bad;
#pragma unroll
  for (int k = 0; k < NPL; ++k) x[k] = tq_load_elem(a.k, off + lane + 32 * k, a.dtype);
  if (a.rc != nullptr) {
#pragma unroll
    for (int k = 0; k < NPL / 2; ++k) {
      const double c = a.rc[static_cast<int64_t>(pos) * (D / 2) + lane + 32 * k];
      const double sn = a.rs[static_cast<int64_t>(pos) * (D / 2) + lane + 32 * k];
      const double u = x[k], w = x[k + NPL / 2];
      x[k] = u * c - w * sn;
      x[k + NPL / 2] = w * c + u * sn;
    }
  }
  const double nu = unit_f64<NPL>(x, a.books, buf[warp], lane, bad);
  uint32_t *krow = reinterpret_cast<uint32_t *>(a.kcode + row * planes * (D / 8));
  double r2 = 0.0;
#pragma unroll
  for (int k = 0; k < NPL; ++k) {
    const int idx = code_f64(x[k], a.books.tk);
    for (int p = 0; p < mbk; ++p) {
      const uint32_t w = __ballot_sync(TQ_FULL, (idx >> p) & 1);
      if (lane == 0) krow[p * NPL + k] = w;
    }
    const double r = x[k] - static_cast<double>(a.books.ck[idx]);
    buf[warp][lane + 32 * k] = r;
    r2 += r * r;
  }
  double rho = 0.0;
  if (a.books.qjl) {
    rho = sqrt(warp_sum_f64(r2));
    __syncwarp();
#pragma unroll
    for (int k = 0; k < NPL; ++k) {
      double z = 0.0;
      for (int j = 0; j < D; ++j)
        z = fma(static_cast<double>(tq_bf16_to_f32(a.S[(lane + 32 * k) * D + j])), buf[warp][j], z);
      const uint32_t w = __ballot_sync(TQ_FULL, z >= 0.0);
      if (lane == 0) krow[mbk * NPL + k] = w;
    }
    __syncwarp();
  }
  if (lane == 0) {
    reinterpret_cast<uint32_t *>(a.kscale)[row] =
        __half_as_ushort(__double2half(nu)) |
        (static_cast<uint32_t>(__half_as_ushort(__double2half(rho))) << 16);
    if (bad && a.status) atomicAdd(a.status, 1u);
  }
#pragma unroll
  for (int k = 0; k < NPL; ++k) x[k] = tq_load_elem(a.v, off + lane + 32 * k, a.dtype);
  const double nv = unit_f64<NPL>(x, a.books, buf[warp], lane, bad);
  uint32_t *vg = a.vcode + (row >> 5) * a.books.bits_v * D;
  const uint32_t bit = 1u << (pos & 31);
#pragma unroll
  for (int k = 0; k < NPL; ++k) {
    const int idx = code_f64(x[k], a.books.tv);
    for (int p = 0; p < a.books.bits_v; ++p) {
      uint32_t *w = vg + p * D + lane + 32 * k;
      if ((idx >> p) & 1)
        atomicOr(w, bit);
      else
        atomicAnd(w, ~bit);
    }
  }
  if (lane == 0) {
    a.vnorm[row] = __half_as_ushort(__double2half(nv));
    if (bad && a.status) atomicAdd(a.status, 1u);
  }
}

}  // namespace

int launch_paged_quantize(const tq_codec *c, const PagedView &p, const void *k, const void *v, int dtype,
                          int64_t st, int64_t sh, const float *rc, const float *rs, const tq_cache *cache,
                          uint32_t *status, cudaStream_t stream) {
  PagedQuantArgs a;
  a.p = p;
  a.k = k;
  a.v = v;
  a.dtype = dtype;
  a.Hkv = cache->Hkv;
  a.st = st;
  a.sh = sh;
  a.rc = rc;
  a.rs = rs;
  a.kcode = cache->kcode;
  a.kscale = cache->kscale;
  a.vcode = cache->vcode;
  a.vnorm = cache->vnorm;
  a.status = status;
  a.S = c->S_dev;
  a.books = c->books;
  const int64_t rows = static_cast<int64_t>(p.N) * cache->Hkv;
  const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
  if (c->d == 64)
    paged_quantize_kernel<64><<<grid, 128, 0, stream>>>(a);
  else
    paged_quantize_kernel<128><<<grid, 128, 0, stream>>>(a);
  tq_count_launch(1);
  return tq_check_launch("paged_quantize_kernel");
}
