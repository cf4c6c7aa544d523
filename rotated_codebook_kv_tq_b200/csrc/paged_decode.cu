// Attention of a few new tokens over a paged compressed cache: the keys of a
// (sequence, KV head) are split over blocks, expanded from their code planes
// straight into tensor-core operand registers, and the blocks' partial sums
// joined by a second kernel.
//
//   l_ij = scale nu_j (<q'_i, c[idx_j]> + coef rho_j (2 <q''_i, sigma_j> - sum q''_i)),
//   q' = Pi RoPE(q), q'' = S q', coef = sqrt(pi/2)/d, sigma_j the 0/1 sketch bits;
//   w_ij = 2^(l_ij log2 e + log2 nu^v_j - M),   out = Pi^T (sum_j w_ij c_v[idx^v_j]) / sum_j w_ij / nu^v_j.
// The value norm rides in the weight, so weights are at most 1 and value
// operands are table entries: both sides keep fp16's 2^-11 at any norm.  Norms,
// logits, maxima and sums are fp32; query, centroid and weight are rounded to
// fp16 once each (2^-11 of an element, against 2^-8 of a bf16 answer).
#include <math_constants.h>

#include <cstdlib>

#include "paged_expand.cuh"
#include "tq_sm100.cuh"

namespace {

constexpr int DW = 8;          // warps of a block
constexpr float F_SIGN = 1024.f;   // 2^10: keeps the scaled q'' of a bit operand inside fp16

struct DecArgs {
  PagedView p;
  const void *q;
  int dtype;
  int64_t st, sh;
  int Hq, Hkv, G;
  const uint8_t *kcode;
  const uint16_t *kscale;
  const uint32_t *vcode;
  const uint16_t *vnorm;
  float scale, qjl_coef;
  const float *rc, *rs;
  void *out;
  int out_dtype;
  const uint16_t *S;
  int qtiles;            // tiles of 8 NT query rows a (sequence, KV head)
  int chunk;             // 32-token groups of a block
  int splits;
  int stages;            // ring slots of a warp
  float *po;             // [N Hq][splits][D] partial sums
  float2 *pml;           // [N Hq][splits] (reference M, denominator)
  uint32_t wait_limit;
  uint32_t lutk[4], lutv[4];   // fp16 table bytes: low 0-3, low 4-7, high 0-3, high 4-7
  TqBooks books;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The fp16 value whose bit pattern is 1 << x (x <= 14): 2^(x - 24) below the
// exponent field, then 2^-14, 2^-13, 2^-11, 2^-7, 2.
__device__ __forceinline__ float bit_value(int x) { return __half2float(__ushort_as_half(1u << x)); }

// Coordinate of thread column t, element `half` (0 / 1 of a register pair) of
// k-step ks, operand register r (0: first, 1: second): the order in which
// nibbles() and the sketch-bit masks leave a plane word.
template <int D>
__device__ __forceinline__ int code_coord(int t, int ks, int r, int half) {
  if (D == 128) return 32 * t + 4 * (4 * (ks & 1) + 2 * r + half) + (ks >> 1);
  return 16 * t + 4 * (2 * r + half) + ks;
}
template <int D>
__device__ __forceinline__ int bit_coord(int t, int ks, int r, int half) {
  const int x = 2 * ks + r;
  return D == 128 ? 32 * t + x + 16 * half : 16 * t + x + 8 * half;
}

// Rows of a (sequence, KV head): row r is new token r / G, head r % G.  Tokens
// visible to the query tile that starts at row lo.
__device__ __forceinline__ int tile_visible(const SeqSpan &sp, int G, int lo, int rows) {
  const int last = min(lo + rows, sp.n * G) - 1;
  return max(0, min(sp.len, sp.len - sp.n + last / G + 1));
}

template <int D, bool K4, bool V4, int NT>
__global__ void __launch_bounds__(DW * 32, NT <= 2 ? 2 : 1) paged_decode_kernel(const __grid_constant__ DecArgs a) {
  constexpr int NPL = D / 32, KS = D / 16, R = 8 * NT, MT = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  uint2 *bc = reinterpret_cast<uint2 *>(smem);                 // [KS][NT][32] code operand
  uint2 *bs = bc + KS * NT * 32;                               // [KS][NT][32] sketch operand
  float4 *colc = reinterpret_cast<float4 *>(bs + KS * NT * 32);   // [R] column constants
  float *q1 = reinterpret_cast<float *>(colc + R);             // [R][D]
  float *q2 = q1 + R * D;                                      // [256 / D][R][D]
  uint64_t *bars = reinterpret_cast<uint64_t *>(q2 + 256 * R);   // [DW][8]
  float *sM = reinterpret_cast<float *>(bars + DW * 8);        // [DW][R], then [DW][R] sums
  uint8_t *ring = reinterpret_cast<uint8_t *>(sM + 2 * DW * R);
  float *osum = reinterpret_cast<float *>(ring);               // [DW][R][D + 4], once the ring is drained

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x, kvh = blockIdx.y / a.qtiles, qt = blockIdx.y % a.qtiles, s = blockIdx.z;
  sm100::pdl_wait();
  const SeqSpan sp = paged_span(a.p, s);
  const int lo = qt * R, nrows = min(R, sp.n * a.G - lo);
  if (nrows <= 0) return;
  const int vis = tile_visible(sp, a.G, lo, R);
  const int g_end = min((split + 1) * a.chunk, (vis + 31) >> 5);
  const int g0 = split * a.chunk + warp;
  if (split * a.chunk >= g_end && split > 0) return;

  const int mbk = a.books.mse_bits_k, planes = mbk + a.books.qjl, nbv = a.books.bits_v;
  const uint32_t kb = 32 * planes * (D / 8), vb = nbv * D * 4;
  const uint32_t stage_bytes = kb + vb + 192;
  uint8_t *mine = ring + static_cast<size_t>(warp) * a.stages * stage_bytes;
  uint64_t *bar = bars + warp * 8;
  if (lane == 0)
    for (int i = 0; i < a.stages; ++i) sm100::mbar_init(&bar[i], 1);
  if (tid == 0) asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncwarp();
  const int cnt = g_end > g0 ? (g_end - g0 + DW - 1) / DW : 0;   // this warp's groups
  const int P = 1 << a.p.page_shift;
  int pages = -1;          // lane i: page of group i of the current 32
  uint32_t valid = 0u, phase = 0u;
  auto issue = [&](int i) {
    if ((i & 31) == 0) {
      const int gi = g0 + (i + lane) * DW;
      pages = i + lane < cnt ? paged_page(a.p, s, gi * 32) : -1;
    }
    const int page = __shfl_sync(TQ_FULL, pages, i & 31), st = i % a.stages;
    valid = page >= 0 ? valid | (1u << st) : valid & ~(1u << st);
    if (page >= 0 && lane == 0) {
      const int64_t row = (static_cast<int64_t>(page) * a.Hkv + kvh) * P + (((g0 + i * DW) * 32) & (P - 1));
      uint8_t *dst = mine + st * stage_bytes;
      sm100::mbar_expect_tx(&bar[st], stage_bytes);
      sm100::bulk_g2s(dst, a.kcode + row * planes * (D / 8), kb, &bar[st]);
      sm100::bulk_g2s(dst + kb, a.vcode + (row >> 5) * nbv * D, vb, &bar[st]);
      sm100::bulk_g2s(dst + kb + vb, a.kscale + row * 2, 128, &bar[st]);
      sm100::bulk_g2s(dst + kb + vb + 128, a.vnorm + row, 64, &bar[st]);
    }
  };
  int issued = 0;
  for (; issued < a.stages && issued < cnt; ++issued) issue(issued);

  // ---- queries, while the first groups arrive: q' by warps, q'' = S q' by
  // threads (row tid % D of S, a 1/(256/D) part of its columns)
  constexpr int PARTS = 256 / D, PW = D / PARTS;
  uint4 srow[PW / 8];
  if (a.books.qjl) {
    const uint4 *src = reinterpret_cast<const uint4 *>(a.S + (tid % D) * D + (tid / D) * PW);
#pragma unroll
    for (int i = 0; i < PW / 8; ++i) srow[i] = src[i];
  }
  {
    // warp w: rows w, w + 8, ..
    float x[NT][NPL];
    int64_t off[NT];
    int at[NT];
#pragma unroll
    for (int z = 0; z < NT; ++z) {
      const int r = warp + DW * z, tok = (lo + r) / a.G;
      at[z] = sp.len - sp.n + tok;
      off[z] = r < nrows && at[z] >= 0
                   ? static_cast<int64_t>(sp.row0 + tok) * a.st + (kvh * a.G + (lo + r) % a.G) * a.sh : -1;
    }
    paged_load_rows<NT, NPL>(x, a.q, off, a.dtype, lane);
    paged_rope_rows<NT, NPL>(x, a.rc, a.rs, at, off, lane);
#pragma unroll
    for (int z = 0; z < NT; ++z) {
      const int r = warp + DW * z;
      if (a.books.pi != nullptr) {
        tq_warp_dense<NPL>(x[z], a.books.pi_t, q1 + r * D, lane);
      } else {
        tq_apply_signs<NPL>(x[z], a.books.dneg, lane);
        tq_warp_wht<NPL, true>(x[z], lane);
#pragma unroll
        for (int k = 0; k < NPL; ++k) x[z][k] *= 1.0f / sqrtf(static_cast<float>(D));
      }
#pragma unroll
      for (int k = 0; k < NPL; ++k) q1[r * D + lane + 32 * k] = x[z][k];
    }
  }
  __syncthreads();
  if (a.books.qjl) {
    float acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = 0.f;
#pragma unroll
    for (int i = 0; i < PW / 8; ++i) {
      const uint32_t w[4] = {srow[i].x, srow[i].y, srow[i].z, srow[i].w};
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 *qv = reinterpret_cast<const float4 *>(q1 + r * D + (tid / D) * PW + 8 * i);
        const float4 u = qv[0], v = qv[1];
        acc[r] = fmaf(__uint_as_float(w[0] << 16), u.x, acc[r]);
        acc[r] = fmaf(__uint_as_float(w[0] & 0xffff0000u), u.y, acc[r]);
        acc[r] = fmaf(__uint_as_float(w[1] << 16), u.z, acc[r]);
        acc[r] = fmaf(__uint_as_float(w[1] & 0xffff0000u), u.w, acc[r]);
        acc[r] = fmaf(__uint_as_float(w[2] << 16), v.x, acc[r]);
        acc[r] = fmaf(__uint_as_float(w[2] & 0xffff0000u), v.y, acc[r]);
        acc[r] = fmaf(__uint_as_float(w[3] << 16), v.z, acc[r]);
        acc[r] = fmaf(__uint_as_float(w[3] & 0xffff0000u), v.w, acc[r]);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) q2[((tid / D) * R + r) * D + tid % D] = acc[r];
  }
  __syncthreads();
  // column constants and power-of-two scales (fp16 operands in [-1, 1])
  for (int r = warp; r < R; r += DW) {
    float m1 = 0.f, m2 = 0.f, sum2 = 0.f, z[NPL];
#pragma unroll
    for (int k = 0; k < NPL; ++k) {
      z[k] = 0.f;
      if (a.books.qjl)
#pragma unroll
        for (int p = 0; p < PARTS; ++p) z[k] += q2[(p * R + r) * D + lane + 32 * k];
      m1 = fmaxf(m1, fabsf(q1[r * D + lane + 32 * k]));
      m2 = fmaxf(m2, fabsf(z[k]));
      sum2 += z[k];
    }
    m1 = tq_warp_max(m1);
    m2 = tq_warp_max(m2);
    sum2 = tq_warp_sum(sum2);
    // exponents kept inside fp32 for any finite query
    const int e1 = m1 > 0.f ? max(-120, ilogbf(m1) + 1) : 0, e2 = m2 > 0.f ? max(-100, ilogbf(m2) + 1) : 0;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < NPL; ++k) {
      q1[r * D + lane + 32 * k] = ldexpf(q1[r * D + lane + 32 * k], -e1);
      q2[r * D + lane + 32 * k] = ldexpf(z[k], -e2);
    }
    if (lane == 0) {
      const float sl = a.scale * 1.4426950408889634f;
      const int pos = sp.len - sp.n + (lo + r) / a.G;
      colc[r] = make_float4(sl * ldexpf(1.f, e1), sl * 2.f * a.qjl_coef * ldexpf(F_SIGN, e2),
                            sl * a.qjl_coef * sum2, __int_as_float(r < nrows ? pos : -1));
    }
  }
  __syncthreads();
  for (int e = tid; e < KS * NT * 32; e += DW * 32) {
    const int l = e & 31, nt = (e >> 5) % NT, ks = (e >> 5) / NT, n = nt * 8 + (l >> 2), tt = l & 3;
    uint32_t wc[2], wsn[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      uint32_t c[2], b[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        c[h] = __half_as_ushort(__float2half_rn(q1[n * D + code_coord<D>(tt, ks, r, h)]));
        const int x = 2 * ks + r;   // bit 15 is shifted down to bit 0
        b[h] = __half_as_ushort(__float2half_rn(q2[n * D + bit_coord<D>(tt, ks, r, h)] *
                                                (1.0f / (F_SIGN * bit_value(x == 15 ? 0 : x)))));
      }
      wc[r] = c[0] | (c[1] << 16);
      wsn[r] = b[0] | (b[1] << 16);
    }
    bc[e] = make_uint2(wc[0], wc[1]);
    bs[e] = make_uint2(wsn[0], wsn[1]);
  }
  __syncthreads();
  sm100::pdl_trigger();

  // ---- groups of 32 tokens.  Row `g` of block b (0..3) of the logits is token
  // 8 b + 4 (g & 1) + g / 2: the order in which the value operand holds tokens.
  float acc_o[MT][NT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc_o[i][n][e] = 0.f;
  float M[NT][2], den[NT][2];
  int limit_min = 0x7fffffff;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      M[n][e] = -CUDART_INF_F;
      den[n][e] = 0.f;
    }
  for (int r = 0; r < R; ++r) limit_min = min(limit_min, r < nrows ? __float_as_int(colc[r].w) : 0x7fffffff);
  const int tok0 = 4 * (g & 1) + (g >> 1);
  bool ok = true;
  for (int i = 0; i < cnt; ++i) {
    const int stg = i % a.stages;
    if ((valid >> stg) & 1u) {
      ok = sm100::mbar_wait(&bar[stg], (phase >> stg) & 1u, a.wait_limit);
      ok = __all_sync(TQ_FULL, ok);
      if (!ok) break;
      phase ^= 1u << stg;
      const uint8_t *base = mine + stg * stage_bytes;
      const int j0 = (g0 + i * DW) * 32;
      // ---- logits, 16 tokens (blocks 2 h and 2 h + 1) at a time
      uint32_t pf[4][NT];     // weights as value-side operand registers, by block
      float lg[2][NT][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float s1[NT][4], s2[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s1[n][e] = s2[n][e] = 0.f;
        uint32_t w[2][4], sg[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint32_t *kr = reinterpret_cast<const uint32_t *>(base) + (8 * (2 * h + b) + tok0) * planes * NPL +
                               (D == 128 ? t : t >> 1);
#pragma unroll
          for (int p = 0; p < 4; ++p) w[b][p] = p < mbk ? kr[p * NPL] : 0u;
          sg[b] = a.books.qjl ? kr[mbk * NPL] : 0u;
          if (D == 64) {
#pragma unroll
            for (int p = 0; p < 4; ++p) w[b][p] >>= 16 * (t & 1);
            sg[b] = prmt(sg[b], 0u, t & 1 ? 0x4342 : 0x4140);
          }
          if (K4) fold_sign(w[b]);
        }
#pragma unroll
        for (int sft = 0; sft < 4; ++sft) {
          uint32_t oa[4], ob[4];
          expand8<K4>(nibbles<K4>(w[0], sft), a.lutk, oa);
          expand8<K4>(nibbles<K4>(w[1], sft), a.lutk, ob);
#pragma unroll
          for (int hf = 0; hf < (D == 128 ? 2 : 1); ++hf) {
            const int ks = D == 128 ? 2 * sft + hf : sft;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint2 b = bc[(ks * NT + n) * 32 + lane];
              mma16816(s1[n], oa[2 * hf], ob[2 * hf], oa[2 * hf + 1], ob[2 * hf + 1], b.x, b.y);
            }
          }
        }
        if (a.books.qjl) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            uint32_t ar[2][2];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const int x = 2 * ks + r;
                ar[b][r] = x == 15 ? (sg[b] >> 15) & 0x00010001u : sg[b] & (0x00010001u << x);
              }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint2 b = bs[(ks * NT + n) * 32 + lane];
              mma16816(s2[n], ar[0][0], ar[1][0], ar[0][1], ar[1][1], b.x, b.y);
            }
          }
        }
        // ---- logits in units of log2, value norm added
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int tk = 8 * (2 * h + b) + tok0;
          const uint32_t sc = reinterpret_cast<const uint32_t *>(base + kb + vb)[tk];
          const float nu = tq_half_to_f32(static_cast<uint16_t>(sc & 0xffffu));
          const float rho = tq_half_to_f32(static_cast<uint16_t>(sc >> 16));
          const float nv = fmaxf(tq_half_to_f32(reinterpret_cast<const uint16_t *>(base + kb + vb + 128)[tk]),
                                 5.9604645e-8f);
          const float lnv = __log2f(nv);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float4 cc = colc[n * 8 + 2 * t + e];
              float v = fmaf(nu, fmaf(cc.x, s1[n][2 * b + e], rho * fmaf(cc.y, s2[n][2 * b + e], -cc.z)), lnv);
              if (j0 + 31 > limit_min) v = j0 + tk <= __float_as_int(cc.w) ? v : -CUDART_INF_F;
              lg[h][n][2 * b + e] = v;
            }
        }
      }
      // ---- reference of the weights: moved only when a weight
      // would exceed 2^8 (fp16 weights are as exact there as at 1)
      bool grow = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) grow |= lg[h][n][e] > M[n][e & 1] + 8.f;
      if (__any_sync(TQ_FULL, grow)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(fmaxf(lg[0][n][e], lg[0][n][e + 2]), fmaxf(lg[1][n][e], lg[1][n][e + 2]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(TQ_FULL, mx, o));
            const float mn = fmaxf(M[n][e], mx);
            const float corr = mn == -CUDART_INF_F ? 1.f : ex2(M[n][e] - mn);
            M[n][e] = mn;
            den[n][e] *= corr;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              acc_o[m][n][e] *= corr;
              acc_o[m][n][e + 2] *= corr;
            }
          }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int tk = 8 * (2 * h + b) + tok0;
          const float nv = fmaxf(tq_half_to_f32(reinterpret_cast<const uint16_t *>(base + kb + vb + 128)[tk]),
                                 5.9604645e-8f);
          const float inv = __frcp_rn(nv);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float e[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float v = lg[h][n][2 * b + c];
              e[c] = v == -CUDART_INF_F ? 0.f : ex2(v - M[n][c]);
              if (v != -CUDART_INF_F) den[n][c] = fmaf(e[c], inv, den[n][c]);
            }
            const __half2 hv = __floats2half2_rn(e[0], e[1]);
            pf[2 * h + b][n] = transpose8x8(*reinterpret_cast<const uint32_t *>(&hv));
          }
        }
      // ---- values: four consecutive coordinates of a thread row at a time
#pragma unroll
      for (int c4 = 0; c4 < NPL; ++c4) {
        uint32_t vw[4][4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (p < nbv) v = *reinterpret_cast<const uint4 *>(base + kb + (p * D + 32 * c4 + 4 * g) * 4);
          vw[0][p] = v.x;
          vw[1][p] = v.y;
          vw[2][p] = v.z;
          vw[3][p] = v.w;
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          uint32_t oa[4], ob[4];
          if (V4) {
            fold_sign(vw[2 * m]);
            fold_sign(vw[2 * m + 1]);
          }
          expand8<V4>(nibbles<V4>(vw[2 * m], t), a.lutv, oa);
          expand8<V4>(nibbles<V4>(vw[2 * m + 1], t), a.lutv, ob);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma16816(acc_o[2 * c4 + m][n], oa[0], ob[0], oa[1], ob[1], pf[0][n], pf[1][n]);
            mma16816(acc_o[2 * c4 + m][n], oa[2], ob[2], oa[3], ob[3], pf[2][n], pf[3][n]);
          }
        }
      }
      __syncwarp();
    }
    if (issued < cnt) {
      issue(issued);
      ++issued;
    }
  }
  if (!ok) {
    // a copy never arrived: let the others land, and answer NaN
    for (int i = 0; i < a.stages; ++i)
      if ((valid >> i) & 1u) sm100::mbar_wait(&bar[i], (phase >> i) & 1u, 1u << 20);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        M[n][e] = 0.f;
        den[n][e] = CUDART_NAN_F;
      }
  }
  // ---- the block's sums: rescale to the common reference, add the warps
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) den[n][e] += __shfl_xor_sync(TQ_FULL, den[n][e], o);
      if (g == 0) {
        sM[warp * R + n * 8 + 2 * t + e] = M[n][e];
        sM[(DW + warp) * R + n * 8 + 2 * t + e] = den[n][e];
      }
    }
  __syncthreads();     // every warp is past its ring as well
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = n * 8 + 2 * t + e;
      float mx = sM[col];
#pragma unroll
      for (int w = 1; w < DW; ++w) mx = fmaxf(mx, sM[w * R + col]);
      const float f = mx == -CUDART_INF_F ? 0.f : ex2(M[n][e] - mx);
#pragma unroll
      for (int c4 = 0; c4 < NPL; ++c4)
        *reinterpret_cast<float4 *>(osum + (warp * R + col) * (D + 4) + 32 * c4 + 4 * g) =
            make_float4(acc_o[2 * c4][n][e] * f, acc_o[2 * c4][n][e + 2] * f, acc_o[2 * c4 + 1][n][e] * f,
                        acc_o[2 * c4 + 1][n][e + 2] * f);
    }
  __syncthreads();
  for (int r = warp; r < nrows; r += DW) {
    float mx = sM[r];
#pragma unroll
    for (int w = 1; w < DW; ++w) mx = fmaxf(mx, sM[w * R + r]);
    float l = 0.f;
#pragma unroll
    for (int w = 0; w < DW; ++w) l += sM[(DW + w) * R + r] * (mx == -CUDART_INF_F ? 0.f : ex2(sM[w * R + r] - mx));
    float x[NPL];
#pragma unroll
    for (int k = 0; k < NPL; ++k) {
      x[k] = 0.f;
#pragma unroll
      for (int w = 0; w < DW; ++w) x[k] += osum[(w * R + r) * (D + 4) + lane + 32 * k];
    }
    const int64_t row = static_cast<int64_t>(sp.row0 + (lo + r) / a.G) * a.Hq + kvh * a.G + (lo + r) % a.G;
    if (a.splits > 1) {
#pragma unroll
      for (int k = 0; k < NPL; ++k) a.po[(row * a.splits + split) * D + lane + 32 * k] = x[k];
      if (lane == 0) a.pml[row * a.splits + split] = make_float2(mx, l);
    } else {
      paged_store_row<D>(x, l, a.books, osum + r * (D + 4), a.out, a.out_dtype, row, lane);
    }
  }
}

// One warp per answer row: the splits' sums joined, rotated back, stored.
template <int D>
__global__ void __launch_bounds__(128) paged_combine_kernel(const __grid_constant__ DecArgs a, int R) {
  constexpr int NPL = D / 32;
  __shared__ float dsc[4][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + warp;
  sm100::pdl_wait();
  if (row >= static_cast<int64_t>(a.p.N) * a.Hq) return;
  const int tok = static_cast<int>(row / a.Hq), h = static_cast<int>(row % a.Hq);
  const int s = paged_find_seq(a.p, tok, 1, 0);
  const SeqSpan sp = paged_span(a.p, s);
  const int i = tok - sp.row0;
  if (i < 0 || i >= sp.n) return;
  const int vis = tile_visible(sp, a.G, (i * a.G + h % a.G) / R * R, R);
  const int n = max(1, ((vis + 31) / 32 + a.chunk - 1) / a.chunk);
  const float2 *ml = a.pml + row * a.splits;
  float mx = -CUDART_INF_F;
  for (int j = lane; j < n; j += 32) mx = fmaxf(mx, ml[j].x);
  mx = tq_warp_max(mx);
  float l = 0.f, x[NPL];
#pragma unroll
  for (int k = 0; k < NPL; ++k) x[k] = 0.f;
#pragma unroll 8
  for (int j = 0; j < n; ++j) {
    const float2 m = ml[j];
    const float f = mx == -CUDART_INF_F ? 0.f : ex2(m.x - mx);
    l = fmaf(m.y, f, l);
#pragma unroll
    for (int k = 0; k < NPL; ++k) x[k] = fmaf(a.po[(row * a.splits + j) * D + lane + 32 * k], f, x[k]);
  }
  paged_store_row<D>(x, l, a.books, dsc[warp], a.out, a.out_dtype, row, lane);
}

struct DecPlan {
  int NT, qtiles, chunk, splits, stages;
  size_t smem;
};

size_t fixed_smem(int d, int NT) {
  const size_t R = 8 * NT;
  return 2 * (d / 16) * NT * 32 * 8 + R * 16 + R * d * 4 + 256 * R * 4 + DW * 8 * 8 + 2 * DW * R * 4;
}

// Query rows a tile: 8, 16 or 32.  Blocks: enough for every SM to hold its two
// (one with 32 rows), but no fewer than 8 groups (one a warp) in a block.
DecPlan plan(const tq_codec *c, int num_seqs, int max_new, int max_len, int Hq, int Hkv) {
  DecPlan p;
  const int rows = max_new * (Hq / Hkv), sms = 148;
  p.NT = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
  p.qtiles = (rows + 8 * p.NT - 1) / (8 * p.NT);
  const int per_sm = p.NT <= 2 ? 2 : 1;
  const int64_t pairs = static_cast<int64_t>(num_seqs) * Hkv * p.qtiles;
  const int groups = std::max(1, (max_len + 31) / 32);
  const int64_t slots = static_cast<int64_t>(sms) * per_sm;
  int64_t want = pairs >= slots ? (4 * slots + pairs - 1) / pairs : slots / pairs;
  want = std::min<int64_t>(std::max<int64_t>(want, 1), (groups + DW - 1) / DW);
  want = std::min<int64_t>(want, 512);
  p.chunk = static_cast<int>((groups + want - 1) / want);
  p.splits = (groups + p.chunk - 1) / p.chunk;
  const int planes = c->mse_bits_k + c->qjl_k;
  const size_t stage = 32 * planes * (c->d / 8) + c->bits_v * c->d * 4 + 192;
  const size_t fixed = fixed_smem(c->d, p.NT);
  const size_t room = (per_sm == 2 ? 113 * 1024 : 226 * 1024) - fixed;
  const size_t merge = static_cast<size_t>(DW) * 8 * p.NT * (c->d + 4) * 4;
  p.stages = static_cast<int>(std::min<size_t>(8, room / (DW * stage)));
  p.smem = fixed + std::max(DW * p.stages * stage, merge);
  return p;
}

template <int D, bool K4, bool V4, int NT>
int run_dec(const DecArgs &a, const DecPlan &pl, cudaStream_t stream) {
  auto kern = paged_decode_kernel<D, K4, V4, NT>;
  int dev = 0;
  cudaGetDevice(&dev);
  static bool done[64] = {};
  if (dev < 64 && !done[dev]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess)
      return tq_check_launch("cudaFuncSetAttribute(paged_decode)");
    done[dev] = true;
  }
  const dim3 grid(pl.splits, a.Hkv * pl.qtiles, a.p.num_seqs);
  if (tq_launch_pdl(kern, grid, dim3(DW * 32), pl.smem, stream, a) != cudaSuccess)
    return tq_check_launch("paged_decode_kernel");
  tq_count_launch(1);
  if (pl.splits == 1) return tq_check_launch("paged_decode_kernel");
  const int64_t rows = static_cast<int64_t>(a.p.N) * a.Hq;
  if (tq_launch_pdl(paged_combine_kernel<D>, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0, stream, a,
                    8 * NT) != cudaSuccess)
    return tq_check_launch("paged_combine_kernel");
  tq_count_launch(1);
  return tq_check_launch("paged_combine_kernel");
}

template <int D, bool K4, bool V4>
int run_dec_nt(const DecArgs &a, const DecPlan &pl, cudaStream_t stream) {
  switch (pl.NT) {
    case 1: return run_dec<D, K4, V4, 1>(a, pl, stream);
    case 2: return run_dec<D, K4, V4, 2>(a, pl, stream);
    default: return run_dec<D, K4, V4, 4>(a, pl, stream);
  }
}

template <int D>
int run_dec_d(const DecArgs &a, const DecPlan &pl, bool k4, bool v4, cudaStream_t stream) {
  if (k4) return v4 ? run_dec_nt<D, true, true>(a, pl, stream) : run_dec_nt<D, true, false>(a, pl, stream);
  return v4 ? run_dec_nt<D, false, true>(a, pl, stream) : run_dec_nt<D, false, false>(a, pl, stream);
}

}  // namespace

size_t paged_decode_workspace_bytes(const tq_codec *c, int N, int num_seqs, int max_new, int max_len, int Hq,
                                    int Hkv) {
  const DecPlan p = plan(c, num_seqs, max_new, max_len, Hq, Hkv);
  if (p.splits == 1) return 16;
  return static_cast<size_t>(N) * Hq * p.splits * (c->d + 2) * sizeof(float) + 16;
}

int launch_paged_decode(const tq_codec *c, const PagedView &p, const void *q, int dtype, int64_t st, int64_t sh,
                        int Hq, const tq_cache *cache, float scale, const float *rc, const float *rs, void *ws,
                        void *out, int out_dtype, cudaStream_t stream) {
  const DecPlan pl = plan(c, p.num_seqs, p.max_new, p.max_len, Hq, cache->Hkv);
  DecArgs a;
  a.p = p;
  a.q = q;
  a.dtype = dtype;
  a.st = st;
  a.sh = sh;
  a.Hq = Hq;
  a.Hkv = cache->Hkv;
  a.G = Hq / cache->Hkv;
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
  a.S = c->S_dev;
  a.qtiles = pl.qtiles;
  a.chunk = pl.chunk;
  a.splits = pl.splits;
  a.stages = pl.stages;
  a.po = static_cast<float *>(ws);
  a.pml = reinterpret_cast<float2 *>(a.po + static_cast<size_t>(p.N) * Hq * pl.splits * c->d);
  a.wait_limit = 1u << 26;
  if (const char *e = getenv("TQ_WAIT_LIMIT")) a.wait_limit = static_cast<uint32_t>(strtoul(e, nullptr, 10));
  byte_table(c->books.ck, c->mse_bits_k, a.lutk);
  byte_table(c->books.cv, c->bits_v, a.lutv);
  a.books = c->books;
  const bool k4 = c->mse_bits_k == 4, v4 = c->bits_v == 4;
  return c->d == 64 ? run_dec_d<64>(a, pl, k4, v4, stream) : run_dec_d<128>(a, pl, k4, v4, stream);
}
