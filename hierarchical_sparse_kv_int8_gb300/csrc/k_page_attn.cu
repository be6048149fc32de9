// Attention of the newest tokens of every sequence over its paged cache.
//
// One warp per (sequence, query, head): it walks the visible positions one by
// one with the running maximum m and sum l of an online softmax in log2 units,
//   m' = max(m, x),  o = o 2^(m - m') + 2^(x - m') v,  l likewise.
#include "pages_internal.cuh"

#include <math_constants.h>

namespace dhs {
namespace {

constexpr int kPaWarps = 4;

template <int D, int KIND>
__device__ __forceinline__ void row_values(const unsigned char *base, const float *sc, int64_t row,
                                           int lane, float (&x)[D / 32]) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const int64_t at = row * D + lane * (D / 32) + i;
    if (KIND == DHS_PAGE_BF16)
      x[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(base)[at]);
    else if (KIND == DHS_PAGE_INT8)
      x[i] = (float)reinterpret_cast<const int8_t *>(base)[at] * sc[row];
    else {
      const uint32_t c = base[at];
      const float m = __uint_as_float((c & 0x7Fu) << 20) * 1.329227995784916e36f;
      x[i] = (c & 0x80u ? -m : m) * sc[row];
    }
  }
}

template <int D, int KIND>
__global__ void __launch_bounds__(kPaWarps * 32)
k_page_attn(const PageView pg, const __nv_bfloat16 *__restrict__ q,
            const int32_t *__restrict__ q_lens, const int32_t *__restrict__ seq_lens,
            const int32_t *__restrict__ table, int width, int n_seqs, int q_len, int hq,
            float scale_log2, __nv_bfloat16 *__restrict__ out, float *__restrict__ lse,
            int32_t *err) {
  const int64_t item = (int64_t)blockIdx.x * kPaWarps + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (item >= (int64_t)n_seqs * q_len * hq) return;
  const int h = (int)(item % hq), j = (int)(item / hq % q_len), i = (int)(item / hq / q_len);
  const int kvh = h / (hq / pg.hkv);
  int nq = q_lens ? q_lens[i] : q_len, len = seq_lens[i];
  if (nq < 0 || nq > q_len || len < 0 || len > (int64_t)width * pg.rows) {
    page_error(err, DC_ROW_RANGE, DHS_SITE_PAGE_ATTEND);
    nq = max(0, min(nq, q_len));
    len = (int)max((int64_t)0, min((int64_t)len, (int64_t)width * pg.rows));
  }
  if (j >= nq) return;
  const int seen = len - nq + j + 1;
  float qv[D / 32], o[D / 32], m = -CUDART_INF_F, l = 0.f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) {
    qv[e] = __bfloat162float(q[item * D + lane * (D / 32) + e]);
    o[e] = 0.f;
  }
  for (int t = 0; t < seen; ++t) {
    int64_t row = page_row(pg, table + (int64_t)i * width, t, err, DHS_SITE_PAGE_ATTEND);
    if (row < 0) continue;
    row += (int64_t)kvh * pg.rows;
    float x[D / 32], s = 0.f;
    row_values<D, KIND>(pg.k, pg.ks, row, lane, x);
#pragma unroll
    for (int e = 0; e < D / 32; ++e) s = fmaf(qv[e], x[e], s);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    s *= scale_log2;
    const float mn = fmaxf(m, s), base = mn == -CUDART_INF_F ? 0.f : mn;
    const float f = exp2f(m - base), p = exp2f(s - base);
    m = mn;
    l = l * f + p;
    row_values<D, KIND>(pg.v, pg.vs, row, lane, x);
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] = o[e] * f + p * x[e];
  }
  // nothing seen: 0; only scores of -infinity: 0 / 0
  const float inv = m == -CUDART_INF_F && l == 0.f && seen <= 0 ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < D / 32; ++e)
    out[item * D + lane * (D / 32) + e] = __float2bfloat16(seen <= 0 ? 0.f : o[e] * inv);
  if (lse && lane == 0)
    lse[item] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.69314718055994531f;
}

bool attend_args(const dhs_pages *pages, int32_t n_seqs, int32_t q_len, int32_t q_heads,
                 PageView *pg) {
  return page_view(pages, pg) && n_seqs >= 0 && q_len >= 1 && q_len <= kMaxKmax && q_heads >= 1 &&
         q_heads % pg->hkv == 0 && (int64_t)q_len * (q_heads / pg->hkv) <= 128;
}

}  // namespace
}  // namespace dhs

extern "C" int64_t dhs_page_attend_workspace(const dhs_pages *pages, int32_t n_seqs, int32_t q_len,
                                             int32_t q_heads) {
  dhs::PageView pg;
  return dhs::attend_args(pages, n_seqs, q_len, q_heads, &pg) ? 0 : -1;
}

extern "C" int dhs_page_attend(const dhs_pages *pages, const void *q, const int32_t *q_lens,
                               const int32_t *seq_lens, const int32_t *page_table,
                               int32_t table_width, int32_t n_seqs, int32_t q_len,
                               int32_t q_heads, float scale, void *out, float *lse,
                               void *workspace, int64_t workspace_bytes, int32_t *err,
                               dhs_stream stream) {
  using namespace dhs;
  PageView pg;
  if (!attend_args(pages, n_seqs, q_len, q_heads, &pg) || table_width < 0 || !(scale >= 0.f) ||
      scale > 3e38f || workspace_bytes < 0)
    return DHS_ERR_INVALID;
  if (n_seqs == 0) return DHS_OK;
  if (!q || !seq_lens || !page_table || !out || ((uintptr_t)q & 15u) || ((uintptr_t)out & 15u) ||
      ((uintptr_t)workspace & 15u))
    return DHS_ERR_INVALID;
  (void)workspace;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const float sl2 = (scale == 0.f ? 1.f / sqrtf((float)pg.d) : scale) * 1.4426950408889634f;
  const int64_t items = (int64_t)n_seqs * q_len * q_heads;
  auto go = [&](auto kern) {
    return launch_prio(kern, dim3((unsigned)((items + kPaWarps - 1) / kPaWarps)),
                       dim3(kPaWarps * 32), 0, s, pg, static_cast<const __nv_bfloat16 *>(q),
                       q_lens, seq_lens, page_table, table_width, n_seqs, q_len, q_heads, sl2,
                       static_cast<__nv_bfloat16 *>(out), lse, err);
  };
  cudaError_t e;
  switch ((pg.d == 128 ? 4 : 0) + pg.kind) {
    case 0: e = go(k_page_attn<64, DHS_PAGE_BF16>); break;
    case 1: e = go(k_page_attn<64, DHS_PAGE_INT8>); break;
    case 2: e = go(k_page_attn<64, DHS_PAGE_E4M3>); break;
    case 4: e = go(k_page_attn<128, DHS_PAGE_BF16>); break;
    case 5: e = go(k_page_attn<128, DHS_PAGE_INT8>); break;
    default: e = go(k_page_attn<128, DHS_PAGE_E4M3>); break;
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return DHS_ERR_CUDA;
  }
  return DHS_OK;
}
