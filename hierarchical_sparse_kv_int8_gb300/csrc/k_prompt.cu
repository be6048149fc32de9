// Causal attention of packed sequences.
//
// One warp per (query token, head): an online softmax over the keys the query
// sees, one key at a time.
#include "pages_internal.cuh"

#include <math_constants.h>

namespace dhs {
namespace {

constexpr int kPrWarps = 4;

struct PromptStrides {
  int64_t qt, qh, kt, kh, vt, vh;
};

template <int D>
__global__ void __launch_bounds__(kPrWarps * 32)
k_prompt(const __nv_bfloat16 *__restrict__ q, const __nv_bfloat16 *__restrict__ k,
         const __nv_bfloat16 *__restrict__ v, const PromptStrides st, int64_t n_q, int64_t n_k,
         const int32_t *__restrict__ cu_q, const int32_t *__restrict__ cu_k, int n_seqs, int hq,
         int hkv, float scale_log2, __nv_bfloat16 *__restrict__ out, float *__restrict__ lse,
         int32_t *err) {
  const int64_t item = (int64_t)blockIdx.x * kPrWarps + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (item >= n_q * hq) return;
  const int64_t tok = item / hq;
  const int h = (int)(item - tok * hq), kvh = h / (hq / hkv);
  const int i = seq_of(cu_q, n_seqs, tok);
  if (i < 0) return;
  const int64_t k0 = cu_k[i], k1 = cu_k[i + 1];
  if (k0 < 0 || k1 < k0 || k1 > n_k || cu_q[i + 1] > n_q || cu_q[i] < 0) {
    page_error(err, DC_ROW_RANGE, DHS_SITE_PROMPT_ATTEND);
    return;
  }
  const int64_t seen = (k1 - k0) - (cu_q[i + 1] - tok) + 1;
  float qv[D / 32], o[D / 32], m = -CUDART_INF_F, l = 0.f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) {
    qv[e] = __bfloat162float(q[tok * st.qt + h * st.qh + lane * (D / 32) + e]);
    o[e] = 0.f;
  }
  for (int64_t t = k0; t < k0 + seen; ++t) {
    const __nv_bfloat16 *kr = k + t * st.kt + kvh * st.kh + lane * (D / 32);
    const __nv_bfloat16 *vr = v + t * st.vt + kvh * st.vh + lane * (D / 32);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) s = fmaf(qv[e], __bfloat162float(kr[e]), s);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    s *= scale_log2;
    const float mn = fmaxf(m, s), base = mn == -CUDART_INF_F ? 0.f : mn;
    const float f = exp2f(m - base), p = exp2f(s - base);
    m = mn;
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] = o[e] * f + p * __bfloat162float(vr[e]);
  }
#pragma unroll
  for (int e = 0; e < D / 32; ++e)
    out[item * D + lane * (D / 32) + e] = __float2bfloat16(seen <= 0 ? 0.f : o[e] / l);
  if (lse && lane == 0)
    lse[item] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.69314718055994531f;
}

bool prompt_args(int64_t n_q, int64_t n_k, int32_t n_seqs, int32_t hq, int32_t hkv, int32_t d) {
  return n_q >= 0 && n_k >= 0 && n_q <= INT32_MAX && n_k <= INT32_MAX && n_seqs >= 0 && hkv >= 1 &&
         hkv <= kPageMaxHeads && hq >= 1 && hq % hkv == 0 && hq / hkv <= 128 &&
         (d == 64 || d == 128);
}

}  // namespace
}  // namespace dhs

extern "C" int64_t dhs_prompt_attend_workspace(int64_t n_q, int64_t n_k, int32_t n_seqs,
                                               int32_t q_heads, int32_t kv_heads,
                                               int32_t head_dim) {
  return dhs::prompt_args(n_q, n_k, n_seqs, q_heads, kv_heads, head_dim) ? 0 : -1;
}

extern "C" int dhs_prompt_attend(const void *q, const void *k, const void *v,
                                 const int64_t *strides, int64_t n_q, int64_t n_k,
                                 const int32_t *cu_q, const int32_t *cu_k, int32_t n_seqs,
                                 int32_t q_heads, int32_t kv_heads, int32_t head_dim, float scale,
                                 void *out, float *lse, void *workspace, int64_t workspace_bytes,
                                 int32_t *err, dhs_stream stream) {
  using namespace dhs;
  if (!prompt_args(n_q, n_k, n_seqs, q_heads, kv_heads, head_dim) || !(scale >= 0.f) ||
      scale > 3e38f || workspace_bytes < 0)
    return DHS_ERR_INVALID;
  if (n_q == 0 || n_seqs == 0) return DHS_OK;
  if (!q || !out || !cu_q || !cu_k || (n_k > 0 && (!k || !v)) || ((uintptr_t)q & 15u) ||
      ((uintptr_t)k & 15u) || ((uintptr_t)v & 15u) || ((uintptr_t)out & 15u) ||
      ((uintptr_t)workspace & 15u))
    return DHS_ERR_INVALID;
  const int64_t d = head_dim;
  PromptStrides st = {q_heads * d, d, kv_heads * d, d, kv_heads * d, d};
  if (strides) {
    for (int i = 0; i < 6; ++i)
      if (strides[i] < 0 || strides[i] % 8 || strides[i] > ((int64_t)1 << 38)) return DHS_ERR_INVALID;
    st = {strides[0], strides[1], strides[2], strides[3], strides[4], strides[5]};
  }
  (void)workspace;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const float sl2 = (scale == 0.f ? 1.f / sqrtf((float)d) : scale) * 1.4426950408889634f;
  const int64_t items = n_q * q_heads;
  auto go = [&](auto kern) {
    return launch_prio(kern, dim3((unsigned)((items + kPrWarps - 1) / kPrWarps)),
                       dim3(kPrWarps * 32), 0, s, static_cast<const __nv_bfloat16 *>(q),
                       static_cast<const __nv_bfloat16 *>(k),
                       static_cast<const __nv_bfloat16 *>(v), st, n_q, n_k, cu_q, cu_k, n_seqs,
                       q_heads, kv_heads, sl2, static_cast<__nv_bfloat16 *>(out), lse, err);
  };
  const cudaError_t e = d == 128 ? go(k_prompt<128>) : go(k_prompt<64>);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return DHS_ERR_CUDA;
  }
  return DHS_OK;
}
