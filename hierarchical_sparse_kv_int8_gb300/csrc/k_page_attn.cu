// Attention of the newest tokens of every sequence over its paged cache: the kernels that see
// every position, and their entry points.
#include "page_attn.cuh"

namespace dhs {

int device_sms(int dev) {
  static std::atomic<int> known[kMaxDevices];
  if (dev < 0 || dev >= kMaxDevices) return 0;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

}  // namespace dhs

extern "C" int64_t dhs_page_attend_workspace(const dhs_pages *pages, int32_t n_seqs, int32_t q_len,
                                             int32_t q_heads) {
  using namespace dhs;
  PageView pg;
  if (!attend_args(pages, n_seqs, q_len, q_heads, &pg)) return -1;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  const int R = q_len * (q_heads / pg.hkv), sms = device_sms(dev);
  if (sms < 1) return -1;
  return pick<false>(pg, R, q_len, [&](auto c) -> int64_t {
    return plan_bytes(n_seqs, pg.hkv) + (int64_t)sms * decltype(c)::OCC * 2 * R * (pg.d + 4) * 4;
  });
}

extern "C" int dhs_page_attend(const dhs_pages *pages, const void *q, const int32_t *q_lens,
                               const int32_t *seq_lens, const int32_t *page_table,
                               int32_t table_width, int32_t n_seqs, int32_t q_len,
                               int32_t q_heads, float scale, void *out, float *lse,
                               void *workspace, int64_t workspace_bytes, int32_t *err,
                               dhs_stream stream) {
  return dhs::attend_call<false>(pages, q, q_lens, seq_lens, page_table, table_width, n_seqs, q_len,
                                 q_heads, 0, 0, scale, out, lse, workspace, workspace_bytes, err,
                                 stream);
}
