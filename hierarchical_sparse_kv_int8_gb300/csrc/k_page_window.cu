// Attention of the newest tokens of every sequence over its paged cache with a sliding window
// and first positions that stay visible: the kernels of page_attn.cuh that go by a list of a
// sequence's blocks, and their entry point.
//
// A query at position p sees (p - window, p] and [0, sinks).  Of a sequence's blocks only those
// are walked, and only their pages looked up, that some of its queries sees: what lies between
// the sinks and the first query's window costs nothing.  The last q_len - 1 positions before the
// last query's window are seen by some queries and not by others, as are the newest q_len - 1.
// Measured (GB300): 128 sequences of up to 102400 positions in a window of 4096 with 4 sinks,
// int8, 16 rows, 45.9 us, of which the bytes take 21 at the measured copy bandwidth: from the
// start through the lengths, a CTA's place, the page table and the first rows it takes 7 us,
// 25 to stream, a second item in a CTA some 7 more, the join 4; in e4m3 45.8, in bf16 54.9 (40 of
// bytes).  One sequence, bf16, 9.6 us.
#include "page_attn.cuh"

extern "C" int dhs_page_attend_window(const dhs_pages *pages, const void *q, const int32_t *q_lens,
                                      const int32_t *seq_lens, const int32_t *page_table,
                                      int32_t table_width, int32_t n_seqs, int32_t q_len,
                                      int32_t q_heads, int32_t window, int32_t sinks, float scale,
                                      void *out, float *lse, void *workspace,
                                      int64_t workspace_bytes, int32_t *err, dhs_stream stream) {
  if (window < 1) return DHS_ERR_INVALID;
  return dhs::attend_call<true>(pages, q, q_lens, seq_lens, page_table, table_width, n_seqs, q_len,
                                q_heads, window, sinks, scale, out, lse, workspace, workspace_bytes,
                                err, stream);
}
