// Shared by the paged-cache and prompt operators: the cache as kernels see it,
// where a position lives in it, and which sequence a packed token belongs to.
#pragma once
#include "dhs_internal.cuh"
#include "ptx_util.cuh"

#include <atomic>

namespace dhs {

constexpr int kPageMaxHeads = 1024;
constexpr int kMaxDevices = 64;
// Sequences of a call at most: loops over them run up to 1024 past the last, in 32 bits.
constexpr int kMaxSeqs = INT32_MAX - 1024;

// Streaming multiprocessors of a device (asked once), 0 on failure.
int device_sms(int dev);

// A kernel's dynamic shared-memory limit, raised once on each device.
struct DeviceSmem {
  std::atomic<int> done[kMaxDevices] = {};
  template <typename F>
  cudaError_t ensure(F *func, int bytes, int dev) {
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    cudaError_t e = same_carveout(func);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done[dev].store(1, std::memory_order_release);
    return e;
  }
};

// The cache, by value.  A "row" is one (page, kv head, page row): head_dim
// elements at row * head_dim and one scale at `row` of the scale arrays.
struct PageView {
  unsigned char *k, *v;
  float *ks, *vs;
  int64_t n_pages;
  int rows, hkv, d, kind;
  uint32_t div_mul;  // pos / rows = pos * div_mul >> div_shift for 0 <= pos < 2^31
  int div_shift;
};

// Whether arrays of 32-bit words (NULL: none) lie where words may lie.
template <typename... P>
bool words(const P *...p) {
  return (((uintptr_t)p | ...) & 3u) == 0;
}

inline bool page_view(const dhs_pages *p, PageView *out) {
  if (!p || !p->k || !p->v || ((uintptr_t)p->k & 15u) || ((uintptr_t)p->v & 15u)) return false;
  if (p->kind < DHS_PAGE_BF16 || p->kind > DHS_PAGE_E4M3) return false;
  if (p->kind != DHS_PAGE_BF16 && (!p->k_scale || !p->v_scale)) return false;
  if (p->kind != DHS_PAGE_BF16 && !words(p->k_scale, p->v_scale)) return false;
  if (p->page_rows < 1 || p->kv_heads < 1 || p->kv_heads > kPageMaxHeads || p->n_pages < 1 ||
      p->n_pages > INT32_MAX || (p->head_dim != 64 && p->head_dim != 128))
    return false;
  out->k = static_cast<unsigned char *>(p->k);
  out->v = static_cast<unsigned char *>(p->v);
  out->ks = p->k_scale;
  out->vs = p->v_scale;
  out->n_pages = p->n_pages;
  out->rows = p->page_rows;
  out->hkv = p->kv_heads;
  out->d = p->head_dim;
  out->kind = p->kind;
  // with 2^s >= rows, ceil(2^(31 + s) / rows) is off by less than 2^-31 of a
  // quotient's unit for every pos < 2^31, and fits 32 bits
  int s = 0;
  while (((int64_t)1 << s) < p->page_rows) ++s;
  out->div_mul = (uint32_t)((((uint64_t)1 << (31 + s)) + p->page_rows - 1) / p->page_rows);
  out->div_shift = 31 + s;
  return true;
}

__device__ __forceinline__ void page_error(int32_t *err, int code, int site) {
  if (err) record_error(err, code, site);
}

// Row (of kv head 0) that holds position `pos` of the sequence whose table
// starts at `tab`, or -1 (recorded) where the table names no page; kv head h's
// row is h * rows further on.  The caller has checked 0 <= pos < width * rows.
__device__ __forceinline__ int64_t page_row(const PageView &p, const int32_t *tab, int pos,
                                            int32_t *err, int site) {
  const int pg = (int)((uint64_t)(uint32_t)pos * p.div_mul >> p.div_shift);
  const int in = pos - pg * p.rows;
  const int32_t page = tab[pg];
  if (page < 0 || page >= p.n_pages) {
    page_error(err, DC_LOC_RANGE, site);
    return -1;
  }
  return (int64_t)page * p.hkv * p.rows + in;
}

// Sequence of packed token `tok`: the i with cu[i] <= tok < cu[i + 1], or -1
// (padding).  For offsets that do not ascend some i or -1 comes back; the
// caller checks what it derives from it.
__device__ __forceinline__ int seq_of(const int32_t *cu, int n, int64_t tok) {
  if (tok < cu[0]) return -1;
  int lo = 0, hi = n;  // cu[lo] <= tok; hi is n or cu[hi] > tok
  while (lo < hi) {
    const int mid = lo + ((hi - lo + 1) >> 1);  // (n may be more than 2^30)
    if (cu[mid] <= tok) lo = mid;
    else hi = mid - 1;
  }
  return lo < n ? lo : -1;
}

}  // namespace dhs
