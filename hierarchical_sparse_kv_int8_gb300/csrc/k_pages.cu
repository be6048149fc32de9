// The paged cache's write (with quantisation) and read-back.
//
// Token cu[i] + u of a packed batch is position p = len_i - n_i + u of sequence
// i and lives in row p mod R of page table[i][p / R].  In the 8-bit kinds each
// (token, head) row x keeps s = max|x| / Q and the codes round(x / s).
//
// Both directions move every byte once and are bound by HBM: a row of 64 or 128
// values is shared by 8 or 16 lanes of 16 bytes, so that the bf16 side is read
// or written in whole 128- and 256-byte rows and the 8-bit side in 64- and
// 128-byte ones; the row's maximum takes three or four shuffles.
#include "pages_internal.cuh"

namespace dhs {
namespace {

constexpr int kPgThreads = 256;
constexpr int kPgTok = 32;  // tokens of a CTA at most (their places in shared memory)
constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100

struct TokenRows {
  unsigned char *k, *v;          // bf16
  int64_t kt, kh, vt, vh;        // strides of a token and a head, in elements
};

// Whether x / s > mid in real numbers, `mid` of at most 8 significant bits:
// the product's rounding error is recovered by the fused multiply-add, and
// x - hi is exact because the two are within a factor of two (x / s is next to
// mid).  Returns -1, 0, 1 for below, equal, above.
__device__ __forceinline__ int side_of(float x, float s, float mid) {
  const float hi = mid * s, lo = fmaf(mid, s, -hi);
  const float d = (x - hi) - lo;
  return d > 0.f ? 1 : (d < 0.f ? -1 : 0);
}

// The code value (a whole number up to 127) of x >= 0: x / s to nearest even.
// y = x * (1 / s) is off by less than 2^-15, which matters only next to a
// half; there the side is decided exactly.
__device__ __forceinline__ float round_int8(float x, float s, float inv) {
  const float y = x * inv;
  float c = rintf(y);
  if (fabsf(fabsf(y - c) - 0.5f) < 1e-3f) {
    const float f = floorf(y), mid = f + 0.5f;
    const int side = side_of(x, s, mid);
    const bool odd = (((int)f) & 1) != 0;
    c = (side > 0 || (side == 0 && odd)) ? f + 1.f : f;
  }
  return fminf(c, 127.f);
}
// The same on the e4m3 grid, whose spacing at y is 2^(max(e, -6) - 3), e the
// exponent of y: y over the spacing is a whole number of at most 16 plus a
// fraction.
__device__ __forceinline__ float round_e4m3(float x, float s, float inv) {
  const float y = x * inv;
  const int e = max((int)(__float_as_uint(y) >> 23) - 127, -6);
  const float up = __uint_as_float((uint32_t)(127 + 3 - e) << 23);    // 2^(3 - e)
  const float step = __uint_as_float((uint32_t)(127 + e - 3) << 23);  // 2^(e - 3)
  const float z = y * up;
  float c = rintf(z);
  if (fabsf(fabsf(z - c) - 0.5f) < 1e-4f) {
    const float f = floorf(z);
    const int side = side_of(x, s, (f + 0.5f) * step);
    const bool odd = (((int)f) & 1) != 0;
    c = (side > 0 || (side == 0 && odd)) ? f + 1.f : f;
  }
  return fminf(c * step, 448.f);
}

// Bits of a finite non-negative value that lies on the e4m3 grid.
__device__ __forceinline__ uint32_t e4m3_bits(float v) {
  const uint32_t u = __float_as_uint(v);
  const int e = (int)(u >> 23) - 127;
  return e >= -6 ? (uint32_t)((e + 7) << 3) | ((u >> 20) & 7u) : (uint32_t)(v * 512.f);
}

// e4m3 code to its value (finite codes).
__device__ __forceinline__ float e4m3_value(uint32_t c) {
  // the code's seven lower bits at a float's exponent and mantissa give the
  // value times 2^-120, subnormals included
  const float m = __uint_as_float((c & 0x7Fu) << 20) * 1.329227995784916e36f;  // 2^120
  return (c & 0x80u) ? -m : m;
}

// Where the tokens of this CTA live: row of kv head 0, -1 none, -2 padding.
__device__ __forceinline__ int64_t place(const PageView &pg, const int32_t *cu,
                                         const int32_t *lens, const int32_t *table, int width,
                                         int n_seqs, int64_t tok, int32_t *err, int site) {
  const int i = seq_of(cu, n_seqs, tok);
  if (i < 0) return -2;
  const int64_t pos = (int64_t)lens[i] - ((int64_t)cu[i + 1] - tok);
  if (pos < 0 || pos >= (int64_t)width * pg.rows || pos > INT32_MAX) {
    page_error(err, DC_ROW_RANGE, site);
    return -1;
  }
  return page_row(pg, table + (int64_t)i * width, (int)pos, err, site);
}

template <int D, int KIND>
__global__ void __launch_bounds__(kPgThreads)
k_page_write(const PageView pg, const TokenRows src, int64_t n_tok, int per_cta,
             const int32_t *__restrict__ cu, const int32_t *__restrict__ lens,
             const int32_t *__restrict__ table, int width, int n_seqs, int32_t *err) {
  constexpr int L = D / 8;  // lanes of a row
  __shared__ int64_t dst[kPgTok];
  const int64_t t0 = (int64_t)blockIdx.x * per_cta;
  const int nt = (int)min((int64_t)per_cta, n_tok - t0);
  if (threadIdx.x < nt)
    dst[threadIdx.x] = place(pg, cu, lens, table, width, n_seqs, t0 + threadIdx.x, err,
                             DHS_SITE_PAGE_WRITE);
  __syncthreads();
  const int sub = threadIdx.x % L;
  // every lane of a warp takes part in the shuffles, with or without a row
  const int total = nt * pg.hkv, rounds = (total + kPgThreads / L - 1) / (kPgThreads / L);
  for (int it = 0; it < rounds; ++it) {
    const int e = it * (kPgThreads / L) + threadIdx.x / L;
    const int t = e / pg.hkv, h = e - t * pg.hkv;
    const int64_t base = e < total ? dst[t] : -2;
    const bool on = base >= 0;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (on)
        w = *reinterpret_cast<const uint4 *>(
            (side ? src.v : src.k) +
            2 * ((t0 + t) * (side ? src.vt : src.kt) + h * (side ? src.vh : src.kh) + sub * 8));
      const int64_t row = base + (int64_t)h * pg.rows;
      unsigned char *out = side ? pg.v : pg.k;
      if (KIND == DHS_PAGE_BF16) {
        if (on) *reinterpret_cast<uint4 *>(out + (row * D + sub * 8) * 2) = w;
        continue;
      }
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
      // the largest magnitude as bits: an infinity or a NaN is the largest
      uint32_t top = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        top = max(top, max(u[i] & 0x7FFFu, (u[i] >> 16) & 0x7FFFu));
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float big = __uint_as_float(top << 16);
      const bool bad = top >= 0x7F80u;
      const float s = (bad || big < kTiny) ? 0.f
                                           : __fdiv_rn(big, KIND == DHS_PAGE_INT8 ? 127.f : 448.f);
      const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
      uint32_t code[2] = {0u, 0u};
      if (s > 0.f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t b = (u[i >> 1] >> ((i & 1) * 16)) & 0xFFFFu;
          const float x = __uint_as_float((b & 0x7FFFu) << 16);
          const bool neg = (b & 0x8000u) != 0u;
          uint32_t c;
          if (KIND == DHS_PAGE_INT8) {
            const int v = (int)round_int8(x, s, inv);
            c = (uint32_t)(neg ? -v : v) & 0xFFu;
          } else {
            c = e4m3_bits(round_e4m3(x, s, inv)) | (neg ? 0x80u : 0u);
          }
          code[i >> 2] |= c << ((i & 3) * 8);
        }
      }
      if (on) {
        *reinterpret_cast<uint2 *>(out + row * D + sub * 8) = make_uint2(code[0], code[1]);
        if (sub == 0) (side ? pg.vs : pg.ks)[row] = bad ? __uint_as_float(0x7FC00000u) : s;
      }
    }
  }
}

template <int D, int KIND>
__global__ void __launch_bounds__(kPgThreads)
k_page_read(const PageView pg, const TokenRows to, int64_t n_tok, int per_cta,
            const int32_t *__restrict__ cu, const int32_t *__restrict__ lens,
            const int32_t *__restrict__ table, int width, int n_seqs, int32_t *err) {
  constexpr int L = D / 8;
  __shared__ int64_t src[kPgTok];
  const int64_t t0 = (int64_t)blockIdx.x * per_cta;
  const int nt = (int)min((int64_t)per_cta, n_tok - t0);
  if (threadIdx.x < nt)
    src[threadIdx.x] = place(pg, cu, lens, table, width, n_seqs, t0 + threadIdx.x, err,
                             DHS_SITE_PAGE_READ);
  __syncthreads();
  const int sub = threadIdx.x % L, total = nt * pg.hkv;
  for (int e = threadIdx.x / L; e < total; e += kPgThreads / L) {
    const int t = e / pg.hkv, h = e - t * pg.hkv;
    const int64_t base = src[t];
    if (base == -2) continue;
    const int64_t row = base + (int64_t)h * pg.rows;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      const unsigned char *in = side ? pg.v : pg.k;
      if (base >= 0) {
        if (KIND == DHS_PAGE_BF16) {
          w = *reinterpret_cast<const uint4 *>(in + (row * D + sub * 8) * 2);
        } else {
          const uint2 c = *reinterpret_cast<const uint2 *>(in + row * D + sub * 8);
          const float s = (side ? pg.vs : pg.ks)[row];
          float x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t b = ((i < 4 ? c.x : c.y) >> ((i & 3) * 8)) & 0xFFu;
            x[i] = (KIND == DHS_PAGE_INT8 ? (float)(int8_t)b : e4m3_value(b)) * s;
          }
          w = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                         pack_bf16(x[6], x[7]));
        }
      }
      *reinterpret_cast<uint4 *>(
          (side ? to.v : to.k) +
          2 * ((t0 + t) * (side ? to.vt : to.kt) + h * (side ? to.vh : to.kh) + sub * 8)) = w;
    }
  }
}

// Tokens of a CTA: enough CTAs to fill the GPU first, then more tokens each.
int tokens_per_cta(int64_t n_tok) {
  int64_t per = n_tok / 608;  // four CTAs on each of 152 SMs
  return (int)(per < 1 ? 1 : (per > kPgTok ? kPgTok : per));
}

int page_copy(bool write, const dhs_pages *pages, void *k, void *v, const int64_t *strides,
              int64_t n_tok, const int32_t *cu, const int32_t *lens, const int32_t *table,
              int32_t width, int32_t n_seqs, int32_t *err, dhs_stream stream) {
  PageView pg;
  if (!page_view(pages, &pg) || n_tok < 0 || n_seqs < 0 || width < 0) return DHS_ERR_INVALID;
  if (n_tok == 0 || n_seqs == 0) return DHS_OK;
  if (!k || !v || !cu || !lens || !table || width < 1 || ((uintptr_t)k & 15u) ||
      ((uintptr_t)v & 15u))
    return DHS_ERR_INVALID;
  if (n_tok > INT32_MAX) return DHS_ERR_CAPACITY;
  TokenRows r;
  r.k = static_cast<unsigned char *>(k);
  r.v = static_cast<unsigned char *>(v);
  r.kt = r.vt = (int64_t)pg.hkv * pg.d;
  r.kh = r.vh = pg.d;
  if (strides) {
    for (int i = 0; i < 4; ++i)
      if (strides[i] < 0 || strides[i] % 8 || strides[i] > ((int64_t)1 << 40)) return DHS_ERR_INVALID;
    r.kt = strides[0];
    r.kh = strides[1];
    r.vt = strides[2];
    r.vh = strides[3];
    // rows that are written must not lie over one another
    if (!write)
      for (int i = 0; i < 4; ++i)
        if ((i & 1 ? pg.hkv > 1 : n_tok > 1) && strides[i] < pg.d) return DHS_ERR_INVALID;
  }
  const int per = tokens_per_cta(n_tok);
  const unsigned grid = (unsigned)((n_tok + per - 1) / per);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto go = [&](auto kern) {
    return launch_prio(kern, dim3(grid), dim3(kPgThreads), 0, s, pg, r, n_tok, per, cu, lens,
                       table, width, n_seqs, err);
  };
  cudaError_t e;
  const int key = (write ? 0 : 8) + (pg.d == 128 ? 4 : 0) + pg.kind;
  switch (key) {
    case 0: e = go(k_page_write<64, DHS_PAGE_BF16>); break;
    case 1: e = go(k_page_write<64, DHS_PAGE_INT8>); break;
    case 2: e = go(k_page_write<64, DHS_PAGE_E4M3>); break;
    case 4: e = go(k_page_write<128, DHS_PAGE_BF16>); break;
    case 5: e = go(k_page_write<128, DHS_PAGE_INT8>); break;
    case 6: e = go(k_page_write<128, DHS_PAGE_E4M3>); break;
    case 8: e = go(k_page_read<64, DHS_PAGE_BF16>); break;
    case 9: e = go(k_page_read<64, DHS_PAGE_INT8>); break;
    case 10: e = go(k_page_read<64, DHS_PAGE_E4M3>); break;
    case 12: e = go(k_page_read<128, DHS_PAGE_BF16>); break;
    case 13: e = go(k_page_read<128, DHS_PAGE_INT8>); break;
    default: e = go(k_page_read<128, DHS_PAGE_E4M3>); break;
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return DHS_ERR_CUDA;
  }
  return DHS_OK;
}

}  // namespace
}  // namespace dhs

extern "C" int dhs_page_write(const dhs_pages *pages, const void *k, const void *v,
                              const int64_t *strides, int64_t n_tokens, const int32_t *cu,
                              const int32_t *seq_lens, const int32_t *page_table,
                              int32_t table_width, int32_t n_seqs, int32_t *err,
                              dhs_stream stream) {
  return dhs::page_copy(true, pages, const_cast<void *>(k), const_cast<void *>(v), strides,
                        n_tokens, cu, seq_lens, page_table, table_width, n_seqs, err, stream);
}

extern "C" int dhs_page_read(const dhs_pages *pages, void *k, void *v, const int64_t *strides,
                             int64_t n_tokens, const int32_t *cu, const int32_t *seq_lens,
                             const int32_t *page_table, int32_t table_width, int32_t n_seqs,
                             int32_t *err, dhs_stream stream) {
  return dhs::page_copy(false, pages, k, v, strides, n_tokens, cu, seq_lens, page_table,
                        table_width, n_seqs, err, stream);
}
