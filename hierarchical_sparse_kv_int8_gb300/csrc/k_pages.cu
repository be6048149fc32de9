// The paged cache's write (with quantisation) and read-back.
//
// Token cu[i] + u of a packed batch is position p = len_i - n_i + u of sequence
// i and lives in row p mod R of page table[i][p / R].  In the 8-bit kinds each
// (token, head) row x keeps s = max|x| / Q and the codes round(x / s).
//
// Both directions move every byte once and are bound by HBM: 37,000 tokens of 8 heads of
// 128 dims are written as e4m3 in 44 us (78 % of the measured copy bandwidth; bf16 to
// bf16 86 %), two times 65536 read back from int8 in 143 us (84 %; bf16 97 %).  A
// thread takes 8 values (bf16) or 16 (8 bits) of a row of keys and of the same row of
// values: 16-byte accesses on both sides but for the bf16 side of 8-bit rows, where it
// is two, and 64 bytes in flight a thread.
#include "pages_quant.cuh"

namespace dhs {
namespace {

constexpr int kPgThreads = 256;
constexpr int kPgTok = 32;  // tokens of a CTA at most (their places in shared memory)
struct TokenRows {
  unsigned char *k, *v;          // bf16
  int64_t kt, kh, vt, vh;        // strides of a token and a head, in elements
};

// Four codes times s as bf16, two a word.
template <int KIND>
__device__ __forceinline__ void dequantise(uint32_t c, float s, uint32_t &lo, uint32_t &hi) {
  float x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = (c >> (i * 8)) & 0xFFu;
    if (KIND == DHS_PAGE_INT8) {
      // 2^23 + (x + 128) as bits, less 2^23 + 128 (a conversion takes the slow pipe)
      x[i] = __fsub_rn(__uint_as_float(0x4B000000u | (b ^ 0x80u)), 8388736.f) * s;
    } else {
      // the code's seven lower bits at a float's exponent and mantissa give the
      // value times 2^-120, subnormals included
      const float m = __uint_as_float(((b & 0x7Fu) << 20) | ((b & 0x80u) << 24));
      x[i] = m * 1.329227995784916e36f * s;
    }
  }
  lo = pack_bf16(x[0], x[1]);
  hi = pack_bf16(x[2], x[3]);
}

template <int D, int KIND>
__global__ void __launch_bounds__(kPgThreads)
k_page_write(const PageView pg, const TokenRows src, int64_t n_tok, int per_cta,
             const int32_t *__restrict__ cu, const int32_t *__restrict__ lens,
             const int32_t *__restrict__ table, int width, int n_seqs, int32_t *err) {
  constexpr int E = KIND == DHS_PAGE_BF16 ? 8 : 16;  // values of a thread
  constexpr int L = D / E;                           // lanes of a row
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
    uint32_t u[2][E / 2];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const uint4 *at = reinterpret_cast<const uint4 *>(
          (side ? src.v : src.k) +
          2 * ((t0 + t) * (side ? src.vt : src.kt) + h * (side ? src.vh : src.kh) + sub * E));
#pragma unroll
      for (int x = 0; x < E / 8; ++x) {
        const uint4 w = on ? at[x] : make_uint4(0u, 0u, 0u, 0u);
        u[side][4 * x] = w.x;
        u[side][4 * x + 1] = w.y;
        u[side][4 * x + 2] = w.z;
        u[side][4 * x + 3] = w.w;
      }
    }
    const int64_t row = base + (int64_t)h * pg.rows;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      unsigned char *out = side ? pg.v : pg.k;
      if (KIND == DHS_PAGE_BF16) {
        if (on)
          *reinterpret_cast<uint4 *>(out + (row * D + sub * E) * 2) =
              make_uint4(u[side][0], u[side][1], u[side][2], u[side][3]);
        continue;
      }
      // the largest magnitude, of both halves of a word at a time: as bits an
      // infinity or a NaN is the largest
      uint32_t two = 0u;
#pragma unroll
      for (int i = 0; i < E / 2; ++i) two = __vmaxu2(two, u[side][i] & 0x7FFF7FFFu);
      uint32_t top = max(two & 0xFFFFu, two >> 16);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float big = __uint_as_float(top << 16);
      const bool bad = top >= 0x7F80u;
      const float s = (bad || big < kTiny) ? 0.f
                                           : __fdiv_rn(big, KIND == DHS_PAGE_INT8 ? 127.f : 448.f);
      uint32_t code[E / 4];
#pragma unroll
      for (int i = 0; i < E / 4; ++i) code[i] = 0u;
      if (s > 0.f) quantise<KIND, E>(u[side], big, s, code);
      if (on) {
        *reinterpret_cast<uint4 *>(out + row * D + sub * E) =
            make_uint4(code[0], code[1], code[E / 4 - 2], code[E / 4 - 1]);
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
  constexpr int E = KIND == DHS_PAGE_BF16 ? 8 : 16;
  constexpr int L = D / E;
  __shared__ int64_t src[kPgTok];
  const int64_t t0 = (int64_t)blockIdx.x * per_cta;
  const int nt = (int)min((int64_t)per_cta, n_tok - t0);
  if (threadIdx.x < nt)
    src[threadIdx.x] = place(pg, cu, lens, table, width, n_seqs, t0 + threadIdx.x, err,
                             DHS_SITE_PAGE_READ);
  __syncthreads();
  const int sub = threadIdx.x % L, total = nt * pg.hkv;
#pragma unroll 2
  for (int e = threadIdx.x / L; e < total; e += kPgThreads / L) {
    const int t = e / pg.hkv, h = e - t * pg.hkv;
    const int64_t base = src[t];
    if (base == -2) continue;
    const int64_t row = base + (int64_t)h * pg.rows;
    uint4 w[2];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      w[side] = make_uint4(0u, 0u, 0u, 0u);
      if (base >= 0) {
        w[side] = *reinterpret_cast<const uint4 *>((side ? pg.v : pg.k) +
                                                   (row * D + sub * E) * (16 / E));
        if (KIND != DHS_PAGE_BF16) s[side] = (side ? pg.vs : pg.ks)[row];
      }
    }
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      uint4 *at = reinterpret_cast<uint4 *>(
          (side ? to.v : to.k) +
          2 * ((t0 + t) * (side ? to.vt : to.kt) + h * (side ? to.vh : to.kh) + sub * E));
      if (KIND == DHS_PAGE_BF16) {
        *at = w[side];
      } else {
        uint4 a, b;
        dequantise<KIND>(w[side].x, s[side], a.x, a.y);
        dequantise<KIND>(w[side].y, s[side], a.z, a.w);
        dequantise<KIND>(w[side].z, s[side], b.x, b.y);
        dequantise<KIND>(w[side].w, s[side], b.z, b.w);
        at[0] = a;
        at[1] = b;
      }
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
  if (!page_view(pages, &pg) || n_tok < 0 || n_seqs < 0 || n_seqs > kMaxSeqs || width < 0)
    return DHS_ERR_INVALID;
  if (n_tok == 0 || n_seqs == 0) return DHS_OK;
  if (!k || !v || !cu || !lens || !table || width < 1 || ((uintptr_t)k & 15u) ||
      ((uintptr_t)v & 15u) || !words(cu, lens, table, err))
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
  }
  // rows that are written must not lie over one another (between keys and values of
  // different strides the caller sees to that)
  if (!write) {
    const int64_t off = (int64_t)((uintptr_t)v - (uintptr_t)k) / 2;
    const bool one = n_tok == 1, single = pg.hkv == 1;
    if (rows_meet(n_tok, pg.hkv, r.kt, r.kh, pg.d, 0, true) ||
        rows_meet(n_tok, pg.hkv, r.vt, r.vh, pg.d, 0, true) ||
        ((one || r.kt == r.vt) && (single || r.kh == r.vh) &&
         rows_meet(n_tok, pg.hkv, r.kt, r.kh, pg.d, off, false)))
      return DHS_ERR_INVALID;
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
