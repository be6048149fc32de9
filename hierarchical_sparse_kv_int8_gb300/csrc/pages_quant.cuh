// Rows on their way into the paged cache: where a packed token lives, and the codes and
// scale of a row in the 8-bit kinds.
//
// Rounding exactly costs a comparison per row, not per value.  With s = max / Q
// rounded to 24 bits, x / s is either at least 2^-13 (e4m3) or 2^-16 (int8) of itself
// away from the middle of two codes, or max / Q and x would meet the middle
// exactly: x Q = middle max is an equation of small whole numbers.  Which side x / s
// falls on there follows from s being rounded down or up, the sign of max - Q s.  So x
// is multiplied by 1 / s times 1 +- 2^-15 (2^-18) by that sign, which moves only those
// values to their side.  Where s is exact (sign 0) a middle is a true tie: for int8 s is
// then a power of two and x / s exact; for e4m3 x / s is rounded to 17 bits first, which
// puts it on the middle again, and the conversion takes the even code.  (With every
// value's side decided by itself the write of 37,000 tokens took 113 us and 40
// instructions a value.)
#pragma once
#include "pages_internal.cuh"

#include <algorithm>

namespace dhs {

constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100

__device__ __forceinline__ uint32_t e4m3_pair_code(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// y rounded to 17 bits (the intrinsics keep the product and differences apart)
__device__ __forceinline__ float bits17(float y) {
  const float t = __fmul_rn(y, 129.f);
  return __fsub_rn(t, __fsub_rn(t, y));
}

// Codes of N bf16 values (two a word) of a row with the largest magnitude `big`
// and scale s, four codes a word.
template <int KIND, int N>
__device__ __forceinline__ void quantise(const uint32_t (&u)[N / 2], float big, float s,
                                         uint32_t (&code)[N / 4]) {
  const float off = fmaf(KIND == DHS_PAGE_INT8 ? -127.f : -448.f, s, big);  // (its sign is exact)
  const float move = KIND == DHS_PAGE_INT8 ? 3.814697265625e-6f : 3.0517578125e-5f;
  const float by = __frcp_rn(s) * (off > 0.f ? 1.f + move : off < 0.f ? 1.f - move : 1.f);
#pragma unroll
  for (int w = 0; w < N / 4; ++w) {
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = u[w * 2 + (i >> 1)];
      x[i] = __uint_as_float(i & 1 ? b & 0xFFFF0000u : b << 16);
    }
    if (KIND == DHS_PAGE_INT8) {
      // 1.5 * 2^23 more leaves the nearest whole number, ties to even, in the low bits
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = fmaf(x[i], by, 12582912.f);
      code[w] = __byte_perm(
          __byte_perm(__float_as_uint(x[0]), __float_as_uint(x[1]), 0x0040),
          __byte_perm(__float_as_uint(x[2]), __float_as_uint(x[3]), 0x0040), 0x5410);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = bits17(x[i] * by);
      code[w] = __byte_perm(e4m3_pair_code(x[0], x[1]), e4m3_pair_code(x[2], x[3]), 0x5410);
    }
  }
}

// Where packed token `tok` lives: row of kv head 0, -1 none (recorded), -2 padding; and its
// position.
__device__ __forceinline__ int64_t place(const PageView &pg, const int32_t *cu,
                                         const int32_t *lens, const int32_t *table, int width,
                                         int n_seqs, int64_t tok, int32_t *err, int site,
                                         int *position = nullptr) {
  const int i = seq_of(cu, n_seqs, tok);
  if (i < 0) return -2;
  const int64_t pos = (int64_t)lens[i] - ((int64_t)cu[i + 1] - tok);
  if (pos < 0 || pos >= (int64_t)width * pg.rows || pos > INT32_MAX) {
    page_error(err, DC_ROW_RANGE, site);
    return -1;
  }
  if (position) *position = (int)pos;
  return page_row(pg, table + (int64_t)i * width, (int)pos, err, site);
}

// Whether a row of d elements at i st + j sh and one at off + i' st + j' sh share an
// element, for any 0 <= i, i' < n and 0 <= j, j' < h; with off = 0 (the rows themselves)
// a row and itself do not count.  For every difference of heads the nearest difference
// of tokens on either side decides.
inline bool rows_meet(int64_t n, int64_t h, int64_t st, int64_t sh, int64_t d, int64_t off, bool same) {
  if (same && (h == 1 || sh >= d) && (n == 1 || st >= (h - 1) * sh + d)) return false;
  const __int128 extent = (__int128)(n - 1) * st + (__int128)(h - 1) * sh + d;
  if (!same && (off >= extent || off <= -extent)) return false;
  for (int64_t dj = same ? 0 : 1 - h; dj < h; ++dj) {
    const int64_t want = -(off + dj * sh);  // what di st has to miss by d
    const int64_t lo = st > 0 ? want / st - (want % st < 0) : 0;
    for (int64_t di = lo; di <= lo + 1; ++di) {
      int64_t x = std::max(1 - n, std::min(n - 1, di));
      if (same && dj == 0 && x == 0) {
        if (n == 1) continue;
        x = 1;
      }
      const int64_t miss = x * st - want;
      if (miss < d && miss > -d) return true;
    }
  }
  return false;
}

}  // namespace dhs
