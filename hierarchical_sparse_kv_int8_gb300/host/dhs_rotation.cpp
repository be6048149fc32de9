// Angular frequencies of a position rotation as turns per position in 64-bit fixed point.
//
// turns = round(f / 2 pi * 2^64) mod 2^64.  f is m 2^e with a whole m below 2^53; with
// 1 / 2 pi to 130 bits after the point (128 that are not zero) the product is a whole number
// of 181 bits, exact but for m times the constant's half of a last bit: less than 2^-13 of
// a unit of the result for every |f| below 2^32.  So a position p below 2^31 turns by less
// than 2^-33 of a turn more or less than it should.
#include "../../include/dhs.h"

#include <cmath>

extern "C" int dhs_rotation_turns(const double *freqs, int32_t n, uint64_t *turns) {
  if (n < 0 || (n > 0 && (!freqs || !turns))) return DHS_ERR_INVALID;
  for (int32_t i = 0; i < n; ++i)
    if (!(std::fabs(freqs[i]) < 4294967296.0)) return DHS_ERR_INVALID;
  // 2^130 / 2 pi, rounded
  constexpr uint64_t hi = 0xa2f9836e4e441529u, lo = 0xfc2757d1f534ddc1u;
  for (int32_t i = 0; i < n; ++i) {
    int e = 0;
    const double f = std::frexp(std::fabs(freqs[i]), &e);       // in [1/2, 1)
    const uint64_t m = (uint64_t)std::ldexp(f, 53);             // f = m 2^(e - 53)
    // w[2] 2^128 + w[1] 2^64 + w[0] = m 2^130 / 2 pi
    const unsigned __int128 low = (unsigned __int128)m * lo;
    const unsigned __int128 high = (unsigned __int128)m * hi + (uint64_t)(low >> 64);
    const uint64_t w[3] = {(uint64_t)low, (uint64_t)high, (uint64_t)(high >> 64)};
    const int shift = 66 + 53 - e;  // bits below a unit of the result; 87 at least
    auto bit_on = [&](int at) -> uint64_t {  // the 64 bits from bit `at` on
      const int k = at / 64, s = at % 64;
      if (k > 2) return 0;
      const uint64_t next = k < 2 ? w[k + 1] : 0;
      return s ? (w[k] >> s) | (next << (64 - s)) : w[k];
    };
    uint64_t t = bit_on(shift);
    t += bit_on(shift - 1) & 1u;    // the nearest whole number
    turns[i] = std::signbit(freqs[i]) ? (uint64_t)0 - t : t;
  }
  return DHS_OK;
}
