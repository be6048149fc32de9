// Norm and position rotation of every head of queries and keys in one pass, and the same
// with keys and values going on into the paged cache.
//
// For a head's row x of D dims: y = x / sqrt(mean(x^2) + eps) * w (or y = x), then for
// pair i < P of its dims (a, b) -> (a c - b s, b c + a s) with c, s = A cos, A sin of
// position * f_i.  Everything between the 16-bit input and the one rounding of the output
// is in 32 bits.
//
// The angle is kept in turns of 64-bit fixed point: position * (f_i / 2 pi) mod 1 is a
// product of whole numbers mod 2^64, exact up to 2^-65 turns of f_i times the position, and
// its upper 32 bits are the argument of a sine and cosine in half turns.  In 32-bit floats a
// position of 100,000 would leave some 2^-8 of an angle; a table of sines and cosines costs
// its own reads and a largest position.  A CTA works out the pairs of its tokens once, for
// all of their heads.
//
// HBM bounds it: each row is read once and written once, with nothing in between that
// another row needs.  What stands in the way is the work per value, so a row's 8 or 16 lanes
// keep their token: what they multiply by (sines, cosines and the norm's weights in one) is
// made once and stays in registers over the heads of a chunk.  A lane holds 8 values of a
// row: 4 and their 4 partners half a rotation away, or 4 pairs of neighbours, so that the
// rotation needs no exchange between lanes and the norm one reduction over the row.
// Measured (GB300, 6.77 TB/s copied), 128 dims, 32 query heads over 8: 25,638 tokens 89 us,
// 87 % of the bytes' time; 51,383 tokens on into pages as bf16 208 us (89 %), as e4m3 228 (75 %:
// 72 % of the issue slots); 64 tokens 4.8 us, of which the lookup of their places is three
// loads that wait for one another.  With sines worked out for every row of every head it was
// 199 and 432 us.
#include "pages_quant.cuh"
#include "tc_util.cuh"

namespace dhs {
namespace {

constexpr int kRoThreads = 256;
constexpr int kRoAhead = 4;  // rows of a lane under way at a time
constexpr int kNoPages = -1;

struct HeadRows {
  const unsigned char *x;
  unsigned char *out;        // nullptr: not wanted
  const float *norm;         // nullptr: none
  int64_t xt, xh, ot, oh;    // strides of a token and a head, in elements
  int heads;
};

struct RotateArgs {
  HeadRows q, k, v;
  const uint64_t *turns;
  const int32_t *positions, *cu, *lens, *table;
  int32_t *err;
  int64_t n_tok;
  float amplitude, eps;
  int pairs, halves, width, n_seqs;
  int chunk, qc, kc;  // heads of a chunk; chunks of queries and of keys
};

// Codes of eight values in 32 bits over the scale's reciprocal, rounded to nearest with
// ties to even.  (The values are off by some half-steps of 32 bits themselves, so no
// quotient is exact here; rows of the cache that come in 16 bits are quantised exactly.)
template <int KIND>
__device__ __forceinline__ void codes_of(const float (&y)[8], float by, uint32_t (&code)[2]) {
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    if (KIND == DHS_PAGE_INT8) {
      uint32_t b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(fmaf(y[4 * w + i], by, 12582912.f));
      code[w] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    } else {
      code[w] = __byte_perm(e4m3_pair_code(y[4 * w] * by, y[4 * w + 1] * by),
                            e4m3_pair_code(y[4 * w + 2] * by, y[4 * w + 3] * by), 0x5410);
    }
  }
}

// CTA (x, y): tokens x * TOK .., chunk y of the heads of queries, then keys, then values.
template <int D, int KIND, bool HALVES>
__global__ void __launch_bounds__(kRoThreads)
k_rotate(const PageView pg, const RotateArgs a) {
  constexpr int L = D / 8, TOK = kRoThreads / L, U = kRoAhead;  // lanes of a row, tokens
  __shared__ int64_t dst[TOK];
  __shared__ int at_pos[TOK];
  pdl_wait();
  const int sub = threadIdx.x % L, mine = threadIdx.x / L;
  const int64_t t0 = (int64_t)blockIdx.x * TOK, tok = t0 + mine;
  const bool there = tok < a.n_tok;
  const int c = blockIdx.y;
  const bool value = c >= a.qc + a.kc, key = !value && c >= a.qc;
  const HeadRows &r = value ? a.v : key ? a.k : a.q;
  const int h0 = (c - (value ? a.qc + a.kc : key ? a.qc : 0)) * a.chunk;
  const int h1 = min(h0 + a.chunk, r.heads);

  // where this lane's 8 values lie: two fours, of which a rotation by halves has pairs
  const int quads = value ? 0 : a.pairs / 4;
  const bool turned = sub < quads, split = HALVES && turned;
  const int e0 = !HALVES || value ? 8 * sub : split ? 4 * sub : 2 * a.pairs + 8 * (sub - quads);
  const int e1 = split ? a.pairs + 4 * sub : e0 + 4;

  const unsigned char *from = r.x + 2 * ((there ? tok : 0) * r.xt + h0 * r.xh);
  uint2 u[U][2];
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const bool on = there && h + i < h1;
      const unsigned char *at = from + (int64_t)(h - h0 + i) * r.xh * 2;
      u[i][0] = on ? *reinterpret_cast<const uint2 *>(at + 2 * e0) : make_uint2(0u, 0u);
      u[i][1] = on ? *reinterpret_cast<const uint2 *>(at + 2 * e1) : make_uint2(0u, 0u);
    }
  };
  load(h0);  // under way with the lookups

  if (KIND != kNoPages || a.pairs > 0) {
    if (threadIdx.x < TOK && t0 + threadIdx.x < a.n_tok) {
      int pos = 0;
      int64_t to = 0;
      if (KIND != kNoPages)
        to = place(pg, a.cu, a.lens, a.table, a.width, a.n_seqs, t0 + threadIdx.x, a.err,
                   DHS_SITE_PAGE_APPEND, &pos);
      dst[threadIdx.x] = to;
      at_pos[threadIdx.x] = a.positions ? a.positions[t0 + threadIdx.x] : pos;
    }
    __syncthreads();
  }
  const int64_t base = !there ? -2 : KIND == kNoPages ? 0 : dst[mine];
  const bool on = base >= 0;
  const bool raw = !r.norm && (value || a.pairs == 0);  // rows go as they come, bit by bit

  // out = y C + (its partners) S: the weights, and the rotation, of this lane's values
  uint64_t C[4], S[4];
  if (!raw) {
    float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}, cw[8], sw[8];
    if (r.norm) {
      *reinterpret_cast<float4 *>(w) = *reinterpret_cast<const float4 *>(r.norm + e0);
      *reinterpret_cast<float4 *>(w + 4) = *reinterpret_cast<const float4 *>(r.norm + e1);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cw[i] = w[i];
      sw[i] = 0.f;
    }
    if (turned && there) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t turn = a.turns[4 * sub + i] * (uint64_t)(int64_t)at_pos[mine];
        float sn, cs;
        sincospif((float)(int32_t)(uint32_t)(turn >> 32) * 4.656612873077393e-10f, &sn, &cs);  // 2^-31
        sn *= a.amplitude;
        cs *= a.amplitude;
        const int p = HALVES ? i : 2 * i, q = HALVES ? 4 + i : 2 * i + 1;
        cw[p] = w[p] * cs;
        sw[p] = -w[q] * sn;
        cw[q] = w[q] * cs;
        sw[q] = w[p] * sn;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      C[i] = pack_f32x2(cw[2 * i], cw[2 * i + 1]);
      S[i] = pack_f32x2(sw[2 * i], sw[2 * i + 1]);
    }
  }

  // one row: heads are of the whole CTA, so every lane takes part in the reductions
  auto finish = [&](int h, const uint2 (&x)[2]) {
    const uint32_t w[4] = {x[0].x, x[0].y, x[1].x, x[1].y};
    uint64_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      y[i] = pack_f32x2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    uint2 b0 = x[0], b1 = x[1];
    if (!raw) {
      if (r.norm) {
        auto squares = [&]() {
          uint64_t two = mul_f32x2(y[0], y[0]);
#pragma unroll
          for (int i = 1; i < 4; ++i) two = fma_f32x2(y[i], y[i], two);
          float ss, s1;
          unpack_f32x2(two, ss, s1);
          ss += s1;
#pragma unroll
          for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          return ss;
        };
        auto times = [&](float f) {
          const uint64_t two = pack_f32x2(f, f);
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = mul_f32x2(y[i], two);
        };
        float ss = squares(), eps = a.eps;
        // squares that leave the range of 32 bits (2^100 and more; below 2^-90 where eps does
        // not outweigh them): once more of the row times 2^-70 or 2^100
        const bool big = !(ss < 1.2676506e30f), small = ss < 8.077936e-28f && eps < 7.8886e-31f;
        if (__any_sync(0xffffffffu, big || small)) {
          const float g = big ? 8.470329472543003e-22f : small ? 1.2676506002282294e30f : 1.f;
          times(g);
          ss = squares();
          eps = eps * g * g;
        }
        times(rsqrtf(fmaf(ss, 1.f / D, eps)));
      }
      uint64_t z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i] = mul_f32x2(y[i], C[i]);
      if (turned) {
        if (HALVES) {
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = fma_f32x2(y[i ^ 2], S[i], z[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float p, q;
            unpack_f32x2(y[i], p, q);
            z[i] = fma_f32x2(pack_f32x2(q, p), S[i], z[i]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = z[i];
      float p[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) unpack_f32x2(y[i], p[2 * i], p[2 * i + 1]);
      b0 = make_uint2(pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]));
      b1 = make_uint2(pack_bf16(p[4], p[5]), pack_bf16(p[6], p[7]));
    }
    const bool live = on && h < h1;
    if (live && r.out) {
      unsigned char *at = r.out + 2 * (tok * r.ot + h * r.oh);
      *reinterpret_cast<uint2 *>(at + 2 * e0) = b0;
      *reinterpret_cast<uint2 *>(at + 2 * e1) = b1;
    }
    if (KIND == kNoPages || !(key || value)) return;
    const int64_t row = base + (int64_t)h * pg.rows;
    unsigned char *out = value ? pg.v : pg.k;
    if (KIND == DHS_PAGE_BF16) {
      if (live) {
        *reinterpret_cast<uint2 *>(out + (row * D + e0) * 2) = b0;
        *reinterpret_cast<uint2 *>(out + (row * D + e1) * 2) = b1;
      }
      return;
    }
    float p[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack_f32x2(y[i], p[2 * i], p[2 * i + 1]);
    uint32_t top = 0u;  // (as bits an infinity or a NaN is the largest)
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(p[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float big = __uint_as_float(top);
    const bool bad = top >= 0x7F800000u;
    const float s = (bad || big < kTiny) ? 0.f
                                         : __fdiv_rn(big, KIND == DHS_PAGE_INT8 ? 127.f : 448.f);
    uint32_t code[2] = {0u, 0u};
    if (s > 0.f) {
      if (raw) quantise<KIND, 8>(w, big, s, code);
      else codes_of<KIND>(p, __frcp_rn(s), code);
    }
    if (live) {
      *reinterpret_cast<uint32_t *>(out + row * D + e0) = code[0];
      *reinterpret_cast<uint32_t *>(out + row * D + e1) = code[1];
      if (sub == 0) (value ? pg.vs : pg.ks)[row] = bad ? __uint_as_float(0x7FC00000u) : s;
    }
  };
  for (int h = h0; h < h1; h += U) {
    if (h > h0) load(h);
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (h + i < h1) finish(h + i, u[i]);
  }
}

// Strides that an address may be made of.
bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0 && s <= ((int64_t)1 << 40); }

// The rows of a caller's heads, or false where they are refused: rows of the output that
// share elements, or that share some with the input but are not the input itself (of the
// same strides; of others the caller sees to that).
bool head_rows(const dhs_heads *h, int64_t n_tok, int d, bool out_wanted, HeadRows *r) {
  if (!h->x || (out_wanted && !h->out) || h->heads < 1 || h->heads > 128 * kPageMaxHeads ||
      ((uintptr_t)h->x & 15u) || ((uintptr_t)h->out & 15u) || ((uintptr_t)h->norm & 15u) ||
      !stride_ok(h->x_token) || !stride_ok(h->x_head) || !stride_ok(h->out_token) ||
      !stride_ok(h->out_head))
    return false;
  if (h->out) {
    if (rows_meet(n_tok, h->heads, h->out_token, h->out_head, d, 0, true)) return false;
    const bool alike = (n_tok == 1 || h->x_token == h->out_token) &&
                       (h->heads == 1 || h->x_head == h->out_head);
    const int64_t off = (int64_t)((uintptr_t)h->out - (uintptr_t)h->x) / 2;
    if (h->out == h->x ? !alike
                       : alike && rows_meet(n_tok, h->heads, h->out_token, h->out_head, d, off, false))
      return false;
  }
  r->x = static_cast<const unsigned char *>(h->x);
  r->out = static_cast<unsigned char *>(h->out);
  r->norm = h->norm;
  r->xt = h->x_token;
  r->xh = h->x_head;
  r->ot = h->out_token;
  r->oh = h->out_head;
  r->heads = h->heads;
  return true;
}

bool rotation_ok(const dhs_rotation *rot, int d, RotateArgs *a) {
  a->turns = nullptr;
  a->pairs = a->halves = 0;
  a->amplitude = 1.f;
  if (!rot) return true;
  if (!rot->turns || ((uintptr_t)rot->turns & 7u) || rot->n_pairs < 4 || rot->n_pairs % 4 ||
      rot->n_pairs > d / 2 || rot->pairing < DHS_ROTATE_HALVES ||
      rot->pairing > DHS_ROTATE_NEIGHBOURS || !(rot->amplitude > 0.f) || rot->amplitude > 1e38f)
    return false;
  a->turns = rot->turns;
  a->pairs = rot->n_pairs;
  a->halves = rot->pairing == DHS_ROTATE_HALVES;
  a->amplitude = rot->amplitude;
  return true;
}

int launch(const PageView &pg, RotateArgs &a, int d, int kind, dhs_stream stream) {
  // Chunks as long as the GPU stays full (their sines, cosines and lookups are made once),
  // one row each where tokens are few: 8 CTAs' lanes a row on each of 152 SMs.
  const int64_t heads = (int64_t)a.q.heads + a.k.heads + a.v.heads;
  const int64_t fill = a.n_tok * heads / (152 * 8 * (kRoThreads / (d / 8)));
  a.chunk = (int)std::max<int64_t>(std::min<int64_t>(std::max<int64_t>(fill, 1), 32),
                                   (heads + 59999) / 60000);
  auto chunks = [&](int n) { return (n + a.chunk - 1) / a.chunk; };
  a.qc = chunks(a.q.heads);
  a.kc = chunks(a.k.heads);
  const int tok = kRoThreads / (d / 8);
  const dim3 grid((unsigned)((a.n_tok + tok - 1) / tok),
                  (unsigned)(a.qc + a.kc + chunks(a.v.heads)));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto go = [&](auto dim, auto k) {
    constexpr int D = decltype(dim)::value, K = decltype(k)::value;
    return a.halves ? launch_pdl(k_rotate<D, K, true>, grid, dim3(kRoThreads), 0, s, pg, a)
                    : launch_pdl(k_rotate<D, K, false>, grid, dim3(kRoThreads), 0, s, pg, a);
  };
  auto kinds = [&](auto dim) {
    switch (kind) {
      case DHS_PAGE_BF16: return go(dim, std::integral_constant<int, DHS_PAGE_BF16>());
      case DHS_PAGE_INT8: return go(dim, std::integral_constant<int, DHS_PAGE_INT8>());
      case DHS_PAGE_E4M3: return go(dim, std::integral_constant<int, DHS_PAGE_E4M3>());
      default: return go(dim, std::integral_constant<int, kNoPages>());
    }
  };
  const cudaError_t e = d == 128 ? kinds(std::integral_constant<int, 128>())
                                 : kinds(std::integral_constant<int, 64>());
  if (e != cudaSuccess) {
    cudaGetLastError();
    return DHS_ERR_CUDA;
  }
  return DHS_OK;
}

}  // namespace
}  // namespace dhs

extern "C" int dhs_rotate(const dhs_rotation *rot, const dhs_heads *q, const dhs_heads *k, float eps,
                          int32_t head_dim, int64_t n_tokens, const int32_t *positions,
                          dhs_stream stream) {
  using namespace dhs;
  RotateArgs a = {};
  if ((head_dim != 64 && head_dim != 128) || n_tokens < 0 || !(eps >= 0.f) || eps > 1e38f ||
      !rotation_ok(rot, head_dim, &a) || (!q && !k))
    return DHS_ERR_INVALID;
  if (n_tokens == 0) return DHS_OK;
  if (n_tokens > INT32_MAX) return DHS_ERR_CAPACITY;
  if ((rot && !positions) || !words(positions) ||
      (q && !head_rows(q, n_tokens, head_dim, true, &a.q)) ||
      (k && !head_rows(k, n_tokens, head_dim, true, &a.k)))
    return DHS_ERR_INVALID;
  a.positions = positions;
  a.n_tok = n_tokens;
  a.eps = eps;
  return launch(PageView{}, a, head_dim, kNoPages, stream);
}

extern "C" int dhs_page_append(const dhs_pages *pages, const dhs_rotation *rot, const dhs_heads *q,
                               const dhs_heads *k, const void *v, const int64_t *v_strides, float eps,
                               int64_t n_tokens, const int32_t *positions, const int32_t *cu,
                               const int32_t *seq_lens, const int32_t *page_table,
                               int32_t table_width, int32_t n_seqs, int32_t *err, dhs_stream stream) {
  using namespace dhs;
  PageView pg;
  RotateArgs a = {};
  if (!page_view(pages, &pg) || n_tokens < 0 || n_seqs < 0 || n_seqs > kMaxSeqs || table_width < 0 ||
      !(eps >= 0.f) || eps > 1e38f || !rotation_ok(rot, pg.d, &a))
    return DHS_ERR_INVALID;
  if (n_tokens == 0 || n_seqs == 0) return DHS_OK;
  if (n_tokens > INT32_MAX) return DHS_ERR_CAPACITY;
  if (!k || !v || ((uintptr_t)v & 15u) || !cu || !seq_lens || !page_table || table_width < 1 ||
      !words(positions, cu, seq_lens, page_table, err) || k->heads != pg.hkv ||
      !head_rows(k, n_tokens, pg.d, false, &a.k) ||
      (q && !head_rows(q, n_tokens, pg.d, true, &a.q)))
    return DHS_ERR_INVALID;
  a.v.x = static_cast<const unsigned char *>(v);
  a.v.xt = (int64_t)pg.hkv * pg.d;
  a.v.xh = pg.d;
  a.v.heads = pg.hkv;
  if (v_strides) {
    if (!stride_ok(v_strides[0]) || !stride_ok(v_strides[1])) return DHS_ERR_INVALID;
    a.v.xt = v_strides[0];
    a.v.xh = v_strides[1];
  }
  a.positions = positions;
  a.cu = cu;
  a.lens = seq_lens;
  a.table = page_table;
  a.err = err;
  a.n_tok = n_tokens;
  a.eps = eps;
  a.width = table_width;
  a.n_seqs = n_seqs;
  return launch(pg, a, pg.d, pg.kind, stream);
}
