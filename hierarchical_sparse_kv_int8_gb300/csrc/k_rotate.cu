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
// another row needs.  A lane holds 8 values of a row: 4 and their 4 partners half a rotation
// away, or 4 pairs of neighbours, so that the rotation needs no exchange between lanes and
// the norm one reduction over the row's 8 or 16 lanes.  A warp's rows are all of one of
// queries, keys and values.
#include "pages_quant.cuh"

namespace dhs {
namespace {

constexpr int kRoThreads = 256;
constexpr int kRoTok = 16;   // tokens of a CTA at most
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
  int pairs, halves, per_cta, width, n_seqs;
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

template <int D, int KIND>
__global__ void __launch_bounds__(kRoThreads)
k_rotate(const PageView pg, const RotateArgs a) {
  constexpr int L = D / 8, RW = 32 / L, ROWS = kRoThreads / L;  // lanes of a row, rows of a warp, CTA
  __shared__ int64_t dst[kRoTok];
  __shared__ int at_pos[kRoTok];
  __shared__ __align__(16) float sh_cos[kRoTok][D / 2], sh_sin[kRoTok][D / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % L;
  const int64_t t0 = (int64_t)blockIdx.x * a.per_cta;
  const int nt = (int)min((int64_t)a.per_cta, a.n_tok - t0);

  // slots of rows: queries, keys, values, each rounded up to whole warps
  auto whole = [](int n) { return (n + RW - 1) / RW * RW; };
  const int nq = nt * a.q.heads, nk = nt * a.k.heads, nv = nt * a.v.heads;
  const int k0 = whole(nq), v0 = k0 + whole(nk), total = v0 + whole(nv);
  const int step = ROWS * gridDim.y;

  // where this lane's 8 values lie, without and with a rotation by halves
  const int quads = a.pairs / 4;
  const bool split = a.halves && sub < quads;
  const int e0 = !a.halves ? 8 * sub : split ? 4 * sub : 2 * a.pairs + 8 * (sub - quads);
  const int e1 = split ? a.pairs + 4 * sub : e0 + 4;

  // the row of a slot: its token and head
  auto row_of = [&](int slot, int &t, int &h) -> const HeadRows & {
    const HeadRows &r = slot < k0 ? a.q : slot < v0 ? a.k : a.v;
    const int x = slot - (slot < k0 ? 0 : slot < v0 ? k0 : v0) + lane / L;
    t = (int)((uint32_t)x / (uint32_t)r.heads);
    h = x - t * r.heads;
    return r;
  };
  auto load = [&](int slot, uint2 (&u)[2]) {
    u[0] = u[1] = make_uint2(0u, 0u);
    if (slot >= total) return;
    int t, h;
    const HeadRows &r = row_of(slot, t, h);
    if (t >= nt) return;
    const unsigned char *at = r.x + 2 * ((t0 + t) * r.xt + h * r.xh);
    const bool value = slot >= v0;
    u[0] = *reinterpret_cast<const uint2 *>(at + 2 * (value ? 8 * sub : e0));
    u[1] = *reinterpret_cast<const uint2 *>(at + 2 * (value ? 8 * sub + 4 : e1));
  };

  int slot = (int)blockIdx.y * ROWS + warp * RW;
  uint2 u[2];
  load(slot, u);  // under way with the lookups

  if (threadIdx.x < nt) {
    int pos = 0;
    int64_t to = 0;
    if (KIND != kNoPages)
      to = place(pg, a.cu, a.lens, a.table, a.width, a.n_seqs, t0 + threadIdx.x, a.err,
                 DHS_SITE_PAGE_APPEND, &pos);
    dst[threadIdx.x] = to;
    at_pos[threadIdx.x] = a.positions ? a.positions[t0 + threadIdx.x] : pos;
  }
  if (a.pairs > 0) {
    __syncthreads();
    for (int e = threadIdx.x; e < nt * a.pairs; e += kRoThreads) {
      const int t = e / a.pairs, i = e - t * a.pairs;
      const uint64_t turn = a.turns[i] * (uint64_t)(int64_t)at_pos[t];
      float s, c;
      sincospif((float)(int32_t)(uint32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31
      sh_cos[t][i] = c * a.amplitude;
      sh_sin[t][i] = s * a.amplitude;
    }
  }
  __syncthreads();

  for (; slot < total; slot += step) {
    uint2 next[2];
    load(slot + step, next);
    int t, h;
    const HeadRows &r = row_of(slot, t, h);
    const int64_t base = t < nt ? dst[t] : -2;
    const bool on = t < nt && base >= 0;
    const bool key = slot >= k0 && slot < v0, value = slot >= v0;  // (of the whole warp)
    const uint32_t w[4] = {u[0].x, u[0].y, u[1].x, u[1].y};
    const bool raw = !r.norm && (value || a.pairs == 0);  // the row goes as it came, bit by bit
    float y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = __uint_as_float(w[i] << 16);
      y[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    if (!value) {
      if (r.norm) {
        auto squares = [&](float g) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float z = y[i] * g;
            ss = fmaf(z, z, ss);
          }
#pragma unroll
          for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          return ss;
        };
        const float ss = squares(1.f);
        float f = rsqrtf(fmaf(ss, 1.f / D, a.eps));
        // squares that leave the range of 32 bits (2^100 and more; below 2^-90 where eps does
        // not outweigh them): once more of the row times 2^-70 or 2^100
        const bool big = !(ss < 1.2676506e30f), small = ss < 8.077936e-28f && a.eps < 7.8886e-31f;
        if (__any_sync(0xffffffffu, big || small)) {
          const float g = big ? 8.470329472543003e-22f : small ? 1.2676506002282294e30f : 1.f;
          f = rsqrtf(fmaf(squares(g), 1.f / D, a.eps * g * g)) * g;
        }
        const float4 g0 = *reinterpret_cast<const float4 *>(r.norm + e0);
        const float4 g1 = *reinterpret_cast<const float4 *>(r.norm + e1);
        y[0] *= f * g0.x;
        y[1] *= f * g0.y;
        y[2] *= f * g0.z;
        y[3] *= f * g0.w;
        y[4] *= f * g1.x;
        y[5] *= f * g1.y;
        y[6] *= f * g1.z;
        y[7] *= f * g1.w;
      }
      if (sub < quads && t < nt) {
        const float4 c4 = *reinterpret_cast<const float4 *>(&sh_cos[t][4 * sub]);
        const float4 s4 = *reinterpret_cast<const float4 *>(&sh_sin[t][4 * sub]);
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float &p = a.halves ? y[i] : y[2 * i], &q = a.halves ? y[4 + i] : y[2 * i + 1];
          const float x = p;
          p = x * c[i] - q * s[i];
          q = q * c[i] + x * s[i];
        }
      }
    }
    const uint2 b0 = raw ? u[0] : make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
    const uint2 b1 = raw ? u[1] : make_uint2(pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
    if (!value) {
      if (on && r.out) {
        unsigned char *at = r.out + 2 * ((t0 + t) * r.ot + h * r.oh);
        *reinterpret_cast<uint2 *>(at + 2 * e0) = b0;
        *reinterpret_cast<uint2 *>(at + 2 * e1) = b1;
      }
    }
    if (KIND != kNoPages && (key || value)) {
      const int64_t row = base + (int64_t)h * pg.rows;
      unsigned char *out = value ? pg.v : pg.k;
      const int f0 = value ? 8 * sub : e0, f1 = value ? f0 + 4 : e1;
      if (KIND == DHS_PAGE_BF16) {
        if (on) {
          *reinterpret_cast<uint2 *>(out + (row * D + f0) * 2) = b0;
          *reinterpret_cast<uint2 *>(out + (row * D + f1) * 2) = b1;
        }
      } else {
        uint32_t top = 0u;  // (as bits an infinity or a NaN is the largest)
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(y[i]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float big = __uint_as_float(top);
        const bool bad = top >= 0x7F800000u;
        const float s = (bad || big < kTiny) ? 0.f
                                             : __fdiv_rn(big, KIND == DHS_PAGE_INT8 ? 127.f : 448.f);
        uint32_t code[2] = {0u, 0u};
        if (s > 0.f) {
          if (raw) quantise<KIND, 8>(w, big, s, code);
          else codes_of<KIND>(y, __frcp_rn(s), code);
        }
        if (on) {
          *reinterpret_cast<uint32_t *>(out + row * D + f0) = code[0];
          *reinterpret_cast<uint32_t *>(out + row * D + f1) = code[1];
          if (sub == 0) (value ? pg.vs : pg.ks)[row] = bad ? __uint_as_float(0x7FC00000u) : s;
        }
      }
    }
    u[0] = next[0];
    u[1] = next[1];
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
  // enough CTAs to fill the GPU first (heads over several where tokens are few), then more
  // tokens of a CTA, which share its sines and cosines
  const int rows_cta = kRoThreads / (d / 8);
  int64_t per = a.n_tok / (8 * 152);
  a.per_cta = (int)(per < 1 ? 1 : (per > kRoTok ? kRoTok : per));
  const int64_t grid = (a.n_tok + a.per_cta - 1) / a.per_cta;
  const int64_t rows = (int64_t)a.per_cta * (a.q.heads + a.k.heads + a.v.heads);
  const int64_t split = std::max<int64_t>(
      1, std::min((rows + rows_cta - 1) / rows_cta, (4 * 152 + grid - 1) / grid));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto go = [&](auto kern) {
    return launch_prio(kern, dim3((unsigned)grid, (unsigned)split), dim3(kRoThreads), 0, s, pg, a);
  };
  cudaError_t e;
  switch ((d == 128 ? 4 : 0) + kind) {
    case -1: e = go(k_rotate<64, kNoPages>); break;
    case 0: e = go(k_rotate<64, DHS_PAGE_BF16>); break;
    case 1: e = go(k_rotate<64, DHS_PAGE_INT8>); break;
    case 2: e = go(k_rotate<64, DHS_PAGE_E4M3>); break;
    case 3: e = go(k_rotate<128, kNoPages>); break;
    case 4: e = go(k_rotate<128, DHS_PAGE_BF16>); break;
    case 5: e = go(k_rotate<128, DHS_PAGE_INT8>); break;
    default: e = go(k_rotate<128, DHS_PAGE_E4M3>); break;
  }
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
