// Attention of the newest tokens of every sequence over its paged cache.
//
// For sequence i and kv head h the R = q_len x G (query, head) pairs, G = q_heads
// / kv_heads, are the rows of one small matrix; S = Q K^T and O = P V run on
// mma.sync m16n8k16 tiles of 16 rows (R is 1 to 128, and what bounds the work is
// the cache's bytes: 16 rows take 4 cycles of tensor core per cached token and
// head against 22 cycles of HBM for its 512 bytes in bf16, 11 in 8 bits).
// The softmax is online in log2 units: with the running maximum m of a row,
//   l = sum 2^(x - m),  O = sum 2^(x - m) v,
// and O and l are rescaled only when m grows by more than 4 (8 bits) or 8 (bf16),
// so weights stay below 2^4 or 2^8.
//
// Work split: the positions of every (sequence, kv head) item are cut into
// blocks, all items' blocks are laid end to end, and CTA b of n takes blocks
// [b T / n, (b + 1) T / n) of the T.  Every CTA so reads the same number of rows
// whatever the lengths are, and an item lies in as many CTAs as its length asks
// for.  An item inside one CTA is finished there; otherwise each CTA leaves (m,
// l, O) of its part in the workspace and a second launch joins the parts in CTA
// order, so bits repeat.  The lengths are read on the device: every CTA adds up
// the block counts itself.
//
// Inside a CTA four warps form WT token groups of WM warps.  A group streams
// tiles of TN positions through a ring of NS stages of shared memory with
// 16-byte cp.async (a row's page is looked up two tiles before its copy is
// waited for, so neither latency is exposed); its warps share the tile, each
// with its own 16 MT rows of Q and O in registers.  Groups need no barrier but
// their own until the item's end, where they are merged through shared memory.
//
// 8-bit rows: the codes become f16 in registers, exactly.  A row of Q is scaled
// by a power of two to fit f16 (exact down to 2^-32 of its largest element, and
// off by 2^-40 of it below), a key's scale multiplies its column of scores.  A
// value's scale multiplies its column of weights over a common power of two, which
// follows the largest scale read so far: f16 then holds a weight times scale to 2^-11,
// or to 2^-31 of the largest weight times the largest scale that the row sees (2^-27
// next to a scale of up to 2^4 times that which the row does not see; the values of
// larger ones are added when the warps' parts are merged).  (Codes to bf16 instead,
// with scaled bf16 weights, took 4 instructions a pair on the half-rate integer
// pipe instead of 1.5 to 2, and bound the kernel.)
// The fragments are read so that no transposition is needed: a thread's 16
// bytes of a key are 16 consecutive dims, which Q's fragments are loaded to
// match, and of a value 16 (8) consecutive output columns of two positions,
// paired by byte permutes.
//
// Positions that a query does not see have weight 0.  0 times an infinity or a
// NaN is not 0, so among the last q_len - 1 positions, the only ones that some
// queries of a sequence see and others do not, values that are not finite are
// set to 0 in shared memory and added afterwards to the queries that see them.
//
// Measured, 32 sequences of 65536 positions, 128 dims, one kv head, in us (and % of the
// measured copy bandwidth): bf16 8 rows 167 (95), 32 rows 173 (91), 64 rows 225 (70),
// 128 rows 510; int8 8 rows 99 (82), 32 rows 178, 64 rows 316, 128 rows 801.  Up to 32
// rows of bf16 the bytes bound it, in 8 bits the conversion to f16 does, and with more
// rows the mma.sync products and the registers that 128 rows leave for nothing else.  One
// sequence of 4096: 9.0 us, of which the join takes 4 to 5 and the way from the lengths
// through the page table to the first rows most of the rest.
#include "pages_internal.cuh"
#include "tc_util.cuh"

#include <math_constants.h>

#include <algorithm>
#include <atomic>

namespace dhs {
namespace {

constexpr int kPaWarps = 4;
constexpr int kPaThreads = kPaWarps * 32;
constexpr float kRescale8 = 4.f, kRescale16 = 8.f;  // 8-bit caches, bf16
// f16 weights: value scales over 2^vref are in [2^6, 2^7) when vref is set and may
// grow to 2^11 before it is set anew, so that a weight is at most 2^15
constexpr int kVrefUp = 6, kVrefMax = 11;

// ------------------------------------------------------------ 8-bit to f16 pairs
// int8: with its sign bit flipped x is u = x + 128, and 0x6400 | u is 1024 + u in
// f16; 1152 less is x, exactly.  e4m3: the conversion instruction, exact too.
__device__ __forceinline__ uint32_t sub_1152(uint32_t t) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(t), "r"(0x64806480u));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_f16(uint32_t two) {
  uint32_t r;
  asm("{\n .reg .b16 h;\n cvt.u16.u32 h, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}\n" : "=r"(r) : "r"(two));
  return r;
}
// the four codes of w as two pairs
template <int KIND>
__device__ __forceinline__ void f16_pairs(uint32_t w, uint32_t &lo, uint32_t &hi) {
  if (KIND == DHS_PAGE_INT8) {
    w ^= 0x80808080u;
    lo = sub_1152(__byte_perm(w, 0x64646464u, 0x4140));
    hi = sub_1152(__byte_perm(w, 0x64646464u, 0x4342));
  } else {
    lo = e4m3_f16(w & 0xFFFFu);
    hi = e4m3_f16(w >> 16);
  }
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <int KIND>
__device__ __forceinline__ void mma_kind(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (KIND == DHS_PAGE_BF16) mma_bf16_16816(d, a, b0, b1);
  else mma_f16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
}

__device__ __forceinline__ void cp_async_4_zfill(void *dst, const void *src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(smem_u32(dst)), "l"(src),
               "r"(bytes));
}

template <int D_, int KIND_, int WM_, int MT_, int NH_, bool SOME_ = KIND_ != DHS_PAGE_BF16>
struct Cfg {
  static constexpr int D = D_, KIND = KIND_, WM = WM_, MT = MT_;
  static constexpr int NH = NH_;                         // 8-row halves of a row tile in use
  static constexpr bool SOME = SOME_;  // value scales that only some rows see are looked for
  static constexpr int WT = kPaWarps / WM;
  static constexpr int W = KIND == DHS_PAGE_BF16 ? 2 : 1;
  static constexpr int RB = D * W;                       // bytes of a row
  static constexpr int CH = RB / 16;                     // 16-byte chunks of a row
  // 8-bit tiles that four warps read are turned into f16 in shared memory once (32 x
  // 64K int8, 128 rows: 916 -> 875 us when it came in; 2 warps: 185 -> 225, so not there)
  static constexpr bool CONV = W == 1 && WM > 2;
  // positions of a group's tile: 8 KB of keys and values per warp of the group
  static constexpr int TN0 = 8192 * WM / (2 * RB);
  static constexpr int TN = TN0 > 64 ? 64 : TN0;
  static constexpr int SUB = MT == 1 && TN >= 32 ? 32 : 16;  // positions scored at a time
  static constexpr int KV = TN * RB;
  static constexpr int STAGE = 2 * KV + (W == 1 ? 2 * TN * 4 : 0);  // keys, values, scales
  static constexpr int NS = 3;
  static constexpr int RING = NS * STAGE;
  static constexpr int RC = CONV ? 2 * D : RB;           // bytes of a row as it is read
  static constexpr int GROUP = RING + (CONV ? 2 * TN * RC : 0);
  static constexpr int ROWS = WM * MT * 16;              // rows of Q that fit
  static constexpr int OPAD = D + 4;
  static constexpr int MERGE = WT * ROWS * OPAD * 4;
  static constexpr int DATA = WT * GROUP > MERGE ? WT * GROUP : MERGE;
  static constexpr int SLOTS = NS + 1;
  static constexpr int OFF_ROW = DATA;                           // int64 [WT][SLOTS][TN]
  static constexpr int OFF_MASK = OFF_ROW + WT * SLOTS * TN * 8; // uint32 [WT][SLOTS][2]
  static constexpr int OFF_ML = OFF_MASK + WT * SLOTS * 8;       // float [WT][ROWS][2]
  static constexpr int OFF_TAB = OFF_ML + WT * ROWS * 8;         // int2 [ROWS]
  static constexpr int OFF_LATE = OFF_TAB + ROWS * 8;            // float [ROWS][kMaxKmax]
  static constexpr int SMEM = OFF_LATE + (SOME ? ROWS * kMaxKmax * 4 : 0);
  static constexpr int OCC = SMEM * 2 <= 226 * 1024 ? 2 : 1;
  static constexpr bool B16 = W == 2 || CONV;            // the products read 16-bit rows
  static constexpr int BLOCK = WT * TN;                  // positions of a block
};

// Physical 16-byte chunk of a row's chunk `c` in shared memory, such that the
// reads below meet no bank twice (ldmatrix takes the same chunk of 8 rows; 8-bit
// keys 4 neighbouring chunks of rows 2i and 2i + 1; 8-bit values 2 chunks of
// every other row).
template <class C>
__device__ __forceinline__ int kchunk(int row, int c) {
  if (C::W == 2) return c ^ (row & 7);
  return C::D == 128 && !C::CONV ? c ^ ((row & 1) << 2) : c;
}
template <class C>
__device__ __forceinline__ int vchunk(int row, int c) {
  if (C::W == 2) return c ^ (row & 7);
  return C::CONV ? c : C::D == 128 ? c ^ (row & 6) : c ^ (row & 2);
}

// a / b for a >= 0, b > 0, in 32 bits where both fit (a 64-bit division takes some
// hundred instructions, and every CTA starts with several)
__device__ __forceinline__ int64_t idiv(int64_t a, int64_t b) {
  return ((uint64_t)a | (uint64_t)b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

__device__ __forceinline__ float2 f16_floats(uint32_t two) {
  float2 r;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "r"(two));
  return r;
}
// code x of the four in w
template <int KIND>
__device__ __forceinline__ float code_value(uint32_t w, int x) {
  const uint32_t c = (w >> (8 * x)) & 0xFFu;
  return KIND == DHS_PAGE_INT8 ? (float)(int8_t)c : f16_floats(e4m3_f16(c)).x;
}

struct AttnArgs {
  const uint16_t *q;
  const int32_t *q_lens, *seq_lens, *table;
  uint16_t *out;
  float *lse;
  int2 *plan;        // [n_seqs][hkv]: first and last CTA of an item in parts, or (-1, -1)
  float *parts;      // [grid][2][R][D + 4]: O, m, l, -
  int32_t *err;
  int width, n_seqs, q_len, hq, G, R;
  float scale_log2;
};

// More than 32 sequences.  Their lengths are read eight to a lane, under way together (1024
// sequences of 200: 53 -> 38 us).
struct SeqLens {
  const int32_t *q_lens, *seq_lens;
  int q_len, n_seqs, most;
};
// Blocks (of one kv head) of sequences i + 32 u + this lane.
template <int BLOCK>
__device__ __forceinline__ void blocks_of_8(const SeqLens &a, int i, int (&n)[8], int32_t *err) {
  const int lane = threadIdx.x & 31;
  int nq[8], len[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int at = i + 32 * u + lane;
    nq[u] = at >= a.n_seqs ? 0 : a.q_lens ? a.q_lens[at] : a.q_len;
    len[u] = at >= a.n_seqs ? 0 : a.seq_lens[at];
  }
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    if (nq[u] < 0 || nq[u] > a.q_len || len[u] < 0 || len[u] > a.most)
      page_error(err, DC_ROW_RANGE, DHS_SITE_PAGE_ATTEND);
    len[u] = max(0, min(len[u], a.most));
    n[u] = nq[u] > 0 ? (int)(((uint32_t)len[u] + BLOCK - 1) / BLOCK) : 0;
  }
}
// This lane's share of all blocks, and the sequences with any.
template <int BLOCK>
__device__ __forceinline__ longlong2 count_blocks(const SeqLens &a, int32_t *err) {
  int64_t sum = 0;
  int some = 0;
  for (int i = 0; i < a.n_seqs; i += 256) {
    int n[8];
    blocks_of_8<BLOCK>(a, i, n, err);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      some += __popc(__ballot_sync(0xffffffffu, n[u] > 0));
      sum += n[u];
    }
  }
  return make_longlong2(sum, some);
}
// The 32 neighbours (their first) among whom unit `want` is, and the units before them.
// (chunk: blocks of a unit)
template <int BLOCK>
__device__ __forceinline__ longlong2 find_neighbours(const SeqLens &a, int64_t want,
                                                     int64_t chunk) {
  int base = 0;
  bool found = false;
  int64_t at = 0;
  for (int i = 0; i < a.n_seqs && !found; i += 256) {
    int n[8];
    blocks_of_8<BLOCK>(a, i, n, nullptr);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int units = chunk == 1 ? n[u] : (int)idiv(n[u] + chunk - 1, chunk);
      const int all = __reduce_add_sync(0xffffffffu, units);
      if (!found && want < at + all) {
        found = true;
        base = i + 32 * u;
      }
      if (!found) at += all;
    }
  }
  return make_longlong2(base, at);
}
// The same as calls: with these loops inside it, the kernel's code for few sequences lies
// apart, which costs where it has to come from memory (L2 flushed before each call: one
// sequence of 4096 18.7 us with them, 16.9 without; 16 of 64K in int8 77 and 73, 8 of up to
// 32K in bf16, 4 tokens each, 41.5 and 39.5).  More than 32 pay for it with 1 to 5 % (61 of
// 8000 in e4m3 106.8 and 107.7, 1024 of 200 in int8, 32 rows each, 63 and 66).
template <int BLOCK>
__device__ __noinline__ longlong2 count_blocks_call(const int32_t *q_lens, const int32_t *seq_lens,
                                                    int q_len, int n_seqs, int most,
                                                    int32_t *err) {
  return count_blocks<BLOCK>(SeqLens{q_lens, seq_lens, q_len, n_seqs, most}, err);
}
template <int BLOCK>
__device__ __noinline__ longlong2 find_neighbours_call(const int32_t *q_lens,
                                                       const int32_t *seq_lens, int q_len,
                                                       int n_seqs, int most, int64_t want,
                                                       int64_t chunk) {
  return find_neighbours<BLOCK>(SeqLens{q_lens, seq_lens, q_len, n_seqs, most}, want, chunk);
}

template <class C>
__global__ void __launch_bounds__(kPaThreads, C::OCC)
k_page_attn(const PageView pg, const AttnArgs a) {
  constexpr int D = C::D, MT = C::MT, WM = C::WM, WT = C::WT, TN = C::TN, NS = C::NS, RB = C::RB;
  constexpr int KIND = C::KIND, SUB = C::SUB, NH = C::NH, RC = C::RC;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int sh_flag;       // values that are not finite were taken out
  __shared__ uint32_t sh_late;  // positions from `common` on that were left out
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wm = warp % WM, wt = warp / WM;      // rows of this warp, token group
  const int gl = wm * 32 + lane;                 // thread within the group
  const int qd = lane & 3, ql = lane >> 2;
  const int hkv = pg.hkv;
  // (a tile past the last position still fits 32 bits)
  const int64_t most = min((int64_t)a.width * pg.rows, (int64_t)INT32_MAX - 1024);

  // queries and visible length of a sequence, and its blocks per kv head
  auto shape = [&](int i, int &nq, int &len) {
    nq = a.q_lens ? a.q_lens[i] : a.q_len;
    len = a.seq_lens[i];
    if (nq < 0 || nq > a.q_len || len < 0 || len > most) {
      page_error(a.err, DC_ROW_RANGE, DHS_SITE_PAGE_ATTEND);
      nq = max(0, min(nq, a.q_len));
      len = (int)max((int64_t)0, min((int64_t)len, most));
    }
  };
  // Blocks (of one kv head) of sequence i + lane; with 32 sequences or fewer each lane
  // keeps what it read.
  const bool few = a.n_seqs <= 32;
  int my_nq = 0, my_len = 0, my_n = 0;
  bool known = false;
  auto blocks = [&](int i) {
    if (known) return my_n;
    my_nq = my_len = 0;
    if (i + lane < a.n_seqs) shape(i + lane, my_nq, my_len);
    my_n = my_nq > 0 ? (int)(((uint32_t)my_len + C::BLOCK - 1) / C::BLOCK) : 0;
    return my_n;
  };

  // (128 rows of bf16 have no register for the calls' sake: 498 us for 32 x 64K, 542 with them)
  constexpr bool kCalls = !(C::W == 2 && MT == 2);
  const SeqLens seqs{a.q_lens, a.seq_lens, a.q_len, a.n_seqs, (int)most};
  // All blocks, and the sequences with any: every warp adds up all of them.
  int64_t sum = 0;
  int some = 0;
  if (few) {
    const int n = blocks(0);
    some = __popc(__ballot_sync(0xffffffffu, n > 0));
    sum = __reduce_add_sync(0xffffffffu, n);  // (32 of them fit 32 bits)
  } else {
    const longlong2 r = kCalls ? count_blocks_call<C::BLOCK>(a.q_lens, a.seq_lens, a.q_len,
                                                             a.n_seqs, (int)most, a.err)
                               : count_blocks<C::BLOCK>(seqs, a.err);
    sum = r.x;
    some = (int)r.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  known = few;
  const int64_t total = sum * hkv;

  // sequences without a block: their queries see nothing
  for (int i = blockIdx.x; i < a.n_seqs; i += gridDim.x) {
    int nq, len;
    shape(i, nq, len);
    if (nq > 0 && len > 0) continue;
    for (int h = tid; h < hkv; h += kPaThreads) a.plan[(int64_t)i * hkv + h] = make_int2(-1, -1);
    if (nq == 0) continue;
    const int64_t base = (int64_t)i * a.q_len * a.hq;
    for (int e = tid; e < nq * a.hq * (D / 8); e += kPaThreads)
      *reinterpret_cast<uint4 *>(a.out + (base * D + (int64_t)e * 8)) = make_uint4(0u, 0u, 0u, 0u);
    if (a.lse)
      for (int e = tid; e < nq * a.hq; e += kPaThreads) a.lse[base + e] = -CUDART_INF_F;
  }
  // CTAs that take part.  An item of b blocks in P parts costs b / P blocks of
  // streaming and P parts of (R, D) in the join, least at P = sqrt(b x block
  // bytes / part bytes); more CTAs than that lengthen a short call.
  const int64_t items = (int64_t)some * hkv;
  const float parts =
      items > 0 ? ceilf(sqrtf((float)total / (float)items * ((float)C::BLOCK * 2 * RB) /
                              (float)(a.R * D * 4)))
                : 0.f;
  int64_t n_parts = (int64_t)((float)items * parts);
  if (n_parts > gridDim.x / C::OCC) n_parts = gridDim.x;
  int n_cta = (int)min(min((int64_t)gridDim.x, total), n_parts);
  // Few long items: a CTA whose blocks belong to two items fills and drains its ring
  // twice (some 4 us), and the others wait for it.  Then each CTA takes one chunk of
  // at most `most_blocks` blocks of one item, of which there are at most n_cta.  Chunks
  // are up to items / n_cta longer than even shares, so many items lose by them.  Both
  // sides, 128 dims, 1 to 32 rows, one item of 8K, 32K or 100K positions and the others of
  // half that to that, means over 8 or 12 such batches: 2 items +0.1 % (-7 to +9), 3 -2.2,
  // 4 -5.1, 6 -3.7, 8 -2.0, 9 -2.3, 10 -1.3, 12 -3.4, 16 -2.4, 24 -2.0, 32 -2.6 (-7 to 0),
  // 48 +0.8 (-3 to +3).  The rule stops at 9 and leaves some 2 % at 10 to 32.
  const bool chunked = items > 1 && items * 32 <= n_cta;
  const int64_t most_blocks =
      chunked ? idiv(total + n_cta - items - 1, max((int64_t)1, n_cta - items)) : 1;
  auto units = [&](int64_t n) { return chunked ? idiv(n + most_blocks - 1, most_blocks) : n; };
  int64_t total_units = total;
  if (chunked) {
    int64_t x = 0;
    for (int i = 0; i < a.n_seqs; i += 32) x += units(blocks(i));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    total_units = x * hkv;
    n_cta = (int)total_units;
  }
  pdl_trigger();  // the join may be placed; it waits for this grid's end
  if ((int)blockIdx.x >= n_cta) return;
  // from here on places are in units: chunks, or blocks
  auto range = [&](int b) -> int64_t { return chunked ? b : idiv(total_units * b, n_cta); };
  const int64_t begin = range(blockIdx.x), end = range(blockIdx.x + 1);

  // the sequence that holds unit `begin`, and the unit it starts at
  int seq = 0, seq_nq = 0, seq_len = 0;
  int64_t seq_at = 0;
  {
    const int64_t want = idiv(begin, hkv);  // in units of one head: only the sequence is looked for
    int64_t at = 0;
    int base = 0;  // its 32 neighbours
    if (!few) {
      const longlong2 r =
          kCalls ? find_neighbours_call<C::BLOCK>(a.q_lens, a.seq_lens, a.q_len, a.n_seqs,
                                                  (int)most, want, most_blocks)
                 : find_neighbours<C::BLOCK>(seqs, want, most_blocks);
      base = (int)r.x;
      at = r.y;
    }
    const int n = (int)units(blocks(base));
    int x = n;  // inclusive sums
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const uint32_t here = __ballot_sync(0xffffffffu, want < at + x);
    const int src = max(0, __ffs(here) - 1);
    seq = base + src;
    seq_at = (at + __shfl_sync(0xffffffffu, x - n, src)) * hkv;
    seq_nq = __shfl_sync(0xffffffffu, my_nq, src);
    seq_len = __shfl_sync(0xffffffffu, my_len, src);
  }
  if (tid == 0) {
    sh_flag = 0;
    sh_late = 0u;
  }
  __syncthreads();

  unsigned char *ring = smem + wt * C::GROUP;
  int64_t *rowbuf = reinterpret_cast<int64_t *>(smem + C::OFF_ROW) + wt * C::SLOTS * TN;
  uint32_t *maskbuf = reinterpret_cast<uint32_t *>(smem + C::OFF_MASK) + wt * C::SLOTS * 2;
  float *ml = reinterpret_cast<float *>(smem + C::OFF_ML);
  float *osm = reinterpret_cast<float *>(smem);
  auto group_sync = [&]() {
    if (WM == 1) __syncwarp();
    else if (WT == 1) __syncthreads();
    else named_sync(1 + wt, WM * 32);
  };

  for (int64_t pos = begin; pos < end && seq < a.n_seqs;) {
    const int nq = seq_nq, len = seq_len;
    const int64_t nb = nq > 0 ? (int64_t)(((uint32_t)len + C::BLOCK - 1) / C::BLOCK) : 0;
    const int64_t nu = units(nb);
    if (pos >= seq_at + nu * hkv) {  // on to the next sequence (empty ones among them)
      seq_at += nu * hkv;
      if (++seq < a.n_seqs) shape(seq, seq_nq, seq_len);
      continue;
    }
    const int kvh = (int)idiv(pos - seq_at, nu);
    const int64_t item0 = seq_at + kvh * nu, item1 = item0 + nu;
    const int64_t stop = min(end, item1);
    // blocks of this item's part
    const int b0 = (int)(chunked ? idiv(nb * (pos - item0), nu) : pos - item0);
    const int nblk = (int)(chunked ? idiv(nb * (stop - item0), nu) : stop - item0) - b0;
    const int32_t *tab = a.table + (int64_t)seq * a.width;

    // ---- Q fragments of this warp's rows: for 16-bit rows k-step s holds dims 16 s ..;
    // for 8-bit ones k index (s, 2 qd + e) is dim 64 j + 16 qd + 4 s + e and (s, 2 qd + 8 + e)
    // is 2 further on, s = 0 .. 3 of the 64 dims of block j
    uint32_t qf[MT][D / 16][4];
    auto load_q = [&]() {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int m = (wm * MT + mt) * 16 + half * 8 + ql, j = m / a.G;
          const bool on = m < a.R && j < nq;
          const uint16_t *src =
              a.q + (((int64_t)seq * a.q_len + j) * a.hq + kvh * a.G + (m - j * a.G)) * D;
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const int lo = C::B16 ? 16 * s + 2 * qd : 64 * (s >> 2) + 16 * qd + 4 * (s & 3);
            const int hi = lo + (C::B16 ? 8 : 2);
            qf[mt][s][half] = on ? *reinterpret_cast<const uint32_t *>(src + lo) : 0u;
            qf[mt][s][2 + half] = on ? *reinterpret_cast<const uint32_t *>(src + hi) : 0u;
          }
        }
    };
    // 8 bits: under way with the lookups and first copies, as the rows' largest elements
    // are wanted before the first tile (189 short sequences 74 -> 69 us); bf16 after them
    // (400 short sequences 94 us, before them 100), and so 128 rows of 8 bits, whose
    // registers are short (32 x 64K took 833 us then, before them 842)
    constexpr bool kEarly = C::W == 1 && MT == 1;
    if (kEarly) load_q();

    // ---- row lookups and copies, tile by tile.  Tile t of the group is
    // positions (b0 + t) * BLOCK + wt * TN ...
    constexpr int LK = (TN + WM * 32 - 1) / (WM * 32);  // lookups of a thread
    // the page (-1: no position there), read ahead of the row that follows from it
    auto lookup = [&](int t, int (&page)[LK]) {
#pragma unroll
      for (int u = 0; u < LK; ++u) {
        const int x = gl + u * WM * 32;
        const int64_t p = (int64_t)(b0 + t) * C::BLOCK + wt * TN + x;
        page[u] = t < nblk && x < TN && p < len
                      ? tab[(uint64_t)(uint32_t)p * pg.div_mul >> pg.div_shift]
                      : INT32_MIN;
      }
    };
    auto keep = [&](int t, const int (&page)[LK]) {
      int64_t *dst = rowbuf + (t % C::SLOTS) * TN;
#pragma unroll
      for (int u = 0; u < LK; ++u) {
        const int x = gl + u * WM * 32;
        const uint32_t p = (uint32_t)((b0 + t) * C::BLOCK + wt * TN + x);
        int64_t row = -1;  // nothing there
        if (page[u] >= 0 && page[u] < pg.n_pages)
          row = ((int64_t)page[u] * hkv + kvh) * pg.rows +
                (p - (uint32_t)((uint64_t)p * pg.div_mul >> pg.div_shift) * pg.rows);
        else if (page[u] != INT32_MIN)
          page_error(a.err, DC_LOC_RANGE, DHS_SITE_PAGE_ATTEND);
        const uint32_t ok = __ballot_sync(0xffffffffu, row >= 0);
        if (x < TN) dst[x] = row;
        if (lane == 0 && (x >> 5) < 2) maskbuf[(t % C::SLOTS) * 2 + (x >> 5)] = ok;
      }
    };
    // In-page offset of the tile that is copied next: a tile inside one page and
    // below the length is one run of memory, copied from one address with constant
    // offsets; others row by row.
    int in_page = (int)((uint32_t)(b0 * C::BLOCK + wt * TN) % (uint32_t)pg.rows);
    const int in_step = C::BLOCK % pg.rows;
    auto copy = [&](int t) {
      // a thread copies one chunk column of every STEP-th row
      constexpr int STEP = WM * 32 / C::CH;
      constexpr int XM = STEP >= 8 ? 7 : STEP - 1;  // x & 7 = (xr & XM) + (u * STEP & 7)
      const int xr = gl / C::CH, c = gl % C::CH;
      if (t < nblk) {
        unsigned char *kst = ring + (t % NS) * C::STAGE, *vst = kst + C::KV;
        float *sc = reinterpret_cast<float *>(vst + C::KV);
        const int64_t *src = rowbuf + (t % C::SLOTS) * TN;
        const int64_t row0 = src[0];
        const bool run = in_page + TN <= pg.rows && row0 >= 0 &&
                         (int64_t)(b0 + t) * C::BLOCK + wt * TN + TN <= len;
        if (run) {
          const unsigned char *gk = pg.k + (row0 + xr) * RB + c * 16;
          const unsigned char *gv = pg.v + (row0 + xr) * RB + c * 16;
#pragma unroll
          for (int u = 0; u < TN / STEP; ++u) {
            const int low = (xr & XM) + (u * STEP & 7);
            cp_async_16(kst + (xr + u * STEP) * RB + kchunk<C>(low, c) * 16, gk + u * STEP * RB);
            cp_async_16(vst + (xr + u * STEP) * RB + vchunk<C>(low, c) * 16, gv + u * STEP * RB);
          }
          if (C::W == 1) {
#pragma unroll
            for (int u = 0; u < LK; ++u) {
              const int x = gl + u * WM * 32;
              if (x < TN) {
                cp_async_4(sc + x, pg.ks + row0 + x);
                cp_async_4(sc + TN + x, pg.vs + row0 + x);
              }
            }
          }
        } else {
#pragma unroll 4
          for (int u = 0; u < TN / STEP; ++u) {
            const int x = xr + u * STEP;
            const int64_t row = src[x];
            const int n = row < 0 ? 0 : 16;
            const int64_t off = (row < 0 ? 0 : row * RB) + c * 16;
            cp_async_16_zfill(kst + x * RB + kchunk<C>(x, c) * 16, pg.k + off, n);
            cp_async_16_zfill(vst + x * RB + vchunk<C>(x, c) * 16, pg.v + off, n);
          }
          if (C::W == 1) {
#pragma unroll
            for (int u = 0; u < LK; ++u) {
              const int x = gl + u * WM * 32;
              if (x < TN) {
                const int64_t row = src[x];
                cp_async_4_zfill(sc + x, pg.ks + (row < 0 ? 0 : row), row < 0 ? 0 : 4);
                cp_async_4_zfill(sc + TN + x, pg.vs + (row < 0 ? 0 : row), row < 0 ? 0 : 4);
              }
            }
          }
        }
      }
      in_page += in_step;
      if (in_page >= pg.rows) in_page -= pg.rows;
      cp_async_commit();
    };

    {
      int page[NS][LK];
#pragma unroll
      for (int t = 0; t < NS; ++t) lookup(t, page[t]);
#pragma unroll
      for (int t = 0; t < NS; ++t) keep(t, page[t]);
    }
    group_sync();
#pragma unroll
    for (int t = 0; t < NS - 1; ++t) copy(t);

    if (!kEarly) load_q();

    // ---- Q in f16 and what a score is multiplied by
    float fr[MT][2];  // by row: softmax scale in log2 units, f16 scaling
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        fr[mt][half] = a.scale_log2;
        if (C::W == 1) {
          uint32_t top = 0u;
#pragma unroll
          for (int s = 0; s < D / 16; ++s)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t x = qf[mt][s][2 * k + half];
              top = max(top, max(x & 0x7FFFu, (x >> 16) & 0x7FFFu));
            }
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          // the largest element goes to [2^14, 2^15) (infinities and NaN stay)
          const int e = top >= 0x7F80u ? 0 : max((int)(top >> 7) - 127 - 14, -110);
          const float down = __uint_as_float((uint32_t)(127 - e) << 23);
          // (above zero, as it multiplies -infinity)
          fr[mt][half] = fmaxf(fr[mt][half] * __uint_as_float((uint32_t)(127 + e) << 23), 1e-37f);
#pragma unroll
          for (int s = 0; s < D / 16; ++s)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t x = qf[mt][s][2 * k + half];
              qf[mt][s][2 * k + half] = pack_f16(__uint_as_float(x << 16) * down,
                                                 __uint_as_float(x & 0xFFFF0000u) * down);
            }
        }
      }
    // visible positions of this thread's rows (idle rows: all, never written)
    int seen[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int j = ((wm * MT + mt) * 16 + half * 8 + ql) / a.G;
        seen[mt][half] = j < nq ? len - nq + j + 1 : len;
      }
    const int common = len - nq + 1;  // positions that every query sees

    float o[MT][D / 8][4], mx[MT][2];
    float l[MT][2];
    int vref = -200;   // 8 bits: weights times scales are over 2^vref
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][i][e] = 0.f;
      mx[mt][0] = mx[mt][1] = -CUDART_INF_F;
      l[mt][0] = l[mt][1] = 0.f;
    }

    for (int t = 0; t < nblk; ++t) {
      cp_async_wait_group<NS - 2>();
      group_sync();
      int ahead[LK];
      lookup(t + NS, ahead);
      copy(t + NS - 1);
      unsigned char *kst = ring + (t % NS) * C::STAGE, *vst = kst + C::KV;
      float *sc = reinterpret_cast<float *>(vst + C::KV);
      const int p0 = (int)((int64_t)(b0 + t) * C::BLOCK) + wt * TN;
      const uint32_t ok0 = maskbuf[(t % C::SLOTS) * 2];
      const uint32_t ok1 = TN > 32 ? maskbuf[(t % C::SLOTS) * 2 + 1] : 0xffffffffu;
      const bool full = TN == 16 ? (ok0 & 0xffffu) == 0xffffu : (ok0 & ok1) == 0xffffffffu;
      const bool masked = !full || p0 + TN > common;
      if (KIND == DHS_PAGE_BF16 && nq > 1 && p0 + TN > common) {
        // values that only some queries see: those that are not finite out
        const int x0 = max(0, common - p0), x1 = min(TN, len - p0);
        for (int e = x0 * C::CH + lane; e < x1 * C::CH; e += 32) {
          const int x = e / C::CH, c = e % C::CH;
          uint4 *at = reinterpret_cast<uint4 *>(vst + x * RB + vchunk<C>(x, c) * 16);
          uint32_t w[4] = {at->x, at->y, at->z, at->w};
          bool bad = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if ((w[i] & 0x7F80u) == 0x7F80u) { w[i] &= 0xFFFF0000u; bad = true; }
            if ((w[i] & 0x7F800000u) == 0x7F800000u) { w[i] &= 0x0000FFFFu; bad = true; }
          }
          if (bad) {
            *at = make_uint4(w[0], w[1], w[2], w[3]);
            sh_flag = 1;
          }
        }
        __syncwarp();
      }
      if (C::W == 1) {
        if (C::SOME && nq > 1 && p0 + TN > common) {
          // Scales that only some rows see (the last q_len - 1) and that are 2^5 times those
          // that all see, or the first of them: following one would cost the rows that do
          // not see it their weights.  Where the power of two does not cover them already,
          // their positions' values are left for the merge.  (Each warp of the group does
          // the same.  This costs 1 to 3 %; a power of two of each row's own cost 4 to 16.)
          int e[2] = {-127, -127}, ref = -127;
#pragma unroll
          for (int u = 0; u < (TN + 31) / 32; ++u) {
            const int x = lane + u * 32;
            const uint32_t b = x < TN ? __float_as_uint(sc[TN + x]) : 0u;
            e[u] = (int)((b < 0x7F800000u ? b : 0u) >> 23) - 127;
            if (p0 + x <= max(p0, common - 1)) ref = max(ref, e[u]);
          }
          ref = __reduce_max_sync(0xffffffffu, ref);
#pragma unroll
          for (int u = 0; u < (TN + 31) / 32; ++u) {
            const int x = lane + u * 32;
            if (p0 + x >= max(common, 0) && e[u] > ref + 4 && e[u] >= vref + kVrefMax) {
              sc[TN + x] = 0.f;
              atomicOr(&sh_late, 1u << (p0 + x - common));
            }
          }
          __syncwarp();
        }
        // the tile's largest value scale (as bits; not one that is not finite)
        uint32_t top = 0u;
#pragma unroll
        for (int u = 0; u < (TN + 31) / 32; ++u) {
          const int x = lane + u * 32;
          const uint32_t b = x < TN ? __float_as_uint(sc[TN + x]) : 0u;
          top = max(top, b < 0x7F800000u ? b : 0u);
        }
        const int e = (int)(__reduce_max_sync(0xffffffffu, top) >> 23) - 127;
        if (e >= vref + kVrefMax) {
          const int to = max(e - kVrefUp, -100);
          const float f = vref < -100 ? 0.f : ex2_approx((float)(vref - to));
          vref = to;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
              for (int x = 0; x < 4; ++x) o[mt][i][x] *= f;
        }
      }
      const unsigned char *kc = kst, *vc = vst;  // the rows as the products read them
      if (C::CONV) {
        unsigned char *f16 = ring + C::RING;
#pragma unroll
        for (int u = 0; u < 2 * TN * C::CH / (WM * 32); ++u) {
          const int e = (gl + u * WM * 32) % (TN * C::CH), x = e / C::CH, c = e % C::CH;
          const int v = (gl + u * WM * 32) / (TN * C::CH);  // keys, then values
          const uint4 w = *reinterpret_cast<const uint4 *>(kst + v * C::KV + e * 16);
          uint4 lo, hi;
          f16_pairs<KIND>(w.x, lo.x, lo.y);
          f16_pairs<KIND>(w.y, lo.z, lo.w);
          f16_pairs<KIND>(w.z, hi.x, hi.y);
          f16_pairs<KIND>(w.w, hi.z, hi.w);
          unsigned char *dst = f16 + v * TN * RC + x * RC;
          *reinterpret_cast<uint4 *>(dst + (((2 * c) ^ (x & 7)) << 4)) = lo;
          *reinterpret_cast<uint4 *>(dst + (((2 * c + 1) ^ (x & 7)) << 4)) = hi;
        }
        kc = f16;
        vc = f16 + TN * RC;
        group_sync();
      }
      const float vdown = C::W == 1 ? __uint_as_float((uint32_t)(127 - max(vref, -100)) << 23) : 1.f;
#pragma unroll
      for (int sub = 0; sub < TN / SUB; ++sub) {
        const int s0 = sub * SUB;
        // scores
        float s[MT][SUB / 8][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < SUB / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][i][e] = 0.f;
        if (C::B16) {
#pragma unroll
          for (int i = 0; i < SUB / 16; ++i)
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              // matrices: positions 0-7 and 8-15 of the 16, each with two chunks
              const int x = s0 + i * 16 + (lane & 7) + ((lane >> 4) << 3);
              const int c = ks * 2 + ((lane >> 3) & 1);
              uint32_t b0r, b1r, b2r, b3r;
              ldmatrix_x4(b0r, b1r, b2r, b3r, kc + x * RC + ((c ^ (x & 7)) << 4));
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma_kind<KIND>(s[mt][2 * i], qf[mt][ks], b0r, b1r);
                mma_kind<KIND>(s[mt][2 * i + 1], qf[mt][ks], b2r, b3r);
              }
            }
        } else {
#pragma unroll
          for (int i = 0; i < SUB / 8; ++i)
#pragma unroll
            for (int jb = 0; jb < D / 64; ++jb) {
              const int x = s0 + i * 8 + ql;
              const uint4 w = *reinterpret_cast<const uint4 *>(
                  kst + x * RB + kchunk<C>(x, jb * 4 + qd) * 16);
              const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int ks = 0; ks < 4; ++ks) {
                uint32_t b0r, b1r;
                f16_pairs<KIND>(ww[ks], b0r, b1r);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                  mma_kind<KIND>(s[mt][i], qf[mt][jb * 4 + ks], b0r, b1r);
              }
            }
        }
        // key scales, masks, the rows' maxima (a row's factor fr comes later)
        float top[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) top[mt][0] = top[mt][1] = -CUDART_INF_F;
#pragma unroll
        for (int i = 0; i < SUB / 8; ++i) {
          float2 ks = make_float2(1.f, 1.f);
          if (C::W == 1) ks = *reinterpret_cast<const float2 *>(sc + s0 + i * 8 + 2 * qd);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < NH; ++h) {
              float2 x = make_float2(s[mt][i][2 * h], s[mt][i][2 * h + 1]);
              if (C::W == 1) x = make_float2(x.x * ks.x, x.y * ks.y);
              if (masked) {
                const int c = s0 + i * 8 + 2 * qd;
                const uint32_t there = c < 32 ? ok0 >> c : ok1 >> (c - 32);
                if (!(there & 1u) || p0 + c >= seen[mt][h]) x.x = -CUDART_INF_F;
                if (!(there & 2u) || p0 + c + 1 >= seen[mt][h]) x.y = -CUDART_INF_F;
              }
              s[mt][i][2 * h] = x.x;
              s[mt][i][2 * h + 1] = x.y;
              top[mt][h] = fmaxf(top[mt][h], fmaxf(x.x, x.y));
            }
        }
        bool grow = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            top[mt][h] = fmaxf(top[mt][h], __shfl_xor_sync(0xffffffffu, top[mt][h], 1));
            top[mt][h] = fmaxf(top[mt][h], __shfl_xor_sync(0xffffffffu, top[mt][h], 2));
            top[mt][h] *= fr[mt][h];
            grow |= top[mt][h] > mx[mt][h] + (C::W == 1 ? kRescale8 : kRescale16);
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < NH; ++h) {
              // (a row that has seen nothing keeps its zeros)
              const float m_new = fmaxf(mx[mt][h], top[mt][h]);
              const float f = mx[mt][h] == -CUDART_INF_F ? 0.f : ex2_approx(mx[mt][h] - m_new);
              mx[mt][h] = m_new;
              l[mt][h] *= f;
#pragma unroll
              for (int i = 0; i < D / 8; ++i) {
                o[mt][i][2 * h] *= f;
                o[mt][i][2 * h + 1] *= f;
              }
            }
        }
        // weights, rounded for the product with V: to bf16 (at most 2^-8 of each) or,
        // times the value's scale, to f16 (2^-11, or as said at the top); l takes the
        // weights unrounded.  -inf - -inf must not
        // arise in a row that has seen nothing yet
        uint32_t pf[MT][SUB / 16][4];
        if (NH == 1) {
#pragma unroll
          for (int i = 0; i < SUB / 16; ++i) pf[0][i][1] = pf[0][i][3] = 0u;
        }
#pragma unroll
        for (int i = 0; i < SUB / 8; ++i) {
          float2 vs = make_float2(1.f, 1.f);
          if (C::W == 1)
            vs = *reinterpret_cast<const float2 *>(sc + TN + s0 + i * 8 + 2 * qd);
          vs.x *= vdown;
          vs.y *= vdown;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < NH; ++h) {
              const float b = mx[mt][h] == -CUDART_INF_F ? 0.f : -mx[mt][h];
              float2 p = make_float2(ex2_approx(fmaf(s[mt][i][2 * h], fr[mt][h], b)),
                                     ex2_approx(fmaf(s[mt][i][2 * h + 1], fr[mt][h], b)));
              l[mt][h] += p.x + p.y;
              if (C::W == 1) {
                p.x *= vs.x;
                p.y *= vs.y;
                if (masked) {  // (a scale that is not finite at a masked place)
                  const int c = s0 + i * 8 + 2 * qd;
                  const uint32_t there = c < 32 ? ok0 >> c : ok1 >> (c - 32);
                  if (!(there & 1u) || p0 + c >= seen[mt][h]) p.x = 0.f;
                  if (!(there & 2u) || p0 + c + 1 >= seen[mt][h]) p.y = 0.f;
                }
                pf[mt][i >> 1][(i & 1) * 2 + h] = pack_f16(p.x, p.y);
              } else {
                pf[mt][i >> 1][(i & 1) * 2 + h] = pack_bf16(p.x, p.y);
              }
            }
        }
        // O += P V
#pragma unroll
        for (int i = 0; i < SUB / 16; ++i) {
          if (C::B16) {
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
              const int x = s0 + i * 16 + (lane & 15);
              const int c = n * 2 + (lane >> 4);
              uint32_t b0r, b1r, b2r, b3r;
              ldmatrix_x4_trans(b0r, b1r, b2r, b3r, vc + x * RC + ((c ^ (x & 7)) << 4));
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma_kind<KIND>(o[mt][2 * n], pf[mt][i], b0r, b1r);
                mma_kind<KIND>(o[mt][2 * n + 1], pf[mt][i], b2r, b3r);
              }
            }
          } else {
            // output column n of tile c is dim n * (D / 8) + c; this thread's
            // n = ql of positions 2 qd, 2 qd + 1, 2 qd + 8, 2 qd + 9
            constexpr int NW = D / 32;  // words of a thread per position
            uint32_t w[4][NW];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int x = s0 + i * 16 + 2 * qd + (e & 1) + (e >> 1) * 8;
              if (D == 128) {
                const uint4 y = *reinterpret_cast<const uint4 *>(
                    vst + x * RB + vchunk<C>(x, ql) * 16);
                w[e][0] = y.x;
                w[e][1] = y.y;
                w[e][NW - 2] = y.z;
                w[e][NW - 1] = y.w;
              } else {
                const uint2 y = *reinterpret_cast<const uint2 *>(
                    vst + x * RB + vchunk<C>(x, ql >> 1) * 16 + (ql & 1) * 8);
                w[e][0] = y.x;
                w[e][1] = y.y;
              }
            }
#pragma unroll
            for (int c4 = 0; c4 < NW; ++c4) {
              // the two positions' bytes side by side, then four pairs of each half
              uint32_t b0r[4], b1r[4];
              f16_pairs<KIND>(__byte_perm(w[0][c4], w[1][c4], 0x5140), b0r[0], b0r[1]);
              f16_pairs<KIND>(__byte_perm(w[0][c4], w[1][c4], 0x7362), b0r[2], b0r[3]);
              f16_pairs<KIND>(__byte_perm(w[2][c4], w[3][c4], 0x5140), b1r[0], b1r[1]);
              f16_pairs<KIND>(__byte_perm(w[2][c4], w[3][c4], 0x7362), b1r[2], b1r[3]);
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                  mma_kind<KIND>(o[mt][c4 * 4 + c], pf[mt][i], b0r[c], b1r[c]);
            }
          }
        }
      }
      keep(t + NS, ahead);
    }

    // ---- merge the groups: ml [WT][ROWS] and O scaled to the rows' maxima
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        l[mt][h] += __shfl_xor_sync(0xffffffffu, l[mt][h], 1);
        l[mt][h] += __shfl_xor_sync(0xffffffffu, l[mt][h], 2);
        const int m = (wm * MT + mt) * 16 + h * 8 + ql;
        if (qd == 0)
          *reinterpret_cast<float2 *>(ml + (wt * C::ROWS + m) * 2) = make_float2(mx[mt][h], l[mt][h]);
      }
    cp_async_wait_all();
    __syncthreads();
    const bool patch = sh_flag != 0;
    const uint32_t late = C::SOME ? sh_late : 0u;
    float *late_w = reinterpret_cast<float *>(smem + C::OFF_LATE);  // a row's weights
    const bool whole = pos == item0 && stop == item1;
    const int slot = pos > item0 ? 0 : 1;
    float *part = a.parts + ((int64_t)blockIdx.x * 2 + slot) * a.R * (D + 4);
    int2 *tab_of = reinterpret_cast<int2 *>(smem + C::OFF_TAB);
    // a row's maximum and sum over the groups; its place (-1: an idle query) and the
    // factor of its output (negative: it sees nothing)
    if (tid < a.R) {
      const int m = tid, j = m / a.G, sees = len - nq + j + 1;
      float top = -CUDART_INF_F, den = 0.f;
#pragma unroll
      for (int g = 0; g < WT; ++g) top = fmaxf(top, ml[(g * C::ROWS + m) * 2]);
#pragma unroll
      for (int g = 0; g < WT; ++g) {
        const float2 x = *reinterpret_cast<const float2 *>(ml + (g * C::ROWS + m) * 2);
        const float f = x.x == -CUDART_INF_F ? (x.y != x.y ? 1.f : 0.f) : ex2_approx(x.x - top);
        den += x.y * f;
      }
      if (C::SOME && late) {
        const uint16_t *src =
            a.q + (((int64_t)seq * a.q_len + j) * a.hq + kvh * a.G + (m - j * a.G)) * D;
        for (int i = 0; i < kMaxKmax - 1; ++i) {
          if (!(late >> i & 1u) || common + i >= sees) continue;
          const int64_t row = page_row(pg, tab, common + i, nullptr, 0) + (int64_t)kvh * pg.rows;
          float x = 0.f;
          for (int c = 0; c < D; c += 4) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(pg.k + row * RB + c);
#pragma unroll
            for (int y = 0; y < 4; ++y)
              x = fmaf(__uint_as_float((uint32_t)src[c + y] << 16), code_value<KIND>(w, y), x);
          }
          late_w[m * kMaxKmax + i] = ex2_approx(x * pg.ks[row] * a.scale_log2 -
                                                (top == -CUDART_INF_F ? 0.f : top));
        }
      }
      const int at = j < nq ? j * a.hq + (m - j * a.G) : -1;
      tab_of[m] = make_int2(at, __float_as_int(sees <= 0 ? -1.f : 1.f / den));  // (only -inf: 0 / 0)
      if (j < nq) {
        if (!whole) {
          *reinterpret_cast<float2 *>(part + m * (D + 4) + D) = make_float2(top, den);
        } else if (a.lse) {
          a.lse[(int64_t)seq * a.q_len * a.hq + kvh * a.G + at] =
              top == CUDART_INF_F ? top
              : den == 0.f        ? -CUDART_INF_F
                                  : (top + log2f(den)) * 0.69314718055994531f;
        }
      }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const int m = (wm * MT + mt) * 16 + h * 8 + ql;
        float top = -CUDART_INF_F;
#pragma unroll
        for (int g = 0; g < WT; ++g) top = fmaxf(top, ml[(g * C::ROWS + m) * 2]);
        // O to the item's maximum so far, and from its power of two
        const float up = C::W == 1 ? (float)max(vref, -100) : 0.f;
        const float f = mx[mt][h] == -CUDART_INF_F ? 0.f : ex2_approx(mx[mt][h] - top + up);
        // (not zero times a NaN: a row of NaN scores keeps m = -inf and O = NaN)
        const bool nan = l[mt][h] != l[mt][h];
        float *dst = osm + (wt * C::ROWS + m) * C::OPAD;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const float x = nan ? CUDART_NAN_F : o[mt][i][2 * h] * f;
          const float y = nan ? CUDART_NAN_F : o[mt][i][2 * h + 1] * f;
          if (C::B16) {
            *reinterpret_cast<float2 *>(dst + 8 * i + 2 * qd) = make_float2(x, y);
          } else {
            dst[2 * qd * (D / 8) + i] = x;
            dst[(2 * qd + 1) * (D / 8) + i] = y;
          }
        }
      }
    __syncthreads();

    if (tid == 0) {  // every thread has read them
      sh_flag = 0;
      sh_late = 0u;
    }
    // one row's 4 dims at a time
    uint16_t *out0 = a.out + ((int64_t)seq * a.q_len * a.hq + kvh * a.G) * D;
    for (int e = tid; e < a.R * (D / 4); e += kPaThreads) {
      const int m = e / (D / 4), d4 = (e % (D / 4)) * 4;
      const int2 tb = tab_of[m];
      if (tb.x < 0) continue;
      float4 acc = *reinterpret_cast<const float4 *>(osm + m * C::OPAD + d4);
#pragma unroll
      for (int g = 1; g < WT; ++g) {
        const float4 y = *reinterpret_cast<const float4 *>(osm + (g * C::ROWS + m) * C::OPAD + d4);
        acc.x += y.x;
        acc.y += y.y;
        acc.z += y.z;
        acc.w += y.w;
      }
      if (C::SOME && late) {
        for (int i = 0; i < kMaxKmax - 1; ++i) {
          if (!(late >> i & 1u) || common + i >= len - nq + m / a.G + 1) continue;
          const int64_t row = page_row(pg, tab, common + i, nullptr, 0) + (int64_t)kvh * pg.rows;
          const uint32_t w = *reinterpret_cast<const uint32_t *>(pg.v + row * RB + d4);
          const float p = late_w[m * kMaxKmax + i], vs = pg.vs[row];
          acc.x += p * (vs * code_value<KIND>(w, 0));
          acc.y += p * (vs * code_value<KIND>(w, 1));
          acc.z += p * (vs * code_value<KIND>(w, 2));
          acc.w += p * (vs * code_value<KIND>(w, 3));
        }
      }
      if (KIND == DHS_PAGE_BF16 && patch) {
        // the values taken out above, for the queries that see them
        const int64_t lo = max((int64_t)max(0, common), (int64_t)b0 * C::BLOCK);
        const int64_t hi = min((int64_t)len - nq + m / a.G + 1, (int64_t)(b0 + nblk) * C::BLOCK);
        for (int64_t p = lo; p < hi; ++p) {
          int64_t row = page_row(pg, tab, (int)p, a.err, DHS_SITE_PAGE_ATTEND);
          if (row < 0) continue;
          row += (int64_t)kvh * pg.rows;
          const uint2 w = *reinterpret_cast<const uint2 *>(pg.v + row * RB + d4 * 2);
          const uint32_t b[4] = {w.x << 16, w.x & 0xFFFF0000u, w.y << 16, w.y & 0xFFFF0000u};
          float *c4[4] = {&acc.x, &acc.y, &acc.z, &acc.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if ((b[i] & 0x7F800000u) == 0x7F800000u) *c4[i] += __uint_as_float(b[i]);
        }
      }
      if (whole) {
        const float inv = __int_as_float(tb.y);
        *reinterpret_cast<uint2 *>(out0 + (int64_t)tb.x * D + d4) =
            inv < 0.f ? make_uint2(0u, 0u)
                      : make_uint2(pack_bf16(acc.x * inv, acc.y * inv),
                                   pack_bf16(acc.z * inv, acc.w * inv));
      } else {
        *reinterpret_cast<float4 *>(part + m * (D + 4) + d4) = acc;
      }
    }
    if (pos == item0 && tid == 0) {
      // for the join: the CTAs that share the item
      auto owner = [&](int64_t blk) {  // largest b with range(b) <= blk (a unit)
        int b = (int)min((int64_t)n_cta - 1, idiv((blk + 1) * n_cta - 1, total_units));
        while (b > 0 && range(b) > blk) --b;
        while (b + 1 < n_cta && range(b + 1) <= blk) ++b;
        return b;
      };
      a.plan[(int64_t)seq * hkv + kvh] =
          whole ? make_int2(-1, -1) : make_int2(blockIdx.x, owner(item1 - 1));
    }
    __syncthreads();  // shared memory goes to the next item
    pos = stop;
  }
}

// Joins an item's parts: out = sum_p w_p O_p / sum_p w_p l_p, w_p = 2^(m_p - max m).
// One row is shared by SPLIT warps, each with every SPLIT-th part and a running
// maximum of its own; eight parts' loads are under way at a time, as it is their
// latency that the join takes.
template <int D, int SPLIT>
__global__ void __launch_bounds__(128)
k_page_join(const AttnArgs a, int hkv, int width_rows) {
  constexpr int V = D / 32, AHEAD = 8;  // dims of a lane
  __shared__ float red[4][D + 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, part0 = warp % SPLIT;
  const int64_t e = (int64_t)blockIdx.x * (4 / SPLIT) + warp / SPLIT;
  const bool on = e < (int64_t)a.n_seqs * hkv * a.R;
  const int m = on ? (int)(e % a.R) : 0;
  const int64_t item = on ? e / a.R : 0;
  const int seq = (int)(item / hkv), kvh = (int)(item % hkv), j = m / a.G;
  int nq = a.q_lens ? a.q_lens[seq] : a.q_len;
  nq = max(0, min(nq, a.q_len));
  const int len = max(0, min(a.seq_lens[seq], width_rows));
  pdl_wait();
  const int2 pl = on ? a.plan[item] : make_int2(-1, -1);
  const bool live = pl.x >= 0 && j < nq;
  float top = -CUDART_INF_F, den = 0.f, acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  for (int c0 = pl.x + part0; live && c0 <= pl.y; c0 += AHEAD * SPLIT) {
    float2 ml[AHEAD], o[AHEAD][V / 2];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int c = c0 + k * SPLIT;
      const float *src = a.parts + (((int64_t)c * 2 + (c == pl.x ? 1 : 0)) * a.R + m) * (D + 4);
      const bool in = c <= pl.y;
      ml[k] = in ? *reinterpret_cast<const float2 *>(src + D) : make_float2(-CUDART_INF_F, 0.f);
#pragma unroll
      for (int i = 0; i < V / 2; ++i)
        o[k][i] = in ? *reinterpret_cast<const float2 *>(src + lane * V + 2 * i)
                     : make_float2(0.f, 0.f);
    }
    float now = top;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) now = fmaxf(now, ml[k].x);
    const float f0 = top == -CUDART_INF_F ? (den != den ? 1.f : 0.f) : ex2_approx(top - now);
    den *= f0;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] *= f0;
    top = now;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      // (a part that saw nothing weighs nothing; one of NaN scores has m = -inf too)
      const float f = ml[k].x == -CUDART_INF_F ? (ml[k].y != ml[k].y ? 1.f : 0.f)
                                               : ex2_approx(ml[k].x - now);
      den += ml[k].y * f;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        acc[2 * i] += o[k][i].x * f;
        acc[2 * i + 1] += o[k][i].y * f;
      }
    }
  }
  if (SPLIT > 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) red[warp][lane * V + i] = acc[i];
    if (lane == 0) {
      red[warp][D] = top;
      red[warp][D + 1] = den;
    }
    __syncthreads();
    if (part0 != 0) return;
    float all = top;
#pragma unroll
    for (int w = 1; w < SPLIT; ++w) all = fmaxf(all, red[warp + w][D]);
    den = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll
    for (int w = 0; w < SPLIT; ++w) {
      const float t = red[warp + w][D], d = red[warp + w][D + 1];
      const float f = t == -CUDART_INF_F ? (d != d ? 1.f : 0.f) : ex2_approx(t - all);
      den += d * f;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += red[warp + w][lane * V + i] * f;
    }
    top = all;
  }
  if (!live) return;
  const int sees = len - nq + j + 1;
  const float inv = 1.f / den;
  const int64_t row = ((int64_t)seq * a.q_len + j) * a.hq + kvh * a.G + (m - j * a.G);
#pragma unroll
  for (int i = 0; i < V; i += 2)
    *reinterpret_cast<uint32_t *>(a.out + row * D + lane * V + i) =
        sees <= 0 ? 0u : pack_bf16(acc[i] * inv, acc[i + 1] * inv);
  if (a.lse && lane == 0)
    a.lse[row] = top == CUDART_INF_F ? top
                 : den == 0.f        ? -CUDART_INF_F
                                     : (top + log2f(den)) * 0.69314718055994531f;
}

bool attend_args(const dhs_pages *pages, int32_t n_seqs, int32_t q_len, int32_t q_heads,
                 PageView *pg) {
  return page_view(pages, pg) && n_seqs >= 0 && n_seqs <= kMaxSeqs && q_len >= 1 &&
         q_len <= kMaxKmax && q_heads >= 1 && q_heads % pg->hkv == 0 &&
         (int64_t)q_len * (q_heads / pg->hkv) <= 128;
}

int64_t plan_bytes(int32_t n_seqs, int hkv) {
  return ((int64_t)n_seqs * hkv * 8 + 255) / 256 * 256;
}

// Calls f with the configuration for R rows.  8 rows take half of a row tile's
// softmax, 16 rows fit one warp and four token groups stream at once; more rows take
// more warps of the same tile, and above 64 two row tiles a warp.  With one token a
// sequence every row sees every position, and up to 16 rows of 8 bits, the usual
// decode, leave out what looks for others (128 x 100K int8: 451 -> 446 us).
template <int D, int KIND, class F>
auto pick_rows(int R, int q_len, F f) {
  if (KIND != DHS_PAGE_BF16 && q_len == 1 && R <= 16)
    return R <= 8 ? f(Cfg<D, KIND, 1, 1, 1, false>()) : f(Cfg<D, KIND, 1, 1, 2, false>());
  if (R <= 8) return f(Cfg<D, KIND, 1, 1, 1>());
  if (R <= 16) return f(Cfg<D, KIND, 1, 1, 2>());
  if (R <= 32) return f(Cfg<D, KIND, 2, 1, 2>());
  if (R <= 64) return f(Cfg<D, KIND, 4, 1, 2>());
  return f(Cfg<D, KIND, 4, 2, 2>());
}
template <class F>
auto pick(const PageView &pg, int R, int q_len, F f) {
  switch ((pg.d == 128 ? 4 : 0) + pg.kind) {
    case 0: return pick_rows<64, DHS_PAGE_BF16>(R, q_len, f);
    case 1: return pick_rows<64, DHS_PAGE_INT8>(R, q_len, f);
    case 2: return pick_rows<64, DHS_PAGE_E4M3>(R, q_len, f);
    case 4: return pick_rows<128, DHS_PAGE_BF16>(R, q_len, f);
    case 5: return pick_rows<128, DHS_PAGE_INT8>(R, q_len, f);
    default: return pick_rows<128, DHS_PAGE_E4M3>(R, q_len, f);
  }
}

}  // namespace

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
  return pick(pg, R, q_len, [&](auto c) -> int64_t {
    return plan_bytes(n_seqs, pg.hkv) + (int64_t)sms * decltype(c)::OCC * 2 * R * (pg.d + 4) * 4;
  });
}

extern "C" int dhs_page_attend(const dhs_pages *pages, const void *q, const int32_t *q_lens,
                               const int32_t *seq_lens, const int32_t *page_table,
                               int32_t table_width, int32_t n_seqs, int32_t q_len,
                               int32_t q_heads, float scale, void *out, float *lse,
                               void *workspace, int64_t workspace_bytes, int32_t *err,
                               dhs_stream stream) {
  using namespace dhs;
  PageView pg;
  if (!attend_args(pages, n_seqs, q_len, q_heads, &pg) || table_width < 0 || !(scale >= 0.f) ||
      scale > 1e38f || workspace_bytes < 0)
    return DHS_ERR_INVALID;
  if (n_seqs == 0) return DHS_OK;
  if (!q || !seq_lens || !page_table || !out || !workspace || ((uintptr_t)q & 15u) ||
      ((uintptr_t)out & 15u) || ((uintptr_t)workspace & 15u) ||
      !words(q_lens, seq_lens, page_table, lse, err))
    return DHS_ERR_INVALID;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return DHS_ERR_CUDA;
  }
  const int sms = device_sms(dev);
  if (sms < 1) return DHS_ERR_CUDA;
  AttnArgs a;
  a.q = static_cast<const uint16_t *>(q);
  a.q_lens = q_lens;
  a.seq_lens = seq_lens;
  a.table = page_table;
  a.out = static_cast<uint16_t *>(out);
  a.lse = lse;
  a.plan = static_cast<int2 *>(workspace);
  a.parts = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) +
                                      plan_bytes(n_seqs, pg.hkv));
  a.err = err;
  a.width = table_width;
  a.n_seqs = n_seqs;
  a.q_len = q_len;
  a.hq = q_heads;
  a.G = q_heads / pg.hkv;
  a.R = q_len * a.G;
  a.scale_log2 = (scale == 0.f ? 1.f / sqrtf((float)pg.d) : scale) * 1.4426950408889634f;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return pick(pg, a.R, q_len, [&](auto c) -> int {
    using C = decltype(c);
    const int grid = sms * C::OCC;
    if (workspace_bytes < plan_bytes(n_seqs, pg.hkv) + (int64_t)grid * 2 * a.R * (C::D + 4) * 4)
      return DHS_ERR_INVALID;
    static DeviceSmem granted;
    const int64_t rows = (int64_t)n_seqs * pg.hkv * a.R;
    if (rows > INT32_MAX) return DHS_ERR_CAPACITY;
    const int width_rows =
        (int)std::min<int64_t>((int64_t)table_width * pg.rows, (int64_t)INT32_MAX - 1024);
    // few rows: four warps a row
    const bool few = rows <= 4 * sms;
    const unsigned jgrid = (unsigned)(few ? rows : (rows + 3) / 4);
    if (granted.ensure(k_page_attn<C>, C::SMEM, dev) != cudaSuccess ||
        launch_prio(k_page_attn<C>, dim3(grid), dim3(kPaThreads), C::SMEM, s, pg, a) !=
            cudaSuccess ||
        launch_pdl(few ? k_page_join<C::D, 4> : k_page_join<C::D, 1>, dim3(jgrid), dim3(128), 0, s,
                   a, pg.hkv, width_rows) != cudaSuccess) {
      cudaGetLastError();
      return DHS_ERR_CUDA;
    }
    return DHS_OK;
  });
}
