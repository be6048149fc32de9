// Attention of a chunk of new tokens of every sequence over its paged cache, with or without
// a sliding window and first tokens that stay visible, on the fifth-generation tensor cores.
//
// A token at position p sees the positions t <= p with t > p - window or t < sinks (all t <= p
// without a window).  For kv head g the rows of the score matrix are (token, head) pairs, the
// G = q_heads / kv_heads heads of a token next to one another: 128 rows are tpt = 128 / G
// tokens, an item of work is two such row tiles (2 tpt consecutive tokens of one sequence) and
// the key tiles of 128 positions that any of them sees: those of the sinks and those from the
// window's start to the last token's place.
//   S_i = Q_i K^T (M 128, N 128, K D), P_i = 2^(c S_i - m_i), O_i += P_i V.
//
// Warps 0-7 and 8-15 are the softmax threads of row tile 0 and 1, two threads a row, each with
// half of a tile's columns; warp 16 issues all MMAs in the order P0 V(t), Q0 K(t+1), P1 V(t),
// Q1 K(t+1), so that the tensor cores work for one row tile while the other's softmax runs;
// P lies over S in tensor memory.  Warp 17 works out the items and fetches Q.  (The order of
// the products, the softmax and its bounded waits are those of the prompt kernel, and so are
// their reasons.)
//
// Pages.  A tile of 128 positions comes in boxes of the largest power of two that divides the
// page's rows: a box lies in one page, whichever page size there is.  A box of which no position
// is wanted, or whose page is not in the cache, is fetched from beyond the cache's end, which
// TMA fills with zeros, and so nothing is read that the page table does not name.
//
// bf16: the boxes go straight into the 128-byte-swizzled tiles that the MMAs read (warps 17
// and 19: an issued copy takes a warp some 55 cycles, and every instruction that a tile costs
// them ten or more beside the softmax); warp 18 sets values to 0 that are not
// finite and that some row does not see (0 times an infinity is not 0), and the rows that see
// them get them added at the end.
// 8 bits: three warps fetch the codes of keys and three those of values, and turn them into
// bf16, exactly, in the MMAs' tiles.  A key's scale
// multiplies its column of scores in 32 bits and a value's its column of weights before their
// one rounding to bf16, so that neither codes nor scales are rounded.
//
// Work split.  An item's cost is taken as the positions it walks and some tiles' worth for its
// own sake; all items' costs are laid end to end, sequence by sequence, and CTA b of n takes
// the b-th n-th.  An item cut by such a border is walked in parts by several CTAs, which leave
// (O, m, l) in the workspace for a join; a border near an item's end is moved there.  Every CTA
// so has the same work whatever the lengths are (one chunk of a long prompt beside sequences
// that decode one token), and the sums of costs have a closed form, so that a CTA finds its
// place by two searches.  Lengths are read on the device, and bits repeat.
//
// Measured, the two launches inside a captured graph (GB300, 1904 TFLOP/s and 6.77 TB/s
// measured, 1687 TFLOP/s held for seconds):
//   8192 new tokens at the end of 32768, 16 heads over 1, 128 dims: bf16 1.09 ms, 1757 TFLOP/s,
//   over the rate held under the power limit; int8 1.69, e4m3 1.76.  With codes the softmax
//   threads have the scales' products beside their own (a tile's chain is some 2400 cycles in
//   bf16, 1450 of them softmax) and share their issue slots with the warps that turn codes, which
//   are busy all the time.
//   64 dims: bf16 0.89 ms (S = Q K^T takes half the time, the softmax the same), int8 1.43.
//   64 sequences that decode one token each over up to 8192 positions, 32 heads over 8: bf16
//   218 us, 6.2 TB/s; int8 272, 2.56 TB/s, bound by turning codes that 4 rows make use of.
//   25 such sequences and chunks of 512 and 368 tokens: bf16 172 us, int8 237, e4m3 249.
//   4096 and 2485 new tokens in a window of 1024 with 4 sinks, 32 heads over 8, 64 dims: bf16
//   119 us, e4m3 149: items of some ten tiles, of which an item's start and end take as much
//   time as two and masks as much as two more.
//   77 new tokens at the end of 1100, 8 heads over 1: 20.5 us, latency from end to end.
#include "pages_internal.cuh"
#include "attn_tc.cuh"

#include <math_constants.h>

#include <algorithm>

namespace dhs {
namespace {

constexpr int kChSoftmax = 512;  // two row tiles, two warpgroups each
constexpr int kChM = 128, kChN = 128, kChH = kChN / 2;
constexpr int kChMma = 16, kChLoad = 17;
constexpr int kChClean = 18, kChLoadV = 19;  // bf16
constexpr int kChTurn = 18;                  // 8 bits: the first of six
// Microseconds that a wait lasts at most, and that a CTA's last ones do, for copies and
// products in flight.  In a build for tests the first is a variable.
constexpr uint32_t kChLastUs = 2000000;
#ifdef DHS_TEST_WAITS
}  // namespace
}  // namespace dhs
extern "C" uint32_t dhs_chunk_wait_us;
uint32_t dhs_chunk_wait_us = 2000000;
namespace dhs {
namespace {
#else
constexpr uint32_t dhs_chunk_wait_us = 2000000;
#endif
constexpr float kChRescale = 8.f;
constexpr uint32_t kChCols = 512;   // tensor memory: S0, S1 (P over them), O0, O1
constexpr int kChOver = 3 * kChN;   // what an item costs besides its positions
constexpr int kChLone = 3;          // quarters of a position's cost where there is one row tile
constexpr int kChLeast = 3 * kChN;  // cost of a CTA's share at least
// A border this many tiles from an item's end, or fewer, is moved there: an eighth of a share, 2
// to 8 tiles.  A cut costs what a CTA writes and the join reads for it, so long shares rather
// differ by as much (4096 and 2485 new tokens in a window of 1024, 32 heads over 8 of 64 dims,
// bf16: 143 us with 2 tiles at most, 119 with 8), short ones, whose time is the longest share's,
// do not.
constexpr int kChSnap = 2, kChSnapMost = 8, kChSnapPart = 8;

struct ChunkArgs {
  PageView pg;
  const int32_t *cu, *lens, *table;
  uint16_t *out;
  float *lse, *parts;        // parts: [CTAs][2][256][D]
  float2 *ml;                // [CTAs][2][256]: a row's maximum and sum
  int4 *plan;                // [CTAs][2]: the item that this CTA begins and others go on with
                             // (first token's row, tokens, kv head, last CTA or -1), and
                             // (first position, whether this CTA goes on with another's, -, -)
  int32_t *status;           // [CTAs]: a wait of the CTA ran out
  int32_t *err;
  int64_t n_tok, cap;        // cap: positions that an item's cost counts at most
  int n_seqs, width, most, hq, G, tpt, box, window, sinks;
  uint32_t wait_us;
  int out32;                 // out lies on 32-byte boundaries
  float scale_log2;
};

template <int D, int KIND>
struct ChCfg {
  static constexpr bool W8 = KIND != DHS_PAGE_BF16;
  static constexpr int HALVES = D / 64;
  static constexpr int TILE = 128 * D * 2;    // a Q, K or V tile as the MMAs read it
  static constexpr int HALF = 128 * 128;      // 64 dims of its 128 rows
  static constexpr int KS = D == 64 ? 4 : W8 ? 2 : 3, VS = D == 64 ? 4 : 2, SLOTS = KS + VS;
  // 32 rows of codes: of 64 bytes one after another, or, where each comes in a box of its own,
  // on the 128-byte boundaries that TMA writes to
  static constexpr int QUARTER = 32 * 128;
  static constexpr int TURN = W8 ? 3 : 0;     // warps that turn keys' codes, and values'
  static constexpr int THREADS = kChSoftmax + (W8 ? 256 : 128);
  // What the softmax threads know of a key tile: positions whose page is not in the cache, and
  // scales.  Tile m's is filled when its slot is free of tile m - KS, or, in 8 bits with its
  // codes, a tile sooner; by then the softmax is over with tile m - KS - 2 or m - KS - 3.
  static constexpr int NE = 8;
  static constexpr int ENTRY = 16 + (W8 ? 2 * 128 * 4 : 0);
  static constexpr int OFF_KV = 2 * TILE;
  static constexpr int OFF_RAW = OFF_KV + SLOTS * TILE;
  static constexpr int OFF_RED = OFF_RAW + 2 * TURN * QUARTER;  // float [2 tiles][2 halves][128]
  static constexpr int OFF_ENTRY = OFF_RED + 2 * 2 * 128 * 4;
  static constexpr int OFF_BAR = OFF_ENTRY + NE * ENTRY;
  static constexpr int CLEAN = 4;             // value tiles gone over and not yet used, at most
  static constexpr int BARS = 3 + 2 * SLOTS + (W8 ? 0 : CLEAN) + 2 * TURN + 8 + 4 + 8;
  static constexpr int OFF_TMEM = OFF_BAR + BARS * 8;
  // int [4]: abort, whether pages were missing, bad values by item parity
  static constexpr int OFF_MISC = OFF_TMEM + 16;
  static constexpr int OFF_ITEM = OFF_MISC + 16;  // ChunkItem [2]
  static constexpr int SMEM = OFF_ITEM + 2 * 64;
  static_assert(NE >= KS + (W8 ? 3 : 2), "entries of key tiles");
  static_assert(SMEM <= 227 * 1024, "shared memory of the chunk kernel");
};

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, int x, int y, int z,
                                            int w, void *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void cp_async_4_or_0(void *dst, const void *src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(smem_u32(dst)), "l"(src),
               "r"(bytes));
}

// Two codes a word (the bytes of a that `sel` names) as bf16, exactly.  int8: 0x43 over a code's
// bits is 128 + its lower seven, plus 128 more in the exponent if it is negative; less 128 or 256.
// e4m3: the lower seven bits at a bf16's exponent and mantissa are the value times 2^-120,
// subnormals included.
template <int KIND>
__device__ __forceinline__ uint32_t two_codes(uint32_t a, bool upper) {
  uint32_t r;
  if (KIND == DHS_PAGE_INT8) {
    const uint32_t t = __byte_perm(a, 0x43434343u, upper ? 0x4342 : 0x4140);
    asm("sub.rn.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(t & 0xFF7FFF7Fu), "r"(t & 0xFF80FF80u));
  } else {
    const uint32_t t = __byte_perm(a, 0u, upper ? 0x3424 : 0x1404);
    asm("mul.rn.bf16x2 %0, %1, %2;\n"
        : "=r"(r)
        : "r"((t & 0x80008000u) | ((t >> 4) & 0x07F007F0u)), "r"(0x7B807B80u));
  }
  return r;
}

// A sequence's first token, new tokens and what its positions are ahead of them; false
// (recorded) for offsets or a length out of range.
__device__ __forceinline__ bool chunk_seq(const ChunkArgs &a, int i, int &q0, int &nq, int &off,
                                          bool record) {
  q0 = a.cu[i];
  const int64_t q1 = a.cu[i + 1];
  const int len = a.lens[i];
  nq = off = 0;
  if (q0 < 0 || q1 < q0 || q1 > a.n_tok || (q1 > q0 && (len < 0 || len > a.most))) {
    if (record) page_error(a.err, DC_ROW_RANGE, DHS_SITE_PAGE_CHUNK);
    return false;
  }
  nq = (int)(q1 - q0);
  off = len - nq;
  return true;
}

// One piece of work: two row tiles of a sequence and key tiles that they walk, the j0-th and
// following of the item's list: tile n of the list is n (the sinks') below ns, n + gap from there.
struct ChunkItem {
  int row0, ntok, seq, kvh;  // the first token's row (< 0: no more work), tokens of the item
  int p0;                    // the first token's position
  int j0, n0, n1;            // of the list: first tile, and how many either row tile walks (one
                             // row tile of two tiles and more: see `dual` below)
  int ns, gap;
  int slot;                  // of the parts, or -1: the whole item
  int tiles;                 // key tiles of this CTA before this piece
};
static_assert(sizeof(ChunkItem) <= 64, "");

__device__ __forceinline__ int tile_of(int ns, int gap, int n) { return n < ns ? n : n + gap; }

// The pieces of CTA b, in order.  All lanes of a warp; what comes back is lane-uniform.
struct ChunkSchedule {
  const ChunkArgs &a;
  int lane, span, n_cta, hkv;
  int64_t begin, end, share;
  int rest;                        // all costs: share * n_cta + rest
  // the item to come: sequence, kv head, place in the sequence, where its cost starts
  int seq, kvh, r, q0, nq, off, R;
  int base, my_q0, my_nq, my_off;  // this lane's of 32 sequences
  int64_t at, per, m;
  // for the join
  int4 first;
  int first_pos, cont;

  // the items r < m of a sequence cost max(o, 0) + (r + 1) span, later ones the cap
  __device__ int64_t below_cap(int o) const {
    if (a.window == 0) return INT32_MAX;
    const int64_t left = a.cap - 1 - max(o, 0);
    return left < span ? 0 : (int64_t)((uint32_t)left / (uint32_t)span);
  }
  // cost of a sequence's first j items; a single row tile has two key tiles at a time
  __device__ int64_t upto(int j, int n, int o, int64_t m) const {
    const int64_t x = min((int64_t)j, m);
    if (n <= a.tpt) return j == 0 ? 0 : (x * (max(o, 0) + span) + (j - x) * a.cap) * kChLone / 4 + kChOver;
    return x * max(o, 0) + (int64_t)span * (x * (x + 1) / 2) + (j - x) * a.cap + (int64_t)j * kChOver;
  }
  __device__ int64_t cost_of(int i, bool record) const {
    int x0, n, o;
    if (i >= a.n_seqs || !chunk_seq(a, i, x0, n, o, record)) return 0;
    return upto((int)((uint32_t)(n + span - 1) / (uint32_t)span), n, o, below_cap(o)) * hkv;
  }
  __device__ int64_t border(int b) const {
    return share * b + (int64_t)((uint32_t)rest * (uint32_t)b / (uint32_t)n_cta);
  }
  __device__ void enter(int i) {  // sequence i is the one to come
    seq = i;
    kvh = r = 0;
    if (i < base || i >= base + 32) {
      base = i;
      my_q0 = my_nq = my_off = 0;
      if (i + lane < a.n_seqs) chunk_seq(a, i + lane, my_q0, my_nq, my_off, false);
    }
    q0 = __shfl_sync(0xffffffffu, my_q0, i - base);
    nq = __shfl_sync(0xffffffffu, my_nq, i - base);
    off = __shfl_sync(0xffffffffu, my_off, i - base);
    R = (int)((uint32_t)(nq + span - 1) / (uint32_t)span);
    m = below_cap(off);
    per = upto(R, nq, off, m);
  }
  __device__ ChunkSchedule(const ChunkArgs &args, int l) : a(args), lane(l) {
    span = 2 * a.tpt;
    hkv = a.pg.hkv;
    first = make_int4(0, 0, 0, -1);
    first_pos = cont = 0;
    base = -64;
    int64_t total = 0, mine = 0;
    for (int i = 0; i < a.n_seqs; i += 32) {
      mine = cost_of(i + lane, true);
      total += mine;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    n_cta = (int)min((int64_t)gridDim.x, (total + kChLeast - 1) / kChLeast);
    seq = a.n_seqs;
    at = begin = end = 0;
    if ((int)blockIdx.x >= n_cta) return;
    share = (total | n_cta) >> 32 ? total / n_cta : (int64_t)((uint32_t)total / (uint32_t)n_cta);
    rest = (int)(total - share * n_cta);
    begin = border(blockIdx.x);
    end = border(blockIdx.x + 1);
    // the sequence in which the share begins
    for (int i = 0; i < a.n_seqs; i += 32) {
      const int64_t c = a.n_seqs <= 32 ? mine : cost_of(i + lane, false);
      int64_t x = c;  // inclusive sums
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const uint32_t here = __ballot_sync(0xffffffffu, begin < at + x);
      if (here) {
        const int src = __ffs(here) - 1;
        at += __shfl_sync(0xffffffffu, x - c, src);
        enter(i + src);
        break;
      }
      at += __shfl_sync(0xffffffffu, x, 31);
    }
    if (seq >= a.n_seqs) return;
    kvh = (int)(((begin - at) | per) >> 32 ? (begin - at) / per
                                           : (int64_t)((uint32_t)(begin - at) / (uint32_t)per));
    at += kvh * per;
    int lo = 0, hi = R - 1;  // the last item that starts at or before `begin`
    while (lo < hi) {
      const int mid = (int)(((int64_t)lo + hi + 1) >> 1);
      if (at + upto(mid, nq, off, m) <= begin) lo = mid;
      else hi = mid - 1;
    }
    r = lo;
    at += upto(r, nq, off, m);
  }
  // (of an item of nt tiles that starts at `at` and costs c) the tile at which border x cuts it
  __device__ int cut(int64_t x, int64_t c, int nt) const {
    // (both CTAs at a border work out the same numbers)
    const int t = min(nt, (int)((float)nt * ((float)(x - at) / (float)c)));
    const int snap = (int)max((int64_t)kChSnap, min((int64_t)kChSnapMost, share / (kChSnapPart * kChN)));
    return t < snap ? 0 : nt - t < snap ? nt : t;
  }
  __device__ bool next(ChunkItem &it) {
    while (seq < a.n_seqs && at < end) {
      const int64_t c = R > 0 ? upto(r + 1, nq, off, m) - upto(r, nq, off, m) : 0;
      bool own = false;
      if (R > 0) {
        const int tok0 = r * span, ntok = min(span, nq - tok0), p0 = off + tok0;
        // tiles before the end of what either row tile's last token sees
        const int e0 = (max(0, p0 + min(a.tpt, ntok)) + kChN - 1) / kChN;
        const int e1 = (max(0, p0 + ntok) + kChN - 1) / kChN;
        int ns = 0, w0 = 0;  // tiles of the sinks, the window's first
        if (a.window > 0) {
          ns = (int)(((int64_t)a.sinks + kChN - 1) / kChN);
          w0 = max(ns, (int)(max((int64_t)0, (int64_t)p0 - a.window + 1) / kChN));
        }
        auto listed = [&](int e) { return min(e, ns) + max(0, e - w0); };
        const int l0 = listed(e0), nt = listed(e1);
        const int lo = at < begin ? cut(begin, c, nt) : 0;
        const int hi = at + c > end ? cut(end, c, nt) : nt;
        own = lo < hi || (nt == 0 && at >= begin);
        if (own) {
          const bool whole = lo == 0 && hi == nt;
          it.row0 = q0 + tok0;
          it.ntok = ntok;
          it.seq = seq;
          it.kvh = kvh;
          it.p0 = p0;
          it.j0 = lo;
          it.n0 = max(0, min(l0, hi) - lo);
          it.n1 = ntok > a.tpt ? hi - lo : 0;
          it.ns = ns;
          it.gap = w0 - ns;
          it.slot = whole ? -1 : lo > 0 ? 0 : 1;
          if (!whole && lo > 0) cont = 1;
          if (!whole && lo == 0) {
            // the last CTA that has some of this item
            int b = min(n_cta - 1, (int)((float)(at + c) / (float)max((int64_t)1, share)));
            while (b > 0 && border(b) >= at + c) --b;
            while (b + 1 < n_cta && border(b + 1) < at + c) ++b;
            first = make_int4(it.row0, ntok, kvh, b);
            first_pos = p0;
          }
        }
      }
      // on to the next one
      at += c;
      if (++r >= R) {
        r = 0;
        if (R == 0 || ++kvh >= hkv) enter(seq + 1);
      }
      if (own) return true;
    }
    return false;
  }
};

template <int D, int KIND, bool WIN>
__global__ void __launch_bounds__(ChCfg<D, KIND>::THREADS, 1)
k_chunk(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
        const __grid_constant__ CUtensorMap mv, const __grid_constant__ ChunkArgs a) {
  using C = ChCfg<D, KIND>;
  constexpr bool W8 = C::W8;
  // no static shared memory: the dynamic part starts on the boundary it asks for
  extern __shared__ __align__(1024) unsigned char smem[];
  int *misc = reinterpret_cast<int *>(smem + C::OFF_MISC);
  volatile int *abort_v = misc, *missing = misc + 1, *bad_values = misc + 2;
  auto item_of = [&](int k) -> ChunkItem & {
    return *reinterpret_cast<ChunkItem *>(smem + C::OFF_ITEM + (k & 1) * 64);
  };
  if ((smem_u32(smem) & 1023u) != 0u) {  // (the swizzle pattern follows address bits)
    pdl_wait();
    if (threadIdx.x == 0) {
      a.status[blockIdx.x] = 1;
      a.plan[2 * blockIdx.x] = make_int4(0, 0, 0, -1);
    }
    page_error(a.err, DC_CAPACITY, DHS_SITE_PAGE_CHUNK);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
  uint64_t *q_full = bars, *q_empty = bars + 1, *mma_done = bars + 2, *full = bars + 3,
           *empty = full + C::SLOTS, *clean = empty + C::SLOTS, *raw = clean + (W8 ? 0 : C::CLEAN);
  uint64_t *s_full = raw + 2 * C::TURN, *p_full = s_full + 2, *pv_done = s_full + 4,
           *o_empty = s_full + 6, *item_full = s_full + 8, *item_empty = s_full + 10,
           *half_in = s_full + 12, *half_read = s_full + 16;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_TMEM);
  if (tid == kChLoad * 32) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(mma_done, 1);
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(&full[i], W8 ? 4 : 1);          // 8 bits: a tile's quarters
      mbar_init(&empty[i], 1);
    }
    if (!W8)
      for (int i = 0; i < C::CLEAN; ++i) mbar_init(&clean[i], 1);
    for (int i = 0; i < 2 * C::TURN; ++i) mbar_init(&raw[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kChSoftmax / 64);   // one arrival per warp
      mbar_init(&pv_done[i], 1);
      mbar_init(&o_empty[i], kChSoftmax / 64);
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], C::THREADS / 32 - 1);  // all warps but the loader's
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&half_in[i], 2);
      mbar_init(&half_read[i], 2);
      misc[i] = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    fence_proxy_async_smem();
  }
  if (tid == kChLoad * 32 + 1) {
    tma_prefetch(&mq);
    tma_prefetch(&mk);
    tma_prefetch(&mv);
  }
  pdl_wait();  // (what is above needs nothing of the launch before, nor takes what it may want)
  if (warp == kChMma) tmem_alloc(tmem_slot, kChCols);
  pdl_trigger();  // the join may be placed; it waits for this grid's end
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0u;  // all 512 columns are this CTA's

  // (whether what is waited for has come)
  auto wait = [&](uint64_t *bar, uint32_t parity, bool force = false) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint32_t since = global_us();
    do {
      if (!force && *abort_v) return false;
      if (global_us() - since >= (force ? kChLastUs : a.wait_us)) {
        page_error(a.err, DC_TIMEOUT, DHS_SITE_PAGE_CHUNK);
        *abort_v = 1;
        return false;
      }
    } while (!mbar_try_wait(bar, parity));
    return true;
  };
  auto given_up = [&]() { return __any_sync(0xffffffffu, *abort_v) != 0; };
  // Slot of the n-th K or V tile since the start, and the parity of its use.  (All counts run
  // over a CTA's pieces: every wait is for the phase after the one waited for last.)
  auto kslot = [&](uint32_t n) { return n % C::KS; };
  auto vslot = [&](uint32_t n) { return C::KS + n % C::VS; };
  auto kpar = [&](uint32_t n) { return (n / C::KS) & 1u; };
  auto vpar = [&](uint32_t n) { return (n / C::VS) & 1u; };
  auto item_par = [&](int k) { return (uint32_t)(k >> 1) & 1u; };
  auto bad_of = [&](uint32_t n) {
    return reinterpret_cast<uint32_t *>(smem + C::OFF_ENTRY + (n % C::NE) * C::ENTRY);
  };
  auto scales_of = [&](uint32_t n) { return reinterpret_cast<float *>(bad_of(n) + 4); };
  // the k-th piece, read and released by every warp but the loader's
  auto take = [&](int k) {
    wait(&item_full[k & 1], item_par(k));
    __syncwarp();
    const ChunkItem it = item_of(k);
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_empty[k & 1]);
    return it;
  };
  // The page of position `pos` of a piece's sequence as the table has it (INT32_MIN: none of
  // the positions up to `to` is wanted) and the row in it; asked for a tile ahead of its use.
  auto ask = [&](const ChunkItem &it, int pos, int to, int &in) {
    const bool want = pos <= it.p0 + it.ntok - 1 && (!WIN || to > it.p0 - a.window || pos < a.sinks);
    const int pg = (int)((uint64_t)(uint32_t)pos * a.pg.div_mul >> a.pg.div_shift);
    in = pos - pg * a.pg.rows;
    return want ? a.table[(int64_t)it.seq * a.width + pg] : INT32_MIN;
  };
  const uint32_t pages = (uint32_t)a.pg.n_pages;
  auto there = [&](int page) { return (uint32_t)page < pages; };
  // bf16: the boxes of a key or value tile; a lane has box lane, lane + 32, ...  (One warp has
  // some 2300 cycles for all that it does for a tile, so the usual case, pages of which no more
  // than 32 boxes make a tile, passes by the others.)
  const int boxes = kChN / a.box;
  struct Boxes {
    int page[4], in[4];
  };
  auto ask_tile = [&](const ChunkItem &it, int n, Boxes &b) {
    const int pos = tile_of(it.ns, it.gap, it.j0 + n) * kChN + lane * a.box;
    b.page[0] = INT32_MIN;
    if (lane < boxes) b.page[0] = ask(it, pos, pos + a.box - 1, b.in[0]);
    if (boxes > 32) {
#pragma unroll
      for (int r = 1; r < 4; ++r) {
        b.page[r] = INT32_MIN;
        const int p = pos + 32 * r * a.box;
        if (lane + 32 * r < boxes) b.page[r] = ask(it, p, p + a.box - 1, b.in[r]);
      }
    }
  };
  auto fetch_tile = [&](const ChunkItem &it, const CUtensorMap *map, uint32_t slot, const Boxes &b) {
    if (lane == 0) mbar_arrive_expect_tx(&full[slot], (uint32_t)C::TILE);
    unsigned char *to = smem + C::OFF_KV + slot * C::TILE + lane * a.box * 128;
    auto box = [&](int r) {
      const int page = there(b.page[r]) ? b.page[r] : (int)pages;
#pragma unroll
      for (int h = 0; h < C::HALVES; ++h)
        tma_load_4d(to + h * C::HALF + 32 * r * a.box * 128, map, h * 64, b.in[r], it.kvh, page,
                    &full[slot]);
    };
    if (lane < boxes) box(0);
    if (boxes > 32) {
#pragma unroll
      for (int r = 1; r < 4; ++r)
        if (lane + 32 * r < boxes) box(r);
    }
    __syncwarp();
  };

  // (8 bits: of the 80 registers a thread at launch, 512 x 96 and 256 x 48 are made; every warp
  // of a warpgroup asks in the same place)
  if (warp >= kChMma) {
  if (W8) asm volatile("setmaxnreg.dec.sync.aligned.u32 48;\n");
  if (warp == kChLoad) {
    // --------------------------------------------------- pieces and Q, in bf16 also K
    ChunkSchedule plan(a, lane);
    uint32_t kn = 0, qn = 0, tiles = 0;
    for (int k = 0;; ++k) {
      ChunkItem it = {};
      const bool more = plan.next(it);
      if (!more) it.row0 = -1;
      it.tiles = (int)tiles;
      if (k >= 2) wait(&item_empty[k & 1], item_par(k) ^ 1u);
      __syncwarp();
      if (given_up()) break;
      if (lane == 0) {
        item_of(k) = it;
        mbar_arrive(&item_full[k & 1]);
      }
      if (!more) break;
      const int nt = max(it.n0, it.n1);
      tiles += nt;
      if (lane == 0 && nt > 0) {  // (qn is this lane's alone)
        const int ntile = it.n1 > 0 ? 2 : 1;
        if (qn > 0) wait(q_empty, (qn - 1) & 1u);
        if (!*abort_v) {
          mbar_arrive_expect_tx(q_full, (uint32_t)(ntile * C::HALVES * a.G * a.tpt * 128));
          for (int i = 0; i < ntile; ++i)
            for (int h = 0; h < C::HALVES; ++h)
              tma_load_3d(smem + i * C::TILE + h * C::HALF, &mq, h * 64, it.kvh * a.G,
                          it.row0 + i * a.tpt, q_full);
          ++qn;
        }
      }
      __syncwarp();
      if (given_up()) break;
      if (!W8 && nt > 0) {
        Boxes now, next;
        ask_tile(it, 0, next);
        for (int n = 0; n < nt; ++n) {
          now = next;
          if (n + 1 < nt) ask_tile(it, n + 1, next);
          if (kn >= (uint32_t)C::KS) wait(&empty[kslot(kn)], kpar(kn) ^ 1u);
          if (given_up()) break;
          // wanted positions that are not there
          uint32_t *e = bad_of(kn);
          if (lane == 0) *reinterpret_cast<uint4 *>(e) = make_uint4(0u, 0u, 0u, 0u);
          auto gone = [&](int r) { return now.page[r] != INT32_MIN && !there(now.page[r]); };
          if (__any_sync(0xffffffffu, gone(0) || (boxes > 32 && (gone(1) || gone(2) || gone(3))))) {
            __syncwarp();
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (lane + 32 * r < boxes && gone(r)) {
                page_error(a.err, DC_LOC_RANGE, DHS_SITE_PAGE_CHUNK);
                *missing = 1;
                for (int x = (lane + 32 * r) * a.box; x < (lane + 32 * r + 1) * a.box; ++x)
                  atomicOr(&e[x >> 5], 1u << (x & 31));
              }
            __syncwarp();
          }
          fetch_tile(it, &mk, kslot(kn), now);
          ++kn;
        }
        if (given_up()) break;
      }
    }
    if (lane == 0) {
      a.plan[2 * blockIdx.x] = plan.first;
      a.plan[2 * blockIdx.x + 1] = make_int4(plan.first_pos, plan.cont, 0, 0);
      // every copy has landed before the CTA ends
      if (qn > 0) wait(q_full, (qn - 1) & 1u, true);
      for (uint32_t i = kn > C::KS ? kn - C::KS : 0; i < kn; ++i) wait(&full[kslot(i)], kpar(i), true);
    }
    __syncwarp();
  } else if (warp == kChMma) {
    // ----------------------------------------------------------------- products
    constexpr uint32_t kIdescQK = tc_idesc_bf16(kChM, kChN, 0, 0);
    constexpr uint32_t kIdescPV = tc_idesc_bf16(kChM, D, 0, 1);
    const uint32_t sQ = smem_u32(smem), sKV = smem_u32(smem + C::OFF_KV);
    auto qk = [&](int i, uint32_t c, int of) {  // row tile i, whose Q is the `of`-th
      const uint64_t q = tc_desc_sw128(sQ + of * C::TILE, 16, 1024);
      const uint64_t k = tc_desc_sw128(sKV + kslot(c) * C::TILE, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t o = ((kk >> 2) * C::HALF + (kk & 3) * 32) >> 4;
        warp_mma(i * kChN, q + o, k + o, kIdescQK, kk);
      }
      warp_commit(&s_full[i]);
    };
    auto pv = [&](int i, uint32_t c, int n) {
      const uint64_t v = tc_desc_sw128(sKV + vslot(c) * C::TILE, C::HALF, 1024);
#pragma unroll
      for (int kk = 0; kk < kChN / 16; ++kk)
        warp_mma_ta(2 * kChN + i * D, i * kChN + kk * 8, v + kk * 128, kIdescPV, n | kk);
    };
    uint32_t kn = 0, vn = 0, qn = 0, pn[2] = {0, 0}, on[2] = {0, 0};
    for (int k = 0;; ++k) {
      const ChunkItem it = take(k);
      if (given_up() || it.row0 < 0) break;
      const int nt = max(it.n0, it.n1);
      if (nt == 0) continue;
      const bool dual = it.n1 == 0 && nt > 1;
      auto values_in = [&]() {
        if (W8) wait(&full[vslot(vn)], vpar(vn));
        else wait(&clean[vn % C::CLEAN], (vn / C::CLEAN) & 1u);
      };
      auto key_in = [&](uint32_t c) {
        wait(&full[kslot(c)], kpar(c));
        __syncwarp();
        tc_fence_after();
      };
      auto weights_in = [&](int i) {
        wait(&p_full[i], pn[i] & 1u);
        ++pn[i];
        __syncwarp();
        tc_fence_after();
      };
      // (the last piece's O has been read, before the first product over it)
      auto o_free = [&](int i) {
        if (on[i] > 0) wait(&o_empty[i], (on[i] - 1) & 1u);
        ++on[i];
      };
      wait(q_full, qn & 1u);
      ++qn;
      key_in(kn);
      if (dual) {
        // one row tile: its even and odd key tiles are walked as two, side by side, and
        // put together by the softmax threads
        qk(0, kn, 0);
        warp_commit(&empty[kslot(kn)]);
        ++kn;
        key_in(kn);
        qk(1, kn, 0);
        warp_commit(&empty[kslot(kn)]);
        ++kn;
        if (nt == 2) warp_commit(q_empty);
        for (int n = 0; n < nt; ++n) {
          if ((n & 15) == 15 && given_up()) break;
          values_in();
          auto step = [&](int i) {
            // (what is here already is waited for first: only the weights' wait is long.  Keys
            // in 8 bits may not be here yet)
            if (n < 2) o_free(i);
            if (!W8 && n + 2 < nt) key_in(kn);
            weights_in(i);
            pv(i, vn, n >> 1);
            if (n + 2 >= nt) warp_commit(&pv_done[i]);
            warp_commit(&empty[vslot(vn)]);
            ++vn;
            if (n + 2 < nt) {
              if (W8) key_in(kn);
              qk(i, kn, 0);
              warp_commit(&empty[kslot(kn)]);
              ++kn;
              if (n + 3 == nt) warp_commit(q_empty);
            }
          };
          if (n & 1) step(1);
          else step(0);
        }
        continue;
      }
      if (it.n0 > 0) qk(0, kn, 0);
      if (it.n1 > 0) qk(1, kn, 1);
      warp_commit(&empty[kslot(kn)]);
      if (nt == 1) warp_commit(q_empty);
      ++kn;
      for (int n = 0; n < nt; ++n) {
        if ((n & 15) == 15 && given_up()) break;
        // (bf16: as above.  8192 tokens over 32768 of 64 dims 0.91 -> 0.89 ms, 128 dims the same.
        // With a warp for each row tile's MMAs the two tiles' products interleave, and each is there
        // later: 1.13 -> 1.49 ms)
        values_in();
        if (!W8 && n + 1 < nt) key_in(kn);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int ni = i ? it.n1 : it.n0;
          if (n < ni) {
            if (n == 0) o_free(i);
            weights_in(i);
            pv(i, vn, n);
            if (n + 1 == ni) warp_commit(&pv_done[i]);
          }
          if (n + 1 < ni) {
            if (W8) key_in(kn);
            qk(i, kn, i);
          }
        }
        warp_commit(&empty[vslot(vn)]);
        ++vn;
        if (n + 1 < nt) {
          warp_commit(&empty[kslot(kn)]);
          ++kn;
          if (n + 2 == nt) warp_commit(q_empty);
        }
      }
    }
    warp_commit(mma_done);
    wait(mma_done, 0u, true);
    __syncwarp();
  } else if (W8 && warp >= kChTurn) {
    // ---------------- 8 bits: keys (warps 18, 20, 21) and values (19, 22, 23) into bf16
    // A warp has every third quarter and room for one: its codes are fetched while the other
    // two warps work.
    const bool v = warp == 19 || warp >= 22;
    const uint32_t mine = warp < 20 ? 0 : warp < 22 ? warp - 19 : warp - 21;
    unsigned char *room = smem + C::OFF_RAW + ((v ? C::TURN : 0) + mine) * C::QUARTER;
    uint64_t *landed = &raw[(v ? C::TURN : 0) + mine];
    const int pitch = D == 64 && a.box == 1 ? 128 : D;
    // 16 codes at a time: chunk y of a row's 64 dims.  8 lanes that go together have rows x and
    // x ^ 5, so that they meet no bank twice, neither among the codes (128-byte rows are swizzled)
    // nor where the 32 bytes go as bf16.
    const int y = lane & 3, xl = (lane >> 3) ^ (lane & 4 ? 5 : 0);
    const uint32_t from = xl * pitch + (D == 128 ? y ^ xl : y) * 16;
    const uint32_t to0 = xl * 128 + (((2 * y) ^ xl) << 4), to1 = to0 ^ 16;
    uint32_t tn = 0, used = 0, issued = 0;  // tiles; quarters of this warp
    for (int k = 0;; ++k) {
      const ChunkItem it = take(k);
      if (given_up() || it.row0 < 0) break;
      const uint32_t end = 4 * (tn + max(it.n0, it.n1));
      auto place = [&](uint32_t g) {  // this lane's position of quarter g
        return tile_of(it.ns, it.gap, it.j0 + (int)((g >> 2) - tn)) * kChN + 32 * (int)(g & 3) + lane;
      };
      // the first quarter of this warp's in the piece, its pages and those of the next
      uint32_t g = 4 * tn + (mine + 3 - (4 * tn) % 3) % 3;
      int in = 0, in1 = 0, page = INT32_MIN, page1 = INT32_MIN;
      if (g < end) page = ask(it, place(g), place(g), in);
      if (g + 3 < end) page1 = ask(it, place(g + 3), place(g + 3), in1);
      auto fetch = [&](uint32_t g) {  // codes and scales of quarter g, whose page is known
        if (g < end) {
          const bool ok = there(page);
          const uint32_t c = g >> 2;
          const int q = g & 3;
          if (!v) {  // (the softmax wants both scales with the keys)
            const bool gone = page != INT32_MIN && !ok;
            if (gone) {
              page_error(a.err, DC_LOC_RANGE, DHS_SITE_PAGE_CHUNK);
              *missing = 1;
            }
            const uint32_t bad = __ballot_sync(0xffffffffu, gone);
            if (lane == 0) bad_of(c)[q] = bad;
            const int64_t row = ok ? ((int64_t)page * a.pg.hkv + it.kvh) * a.pg.rows + in : 0;
            float *to = scales_of(c) + 32 * q + lane;
            cp_async_4_or_0(to, a.pg.ks + row, ok ? 4 : 0);
            cp_async_4_or_0(to + 128, a.pg.vs + row, ok ? 4 : 0);
          }
          // a box is in one page: any of its positions that is there tells which
          const int first = lane & ~(a.box - 1);
          const uint32_t all = a.box == 32 ? ~0u : (1u << a.box) - 1u;
          const uint32_t in_box = (__ballot_sync(0xffffffffu, ok) >> first) & all;
          const int of = __shfl_sync(0xffffffffu, page, first + max(0, __ffs(in_box) - 1));
          if (lane == 0) mbar_arrive_expect_tx(landed, (uint32_t)(32 * D));
          __syncwarp();
          if (lane == first)
            tma_load_4d(room + lane * pitch, v ? &mv : &mk, 0, in, it.kvh,
                        in_box ? of : (int)pages, landed);
          ++issued;
        }
        cp_async_commit();
        page = page1;
        in = in1;
        page1 = g + 6 < end ? ask(it, place(g + 6), place(g + 6), in1) : INT32_MIN;
      };
      fetch(g);
      for (; g < end; g += 3) {
        const uint32_t c = g >> 2, slot = v ? vslot(c) : kslot(c);
        wait(landed, used & 1u);
        if (c >= (uint32_t)(v ? C::VS : C::KS)) wait(&empty[slot], (v ? vpar(c) : kpar(c)) ^ 1u);
        __syncwarp();
        if (given_up()) break;
        ++used;
        unsigned char *dst = smem + C::OFF_KV + slot * C::TILE + (g & 3) * (32 * 128);
        constexpr int B = D == 128 ? 4 : 2;  // chunks at a time: half of the quarter
        uint4 w[B];
        auto read = [&](int part) {
#pragma unroll
          for (int e = 0; e < B; ++e)
            w[e] = *reinterpret_cast<const uint4 *>(
                room + (D == 128 ? (from ^ ((e & 1) * 64)) + (2 * part + (e >> 1)) * 1024
                                 : from + (2 * part + e) * 8 * pitch));
        };
        auto write = [&](int part) {
#pragma unroll
          for (int e = 0; e < B; ++e) {
            uint4 lo, hi;
            lo.x = two_codes<KIND>(w[e].x, false);
            lo.y = two_codes<KIND>(w[e].x, true);
            lo.z = two_codes<KIND>(w[e].y, false);
            lo.w = two_codes<KIND>(w[e].y, true);
            hi.x = two_codes<KIND>(w[e].z, false);
            hi.y = two_codes<KIND>(w[e].z, true);
            hi.z = two_codes<KIND>(w[e].w, false);
            hi.w = two_codes<KIND>(w[e].w, true);
            unsigned char *at = dst + (D == 128 ? (e & 1) * C::HALF + (2 * part + (e >> 1)) * 1024
                                                : (2 * part + e) * 1024);
            *reinterpret_cast<uint4 *>(at + to0) = lo;
            *reinterpret_cast<uint4 *>(at + to1) = hi;
          }
        };
        read(0);
        write(0);
        read(1);
        __syncwarp();  // every lane has its codes
        fetch(g + 3);
        write(1);
        cp_async_wait_group<1>();  // this quarter's scales are in (the next one's may be under way)
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[slot]);
      }
      tn += max(it.n0, it.n1);
      if (given_up()) break;
    }
    cp_async_wait_all();
    // every copy has landed before the CTA ends
    if (used < issued) wait(landed, used & 1u, true);
    __syncwarp();
  } else if (!W8 && warp == kChLoadV) {
    // ------------------------------------------------------------- bf16: V's copies
    uint32_t vn = 0;
    for (int k = 0;; ++k) {
      const ChunkItem it = take(k);
      if (given_up() || it.row0 < 0) break;
      const int nt = max(it.n0, it.n1);
      Boxes now, next;
      if (nt > 0) ask_tile(it, 0, next);
      for (int n = 0; n < nt; ++n) {
        now = next;
        if (n + 1 < nt) ask_tile(it, n + 1, next);
        if (vn >= (uint32_t)C::VS) wait(&empty[vslot(vn)], vpar(vn) ^ 1u);
        if (given_up()) break;
        fetch_tile(it, &mv, vslot(vn), now);
        ++vn;
      }
      if (given_up()) break;
    }
    if (lane == 0)
      for (uint32_t i = vn > C::VS ? vn - C::VS : 0; i < vn; ++i) wait(&full[vslot(i)], vpar(i), true);
    __syncwarp();
  } else if (!W8 && warp == kChClean) {
    // ------------------------------------------------------------------- values
    uint32_t vn = 0;
    for (int k = 0;; ++k) {
      const ChunkItem it = take(k);
      if (given_up() || it.row0 < 0) break;
      const int last = it.p0 + it.ntok - 1;
      for (int n = 0; n < max(it.n0, it.n1); ++n, ++vn) {
        wait(&full[vslot(vn)], vpar(vn));
        if (given_up()) break;
        const int t0 = tile_of(it.ns, it.gap, it.j0 + n) * kChN;
        // rows of the tile that not every row of the item sees: [0, r1) below the window of
        // the last token (sinks excepted), and from r0 on, after the first token
        const int r0 = max(0, it.p0 + 1 - t0);
        const int r1 = WIN ? min(kChN, last - a.window + 1 - t0) : 0;
        if (r0 < kChN || r1 > 0) {
          unsigned char *v = smem + C::OFF_KV + vslot(vn) * C::TILE;
          // Row r's 64 dims of half h are the 128 bytes at h * HALF + r * 128.  An exponent
          // of ones plus one carries into the sign's place: eight values cost a dozen
          // instructions, and the slow loop runs only if some are not finite.
          auto some = [&](int x) { return x >= r0 || (WIN && x < r1 && t0 + x >= a.sinks); };
          uint32_t any = 0u;
#pragma unroll 8
          for (int e = lane; e < kChN * 8; e += 32) {
            if (!some(e >> 3)) continue;
#pragma unroll
            for (int h = 0; h < C::HALVES; ++h) {
              const uint4 w = *reinterpret_cast<const uint4 *>(v + h * C::HALF + e * 16);
              any |= (w.x & 0x7F807F80u) + 0x00800080u;
              any |= (w.y & 0x7F807F80u) + 0x00800080u;
              any |= (w.z & 0x7F807F80u) + 0x00800080u;
              any |= (w.w & 0x7F807F80u) + 0x00800080u;
            }
          }
          bool found = false;
          for (int e = lane; (any & 0x80008000u) != 0u && e < kChN * 8; e += 32) {
            if (!some(e >> 3)) continue;
#pragma unroll
            for (int h = 0; h < C::HALVES; ++h) {
              uint4 *at = reinterpret_cast<uint4 *>(v + h * C::HALF + e * 16);
              uint32_t w[4] = {at->x, at->y, at->z, at->w};
              bool bad = false;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if ((w[i] & 0x7F80u) == 0x7F80u) { w[i] &= 0xFFFF0000u; bad = true; }
                if ((w[i] & 0x7F800000u) == 0x7F800000u) { w[i] &= 0x0000FFFFu; bad = true; }
              }
              if (bad) {
                *at = make_uint4(w[0], w[1], w[2], w[3]);
                found |= t0 + (e >> 3) <= last;
              }
            }
          }
          if (found) bad_values[k & 1] = k + 1;
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&clean[vn % C::CLEAN]);
      }
    }
    __syncwarp();
  }
  } else {
    if (W8) asm volatile("setmaxnreg.inc.sync.aligned.u32 96;\n");
    // ------------------------------------------------------------------ softmax
    const int i = warp >> 3, hg = (warp >> 2) & 1, m = tid & 127;
    const int tloc = m / a.G, h = m - tloc * a.G;
    const int pair = 1 + i * 4 + (warp & 3);  // barrier of the two warps of these rows
    const uint32_t lrow = (uint32_t)((warp & 3) * 32) << 16;
    // this thread's half of the row's scores, and of its output columns
    const uint32_t tS = tmem + lrow + i * kChN + hg * kChH;
    const uint32_t tP = tmem + lrow + i * kChN + hg * (kChH / 2);
    const uint32_t tO = tmem + lrow + 2 * kChN + i * D + hg * (D / 2);
    float *red = reinterpret_cast<float *>(smem + C::OFF_RED) + i * 256;
    const float sl2 = a.scale_log2;
    const uint64_t sl22 = pack_f32x2(sl2, sl2);
    // Whether columns that no row of a warp sees are gone past.  In bf16 the branches cost every
    // tile more than that saves (8192 tokens over 32768 1.09 -> 1.15 ms, 64 dims 0.89 -> 0.96, in a
    // window 119 -> 124 us), in 8 bits with 128 dims and no window they save nothing; windowed
    // chunks in e4m3 take 149 us instead of 155 with them, long ones of 64 dims in int8 1.43 ms
    // instead of 1.73.
    constexpr bool SKIP = W8 && (WIN || D == 64);
    uint32_t sn = 0, pieces = 0, hn = 0;  // key tiles of this row tile; pieces walked as two halves
    for (int k = 0;; ++k) {
      // the piece stays in shared memory until its rows are written: few of its fields are
      // wanted in the loop, where registers are short
      wait(&item_full[k & 1], item_par(k));
      __syncwarp();
      volatile const ChunkItem &it = item_of(k);
      // (the warps of a pair leave together: they meet at barriers below, also after a wait
      // has run out)
      if (named_or(pair, 64, *abort_v != 0) || it.row0 < 0) break;
      // one row tile of several key tiles: row tile 0's threads have the even tiles, row tile
      // 1's the odd ones, of the same rows
      const bool dual = it.n1 == 0 && it.n0 > 1;
      const int ni = dual ? (it.n0 + 1 - i) >> 1 : i ? it.n1 : it.n0, ti = dual ? 0 : i;
      const int tstep = dual ? 2 : 1;
      int tile = it.j0 + (dual ? i : 0);      // of the list
      uint32_t en = (uint32_t)(it.tiles + (dual ? i : 0));  // the key tile's entry
      int lim0;  // columns of tile 0 that this row's half sees
      int least; // tiles from this one on have columns that some row does not see
      int wend = 0;  // tiles before this position have columns behind some row's window
      {
        const int tok = ti * a.tpt + tloc, ntok = it.ntok, p0 = it.p0;
        lim0 = (tloc < a.tpt && tok < ntok ? p0 + tok + 1 : 0) - hg * kChH;
        least = p0 + ti * a.tpt + 1;
        if (WIN) wend = max(p0, -1024) + min((ti + 1) * a.tpt, ntok) - a.window;
      }
      float m_run = -CUDART_INF_F, l = 0.f;
      const int ns = WIN ? it.ns : 0, gap = WIN ? it.gap : 0;
      for (int n = 0; n < ni; ++n, ++sn, en += tstep, tile += tstep) {
        wait(&s_full[i], sn & 1u);
        __syncwarp();
        tc_fence_after();
        uint32_t s0[32], s1[32];
        tmem_ld32(tS, s0);
        tmem_ld32(tS + 32, s1);
        tmem_wait_ld();
        const int first = (WIN ? tile_of(ns, gap, tile) : tile) * kChN;
        const float *sc = scales_of(en) + hg * kChH;
        uint2 out_of = make_uint2(0u, 0u);  // positions that are not there
        if (*missing) out_of = *reinterpret_cast<const uint2 *>(bad_of(en) + hg * 2);
        const bool masked = first + kChN > least || (out_of.x | out_of.y) != 0u ||
                            (WIN && first < wend && first + kChN > a.sinks);
        // Columns that this row does not see, and whether no row of the warp sees any of 32.  (A
        // warp's rows are few tokens: most groups of columns are seen by all of them or by none.)
        uint32_t hid0 = 0u, hid1 = 0u;
        bool none0 = false, none1 = false;
        if (masked) {
          const int lim = lim0 - first;  // columns below this one are not after the row
          auto below = [](int x) { return x <= 0 ? 0u : x >= 32 ? ~0u : (1u << x) - 1u; };
          hid0 = out_of.x | ~below(lim);
          hid1 = out_of.y | ~below(lim - 32);
          if (WIN) {
            const int w = lim - a.window, s = a.sinks - first - hg * kChH;
            hid0 |= below(w) & ~below(s);
            hid1 |= below(w - 32) & ~below(s - 32);
          }
          if (SKIP) {
            none0 = __all_sync(0xffffffffu, hid0 == ~0u);
            none1 = __all_sync(0xffffffffu, hid1 == ~0u);
          }
        }
        if (W8) {
          auto scaled = [&](uint32_t(&s)[32], const float *by) {
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              const float4 f = *reinterpret_cast<const float4 *>(by + c);
              float u, w;
              unpack_f32x2(mul_f32x2(pack_f32x2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])),
                                     pack_f32x2(f.x, f.y)), u, w);
              s[c] = __float_as_uint(u);
              s[c + 1] = __float_as_uint(w);
              unpack_f32x2(mul_f32x2(pack_f32x2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])),
                                     pack_f32x2(f.z, f.w)), u, w);
              s[c + 2] = __float_as_uint(u);
              s[c + 3] = __float_as_uint(w);
            }
          };
          if (!SKIP || !none0) scaled(s0, sc);
          if (!SKIP || !none1) scaled(s1, sc + 32);
        }
        if (masked) {
          auto hide = [](uint32_t(&s)[32], uint32_t hid) {
#pragma unroll
            for (int g = 0; g < 32; g += 8)
              if (!(WIN || SKIP) || __any_sync(0xffffffffu, (hid >> g & 0xFFu) != 0u)) {
#pragma unroll
                for (int c = g; c < g + 8; ++c)
                  if (hid >> c & 1u) s[c] = 0xFF800000u;
              }
          };
          hide(s0, hid0);
          hide(s1, hid1);
        }
        float mx0 = -CUDART_INF_F, mx1 = mx0;
#pragma unroll
        for (int c = 0; c < 32; c += 2) {  // (three-operand maxima)
          mx0 = max3(mx0, __uint_as_float(s0[c]), __uint_as_float(s0[c + 1]));
          mx1 = max3(mx1, __uint_as_float(s1[c]), __uint_as_float(s1[c + 1]));
        }
        float mx = fmaxf(mx0, mx1) * sl2;
        // The two warps that share 32 rows meet here, which also separates the halves'
        // reads of S from their writes of P.  Rows whose maximum grew much are rare:
        // only then do the halves exchange their maxima.
        if (named_or(pair, 64, mx > m_run + kChRescale)) {
          red[hg * 128 + m] = mx;
          named_sync(pair, 64);
          mx = fmaxf(mx, red[(hg ^ 1) * 128 + m]);
          named_sync(pair, 64);
          if (__any_sync(0xffffffffu, mx > m_run + kChRescale)) {
            const float m_new = fmaxf(m_run, mx);
            const float f = m_run == -CUDART_INF_F ? 0.f : ex2_approx(m_run - m_new);
            m_run = m_new;
            l *= f;
            if (n > 0) {  // (the product of tile n - 1 was complete before S of tile n)
#pragma unroll 1
              for (int c = 0; c < D / 2; c += 16) {
                uint32_t o[16];
                tmem_ld16(tO + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                tmem_st16(tO + c, o);
              }
            }
          }
        }
        // -inf - -inf must not arise in a row that has seen nothing
        const float b = m_run == -CUDART_INF_F ? 0.f : -m_run;
        uint64_t l2 = pack_f32x2(0.f, 0.f);
        const uint64_t b2 = pack_f32x2(b, b);
        uint32_t p[16];
        // weights (8 bits: times their value's scale) are rounded to bf16 for the product, at
        // most 2^-8 of each; l takes them unrounded
        auto weights = [&](const uint32_t(&s)[32], const float *by, uint32_t hid, bool none) {
          if (SKIP && none) {
#pragma unroll
            for (int x = 0; x < 16; ++x) p[x] = 0u;
            return;
          }
          float4 f4;
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            float u, w;
            unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[2 * x]),
                                              __uint_as_float(s[2 * x + 1])), sl22, b2), u, w);
            u = ex2_approx(u);
            w = ex2_approx(w);
            uint64_t two = pack_f32x2(u, w);
            l2 = add_f32x2(l2, two);
            if (W8) {
              if (x % 2 == 0) f4 = *reinterpret_cast<const float4 *>(by + 2 * x);
              unpack_f32x2(mul_f32x2(two, x % 2 ? pack_f32x2(f4.z, f4.w) : pack_f32x2(f4.x, f4.y)), u, w);
            }
            p[x] = pack_bf16(u, w);
          }
          if (W8 && masked) {
            // a scale that is not finite at a hidden place: 0 times it is NaN, which the sum shows
            uint32_t sum = p[0];
#pragma unroll
            for (int x = 1; SKIP && x < 16; ++x)
              asm("add.rn.bf16x2 %0, %0, %1;\n" : "+r"(sum) : "r"(p[x]));
            if (!SKIP || ((sum & 0x7F807F80u) + 0x00800080u) & 0x80008000u) {
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                if (hid >> (2 * x) & 1u) p[x] &= 0xFFFF0000u;
                if (hid >> (2 * x + 1) & 1u) p[x] &= 0x0000FFFFu;
              }
            }
          }
        };
        weights(s0, sc + 128, hid0, none0);
        tmem_st16(tP, p);
        weights(s1, sc + 160, hid1, none1);
        tmem_st16(tP + 16, p);
        {
          float l0, l1;
          unpack_f32x2(l2, l0, l1);
          l += l0 + l1;
        }
        tmem_wait_st();  // (of the rescaled O, too)
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[i]);
      }
      red[hg * 128 + m] = l;
      bool bad = false;
      if (ni > 0) {
        wait(&pv_done[i], pieces++ & 1u);
        __syncwarp();
        tc_fence_after();
      }
      if (dual && i == 1) {
        // this half's maximum, sum and O go to the threads of row tile 0
        named_sync(pair, 64);
        l += red[(hg ^ 1) * 128 + m];
        named_sync(pair, 64);
        red[hg * 128 + m] = hg ? l : m_run;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&half_in[warp & 3]);
        wait(&half_read[warp & 3], hn & 1u);
        ++hn;
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&o_empty[1]);
          mbar_arrive(&item_empty[k & 1]);
        }
        continue;
      }
      uint32_t o[D / 2];
      if (ni > 0) {
#pragma unroll
        for (int c = 0; c < D / 2; c += 32)
          tmem_ld32(tO + c, *reinterpret_cast<uint32_t(*)[32]>(&o[c]));
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_empty[i]);
      } else {
#pragma unroll
        for (int x = 0; x < D / 2; ++x) o[x] = 0u;
      }
      if (dual) {  // the other half is there
        wait(&half_in[warp & 3], hn & 1u);
        ++hn;
      }
      // Rows of a piece for which a wait ran out (whoever's it was: it is known by the time
      // what it waited for arrives here) are not written, nor half of them.
      const bool lost = named_or(pair, 64, *abort_v != 0);
      l += red[(hg ^ 1) * 128 + m];  // the row's sum over both halves
      // (read before this piece's place is given up: the one after next uses it again)
      bad = !W8 && bad_values[k & 1] == k + 1;
      if (dual) {
        tc_fence_after();
        const float m1 = red[256 + m], l1 = red[256 + 128 + m];
        const float top = fmaxf(m_run, m1);
        // (tiles that a row does not see weigh nothing; NaN scores have m = -inf too)
        const float f0 = m_run == -CUDART_INF_F ? (l != l ? 1.f : 0.f) : ex2_approx(m_run - top);
        const float f1 = m1 == -CUDART_INF_F ? (l1 != l1 ? 1.f : 0.f) : ex2_approx(m1 - top);
        m_run = top;
        l = l * f0 + l1 * f1;
#pragma unroll
        for (int c = 0; c < D / 2; c += 16) {
          uint32_t x[16];
          tmem_ld16(tO + D + c, x);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e)
            o[c + e] = __float_as_uint(__uint_as_float(o[c + e]) * f0 + __uint_as_float(x[e]) * f1);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&half_read[warp & 3]);
      }
      const int tok = ti * a.tpt + tloc, ntok = it.ntok, p0 = it.p0, slot = it.slot;
      const int row0 = it.row0, kvh = it.kvh, seq = it.seq, j0 = it.j0;
      const int walked = dual ? it.n0 : ni;
      const bool valid = tloc < a.tpt && tok < ntok && !lost;
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[k & 1]);
      if (valid && bad) {
        // values that were taken out, for the positions of this piece's tiles that this row sees
        const int pos = p0 + tok, last = p0 + ntok - 1;
        for (int n = 0; n < walked; ++n) {
          const int t0 = (WIN ? tile_of(ns, gap, j0 + n) : j0 + n) * kChN;
          const int from = WIN ? max(t0, 0) : max(t0, p0 + 1);
          for (int t = from; t < min(t0 + kChN, pos + 1); ++t) {
            if (WIN && t < a.sinks && t <= p0) continue;              // (every row sees it)
            if (WIN && t >= a.sinks && t <= pos - a.window) continue; // this one does not
            if (WIN && t <= p0 && t > last - a.window) continue;
            const int pg = (int)((uint64_t)(uint32_t)t * a.pg.div_mul >> a.pg.div_shift);
            const int page = a.table[(int64_t)seq * a.width + pg];
            if (page < 0 || page >= a.pg.n_pages) continue;
            const uint16_t *src =
                reinterpret_cast<const uint16_t *>(a.pg.v) +
                (((int64_t)page * a.pg.hkv + kvh) * a.pg.rows + (t - pg * a.pg.rows)) * D + hg * (D / 2);
#pragma unroll
            for (int x = 0; x < D / 2; ++x) {
              const uint32_t u = (uint32_t)src[x] << 16;
              if ((u & 0x7F800000u) == 0x7F800000u)
                o[x] = __float_as_uint(__uint_as_float(o[x]) + __uint_as_float(u));
            }
          }
        }
      }
      if (valid) {
        if (slot >= 0) {
          const int64_t place = ((int64_t)blockIdx.x * 2 + slot) * 256 + i * 128 + m;
          float *to = a.parts + place * D + hg * (D / 2);
#pragma unroll
          for (int x = 0; x < D / 2; x += 8)  // whole 32-byte sectors
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(to + x),
                         "r"(o[x]), "r"(o[x + 1]), "r"(o[x + 2]), "r"(o[x + 3]), "r"(o[x + 4]),
                         "r"(o[x + 5]), "r"(o[x + 6]), "r"(o[x + 7])
                         : "memory");
          if (hg == 0) a.ml[place] = make_float2(m_run, l);
        } else {
          const int64_t row = (int64_t)(row0 + tok) * a.hq + kvh * a.G + h;
          const bool sees = p0 + tok >= 0;
          const float inv = 1.f / l;  // only scores of -inf: 0 / 0
          uint16_t *to = a.out + row * D + hg * (D / 2);
#pragma unroll
          for (int x = 0; x < D / 2; x += 16) {
            uint32_t w[8];
#pragma unroll
            for (int y = 0; y < 8; ++y)
              w[y] = sees ? pack_bf16(__uint_as_float(o[x + 2 * y]) * inv,
                                      __uint_as_float(o[x + 2 * y + 1]) * inv)
                          : 0u;
            if (a.out32) {
              asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(to + x),
                           "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]),
                           "r"(w[6]), "r"(w[7])
                           : "memory");
            } else {
              *reinterpret_cast<uint4 *>(to + x) = make_uint4(w[0], w[1], w[2], w[3]);
              *reinterpret_cast<uint4 *>(to + x + 8) = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
          if (a.lse && hg == 0)
            a.lse[row] = m_run == CUDART_INF_F ? m_run
                         : l == 0.f            ? -CUDART_INF_F
                                               : (m_run + log2f(l)) * 0.69314718055994531f;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kChMma) tmem_dealloc(*tmem_slot, kChCols);
  if (tid == 0) a.status[blockIdx.x] = *abort_v;
}

// Joins the items' parts: sum_p w_p O_p / sum_p w_p l_p, w_p = 2^(m_p - max m).  Every block
// lists the items that were cut, and all warps share their rows, a row at a time.
constexpr int kChMostCtas = 256;
template <int D>
__global__ void __launch_bounds__(256)
k_chunk_join(const __grid_constant__ ChunkArgs a, int ctas) {
  constexpr int V = D / 32, AHEAD = 4;  // dims of a lane; parts under way at a time
  __shared__ int begun[kChMostCtas], counts[8];
  __shared__ unsigned char goes_on[kChMostCtas];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  // (in the order of the CTAs: all blocks go by the same list)
  bool begins = false, lost = false;
  if (threadIdx.x < ctas) {
    begins = a.plan[2 * threadIdx.x].w >= 0;
    goes_on[threadIdx.x] = a.plan[2 * threadIdx.x + 1].y != 0;
    lost = a.status[threadIdx.x] != 0;
  }
  const uint32_t some = __ballot_sync(0xffffffffu, begins);
  if (lane == 0) counts[warp] = __popc(some);
  // a wait that ran out in any CTA: no row is joined (which of them are whole is not known)
  if (__syncthreads_or(lost)) return;
  int cut = 0, at = 0;
  for (int w = 0; w < 8; ++w) {
    if (w == warp) at = cut;
    cut += counts[w];
  }
  if (begins) begun[at + __popc(some & ((1u << lane) - 1u))] = threadIdx.x;
  __syncthreads();
  for (int e = blockIdx.x * 8 + warp; e < cut * 256; e += gridDim.x * 8) {
    const int w = e % 256, i = w >> 7, m = w & 127, b = begun[e / 256];
    const int4 pl = a.plan[2 * b];
    const int tloc = m / a.G, h = m - tloc * a.G, tok = i * a.tpt + tloc;
    if (tloc >= a.tpt || tok >= pl.y) continue;
    float top = -CUDART_INF_F, den = 0.f, acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    for (int c0 = b; c0 <= pl.w; c0 += AHEAD) {
      float2 ml[AHEAD];
      float o[AHEAD][V];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int c = c0 + u;
        const bool in = c <= pl.w && (c == b || goes_on[c]);
        const int64_t place = ((int64_t)c * 2 + (c == b ? 1 : 0)) * 256 + w;
        ml[u] = in ? a.ml[place] : make_float2(-CUDART_INF_F, 0.f);
#pragma unroll
        for (int v = 0; v < V; v += 2) {
          const float2 y = in ? *reinterpret_cast<const float2 *>(a.parts + place * D + lane * V + v)
                              : make_float2(0.f, 0.f);
          o[u][v] = y.x;
          o[u][v + 1] = y.y;
        }
      }
      float now = top;
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) now = fmaxf(now, ml[u].x);
      // (a part that saw nothing weighs nothing; one of NaN scores has m = -inf too)
      const float f0 = top == -CUDART_INF_F ? (den != den ? 1.f : 0.f) : ex2_approx(top - now);
      den *= f0;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] *= f0;
      top = now;
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const float f = ml[u].x == -CUDART_INF_F ? (ml[u].y != ml[u].y ? 1.f : 0.f)
                                                 : ex2_approx(ml[u].x - now);
        den += ml[u].y * f;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] += o[u][v] * f;
      }
    }
    const int64_t row = (int64_t)(pl.x + tok) * a.hq + pl.z * a.G + h;
    const bool sees = a.plan[2 * b + 1].x + tok >= 0;
    const float inv = 1.f / den;
#pragma unroll
    for (int v = 0; v < V; v += 2)
      *reinterpret_cast<uint32_t *>(a.out + row * D + lane * V + v) =
          sees ? pack_bf16(acc[v] * inv, acc[v + 1] * inv) : 0u;
    if (a.lse && lane == 0)
      a.lse[row] = top == CUDART_INF_F ? top
                   : den == 0.f        ? -CUDART_INF_F
                                       : (top + log2f(den)) * 0.69314718055994531f;
  }
}

bool chunk_args(const dhs_pages *pages, int64_t n_tok, int32_t n_seqs, int32_t hq, PageView *pg) {
  return page_view(pages, pg) && n_tok >= 0 && n_tok <= INT32_MAX - 256 && n_seqs >= 0 &&
         n_seqs <= kMaxSeqs && hq >= 1 && hq % pg->hkv == 0 && hq / pg->hkv <= 128;
}

// CTAs of a call, one on an SM; 0 on failure.
int chunk_ctas(int dev) { return std::min(device_sms(dev), kChMostCtas); }

// Workspace of n CTAs: parts, their maxima and sums, plan and status; parts start at the next
// 32-byte boundary.
int64_t chunk_bytes(int n, int d) {
  return (int64_t)n * 2 * 256 * (d * 4 + 8) + (int64_t)n * (2 * 16 + 16) + 32;
}

// The cache's rows [page][kv head][page row][d], boxes of `box` rows: 64 bf16, or a row's
// codes; swizzled where that is 128 bytes.
bool encode_pages(EncodeTiled f, CUtensorMap *m, void *p, const PageView &pg, int box) {
  const bool w8 = pg.kind != DHS_PAGE_BF16;
  const cuuint64_t rb = (cuuint64_t)pg.d * (w8 ? 1 : 2);
  const cuuint64_t dims[4] = {(cuuint64_t)pg.d, (cuuint64_t)pg.rows, (cuuint64_t)pg.hkv,
                              (cuuint64_t)pg.n_pages};
  const cuuint64_t strides[3] = {rb, rb * pg.rows, rb * pg.rows * pg.hkv};
  const cuuint32_t b[4] = {w8 ? (cuuint32_t)pg.d : 64u, (cuuint32_t)box, 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return f(m, w8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, p, dims,
           strides, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
           w8 && pg.d == 64 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_queries(EncodeTiled f, CUtensorMap *m, const void *p, int64_t tokens, int heads, int d,
                    int64_t st, int64_t sh, int box_heads, int box_tokens) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)sh * 2, (cuuint64_t)st * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
  const cuuint32_t one[3] = {1, 1, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box, one,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How long a wait may take: as for prompts, 20 us for each key tile that an item can have and
// 5 us for each sequence beside two seconds; half an hour at most.
uint32_t chunk_wait_us(int64_t positions, int32_t n_seqs) {
  const uint64_t least = dhs_chunk_wait_us;
  return (uint32_t)std::min<uint64_t>(
      least + least * (uint64_t)(positions / kChN + 1) / 100000 + least * (uint64_t)n_seqs / 400000,
      1800000000u);
}

}  // namespace
}  // namespace dhs

extern "C" int64_t dhs_page_chunk_workspace(const dhs_pages *pages, int64_t n_tokens,
                                            int32_t n_seqs, int32_t q_heads) {
  using namespace dhs;
  PageView pg;
  if (!chunk_args(pages, n_tokens, n_seqs, q_heads, &pg)) return -1;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  const int ctas = chunk_ctas(dev);
  return ctas < 1 ? -1 : chunk_bytes(ctas, pg.d);
}

extern "C" int dhs_page_chunk(const dhs_pages *pages, const void *q, const int64_t *q_strides,
                              int64_t n_tokens, const int32_t *cu, const int32_t *seq_lens,
                              const int32_t *page_table, int32_t table_width, int32_t n_seqs,
                              int32_t q_heads, int32_t window, int32_t sinks, float scale, void *out,
                              float *lse, void *workspace, int64_t workspace_bytes, int32_t *err,
                              dhs_stream stream) {
  using namespace dhs;
  ChunkArgs a = {};
  if (!chunk_args(pages, n_tokens, n_seqs, q_heads, &a.pg) || table_width < 0 || window < 0 ||
      sinks < 0 || (sinks > 0 && window == 0) || !(scale >= 0.f) || scale > 1e38f ||
      workspace_bytes < 0)
    return DHS_ERR_INVALID;
  if (n_tokens == 0 || n_seqs == 0) return DHS_OK;
  if (!q || !cu || !seq_lens || !page_table || table_width < 1 || !out || !workspace ||
      ((uintptr_t)q & 15u) || ((uintptr_t)out & 15u) || ((uintptr_t)workspace & 15u) ||
      !words(cu, seq_lens, page_table, lse, err))
    return DHS_ERR_INVALID;
  const int64_t d = a.pg.d;
  int64_t st[2] = {q_heads * d, d};
  if (q_strides)
    for (int i = 0; i < 2; ++i) {
      const bool used = (i ? q_heads : n_tokens) > 1;
      if (q_strides[i] < 0 || q_strides[i] % 8 || q_strides[i] >= ((int64_t)1 << 38) ||
          (used && q_strides[i] < d))
        return DHS_ERR_INVALID;
      if (used) st[i] = q_strides[i];
    }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return DHS_ERR_CUDA;
  }
  const int ctas = chunk_ctas(dev);
  EncodeTiled enc = encoder();
  if (ctas < 1 || !enc) return DHS_ERR_CUDA;
  if (workspace_bytes < chunk_bytes(ctas, (int)d)) return DHS_ERR_INVALID;
  a.cu = cu;
  a.lens = seq_lens;
  a.table = page_table;
  a.out = static_cast<uint16_t *>(out);
  a.lse = lse;
  unsigned char *w = reinterpret_cast<unsigned char *>(((uintptr_t)workspace + 31) & ~(uintptr_t)31);
  a.parts = reinterpret_cast<float *>(w);
  a.ml = reinterpret_cast<float2 *>(w + (int64_t)ctas * 2 * 256 * d * 4);
  a.plan = reinterpret_cast<int4 *>(a.ml + (int64_t)ctas * 2 * 256);
  a.status = reinterpret_cast<int32_t *>(a.plan + 2 * ctas);
  a.err = err;
  a.n_tok = n_tokens;
  a.n_seqs = n_seqs;
  a.width = table_width;
  // (a tile's positions run up to 1024 past the last token, in 32 bits)
  a.most = (int)std::min<int64_t>((int64_t)table_width * a.pg.rows, (int64_t)INT32_MAX - 1024);
  a.hq = q_heads;
  a.G = q_heads / a.pg.hkv;
  a.tpt = kChM / a.G;
  a.box = 1;
  const int most_box = a.pg.kind == DHS_PAGE_BF16 ? 128 : 32;  // (a tile, a quarter)
  while (a.box < most_box && a.pg.rows % (2 * a.box) == 0) a.box *= 2;
  a.window = std::min(window, INT32_MAX - 1024);  // (no sequence is longer)
  a.sinks = sinks;
  a.cap = window > 0 ? std::min<int64_t>((int64_t)window + sinks + 2 * a.tpt + 2 * kChN, (int64_t)1 << 31)
                     : (int64_t)1 << 31;
  a.wait_us = chunk_wait_us(a.most, n_seqs);
  a.out32 = ((uintptr_t)out & 31u) == 0;
  a.scale_log2 = (scale == 0.f ? 1.f / sqrtf((float)d) : scale) * 1.4426950408889634f;
  // costs are summed in 64 bits and multiplied by tiles and CTAs
  const int64_t items = n_tokens / (2 * a.tpt) + std::min<int64_t>(n_seqs, n_tokens);
  if ((__int128)items * a.pg.hkv * (std::min<int64_t>(a.most, a.cap) + 4 * kChN) >= (__int128)1 << 53)
    return DHS_ERR_CAPACITY;
  CUtensorMap mq = {}, mk = {}, mv = {};
  if (!encode_queries(enc, &mq, q, n_tokens, q_heads, (int)d, st[0], st[1], a.G, a.tpt) ||
      !encode_pages(enc, &mk, a.pg.k, a.pg, a.box) || !encode_pages(enc, &mv, a.pg.v, a.pg, a.box))
    return DHS_ERR_INVALID;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto run = [&](auto kern, auto cfg, auto) -> cudaError_t {  // (one for each kernel: their types)
    using C = decltype(cfg);
    static DeviceSmem granted;
    cudaError_t e = granted.ensure(kern, C::SMEM, dev);
    if (e == cudaSuccess)
      e = launch_pdl(kern, dim3((unsigned)ctas), dim3(C::THREADS), (size_t)C::SMEM, s, mq, mk, mv, a);
    return e;
  };
  auto kinds = [&](auto dim, auto win) -> cudaError_t {
    constexpr int D = decltype(dim)::value;
    constexpr bool W = decltype(win)::value;
    cudaError_t e;
    switch (a.pg.kind) {
      case DHS_PAGE_BF16: e = run(k_chunk<D, DHS_PAGE_BF16, W>, ChCfg<D, DHS_PAGE_BF16>(), win); break;
      case DHS_PAGE_INT8: e = run(k_chunk<D, DHS_PAGE_INT8, W>, ChCfg<D, DHS_PAGE_INT8>(), win); break;
      default: e = run(k_chunk<D, DHS_PAGE_E4M3, W>, ChCfg<D, DHS_PAGE_E4M3>(), win); break;
    }
    if (e == cudaSuccess)
      e = launch_pdl(k_chunk_join<D>, dim3((unsigned)(8 * ctas)), dim3(256), 0, s, a, ctas);
    return e;
  };
  auto windows = [&](auto dim) -> cudaError_t {
    return window > 0 ? kinds(dim, std::true_type()) : kinds(dim, std::false_type());
  };
  const cudaError_t e = d == 128 ? windows(std::integral_constant<int, 128>())
                                 : windows(std::integral_constant<int, 64>());
  if (e != cudaSuccess) {
    cudaGetLastError();
    return DHS_ERR_CUDA;
  }
  return DHS_OK;
}
