// Causal attention of packed sequences on the fifth-generation tensor cores.
//
// For kv head g the rows of the score matrix are (token, head) pairs, the G =
// q_heads / kv_heads heads of a token next to one another: 128 rows are tpt =
// 128 / G tokens (the rest of the 128 idle when G does not divide it), so that
// grouped heads share every key and value tile and the causal edge of a tile is
// tpt positions wide.  An item of work is two such row tiles (2 tpt consecutive
// tokens of one sequence), walking the keys that they see in tiles of 128:
//   S_i = Q_i K^T (M 128, N 128, K D), P_i = 2^(c S_i - m_i), O_i += P_i V.
// One CTA per SM walks a fixed list of items (PromptSchedule), so that the copies
// and first products of an item run while the rows of the one before are written.
//
// Warps 0-7 and 8-15 are the softmax threads of row tile 0 and 1, two threads a
// row, each with half of a tile's columns: they read S from tensor memory, keep the
// row's maximum m (O is rescaled only when it grows by more than kPrRescale) and its
// sum l in 32 bits, and write P in bf16 over S in tensor memory, from where the second
// product reads it.  (With one thread a row the softmax of a tile took 2500 cycles
// against the 1024 of the other row tile's products, and bound the kernel: 1.02 ms
// then, 0.73 with two.)  Warp 16 issues all MMAs, for each value tile t in the
// order  P0 V(t), Q0 K(t+1), P1 V(t), Q1 K(t+1): while one row tile's softmax runs,
// the tensor cores work for the other.  S_i(t + 1) overwrites P_i(t), which the MMA
// issued just before it reads: MMAs run in the order of their issue.  Warp 17 works
// out the items and fetches Q and the rings of K and V tiles with tiled TMA copies in
// the 128-byte-swizzled layout.
//
// A weight is 0 where a row does not see a key, but 0 times an infinity or a NaN is
// not 0: warps 18-19 go over the value tiles at the causal edge and the sequence's
// end before they are used, set what is not finite there to 0, and remember it; the
// rows that do see such a value get it added at the end, value by value.
//
// With few row tiles the keys are split over several items, which leave (O, m, l) in
// the workspace for a join (prompt_splits says when).
//
// Waits are bounded, by a time that follows the work a wait may last for
// (prompt_wait_us); one that runs out records an error and lets the CTA finish: rows that
// are not written yet stay as they were, the loader waits for its copies and the MMA
// warp for its products before tensor memory is freed.  With key splits each CTA leaves
// word of it for the join, which then writes no row at all.
//
// Measured (16 heads of one kv head, 128 dims): 16384 tokens of one sequence 0.60 ms,
// 1830 TFLOP/s, 95 % of the measured matrix rate, in calls with pauses between; 0.66 ms
// and 86 % (98 % of the rate held for seconds) in calls without, where the power limit
// lowers the clock; 8192 tokens 0.166 ms.  At 64 dims Q K^T
// takes half the time, P V as long as at 128 and a tile's softmax the same: 16384 tokens
// reach 1110 TFLOP/s with the tensor pipe busy for 44 % of the cycles, the issue slots
// for 54 and the exponentials' pipe for 44: what bounds it is the chain of a tile's
// softmax (read S, maximum, exponentials, write P), of which two run side by side.  16
// ragged sequences of up to 2048 tokens (32 heads over 8) reach 1180 (1090 in calls
// without pauses): an item costs some 3 tiles' time besides its tiles (the first S, the
// rows' writing).
#include "pages_internal.cuh"
#include "attn_tc.cuh"

#include <math_constants.h>

#include <algorithm>

namespace dhs {
namespace {

constexpr int kPrSoftmax = 512;  // two row tiles, two warpgroups each
constexpr int kPrThreads = kPrSoftmax + 128;
constexpr int kPrM = 128, kPrN = 128, kPrH = kPrN / 2;
constexpr int kMmaWarp = 16, kLoadWarp = 17, kCleanWarp = 18;
// Microseconds that a wait lasts at most (see prompt_wait_us), and that the last ones of
// a CTA do, for copies and products in flight.  In a build for tests the first is a
// variable.
constexpr uint32_t kPrLastUs = 2000000;
#ifdef DHS_TEST_WAITS
}  // namespace
}  // namespace dhs
extern "C" uint32_t dhs_prompt_wait_us;
uint32_t dhs_prompt_wait_us = 2000000;
namespace dhs {
namespace {
#else
constexpr uint32_t dhs_prompt_wait_us = 2000000;
#endif
constexpr float kPrRescale = 8.f;
constexpr int kPrSplits = 64;      // key splits at most
constexpr uint32_t kPrCols = 512;  // S0, S1 (P over them), O0, O1

struct PromptArgs {
  const uint16_t *v;
  int64_t vt, vh;            // strides of v, for values that are not finite
  const int32_t *cu_q, *cu_k;
  uint16_t *out;
  float *lse, *parts;
  int32_t *status;           // [CTAs] in the workspace: a wait of the CTA ran out
  int32_t *err;
  int64_t n_q, n_k;
  int n_seqs, hq, hkv, G, tpt, nsplit, ctas;
  uint32_t wait_us;
  int64_t most;              // row-tile pairs there can be
  int out32;                 // out lies on 32-byte boundaries
  float scale_log2;
};

template <int D>
struct PrCfg {
  static constexpr int HALVES = D / 64;
  static constexpr int TILE = 128 * D * 2;          // a Q, K or V tile
  static constexpr int HALF = 128 * 128;            // 64 dims of its 128 rows
  // K and V tiles in flight, in a ring each: who waits for a ring's copies waits for
  // every one of them.  (A wait that skips a phase of its barrier, as for every other
  // copy of a common ring, takes the phase before last for the one it waits for
  // while the last is still open.)
  static constexpr int KS = D == 128 ? 3 : 4, VS = D == 128 ? 2 : 4, SLOTS = KS + VS;
  static constexpr int OFF_KV = 2 * TILE;
  static constexpr int OFF_RED = OFF_KV + SLOTS * TILE;  // float [2 tiles][2 halves][128]
  static constexpr int OFF_BAR = OFF_RED + 2 * 2 * 128 * 4;
  static constexpr int CLEAN = 4;                   // value tiles gone over and not yet used, at most
  static constexpr int BARS = 3 + 2 * SLOTS + CLEAN + 8 + 4;
  static constexpr int OFF_TMEM = OFF_BAR + BARS * 8;
  static constexpr int OFF_MISC = OFF_TMEM + 16;    // int [4]: abort, -, bad values by item parity
  static constexpr int OFF_ITEM = OFF_MISC + 16;    // PromptItem [2]
  static constexpr int SMEM = OFF_ITEM + 2 * 64;
};
static_assert(PrCfg<128>::SMEM <= 227 * 1024, "shared memory of the prompt kernel");

// What calls without a record of their own find, one for each device.
__device__ int32_t device_record[2];

__device__ __forceinline__ void prompt_error(const PromptArgs &a, int code) {
  page_error(a.err, code, DHS_SITE_PROMPT_ATTEND);
}

// A sequence's queries and keys; false (recorded) for offsets out of range.
__device__ __forceinline__ bool prompt_seq(const PromptArgs &a, int i, int &q0, int &nq, int &k0,
                                           int &nk, bool record = true) {
  q0 = a.cu_q[i];
  k0 = a.cu_k[i];
  const int64_t q1 = a.cu_q[i + 1], k1 = a.cu_k[i + 1];
  if (q0 < 0 || q1 < q0 || q1 > a.n_q || k0 < 0 || k1 < k0 || k1 > a.n_k) {
    if (record) prompt_error(a, DC_ROW_RANGE);
    nq = nk = 0;
    return false;
  }
  nq = (int)(q1 - q0);
  nk = (int)(k1 - k0);
  return true;
}

// One piece of work: two row tiles of a sequence and the key tiles they walk.
struct PromptItem {
  int q0, nq, k0, nk;   // the sequence; q0 < 0: no more work
  int tok0, kvh, part;  // row tile 0's first token, kv head, key split
  int t0, n0, n1;       // first key tile, and how many either row tile walks
};
static_assert(sizeof(PromptItem) <= 64, "");

// The items of CTA b: items are ordered by the tile's place in its sequence, the
// last places (the longest walks) first, over all sequences, kv heads and key
// splits; the CTAs take them in turn, forth and back, which balances them within
// about one short item.  All lanes of a warp; the next item comes back in lane-uniform
// registers.
struct PromptSchedule {
  const PromptArgs &a;
  int lane, span, q0, nq, k0, nk, tiles, top, items;

  __device__ int load(int i, bool record) {
    q0 = nq = k0 = nk = 0;
    if (i < a.n_seqs) prompt_seq(a, i, q0, nq, k0, nk, record);
    return (nq + span - 1) / span;
  }
  // the same for eight sequences of this lane at a time, whose loads are under way
  // together (1024 prompts of one token: 176 -> 141 us)
  __device__ void load8(int i, int (&n)[8]) {
#pragma unroll
    for (int u = 0; u < 8; ++u) n[u] = load(i + 32 * u + lane, false);
  }
  __device__ PromptSchedule(const PromptArgs &args, int l) : a(args), lane(l), span(2 * args.tpt) {
    int64_t total = 0;
    top = 0;
    for (int i = 0; i < a.n_seqs; i += 32) {
      tiles = load(i + lane, true);  // (32 sequences or fewer stay in registers)
      total += (int64_t)__reduce_add_sync(0xffffffffu, (unsigned)tiles);
      top = max(top, __reduce_max_sync(0xffffffffu, tiles));
    }
    items = (int)min(total, a.most) * a.hkv * a.nsplit;  // (the host keeps this in 31 bits)
  }
  // tiles whose place in their sequence is j or later
  __device__ int from(int j) {
    if (a.n_seqs <= 32) return __reduce_add_sync(0xffffffffu, max(0, tiles - j));
    int n = 0, x[8];
    for (int i = 0; i < a.n_seqs; i += 256) {
      load8(i, x);
#pragma unroll
      for (int u = 0; u < 8; ++u) n += max(0, x[u] - j);
    }
    return __reduce_add_sync(0xffffffffu, n);
  }
  __device__ bool item(int k, PromptItem &it) {
    const int64_t w = (int64_t)k * gridDim.x +
                      (k & 1 ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
    if (w >= items) return false;
    const uint32_t per = (uint32_t)(a.hkv * a.nsplit);
    const int t = (int)((uint32_t)w / per), in = (int)((uint32_t)w % per);
    it.part = a.nsplit == 1 ? 0 : (int)((uint32_t)in / (uint32_t)a.hkv);
    it.kvh = in - it.part * a.hkv;
    it.q0 = it.nq = it.k0 = it.nk = 0;
    // the place: from(place + 1) <= t < from(place)
    int lo = 0, hi = top - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (from(mid) > t) lo = mid;
      else hi = mid - 1;
    }
    // the sequence: the (t - from(place + 1))-th of those that have it
    int nth = t - from(lo + 1);
    int base = 0;  // its 32 neighbours
    if (a.n_seqs > 32) {
      bool found = false;
      for (int i = 0; i < a.n_seqs && !found; i += 256) {
        int x[8];
        load8(i, x);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int n = __popc(__ballot_sync(0xffffffffu, x[u] > lo));
          if (!found && nth < n) {
            found = true;
            base = i + 32 * u;
          }
          if (!found) nth -= n;
        }
      }
      tiles = load(base + lane, false);
    }
    const uint32_t has = __ballot_sync(0xffffffffu, tiles > lo);
    if (nth < __popc(has)) {
      const bool me = tiles > lo && __popc(has & ((1u << lane) - 1u)) == nth;
      const int src = __ffs(__ballot_sync(0xffffffffu, me)) - 1;
      it.q0 = __shfl_sync(0xffffffffu, q0, src);
      it.nq = __shfl_sync(0xffffffffu, nq, src);
      it.k0 = __shfl_sync(0xffffffffu, k0, src);
      it.nk = __shfl_sync(0xffffffffu, nk, src);
    }
    it.tok0 = lo * span;
    const int off = it.nk - it.nq + 1, tok1 = it.tok0 + a.tpt;
    const int last0 = min(tok1, it.nq) - 1, last1 = min(tok1 + a.tpt, it.nq) - 1;
    // key tiles that any row sees, this split's, and either row tile's (T is below
    // 2^24 and there are at most kPrSplits parts: 32 bits hold the products)
    const int T = (max(0, off + max(last0, last1)) + kPrN - 1) / kPrN;
    it.t0 = a.nsplit == 1 ? 0 : (int)((uint32_t)T * it.part / (uint32_t)a.nsplit);
    const int t1 = a.nsplit == 1 ? T : (int)((uint32_t)T * (it.part + 1) / (uint32_t)a.nsplit);
    const int e0 = min(t1, (max(0, off + last0) + kPrN - 1) / kPrN);
    const int e1 = last1 >= tok1 ? min(t1, (max(0, off + last1) + kPrN - 1) / kPrN) : it.t0;
    it.n0 = max(0, e0 - it.t0);
    it.n1 = max(0, e1 - it.t0);
    return true;
  }
};

template <int D>
__global__ void __launch_bounds__(kPrThreads, 1)
k_prompt(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
         const __grid_constant__ CUtensorMap mv, const PromptArgs a) {
  using C = PrCfg<D>;
  // no static shared memory: the dynamic part starts on the boundary it asks for
  extern __shared__ __align__(1024) unsigned char smem[];
  int *misc = reinterpret_cast<int *>(smem + C::OFF_MISC);
  volatile int *abort_v = misc, *bad_values = misc + 2;
  auto item_of = [&](int k) -> PromptItem & {
    return *reinterpret_cast<PromptItem *>(smem + C::OFF_ITEM + (k & 1) * 64);
  };
  if ((smem_u32(smem) & 1023u) != 0u) {  // (the swizzle pattern follows address bits)
    if (a.nsplit > 1 && threadIdx.x == 0) a.status[blockIdx.x] = 1;
    prompt_error(a, DC_CAPACITY);
    return;
  }
  // (a warp's number by a shuffle: the compiler then knows that the roles' branches are
  // the same for a whole warp and keeps the MMAs' operands in uniform registers; moves
  // into them had made the issue of an MMA cost what its execution does, 0.644 ms for
  // 16384 tokens instead of 0.599)
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
  uint64_t *q_full = bars, *q_empty = bars + 1, *mma_done = bars + 2, *full = bars + 3,
           *empty = full + C::SLOTS, *clean = empty + C::SLOTS;
  uint64_t *s_full = clean + C::CLEAN, *p_full = s_full + 2, *pv_done = s_full + 4,
           *o_empty = s_full + 6, *item_full = s_full + 8, *item_empty = s_full + 10;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_TMEM);
  if (tid == kLoadWarp * 32) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(mma_done, 1);
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::CLEAN; ++i) mbar_init(&clean[i], 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kPrSoftmax / 64);   // one arrival per warp
      mbar_init(&pv_done[i], 1);
      mbar_init(&o_empty[i], kPrSoftmax / 64);
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], kPrSoftmax / 32 + 3);  // all warps but the loader's
    }
    for (int i = 0; i < 4; ++i) misc[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, kPrCols);
  if (tid == kLoadWarp * 32 + 1) {
    tma_prefetch(&mq);
    if (a.n_k > 0) {  // (without keys their maps are not made)
      tma_prefetch(&mk);
      tma_prefetch(&mv);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // All 512 columns are this CTA's, so they start at column 0 (lane 0), and the
  // addresses below are constants.
  constexpr uint32_t tmem = 0u;

  auto wait = [&](uint64_t *bar, uint32_t parity, bool force = false) {
    if (mbar_try_wait(bar, parity)) return;
    const uint32_t since = global_us();  // (a poll that fails has waited for some 5 us)
    do {
      if (!force && *abort_v) return;
      if (global_us() - since >= (force ? kPrLastUs : a.wait_us)) {
        prompt_error(a, DC_TIMEOUT);
        *abort_v = 1;
        return;
      }
    } while (!mbar_try_wait(bar, parity));
  };
  auto given_up = [&]() { return __any_sync(0xffffffffu, *abort_v) != 0; };
  // Slot of the n-th K or V tile since the start, and the parity of its use.  (All
  // counts below run over a CTA's items: every wait is for the phase after the one
  // that its waiter waited for last.)
  auto kslot = [&](uint32_t n) { return n % C::KS; };
  auto vslot = [&](uint32_t n) { return C::KS + n % C::VS; };
  auto kpar = [&](uint32_t n) { return (n / C::KS) & 1u; };
  auto vpar = [&](uint32_t n) { return (n / C::VS) & 1u; };
  auto item_par = [&](int k) { return (uint32_t)(k >> 1) & 1u; };
  // the k-th item, read and released by every warp but the loader's
  auto take = [&](int k) {
    wait(&item_full[k & 1], item_par(k));
    __syncwarp();
    const PromptItem it = item_of(k);
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_empty[k & 1]);
    return it;
  };

  if (warp == kLoadWarp) {
    // --------------------------------------------------------- items and copies
    PromptSchedule plan(a, lane);
    uint32_t kn = 0, vn = 0, qn = 0;  // copies issued
    for (int k = 0;; ++k) {
      PromptItem it;
      const bool more = plan.item(k, it);
      if (!more) it.q0 = -1;
      if (k >= 2) wait(&item_empty[k & 1], item_par(k) ^ 1u);
      __syncwarp();
      if (given_up()) break;
      if (lane == 0) {
        item_of(k) = it;
        mbar_arrive(&item_full[k & 1]);
      }
      if (!more) break;
      const int nt = max(it.n0, it.n1);
      if (lane == 0 && nt > 0) {
        const int ntile = it.n1 > 0 ? 2 : 1;
        if (qn > 0) wait(q_empty, (qn - 1) & 1u);
        if (!*abort_v) {
          mbar_arrive_expect_tx(q_full, (uint32_t)(ntile * C::HALVES * a.G * a.tpt * 128));
          for (int i = 0; i < ntile; ++i)
            for (int h = 0; h < C::HALVES; ++h)
              tma_load_3d(smem + i * C::TILE + h * C::HALF, &mq, h * 64, it.kvh * a.G,
                          it.q0 + it.tok0 + i * a.tpt, q_full);
          ++qn;
        }
        for (int n = 0; n < 2 * nt && !*abort_v; ++n) {  // K, V, K, V, ...
          const bool v = n & 1;
          const uint32_t c = v ? vn : kn, t = v ? vslot(c) : kslot(c);
          if (c >= (uint32_t)(v ? C::VS : C::KS)) wait(&empty[t], (v ? vpar(c) : kpar(c)) ^ 1u);
          if (*abort_v) break;
          mbar_arrive_expect_tx(&full[t], (uint32_t)C::TILE);
          for (int h = 0; h < C::HALVES; ++h)
            tma_load_3d(smem + C::OFF_KV + t * C::TILE + h * C::HALF, v ? &mv : &mk, h * 64, it.kvh,
                        it.k0 + (it.t0 + (n >> 1)) * kPrN, &full[t]);
          if (v) ++vn;
          else ++kn;
        }
      }
      __syncwarp();
    }
    if (lane == 0) {
      // every copy has landed before the CTA ends
      if (qn > 0) wait(q_full, (qn - 1) & 1u, true);
      for (uint32_t i = kn > C::KS ? kn - C::KS : 0; i < kn; ++i) wait(&full[kslot(i)], kpar(i), true);
      for (uint32_t i = vn > C::VS ? vn - C::VS : 0; i < vn; ++i) wait(&full[vslot(i)], vpar(i), true);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ----------------------------------------------------------------- products
    constexpr uint32_t kIdescQK = tc_idesc_bf16(kPrM, kPrN, 0, 0);
    constexpr uint32_t kIdescPV = tc_idesc_bf16(kPrM, D, 0, 1);
    const uint32_t sQ = smem_u32(smem), sKV = smem_u32(smem + C::OFF_KV);
    auto qk = [&](int i, uint32_t c) {
      const uint64_t q = tc_desc_sw128(sQ + i * C::TILE, 16, 1024);
      const uint64_t k = tc_desc_sw128(sKV + kslot(c) * C::TILE, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t o = ((kk >> 2) * C::HALF + (kk & 3) * 32) >> 4;
        warp_mma(i * kPrN, q + o, k + o, kIdescQK, kk);
      }
      warp_commit(&s_full[i]);
    };
    auto pv = [&](int i, uint32_t c, int n) {
      const uint64_t v = tc_desc_sw128(sKV + vslot(c) * C::TILE, C::HALF, 1024);
#pragma unroll
      for (int kk = 0; kk < kPrN / 16; ++kk)
        warp_mma_ta(2 * kPrN + i * D, i * kPrN + kk * 8, v + kk * 128, kIdescPV, n | kk);
    };
    uint32_t kn = 0, vn = 0, qn = 0, pn[2] = {0, 0}, on[2] = {0, 0};
    for (int k = 0;; ++k) {
      const PromptItem it = take(k);
      if (given_up() || it.q0 < 0) break;
      const int nt = max(it.n0, it.n1);
      if (nt == 0) continue;
      // the last item's O has been read
      for (int i = 0; i < 2; ++i)
        if ((i ? it.n1 : it.n0) > 0 && on[i] > 0) wait(&o_empty[i], (on[i] - 1) & 1u);
      // S of a row tile may be written at once: the P that the last item's final
      // product read there was issued before
      wait(q_full, qn & 1u);
      ++qn;
      wait(&full[kslot(kn)], kpar(kn));
      __syncwarp();
      tc_fence_after();
      if (it.n0 > 0) qk(0, kn);
      if (it.n1 > 0) qk(1, kn);
      warp_commit(&empty[kslot(kn)]);
      if (nt == 1) warp_commit(q_empty);
      ++kn;
      for (int n = 0; n < nt; ++n) {
        if ((n & 15) == 15 && given_up()) break;
        wait(&clean[vn % C::CLEAN], (vn / C::CLEAN) & 1u);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int ni = i ? it.n1 : it.n0;
          if (n < ni) {
            wait(&p_full[i], pn[i] & 1u);
            ++pn[i];
            __syncwarp();
            tc_fence_after();
            pv(i, vn, n);
            if (n + 1 == ni) {
              warp_commit(&pv_done[i]);
              ++on[i];
            }
          }
          if (n + 1 < ni) {
            wait(&full[kslot(kn)], kpar(kn));
            __syncwarp();
            tc_fence_after();
            qk(i, kn);
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
  } else if (warp >= kCleanWarp) {
    // ------------------------------------------------------------------- values
    uint32_t vn = 0;
    for (int k = 0;; ++k) {
      const PromptItem it = take(k);
      if (given_up() || it.q0 < 0) break;
      const int common = it.nk - it.nq + 1 + it.tok0;  // keys that every row of the item sees
      for (int n = 0; n < max(it.n0, it.n1); ++n, ++vn) {
        wait(&full[vslot(vn)], vpar(vn));
        if (given_up()) break;
        const int r0 = max(0, common - (it.t0 + n) * kPrN);
        if (r0 < kPrN) {
          unsigned char *v = smem + C::OFF_KV + vslot(vn) * C::TILE;
          const int inside = it.nk - (it.t0 + n) * kPrN;  // rows of this sequence
          // Row r's 64 dims of half h are the 128 bytes at h * HALF + r * 128.  An
          // exponent of ones plus one carries into the sign's place: eight values cost
          // a dozen instructions, and the slow loop runs only if some are not finite.
          uint32_t any = 0u;
#pragma unroll 8
          for (int e = r0 * 8 + (warp - kCleanWarp) * 32 + lane; e < kPrN * 8; e += 64) {
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
          for (int e = r0 * 8 + (warp - kCleanWarp) * 32 + lane;
               (any & 0x80008000u) != 0u && e < kPrN * 8; e += 64) {
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
                found |= (e >> 3) < inside;
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
  } else {
    // ------------------------------------------------------------------ softmax
    const int i = warp >> 3, hg = (warp >> 2) & 1, m = tid & 127;
    const int tloc = m / a.G, h = m - tloc * a.G;
    const int pair = 1 + i * 4 + (warp & 3);  // barrier of the two warps of these rows
    const uint32_t lrow = (uint32_t)((warp & 3) * 32) << 16;
    // this thread's half of the row's scores, and of its output columns
    const uint32_t tS = tmem + lrow + i * kPrN, tO = tmem + lrow + 2 * kPrN + i * D + hg * (D / 2);
    float *red = reinterpret_cast<float *>(smem + C::OFF_RED) + i * 256;
    const float sl2 = a.scale_log2;
    const uint64_t sl22 = pack_f32x2(sl2, sl2);
    uint32_t sn = 0, on = 0;
    for (int k = 0;; ++k) {
      // the item stays in shared memory until its rows are written: few of its
      // fields are wanted in the loop, where registers are short
      wait(&item_full[k & 1], item_par(k));
      __syncwarp();
      volatile const PromptItem &it = item_of(k);
      // (the warps of a pair leave together: they meet at barriers below, also after a
      // wait has run out)
      if (named_or(pair, 64, *abort_v != 0) || it.q0 < 0) break;
      const int t0 = it.t0, ni = i ? it.n1 : it.n0;
      int lim0;  // columns of tile 0 that this row's half sees
      int least; // tiles from this one on have columns that some row does not see
      {
        const int off = it.nk - it.nq + 1, tok = it.tok0 + i * a.tpt + tloc;
        const bool valid = tloc < a.tpt && tok < it.nq;
        lim0 = (valid ? off + tok : 0) - hg * kPrH;
        least = off + it.tok0 + i * a.tpt;
      }
      float m_run = -CUDART_INF_F, l = 0.f;
      for (int n = 0; n < ni; ++n, ++sn) {
        wait(&s_full[i], sn & 1u);
        __syncwarp();
        tc_fence_after();
        uint32_t s0[32], s1[32];
        tmem_ld32(tS + hg * kPrH, s0);
        tmem_ld32(tS + hg * kPrH + 32, s1);
        tmem_wait_ld();
        const int first = (t0 + n) * kPrN;
        if (first + kPrN > least) {
          const int lim = lim0 - first;  // columns this row sees
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            if (c >= lim) s0[c] = 0xFF800000u;
            if (c + 32 >= lim) s1[c] = 0xFF800000u;
          }
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
        if (named_or(pair, 64, mx > m_run + kPrRescale)) {
          red[hg * 128 + m] = mx;
          named_sync(pair, 64);
          mx = fmaxf(mx, red[(hg ^ 1) * 128 + m]);
          named_sync(pair, 64);
          if (__any_sync(0xffffffffu, mx > m_run + kPrRescale)) {
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
        // weights are rounded to bf16 for the product (at most 2^-8 of each); l is not
        auto weights = [&](const uint32_t(&s)[32]) {
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            float u, w;
            unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[2 * x]),
                                              __uint_as_float(s[2 * x + 1])), sl22, b2), u, w);
            u = ex2_approx(u);
            w = ex2_approx(w);
            l2 = add_f32x2(l2, pack_f32x2(u, w));
            p[x] = pack_bf16(u, w);
          }
        };
        weights(s0);
        tmem_st16(tS + hg * (kPrH / 2), p);
        weights(s1);
        tmem_st16(tS + hg * (kPrH / 2) + 16, p);
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
      uint32_t o[D / 2];
      if (ni > 0) {
        wait(&pv_done[i], on & 1u);
        ++on;
        __syncwarp();
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < D / 2; c += 32)
          tmem_ld32(tO + c, *reinterpret_cast<uint32_t(*)[32]>(&o[c]));
        tmem_wait_ld();
        tc_fence_before();
        // (read before this item's place is given up: the one after next uses it again)
        bad = bad_values[k & 1] == k + 1;
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_empty[i]);
      } else {
#pragma unroll
        for (int x = 0; x < D / 2; ++x) o[x] = 0u;
      }
      // Rows of an item for which a wait ran out (whoever's it was: it is known by the
      // time what it waited for arrives here) are not written, nor half of them.
      const bool lost = named_or(pair, 64, *abort_v != 0);
      l += red[(hg ^ 1) * 128 + m];  // the row's sum over both halves
      const int off = it.nk - it.nq + 1, tok = it.tok0 + i * a.tpt + tloc;
      const int q0 = it.q0, k0 = it.k0, kvh = it.kvh, part_no = it.part, common = off + it.tok0;
      const bool valid = tloc < a.tpt && tok < it.nq && !lost;
      const int seen = valid ? off + tok : 0;  // may be negative
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[k & 1]);
      if (valid && bad) {
        // values that were taken out, for the keys that this row sees in this item's tiles
        const int lo = max(max(common, 0), t0 * kPrN);
        const int hi = min(seen, (t0 + ni) * kPrN);
        for (int p = lo; p < hi; ++p) {
          const uint16_t *src =
              a.v + (int64_t)(k0 + p) * a.vt + (int64_t)kvh * a.vh + hg * (D / 2);
#pragma unroll
          for (int x = 0; x < D / 2; ++x) {
            const uint32_t u = (uint32_t)src[x] << 16;
            if ((u & 0x7F800000u) == 0x7F800000u)
              o[x] = __float_as_uint(__uint_as_float(o[x]) + __uint_as_float(u));
          }
        }
      }
      if (valid) {
        const int64_t row = (int64_t)(q0 + tok) * a.hq + kvh * a.G + h;
        if (a.nsplit > 1) {
          float *part = a.parts + ((int64_t)part_no * a.n_q * a.hq + row) * (D + 2);
#pragma unroll
          for (int x = 0; x < D / 2; x += 2)
            *reinterpret_cast<float2 *>(part + hg * (D / 2) + x) =
                make_float2(__uint_as_float(o[x]), __uint_as_float(o[x + 1]));
          if (hg == 0) *reinterpret_cast<float2 *>(part + D) = make_float2(m_run, l);
        } else {
          const float inv = 1.f / l;  // only scores of -inf: 0 / 0
          uint16_t *to = a.out + row * D + hg * (D / 2);
#pragma unroll
          for (int x = 0; x < D / 2; x += 16) {
            uint32_t w[8];
#pragma unroll
            for (int y = 0; y < 8; ++y)
              w[y] = seen > 0 ? pack_bf16(__uint_as_float(o[x + 2 * y]) * inv,
                                          __uint_as_float(o[x + 2 * y + 1]) * inv)
                              : 0u;
            if (a.out32) {  // whole 32-byte sectors
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
  if (warp == kMmaWarp) tmem_dealloc(*tmem_slot, kPrCols);
  if (a.nsplit > 1 && tid == 0) a.status[blockIdx.x] = *abort_v;
}

// Joins the parts of a row: sum_s w_s O_s / sum_s w_s l_s, w_s = 2^(m_s - max m).
template <int D>
__global__ void __launch_bounds__(128)
k_prompt_join(const PromptArgs a) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + threadIdx.x / 32, rows = a.n_q * a.hq;
  pdl_wait();
  // (which parts are missing is not known; each warp reading all words for itself, beside
  // its parts, took up to 3 us longer)
  int lost = 0;
  for (int c = threadIdx.x; c < a.ctas; c += 128) lost |= a.status[c];
  if (__syncthreads_or(lost) || row >= rows) return;
  const int64_t tok = row / a.hq;
  const int i = seq_of(a.cu_q, a.n_seqs, tok);
  if (i < 0) return;
  int q0, nq, k0, nk;
  if (!prompt_seq(a, i, q0, nq, k0, nk) || tok < q0 || tok >= q0 + nq) return;
  const bool some = nk - nq + (int)(tok - q0) + 1 > 0;
  const float *p = a.parts + row * (D + 2);
  const int64_t step = rows * (D + 2);
  float top = -CUDART_INF_F, den = 0.f, acc[V];
#pragma unroll
  for (int x = 0; x < V; ++x) acc[x] = 0.f;
  for (int s = 0; s < a.nsplit; ++s) top = fmaxf(top, p[s * step + D]);
#pragma unroll 4
  for (int s = 0; s < a.nsplit; ++s) {
    const float2 ml = *reinterpret_cast<const float2 *>(p + s * step + D);
    const float f = ml.x == -CUDART_INF_F ? (ml.y != ml.y ? 1.f : 0.f) : ex2_approx(ml.x - top);
    den += ml.y * f;
#pragma unroll
    for (int x = 0; x < V; x += 2) {
      const float2 o = *reinterpret_cast<const float2 *>(p + s * step + lane * V + x);
      acc[x] += o.x * f;
      acc[x + 1] += o.y * f;
    }
  }
  const float inv = 1.f / den;
#pragma unroll
  for (int x = 0; x < V; x += 2)
    *reinterpret_cast<uint32_t *>(a.out + row * D + lane * V + x) =
        some ? pack_bf16(acc[x] * inv, acc[x + 1] * inv) : 0u;
  if (a.lse && lane == 0)
    a.lse[row] = top == CUDART_INF_F ? top
                 : den == 0.f        ? -CUDART_INF_F
                                     : (top + log2f(den)) * 0.69314718055994531f;
}

bool prompt_args(int64_t n_q, int64_t n_k, int32_t n_seqs, int32_t hq, int32_t hkv, int32_t d) {
  // (a tile's positions run up to 256 past the last token, in 32 bits)
  constexpr int64_t most = INT32_MAX - 256;
  return n_q >= 0 && n_k >= 0 && n_q <= most && n_k <= most && n_seqs >= 0 &&
         n_seqs <= kMaxSeqs && hkv >= 1 && hkv <= kPageMaxHeads && hq >= 1 && hq % hkv == 0 &&
         hq / hkv <= 128 && (d == 64 || d == 128);
}

// Most row-tile pairs n_q tokens of n_seqs sequences can make.
int64_t prompt_tiles(int64_t n_q, int32_t n_seqs, int G) {
  const int64_t span = 2 * (128 / G);
  return n_q / span + std::min<int64_t>(n_seqs, n_q);
}

// Key splits: as many as make the longest CTA shortest.  With I row-tile pairs (times
// kv heads) of T key tiles, n splits deal I n items of T / n tiles to the SMs in
// ceil(I n / SMs) turns; an item costs some 3 tiles' time besides its tiles, a join
// some 6.  (Two 500-token chunks over 32K keys, 32 pairs: 4 splits, 92 us instead of
// 330.)  The average stands for every sequence: 500 tokens over 100K keys (8 heads over 2,
// 128 dims) take 147 us by themselves and 980 beside 30 prompts of 50 tokens, which lower
// it to no split.
int prompt_splits(int64_t n_q, int64_t n_k, int32_t n_seqs, int hq, int hkv, int sms) {
  if (n_q == 0 || n_seqs == 0) return 1;
  const int64_t items = prompt_tiles(n_q, n_seqs, hq / hkv) * hkv;
  // an average row's keys: all of the sequence but half of its queries
  const int64_t tiles =
      std::max<int64_t>(0, n_k - std::min(n_q, n_k) / 2) / n_seqs / kPrN + 1;
  int best = 1;
  int64_t least = INT64_MAX;
  for (int n = 1; n <= kPrSplits && (n == 1 || tiles / n >= 4); ++n) {
    const int64_t cost = (items * n + sms - 1) / sms * ((tiles + n - 1) / n + 3) + (n > 1 ? 6 : 0);
    if (cost < least) {
      least = cost;
      best = n;
    }
  }
  return best;
}

// Bytes of the parts' workspace: (O, m, l) of every row and split, then a word a CTA.
int64_t prompt_bytes(int nsplit, int64_t n_q, int hq, int d, int sms) {
  return nsplit > 1 ? (int64_t)nsplit * n_q * hq * (d + 2) * 4 + (int64_t)sms * 4 : 0;
}

// How long a wait may take.  Some last as long as an item (a row tile without work waits
// for the next one) or as the search for one among all sequences: beside two seconds,
// 20 us for each key tile there can be, which takes 0.3 to 0.5 us, and 5 us for each
// sequence, which takes some 0.1; half an hour at most.
uint32_t prompt_wait_us(int64_t n_k, int32_t n_seqs) {
  const uint64_t least = dhs_prompt_wait_us;
  return (uint32_t)std::min<uint64_t>(
      least + least * (uint64_t)(n_k / kPrN + 1) / 100000 + least * (uint64_t)n_seqs / 400000,
      1800000000u);
}

// The device's record (its address asked for once; chosen in the kernel it would cost
// registers where there are none), or nullptr.
int32_t *record_of(int dev) {
  static std::atomic<int32_t *> known[kMaxDevices];
  if (dev < 0 || dev >= kMaxDevices) return nullptr;
  int32_t *p = known[dev].load(std::memory_order_acquire);
  if (!p) {
    void *at = nullptr;
    if (cudaGetSymbolAddress(&at, device_record) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    p = static_cast<int32_t *>(at);
    known[dev].store(p, std::memory_order_release);
  }
  return p;
}

// [tokens][heads][d] of bf16, boxes of 64 dims x box_heads x box_tokens.
bool encode(EncodeTiled f, CUtensorMap *m, const void *p, int64_t tokens, int heads, int d,
            int64_t st, int64_t sh, int box_heads, int box_tokens) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)sh * 2, (cuuint64_t)st * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
  const cuuint32_t one[3] = {1, 1, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box, one,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace dhs

extern "C" int64_t dhs_prompt_attend_workspace(int64_t n_q, int64_t n_k, int32_t n_seqs,
                                               int32_t q_heads, int32_t kv_heads,
                                               int32_t head_dim) {
  using namespace dhs;
  if (!prompt_args(n_q, n_k, n_seqs, q_heads, kv_heads, head_dim)) return -1;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  const int sms = device_sms(dev);
  if (sms < 1) return -1;
  const int n = prompt_splits(n_q, n_k, n_seqs, q_heads, kv_heads, sms);
  return prompt_bytes(n, n_q, q_heads, head_dim, sms);
}

extern "C" int dhs_prompt_attend(const void *q, const void *k, const void *v,
                                 const int64_t *strides, int64_t n_q, int64_t n_k,
                                 const int32_t *cu_q, const int32_t *cu_k, int32_t n_seqs,
                                 int32_t q_heads, int32_t kv_heads, int32_t head_dim, float scale,
                                 void *out, float *lse, void *workspace, int64_t workspace_bytes,
                                 int32_t *err, dhs_stream stream) {
  using namespace dhs;
  if (!prompt_args(n_q, n_k, n_seqs, q_heads, kv_heads, head_dim) || !(scale >= 0.f) ||
      scale > 1e38f || workspace_bytes < 0)
    return DHS_ERR_INVALID;
  if (n_q == 0 || n_seqs == 0) return DHS_OK;
  if (!q || !out || !cu_q || !cu_k || (n_k > 0 && (!k || !v)) || ((uintptr_t)q & 15u) ||
      ((uintptr_t)k & 15u) || ((uintptr_t)v & 15u) || ((uintptr_t)out & 15u) ||
      ((uintptr_t)workspace & 15u) || !words(cu_q, cu_k, lse, err))
    return DHS_ERR_INVALID;
  const int64_t d = head_dim;
  int64_t st[6] = {q_heads * d, d, kv_heads * d, d, kv_heads * d, d};
  if (strides)
    for (int i = 0; i < 6; ++i) {
      const bool used = (i & 1) ? (i == 1 ? q_heads : kv_heads) > 1 : (i == 0 ? n_q : n_k) > 1;
      if (strides[i] < 0 || strides[i] % 8 || strides[i] >= ((int64_t)1 << 38) ||
          (used && strides[i] < d))
        return DHS_ERR_INVALID;
      if (used) st[i] = strides[i];
    }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return DHS_ERR_CUDA;
  }
  const int sms = device_sms(dev);
  EncodeTiled enc = encoder();
  if (!err) err = record_of(dev);
  if (sms < 1 || !enc || !err) return DHS_ERR_CUDA;
  PromptArgs a;
  a.v = static_cast<const uint16_t *>(v);
  a.vt = st[4];
  a.vh = st[5];
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.out = static_cast<uint16_t *>(out);
  a.lse = lse;
  a.parts = static_cast<float *>(workspace);
  a.err = err;
  a.n_q = n_q;
  a.n_k = n_k;
  a.n_seqs = n_seqs;
  a.hq = q_heads;
  a.hkv = kv_heads;
  a.G = q_heads / kv_heads;
  a.tpt = kPrM / a.G;
  a.nsplit = prompt_splits(n_q, n_k, n_seqs, q_heads, kv_heads, sms);
  a.scale_log2 = (scale == 0.f ? 1.f / sqrtf((float)d) : scale) * 1.4426950408889634f;
  const int64_t bytes = prompt_bytes(a.nsplit, n_q, q_heads, head_dim, sms);
  if (bytes > 0 && (!workspace || workspace_bytes < bytes)) return DHS_ERR_INVALID;
  a.wait_us = prompt_wait_us(n_k, n_seqs);
  a.most = prompt_tiles(n_q, n_seqs, a.G);
  a.out32 = ((uintptr_t)out & 31u) == 0;
  const int64_t items = a.most * kv_heads * a.nsplit;
  if (items > INT32_MAX) return DHS_ERR_CAPACITY;
  a.ctas = (int)std::min<int64_t>(items, sms);
  a.status = bytes > 0 ? reinterpret_cast<int32_t *>(static_cast<unsigned char *>(workspace) +
                                                     bytes) - sms
                       : nullptr;
  CUtensorMap mq = {}, mk = {}, mv = {};
  if (!encode(enc, &mq, q, n_q, q_heads, (int)d, st[0], st[1], a.G, a.tpt)) return DHS_ERR_INVALID;
  if (n_k > 0 && (!encode(enc, &mk, k, n_k, kv_heads, (int)d, st[2], st[3], 1, kPrN) ||
                  !encode(enc, &mv, v, n_k, kv_heads, (int)d, st[4], st[5], 1, kPrN)))
    return DHS_ERR_INVALID;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto go = [&](auto dim) -> cudaError_t {
    constexpr int D = decltype(dim)::value;
    static DeviceSmem granted;
    cudaError_t e = granted.ensure(k_prompt<D>, PrCfg<D>::SMEM, dev);
    if (e == cudaSuccess)
      e = launch_prio(k_prompt<D>, dim3((unsigned)a.ctas), dim3(kPrThreads),
                      (size_t)PrCfg<D>::SMEM, s, mq, mk, mv, a);
    if (e == cudaSuccess && a.nsplit > 1)
      e = launch_pdl(k_prompt_join<D>, dim3((unsigned)((n_q * q_heads + 3) / 4)), dim3(128), 0, s,
                     a);
    return e;
  };
  const cudaError_t e = d == 128 ? go(std::integral_constant<int, 128>())
                                 : go(std::integral_constant<int, 64>());
  if (e != cudaSuccess) {
    cudaGetLastError();
    return DHS_ERR_CUDA;
  }
  return DHS_OK;
}

extern "C" int dhs_prompt_errors(int32_t *found, dhs_stream stream) {
  using namespace dhs;
  if (!found) return DHS_ERR_INVALID;
  static const int32_t none[2] = {0, 0};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e =
      cudaMemcpyFromSymbolAsync(found, device_record, sizeof none, 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && found[0] != 0) {
    e = cudaMemcpyToSymbolAsync(device_record, none, sizeof none, 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return DHS_ERR_CUDA;
  }
  return DHS_OK;
}
