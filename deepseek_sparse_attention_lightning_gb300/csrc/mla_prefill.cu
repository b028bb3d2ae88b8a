// mla_prefill.cu -- latent attention in its expanded form for prompts: every
// head has its own keys (128 dims) and values (128 dims), expanded from the
// latent rows by the model's up-projection, and all heads share the 64-dim
// rope key that is cached beside the latent ("Deepseek Details", section
// "DSA": the latent 512 + rope 64; the expanded form is the textbook one).
//
//   x[i, j] = sm_scale * (q[i, 0:128] . k[j] + q[i, 128:192] . k_rope[j])
//   out[i]  = sum_j softmax(x[i])[j] * v[j],   lse[i] = log sum_j exp(x[i, j])
//
// over the keys j < lim[i]: all of the request's, or up to the query's own
// token (the queries are the last of the request's tokens).  Requests are
// packed one after another.
//
// Bound by the matrix pipe: 640 flop a visible pair, against two ring granules'
// worth of traffic a key tile.  One CTA = 256 queries of one head, as two query
// tiles of 128 (M = 128): while one tile's scores are in the softmax, the matrix
// pipe works on the other's.  Measured: one prompt of 8192 tokens, 128 heads,
// 1.70 to 1.77 ms by the machine = 1550 to 1615 TFLOP/s over the visible pairs (81
// to 84 % of the measured matrix rate); 8 ragged prompts of 414 .. 2047, 479 to 509
// us; every query over all of 4096 keys, 862 us = 1594 TFLOP/s.
//
// Tensor memory (512 columns): S of the two tiles (128 each, fp32), O of the
// two (128 each).  P (bf16, 64 columns) overwrites the S it came from and is
// the A operand of P V, so it never passes through shared memory.
// Shared memory: q of both tiles (96 KB), and a ring of eight 16 KB granules,
// each 128 keys x 64 dims (128B swizzle) in the order in which they are read:
// the three atoms of a key tile's K (the third is the shared rope key), then
// the two of its V.
//
// MMA order: QK0(j), PV1(j-1), QK1(j), PV0(j), QK0(j+1), ...: a tile's softmax
// has the other tile's P V and Q K^T (1280 cycles of matrix work) to hide in.
//
// A grid of one CTA for each 256 queries of a head (and at most one more a
// request), late queries (most keys) first, heads that fit into L2 together; but
// a CTA that runs goes on with the work of CTAs that have not started (a request
// for one is under way while the CTA works), so that its copies run into the next
// item while this one's last tiles and output are under way, and the SMs end
// close together.
//
// Few items with many keys (a short chunk over a long prefix, few heads): the
// CTAs of a cluster share an item's key tiles, leave their outputs and
// (maximum, sum) in shared memory, and each joins some of the rows from all of
// them.  Such CTAs have one item each.  choose_parts has the rule and figures.
//
// Warps 0-3 and 4-7: softmax and epilogue of query tile 0 and 1, a row a
// thread.  Warp 8: copies.  Warp 9: MMAs, issued from uniform control flow.
// Warps 10 and 11: the query offsets' order, which no output is stored before.
// The running maximum is raised lazily (by 2^8 at least), by the row's own
// thread, which then rescales its row of O.  P is rounded to bf16 for the
// matrix pipe (it takes operands of one type, and values are bf16), its sum kept
// unrounded in fp32.
//
// Keys behind a request's end (the next request's rows in the packed tensors)
// get probability zero, and their rows of V are cleared in shared memory: they
// may hold anything.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>

#include "dsa_ptx.cuh"
#include "dsa_internal.h"

DSA_DEFINE_ERROR_WORD(mla_prefill)

namespace dsa {
namespace {

constexpr int kTile = 128;                     // queries of a tile, keys of a tile
constexpr int kCtaRows = 2 * kTile;
constexpr int kQAtoms = 3;                     // 192 dims
constexpr int kAtomBytes = kTile * 128;        // 128 rows x 64 dims: 16 KB
constexpr int kRing = 8;
constexpr int kPerTile = 5;                    // granules of a key tile: 3 of K, 2 of V
constexpr int kHeadDim = 128;
constexpr int kOffQ = 0;
constexpr int kOffRing = 2 * kQAtoms * kAtomBytes;
constexpr int kOffBar = kOffRing + kRing * kAtomBytes;
constexpr int kKGranules = 3;
constexpr int kNumBars = 24;
constexpr int kOffTaken = kOffBar + kNumBars * 8;     // an answer of 16 bytes
constexpr int kOffItem = kOffTaken + 16;             // two records
constexpr int kOffSlot = kOffItem + 2 * 48;
constexpr int kOffFalling = kOffSlot + 4, kOffOrder = kOffSlot + 8;      // the query offsets' order
constexpr int kSmemBytes = kOffSlot + 16 + 1024;
static_assert(kOffTaken % 16 == 0, "alignment");
static_assert(kSmemBytes <= 232448, "shared memory");
constexpr int kThreads = 384;                  // two softmax warpgroups; copies, MMAs, two that check offsets
// Registers: launched with 168 a thread (384 x 168 = 64512); the softmax holds a
// row of 128 scores and takes 216, the third warpgroup keeps 72 (256 x 216 +
// 128 x 72 = 64512).
constexpr int kSoftRegs = 216, kOtherRegs = 72;
static_assert(256 * kSoftRegs + 128 * kOtherRegs <= 384 * 168, "registers");
constexpr int kSoftWarps = 8;
constexpr int kItemReaders = kSoftWarps + 1;   // and the MMA warp
constexpr int kMaxParts = 8;                   // CTAs of a cluster that share an item's keys
constexpr int kColS = 0, kColO = 256, kTmemCols = 512;
constexpr float kRaiseLog2 = 8.0f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// mbar_wait and mbar_test_wait by a whole warp: the same answer in every lane.
// (A phase may complete between two lanes' tests; lanes that then took different
// branches would meet in different votes and shuffles.)
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

__device__ __forceinline__ bool warp_test(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_test_wait(bar, parity));
}

// Keys a query row sees: its own token and those before it, or all.
__device__ __forceinline__ int key_limit(int row, int qlen, int klen, int causal) {
  return causal ? max(0, klen - qlen + row + 1) : klen;
}

// The work of one CTA (or cluster) of the grid: 256 queries of a head.
struct Item {
  int work;                  // it has queries (a record: 0 ends the CTA's work)
  int head, row0;            // first query row of the request
  int q0, k0, qlen, klen;    // the request in the packed tensors
  int nt0, nt1;              // key tiles of the two query tiles
  int base;                  // key tiles of the CTA's items before it
};
static_assert(sizeof(Item) <= 48, "record");

// Request r begins at slot (cu_q[r] + 255 r) / 256 of the grid's x: that leaves
// it as many slots as it has blocks of 256 queries, or one more (a single request
// none), and the slot of a CTA needs no walk over the requests before it to find
// its own.  (Offsets behind the packed tensor move no slot of the requests inside,
// and give slots that the grid does not have.)
__device__ __forceinline__ int first_slot(const MlaPrefillLaunch& p, int r) {
  return static_cast<int>((static_cast<uint32_t>(max(0, __ldg(p.cu_q + r))) + (kCtaRows - 1u) * r) / kCtaRows);
}

// Whether the query offsets decrease anywhere, looked for by `threads` threads
// (the answer is a thread's own).  Requests then share rows, and slots are not
// theirs: nothing of the call is written.  Offsets outside the packed tensor are
// reported here too (they need not have a slot); their requests are skipped.
__device__ __forceinline__ bool falling_offsets(const MlaPrefillLaunch& p, int tid, int threads) {
  bool falls = false, outside = false;
#pragma unroll 8
  for (int r = tid; r < p.batch; r += threads) {
    const int a = __ldg(p.cu_q + r), b = __ldg(p.cu_q + r + 1);
    falls |= b < a;
    outside |= a < 0 || b > p.total_q;
  }
  if (falls || outside) raise_error(kErrCheck);
  return falls;
}

// Item i of the grid: head groups one after another, in a group the slots, a
// slot's heads next to each other.
__device__ __forceinline__ Item item_of(const MlaPrefillLaunch& p, int i) {
  const int group = i / (p.slots * p.head_group), first = group * p.head_group;
  const int heads = min(p.head_group, p.heads - first), at = i - first * p.slots;
  const int x = at / heads, y = first + at % heads;
  int lo = 0, hi = p.batch;      // first_slot(lo) <= x < first_slot(hi), were it asked
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first_slot(p, mid) <= x) lo = mid;
    else hi = mid;
  }
  Item it;
  it.base = 0;
  it.head = y;
  it.q0 = __ldg(p.cu_q + lo);
  it.k0 = __ldg(p.cu_k + lo);
  it.qlen = __ldg(p.cu_q + lo + 1) - it.q0;
  it.klen = __ldg(p.cu_k + lo + 1) - it.k0;
  // Late queries see the most keys: they start first.
  it.row0 = (first_slot(p, lo + 1) - 1 - x) * kCtaRows;
  // Offsets outside the packed tensors, or a length above max_q, are reported;
  // the request's rows are left as they were, or not all of them written.
  const bool bad = it.q0 < 0 || it.k0 < 0 || it.qlen < 0 || it.klen < 0 ||
                   it.qlen > p.total_q - it.q0 || it.klen > p.total_k - it.k0;
  const bool far = it.row0 >= (p.max_q + kCtaRows - 1) / kCtaRows * kCtaRows;
  it.work = !bad && !far && it.row0 >= 0 && it.row0 < it.qlen ? 1 : 0;
  if (bad || (far && it.row0 < it.qlen)) raise_error(kErrCheck);
  auto tiles_from = [&](int first) {
    if (!it.work || first >= it.qlen) return 0;
    const int lim = key_limit(min(first + kTile, it.qlen) - 1, it.qlen, it.klen, p.causal);
    return (min(lim, it.klen) + kTile - 1) / kTile;
  };
  it.nt0 = tiles_from(it.row0);
  it.nt1 = tiles_from(it.row0 + kTile);
  return it;
}

// Part `rank` of `parts` of an item's key tiles, as an item of its own (keys and
// limits count from the part's first).
__device__ __forceinline__ void keep_part(Item& it, int rank, int parts) {
  const int nt = max(it.nt0, it.nt1), lo = nt * rank / parts, hi = nt * (rank + 1) / parts;
  it.nt0 = min(max(it.nt0 - lo, 0), hi - lo);
  it.nt1 = min(max(it.nt1 - lo, 0), hi - lo);
  it.k0 += lo * kTile;
  it.klen -= lo * kTile;
}

// Joins the parts of an item whose keys the kParts CTAs of a cluster shared.
// Each CTA has left its rows' unscaled outputs (512 bytes a row, 16-byte piece i
// of row r at i ^ (r & 31)) at `o` and their (maximum, sum) at `stat` of its
// shared memory, and joins rows rank, rank + kParts, ...  A warp takes kRows rows
// at a time (six to eight loads in flight): lane kParts * r + c weighs part c of
// row r, and every lane has four of each row's values.
template <int kParts>
__device__ __forceinline__ void join_parts(const MlaPrefillLaunch& p, const Item& it, uint32_t o, uint32_t stat,
                                           int rank, int warp, int lane) {
  constexpr int kRows = kMaxParts / kParts;
  const float ninf = __int_as_float(0xff800000);
  const int rows = min(kCtaRows, it.qlen - it.row0);
  const int my_r = min(lane / kParts, kRows - 1), my_c = lane % kParts;      // (the lanes left over repeat)
  const long long at0 = static_cast<long long>(it.q0 + it.row0) * p.heads + it.head;
  for (int i0 = rank + kParts * kRows * warp; i0 < rows; i0 += kParts * kRows * kSoftWarps) {
    float4 v[kRows][kParts];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int i = min(i0 + kParts * r, kCtaRows - 1);
#pragma unroll
      for (int c = 0; c < kParts; ++c)
        v[r][c] = ld_shared_cluster_f4(mapa_shared(o + i * kHeadDim * 4 + ((lane ^ (i & 31)) << 4), c));
    }
    const int mine = i0 + kParts * my_r;
    const float2 st = ld_shared_cluster_f2(mapa_shared(stat + min(mine, kCtaRows - 1) * 8, my_c));
    float top = ninf, tot = 0.f;
#pragma unroll
    for (int c = 0; c < kParts; ++c)
      top = fmaxf(top, __shfl_sync(0xffffffffu, st.x, kParts * my_r + c));
    const float w = ex2(st.x - (top > ninf ? top : 0.f));
#pragma unroll
    for (int c = 0; c < kParts; ++c) tot += __shfl_sync(0xffffffffu, w * st.y, kParts * my_r + c);
    const bool any = tot > 0.f || tot != tot;
    const float scale = any ? w / tot : 0.f;
    if (p.lse && my_c == 0 && lane < kParts * kRows && mine < rows)
      p.lse[at0 + static_cast<long long>(mine) * p.heads] = any ? (top + log2f(tot)) * kLn2 : ninf;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c = 0; c < kParts; ++c) {
        const float f = __shfl_sync(0xffffffffu, scale, kParts * r + c);
        a = make_float4(fmaf(f, v[r][c].x, a.x), fmaf(f, v[r][c].y, a.y), fmaf(f, v[r][c].z, a.z),
                        fmaf(f, v[r][c].w, a.w));
      }
      const int i = i0 + kParts * r;
      if (i < rows)
        reinterpret_cast<uint2*>(p.out + (at0 + static_cast<long long>(i) * p.heads) * kHeadDim)[lane] =
            make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    mla_prefill_kernel(const __grid_constant__ CUtensorMap tmap_q,
                       const __grid_constant__ CUtensorMap tmap_kv,
                       const __grid_constant__ CUtensorMap tmap_rope, const MlaPrefillLaunch p) {
  extern __shared__ uint8_t smem_raw[];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const float ninf = __int_as_float(0xff800000);

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffSlot);
  volatile int* falling = reinterpret_cast<int*>(smem + kOffFalling);
  const uint32_t bar0 = sbase + kOffBar;
// K / V of key tile j, counted over the CTA's items (at most two of each are in
// the ring): landed, and read.
#define K_FULL(j) (bar0 + 8u * ((j) & 1))
#define V_FULL(j) (bar0 + 16u + 8u * ((j) & 1))
#define K_EMPTY(j) (bar0 + 32u + 8u * ((j) & 1))
#define V_EMPTY(j) (bar0 + 48u + 8u * ((j) & 1))
#define PARITY(j) (((j) >> 1) & 1)
// Of query tile q: q landed / read by its last Q K^T, scores, probabilities,
// output of the item complete.
#define Q_FULL(q) (bar0 + 64u + 8u * (q))
#define Q_EMPTY(q) (bar0 + 80u + 8u * (q))
#define S_FULL(q) (bar0 + 96u + 8u * (q))
#define O_FULL(q) (bar0 + 112u + 8u * (q))
#define P_FULL(q) (bar0 + 128u + 8u * (q))
#define DRAIN (bar0 + 144u)
#define TAKEN (bar0 + 152u)
// Item k's record written / no longer needed by any role.
#define ITEM_FULL(k) (bar0 + 160u + 8u * ((k) & 1))
#define ITEM_EMPTY(k) (bar0 + 176u + 8u * ((k) & 1))
// The query offsets have been looked through.
#define ORDER (sbase + kOffOrder)

  if (warp == 8 && lane == 0) {
    for (int q = 0; q < 2; ++q) {
      mbar_init(K_FULL(q), 1);
      mbar_init(V_FULL(q), 1);
      mbar_init(K_EMPTY(q), 1);
      mbar_init(V_EMPTY(q), 1);
      mbar_init(Q_FULL(q), 1);
      mbar_init(Q_EMPTY(q), 1);
      mbar_init(ITEM_FULL(q), 1);
      mbar_init(ITEM_EMPTY(q), kItemReaders);
      mbar_init(S_FULL(q), 1);
      mbar_init(P_FULL(q), kTile);
      mbar_init(O_FULL(q), 1);
    }
    mbar_init(DRAIN, 1);
    mbar_init(TAKEN, 1);
    mbar_init(ORDER, 2);
    *falling = 0;
    fence_mbar_init();
    prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_kv);
    prefetch_tmap(&tmap_rope);
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  const Item* items = reinterpret_cast<const Item*>(smem + kOffItem);      // 48 bytes apart
  auto record = [&](int k) -> const Item& {
    return *reinterpret_cast<const Item*>(reinterpret_cast<const uint8_t*>(items) + 48 * (k & 1));
  };

  if (warp >= 8) {
    setmaxnreg_dec<kOtherRegs>();
    if (warp == 8) {
      // ------------------------------------------------------------- copies
      if (lane == 0) {
        bool ok = true;
        int n = 0;                                          // granules so far
        int uses0 = 0, uses1 = 0;                           // items that had each query tile
        const uint64_t pol_rope = policy_evict_last();      // every head reads it
        Item it = item_of(p, static_cast<int>(blockIdx.x) / p.parts);
        if (p.parts > 1) keep_part(it, static_cast<int>(blockIdx.x) % p.parts, p.parts);
        int base = 0, k = 0, asked = 0;
        bool more = true;
        while (ok) {
          if (it.work || !more) {
            // The other roles work from the record (one with work = 0 ends them).
            if (k >= 2 && !(ok = mbar_wait(ITEM_EMPTY(k), PARITY(k) ^ 1))) break;
            it.base = base;
            if (!more) it.work = 0;
            const_cast<Item&>(record(k)) = it;
            mbar_arrive(ITEM_FULL(k));
            ++k;
            if (!more) break;
          }
          const int ntmax = max(it.nt0, it.nt1);
          for (int j = 0; ok && j < ntmax; ++j) {
            for (int g = 0; g < kPerTile; ++g, ++n) {
              // The granule's slot held granule n - kRing, of an earlier tile.
              const int old = n - kRing, oj = old / kPerTile;
              if (old >= 0 &&
                  !(ok = mbar_wait(old % kPerTile < kKGranules ? K_EMPTY(oj) : V_EMPTY(oj), PARITY(oj))))
                break;
              const uint32_t bar = g < kKGranules ? K_FULL(base + j) : V_FULL(base + j);
              if (g == 0) mbar_expect_tx(bar, kKGranules * kAtomBytes);
              if (g == kKGranules) mbar_expect_tx(bar, (kPerTile - kKGranules) * kAtomBytes);
              const uint32_t dst = sbase + kOffRing + (n % kRing) * kAtomBytes;
              const int row = it.k0 + j * kTile;
              if (g == 2) tma_load_2d(dst, &tmap_rope, 0, row, bar, pol_rope);
              else tma_load_4d(dst, &tmap_kv, 0, row, g < 2 ? g : g - 1, it.head, bar);
              if (j == 0 && g < 2 && (g == 0 ? it.nt0 : it.nt1) > 0) {
                const int used = g == 0 ? uses0++ : uses1++;
                if (used > 0 && !(ok = mbar_wait(Q_EMPTY(g), (used - 1) & 1))) break;
                mbar_expect_tx(Q_FULL(g), kQAtoms * kAtomBytes);
                tma_load_4d(sbase + kOffQ + g * kQAtoms * kAtomBytes, &tmap_q, 0,
                            it.q0 + it.row0 + g * kTile, 0, it.head, Q_FULL(g));
              }
            }
          }
          base += ntmax;
          // The next item, once this one's copies are under way (not earlier:
          // items go to the CTAs that come free first).
          if (!ok) break;
          if (p.parts > 1) {
            more = false;
            continue;
          }
          mbar_expect_tx(TAKEN, 16);
          take_cta(sbase + kOffTaken, TAKEN);
          if (!(ok = mbar_wait(TAKEN, asked++ & 1))) break;
          uint32_t x, y, z;
          more = taken_cta(sbase + kOffTaken, x, y, z);
          fence_proxy_async_smem();      // read before the next answer is written there
          if (more) it = item_of(p, x);
        }
        if (!ok) raise_error(kErrTimeout);
        // No copy is in flight when the CTA ends.  (After a wait that ran out, the
        // copies before it have had that long to land.)
        if (ok)
          for (int j = max(0, base - 2); j < base; ++j) {
            mbar_wait(K_FULL(j), PARITY(j));
            mbar_wait(V_FULL(j), PARITY(j));
          }
        if (ok && uses0 > 0) mbar_wait(Q_FULL(0), (uses0 - 1) & 1);
        if (ok && uses1 > 0) mbar_wait(Q_FULL(1), (uses1 - 1) & 1);
      }
      __syncwarp();
    } else if (warp == 9) {
      // --------------------------------------------------------------- MMAs
      const uint32_t el = elect_one() ? 1u : 0u;
      constexpr uint32_t idesc_qk = make_idesc(1, 1, 0, 0, kTile, kTile);
      constexpr uint32_t idesc_pv = make_idesc(1, 1, 0, 1, 64, kTile);
      const uint64_t dq0 = smem_desc_sw128(sbase + kOffQ, 16, 1024);
      const uint64_t dr0 = smem_desc_sw128(sbase + kOffRing, 16, 1024);
      // (V: MN-major, an MMA for each granule's 64 dims: with A in tensor memory
      // N = 64 runs at the full rate, and granules need not lie side by side.)
      bool ok = true;
      // A phase is tested before the last MMAs of the step before go out, so that
      // the test's latency hides behind them; `want` waits only if it was not
      // complete then.
      uint32_t done_bar = 0, done_parity = 0;
      auto want = [&](uint32_t bar, uint32_t parity) {
        if (ok && !(done_bar == bar && done_parity == parity)) ok = warp_wait(bar, parity);
        done_bar = 0;
      };
      auto peek = [&](uint32_t bar, uint32_t parity) {
        if (warp_test(bar, parity)) {
          done_bar = bar;
          done_parity = parity;
        }
      };
      // (A phase that completed stays the barrier's latest until its data has
      // been used, so a remembered answer does not go stale before that; it is
      // dropped after a use.)
      // Descriptor offset of granule g of tile t, broadcast: the compiler then
      // knows it to be the same in every lane and keeps it in uniform registers.
      auto slot_of = [&](int t, int g) -> uint64_t {
        return static_cast<uint32_t>(
            __shfl_sync(0xffffffffu, (((t * kPerTile + g) % kRing) * kAtomBytes) >> 4, 0));
      };
      // Q K^T and P V of query tile q over key tile t (counted over the items);
      // next_bar: what the step after it waits for.
      auto qk = [&](int q, int t, uint32_t next_bar, uint32_t next_parity) {
#pragma unroll
        for (int a = 0; a < kQAtoms; ++a) {
          const uint64_t dk = dr0 + slot_of(t, a);
          const uint64_t dq = dq0 + static_cast<uint64_t>(((q * kQAtoms + a) * kAtomBytes) >> 4);
          if (a == kQAtoms - 1) peek(next_bar, next_parity);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16_ss_uni(tmem + kColS + kTile * q, dq + static_cast<uint64_t>((32 * k) >> 4),
                           dk + static_cast<uint64_t>((32 * k) >> 4), idesc_qk, (a > 0 || k > 0) ? 1u : 0u, el);
        }
        if (el) tc_commit(S_FULL(q));
        __syncwarp();
      };
      auto pv = [&](int q, int t, bool first, uint32_t next_bar, uint32_t next_parity) {
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const uint64_t dv = dr0 + slot_of(t, kKGranules + a);
          if (a == 1) peek(next_bar, next_parity);
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            mma_f16_ts_uni(tmem + kColO + kHeadDim * q + 64 * a, tmem + kColS + kTile * q + 8 * k,
                           dv + static_cast<uint64_t>((2048 * k) >> 4), idesc_pv, (!first || k > 0) ? 1u : 0u,
                           el);
        }
      };
      auto commit = [&](uint32_t bar) {
        if (el) tc_commit(bar);
        __syncwarp();
      };
      int base = 0, c0 = 0, c1 = 0;          // key tiles so far: all, and of each query tile
      int items0 = 0, items1 = 0;            // items that had each query tile
      // P V of query tile 1 goes out one step late, after Q K^T of query tile 0
      // over the next key tile (the next item's first, at the end of one).
      bool held = false, held_pv = false, held_v = false, held_first = false, held_last = false;
      int held_t = 0, held_c = 0;
      auto issue_held = [&](uint32_t next_bar, uint32_t next_parity) {
        if (!held || !ok) return;
        held = false;
        if (held_pv) {
          if (!held_v) ok = warp_wait(V_FULL(held_t), PARITY(held_t));
          want(P_FULL(1), held_c & 1);
          tc_fence_after();
          if (!ok) return;
          pv(1, held_t, held_first, next_bar, next_parity);
          if (held_last) commit(O_FULL(1));
        }
        commit(V_EMPTY(held_t));
      };
      for (int item = 0; ok; ++item) {
        // (What is held back does not wait for a record, or an item without keys,
        // to come.)
        if (!warp_test(ITEM_FULL(item), PARITY(item))) issue_held(DRAIN, 0);
        if (!(ok = ok && warp_wait(ITEM_FULL(item), PARITY(item)))) break;
        const int work = __shfl_sync(0xffffffffu, record(item).work, 0);
        const int nt0 = __shfl_sync(0xffffffffu, record(item).nt0, 0);
        const int nt1 = __shfl_sync(0xffffffffu, record(item).nt1, 0), ntmax = max(nt0, nt1);
        if (lane == 0) mbar_arrive(ITEM_EMPTY(item));
        if (!work) break;
        if (ntmax == 0) issue_held(DRAIN, 0);
        for (int j = 0; ok && j < ntmax; ++j) {
          const int t = base + j;
          if (j < nt0) {
            // (A new item's q and first keys may not have landed yet: then the
            // P V that is held back does not wait for them.)
            if (j == 0) {
              if (held && !(warp_test(Q_FULL(0), items0 & 1) && warp_test(K_FULL(t), PARITY(t))))
                issue_held(K_FULL(t), PARITY(t));
              ok = ok && warp_wait(Q_FULL(0), items0 & 1);
              ++items0;
            }
            want(K_FULL(t), PARITY(t));
            tc_fence_after();
            if (!ok) break;
            qk(0, t, P_FULL(1), held_c & 1);
            if (j == nt0 - 1) commit(Q_EMPTY(0));
          }
          issue_held(K_FULL(t), PARITY(t));
          if (!ok) break;
          if (j < nt1) {
            if (j == 0) {
              ok = warp_wait(Q_FULL(1), items1 & 1);
              ++items1;
            }
            if (j >= nt0) want(K_FULL(t), PARITY(t));
            tc_fence_after();
            if (!ok) break;
            qk(1, t, P_FULL(0), c0 & 1);
            if (j == nt1 - 1) commit(Q_EMPTY(1));
          }
          commit(K_EMPTY(t));
          if (j < nt0) {
            ok = warp_wait(V_FULL(t), PARITY(t));
            want(P_FULL(0), c0 & 1);
            tc_fence_after();
            if (!ok) break;
            pv(0, t, j == 0, K_FULL(t + 1), PARITY(t + 1));
            if (j == nt0 - 1) commit(O_FULL(0));
            ++c0;
          }
          held = true;
          held_pv = j < nt1;
          held_v = j < nt0;
          held_first = j == 0;
          held_last = j == nt1 - 1;
          held_t = t;
          held_c = c1;
          if (j < nt1) ++c1;
        }
        base += ntmax;
      }
      issue_held(DRAIN, 0);
      if (!ok && el) raise_error(kErrTimeout);
      if (el) tc_commit(DRAIN);      // every MMA is done before TMEM is freed
      __syncwarp();
      mbar_wait(DRAIN, 0);
    } else {
      // ------------------------------------------------ order of the offsets
      const bool falls = __any_sync(0xffffffffu, falling_offsets(p, (warp - 10) * 32 + lane, 64));
      if (lane == 0) {
        if (falls) *falling = 1;
        mbar_arrive(ORDER);
      }
    }
    __syncwarp();
    if (p.parts > 1) cluster_sync();      // the softmax warps' parts are written
  } else {
    // ---------------------------------------------- softmax and epilogue
    setmaxnreg_inc<kSoftRegs>();
    const int q = warp >> 2, w4 = warp & 3;
    const uint32_t tS = tmem + (static_cast<uint32_t>(w4 * 32) << 16) + kColS + kTile * q;
    const uint32_t tO = tmem + (static_cast<uint32_t>(w4 * 32) << 16) + kColO + kHeadDim * q;
    const float sc = p.sm_scale * kLog2e;
    bool ok = true;
    int phase = 0;             // parities: bit 0 of the scores, bit 1 of the outputs
    int n = 0;                 // key tiles of the item
    float mrun = ninf, lrun = 0.f;
    // (Ahead of the items: the offsets have been looked through before the first
    // scores come, but for tens of thousands of requests: 23 us of 1765 for 65535.
    // Asked for in the first item's epilogue, 1 % of every item, 31 to 50 ns.)
    const bool known = warp_wait(ORDER, 0), refused = !known || *falling;
    ok = known;
    for (int item = 0; ok; ++item) {
      if (!(ok = warp_wait(ITEM_FULL(item), PARITY(item)))) break;
      const int row = q * kTile + w4 * 32 + lane;     // from the item's first
      int lim, vlive;
      {
        const Item& it = record(item);
        if (!it.work) break;
        n = q == 0 ? it.nt0 : it.nt1;
        lim = min(it.klen, key_limit(it.row0 + row, it.qlen, it.klen, p.causal));
        // Keys of the request behind the tile's start, where this query tile is
        // the first to read the tile's V.
        vlive = it.klen;
      }
      mrun = ninf;
      lrun = 0.f;
      for (int j = 0; j < n; ++j, phase ^= 1, lim -= kTile, vlive -= kTile) {
        if (ok && !mbar_wait(S_FULL(q), phase & 1)) ok = false;
        tc_fence_after();
        uint32_t s[128];
        tmem_ld128(tS, s);
        const int seen = lim;
        float mx[4] = {ninf, ninf, ninf, ninf};
        if (__any_sync(0xffffffffu, seen < kTile)) {
  #pragma unroll
          for (int e = 0; e < kTile; ++e)
            if (e >= seen) s[e] = __float_as_uint(ninf);
        }
  #pragma unroll
        for (int e = 0; e < kTile; e += 2)
          mx[(e >> 1) & 3] = max3(mx[(e >> 1) & 3], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
        const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
        const bool raise = tmax > mrun + kRaiseLog2;
        const bool rescale = raise && mrun > ninf;
        if (__any_sync(0xffffffffu, rescale)) {
          // (P V of the tile before is done: it was issued before this Q K^T.)
          const float f = rescale ? ex2(mrun - tmax) : 1.f;
  #pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * c, o);
  #pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(tO + 32 * c, o);
          }
          lrun *= f;
        }
        if (raise) mrun = tmax;
        const float mref = mrun > ninf ? mrun : 0.f;
        // Rows of V behind the request's end are cleared, by the first query
        // tile that reads them.
        if (vlive < kTile && (q == 0 || j >= record(item).nt0)) {
          const int t = record(item).base + j;
          if (ok && !mbar_wait(V_FULL(t), PARITY(t))) ok = false;
  #pragma unroll 1
          for (int a = 0; a < 2; ++a) {
            uint4* v = reinterpret_cast<uint4*>(smem + kOffRing + ((t * kPerTile + 3 + a) % kRing) * kAtomBytes);
            for (int e = (threadIdx.x & 127) + vlive * 8; e < kAtomBytes / 16; e += 128)
              v[e] = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        // P V over the first 64 keys starts while the others' exponentials run.
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  #pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
  #pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x = fma2(make_float2(__uint_as_float(s[32 * c + 2 * e]),
                                              __uint_as_float(s[32 * c + 2 * e + 1])),
                                  make_float2(sc, sc), make_float2(-mref, -mref));
            const float2 w = make_float2(ex2(x.x), ex2(x.y));
            ls[e & 1] = add2(ls[e & 1], w);
            pk[e] = pack_bf16x2(w.x, w.y);
          }
          tmem_st16_async(tS + 16 * c, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(P_FULL(q));
        lrun += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
      }
      if (n > 0) {
        if (ok && !mbar_wait(O_FULL(q), (phase >> 1) & 1)) ok = false;
        tc_fence_after();
        phase ^= 2;
      }
      const Item& it = record(item);
      if (p.parts == 1 && !refused && it.row0 + q * kTile < it.qlen) {
        const bool live = it.row0 + row < it.qlen;
        const bool any = lrun > 0.f || lrun != lrun;
        const float inv = any ? 1.f / lrun : 0.f;
        const long long at = static_cast<long long>(it.q0 + it.row0 + row) * p.heads + it.head;
        uint4* dst = reinterpret_cast<uint4*>(p.out + at * kHeadDim);
  #pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          if (n > 0) tmem_ld32(tO + 32 * c, o);
          if (!live) continue;
          uint32_t w[2][8];
  #pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e >> 3][e & 7] =
                any ? pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv) : 0u;
  #pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (p.out_wide) {
              st_global_32(dst + 4 * c + 2 * e, w[e]);
            } else {
              dst[4 * c + 2 * e] = make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
              dst[4 * c + 2 * e + 1] = make_uint4(w[e][4], w[e][5], w[e][6], w[e][7]);
            }
          }
        }
        if (live && p.lse) p.lse[at] = any ? (mrun + log2f(lrun)) * kLn2 : ninf;
      }
      tc_fence_before();
      ok = __all_sync(0xffffffffu, ok);
      if (lane == 0) mbar_arrive(ITEM_EMPTY(item));
    }
    if (!ok && lane == 0) raise_error(kErrTimeout);
    if (p.parts > 1) {
      const int row = threadIdx.x;
      float4* o_row = reinterpret_cast<float4*>(smem + kOffRing + row * 512);
      named_bar_sync(1, 2 * kTile);      // both query tiles' MMAs are done: the ring and q are free
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        if (n > 0) tmem_ld32(tO + 32 * c, o);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          o_row[(8 * c + e) ^ (row & 31)] =
              n > 0 ? make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                  __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]))
                    : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      reinterpret_cast<float2*>(smem + kOffQ)[row] = make_float2(mrun, lrun);
      tc_fence_before();
      __syncwarp();
      cluster_sync();
      const Item it = record(0);
      const int rank = static_cast<int>(cluster_ctarank());
      if (ok && it.work && !refused) {
        const uint32_t o = sbase + kOffRing, stat = sbase + kOffQ;
        switch (p.parts) {
          case 2: join_parts<2>(p, it, o, stat, rank, warp, lane); break;
          case 3: join_parts<3>(p, it, o, stat, rank, warp, lane); break;
          case 4: join_parts<4>(p, it, o, stat, rank, warp, lane); break;
          case 5: join_parts<5>(p, it, o, stat, rank, warp, lane); break;
          case 6: join_parts<6>(p, it, o, stat, rank, warp, lane); break;
          case 7: join_parts<7>(p, it, o, stat, rank, warp, lane); break;
          default: join_parts<8>(p, it, o, stat, rank, warp, lane); break;
        }
      }
      __syncwarp();
    }
  }
  __syncthreads();
  if (p.parts > 1) cluster_sync();      // the others have read this CTA's part
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
#undef K_FULL
#undef V_FULL
#undef K_EMPTY
#undef V_EMPTY
#undef PARITY
#undef Q_FULL
#undef S_FULL
#undef P_FULL
#undef O_FULL
#undef Q_EMPTY
#undef TAKEN
#undef ITEM_FULL
#undef ITEM_EMPTY
#undef DRAIN
#undef ORDER
}

}  // namespace

namespace {

// Clusters of `parts` CTAs that run at a time on the current device.
int clusters_at_once(int parts) {
  static std::atomic<int> known[64][kMaxParts + 1];
  const int sms = device_sm_count();
  if (parts == 1) return sms;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return sms / parts;
  int n = known[dev][parts].load(std::memory_order_relaxed);
  if (n > 0) return n;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = parts;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(parts);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, mla_prefill_kernel, &cfg) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();
    n = sms / parts;
  }
  known[dev][parts].store(n, std::memory_order_relaxed);
  return n;
}

// Heads whose items run together.  Late items are long and early ones short, so
// the order late to early over all heads ends with short ones and the SMs end
// close together; but heads that run together share L2, and each item reads a
// head's keys from its first.  So as many as have 48 MB of keys and values, in
// groups of equal size.  Measured for one head after another / 16 / 48 / 96 MB /
// all heads together, us: 4096 tokens, 32 heads, 143 / 143 / 115 / 117 / 117; 4000,
// 16 heads, 94 / 66 / 66 / 66 / 66; 6000, 32 heads, 268 / 252 / 229 / 232 / 231; 8192,
// 128 heads, 1712 / 1749 / 1698 / 1659 / 1751; 3000, 128 heads, 270 / 258 / 252 / 258 /
// 274; 8 of 1037, 128 heads, 397 / 393 / 397 / 432 / 432.
int heads_at_once(const MlaPrefillLaunch& a) {
  const double bytes = 48 << 20, head = static_cast<double>(a.total_k) / a.batch * 2 * kHeadDim * 2;
  const int groups = static_cast<int>(std::ceil(a.heads / std::max(1.0, std::min<double>(a.heads, bytes / (head + 1)))));
  return (a.heads + groups - 1) / groups;
}

// CTAs that share an item's keys.  Costs in key tiles (1.75 us), from the mean
// lengths (the lengths themselves are on the device): the late items' tiles, 4
// for the start and end of an item of one CTA, 5.5 + 0.3 c with the join of c
// parts; items that come in rounds leave SMs idle in the last one.  Measured for
// 1 / 2 / 4 / 6 / 8 parts, us: 1 query over 16000 keys, 8 heads, 199 / 113 / 64 /
// 46 / 38; 64 over 16000, 24 heads, 201 / 109 / 64 / 91 / 74 (5: 58); 1000 over
// 5000, 16 heads, 79 / 51 / 62 / 74 / 106; 1000 over 1000, 25 / 23 / 33 / 46 /
// 68; 2 x 512 over 16513, 128 heads, 922 / 875 / 1027 / 1144 / 1365; 77 over 77, 16
// heads, 11 / 15 / 15 / 15 / 24.
int choose_parts(const MlaPrefillLaunch& a) {
  const double queries = static_cast<double>(a.total_q) / a.batch;
  const double blocks = std::max(1.0, std::ceil(queries / kCtaRows));      // of a request
  const double items = blocks * a.batch * a.heads;
  const double keys = static_cast<double>(a.total_k) / a.batch / kTile;    // key tiles of a late item ...
  if (keys <= 4) return 1;                                                 // two parts cost 8 at least
  const double spread =                                                    // ... and how many fewer an early one has
      a.causal ? std::min(keys, queries * (blocks - 1) / blocks / kTile) : 0;
  int best = 1;
  double best_cost = 0;
  for (int c = 1; c <= kMaxParts; ++c) {
    const double extra = c == 1 ? 4 : 5.5 + 0.3 * c, n = clusters_at_once(c);
    const double most = std::ceil(keys / c) + extra;
    const double mean = (keys - spread / 2) / c + extra, least = (keys - spread) / c + extra;
    const double cost = std::max(most, (items * mean + (std::ceil(items / n) * n - items) * least) / n);
    if (c == 1 || cost < 0.97 * best_cost) {
      best = c;
      best_cost = cost;
    }
  }
  return best;
}

}  // namespace

namespace {
long long slots_of(const MlaPrefillLaunch& a) { return (a.total_q + (kCtaRows - 1LL) * a.batch) / kCtaRows; }
}  // namespace

long long mla_prefill_items(const MlaPrefillLaunch& a) { return slots_of(a) * a.heads; }

cudaError_t launch_mla_prefill(MlaPrefillLaunch a, cudaStream_t s) {
  // Outputs of a thread's row are stored 32 bytes (a whole sector) at a time
  // where they are aligned so.
  a.out_wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
  const uint64_t H = a.heads, Tq = a.total_q, Tk = a.total_k > 0 ? a.total_k : 1;
  // Rows as 64-dim atoms (a box: 128 rows of one or three atoms of a head).
  const uint64_t qdims[4] = {64, Tq, kQAtoms, H}, qstr[3] = {H * 384, 128, 384};
  const uint64_t kdims[4] = {64, Tk, 4, H}, kstr[3] = {H * 512, 128, 512};
  const uint32_t qbox[4] = {64, kTile, kQAtoms, 1}, kbox[4] = {64, kTile, 1, 1};
  CUtensorMap tq, tk, tr;
  if (!encode_tmap_nd(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, 4, qdims, qstr, qbox,
                      CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tmap_nd(&tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.kv, 4, kdims, kstr, kbox,
                      CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tmap_2d(&tr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.k_rope, 64, Tk,
                      static_cast<uint64_t>(a.ld_rope) * 2, 64, kTile, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(mla_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSmemBytes);
  if (e != cudaSuccess) return e;
  a.parts = choose_parts(a);
  a.slots = static_cast<int>(slots_of(a));
  a.head_group = heads_at_once(a);
  const long long ctas = mla_prefill_items(a) * a.parts;
  if (ctas > INT_MAX) return cudaErrorInvalidValue;      // (parts are 1 where there are many items)
  const dim3 grid(static_cast<unsigned>(ctas));
  return launch_kernel(mla_prefill_kernel, grid, dim3(kThreads), kSmemBytes, s, false, a.parts, tq, tk, tr, a);
}

}  // namespace dsa
