// gqa_prefill.cu -- attention over packed prompts for layers with grouped heads:
// G query heads share a key / value head of 64 or 128 dims (the textbook form).
//
//   x[i, j] = sm_scale * q[i] . k[j],  out[i] = sum_j softmax(x[i])[j] * v[j],
//   lse[i] = log sum_j exp(x[i, j])
//
// over the keys j < lim[i]: all of the request's, or up to the query's own token
// (the queries are the last of the request's tokens).  Requests are packed one
// after another.
//
// The rows of a query tile (M = 128) are the G heads of 128 / G queries, head
// fastest: they read the same keys, so a short prompt fills tiles that a tile a
// head would leave nearly empty, a key tile is read once for all of a group, and
// at the diagonal a tile covers few queries, so little of what it computes is
// masked.  (Rows 128 / G * G and up, where G is no divisor, are computed and not
// used.)
//
// D = 128 is bound by the matrix pipe (512 flop a visible pair): 4096 queries over
// 4096 keys, 64 heads on 8, take 317 us, 1.73 PFLOP/s, 91 % of the measured matrix
// rate; a prompt of 8192 with a causal mask 640 us (1.72).  D = 64 is bound by the
// softmax, which has as many exponentials for half the products: 263 us for the
// first (1.05 PFLOP/s), the matrix pipe and the special function units 44 % busy
// each.  (Without the exponentials and the maximum, whose results it could not do
// without, it would take 195.)
//
// One CTA = two query tiles over the same keys: while one tile's scores are in the
// softmax, the matrix pipe works on the other's.
//
// Tensor memory (512 columns): S (fp32) of the two tiles, one buffer of 128 keys each
// (D = 128), two of 96 (D = 64: Q K^T of the next key tile is done while this one's
// is in the softmax; 16 ragged prompts, 32 heads: one buffer of 128 158 us, two of 96
// 137; three query tiles with one buffer of 96 each, 141), and O of the two.  P (bf16)
// overwrites the S it came from and is the A operand of P V, so it never passes
// through shared memory.
// Shared memory: q of both tiles, and a ring of key tiles, K and V of each in atoms of
// 64 dims (128B swizzle).
//
// Each query tile has an MMA warp of its own, which answers that tile's probabilities
// at once, whatever the other is at.  (One for both in a fixed order: 321 us for the
// 4096 by 4096 above, instead of 317.)
//
// A grid of one CTA for each block of two query tiles of a key head (and at most
// one more a request), late queries (most keys) first, heads that fit into L2
// together; but a CTA that runs goes on with the work of CTAs that have not started
// (a request for one is under way while the CTA works), so that its copies run into
// the next item while this one's last tiles and output are under way, and the SMs
// end close together.
//
// Few items with many keys (a short chunk over a long prefix, few heads; or the last
// ones of a call, which would leave most SMs idle): the CTAs
// of a cluster share an item's key tiles, leave their outputs and (maximum, sum)
// in shared memory, and each joins some of the rows from all of them.  Such CTAs
// have one item each.  choose_plan has the rule and figures.
//
// Warps 0-3 and 4-7: softmax and epilogue of query tile 0 and 1, a row a thread.
// Warp 8: copies.  Warps 9 and 10: MMAs of query tile 0 and 1, issued from uniform
// control flow.  Warp 11: the query offsets' order, which no output is stored before.
// (16 softmax warps, half a row a thread, D = 64: 317 us instead of 270.)  The running
// maximum is raised lazily (by 2^8 at least), by the row's own thread, which then
// rescales its row of O.  P is rounded to bf16 for the matrix pipe (it takes
// operands of one type, and values are bf16), its sum kept unrounded in fp32.
//
// Keys behind a request's end (the next request's rows in the packed tensors) get
// probability zero, and their rows of V are cleared in shared memory: they may
// hold anything.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>

#include "dsa_ptx.cuh"
#include "dsa_internal.h"

DSA_DEFINE_ERROR_WORD(gqa_prefill)

namespace dsa {
namespace {

constexpr int kTile = 128;                     // rows of a query tile
constexpr int kAtomBytes = kTile * 128;        // 128 rows x 64 dims: 16 KB
constexpr int kNumBars = 40;

// Shared memory for heads of kDim dims.
template <int kDim>
struct Geo {
  static constexpr int kAtoms = kDim / 64;
  // Keys of a key tile, and buffers of scores: with two, Q K^T of a query tile's next key
  // tile is done while this one's is in the softmax (D = 64: 4 x 96 columns of tensor
  // memory, and 2 x 64 of outputs; D = 128 leaves room for one of 128).
  static constexpr int kBufs = kDim == 128 ? 1 : 2, kKeys = kDim == 128 ? 128 : 96;
  static constexpr int kColO = 2 * kBufs * kKeys;
  static_assert(kColO + 2 * kDim <= 512, "tensor memory");
  static constexpr int kOperand = kAtoms * kAtomBytes;      // q of a tile
  static constexpr int kKeyAtom = kKeys * 128, kKeyOperand = kAtoms * kKeyAtom;      // K or V of a key tile
  static constexpr int kStages = kDim == 128 ? 2 : 4;       // key tiles in the ring
  static constexpr int kOffQ = 0;
  static constexpr int kOffRing = 2 * kOperand;             // a stage: K, V
  static constexpr int kOffBar = kOffRing + kStages * 2 * kKeyOperand;
  static constexpr int kOffTaken = kOffBar + kNumBars * 8;  // an answer of 16 bytes
  static constexpr int kOffItem = kOffTaken + 16;           // two records
  static constexpr int kOffSlot = kOffItem + 2 * 48;
  static constexpr int kOffFalling = kOffSlot + 4, kOffOrder = kOffSlot + 8;      // the query offsets' order
  static constexpr int kSmemBytes = kOffSlot + 16 + 1024;
  static_assert(kOffTaken % 16 == 0, "alignment");
  static_assert(kSmemBytes <= 232448, "shared memory");
  static_assert(2 * kTile * kDim * 4 <= kStages * 2 * kKeyOperand, "a part's outputs lie in the ring");
};
constexpr int kThreads = 384;                  // two softmax warpgroups; copies, MMAs, the offsets
// Registers: launched with 168 a thread (384 x 168 = 64512); the softmax holds a
// row of 128 scores and takes 216, the third warpgroup keeps 72 (256 x 216 +
// 128 x 72 = 64512).
constexpr int kSoftRegs = 216, kOtherRegs = 72;
static_assert(256 * kSoftRegs + 128 * kOtherRegs <= 384 * 168, "registers");
constexpr int kSoftWarps = 8;
constexpr int kItemReaders = kSoftWarps + 2;   // and the MMA warps
constexpr int kMaxParts = 8;                   // CTAs of a cluster that share an item's keys
constexpr int kColS = 0, kTmemCols = 512;
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

// Keys a query sees: its own token and those before it, or all.
__device__ __forceinline__ int key_limit(int query, int qlen, int klen, int causal) {
  return causal ? max(0, klen - qlen + query + 1) : klen;
}

// The work of one CTA (or cluster) of the grid: two query tiles of a key head.
struct Item {
  int work;                  // it has queries (a record: 0 ends the CTA's work)
  int head, row0;            // key head; first query of the request
  int q0, k0, qlen, klen;    // the request in the packed tensors
  int nt0, nt1;              // key tiles of the two query tiles
  int base;                  // key tiles of the CTA's items before it
};
static_assert(sizeof(Item) <= 48, "record");

// Request r begins at slot (cu_q[r] + (n - 1) r) / n of the grid's x, for blocks of n
// queries: that leaves it as many slots as it has blocks, or one more (a single
// request none), and the slot of a CTA needs no walk over the requests before it to
// find its own.  (Offsets behind the packed tensor move no slot of the requests
// inside, and give slots that the grid does not have.)
__device__ __forceinline__ int first_slot(const GqaPrefillLaunch& p, int r) {
  const uint32_t n = 2 * p.tile_q;
  return static_cast<int>((static_cast<uint32_t>(max(0, __ldg(p.cu_q + r))) + (n - 1) * r) / n);
}

// Whether the query offsets decrease anywhere, looked for by `threads` threads
// (the answer is a thread's own).  Requests then share rows, and slots are not
// theirs: nothing of the call is written.  Offsets outside the packed tensor are
// reported here too (they need not have a slot); their requests are skipped.
__device__ __forceinline__ bool falling_offsets(const GqaPrefillLaunch& p, int tid, int threads) {
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

// Item i of the call, the launch's first and so many more: head groups one after
// another, in a group the slots, a slot's heads next to each other.
template <int kKeys>
__device__ __forceinline__ Item item_of(const GqaPrefillLaunch& p, int from_first) {
  const int i = p.first_item + from_first;
  const int block = 2 * p.tile_q;
  const int group = i / (p.slots * p.head_group), first = group * p.head_group;
  const int heads = min(p.head_group, p.kv_heads - first), at = i - first * p.slots;
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
  it.row0 = (first_slot(p, lo + 1) - 1 - x) * block;
  // Offsets outside the packed tensors, or a length above max_q, are reported;
  // the request's rows are left as they were, or not all of them written.
  const bool bad = it.q0 < 0 || it.k0 < 0 || it.qlen < 0 || it.klen < 0 ||
                   it.qlen > p.total_q - it.q0 || it.klen > p.total_k - it.k0;
  const bool far = it.row0 >= (p.max_q + block - 1LL) / block * block;
  it.work = !bad && !far && it.row0 >= 0 && it.row0 < it.qlen ? 1 : 0;
  if (bad || (far && it.row0 < it.qlen)) raise_error(kErrCheck);
  auto tiles_from = [&](int first) {
    if (!it.work || first >= it.qlen) return 0;
    const int lim = key_limit(min(first + p.tile_q, it.qlen) - 1, it.qlen, it.klen, p.causal);
    return (min(lim, it.klen) + kKeys - 1) / kKeys;
  };
  it.nt0 = tiles_from(it.row0);
  it.nt1 = tiles_from(it.row0 + p.tile_q);
  return it;
}

// Part `rank` of `parts` of an item's key tiles, as an item of its own (keys and
// limits count from the part's first).
template <int kKeys>
__device__ __forceinline__ void keep_part(Item& it, int rank, int parts) {
  const int nt = max(it.nt0, it.nt1), lo = nt * rank / parts, hi = nt * (rank + 1) / parts;
  it.nt0 = min(max(it.nt0 - lo, 0), hi - lo);
  it.nt1 = min(max(it.nt1 - lo, 0), hi - lo);
  it.k0 += lo * kKeys;
  it.klen -= lo * kKeys;
}

// Joins the parts of an item whose keys the kParts CTAs of a cluster shared.
// Each CTA has left its rows' unscaled outputs (16-byte piece i of row r at
// i ^ (r % pieces)) at `o` and their (maximum, sum) at `stat` of its shared memory,
// and joins rows rank, rank + kParts, ...  A warp takes kRows rows at a time (six to
// eight loads in flight): lane kParts * r + c weighs part c of row r, and every lane
// has kDim / 32 of each row's values.
template <int kDim, int kParts>
__device__ __forceinline__ void join_parts(const GqaPrefillLaunch& p, const Item& it, uint32_t o, uint32_t stat,
                                           int rank, int warp, int lane) {
  constexpr int kRows = kMaxParts / kParts, kPieces = kDim / 4, kValues = kDim / 32;
  const float ninf = __int_as_float(0xff800000);
  const int my_r = min(lane / kParts, kRows - 1), my_c = lane % kParts;      // (the lanes left over repeat)
  // Row i's place in out and lse, or -1.
  auto place = [&](int i) -> long long {
    const int r = i & (kTile - 1), query = it.row0 + (i / kTile) * p.tile_q + r / p.group;
    if (i >= 2 * kTile || r >= p.tile_q * p.group || query >= it.qlen) return -1;
    return static_cast<long long>(it.q0 + query) * p.heads + it.head * p.group + r % p.group;
  };
  for (int i0 = rank + kParts * kRows * warp; i0 < 2 * kTile; i0 += kParts * kRows * kSoftWarps) {
    float v[kRows][kParts][kValues];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int i = min(i0 + kParts * r, 2 * kTile - 1);
#pragma unroll
      for (int c = 0; c < kParts; ++c) {
        const uint32_t row = o + i * kDim * 4;
        if constexpr (kDim == 128) {
          const float4 w = ld_shared_cluster_f4(mapa_shared(row + ((lane ^ (i & 31)) << 4), c));
          v[r][c][0] = w.x;
          v[r][c][1] = w.y;
          v[r][c][2] = w.z;
          v[r][c][3] = w.w;
        } else {
          const float2 w = ld_shared_cluster_f2(mapa_shared(row + (((lane >> 1) ^ (i & (kPieces - 1))) << 4) + 8 * (lane & 1), c));
          v[r][c][0] = w.x;
          v[r][c][1] = w.y;
        }
      }
    }
    const int mine = i0 + kParts * my_r;
    const float2 st = ld_shared_cluster_f2(mapa_shared(stat + min(mine, 2 * kTile - 1) * 8, my_c));
    float top = ninf, tot = 0.f;
#pragma unroll
    for (int c = 0; c < kParts; ++c)
      top = fmaxf(top, __shfl_sync(0xffffffffu, st.x, kParts * my_r + c));
    const float w = ex2(st.x - (top > ninf ? top : 0.f));
#pragma unroll
    for (int c = 0; c < kParts; ++c) tot += __shfl_sync(0xffffffffu, w * st.y, kParts * my_r + c);
    const bool any = tot > 0.f || tot != tot;
    const float scale = any ? w / tot : 0.f;
    if (p.lse && my_c == 0 && lane < kParts * kRows && place(mine) >= 0)
      p.lse[place(mine)] = any ? (top + log2f(tot)) * kLn2 : ninf;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float a[kValues];
#pragma unroll
      for (int e = 0; e < kValues; ++e) a[e] = 0.f;
#pragma unroll
      for (int c = 0; c < kParts; ++c) {
        const float f = __shfl_sync(0xffffffffu, scale, kParts * r + c);
#pragma unroll
        for (int e = 0; e < kValues; ++e) a[e] = fmaf(f, v[r][c][e], a[e]);
      }
      const long long at = place(i0 + kParts * r);
      if (at < 0) continue;
      if constexpr (kDim == 128)
        reinterpret_cast<uint2*>(p.out + at * kDim)[lane] = make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
      else
        reinterpret_cast<uint32_t*>(p.out + at * kDim)[lane] = pack_bf16x2(a[0], a[1]);
    }
  }
}

template <int kDim>
__global__ void __launch_bounds__(kThreads, 1)
    gqa_prefill_kernel(const __grid_constant__ CUtensorMap tmap_q,
                       const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, const GqaPrefillLaunch p) {
  using T = Geo<kDim>;
  constexpr int kStages = T::kStages, kKeys = T::kKeys;
  extern __shared__ uint8_t smem_raw[];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const float ninf = __int_as_float(0xff800000);

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + T::kOffSlot);
  volatile int* falling = reinterpret_cast<int*>(smem + T::kOffFalling);
  const uint32_t bar0 = sbase + T::kOffBar;
// K / V of key tile j, counted over the CTA's items: landed, and read.
#define K_FULL(j) (bar0 + 8u * ((j) % kStages))
#define V_FULL(j) (bar0 + 32u + 8u * ((j) % kStages))
#define K_EMPTY(j) (bar0 + 64u + 8u * ((j) % kStages))
#define V_EMPTY(j) (bar0 + 96u + 8u * ((j) % kStages))
#define STAGE_PARITY(j) (((j) / kStages) & 1)
#define PARITY(j) (((j) >> 1) & 1)
// Of query tile q: q landed / read by its last Q K^T; of its c-th key tile: scores,
// probabilities, P V done (kBufs 2: one may come before the last has been waited for).
#define Q_FULL(q) (bar0 + 128u + 8u * (q))
#define Q_EMPTY(q) (bar0 + 144u + 8u * (q))
#define S_FULL(q, c) (bar0 + 160u + 16u * (q) + 8u * ((c) % T::kBufs))
#define PV_DONE(q, c) (bar0 + 256u + 16u * (q) + 8u * ((c) % T::kBufs))
#define P_FULL(q, c) (bar0 + 192u + 16u * (q) + 8u * ((c) % T::kBufs))
#define UNIT_PARITY(c) (((c) / T::kBufs) & 1)
#define DRAIN(q) (bar0 + 288u + 8u * (q))
#define TAKEN (bar0 + 304u)
// Item k's record written / no longer needed by any role.
#define ITEM_FULL(k) (bar0 + 224u + 8u * ((k) & 1))
#define ITEM_EMPTY(k) (bar0 + 240u + 8u * ((k) & 1))
// The query offsets have been looked through.
#define ORDER (sbase + T::kOffOrder)

  if (warp == 8 && lane == 0) {
    for (int st = 0; st < kStages; ++st) {
      mbar_init(K_FULL(st), 1);
      mbar_init(V_FULL(st), 1);
      mbar_init(K_EMPTY(st), 2);      // an MMA warp of each query tile
      mbar_init(V_EMPTY(st), 2);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(Q_FULL(q), 1);
      mbar_init(Q_EMPTY(q), 1);
      mbar_init(ITEM_FULL(q), 1);
      mbar_init(ITEM_EMPTY(q), kItemReaders);
      for (int c = 0; c < T::kBufs; ++c) {
        mbar_init(S_FULL(q, c), 1);
        mbar_init(P_FULL(q, c), kTile);
        mbar_init(PV_DONE(q, c), 1);
      }
    }
    mbar_init(DRAIN(0), 1);
    mbar_init(DRAIN(1), 1);
    mbar_init(TAKEN, 1);
    mbar_init(ORDER, 1);
    *falling = 0;
    fence_mbar_init();
    prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  const Item* items = reinterpret_cast<const Item*>(smem + T::kOffItem);      // 48 bytes apart
  auto record = [&](int k) -> const Item& {
    return *reinterpret_cast<const Item*>(reinterpret_cast<const uint8_t*>(items) + 48 * (k & 1));
  };

  if (warp >= 8) {
    setmaxnreg_dec<kOtherRegs>();
    if (warp == 8) {
      // ------------------------------------------------------------- copies
      if (lane == 0) {
        bool ok = true;
        int uses0 = 0, uses1 = 0;                           // items that had each query tile
        const uint32_t q_bytes = T::kAtoms * p.tile_q * p.group * 128;
        Item it = item_of<kKeys>(p, static_cast<int>(blockIdx.x) / p.parts);
        if (p.parts > 1) keep_part<kKeys>(it, static_cast<int>(blockIdx.x) % p.parts, p.parts);
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
            const int t = base + j, row = it.k0 + j * kKeys;
            const uint32_t dst = sbase + T::kOffRing + (t % kStages) * 2 * T::kKeyOperand;
            if (t >= kStages && !(ok = mbar_wait(K_EMPTY(t), STAGE_PARITY(t - kStages)))) break;
            mbar_expect_tx(K_FULL(t), T::kKeyOperand);
            tma_load_4d(dst, &tmap_k, 0, row, 0, it.head, K_FULL(t));
            if (j == 0) {
              for (int g = 0; ok && g < 2; ++g) {
                if ((g == 0 ? it.nt0 : it.nt1) == 0) continue;
                const int used = g == 0 ? uses0++ : uses1++;
                if (used > 0 && !(ok = mbar_wait(Q_EMPTY(g), (used - 1) & 1))) break;
                mbar_expect_tx(Q_FULL(g), q_bytes);
                for (int a = 0; a < T::kAtoms; ++a)
                  tma_load_5d(sbase + T::kOffQ + g * T::kOperand + a * kAtomBytes, &tmap_q, 0, 0,
                              it.q0 + it.row0 + g * p.tile_q, a, it.head, Q_FULL(g));
              }
              if (!ok) break;
            }
            if (t >= kStages && !(ok = mbar_wait(V_EMPTY(t), STAGE_PARITY(t - kStages)))) break;
            mbar_expect_tx(V_FULL(t), T::kKeyOperand);
            tma_load_4d(dst + T::kKeyOperand, &tmap_v, 0, row, 0, it.head, V_FULL(t));
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
          take_cta(sbase + T::kOffTaken, TAKEN);
          if (!(ok = mbar_wait(TAKEN, asked++ & 1))) break;
          uint32_t x, y, z;
          more = taken_cta(sbase + T::kOffTaken, x, y, z);
          fence_proxy_async_smem();      // read before the next answer is written there
          if (more) it = item_of<kKeys>(p, x);
        }
        if (!ok) raise_error(kErrTimeout);
        // No copy is in flight when the CTA ends.  (After a wait that ran out, the
        // copies before it have had that long to land.)
        if (ok)
          for (int j = max(0, base - kStages); j < base; ++j) {
            mbar_wait(K_FULL(j), STAGE_PARITY(j));
            mbar_wait(V_FULL(j), STAGE_PARITY(j));
          }
        if (ok && uses0 > 0) mbar_wait(Q_FULL(0), (uses0 - 1) & 1);
        if (ok && uses1 > 0) mbar_wait(Q_FULL(1), (uses1 - 1) & 1);
      }
      __syncwarp();
    } else if (warp < 11) {
      // --------------------------------------------------------------- MMAs
      // A warp a query tile, each on its own: it answers its tile's probabilities at
      // once, whatever the other is at.
      const int q = warp - 9;
      const uint32_t el = elect_one() ? 1u : 0u;
      constexpr uint32_t idesc_qk = make_idesc(1, 1, 0, 0, kKeys, kTile);
      constexpr uint32_t idesc_pv = make_idesc(1, 1, 0, 1, kDim, kTile);
      const uint64_t dq = smem_desc_sw128(sbase + T::kOffQ + q * T::kOperand, 16, 1024);
      const uint64_t dk0 = smem_desc_sw128(sbase + T::kOffRing, 16, 1024);
      const uint64_t dv0 = smem_desc_sw128(sbase + T::kOffRing + T::kKeyOperand, T::kKeyAtom, 1024);      // MN-major
      const uint32_t ts0 = tmem + kColS + T::kBufs * kKeys * q, to = tmem + T::kColO + kDim * q;
      bool ok = true;
      // A phase is tested before the last MMAs of the step before go out, so that
      // the test's latency hides behind them; `want` waits only if it was not
      // complete then.
      bool done = false;
      auto want = [&](uint32_t bar, uint32_t parity) {
        if (ok && !done) ok = warp_wait(bar, parity);
        done = false;
      };
      // Descriptor offset of tile t's stage, broadcast: the compiler then knows it to
      // be the same in every lane and keeps it in uniform registers.
      auto stage_of = [&](int t) -> uint64_t {
        return static_cast<uint32_t>(__shfl_sync(0xffffffffu, ((t % kStages) * 2 * T::kKeyOperand) >> 4, 0));
      };
      auto commit = [&](uint32_t bar) {
        if (el) tc_commit(bar);
        __syncwarp();
      };
      // Column of the scores of this query tile's c-th key tile.
      auto col_s = [&](int c) -> uint32_t {
        if (T::kBufs == 1) return ts0;
        return ts0 + static_cast<uint32_t>(__shfl_sync(0xffffffffu, (c % T::kBufs) * kKeys, 0));
      };
      // Q K^T over tile t, this query tile's c-th (the item's last: q is free then).
      auto qk = [&](int t, int c, bool last) {
        const uint64_t dk = dk0 + stage_of(t);
        const uint32_t ts = col_s(c);
        want(K_FULL(t), STAGE_PARITY(t));
        tc_fence_after();
        if (!ok) return;
#pragma unroll
        for (int a = 0; a < T::kAtoms; ++a)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16_ss_uni(ts, dq + static_cast<uint64_t>((a * kAtomBytes + 32 * k) >> 4),
                           dk + static_cast<uint64_t>((a * T::kKeyAtom + 32 * k) >> 4), idesc_qk, (a > 0 || k > 0) ? 1u : 0u, el);
        commit(S_FULL(q, c));
        commit(K_EMPTY(t));
        if (last) commit(Q_EMPTY(q));
      };
      int t = 0, c = 0, uses = 0;      // key tiles so far: all, and of this query tile; items that had it
      for (int item = 0; ok; ++item) {
        if (!(ok = warp_wait(ITEM_FULL(item), PARITY(item)))) break;
        const int work = __shfl_sync(0xffffffffu, record(item).work, 0);
        const int nt0 = __shfl_sync(0xffffffffu, record(item).nt0, 0);
        const int nt1 = __shfl_sync(0xffffffffu, record(item).nt1, 0), ntmax = max(nt0, nt1), nt = q == 0 ? nt0 : nt1;
        if (lane == 0) mbar_arrive(ITEM_EMPTY(item));
        if (!work) break;
        if (nt > 0) {
          ok = warp_wait(Q_FULL(q), uses++ & 1);
          if (T::kBufs == 2) qk(t, c, nt == 1);
        }
        for (int j = 0; ok && j < nt; ++j, ++t, ++c) {
          // (kBufs 2: P V of the tile before has gone out, so the buffer that its scores
          // were in can be written.)
          if (T::kBufs == 1) qk(t, c, j == nt - 1);
          else if (j + 1 < nt) qk(t + 1, c + 1, j + 1 == nt - 1);
          const uint64_t dv = dv0 + stage_of(t);
          const uint32_t ts = col_s(c);
          ok = ok && warp_wait(V_FULL(t), STAGE_PARITY(t)) && warp_wait(P_FULL(q, c), UNIT_PARITY(c));
          tc_fence_after();
          if (!ok) break;
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k) {
            if (k == kKeys / 32) done = warp_test(K_FULL(t + T::kBufs), STAGE_PARITY(t + T::kBufs));
            mma_f16_ts_uni(to, ts + 8 * k, dv + static_cast<uint64_t>((2048 * k) >> 4), idesc_pv, (j > 0 || k > 0) ? 1u : 0u, el);
          }
          if (T::kBufs == 2 || j == nt - 1) commit(PV_DONE(q, T::kBufs == 2 ? c : 0));
          commit(V_EMPTY(t));
        }
        // Tiles that the other query tile alone reads.  (Each in its time: a phase of
        // their barriers takes both warps' arrivals.)
        if (T::kBufs == 2) done = false;
        for (int j = nt; ok && j < ntmax; ++j, ++t) {
          want(K_FULL(t), STAGE_PARITY(t));
          if (lane == 0) mbar_arrive(K_EMPTY(t));
          ok = ok && warp_wait(V_FULL(t), STAGE_PARITY(t));
          if (lane == 0) mbar_arrive(V_EMPTY(t));
        }
      }
      if (!ok && el) raise_error(kErrTimeout);
      if (el) tc_commit(DRAIN(q));      // every MMA is done before TMEM is freed
      __syncwarp();
      mbar_wait(DRAIN(q), 0);
    } else {
      // ------------------------------------------------ order of the offsets
      const bool falls = __any_sync(0xffffffffu, falling_offsets(p, lane, 32));
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
    const uint32_t lanes = tmem + (static_cast<uint32_t>(w4 * 32) << 16);
    const uint32_t tO = lanes + T::kColO + kDim * q;
    const float sc = p.sm_scale * kLog2e;
    // This thread's row: head my_head of the group, of the tile's query my_query.
    const int row_t = w4 * 32 + lane, my_query = row_t / p.group, my_head = row_t - my_query * p.group;
    const bool used = my_query < p.tile_q;
    bool ok = true;
    int c = 0, outs = 0;       // key tiles so far, items that had some
    int n = 0;                 // key tiles of the item
    float mrun = ninf, lrun = 0.f;
    // (Ahead of the items: the offsets have been looked through before the first
    // scores come, but for tens of thousands of requests: 23 us of 1765 for 65535.
    // Asked for in the first item's epilogue, 1 % of every item, 31 to 50 ns.)
    const bool known = warp_wait(ORDER, 0), refused = !known || *falling;
    ok = known;
    for (int item = 0; ok; ++item) {
      if (!(ok = warp_wait(ITEM_FULL(item), PARITY(item)))) break;
      const int query = q * p.tile_q + my_query;      // from the item's first
      int lim, vlive;
      {
        const Item& it = record(item);
        if (!it.work) break;
        n = q == 0 ? it.nt0 : it.nt1;
        // (A row behind the tile's last query sees what that one does: were it to see
        // nothing, its warp would mask every tile, 571 us instead of 495 for four chunks of
        // 500 over 16001 keys in groups of five heads.)
        const int seer = it.row0 + q * p.tile_q + min(my_query, p.tile_q - 1);
        lim = min(it.klen, key_limit(seer, it.qlen, it.klen, p.causal));
        // Keys of the request behind the tile's start, where this query tile is
        // the first to read the tile's V.
        vlive = it.klen;
      }
      mrun = ninf;
      lrun = 0.f;
      for (int j = 0; j < n; ++j, ++c, lim -= kKeys, vlive -= kKeys) {
        const uint32_t tS = lanes + kColS + kKeys * (T::kBufs * q + c % T::kBufs);
        if (ok && !mbar_wait(S_FULL(q, c), UNIT_PARITY(c))) ok = false;
        tc_fence_after();
        uint32_t s[kKeys];
        if constexpr (kKeys == 128) tmem_ld128(tS, s);
        else tmem_ld96(tS, s);
        const int seen = lim;
        float mx[4] = {ninf, ninf, ninf, ninf};
        if (__any_sync(0xffffffffu, seen < kKeys)) {
#pragma unroll
          for (int e = 0; e < kKeys; ++e)
            if (e >= seen) s[e] = __float_as_uint(ninf);
        }
#pragma unroll
        for (int e = 0; e < kKeys; e += 2)
          mx[(e >> 1) & 3] = max3(mx[(e >> 1) & 3], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
        const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
        const bool raise = tmax > mrun + kRaiseLog2;
        const bool rescale = raise && mrun > ninf && used;
        if (__any_sync(0xffffffffu, rescale)) {
          // (kBufs 1: P V of the tile before is done: it was issued before this Q K^T.)
          if (T::kBufs == 2) {
            if (ok && !mbar_wait(PV_DONE(q, c - 1), UNIT_PARITY(c - 1))) ok = false;
            tc_fence_after();
          }
          const float f = rescale ? ex2(mrun - tmax) : 1.f;
#pragma unroll 1
          for (int d = 0; d < kDim; d += 32) {
            uint32_t o[32];
            tmem_ld32(tO + d, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(tO + d, o);
          }
          lrun *= f;
        }
        if (raise) mrun = tmax;
        const float mref = mrun > ninf ? mrun : 0.f;
        // Rows of V behind the request's end are cleared, by both query tiles (either's
        // P V may come first).
        if (vlive < kKeys) {
          const int t = record(item).base + j;
          if (ok && !mbar_wait(V_FULL(t), STAGE_PARITY(t))) ok = false;
#pragma unroll 1
          for (int a = 0; a < T::kAtoms; ++a) {
            uint4* v = reinterpret_cast<uint4*>(smem + T::kOffRing + ((t % kStages) * 2 + 1) * T::kKeyOperand + a * T::kKeyAtom);
            for (int e = (threadIdx.x & 127) + vlive * 8; e < T::kKeyAtom / 16; e += 128)
              v[e] = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int g = 0; g < kKeys / 32; ++g) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x = fma2(make_float2(__uint_as_float(s[32 * g + 2 * e]),
                                              __uint_as_float(s[32 * g + 2 * e + 1])),
                                  make_float2(sc, sc), make_float2(-mref, -mref));
            const float2 w = make_float2(ex2(x.x), ex2(x.y));
            ls[e & 1] = add2(ls[e & 1], w);
            pk[e] = pack_bf16x2(w.x, w.y);
          }
          tmem_st16_async(tS + 16 * g, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(P_FULL(q, c));
        lrun += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
      }
      if (n > 0) {
        if (ok && !(T::kBufs == 2 ? mbar_wait(PV_DONE(q, c - 1), UNIT_PARITY(c - 1)) : mbar_wait(PV_DONE(q, 0), outs & 1))) ok = false;
        tc_fence_after();
        ++outs;
      }
      const Item& it = record(item);
      if (p.parts == 1 && !refused && it.row0 + q * p.tile_q < it.qlen) {
        const bool live = used && it.row0 + query < it.qlen;
        const bool any = lrun > 0.f || lrun != lrun;
        const float inv = any ? 1.f / lrun : 0.f;
        const long long at = static_cast<long long>(it.q0 + it.row0 + query) * p.heads + it.head * p.group + my_head;
        uint4* dst = reinterpret_cast<uint4*>(p.out + at * kDim);
#pragma unroll 1
        for (int c = 0; c < kDim / 32; ++c) {
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
      float4* o_row = reinterpret_cast<float4*>(smem + T::kOffRing + row * kDim * 4);
      named_bar_sync(1, 2 * kTile);      // both query tiles' MMAs are done: the ring and q are free
#pragma unroll 1
      for (int c = 0; c < kDim / 32; ++c) {
        uint32_t o[32];
        if (n > 0) tmem_ld32(tO + 32 * c, o);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          o_row[(8 * c + e) ^ (row & (kDim / 4 - 1))] =
              n > 0 ? make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                  __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]))
                    : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      reinterpret_cast<float2*>(smem + T::kOffQ)[row] = make_float2(mrun, lrun);
      tc_fence_before();
      __syncwarp();
      cluster_sync();
      const Item it = record(0);
      const int rank = static_cast<int>(cluster_ctarank());
      if (ok && it.work && !refused) {
        const uint32_t o = sbase + T::kOffRing, stat = sbase + T::kOffQ;
        switch (p.parts) {
          case 2: join_parts<kDim, 2>(p, it, o, stat, rank, warp, lane); break;
          case 3: join_parts<kDim, 3>(p, it, o, stat, rank, warp, lane); break;
          case 4: join_parts<kDim, 4>(p, it, o, stat, rank, warp, lane); break;
          case 5: join_parts<kDim, 5>(p, it, o, stat, rank, warp, lane); break;
          case 6: join_parts<kDim, 6>(p, it, o, stat, rank, warp, lane); break;
          case 7: join_parts<kDim, 7>(p, it, o, stat, rank, warp, lane); break;
          default: join_parts<kDim, 8>(p, it, o, stat, rank, warp, lane); break;
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
#undef STAGE_PARITY
#undef Q_FULL
#undef S_FULL
#undef P_FULL
#undef PV_DONE
#undef UNIT_PARITY
#undef Q_EMPTY
#undef TAKEN
#undef ITEM_FULL
#undef ITEM_EMPTY
#undef DRAIN
#undef ORDER
}

}  // namespace

namespace {

template <int kDim>
struct Host {
  // Clusters of `parts` CTAs that run at a time on the current device.
  static int clusters_at_once(int parts) {
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
    cfg.dynamicSmemBytes = Geo<kDim>::kSmemBytes;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, gqa_prefill_kernel<kDim>, &cfg) != cudaSuccess || n < 1) {
      (void)cudaGetLastError();
      n = sms / parts;
    }
    known[dev][parts].store(n, std::memory_order_relaxed);
    return n;
  }

  // How the call is launched: its first `whole` items a CTA each, then the rest, `parts`
  // CTAs (a cluster) an item.
  struct Plan {
    long long whole;
    int parts;
  };

  // Costs in key tiles, from the mean lengths (the lengths themselves are on the device):
  // the late items' tiles, 4 for the start and end of an item of one CTA, 5.5 + 0.3 c with
  // the join of c parts; items that come in rounds leave SMs idle in the last one.  So
  // that a last round which leaves many idle may share its keys alone, after whole
  // rounds, for the cost of a second launch: where the call is one request, whose
  // lengths are known.  (Several leave empty blocks in places that the host does not
  // know: four chunks of 504, 48 heads, 530 us with all items a CTA each, 582 shared so.)
  // us:
  //   parts 1 .. 8 of all items (chosen *): a query over 16002 keys, 64 heads on 8, 161
  //   91 65 51 44 38 34 32*; 64 queries, 24 heads, 208 114 83 66 58 50 47 43*; 1000
  //   queries over 5000, 32 heads, 62* 77 92; 4 chunks of 512 over 16001 more, 40 heads,
  //   547 487*;
  //   all items alike, or the last round's keys shared: 1300 queries over 16001 more, 64
  //   heads on 8, 507 and 470; 4572 over 7211 more, 20 heads on 4, 325 and 296; 2642 over
  //   24501 more, 16 heads of 64 dims on one, 322 and 280.
  static Plan choose_plan(const GqaPrefillLaunch& a) {
    const double queries = static_cast<double>(a.total_q) / a.batch;
    const double blocks = std::max(1.0, std::ceil(queries / (2 * a.tile_q)));      // of a request
    const double items = blocks * a.batch * a.kv_heads;
    const double keys = static_cast<double>(a.total_k) / a.batch / Geo<kDim>::kKeys;    // key tiles of a late item ...
    Plan best = {0, 1};
    if (keys <= 4) return best;                                              // two parts cost 8 at least
    const double spread =                                                    // ... and how many fewer an early one has
        a.causal ? std::min(keys, queries * (blocks - 1) / blocks / Geo<kDim>::kKeys) : 0;
    const double sms = clusters_at_once(1), mean1 = keys - spread / 2 + 4;
    const double whole = std::floor(items / sms) * sms, rest = items - whole;
    double best_cost = 0;
    for (int c = 1; c <= kMaxParts; ++c) {
      const double extra = c == 1 ? 4 : 5.5 + 0.3 * c, n = clusters_at_once(c);
      const double most = std::ceil(keys / c) + extra;
      const double mean = (keys - spread / 2) / c + extra, least = (keys - spread) / c + extra;
      const double cost = std::max(most, (items * mean + (std::ceil(items / n) * n - items) * least) / n);
      if (c == 1 || cost < 0.97 * best_cost) {
        best = {0, c};
        best_cost = cost;
      }
      if (c == 1 || a.batch > 1 || whole == 0 || rest == 0) continue;
      const double after = whole * mean1 / sms + std::ceil(rest / n) * mean + 8;
      if (after < 0.97 * best_cost) {
        best = {static_cast<long long>(whole), c};
        best_cost = after;
      }
    }
    return best;
  }

  static cudaError_t launch(GqaPrefillLaunch a, long long items, cudaStream_t s) {
    using T = Geo<kDim>;
    const uint64_t H = a.heads, K = a.kv_heads, G = a.group, Tq = a.total_q, Tk = a.total_k > 0 ? a.total_k : 1;
    // Queries as (64-dim piece, head of the group, query, atom, key head), so that a
    // box brings one atom of a tile's rows; keys as (piece, row, atom, head).
    const uint64_t qdims[5] = {64, G, Tq, T::kAtoms, K};
    const uint64_t qstr[4] = {kDim * 2, static_cast<uint64_t>(a.ld_q) * 2, 128, G * kDim * 2};
    const uint32_t qbox[5] = {64, static_cast<uint32_t>(G), static_cast<uint32_t>(a.tile_q), 1, 1};
    // (Without a key q stands in for k and v, whose strides say nothing then.)
    const uint64_t ld_k = a.total_k > 0 ? a.ld_k : H * kDim, ld_v = a.total_k > 0 ? a.ld_v : H * kDim;
    const uint64_t kdims[4] = {64, Tk, T::kAtoms, K}, kstr[3] = {ld_k * 2, 128, kDim * 2}, vstr[3] = {ld_v * 2, 128, kDim * 2};
    const uint32_t kbox[4] = {64, T::kKeys, T::kAtoms, 1};
    CUtensorMap tq, tk, tv;
    if (!encode_tmap_nd(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, 5, qdims, qstr, qbox, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_nd(&tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.k, 4, kdims, kstr, kbox, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_nd(&tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.v, 4, kdims, vstr, kbox, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(gqa_prefill_kernel<kDim>, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmemBytes);
    if (e != cudaSuccess) return e;
    const Plan plan = choose_plan(a);
    if ((items - plan.whole) * plan.parts > INT_MAX) return cudaErrorInvalidValue;      // (parts are 1 where there are many items)
    auto run = [&](long long first, long long count, int parts) {
      a.first_item = static_cast<int>(first);
      a.parts = parts;
      return launch_kernel(gqa_prefill_kernel<kDim>, dim3(static_cast<unsigned>(count * parts)), dim3(kThreads), T::kSmemBytes, s,
                           false, parts, tq, tk, tv, a);
    };
    if (plan.whole > 0 && (e = run(0, plan.whole, 1)) != cudaSuccess) return e;
    return run(plan.whole, items - plan.whole, plan.parts);
  }
};

// Key heads whose items run together.  Late items are long and early ones short, so
// the order late to early over all heads ends with short ones and the SMs end close
// together; but heads that run together share L2, and each item reads a head's keys
// from its first.  So as many as have 48 MB of keys and values, in groups of equal
// size.  (16384 queries, 64 heads on 32, causal: 2.61 ms; all heads together 2.84, one
// at a time 2.63.  32768, 64 heads on 8: 9.94, 10.35, 10.20.)
int heads_at_once(const GqaPrefillLaunch& a) {
  const double bytes = 48 << 20, head = static_cast<double>(a.total_k) / a.batch * 2 * a.dim * 2;
  const int groups = static_cast<int>(std::ceil(a.kv_heads / std::max(1.0, std::min<double>(a.kv_heads, bytes / (head + 1)))));
  return (a.kv_heads + groups - 1) / groups;
}

int tile_queries(const GqaPrefillLaunch& a) { return kTile / (a.heads / a.kv_heads); }

long long slots_of(const GqaPrefillLaunch& a) {
  const long long block = 2 * tile_queries(a);
  return (a.total_q + (block - 1) * a.batch) / block;
}

}  // namespace

long long gqa_prefill_items(const GqaPrefillLaunch& a) { return slots_of(a) * a.kv_heads; }

cudaError_t launch_gqa_prefill(GqaPrefillLaunch a, cudaStream_t s) {
  a.group = a.heads / a.kv_heads;
  a.tile_q = tile_queries(a);
  // Outputs of a thread's row are stored 32 bytes (a whole sector) at a time
  // where they are aligned so.
  a.out_wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
  a.slots = static_cast<int>(slots_of(a));
  a.head_group = heads_at_once(a);
  const long long items = gqa_prefill_items(a);
  return a.dim == 128 ? Host<128>::launch(a, items, s) : Host<64>::launch(a, items, s);
}

}  // namespace dsa
