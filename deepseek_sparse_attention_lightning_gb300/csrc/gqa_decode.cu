// gqa_decode.cu -- attention of a decode step's queries over the paged cache of a
// layer with grouped heads (the textbook form): G query heads share a key / value
// head of 64 or 128 dims, a request has n_q queries.
//
//   x[row, s] = sm_scale * q[row] . k[s]      (s < vis[row])
//   out[row]  = sum_s softmax(x)[s] * v[s],   lse = log sum_s exp(x)
//
// Bound by HBM: every key and value is read once, for n_q * G rows that share it.  64
// heads on 8, bf16: 8 requests of 131072 tokens 602 us (7.1 TB/s; the measured copy
// rate is 6.8), 8 of 32768 160 us (6.7 TB/s).  FP8, 8 of 32768: 98 us (5.7 TB/s: a
// tile's way through the softmax, some 1500 cycles, is as long as its copy).  A short
// context is bound by latency: 1 request of 4096, 32 heads, 10.9 us, of which the bytes
// take 2.4.
//
// The rows of a request and key head are one row tile (M = 128; more queries than
// fit: several), its keys tiles of two pages (128 tokens).  With few rows the MMAs
// have room to spare (1024 cycles a tile of 64 KB, which takes ~2800 to read), and
// the softmax's latency would bound the kernel instead: a thread that walks a row's
// 128 scores.  So up to 32 rows stand four times in the tile, once in each 32 lanes
// of tensor memory, up to 64 twice: every copy has the same scores, and its threads
// take a quarter (half) of the tile's keys, with a maximum, a sum and an output of
// their own, joined where the stretch ends.  (P of the other keys is zero; it is
// stored once, a copy's own columns each tile.)
//
// Tensor memory: two buffers of S (128 columns), two of P (bf16, 64), O (D).
// Shared memory: q, and a ring of granules, K and V of the key tiles in turn, that
// the copies run ahead in (a page of a head is one contiguous block).
//
// Work: the key tiles of all requests and heads (and what it costs to begin one)
// form one line that is cut evenly over the CTAs, one an SM.  An item (request, key
// head, row tile) that spans CTAs is joined by gqa_merge_kernel from fp32 partials
// and their log-sum-exps.
//
// Roles (256 threads): warp 0 copies, warp 1 MMAs (Q K^T of tile j + 1 runs while
// tile j is in the softmax), warps 4-7 softmax and epilogue, warp 3 the outputs of
// requests without tokens.  The running maximum is raised lazily (only when a tile
// exceeds it by 2^8 does the output get rescaled).  P is rounded to bf16 for the
// matrix pipe (as values are); its sum is kept unrounded in fp32.
//
// Rows of V that no query sees (behind the request's end in its last page, a page
// that is not there or whose id is out of range) are cleared in shared memory
// before P V: their probabilities are zero, but what lies there may be NaN.
//
// Up to 16 rows (kNarrow; most decode steps) lie in the first 16 lanes of a copy and
// are read as 16 lanes x 8 columns, two rows a thread (up to 8 FP8 rows: one), so that
// all lanes of the warp work on them (FP8, 32 ragged requests of 16384 .. 65536, with
// codes made fp16: 629 us by a row a thread, 534 so).
//
// FP8 rows (kFp8; 128 dims): a key or value is its E4M3 code times its row's scale,
// half the bytes, so half the time for the rest.  Nothing is converted for Q K^T: it
// runs on E4M3, the query in two parts, q / 2^e = hi + lo, each E4M3 (a bf16 value
// has 8 bits, a code 4: the sum is exact for values down to 2^-9 of the row's largest,
// and off by 2^-17 of that below).  The key's scale goes to the score.  The value's
// scale goes into the probability through its exponent: with z = x + log2(scale), P =
// 2^(z - m) under a running maximum of z, so that no scale takes P above fp16's range; the
// sum takes P / scale.
//
//   Up to 16 rows (kParts): P V on codes too.  P, rounded to fp16, is four E5M2 parts
//   (its upper byte, the upper byte of what is left, ...), which lose what lies below
//   2^-29 of the largest; the running maximum is raised from 2^2 on, to keep it there.
//   The query's two parts, and P's, stand sixteen lanes apart in a copy: half the MMAs
//   of two products, and the scores are added where they are read, the outputs with
//   those of the copies.  A thread holds pairs of keys 8 apart, so the copies bring V's
//   rows in the order 0 1 8 9 2 3 10 11 ... and the pairs make bytes of one column.
//   768 cycles of MMAs a tile, 32 KB.  (421 us for the requests above, 2.77 GB: 6.6
//   TB/s.)
//
//   More rows: the query's parts side by side, into the same scores; V's codes become
//   fp16 (exactly) in eight warps of their own, which the conversions bound.
//
//   (P in E4M3 parts would drop keys below 2^-17 of the largest, which a long context
//   can have many of.)
//
//   So what P loses is relative to the largest weight times scale, whatever the codes of
//   that row: a weight times scale 2^-24 of it still has 5 bits, and what lies below 2^-29
//   (more rows: 2^-31) adds to the sum alone.  Rows of a request may differ so much where
//   they bring little; but a row of zeros brings nothing, and dsa_kv_write_fp8 gives it
//   scale 1, far above a row's of small values.  So such rows (scale 1, all codes zero) are
//   looked for and count with kLeastScale: their P is as small as it gets, and their weight
//   is in the sum all the same.  (The search for scales of 1 costs 0 to 1 %: 32 ragged
//   requests 434 -> 436 us in calls of three states; where every row's scale is 1, each
//   tile's codes are looked at, 446.)
#include <cuda_fp8.h>

#include <algorithm>

#include "dsa_ptx.cuh"
#include "dsa_internal.h"

DSA_DEFINE_ERROR_WORD(gqa_decode)

namespace dsa {
namespace {

constexpr int kRows = 128;                     // of a row tile (M)
constexpr int kKeys = 2 * kPage;               // of a key tile
constexpr int kAtomBytes = kRows * 128;        // 128 rows x 64 dims
constexpr int kPageAtom = kPage * 128;         // 64 rows x 64 dims
constexpr int kThreads = 256, kThreadsFp8 = 512, kThreadsParts = 384, kSoftThreads = 128;
constexpr int kDequantWarps = 8, kParamWarps = 4;      // FP8; the latter of the former
// FP8, registers a thread (launched with 128 each): copies and MMAs, softmax, two
// warpgroups of dequantisation.
constexpr int kRegsMma = 88, kRegsSoft = 216, kRegsDequant = 104;
static_assert(kRegsMma + kRegsSoft + 2 * kRegsDequant <= 4 * 128, "registers");
// What an item's queries and output cost, in key tiles: bf16, FP8 (whose tiles take half
// the time).  128 requests of 100 .. 900 bf16 tokens: 60.0 us for 1, 58.7 for 2, 59.7 for
// 3; 64 of 1000 .. 6000 FP8 tokens: 100.8 for 1, 97.3 for 2, 90.6 for 4, 91.7 for 6.
constexpr int kStretchBf16 = 2, kStretchFp8 = 4;
constexpr int kColS = 0, kColP = 256, kColO = 384, kTmemCols = 512;
constexpr int kStage = kSoftThreads * 32 * 4;  // 32 columns of a copy's rows, fp32
constexpr float kRaiseLog2 = 8.0f, kRaiseParts = 2.0f, kShiftFp8 = 7.0f, kShiftParts = 13.0f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// Smaller value scales count as this one (a row of values below 2^-71, to which dsa_kv_write_fp8
// may give a subnormal scale): P / scale is 2^95 at most, and 2^31 of them stay in fp32's range.
constexpr float kLeastScale = 0x1p-80f;

// kParts: FP8 rows whose P V runs on codes, P in parts; kDequant: whose codes become
// fp16 first.
template <int kDim, bool kNarrow, bool kFp8>
struct Geo {
  static constexpr bool kParts = kFp8 && kNarrow, kDequant = kFp8 && !kNarrow;
  static constexpr int kAtoms = kDim / 64;
  static constexpr int kOperand = kAtoms * kAtomBytes;      // q, or K or V of a tile for the MMAs (16-bit)
  static constexpr int kQBytes = kParts ? kAtomBytes : kOperand;       // (FP8: both parts, one below the other or side by side)
  static constexpr int kGranule = kFp8 ? kKeys * kDim : kOperand;      // K or V of a tile as it is cached
  static constexpr int kPageBytes = kGranule / 2;
  static constexpr int kRing = kParts ? 10 : kFp8 ? 6 : kDim == 128 ? 5 : 8;      // granules
  static constexpr int kStages = kDequant ? 1 : 2;                     // staging buffers of the epilogue
  static constexpr int kOffQ = 0;
  static constexpr int kOffRing = kQBytes;
  static constexpr int kOffV16 = kOffRing + kRing * kGranule;          // kDequant: two tiles of V in fp16
  static constexpr int kOffStage = kOffV16 + (kDequant ? 2 * kOperand : 0);
  static constexpr int kOffXchg = kOffStage + kStages * kStage;        // (maximum, sum) of 128 threads
  static constexpr int kOffScale = kOffXchg + kSoftThreads * 8;        // FP8, a tile in the ring: 128 key scales, 128 value scales
  static constexpr int kOffParam = kOffScale + (kFp8 ? kRing / 2 * 2 * kKeys * 4 : 0);      // two tiles: kk, lg, 1 / scale
  static constexpr int kOffQScale = kOffParam + (kFp8 ? 2 * 3 * kKeys * 4 : 0);             // four stretches: 2^e of a row
  static constexpr int kOffBar = kOffQScale + (kFp8 ? 4 * kRows * 4 : 0);
  static constexpr int kOffInfo = kOffBar + 40 * 8;      // (34 barriers)
  static constexpr int kSmemBytes = kOffInfo + 48 + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory");
  static_assert(!kFp8 || (kDim == 128 && kRing % 2 == 0), "FP8");
};

// mbar_wait by a whole warp: the same answer in every lane.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// Tokens of request r: seqlens[r], at least 0 and at most what its row of the page
// table covers (more is an error the kernel reports).
__device__ __forceinline__ int request_len(const GqaDecodeLaunch& p, int r) {
  const int s = __ldg(p.seqlens + r);
  if (s > p.max_pages * kPage) {
    raise_error(kErrCheck);
    return p.max_pages * kPage;
  }
  return s < 0 ? 0 : s;
}

__device__ __forceinline__ int tiles_of(int len) { return (len + kKeys - 1) / kKeys; }
template <int kStretch>
__device__ __forceinline__ int units_of(int len) {
  return len > 0 ? tiles_of(len) + kStretch : 0;
}

// The line: for each item with tokens kStretch units and one a key tile, the items
// of a request one after another.  It is cut into parts from unit kStretch on, so
// that the first item's tiles alone count; a cut among an item's kStretch units
// falls before its first tile.
struct Line {
  long long total;
  int parts;
};

template <int kStretch>
__device__ __forceinline__ long long cut(const Line& ln, int g) {
  return kStretch + (ln.total - kStretch) * g / ln.parts;
}

// (one warp) The line of all requests.
template <int kStretch>
__device__ __forceinline__ Line scan_total(const GqaDecodeLaunch& p, int lane) {
  const int items = p.kv_heads * p.row_tiles;      // of a request
  long long n = 0;
  for (int r = lane; r < p.batch; r += 32) n += units_of<kStretch>(request_len(p, r));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  Line ln;
  ln.total = n * items;
  const long long most = (ln.total - kStretch + p.min_tiles - 1) / p.min_tiles;
  ln.parts = most < p.ctas ? static_cast<int>(most < 1 ? 1 : most) : p.ctas;
  return ln;
}

// (one warp) The item that holds unit `at` of the line (at < total): its request,
// which of the request's it is, and the line position of its first unit.
template <int kStretch>
__device__ __forceinline__ void locate(const GqaDecodeLaunch& p, long long at, int lane, int& req, int& item,
                                       long long& first) {
  const int items = p.kv_heads * p.row_tiles;
  long long base = 0;
  req = item = 0;
  first = 0;
  for (int r0 = 0; r0 < p.batch; r0 += 32) {
    const int r = r0 + lane;
    const long long n = r < p.batch ? static_cast<long long>(units_of<kStretch>(request_len(p, r))) * items : 0;
    long long incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, base + incl > at);
    if (hit) {
      const int l = __ffs(hit) - 1;
      req = r0 + l;
      const long long begin = base + __shfl_sync(0xffffffffu, incl - n, l);
      const int each = static_cast<int>(__shfl_sync(0xffffffffu, n, l) / items);
      item = static_cast<int>((at - begin) / each);
      first = begin + static_cast<long long>(item) * each;
      return;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// The stretches of items in a CTA's part [pos, hi) of the line, in order.
template <int kStretch>
struct Walk {
  long long pos, hi;     // next unit of the line, end of the part
  int req, item;         // of the stretch
  int unit;              // unit of the item at pos
  int len, nt;           // the request's tokens and key tiles
  int t0, t1;            // the stretch's tiles
  __device__ __forceinline__ bool next(const GqaDecodeLaunch& p) {
    while (pos < hi) {
      if (unit == nt + kStretch || nt == 0) {     // on to the next item
        ++item;
        unit = 0;
        if (nt == 0 || item == p.kv_heads * p.row_tiles) {
          item = 0;
          do {      // (the line has units left: a request with tokens comes)
            ++req;
            len = request_len(p, req);
            nt = tiles_of(len);
          } while (nt == 0);
        }
      }
      const long long left = hi - pos;
      const int end = static_cast<int>(left < nt + kStretch - unit ? unit + left : nt + kStretch);
      t0 = max(0, unit - kStretch);
      t1 = max(0, end - kStretch);
      pos += end - unit;
      unit = end;
      if (t1 > t0) return true;
    }
    return false;
  }
};

// Page ids of a stretch's tiles, 32 at a time (an id a lane) and one batch ahead:
// kNone behind the request's last page, kBad for an id outside the cache.
struct PageBatch {
  static constexpr int kNone = -1, kBad = -2, kTiles = 16;      // tiles of a batch
  const int32_t* table;
  int pages, num_pages, t0, now, ahead;
  __device__ __forceinline__ int get(int i) const {
    if (i >= pages) return kNone;
    const int id = __ldg(table + i);
    return id >= 0 && id < num_pages ? id : kBad;
  }
  template <int kStretch>
  __device__ __forceinline__ PageBatch(const GqaDecodeLaunch& p, const Walk<kStretch>& wk, int lane)
      : table(p.page_table + static_cast<long long>(wk.req) * p.max_pages), pages((wk.len + kPage - 1) / kPage),
        num_pages(p.num_pages), t0(wk.t0), now(0) {
    ahead = get(2 * t0 + lane);
  }
  // Before tile t's pages are asked for, t going up by one.
  __device__ __forceinline__ bool advance(int t, int lane) {
    if (((t - t0) & (kTiles - 1)) != 0) return false;
    now = ahead;
    ahead = get(2 * (t + kTiles) + lane);
    return true;
  }
  // Page h of tile t.
  __device__ __forceinline__ int page(int t, int h) const {
    return __shfl_sync(0xffffffffu, now, 2 * ((t - t0) & (kTiles - 1)) + h);
  }
};

template <int kN>
__device__ __forceinline__ void tmem_ld_cols(uint32_t addr, uint32_t (&r)[kN]) {
  if constexpr (kN == 32) tmem_ld32(addr, r);
  else if constexpr (kN == 64) tmem_ld64(addr, r);
  else tmem_ld128(addr, r);
}

// kNarrow: 8 or 16, where the tile has so many rows at most (a thread has one or two), else 0.
template <int kDim, int kCopies, int kNarrow, bool kFp8>
__global__ void __launch_bounds__(!kFp8 ? kThreads : kNarrow ? kThreadsParts : kThreadsFp8, 1)
    gqa_decode_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v, const GqaDecodeLaunch p) {
  using T = Geo<kDim, (kNarrow > 0), kFp8>;
  constexpr bool kParts = T::kParts, kDequant = T::kDequant;
  constexpr int kCols = kKeys / kCopies;         // keys of a softmax thread
  constexpr int kStretch = kFp8 ? kStretchFp8 : kStretchBf16;
  constexpr int kCopyRows = kRows / kCopies;     // lanes of a copy
  constexpr int kSets = kParts ? 2 * kCopies : kCopies, kSetRows = kRows / kSets;      // outputs to be added up
  constexpr int kMine = kNarrow / 8;             // rows of a softmax thread (kNarrow)
  static_assert(!kNarrow || kCopies == 4, "a warp a copy");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const float ninf = __int_as_float(0xff800000);
  const uint32_t bar0 = sbase + T::kOffBar;
// Granule n (K of tile i: 2 i, V: 2 i + 1): landed, and read.
#define FULL(n) (bar0 + 8u * ((n) % T::kRing))
#define EMPTY(n) (bar0 + 80u + 8u * ((n) % T::kRing))
#define RING_PARITY(n) (((n) / T::kRing) & 1)
// q of a stretch landed / read; O read by the epilogue; of tile i: scores, probabilities, P V done.
#define Q_FULL (bar0 + 160u)
#define Q_EMPTY (bar0 + 168u)
#define O_FREE (bar0 + 176u)
#define DRAIN (bar0 + 184u)
#define S_FULL(i) (bar0 + 192u + 8u * ((i) & 1))
#define P_FULL(i) (bar0 + 208u + 8u * ((i) & 1))
#define PV_DONE(i) (bar0 + 224u + 8u * ((i) & 1))
#define PARITY2(i) (((i) >> 1) & 1)
// (FP8) Of tile i: scales ready for the softmax, V in fp16.
#define PARAM_FULL(i) (bar0 + 240u + 8u * ((i) & 1))
#define V16_FULL(i) (bar0 + 256u + 8u * ((i) & 1))
  long long* info = reinterpret_cast<long long*>(smem + T::kOffInfo);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + T::kOffInfo + 40);

  if (warp == 0 && lane == 0) {
    for (int n = 0; n < T::kRing; ++n) {
      mbar_init(FULL(n), 1);
      mbar_init(EMPTY(n), (n & 1) ? (kDequant ? kDequantWarps : 1) : (kFp8 ? 1 + kParamWarps : 1));
    }
    mbar_init(Q_FULL, kParts ? kParamWarps : kFp8 ? kDequantWarps : 1);
    mbar_init(Q_EMPTY, 1);
    mbar_init(O_FREE, kSoftThreads / 32);
    mbar_init(DRAIN, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(S_FULL(i), 1);
      mbar_init(P_FULL(i), kSoftThreads / 32);
      mbar_init(PV_DONE(i), 1);
      if (kFp8) {
        mbar_init(PARAM_FULL(i), kParamWarps);
        mbar_init(V16_FULL(i), kDequantWarps);
      }
    }
    fence_mbar_init();
    if (!kFp8) prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  if (warp == 3) {
    const Line ln = scan_total<kStretch>(p, lane);
    const int part = blockIdx.x;
    long long lo = 0, hi = 0, first = 0;
    int req = 0, item = 0;
    if (part < ln.parts && ln.total > 0) {
      lo = cut<kStretch>(ln, part);
      hi = cut<kStretch>(ln, part + 1);
      if (hi > lo) locate<kStretch>(p, lo, lane, req, item, first);
    }
    // What the merge has to join: the item that this part's first cut falls into, if
    // it is the first cut inside that item, and its last part.
    if (lane == 0) {
      int4 join = make_int4(-1, 0, 0, 0);
      const long long tile0 = first + kStretch;
      if (part > 0 && hi > lo && lo > tile0 && cut<kStretch>(ln, part - 1) <= tile0) {
        const long long end = tile0 + tiles_of(request_len(p, req)) - kStretch;      // the item's, from unit kStretch
        join = make_int4(req, item, static_cast<int>((end * ln.parts - 1) / (ln.total - kStretch)), 0);
      }
      p.joins[part] = join;
      info[0] = lo;
      info[1] = hi;
      info[2] = first;
      info[3] = static_cast<long long>(item) << 32 | req;
    }
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  Walk<kStretch> wk;
  wk.pos = info[0];
  wk.hi = info[1];
  wk.req = static_cast<int>(info[3] & 0xffffffff);
  wk.item = static_cast<int>(info[3] >> 32);
  wk.len = request_len(p, wk.req);
  wk.nt = tiles_of(wk.len);
  wk.unit = static_cast<int>(wk.pos - info[2]);
  wk.t0 = wk.t1 = 0;

  if (warp < 4) {
  if constexpr (kDequant) setmaxnreg_dec<kRegsMma>();
  if (warp == 0) {
    // ------------------------------------------------------------- copies
    bool ok = true;
    int it = 0, seg = 0;
    const uint32_t q_bytes = kCopies * T::kAtoms * p.tile_rows * 128;
    for (; ok && wk.next(p); ++seg) {
      PageBatch pages(p, wk, lane);
      const int head = wk.item / p.row_tiles, mtile = wk.item % p.row_tiles;
      for (int t = wk.t0; ok && t < wk.t1; ++t, ++it) {
        if (pages.advance(t, lane) && pages.now == PageBatch::kBad) raise_error(kErrCheck);
        const int page[2] = {pages.page(t, 0), pages.page(t, 1)};
        const uint32_t present = (page[0] >= 0) + (page[1] >= 0);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int n = 2 * it + g;
          if (n >= T::kRing && ok && !mbar_wait(EMPTY(n), RING_PARITY(n - T::kRing))) ok = false;
          if (ok && lane == 0) {
            // (FP8: the scales of keys and values come with the keys.)
            mbar_expect_tx(FULL(n), present * (T::kPageBytes + (kFp8 && g == 0 ? 2 * kPage * 4 : 0)));
            const uint32_t dst = sbase + T::kOffRing + (n % T::kRing) * T::kGranule;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (page[h] < 0) continue;
              if constexpr (kFp8) {
                const long long at = (static_cast<long long>(page[h]) * p.kv_heads + head) * kPage;      // its first row
                if (kParts && g == 1)
                  tma_load_5d(dst + h * T::kPageBytes, &tmap_v, 0, 0, 0, 0, static_cast<int>(at / 16), FULL(n));
                else
                  tma_load_4d(dst + h * T::kPageBytes, g == 0 ? &tmap_k : &tmap_v, 0, 0, head, page[h], FULL(n));
                if (g == 0) {
                  const uint32_t to = sbase + T::kOffScale + (it % (T::kRing / 2)) * 2 * kKeys * 4 + h * kPage * 4;
                  bulk_load(to, p.k_scale + at, kPage * 4, FULL(n));
                  bulk_load(to + kKeys * 4, p.v_scale + at, kPage * 4, FULL(n));
                }
              } else {
#pragma unroll
                for (int a = 0; a < T::kAtoms; ++a)
                  tma_load_5d(dst + a * kAtomBytes + h * kPageAtom, g == 0 ? &tmap_k : &tmap_v, 0, 0, a, head, page[h],
                              FULL(n));
              }
            }
          }
          if (!kFp8 && g == 0 && t == wk.t0) {
            if (seg > 0 && ok && !mbar_wait(Q_EMPTY, (seg - 1) & 1)) ok = false;
            if (ok && lane == 0) {
              mbar_expect_tx(Q_FULL, q_bytes);
              for (int c = 0; c < kCopies; ++c)
                for (int a = 0; a < T::kAtoms; ++a)
                  tma_load_5d(sbase + T::kOffQ + a * kAtomBytes + c * kCopyRows * 128, &tmap_q, 0, 0,
                              wk.req * p.nq + mtile * p.tile_q, a, head, Q_FULL);
            }
          }
          ok = __all_sync(0xffffffffu, ok);
        }
      }
    }
    if (!ok && lane == 0) raise_error(kErrTimeout);
  } else if (warp == 1) {
    // --------------------------------------------------------------- MMAs
    // The whole warp runs this; one lane issues.
    const uint32_t el = elect_one() ? 1u : 0u;
    constexpr uint32_t kFmt = kFp8 ? 0 : 1;      // E4M3 and fp16, or bf16
    constexpr uint32_t idesc_qk = make_idesc(kFmt, kFmt, 0, 0, kKeys, kRows);
    constexpr uint32_t idesc_pv = make_idesc(kParts ? 1 : kFmt, kFmt, 0, 1, kDim, kRows);      // (kParts: E5M2 and E4M3)
    const uint64_t dq = smem_desc_sw128(sbase + T::kOffQ, 16, 1024);
    const uint64_t dk0 = smem_desc_sw128(sbase + T::kOffRing, 16, 1024);
    const uint64_t dv0 = smem_desc_sw128(sbase + (kDequant ? T::kOffV16 : T::kOffRing), kAtomBytes, 1024);      // MN-major
    auto slot_of = [&](int slot, int bytes) -> uint64_t {
      return static_cast<uint32_t>(__shfl_sync(0xffffffffu, (slot * bytes) >> 4, 0));
    };
    bool ok = true;
    int it = 0, npv = 0;
    // P V of tile npv (its stretch's first: the output starts at zero, once the
    // epilogue has read the stretch before).
    int pv_seg = 0, pv_left = 0;
    Walk<kStretch> pvw = wk;
    auto issue_pv = [&]() -> bool {
      bool fresh = false;
      if (pv_left == 0) {
        pvw.next(p);
        pv_left = pvw.t1 - pvw.t0;
        fresh = true;
        if (pv_seg > 0 && !warp_wait(O_FREE, (pv_seg - 1) & 1)) return false;
        ++pv_seg;
      }
      const int n = 2 * npv + 1;
      if (!(kDequant ? warp_wait(V16_FULL(npv), PARITY2(npv)) : warp_wait(FULL(n), RING_PARITY(n))) ||
          !warp_wait(P_FULL(npv), PARITY2(npv)))
        return false;
      tc_fence_after();
      const uint64_t dv = dv0 + slot_of(kDequant ? npv & 1 : n % T::kRing, kDequant ? T::kOperand : T::kGranule);
      const uint32_t tp = tmem + kColP + 64 * (npv & 1);
#pragma unroll
      for (int k = 0; k < kKeys / 16; ++k)
        if constexpr (kParts)      // (the first and second parts' 32 keys at a time, then the others')
          mma_f8_ts_uni(tmem + kColO, tp + 8 * k, dv + static_cast<uint64_t>((4096 * (k & 3)) >> 4), idesc_pv,
                        (!fresh || k > 0) ? 1u : 0u, el);
        else
          mma_f16_ts_uni(tmem + kColO, tp + 8 * k, dv + static_cast<uint64_t>((2048 * k) >> 4), idesc_pv,
                         (!fresh || k > 0) ? 1u : 0u, el);
      if (el) {
        if (!kDequant) tc_commit(EMPTY(n));
        tc_commit(PV_DONE(npv));
      }
      __syncwarp();
      --pv_left;
      ++npv;
      return true;
    };
    for (int seg = 0; ok && wk.next(p); ++seg) {
      if (!(ok = warp_wait(Q_FULL, seg & 1))) break;
      for (int t = wk.t0; t < wk.t1; ++t, ++it) {
        // (Scores of tile it - 2 were read: its P V was issued, after its P_FULL.)
        const int n = 2 * it;
        if (!(ok = warp_wait(FULL(n), RING_PARITY(n)))) break;
        tc_fence_after();
        const uint64_t dk = dk0 + slot_of(n % T::kRing, T::kGranule);
        const uint32_t ts = tmem + kColS + kKeys * (it & 1);
#pragma unroll
        for (int a = 0; a < (kParts ? 1 : T::kAtoms); ++a)      // (FP8: the query's parts, over the same keys)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if constexpr (kFp8)
              mma_f8_ss_uni(ts, dq + static_cast<uint64_t>((a * kAtomBytes + 32 * k) >> 4),
                            dk + static_cast<uint64_t>((32 * k) >> 4), idesc_qk, (a > 0 || k > 0) ? 1u : 0u, el);
            else
              mma_f16_ss_uni(ts, dq + static_cast<uint64_t>((a * kAtomBytes + 32 * k) >> 4),
                           dk + static_cast<uint64_t>((a * kAtomBytes + 32 * k) >> 4), idesc_qk, (a > 0 || k > 0) ? 1u : 0u, el);
        if (el) {
          tc_commit(EMPTY(n));
          tc_commit(S_FULL(it));
          if (t == wk.t1 - 1) tc_commit(Q_EMPTY);
        }
        __syncwarp();
        if (it > 0 && !(ok = issue_pv())) break;
      }
    }
    if (ok && it > 0) ok = issue_pv();
    if (!ok && el) raise_error(kErrTimeout);
    if (el) tc_commit(DRAIN);      // every MMA is done before TMEM is freed
    __syncwarp();
    mbar_wait(DRAIN, 0);
    __syncwarp();
  } else if (warp == 3) {
    // Requests without tokens (no part of the line is theirs).
    const int rows = p.nq * p.heads;
    for (int r = blockIdx.x; r < p.batch; r += gridDim.x) {
      if (request_len(p, r) > 0) continue;
      const long long row0 = static_cast<long long>(r) * rows;
      uint4* dst = reinterpret_cast<uint4*>(p.out + row0 * kDim);
      for (int e = lane; e < rows * (kDim / 8); e += 32) dst[e] = make_uint4(0u, 0u, 0u, 0u);
      if (p.lse)
        for (int e = lane; e < rows; e += 32) p.lse[row0 + e] = ninf;
    }
  }
  } else if (kFp8 && warp >= 8) {
    // ------------------------------- queries, scales and values of FP8 rows
    // A warp converts four rows of V at a time: eight neighbouring lanes hold four
    // 16-code chunks of each of two rows, of different halves (reads) and with
    // different swizzles (writes): both fall on distinct banks.
    if constexpr (kFp8) {
    if constexpr (kDequant) setmaxnreg_dec<kRegsDequant>();
    constexpr int kRowsAtOnce = kParts ? 16 : 32;
    const int w = warp - 8, tid = threadIdx.x - 256;
    const int r2 = (lane >> 2) & 1, c = (lane & 3) + 4 * (((lane >> 3) & 1) ^ r2);
    const int row4 = 2 * (lane >> 4) + r2;
    const int group = p.heads / p.kv_heads;
    bool ok = true;
    int it = 0, seg = 0;
    for (; ok && wk.next(p); ++seg) {
      PageBatch pages(p, wk, lane);
      {
        // The query's parts, eight lanes a row (16 values each).
        const int head = wk.item / p.row_tiles, mtile = wk.item % p.row_tiles, piece = tid & 7;
        if (seg > 0 && !mbar_wait(Q_EMPTY, (seg - 1) & 1)) ok = false;
        for (int row0 = 0; row0 < p.tile_rows; row0 += kRowsAtOnce) {
          const int row = row0 + (tid >> 3), i = row / group;
          const int qi = mtile * p.tile_q + i;
          const bool in = row < p.tile_rows && qi < p.nq;
          uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
          if (in) {
            const uint4* src = reinterpret_cast<const uint4*>(
                p.q + ((static_cast<long long>(wk.req) * p.nq + qi) * p.heads + head * group + (row - i * group)) * kDim) + 2 * piece;
            a = __ldg(src);
            b = __ldg(src + 1);
          }
          const uint32_t word[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
          float2 x[8];
          float amax = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] = make_float2(bf16lo_to_f32(word[e]), bf16hi_to_f32(word[e]));
            amax = max3(amax, fabsf(x[e].x), fabsf(x[e].y));
          }
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          // 2^e, so that the largest value lies in [128, 256).
          const int ex = max(static_cast<int>(__float_as_uint(amax) >> 23) - 134, -100);
          const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 v = mul2(x[e], make_float2(down, down));
            const uint32_t h = __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
            const float2 back = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(h), __NV_E4M3)));
            const uint32_t l = __nv_cvt_float2_to_fp8x2(make_float2(v.x - back.x, v.y - back.y), __NV_SATFINITE, __NV_E4M3);
            hi[e >> 1] = (e & 1) ? hi[e >> 1] | h << 16 : h;
            lo[e >> 1] = (e & 1) ? lo[e >> 1] | l << 16 : l;
          }
          if (row < p.tile_rows) {
#pragma unroll
            for (int cp = 0; cp < kCopies; ++cp) {
              const int at = cp * kCopyRows + row;
              uint8_t* dst = smem + T::kOffQ + at * 128 + ((piece ^ (at & 7)) << 4);
              *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              // (kParts: sixteen rows below; a multiple of 8, so swizzled alike.)
              *reinterpret_cast<uint4*>(dst + (kParts ? 16 * 128 : kAtomBytes)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            if (piece == 0)
              reinterpret_cast<float*>(smem + T::kOffQScale)[(seg & 3) * kRows + row] =
                  __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(Q_FULL);
      }
      uint32_t good = 0;
      for (int t = wk.t0; ok && t < wk.t1; ++t, ++it) {
        if (pages.advance(t, lane)) good = __ballot_sync(0xffffffffu, pages.now >= 0);
        const uint32_t ok2 = good >> (2 * ((t - wk.t0) & (PageBatch::kTiles - 1)));
        const int vlive = wk.len - t * kKeys;
        // Scales and V of tile it - 2 have been read.
        if (it >= 2 && !mbar_wait(PV_DONE(it), PARITY2(it - 2))) ok = false;
        if (w < kParamWarps) {
          const int n = 2 * it;
          if (ok && !mbar_wait(FULL(n), RING_PARITY(n))) ok = false;
          const float* scales = reinterpret_cast<const float*>(smem + T::kOffScale) + (it % (T::kRing / 2)) * 2 * kKeys;
          float* par = reinterpret_cast<float*>(smem + T::kOffParam) + (it & 1) * 3 * kKeys;
          const bool seen = tid < vlive && ((ok2 >> (tid / kPage)) & 1u);
          float vs = seen ? fmaxf(scales[kKeys + tid], kLeastScale) : 1.f;
          // A row of zeros, whose scale is 1, counts with the least scale.  (Only where there
          // is such a scale are V's codes waited for.)
          if (__any_sync(0xffffffffu, seen && vs == 1.f)) {
            if (ok && !mbar_wait(FULL(n + 1), RING_PARITY(n + 1))) ok = false;
            const int at = kParts ? (tid & ~15) | ((tid & 8) >> 2) | ((tid & 6) << 1) | (tid & 1) : tid;      // where its codes lie
            const uint4* codes = reinterpret_cast<const uint4*>(smem + T::kOffRing + ((n + 1) % T::kRing) * T::kGranule + at * kDim);
            uint32_t any = 0u;
#pragma unroll
            for (int e = 0; e < kDim / 16; ++e) {      // (neighbouring lanes on different banks)
              const uint4 w4 = codes[(e + lane) % (kDim / 16)];
              any |= w4.x | w4.y | w4.z | w4.w;
            }
            if (seen && vs == 1.f && (any & 0x7f7f7f7fu) == 0u) vs = kLeastScale;
          }
          par[tid] = seen ? scales[tid] : 0.f;
          par[kKeys + tid] = log2f(vs);
          par[2 * kKeys + tid] = 1.f / vs;
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(PARAM_FULL(it));
            mbar_arrive(EMPTY(n));
          }
        }
        if constexpr (kDequant) {
        const int n = 2 * it + 1;
        if (ok && !mbar_wait(FULL(n), RING_PARITY(n))) ok = false;
        const uint8_t* src = smem + T::kOffRing + (n % T::kRing) * T::kGranule + c * 16;
        uint4 raw[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int row = 32 * u + 4 * w + row4;
          raw[u] = *reinterpret_cast<const uint4*>(src + row * 128);
          // Rows that no query sees are zero, whatever the cache holds.
          if (row >= vlive || !((ok2 >> (u >> 1)) & 1u)) raw[u] = make_uint4(0u, 0u, 0u, 0u);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(EMPTY(n));
        uint8_t* dst = smem + T::kOffV16 + (it & 1) * T::kOperand + (c >> 2) * kAtomBytes;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int row = 32 * u + 4 * w + row4, piece = (2 * (c & 3)) ^ (row & 7);
          const uint32_t code[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const __half2_raw f = __nv_cvt_fp8x2_to_halfraw2(
                static_cast<__nv_fp8x2_storage_t>((code[e >> 1] >> (16 * (e & 1))) & 0xFFFFu), __NV_E4M3);
            h[e] = static_cast<uint32_t>(f.x) | static_cast<uint32_t>(f.y) << 16;
          }
          *reinterpret_cast<uint4*>(dst + row * 128 + (piece << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(dst + row * 128 + ((piece ^ 1) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(V16_FULL(it));
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (!ok && lane == 0) raise_error(kErrTimeout);
    }
  } else {
    // ---------------------------------------------- softmax and epilogue
    if constexpr (kDequant) setmaxnreg_inc<kRegsSoft>();
    constexpr float kRaise = kParts ? kRaiseParts : kRaiseLog2, kShift = kParts ? kShiftParts : kFp8 ? kShiftFp8 : 0.f;
    const int tid = threadIdx.x - 128;             // = TMEM lane
    const int w4 = warp & 3;
    const int copy = tid / kCopyRows, set = tid / kSetRows, row = tid % kSetRows;      // row of the tile
    const uint32_t lanebase = static_cast<uint32_t>(w4 * 32) << 16;
    const int group = p.heads / p.kv_heads;
    const int my_q = row / group;
    float2* xchg = reinterpret_cast<float2*>(smem + T::kOffXchg);
    const float sc = p.sm_scale * kLog2e;
    if constexpr (kCopies > 1) {
      // P of the other copies' keys: zero, once.
      uint32_t z[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) z[e] = 0u;
      for (int c = 0; c < 4; ++c) tmem_st32(tmem + lanebase + kColP + 32 * c, z);
    }
    bool ok = true;
    int it = 0, stage = 0, seg = 0;
    for (; wk.next(p); ++seg) {
      PageBatch pages(p, wk, lane);
      const int head = wk.item / p.row_tiles, mtile = wk.item % p.row_tiles;
      const int qi = mtile * p.tile_q + my_q;
      const bool live = my_q < p.tile_q && qi < p.nq;
      // (A row behind the last query's sees what that one does, so that its warp does not
      // mask every tile.  Its scores are of what lies in shared memory: they go nowhere.)
      const int vis = wk.len - (p.nq - 1 - min(mtile * p.tile_q + min(my_q, p.tile_q - 1), p.nq - 1));
      float mrun = ninf, lrun = 0.f;      // maximum and sum (this thread's keys) in the exp2 domain
      // (kNarrow) The same of this thread's rows, lane / 4 and that + 8; their visible
      // tokens, and FP8 their factors.
      float mrun2[2] = {ninf, ninf}, lrun2[2] = {0.f, 0.f}, f2[2] = {0.f, 0.f};
      int vis2[2] = {0, 0};
      if constexpr (kNarrow > 0) {
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
          const int r = min((lane >> 2) + 8 * u, p.tile_rows - 1);
          vis2[u] = wk.len - (p.nq - 1 - min(mtile * p.tile_q + r / group, p.nq - 1));
        }
      }
      uint32_t good = 0;                  // validity of the next 32 page ids
      auto narrow_tile = [&](int t, uint32_t ok2) {
        uint32_t s[16];
        const uint32_t ts = tmem + lanebase + kColS + kKeys * (it & 1) + kCols * copy;
        if constexpr (!kParts) {
          tmem_ld16x32(ts, s);
        } else {
          // The scores of the query's lower part, sixteen lanes on.
          uint32_t lo[16];
          tmem_ld16x32_two(ts, ts + (16u << 16), s, lo);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (((e >> 1) & 1) < kMine) s[e] = __float_as_uint(__uint_as_float(s[e]) + __uint_as_float(lo[e]));
        }
        const int col = 2 * (lane & 3);      // of each eight
        const float* par = reinterpret_cast<const float*>(smem + T::kOffParam) + (it & 1) * 3 * kKeys + kCols * copy + col;
        if constexpr (kFp8) {
          // z = x + log2(value scale), x the score in the exp2 domain.
          if (ok && !mbar_wait(PARAM_FULL(it), PARITY2(it))) ok = false;
          if (t == wk.t0) {
            const float* qs = reinterpret_cast<const float*>(smem + T::kOffQScale) + (seg & 3) * kRows;
#pragma unroll
            for (int u = 0; u < kMine; ++u) f2[u] = sc * qs[min((lane >> 2) + 8 * u, p.tile_rows - 1)];
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 kk = *reinterpret_cast<const float2*>(par + 8 * j);
            const float2 lg = *reinterpret_cast<const float2*>(par + kKeys + 8 * j);
#pragma unroll
            for (int u = 0; u < kMine; ++u) {
              const float2 z = fma2(mul2(make_float2(__uint_as_float(s[4 * j + 2 * u]), __uint_as_float(s[4 * j + 2 * u + 1])), kk),
                                    make_float2(f2[u], f2[u]), lg);
              s[4 * j + 2 * u] = __float_as_uint(z.x);
              s[4 * j + 2 * u + 1] = __float_as_uint(z.y);
            }
          }
        }
        float top[2];
        bool above = false;
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
          const int seen = ((ok2 >> (kCols * copy / kPage)) & 1u) ? vis2[u] - t * kKeys - kCols * copy - col : 0;
          if (seen < 26) {      // (columns 8 j and 8 j + 1 from `col` on)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (8 * (e >> 1) + (e & 1) >= seen) s[4 * (e >> 1) + 2 * u + (e & 1)] = __float_as_uint(ninf);
          }
          float m = ninf;
#pragma unroll
          for (int j = 0; j < 4; ++j) m = max3(m, __uint_as_float(s[4 * j + 2 * u]), __uint_as_float(s[4 * j + 2 * u + 1]));
          top[u] = m * (kFp8 ? 1.f : sc);
          above |= top[u] > mrun2[u] + kRaise;
        }
        // (The row's maximum, over four lanes, is asked for only where one of them is
        // above.)
        if (__any_sync(0xffffffffu, above)) {
          float fac[2] = {1.f, 1.f};
          bool rescale = false;
#pragma unroll
          for (int u = 0; u < kMine; ++u) {
            top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], 1));
            top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], 2));
            const bool raise = top[u] > mrun2[u] + kRaise;
            fac[u] = raise && mrun2[u] > ninf ? ex2(mrun2[u] - top[u]) : 1.f;
            rescale |= raise && mrun2[u] > ninf && (lane >> 2) + 8 * u < p.tile_rows;
            if (raise) mrun2[u] = top[u];
            lrun2[u] *= fac[u];
          }
          if (__any_sync(0xffffffffu, rescale)) {
            // P V of the tile before has to be in the output first.
            if (ok && !mbar_wait(PV_DONE(it - 1), PARITY2(it - 1))) ok = false;
            tc_fence_after();
            const float fa = __shfl_sync(0xffffffffu, fac[0], 4 * (lane & 7)), fb = __shfl_sync(0xffffffffu, fac[1], 4 * (lane & 7));
            const float f = !kParts && lane >= 16 ? 1.f : (lane & 15) < 8 ? fa : fb;
#pragma unroll 1
            for (int c = 0; c < kDim / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tmem + lanebase + kColO + 32 * c, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(tmem + lanebase + kColO + 32 * c, o);
            }
          }
        }
        // (P of tile it - 2 has been read: that P V was issued before this Q K^T.)
        uint32_t pk[8] = {};
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
          const float mref = mrun2[u] > ninf ? mrun2[u] - kShift : 0.f;
          float2 ls = make_float2(0.f, 0.f);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 y = make_float2(__uint_as_float(s[4 * j + 2 * u]), __uint_as_float(s[4 * j + 2 * u + 1]));
            const float2 x = kFp8 ? add2(y, make_float2(-mref, -mref)) : fma2(y, make_float2(sc, sc), make_float2(-mref, -mref));
            const float2 w = make_float2(ex2(x.x), ex2(x.y));
            if constexpr (kFp8) {
              ls = fma2(w, *reinterpret_cast<const float2*>(par + 2 * kKeys + 8 * j), ls);
              pk[2 * j + u] = pack_f16x2(w.x, w.y);
            } else {
              ls = add2(ls, w);
              pk[2 * j + u] = pack_bf16x2(w.x, w.y);
            }
          }
          lrun2[u] += ls.x + ls.y;
        }
        const uint32_t tp = tmem + lanebase + kColP + 64 * (it & 1);
        if constexpr (kParts) {
          // E5M2 is the upper byte of fp16: a part is what that holds of what is left
          // (exact, 11 bits in four parts of 3).  Parts 0 and 1 in the lanes of the
          // query's parts, 2 and 3 in those of 32 columns on; a column holds the 4 keys
          // of two of this thread's pairs (V's rows are ordered so).
          uint32_t left[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) left[e] = pk[e];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t part[4];
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
              for (int u = 0; u < 2; ++u) part[2 * g + u] = __byte_perm(left[4 * g + u], left[4 * g + 2 + u], 0x7531);
            tmem_st16x8_async(tp + ((q & 1) ? 16u << 16 : 0u) + 32 * (q >> 1) + 8 * copy, part);
            if (q < 3)
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint32_t top = left[e] & 0xff00ff00u;
                const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&left[e]), *reinterpret_cast<const __half2*>(&top));
                left[e] = *reinterpret_cast<const uint32_t*>(&d);
              }
          }
        } else {
          tmem_st16x16_async(tp + (kCols / 2) * copy, pk);
        }
      };
      for (int t = wk.t0; t < wk.t1; ++t, ++it) {
        if (pages.advance(t, lane)) good = __ballot_sync(0xffffffffu, pages.now >= 0);
        // Bit h: page h of the tile can be read.
        const uint32_t ok2 = good >> (2 * ((t - wk.t0) & (PageBatch::kTiles - 1)));
        if (ok && !mbar_wait(S_FULL(it), PARITY2(it))) ok = false;
        tc_fence_after();
        if constexpr (kNarrow > 0) {
          narrow_tile(t, ok2);
        } else {
        uint32_t s[kCols];
        tmem_ld_cols<kCols>(tmem + lanebase + kColS + kKeys * (it & 1) + kCols * copy, s);
        const float4* par = reinterpret_cast<const float4*>(smem + T::kOffParam) + (it & 1) * 3 * kKeys / 4 + kCols / 4 * copy;
        if constexpr (kFp8) {
          // z = x + log2(value scale), x the score in the exp2 domain.
          if (ok && !mbar_wait(PARAM_FULL(it), PARITY2(it))) ok = false;
          const float f = sc * reinterpret_cast<const float*>(smem + T::kOffQScale)[(seg & 3) * kRows + min(row, p.tile_rows - 1)];
#pragma unroll
          for (int e = 0; e < kCols; e += 4) {
            const float4 kk = par[e / 4], lg = par[kKeys / 4 + e / 4];
            const float2 f2 = make_float2(f, f);
            const float2 a = fma2(mul2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), make_float2(kk.x, kk.y)), f2, make_float2(lg.x, lg.y));
            const float2 b = fma2(mul2(make_float2(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), make_float2(kk.z, kk.w)), f2, make_float2(lg.z, lg.w));
            s[e] = __float_as_uint(a.x);
            s[e + 1] = __float_as_uint(a.y);
            s[e + 2] = __float_as_uint(b.x);
            s[e + 3] = __float_as_uint(b.y);
          }
        }
        // Visible keys among this thread's: of its page, or of the first and second.
        const int base = vis - t * kKeys - kCols * copy;
        const int page0 = kCols * copy / kPage;
        const int seen0 = ((ok2 >> page0) & 1u) ? base : 0;
        const int seen1 = kCopies > 1 ? seen0 : ((ok2 >> 1) & 1u) ? base : 0;
        if (__any_sync(0xffffffffu, min(seen0, seen1) < kCols)) {
#pragma unroll
          for (int e = 0; e < kCols; ++e)
            if (e >= (e < kPage ? seen0 : seen1)) s[e] = __float_as_uint(ninf);
        }
        float mx[4] = {ninf, ninf, ninf, ninf};
#pragma unroll
        for (int e = 0; e < kCols; e += 2)
          mx[(e >> 1) & 3] = max3(mx[(e >> 1) & 3], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
        const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * (kFp8 ? 1.f : sc);
        const bool raise = tmax > mrun + kRaise;
        const bool rescale = raise && mrun > ninf && live;
        if (__any_sync(0xffffffffu, rescale)) {
          // P V of the tile before has to be in the output first.
          if (ok && !mbar_wait(PV_DONE(it - 1), PARITY2(it - 1))) ok = false;
          tc_fence_after();
          const float f = rescale ? ex2(mrun - tmax) : 1.f;
#pragma unroll 1
          for (int c = 0; c < kDim / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tmem + lanebase + kColO + 32 * c, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(tmem + lanebase + kColO + 32 * c, o);
          }
          lrun *= f;
        }
        if (raise) mrun = tmax;
        // (FP8: P up to 2^15, which leaves fp16 40 powers of two below.)
        const float mref = mrun > ninf ? mrun - kShift : 0.f;
        // (P of tile it - 2 has been read: that P V was issued before this Q K^T.)
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const uint32_t tp = tmem + lanebase + kColP + 64 * (it & 1) + (kCols / 2) * copy;
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = make_float2(__uint_as_float(s[32 * c + 2 * e]), __uint_as_float(s[32 * c + 2 * e + 1]));
            const float2 x = kFp8 ? add2(y, make_float2(-mref, -mref)) : fma2(y, make_float2(sc, sc), make_float2(-mref, -mref));
            const float2 w = make_float2(ex2(x.x), ex2(x.y));
            if constexpr (kFp8) {
              const float4 inv = par[2 * kKeys / 4 + 8 * c + e / 2];
              ls[e & 1] = fma2(w, (e & 1) ? make_float2(inv.z, inv.w) : make_float2(inv.x, inv.y), ls[e & 1]);
              pk[e] = pack_f16x2(w.x, w.y);
            } else {
              ls[e & 1] = add2(ls[e & 1], w);
              pk[e] = pack_bf16x2(w.x, w.y);
            }
          }
          tmem_st16_async(tp + 16 * c, pk);
        }
        lrun += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
        }
        // Rows of V behind every query's view are cleared.
        const int vlive = wk.len - t * kKeys;
        if (!kDequant && (vlive < kKeys || (ok2 & 3u) != 3u)) {
          const int n = 2 * it + 1;
          if (ok && !mbar_wait(FULL(n), RING_PARITY(n))) ok = false;
          uint4* v = reinterpret_cast<uint4*>(smem + T::kOffRing + (n % T::kRing) * T::kGranule);
          for (int e = tid; e < T::kGranule / 16; e += kSoftThreads) {
            const int at = (e >> 3) & (kKeys - 1);
            // (kParts: of each sixteen rows 0 1 8 9 2 3 10 11 ...)
            const int key = kParts ? (at & ~15) | ((at & 2) << 2) | ((at >> 1) & 6) | (at & 1) : at;
            if (key >= vlive || !((ok2 >> (key / kPage)) & 1u)) v[e] = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(P_FULL(it));
      }
      if constexpr (kNarrow > 0) {
        // From a thread's rows to a row a lane.
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          lrun2[u] += __shfl_xor_sync(0xffffffffu, lrun2[u], 1);
          lrun2[u] += __shfl_xor_sync(0xffffffffu, lrun2[u], 2);
          const float m = __shfl_sync(0xffffffffu, mrun2[u], 4 * (lane & 7)), l = __shfl_sync(0xffffffffu, lrun2[u], 4 * (lane & 7));
          if (((lane >> 3) & (kParts ? 1 : 3)) == u) {
            mrun = m;
            lrun = kParts && lane >= 16 ? 0.f : l;      // (counted once)
          }
        }
      }
      // ---------------------------------------------------------- epilogue
      if (ok && !mbar_wait(PV_DONE(it - 1), PARITY2(it - 1))) ok = false;
      tc_fence_after();
      const bool whole = wk.t0 == 0 && wk.t1 == wk.nt;
      // Where row r of the tile goes: its row of out, or of the part's slot.
      const long long slot0 = (static_cast<long long>(blockIdx.x) * 2 + (wk.t0 > 0 ? 0 : 1)) * kRows;
      auto place = [&](int r) -> long long {
        if (!whole) return slot0 + r;
        const int i = r / group;
        return (static_cast<long long>(wk.req) * p.nq + mtile * p.tile_q + i) * p.heads + head * group + (r - i * group);
      };
      float top = mrun, l = lrun;
      if constexpr (kSets > 1) {
        xchg[tid] = make_float2(mrun, lrun);
        named_bar_sync(1, kSoftThreads);
        top = ninf;
        l = 0.f;
        float2 other[kSets];
#pragma unroll
        for (int c = 0; c < kSets; ++c) {
          other[c] = xchg[c * kSetRows + row];
          top = fmaxf(top, other[c].x);
        }
        const float mref = top > ninf ? top : 0.f;
#pragma unroll
        for (int c = 0; c < kSets; ++c) l = fmaf(ex2(other[c].x - mref), other[c].y, l);
      }
      const bool any = l > 0.f || l != l;
      const float w = any ? ex2(mrun - (top > ninf ? top : 0.f)) / l : 0.f;
      if (live && set == 0) {
        const float lse = any ? (top - kShift + log2f(l)) * kLn2 : ninf;
        if (!whole) p.part_lse[place(row)] = lse;
        else if (p.lse) p.lse[place(row)] = lse;
      }
      if constexpr (kSets == 1) {
        const long long at = live ? place(row) : 0;
#pragma unroll 1
        for (int c = 0; c < kDim / 32; ++c) {
          uint32_t o[32];
          __syncwarp();
          tmem_ld32(tmem + lanebase + kColO + 32 * c, o);
          if (!live) continue;
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(p.out + at * kDim + 32 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t h[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                h[j] = any ? pack_bf16x2(__uint_as_float(o[8 * e + 2 * j]) * w, __uint_as_float(o[8 * e + 2 * j + 1]) * w) : 0u;
              dst[e] = make_uint4(h[0], h[1], h[2], h[3]);
            }
          } else {
            float4* dst = reinterpret_cast<float4*>(p.part_o + at * kDim + 32 * c);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e] = any ? make_float4(__uint_as_float(o[4 * e]) * w, __uint_as_float(o[4 * e + 1]) * w,
                                         __uint_as_float(o[4 * e + 2]) * w, __uint_as_float(o[4 * e + 3]) * w)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
      } else {
        // The copies' outputs, weighted, are added up through shared memory, 32 dims
        // at a time (16-byte piece i of a row at i ^ (row & 7)): thread = row and
        // kSets' share of the 32.
        constexpr int kPer = 32 / kSets;                  // dims of a thread
        const int orow = tid / kSets, part = tid % kSets;
        const int oq = orow / group;
        const bool olive = oq < p.tile_q && mtile * p.tile_q + oq < p.nq;
        const long long at = olive ? place(orow) : 0;
#pragma unroll 1
        for (int c = 0; c < kDim / 32; ++c, stage = (stage + 1) % T::kStages) {
          uint32_t o[32];
          __syncwarp();
          tmem_ld32(tmem + lanebase + kColO + 32 * c, o);
          if (T::kStages == 1 && c > 0) named_bar_sync(1, kSoftThreads);      // the others have read it
          float* buf = reinterpret_cast<float*>(smem + T::kOffStage + stage * kStage);
          if (live)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<float4*>(buf + tid * 32 + ((e ^ (tid & 7)) << 2)) =
                  w > 0.f || w != w ? make_float4(__uint_as_float(o[4 * e]) * w, __uint_as_float(o[4 * e + 1]) * w,
                                                  __uint_as_float(o[4 * e + 2]) * w, __uint_as_float(o[4 * e + 3]) * w)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
          named_bar_sync(1, kSoftThreads);
          if (!olive) continue;
          float sum[kPer];
#pragma unroll
          for (int e = 0; e < kPer; ++e) sum[e] = 0.f;
#pragma unroll
          for (int cc = 0; cc < kSets; ++cc) {
            const int src = cc * kSetRows + orow;
#pragma unroll
            for (int e = 0; e < kPer / 4; ++e) {
              const float4 v = *reinterpret_cast<const float4*>(buf + src * 32 + (((part * (kPer / 4) + e) ^ (src & 7)) << 2));
              sum[4 * e] += v.x;
              sum[4 * e + 1] += v.y;
              sum[4 * e + 2] += v.z;
              sum[4 * e + 3] += v.w;
            }
          }
          const long long to = at * kDim + 32 * c + kPer * part;
          if (whole && kPer == 4) {
            *reinterpret_cast<uint2*>(p.out + to) = make_uint2(pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3]));
          } else if (whole) {
#pragma unroll
            for (int e = 0; e < kPer / 8; ++e)
              reinterpret_cast<uint4*>(p.out + to)[e] =
                  make_uint4(pack_bf16x2(sum[8 * e], sum[8 * e + 1]), pack_bf16x2(sum[8 * e + 2], sum[8 * e + 3]),
                             pack_bf16x2(sum[8 * e + 4], sum[8 * e + 5]), pack_bf16x2(sum[8 * e + 6], sum[8 * e + 7]));
          } else {
#pragma unroll
            for (int e = 0; e < kPer / 4; ++e)
              reinterpret_cast<float4*>(p.part_o + to)[e] = make_float4(sum[4 * e], sum[4 * e + 1], sum[4 * e + 2], sum[4 * e + 3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(O_FREE);
    }
    if (!ok && lane == 0) raise_error(kErrTimeout);
  }
  __syncthreads();
  grid_dep_launch();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
#undef FULL
#undef EMPTY
#undef RING_PARITY
#undef Q_FULL
#undef Q_EMPTY
#undef O_FREE
#undef DRAIN
#undef S_FULL
#undef P_FULL
#undef PV_DONE
#undef PARITY2
#undef PARAM_FULL
#undef V16_FULL
}

// Joins the partials of an item that spans CTAs.  Block (i, c): some rows of the
// item whose first cut begins part i + 1, if it is one (the attention kernel wrote
// that down).  Its first part is slot 1 of its CTA (a stretch from the item's
// start), the others slot 0 of theirs.  D / 4 threads a row, kShare such groups on
// one row (each takes every kShare-th batch of four parts), joined in shared memory.
// (1 request of 131072 tokens, 16 heads on one: 26.7 us; a group a row, 43.7.  32
// heads on 8, 4096 tokens: 10.8 and 12.8.  128 requests of 3000 on average: alike.)
constexpr int kMergeThreads = 256, kBatch = 4, kShare = 4;

template <int kDim>
__global__ void __launch_bounds__(kMergeThreads) gqa_merge_kernel(const GqaDecodeLaunch p) {
  constexpr int kTpr = kDim / 4, kGroups = kMergeThreads / kTpr, kRowsBlock = kGroups / kShare;
  __shared__ float4 s_acc[kGroups][kTpr];
  __shared__ float2 s_sum[kGroups];
  const int g = threadIdx.x / kTpr, c4 = threadIdx.x % kTpr, share = g % kShare;
  const int row = blockIdx.y * kRowsBlock + g / kShare;
  const int g0 = blockIdx.x;
  const float ninf = __int_as_float(0xff800000);
  grid_dep_wait();
  const int4 join = p.joins[g0 + 1];
  if (join.x < 0) return;
  const int head = join.y / p.row_tiles, mtile = join.y % p.row_tiles, group = p.heads / p.kv_heads;
  const int qi = mtile * p.tile_q + row / group;
  const bool live = row < p.tile_rows && qi < p.nq;
  const int n = live ? join.z - g0 + 1 : 0;      // parts
  auto slot = [&](int i) { return (static_cast<long long>(g0 + i) * 2 + (i == 0 ? 1 : 0)) * kRows + row; };
  float mx = ninf, tot = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int b0 = share * kBatch; b0 < n; b0 += kShare * kBatch) {
    float4 v[kBatch];
    float e[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const bool in = b0 + u < n;
      const long long s = slot(in ? b0 + u : 0);
      e[u] = in ? p.part_lse[s] : ninf;
      v[u] = reinterpret_cast<const float4*>(p.part_o + s * kDim)[c4];
    }
    float top = mx;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) top = fmaxf(top, e[u]);
    const float mref = top > ninf ? top : 0.f;
    const float f = ex2((mx - mref) * kLog2e);      // (0 for the first batch: its sums are 0)
    mx = top;
    tot *= f;
    acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const float w = ex2((e[u] - mref) * kLog2e);
      // (An empty part holds zeros; its weight is 0.)
      tot += w;
      acc = make_float4(fmaf(w, v[u].x, acc.x), fmaf(w, v[u].y, acc.y), fmaf(w, v[u].z, acc.z), fmaf(w, v[u].w, acc.w));
    }
  }
  s_acc[g][c4] = acc;
  if (c4 == 0) s_sum[g] = make_float2(mx, tot);
  __syncthreads();
  if (share > 0 || !live) return;
#pragma unroll
  for (int u = 1; u < kShare; ++u) mx = fmaxf(mx, s_sum[g + u].x);
  const float mref = mx > ninf ? mx : 0.f;
  tot = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int u = 0; u < kShare; ++u) {
    const float2 st = s_sum[g + u];
    const float w = ex2((st.x - mref) * kLog2e);
    const float4 v = s_acc[g + u][c4];
    tot = fmaf(w, st.y, tot);
    acc = make_float4(fmaf(w, v.x, acc.x), fmaf(w, v.y, acc.y), fmaf(w, v.z, acc.z), fmaf(w, v.w, acc.w));
  }
  const bool any = tot > 0.f || tot != tot;
  const float inv = any ? 1.f / tot : 0.f;
  const long long at = (static_cast<long long>(join.x) * p.nq + qi) * p.heads + head * group + row % group;
  reinterpret_cast<uint2*>(p.out + at * kDim)[c4] = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv),
                                                               pack_bf16x2(acc.z * inv, acc.w * inv));
  if (p.lse && c4 == 0) p.lse[at] = any ? mx + log2f(tot) * kLn2 : ninf;
}

// Keys of a CTA's part of the line, at least: less is not worth a CTA (1 request of 4000
// tokens, 32 heads on 8: 128 11.4 us, 256 10.9, 512 13.1).
constexpr int kMinKeys = 256;

// Queries of a row tile: as many as fit, the tiles of a request alike.
int row_tiles_of(int nq, int group) {
  const int fit = kRows / group;      // (group <= heads <= 128)
  return (nq + fit - 1) / fit;
}

template <int kDim, int kCopies, int kNarrow, bool kFp8>
cudaError_t launch(const GqaDecodeLaunch& a, cudaStream_t s) {
  using T = Geo<kDim, (kNarrow > 0), kFp8>;
  const uint64_t G = a.heads / a.kv_heads, K = a.kv_heads, tokens = static_cast<uint64_t>(a.batch) * a.nq;
  const uint64_t pages = static_cast<uint64_t>(a.num_pages);
  CUtensorMap tq, tk, tv;
  if (kFp8) {
    // Codes as (byte, row of the page, head, page); kParts: values as (byte, r % 2, r / 8
    // % 2, r / 2 % 4, r / 16) of their rows r, in that order.
    const uint64_t dims[4] = {kDim, kPage, K, pages}, str[3] = {kDim, kPage * kDim, K * kPage * kDim};
    const uint32_t box[4] = {kDim, kPage, 1, 1};
    const uint64_t vdims[5] = {kDim, 2, 2, 4, 4 * K * pages}, vstr[4] = {kDim, 8 * kDim, 2 * kDim, 16 * kDim};
    const uint32_t vbox[5] = {kDim, 2, 2, 4, 4};
    if (!encode_tmap_nd(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.k, 4, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !(T::kParts ? encode_tmap_nd(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.v, 5, vdims, vstr, vbox, CU_TENSOR_MAP_SWIZZLE_128B)
                    : encode_tmap_nd(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.v, 4, dims, str, box, CU_TENSOR_MAP_SWIZZLE_NONE)))
      return cudaErrorInvalidValue;
    tq = tk;      // not used
  } else {
    // Queries as (64-dim piece, head of the group, query, atom, key head): a box brings
    // one atom of a tile's rows.  Caches as (piece, row of the page, atom, head, page).
    const uint64_t qdims[5] = {64, G, tokens, T::kAtoms, K};
    const uint64_t qstr[4] = {kDim * 2, static_cast<uint64_t>(a.heads) * kDim * 2, 128, G * kDim * 2};
    const uint32_t qbox[5] = {64, static_cast<uint32_t>(G), static_cast<uint32_t>(a.tile_q), 1, 1};
    const uint64_t cdims[5] = {64, kPage, T::kAtoms, K, pages};
    const uint64_t cstr[4] = {kDim * 2, 128, kPage * kDim * 2, K * kPage * kDim * 2};
    const uint32_t cbox[5] = {64, kPage, 1, 1, 1};
    if (!encode_tmap_nd(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, 5, qdims, qstr, qbox, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_nd(&tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.k, 5, cdims, cstr, cbox, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_nd(&tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.v, 5, cdims, cstr, cbox, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  auto kern = gqa_decode_kernel<kDim, kCopies, kNarrow, kFp8>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmemBytes);
  if (e != cudaSuccess) return e;
  e = launch_kernel(kern, dim3(a.ctas), dim3(!kFp8 ? kThreads : kNarrow ? kThreadsParts : kThreadsFp8), T::kSmemBytes, s, false, 1,
                    tq, tk, tv, a);
  if (e != cudaSuccess || a.ctas == 1) return e;
  constexpr int kPer = kMergeThreads / (kDim / 4) / kShare;      // rows of a block
  return launch_kernel(gqa_merge_kernel<kDim>, dim3(a.ctas - 1, (a.tile_rows + kPer - 1) / kPer), dim3(kMergeThreads), 0, s,
                       true, 1, a);
}

// As many copies of the rows as fit into a tile.
template <int kDim, bool kFp8>
cudaError_t launch_rows(const GqaDecodeLaunch& a, cudaStream_t s) {
  if constexpr (kFp8)      // (bf16: the same time)
    if (a.tile_rows <= 8) return launch<kDim, 4, 8, kFp8>(a, s);
  if (a.tile_rows <= 16) return launch<kDim, 4, 16, kFp8>(a, s);
  if (a.tile_rows <= 32) return launch<kDim, 4, 0, kFp8>(a, s);
  if (a.tile_rows <= 64) return launch<kDim, 2, 0, kFp8>(a, s);
  return launch<kDim, 1, 0, kFp8>(a, s);
}

}  // namespace

// Two stretches of partials a CTA, one CTA an SM.
size_t gqa_decode_workspace(int dim) {
  const size_t ctas = device_sm_count();
  return ctas * (2 * kRows * (dim + 1) * sizeof(float) + sizeof(int4));
}

cudaError_t launch_gqa_decode(GqaDecodeLaunch a, void* ws, cudaStream_t s) {
  const int group = a.heads / a.kv_heads;
  a.row_tiles = row_tiles_of(a.nq, group);
  a.tile_q = (a.nq + a.row_tiles - 1) / a.row_tiles;
  a.tile_rows = a.tile_q * group;
  a.ctas = device_sm_count();
  a.min_tiles = kMinKeys / kKeys;
  a.part_o = static_cast<float*>(ws);
  const size_t slots = static_cast<size_t>(a.ctas) * 2 * kRows;
  a.part_lse = a.part_o + slots * a.dim;
  a.joins = reinterpret_cast<int4*>(a.part_lse + slots);
  if (a.k_scale) return launch_rows<128, true>(a, s);
  return a.dim == 128 ? launch_rows<128, false>(a, s) : launch_rows<64, false>(a, s);
}

}  // namespace dsa
