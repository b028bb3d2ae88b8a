// mla_decode.cu -- latent attention in its absorbed form over every visible
// token of the paged latent cache (no selection), for decode and MTP
// verification ("[SGLang] NSA", section "forward_decode": q_nope absorbed to
// 512 dims + 64 rope dims against 576-dim latent rows whose first 512 dims are
// the values; "MTP and sparse attention: NSA and DSA": the dense MLA the
// sparse layer replaces).
//
//   x[row, s] = sm_scale * q[row] . c[s]      (576 dims, s < vis[row])
//   out[row]  = sum_s softmax(x)[s] * c[s, 0:512],   lse = log sum_s exp(x)
//
// A request's n_q * H query rows are cut into row tiles of 128, its keys into
// tiles of two pages (128 tokens).  The matrix work of a key and a row tile
// (128 x 1088 multiply-adds) against the key's 1152 bytes is close to the GPU's
// ridge, so both pipes matter.
//
// Two CTAs (a cluster on one pair of SMs) share a row tile: tcgen05 with
// cta_group::2 and M = 128, 64 rows in each CTA.  The fp32 output of 64 rows x
// 512 dims takes 256 of a CTA's 512 TMEM columns (64 rows use all 128 lanes:
// lanes 0-63 hold the first half of an MMA's N columns, lanes 64-127 the
// second), which leaves room for double-buffered scores; and each CTA keeps
// only its share of the operands: for Q K^T one of the tile's two pages (64 x
// 576), for P V half of the value dims of both.  A CTA that works alone holds
// half of the output only by computing all of Q K^T twice.
//
// N = 128 for Q K^T: with one page a step (N = 64) an MMA reads 3 KB of shared
// memory for 16 cycles of work and takes 25 (measured); with two it runs at
// its full rate, 32.
//
// Shared memory: q 72 KB (64 rows), K 72 KB in three groups of 3 atoms (64
// dims each), V 64 KB (two pages), P 16 KB.  All of it is single-buffered:
// a K group is free once its MMAs of the tile are done and is needed again a
// P V and two groups' MMAs later, a V page is free after its half of P V, and
// the copies (one tensor copy a K group, two a V page, in the 128B-swizzled
// layout that the MMAs read) have that long.
//
// Work: the key tiles of all requests (and what it costs to begin one) form one
// line that is cut evenly over the CTA pairs (n_q * H > 128: over groups of
// pairs, one pair for each row tile, which walk the same tiles at the same time
// and share them in L2).  A pair may end one request and begin the next; a
// request that spans pairs is joined by mla_merge_kernel from fp32 partials and
// their log-sum-exps.
//
// Roles (256 threads a CTA): warp 0 copies q and K, warp 2 copies V, warp 1
// of the leading CTA issues the MMAs of both, warps 4-7 are softmax and
// epilogue (thread = row and page of the tile; the two threads of a row agree
// on its maximum through shared memory).  Q K^T of tile j + 1 runs while tile
// j is in the softmax.  The running maximum is raised lazily (only when a tile
// exceeds it by 2^8 does the output get rescaled).  P is rounded to bf16 for
// the matrix pipe (as values and keys are); its sum is kept unrounded in fp32,
// so the log-sum-exp has fp32 accuracy.
//
// FP8 latent rows (kFp8; 656 bytes: 512 E4M3 codes, the four 128-dim tiles'
// scales, 64 rope dims in bf16): a tile is one page, which halves K, V and P and
// makes room for three stages of raw codes and scales (25 KB each) that the copy
// engine runs ahead with.  Eight warps dequantise them for K, eight for V: a
// code times its scale in fp32, rounded to bf16, written in the layout that the
// MMAs read.  (Read by the warps themselves, the codes of a two-page tile cost
// more than all else: the load path took 2 of 4.3 us a tile, and 8 ragged
// requests 351 us.)  K's three groups are dims 0-255, 256-511 and rope, which
// is copied as it is.
//
// Rows of V that no query row sees (behind the request's end in its last page,
// or a page whose id is out of range) are cleared in shared memory before P V:
// their probabilities are zero, but stale cache memory may hold NaN.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "dsa_ptx.cuh"
#include "dsa_internal.h"

DSA_DEFINE_ERROR_WORD(mla_dense)

namespace dsa {
namespace {

constexpr int kRowsCta = 64;                              // query rows of a CTA
constexpr int kRowTile = 2 * kRowsCta;
constexpr int kAtoms = kLatentDim / 64;                   // 9 atoms of 64 dims
constexpr int kQBytes = kRowsCta * kLatentDim * 2;        // 72 KB
constexpr int kAtom = 64 * 128;                           // 64 rows x 64 dims of q, V or P: 8 KB
constexpr int kKGroups = 3, kGroupAtoms = kAtoms / kKGroups;
constexpr int kVBytes = 4 * kAtom;                        // one page, this CTA's 256 value dims
static_assert(kRowsCta == 64 && kPage == 64, "atoms of 64 rows");
constexpr int kF8RowBytes = 656, kF8ScaleOff = 512, kF8RopeOff = 528;
constexpr int kRawStages = 3, kRawTile = 32 * 128;        // FP8: codes of 32 rows x 128 dims
constexpr int kRawBytes = 6 * kRawTile + kPage * 16;      // own rows, the other rows' own dims, scales

// A key tile and the shared memory it takes: two pages of bf16 rows, one of FP8
// rows.
template <bool kFp8>
struct Tile {
  static constexpr int kPages = kFp8 ? 1 : 2;
  static constexpr int kKeys = kPages * kPage;
  static constexpr int kHalf = kKeys / 2;                 // keys of K in a CTA, and of a softmax thread
  static constexpr int kKAtom = kHalf * 128;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kQBytes;
  static constexpr int kOffV = kOffK + kAtoms * kKAtom;
  static constexpr int kOffP = kOffV + kPages * kVBytes;
  static constexpr int kOffRaw = kOffP + kPages * kAtom;
  static constexpr int kOffXchg = kOffRaw + (kFp8 ? kRawStages * kRawBytes : 0);      // 2 x 128 floats
  static constexpr int kOffBar = kOffXchg + 2 * 128 * 4;
  static constexpr int kOffInfo = kOffBar + 24 * 8;
  static constexpr int kSmemBytes = kOffInfo + 32 + 1024;
  static constexpr int kStages = kPages;                  // of a warp's output staging
  // What a request's queries and output cost where it begins, in key tiles (128
  // requests of 512 .. 2048 bf16 tokens: 67.5 us for 0, 65.0 for 1, 63.9 for 2, 64.4
  // for 3; 128 of 64 FP8 rows: 33 for 0, 27 for 2).
  static constexpr int kStretch = 2;
  // First atom of K's group g.
  __host__ __device__ static constexpr int group_atom(int g) {
    return kFp8 ? (g < 2 ? 4 * g : 8 + (g - 2)) : kGroupAtoms * g;
  }
};
static_assert(Tile<false>::kSmemBytes <= 232448 && Tile<true>::kSmemBytes <= 232448, "shared memory");
constexpr int kColO = 0, kColS = 256, kTmemCols = 512;    // S: two buffers of a tile's keys / 2 columns
constexpr int kThreads = 256, kThreadsFp8 = 768;
constexpr int kSoftWarps = 4;
constexpr int kStageRow = 64;                             // bytes of a row that an output store takes
// FP8: eight warps dequantise for K, eight for V.  Registers a thread (launched
// with 80 each): copies and MMAs, softmax, dequantisation.  (Shares of 64, 96, 80:
// 251 us for 8 ragged requests of 65536 .. 131072, mean of four runs, against 237;
// 80 each: 244.)
constexpr int kDequantWarps = 8;
constexpr int kRegsMma = 72, kRegsSoft = 88, kRegsDequant = 80;
static_assert(kRegsMma + kRegsSoft + 4 * kRegsDequant <= 6 * 80, "registers");
constexpr float kRaiseLog2 = 8.0f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// mbar_wait by a whole warp: the same answer in every lane.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// Tokens of request r: seqlens[r], at least 0 and at most what its row of the
// page table covers (more is an error the kernel reports).
__device__ __forceinline__ int request_len(const MlaDecodeLaunch& p, int r) {
  const int s = __ldg(p.seqlens + r);
  if (s > p.max_pages * kPage) {
    raise_error(kErrCheck);
    return p.max_pages * kPage;
  }
  return s < 0 ? 0 : s;
}

template <int kKeys>
__device__ __forceinline__ int tiles_of(int len) {
  return (len + kKeys - 1) / kKeys;
}

// The line: for each request with tokens kStretch units and one a key tile.  It is
// cut into groups from unit kStretch on, so that the first request's tiles alone
// count; a cut among a request's kStretch units falls before its first tile.
struct Line {
  long long total;
  int groups;
};

template <int kStretch>
__device__ __forceinline__ long long cut(const Line& ln, int g) {
  return kStretch + (ln.total - kStretch) * g / ln.groups;
}

template <typename T>
__device__ __forceinline__ int units_of(int len) {
  return len > 0 ? tiles_of<T::kKeys>(len) + T::kStretch : 0;
}

// (one warp) The line of all requests.
template <typename T>
__device__ __forceinline__ Line scan_total(const MlaDecodeLaunch& p, int lane) {
  long long n = 0;
  for (int r = lane; r < p.batch; r += 32) n += units_of<T>(request_len(p, r));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  Line ln;
  ln.total = n;
  const long long most = (n - T::kStretch + p.min_tiles - 1) / p.min_tiles;
  ln.groups = most < p.groups ? static_cast<int>(most < 1 ? 1 : most) : p.groups;
  return ln;
}

// (one warp) The request that holds unit `at` of the line (at < total), and the
// line position of its first unit.
template <typename T>
__device__ __forceinline__ void locate(const MlaDecodeLaunch& p, long long at, int lane, int& req,
                                       long long& first) {
  long long base = 0;
  req = 0;
  first = 0;
  for (int r0 = 0; r0 < p.batch; r0 += 32) {
    const int r = r0 + lane;
    const int n = r < p.batch ? units_of<T>(request_len(p, r)) : 0;
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
      first = base + __shfl_sync(0xffffffffu, incl - n, l);
      return;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// The stretches of requests in a group's part [lo, hi) of the line, in order.
template <typename T>
struct Walk {
  long long pos, hi;     // next unit of the line, end of the part
  int req;               // request of the stretch
  int unit;              // unit of it at pos
  int len;               // its tokens
  int t0, t1, nt;        // the stretch's tiles [t0, t1) of the request's nt
  __device__ __forceinline__ bool next(const MlaDecodeLaunch& p) {
    while (pos < hi) {
      if (unit == nt + T::kStretch || nt == 0) {     // on to the next request with tokens
        do {
          ++req;
          len = request_len(p, req);
          nt = tiles_of<T::kKeys>(len);
        } while (nt == 0);
        unit = 0;
      }
      const long long left = hi - pos;
      const int end = static_cast<int>(left < nt + T::kStretch - unit ? unit + left : nt + T::kStretch);
      t0 = max(0, unit - T::kStretch);
      t1 = max(0, end - T::kStretch);
      pos += end - unit;
      unit = end;
      if (t1 > t0) return true;
    }
    return false;
  }
};

// Page ids of a request: table entry i, kNone behind the last page, kBad for an
// id outside the cache.
struct PageIds {
  static constexpr int kNone = -1, kBad = -2;
  const int32_t* table;
  int pages, num_pages;
  __device__ __forceinline__ int get(int i) const {
    if (i >= pages) return kNone;
    const int id = __ldg(table + i);
    return id >= 0 && id < num_pages ? id : kBad;
  }
};

// 16 E4M3 codes times their scale (in fp32), rounded to bf16 as the cache's other
// rows are: the MMAs take no wider operands at their rate.
__device__ __forceinline__ void dequant16(const uint4 raw, float scale, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t o[8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const __half2_raw h01 =
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[q] & 0xFFFFu), __NV_E4M3);
    const __half2_raw h23 =
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[q] >> 16), __NV_E4M3);
    const float2 f01 = mul2(__half22float2(__half2(h01)), make_float2(scale, scale));
    const float2 f23 = mul2(__half22float2(__half2(h23)), make_float2(scale, scale));
    o[2 * q] = pack_bf16x2(f01.x, f01.y);
    o[2 * q + 1] = pack_bf16x2(f23.x, f23.y);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// Pages of a stretch's tiles, 32 ids at a time (an id a lane) and one batch
// ahead.
template <int kPages>
struct PageBatch {
  static constexpr int kTiles = 32 / kPages;      // of a batch
  PageIds ids;
  int t0, now, next;     // first tile of the stretch; ids of this and the next batch
  template <typename T>
  __device__ __forceinline__ PageBatch(const MlaDecodeLaunch& p, const Walk<T>& wk, int lane)
      : ids{p.page_table + static_cast<long long>(wk.req) * p.max_pages, (wk.len + kPage - 1) / kPage,
            p.num_pages},
        t0(wk.t0), now(0) {
    next = ids.get(kPages * t0 + lane);
  }
  // Before tile t's pages are asked for, t going up by one.
  __device__ __forceinline__ bool advance(int t, int lane) {
    if (((t - t0) & (kTiles - 1)) != 0) return false;
    now = next;
    next = ids.get(kPages * (t + kTiles) + lane);
    return true;
  }
  // Page h of tile t.
  __device__ __forceinline__ int page(int t, int h) const {
    return __shfl_sync(0xffffffffu, now, kPages * ((t - t0) & (kTiles - 1)) + h);
  }
};

template <bool kFp8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kFp8 ? kThreadsFp8 : kThreads, 1)
    mla_decode_kernel(const __grid_constant__ CUtensorMap tmap_q,
                      const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v,
                      const __grid_constant__ CUtensorMap tmap_sc,
                      const __grid_constant__ CUtensorMap tmap_out,
                      const __grid_constant__ CUtensorMap tmap_part, const MlaDecodeLaunch p) {
  using T = Tile<kFp8>;
  constexpr int kKeys = T::kKeys;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int worker = blockIdx.x >> 1;
  const int group = worker / p.row_tiles, mtile = worker % p.row_tiles;
  const int rows_req = p.nq * p.heads;
  const float ninf = __int_as_float(0xff800000);

  const uint32_t bar0 = sbase + T::kOffBar;
// In the leading CTA (both CTAs' threads and copies arrive there):
//   Q_FULL, K_FULL(g): q / K group g landed in both CTAs; P_FULL: P written
//   and V landed in both; O_FREE: the epilogue has read the output.
// In both (the MMAs' completion arrives in both): S_FULL(b), K_EMPTY(g),
//   V_EMPTY(h) (P V of page h of the tile done).  In this CTA: V_FULL(h), and
//   (FP8) RAW_FULL(s), RAW_EMPTY(s) of the raw stages.
#define Q_FULL (bar0)
#define O_FREE (bar0 + 8u)
#define DRAIN (bar0 + 16u)
#define P_FULL (bar0 + 24u)
#define K_FULL(g) (bar0 + 32u + 8u * (g))
#define K_EMPTY(g) (bar0 + 56u + 8u * (g))
#define V_FULL(h) (bar0 + 80u + 8u * (h))
#define V_EMPTY(h) (bar0 + 96u + 8u * (h))
#define S_FULL(b) (bar0 + 112u + 8u * (b))
#define RAW_FULL(s) (bar0 + 128u + 8u * (s))
#define RAW_EMPTY(s) (bar0 + 152u + 8u * (s))
  long long* info = reinterpret_cast<long long*>(smem + T::kOffInfo);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + T::kOffInfo + 28);

  if (warp == 0 && lane == 0) {
    mbar_init(Q_FULL, 1);
    mbar_init(O_FREE, 2 * kSoftWarps);
    mbar_init(DRAIN, 1);
    mbar_init(P_FULL, 2 * kSoftWarps);
    for (int g = 0; g < kKGroups; ++g) {
      mbar_init(K_FULL(g), kFp8 && g < 2 ? 2 * kDequantWarps : 1);
      mbar_init(K_EMPTY(g), 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(V_FULL(h), kFp8 ? kDequantWarps : 1);
      mbar_init(V_EMPTY(h), 1);
      mbar_init(S_FULL(h), 1);
    }
    if (kFp8)
      for (int st = 0; st < kRawStages; ++st) {
        mbar_init(RAW_FULL(st), 1);
        mbar_init(RAW_EMPTY(st), 2 * kDequantWarps);
      }
    fence_mbar_init();
    prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  if (warp == 1) {
    tmem_alloc_2cta(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish_2cta();
  }
  if (warp == 3) {
    const Line ln = scan_total<T>(p, lane);
    long long lo = 0, hi = 0, first = 0;
    int req = 0;
    if (group < ln.groups && ln.total > 0) {
      lo = cut<T::kStretch>(ln, group);
      hi = cut<T::kStretch>(ln, group + 1);
      if (hi > lo) locate<T>(p, lo, lane, req, first);
    }
    // What the merge has to join: the request that this group's first cut falls
    // into, if it is the first cut inside that request, and its last group.
    if (mtile == 0 && rank == 0 && lane == 0) {
      int2 join = make_int2(-1, 0);
      const long long tile0 = first + T::kStretch;
      if (group > 0 && hi > lo && lo > tile0 && cut<T::kStretch>(ln, group - 1) <= tile0) {
        const long long tiles = tile0 + tiles_of<kKeys>(request_len(p, req)) - T::kStretch;      // up to its end
        join = make_int2(req, static_cast<int>((tiles * ln.groups - 1) / (ln.total - T::kStretch)));
      }
      p.joins[group] = join;
    }
    if (lane == 0) {
      info[0] = lo;
      info[1] = hi;
      info[2] = (first << 11) | req;      // req < 2^11, first < 2^42
    }
  }
  __syncthreads();
  cluster_sync();     // the other CTA's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  Walk<T> wk;
  wk.pos = info[0];
  wk.hi = info[1];
  wk.req = static_cast<int>(info[2] & 2047);
  wk.len = request_len(p, wk.req);
  wk.nt = tiles_of<kKeys>(wk.len);
  wk.unit = static_cast<int>(wk.pos - (info[2] >> 11));
  wk.t0 = wk.t1 = 0;

  if (warp < 4) {
  if constexpr (kFp8) setmaxnreg_dec<kRegsMma>();
  if (warp == 0) {
    // -------------------------------------------- q and (bf16 rows) K copies
    const uint32_t q_full = mapa_shared(Q_FULL, 0), k_full0 = mapa_shared(K_FULL(0), 0);
    bool ok = true;
    int it = 0;
    while (ok && wk.next(p)) {
      PageBatch<T::kPages> pages(p, wk, lane);
      for (int t = wk.t0; ok && t < wk.t1; ++t, ++it) {
        if (pages.advance(t, lane) && pages.now == PageIds::kBad) raise_error(kErrCheck);
        // (Two pages a tile: each CTA takes one for K.  One: half of it.)
        const int page = max(0, pages.page(t, kFp8 ? 0 : rank));
        const int row = page * kPage + (kFp8 ? T::kHalf * static_cast<int>(rank) : 0);
#pragma unroll
        for (int g = 0; g < kKGroups; ++g) {
          if (it >= 1 && ok && !mbar_wait(K_EMPTY(g), (it - 1) & 1)) ok = false;
          if (!kFp8 && ok && lane == 0) {
            if (rank == 0) mbar_expect_tx(K_FULL(g), 2 * kGroupAtoms * T::kKAtom);
            tma_load_3d_2cta(sbase + T::kOffK + g * kGroupAtoms * T::kKAtom, &tmap_k, 0, row, kGroupAtoms * g,
                             k_full0 + 8u * g);
          }
          if (kFp8 && g == kKGroups - 1 && ok && lane == 0) {
            if (rank == 0) mbar_expect_tx(K_FULL(g), 2 * T::kKAtom);
            tma_load_3d_2cta(sbase + T::kOffK + 8 * T::kKAtom, &tmap_k, kF8RopeOff, row, 0, k_full0 + 8u * g);
          }
          // q of the stretch (Q K^T of the tile before is done with its last
          // group).
          if (g == kKGroups - 1 && t == wk.t0 && ok && lane == 0) {
            if (rank == 0) mbar_expect_tx(Q_FULL, 2 * kQBytes);
            tma_load_3d_2cta(sbase + T::kOffQ, &tmap_q, 0,
                             wk.req * rows_req + mtile * kRowTile + kRowsCta * static_cast<int>(rank), 0, q_full);
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
    }
    if (!ok && lane == 0) raise_error(kErrTimeout);
  } else if (warp == 2) {
    // ----------------------------------------- V copies, or the raw FP8 rows'
    bool ok = true;
    int it = 0;
    while (ok && wk.next(p)) {
      PageBatch<T::kPages> pages(p, wk, lane);
      for (int t = wk.t0; ok && t < wk.t1; ++t, ++it) {
        pages.advance(t, lane);
        if constexpr (kFp8) {
          const int st = it % kRawStages;
          const int row = max(0, pages.page(t, 0)) * kPage, mine = 32 * static_cast<int>(rank);
          if (it >= kRawStages && !mbar_wait(RAW_EMPTY(st), (it / kRawStages - 1) & 1)) ok = false;
          if (ok && lane == 0) {
            // All codes of this CTA's rows (for K and V), its value dims' of the
            // other rows, every row's scales.
            mbar_expect_tx(RAW_FULL(st), kRawBytes);
            const uint32_t dst = sbase + T::kOffRaw + st * kRawBytes;
#pragma unroll
            for (int c = 0; c < 4; ++c) tma_load_3d(dst + c * kRawTile, &tmap_v, 0, row + mine, c, RAW_FULL(st));
#pragma unroll
            for (int n = 0; n < 2; ++n)
              tma_load_3d(dst + (4 + n) * kRawTile, &tmap_v, 0, row + 32 - mine, 2 * n + static_cast<int>(rank),
                          RAW_FULL(st));
            tma_load_3d(dst + 6 * kRawTile, &tmap_sc, kF8ScaleOff, row, 0, RAW_FULL(st));
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int page = max(0, pages.page(t, h));
            if (it >= 1 && ok && !mbar_wait(V_EMPTY(h), (it - 1) & 1)) ok = false;
            if (ok && lane == 0) {
              // Output dims of P V's two MMAs: 256 n + 128 rank .. + 127.
              mbar_expect_tx(V_FULL(h), kVBytes);
              const uint32_t dst = sbase + T::kOffV + h * kVBytes;
              tma_load_3d(dst, &tmap_v, 0, page * kPage, 2 * static_cast<int>(rank), V_FULL(h));
              tma_load_3d(dst + 2 * kAtom, &tmap_v, 0, page * kPage, 4 + 2 * static_cast<int>(rank), V_FULL(h));
            }
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
    }
    if (!ok && lane == 0) raise_error(kErrTimeout);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMAs
    if (rank == 0) {
      // The whole warp runs this; one lane issues.
      const uint32_t el = elect_one() ? 1u : 0u;
      constexpr uint32_t idesc_qk = make_idesc(1, 1, 0, 0, kKeys, kRowTile);
      constexpr uint32_t idesc_pv = make_idesc(1, 1, 0, 1, 256, kRowTile);
      const uint64_t dq = smem_desc_sw128(sbase + T::kOffQ, 16, 1024);
      const uint64_t dk = smem_desc_sw128(sbase + T::kOffK, 16, 1024);
      const uint64_t dp = smem_desc_sw128(sbase + T::kOffP, 16, 1024);
      const uint64_t dv = smem_desc_sw128(sbase + T::kOffV, kAtom, 1024);
      bool ok = true;
      int it = 0, npv = 0;
      // P V of tile npv (its stretch's first: the output starts at zero, once
      // the epilogue has read the stretch before).
      int pv_seg = 0, pv_left = 0;
      Walk<T> pvw = wk;
      auto issue_pv = [&]() -> bool {
        uint32_t fresh = 0;
        if (pv_left == 0) {
          pvw.next(p);
          pv_left = pvw.t1 - pvw.t0;
          fresh = 1;
          if (pv_seg > 0 && !warp_wait(O_FREE, (pv_seg - 1) & 1)) return false;
          ++pv_seg;
        }
        if (!warp_wait(P_FULL, npv & 1)) return false;
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < T::kPages; ++h) {
#pragma unroll
          for (int j = 0; j < kPage / 16; ++j)
#pragma unroll
            for (int n = 0; n < 2; ++n)
              mma_f16_ss_2cta(tmem + kColO + 128 * n, dp + static_cast<uint64_t>((h * kAtom + 32 * j) >> 4),
                              dv + static_cast<uint64_t>((h * kVBytes + n * 2 * kAtom + j * 2048) >> 4),
                              idesc_pv, (h > 0 || j > 0 || !fresh) ? 1u : 0u, el);
          if (el) tc_commit_2cta(V_EMPTY(h), 3);
          __syncwarp();
        }
        --pv_left;
        ++npv;
        return true;
      };
      for (int seg = 0; ok && wk.next(p); ++seg) {
        if (!warp_wait(Q_FULL, seg & 1)) {
          ok = false;
          break;
        }
        for (int t = wk.t0; t < wk.t1; ++t, ++it) {
          // (Scores of tile it - 2 were read: its P V was issued, after its
          // P_FULL.)
#pragma unroll
          for (int g = 0; g < kKGroups; ++g) {
            if (!(ok = ok && warp_wait(K_FULL(g), it & 1))) break;
            tc_fence_after();
#pragma unroll
            for (int a = T::group_atom(g); a < T::group_atom(g + 1); ++a)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                mma_f16_ss_2cta(tmem + kColS + T::kHalf * (it & 1),
                                dq + static_cast<uint64_t>((a * kAtom + j * 32) >> 4),
                                dk + static_cast<uint64_t>((a * T::kKAtom + j * 32) >> 4), idesc_qk,
                                (a > 0 || j > 0) ? 1u : 0u, el);
            if (el) tc_commit_2cta(K_EMPTY(g), 3);
            __syncwarp();
          }
          if (!ok) break;
          if (el) tc_commit_2cta(S_FULL(it & 1), 3);
          __syncwarp();
          if (it > 0 && !(ok = issue_pv())) break;
        }
      }
      if (ok && it > 0) ok = issue_pv();
      if (!ok && el) raise_error(kErrTimeout);
      if (el) tc_commit_2cta(DRAIN, 1);      // every MMA is done before TMEM is freed
      __syncwarp();
      mbar_wait(DRAIN, 0);
    }
    __syncwarp();
  } else if (warp == 3 && mtile == 0) {
    // Requests without tokens (no page of the line is theirs).
    for (int r = group * 2 + static_cast<int>(rank); r < p.batch; r += 2 * p.groups) {
      if (request_len(p, r) > 0) continue;
      const long long row0 = static_cast<long long>(r) * rows_req;
      uint4* dst = reinterpret_cast<uint4*>(p.out + row0 * kVDim);
      for (long long e = lane; e < static_cast<long long>(rows_req) * (kVDim / 8); e += 32)
        dst[e] = make_uint4(0u, 0u, 0u, 0u);
      if (p.lse)
        for (int e = lane; e < rows_req; e += 32) p.lse[row0 + e] = ninf;
    }
  }
  } else if (kFp8 && warp >= 8) {
    // ------------------------------------------- FP8 rows to bf16 operands
    // A warp takes two rows at a time: lane = row r2 of the two and 16-code
    // chunk c of two 128-dim tiles of it.  Eight neighbouring lanes hold four
    // chunks of each row, of different halves of the tile (reads) and with
    // different swizzles (writes): both fall on distinct banks.
    const int r2 = (lane >> 2) & 1, c = ((lane & 3) | ((lane >> 3) << 2)) ^ (r2 << 2);
    const bool for_k = warp < 8 + kDequantWarps;
    const int w = warp & (kDequantWarps - 1);
    // K: rows 4 w .. of this CTA's 32, of dims 0-255, then 256-511.  V: rows 8 w
    // .. of 64, of this CTA's value dims (code tiles rank and 2 + rank).
    const int row0 = (for_k ? 4 : 8) * w + r2;
    const bool own = for_k || (w >> 2) == static_cast<int>(rank);
    const uint32_t k_full0 = mapa_shared(K_FULL(0), 0);
    bool ok = true;
    int it = 0;
    setmaxnreg_dec<kRegsDequant>();
    while (ok && wk.next(p)) {
      PageBatch<T::kPages> pages(p, wk, lane);
      for (int t = wk.t0; ok && t < wk.t1; ++t, ++it) {
        const int st = it % kRawStages;
        const uint8_t* stage = smem + T::kOffRaw + st * kRawBytes;
        const float* scales = reinterpret_cast<const float*>(stage + 6 * kRawTile);
        pages.advance(t, lane);
        if (!mbar_wait(RAW_FULL(st), (it / kRawStages) & 1)) ok = false;
        uint4 raw[4];
        float scale[4];
        if (for_k) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int row = row0 + 2 * (u & 1), tile = 2 * (u >> 1) + (c >> 3);
            raw[u] = *reinterpret_cast<const uint4*>(stage + tile * kRawTile + row * 128 + (c & 7) * 16);
            scale[u] = scales[(32 * rank + row) * 4 + tile];
          }
        } else {
          // Rows that no query sees are zero, whatever the cache holds.
          const int live = pages.page(t, 0) >= 0 ? wk.len - t * kKeys : 0;
          const uint8_t* src = stage + (own ? rank + 2 * (c >> 3) : 4 + (c >> 3)) * kRawTile + (c & 7) * 16;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int row = row0 + 2 * u;
            raw[u] = *reinterpret_cast<const uint4*>(src + (row & 31) * 128);
            scale[u] = scales[row * 4 + rank + 2 * (c >> 3)];
            if (row >= live) {
              raw[u] = make_uint4(0u, 0u, 0u, 0u);
              scale[u] = 0.f;
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(RAW_EMPTY(st));
        if (for_k) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (it >= 1 && ok && !mbar_wait(K_EMPTY(g), (it - 1) & 1)) ok = false;
            uint8_t* dst = smem + T::kOffK + (4 * g + (c >> 2)) * T::kKAtom;
#pragma unroll
            for (int u = 2 * g; u < 2 * g + 2; ++u) {
              const int row = row0 + 2 * (u & 1), piece = (2 * (c & 3)) ^ (row & 7);
              uint4 lo, hi;
              dequant16(raw[u], scale[u], lo, hi);
              *reinterpret_cast<uint4*>(dst + row * 128 + (piece << 4)) = lo;
              *reinterpret_cast<uint4*>(dst + row * 128 + ((piece ^ 1) << 4)) = hi;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote_async(k_full0 + 8u * g);
          }
        } else {
          if (it >= 1 && ok && !mbar_wait(V_EMPTY(0), (it - 1) & 1)) ok = false;
          uint8_t* dst = smem + T::kOffV + (c >> 2) * kAtom;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int row = row0 + 2 * u, piece = (2 * (c & 3)) ^ (row & 7);
            uint4 lo, hi;
            dequant16(raw[u], scale[u], lo, hi);
            *reinterpret_cast<uint4*>(dst + row * 128 + (piece << 4)) = lo;
            *reinterpret_cast<uint4*>(dst + row * 128 + ((piece ^ 1) << 4)) = hi;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(V_FULL(0));
        }
        ok = __all_sync(0xffffffffu, ok);
      }
    }
    if (!ok && lane == 0) raise_error(kErrTimeout);
  } else {
    // ---------------------------------------------- softmax and epilogue
    if constexpr (kFp8) setmaxnreg_inc<kRegsSoft>();
    const int tid = threadIdx.x - 128;             // = TMEM lane; half: of the tile's keys, and of O's dims
    const int w4 = warp & 3;
    const int row = tid & 63, half = tid >> 6;
    const uint32_t lanebase = static_cast<uint32_t>(w4 * 32) << 16;
    const int rrow = mtile * kRowTile + kRowsCta * static_cast<int>(rank) + row;   // row of the request
    const bool live = rrow < rows_req;
    const int qi = live ? rrow / p.heads : 0;
    float* xchg = reinterpret_cast<float*>(smem + T::kOffXchg);
    const uint32_t p_full = mapa_shared(P_FULL, 0), o_free = mapa_shared(O_FREE, 0);
    const float sc = p.sm_scale * kLog2e;
    bool ok = true;
    int it = 0;
    while (wk.next(p)) {
      PageBatch<T::kPages> pages(p, wk, lane);
      const int vis = live ? wk.len - (p.nq - 1 - qi) : 0;
      float mrun = ninf, lrun = 0.f;      // maximum and sum (this thread's keys) in the exp2 domain
      uint32_t good = 0;                  // validity of the next 32 page ids
      for (int t = wk.t0; t < wk.t1; ++t, ++it) {
        const int b = it & 1;
        if (pages.advance(t, lane)) good = __ballot_sync(0xffffffffu, pages.now >= 0);
        // Bit h: page h of the tile can be read.
        const uint32_t ok2 = good >> (T::kPages * ((t - wk.t0) & (32 / T::kPages - 1)));
        if (ok && !mbar_wait(S_FULL(b), (it >> 1) & 1)) ok = false;
        tc_fence_after();
        uint32_t sr[T::kHalf];
        if constexpr (kFp8) tmem_ld32(tmem + lanebase + kColS + T::kHalf * b, sr);
        else tmem_ld64(tmem + lanebase + kColS + T::kHalf * b, sr);
        // Visible keys among this thread's.
        const int seen = ((ok2 >> (kFp8 ? 0 : half)) & 1u) ? vis - t * kKeys - T::kHalf * half : 0;
        float tmax = ninf;
        if (seen >= T::kHalf) {
#pragma unroll
          for (int j = 0; j < T::kHalf; j += 2)
            tmax = max3(tmax, __uint_as_float(sr[j]), __uint_as_float(sr[j + 1]));
        } else {
#pragma unroll
          for (int j = 0; j < T::kHalf; ++j) {
            if (j >= seen) sr[j] = __float_as_uint(ninf);
            tmax = fmaxf(tmax, __uint_as_float(sr[j]));
          }
        }
        // The row's maximum over both halves (the two threads of a row are in
        // warps w and w + 2).
        xchg[b * 128 + tid] = tmax;
        named_bar_sync(1 + (w4 & 1), 64);
        tmax = fmaxf(tmax, xchg[b * 128 + (tid ^ 64)]) * sc;
        const bool raise = tmax > mrun + kRaiseLog2;
        const bool rescale = raise && mrun > ninf;
        if (__any_sync(0xffffffffu, rescale)) {
          // P V of the tile before has to be in the output first.
          if (ok && !mbar_wait(V_EMPTY(T::kPages - 1), (it - 1) & 1)) ok = false;
          tc_fence_after();
          const float f = rescale ? ex2(mrun - tmax) : 1.f;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t o[32];
            tmem_ld32(tmem + lanebase + kColO + 32 * c, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(tmem + lanebase + kColO + 32 * c, o);
          }
          lrun *= f;
        }
        if (raise) mrun = tmax;
        const float mref = mrun > ninf ? mrun : 0.f;
        // P of the tile before has been read: its P V runs before the next Q K^T,
        // which the exponentials then have to hide in.
        if (it >= 1 && ok && !mbar_wait(V_EMPTY(T::kPages - 1), (it - 1) & 1)) ok = false;
        uint8_t* prow = smem + T::kOffP + (kFp8 ? 0 : half * kAtom) + row * 128;
        const int chunk0 = kFp8 ? 4 * half : 0;
        float2 ls = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < T::kHalf / 8; ++c) {
          uint32_t pk[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 x = fma2(make_float2(__uint_as_float(sr[8 * c + 2 * j]), __uint_as_float(sr[8 * c + 2 * j + 1])),
                                  make_float2(sc, sc), make_float2(-mref, -mref));
            const float2 e = make_float2(ex2(x.x), ex2(x.y));
            ls = add2(ls, e);
            pk[j] = pack_bf16x2(e.x, e.y);
          }
          *reinterpret_cast<uint4*>(prow + (((chunk0 + c) ^ (row & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        lrun += ls.x + ls.y;
#pragma unroll
        for (int h = 0; h < T::kPages; ++h) {
          if (ok && !mbar_wait(V_FULL(h), it & 1)) ok = false;
          // Rows of V behind every query's view are cleared.
          const int vlive = ((ok2 >> h) & 1u) ? wk.len - t * kKeys - kPage * h : 0;
          if (!kFp8 && vlive < kPage) {
            uint4* v = reinterpret_cast<uint4*>(smem + T::kOffV + h * kVBytes);
            for (int e = tid; e < kVBytes / 16; e += 128)
              if (((e >> 3) & (kPage - 1)) >= vlive) v[e] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote_async(p_full);
      }
      // ---------------------------------------------------------- epilogue
      if (ok && !mbar_wait(V_EMPTY(T::kPages - 1), (it - 1) & 1)) ok = false;
      tc_fence_after();
      // Row sum over both halves (the buffer that the last tile did not use).
      xchg[(it & 1) * 128 + tid] = lrun;
      named_bar_sync(1 + (w4 & 1), 64);
      const float l = lrun + xchg[(it & 1) * 128 + (tid ^ 64)];
      named_bar_sync(1 + (w4 & 1), 64);
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
      const float lse = l > 0.f || l != l ? (mrun + log2f(l)) * kLn2 : ninf;
      const bool whole = wk.t0 == 0 && wk.t1 == wk.nt;
      const bool whole_warp = (rrow | 31) < rows_req;      // (rrow - lane is a multiple of 32)
      const long long grow = static_cast<long long>(wk.req) * rows_req + rrow;
      const long long slot = (static_cast<long long>(worker) * 2 + (wk.t0 > 0 ? 0 : 1)) * kRowTile +
                             kRowsCta * static_cast<int>(rank) + row;
      if (whole_warp) {
        // 32 rows at once: staged in this warp's part of the P tile (swizzled, so
        // that rows' 16-byte pieces fall on distinct banks) and written by a
        // tensor store, 64 bytes a row at a time.  Stored from registers, every
        // instruction touches 32 lines: 4 us for a stretch's 64 x 512 floats.
        // (FP8: the two warps of a row share 4 KB of P, and write it again only
        // after the barrier of the next tile's maximum.)
        uint8_t* stage0 = smem + T::kOffP + (row & 32) * 128 + half * (kFp8 ? 2048 : kAtom);
        const int row_w = static_cast<int>((whole ? grow : slot) - lane);
        int buf = 0;
        auto put = [&](const uint32_t* v, int dim) {
          uint8_t* stage = stage0 + buf * 2048;
          if (lane == 0) bulk_wait_read<T::kStages - 1>();      // this buffer's store before
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(stage + lane * kStageRow + ((e ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(whole ? &tmap_out : &tmap_part, smem_u32(stage), dim, row_w);
            bulk_commit();
          }
          buf = (buf + 1) % T::kStages;
        };
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t o[32];
          tmem_ld32(tmem + lanebase + kColO + 32 * c, o);
          const int dim = 256 * (c >> 2) + 128 * half + 32 * (c & 3);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
          if (whole) {
            uint32_t h[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              h[e] = pack_bf16x2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
            put(h, dim);
          } else {
            put(o, dim);
            put(o + 16, dim + 16);
          }
        }
        if (lane == 0) bulk_wait_read<0>();      // before the next P is written there
        __syncwarp();
      } else {
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t o[32];
          tmem_ld32(tmem + lanebase + kColO + 32 * c, o);
          const int dim = 256 * (c >> 2) + 128 * half + 32 * (c & 3);
          if (!live) continue;
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(p.out + grow * kVDim + dim);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              dst[e] = make_uint4(
                  pack_bf16x2(__uint_as_float(o[8 * e]) * inv, __uint_as_float(o[8 * e + 1]) * inv),
                  pack_bf16x2(__uint_as_float(o[8 * e + 2]) * inv, __uint_as_float(o[8 * e + 3]) * inv),
                  pack_bf16x2(__uint_as_float(o[8 * e + 4]) * inv, __uint_as_float(o[8 * e + 5]) * inv),
                  pack_bf16x2(__uint_as_float(o[8 * e + 6]) * inv, __uint_as_float(o[8 * e + 7]) * inv));
          } else {
            float4* dst = reinterpret_cast<float4*>(p.part_o + slot * kVDim + dim);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e] = make_float4(__uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                                   __uint_as_float(o[4 * e + 2]) * inv, __uint_as_float(o[4 * e + 3]) * inv);
          }
        }
      }
      if (live && half == 0) {
        if (!whole) p.part_lse[slot] = lse;
        else if (p.lse) p.lse[grow] = lse;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote_async(o_free);
    }
    if (lane == 0) bulk_wait_all();      // the stores are done before the CTA ends
    if (!ok && lane == 0) raise_error(kErrTimeout);
  }
  __syncthreads();
  grid_dep_launch();
  cluster_sync();     // no arrival is under way to a CTA that has ended
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_2cta(tmem, kTmemCols);
  }
#undef Q_FULL
#undef O_FREE
#undef DRAIN
#undef K_FULL
#undef K_EMPTY
#undef V_FULL
#undef V_EMPTY
#undef S_FULL
#undef RAW_FULL
#undef RAW_EMPTY
#undef P_FULL
}

// Joins the partials of a request that spans groups.  Block (i, c): kRows rows
// of the request whose first cut begins group i + 1, if it is one (the attention
// kernel wrote that down: looking it up again in every block made the merge 21 us
// of 80).  The request's first part is slot 1 of its group (a stretch from the
// request's start), the others slot 0 of theirs.
//
// Eight 16-byte loads in flight a thread: of eight parts, 128 threads a row, or,
// where requests have two or three parts and there are many rows, of two, a warp
// a row (128 requests of 512 .. 2048 tokens, 128 heads: the call takes 68 us
// instead of 76; 1 of 4096, 16 heads, where that way is the slower: 20.5 against
// 16.4).  Few rows of many parts: four such groups of threads share a row (kShare;
// 1 request of 131072, 16 heads, 76 parts: 55 us instead of 61; with 512 rows of
// 19 parts, 78 against 70).
constexpr int kMergeThreads = 128;

template <int kParts, int kShare>
__global__ void __launch_bounds__(kMergeThreads * kShare) mla_merge_kernel(const MlaDecodeLaunch p) {
  constexpr int kVecs = 8 / kParts;                          // of a row, a thread
  constexpr int kTpr = kVDim / 4 / kVecs, kRows = kMergeThreads / kTpr;
  const int rows_req = p.nq * p.heads;
  static_assert(kShare == 1 || kRows == 1, "the groups of a block share a row");
  const int share = threadIdx.x / kMergeThreads;
  const int rrow = blockIdx.y * kRows + (kShare > 1 ? 0 : threadIdx.x / kTpr);
  const int c4 = threadIdx.x % kTpr;
  const int m = rrow / kRowTile, lrow = rrow % kRowTile;
  const int g0 = blockIdx.x;
  const float ninf = __int_as_float(0xff800000);
  grid_dep_wait();
  const int2 join = p.joins[g0 + 1];
  if (join.x < 0 || rrow >= rows_req) return;
  const int n = join.y - g0 + 1;      // parts
  auto slot = [&](int i) {
    return (static_cast<long long>((g0 + i) * p.row_tiles + m) * 2 + (i == 0 ? 1 : 0)) * kRowTile + lrow;
  };
  float mx = ninf, tot = 0.f;
  float4 acc[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int b0 = share * kParts; b0 < n; b0 += kShare * kParts) {
    float4 v[kParts][kVecs];
    float e[kParts];
#pragma unroll
    for (int u = 0; u < kParts; ++u) {
      const bool in = b0 + u < n;
      const long long s = slot(in ? b0 + u : 0);
      e[u] = in ? p.part_lse[s] : ninf;
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        v[u][i] = reinterpret_cast<const float4*>(p.part_o + s * kVDim)[c4 + kTpr * i];
    }
    float top = mx;
#pragma unroll
    for (int u = 0; u < kParts; ++u) top = fmaxf(top, e[u]);
    const float mref = top > ninf ? top : 0.f;
    const float f = ex2((mx - mref) * kLog2e);      // (0 for the first batch: its sums are 0)
    mx = top;
    tot *= f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      acc[i] = make_float4(acc[i].x * f, acc[i].y * f, acc[i].z * f, acc[i].w * f);
#pragma unroll
    for (int u = 0; u < kParts; ++u) {
      const float w = ex2((e[u] - mref) * kLog2e);
      // (An empty part holds zeros; its weight is 0.)
      tot += w;
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        acc[i] = make_float4(fmaf(w, v[u][i].x, acc[i].x), fmaf(w, v[u][i].y, acc[i].y),
                             fmaf(w, v[u][i].z, acc[i].z), fmaf(w, v[u][i].w, acc[i].w));
    }
  }
  if constexpr (kShare > 1) {
    __shared__ float4 s_acc[kShare - 1][kMergeThreads];
    __shared__ float2 s_sum[kShare - 1];
    if (share > 0) {
      s_acc[share - 1][c4] = acc[0];
      if (c4 == 0) s_sum[share - 1] = make_float2(mx, tot);
    }
    __syncthreads();
    if (share > 0) return;
    float top = mx;
#pragma unroll
    for (int u = 0; u < kShare - 1; ++u) top = fmaxf(top, s_sum[u].x);
    const float mref = top > ninf ? top : 0.f;
    const float f = ex2((mx - mref) * kLog2e);
    mx = top;
    tot *= f;
    acc[0] = make_float4(acc[0].x * f, acc[0].y * f, acc[0].z * f, acc[0].w * f);
#pragma unroll
    for (int u = 0; u < kShare - 1; ++u) {
      const float w = ex2((s_sum[u].x - mref) * kLog2e);
      const float4 v = s_acc[u][c4];
      tot = fmaf(w, s_sum[u].y, tot);
      acc[0] = make_float4(fmaf(w, v.x, acc[0].x), fmaf(w, v.y, acc[0].y), fmaf(w, v.z, acc[0].z),
                           fmaf(w, v.w, acc[0].w));
    }
  }
  const bool any = tot > 0.f || tot != tot;
  const float inv = any ? 1.f / tot : 0.f;
  const long long grow = static_cast<long long>(join.x) * rows_req + rrow;
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
    reinterpret_cast<uint2*>(p.out + grow * kVDim)[c4 + kTpr * i] = make_uint2(
        pack_bf16x2(acc[i].x * inv, acc[i].y * inv), pack_bf16x2(acc[i].z * inv, acc[i].w * inv));
  if (p.lse && c4 == 0) p.lse[grow] = any ? mx + log2f(tot) * kLn2 : ninf;
}

constexpr int kMinKeys = 256;   // of a group's part of the line, at least

}  // namespace

// Row tiles of a request, groups of CTA pairs (one pair a row tile), and the
// bytes of the partials: two stretches a pair.
void mla_decode_plan(int nq, int heads, int* row_tiles, int* groups, size_t* ws_bytes) {
  const int mt = (nq * heads + kRowTile - 1) / kRowTile;
  int g = device_sm_count() / 2 / mt;
  if (g < 1) g = 1;
  *row_tiles = mt;
  *groups = g;
  *ws_bytes = static_cast<size_t>(g) * mt * 2 * kRowTile * (kVDim + 1) * sizeof(float) + g * sizeof(int2);
}

cudaError_t launch_mla_decode(MlaDecodeLaunch a, void* ws, cudaStream_t s) {
  size_t bytes;
  mla_decode_plan(a.nq, a.heads, &a.row_tiles, &a.groups, &bytes);
  a.part_o = static_cast<float*>(ws);
  const size_t slots = static_cast<size_t>(a.groups) * a.row_tiles * 2 * kRowTile;
  a.part_lse = a.part_o + slots * kVDim;
  a.joins = reinterpret_cast<int2*>(a.part_lse + slots);
  // Rows as 64-dim atoms: one copy brings a box of rows x atoms, each atom's
  // rows 128 bytes apart (128B swizzle).
  const uint64_t qrows = static_cast<uint64_t>(a.batch) * a.nq * a.heads;
  const uint64_t crows = static_cast<uint64_t>(a.num_pages) * kPage;
  const uint64_t strides[2] = {kLatentDim * 2, 128};
  const uint64_t qdims[3] = {64, qrows, kAtoms}, cdims[3] = {64, crows, kAtoms};
  const uint32_t qbox[3] = {64, kRowsCta, kAtoms}, kbox[3] = {64, kPage, kGroupAtoms},
                 vbox[3] = {64, kPage, 2};
  const bool fp8 = a.kv8 != nullptr;
  a.min_tiles = kMinKeys / (fp8 ? Tile<true>::kKeys : Tile<false>::kKeys);
  CUtensorMap tq, tk, tv, ts;
  if (!encode_tmap_nd(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, 3, qdims, strides, qbox,
                      CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  if (fp8) {
    // The rows as bytes: the rope dims laid out like a bf16 atom, the codes of
    // 32 rows x 128 dims, and the scales.
    const uint64_t rdims[3] = {kF8RowBytes, crows, 1}, rstr[2] = {kF8RowBytes, crows * kF8RowBytes};
    const uint64_t tdims[3] = {128, crows, 4}, tstr[2] = {kF8RowBytes, 128};
    const uint32_t rbox[3] = {128, 32, 1}, tbox[3] = {128, 32, 1}, sbox[3] = {16, kPage, 1};
    if (!encode_tmap_nd(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.kv8, 3, rdims, rstr, rbox,
                        CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_nd(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.kv8, 3, tdims, tstr, tbox,
                        CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !encode_tmap_nd(&ts, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.kv8, 3, rdims, rstr, sbox,
                        CU_TENSOR_MAP_SWIZZLE_NONE))
      return cudaErrorInvalidValue;
  } else if (!encode_tmap_nd(&tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.kv, 3, cdims, strides, kbox,
                             CU_TENSOR_MAP_SWIZZLE_128B) ||
             !encode_tmap_nd(&tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.kv, 3, cdims, strides, vbox,
                             CU_TENSOR_MAP_SWIZZLE_128B)) {
    return cudaErrorInvalidValue;
  }
  if (!fp8) ts = tq;      // not used
  CUtensorMap to, tp;
  const uint64_t odims[2] = {kVDim, qrows}, ostr[1] = {kVDim * 2};
  const uint64_t pdims[2] = {kVDim, slots}, pstr[1] = {kVDim * 4};
  const uint32_t obox[2] = {kStageRow / 2, 32}, pbox[2] = {kStageRow / 4, 32};
  if (!encode_tmap_nd(&to, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.out, 2, odims, ostr, obox,
                      CU_TENSOR_MAP_SWIZZLE_64B) ||
      !encode_tmap_nd(&tp, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.part_o, 2, pdims, pstr, pbox,
                      CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  const int smem = fp8 ? Tile<true>::kSmemBytes : Tile<false>::kSmemBytes;
  auto kern = fp8 ? mla_decode_kernel<true> : mla_decode_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_kernel(kern, dim3(2 * a.groups * a.row_tiles), dim3(fp8 ? kThreadsFp8 : kThreads), smem, s,
                    false, 1, tq, tk, tv, ts, to, tp, a);
  if (e != cudaSuccess || a.groups == 1) return e;
  const int rows = a.nq * a.heads;
  auto merge = [&](void (*k)(const MlaDecodeLaunch), int per, int share) {
    return launch_kernel(k, dim3(a.groups - 1, (rows + per - 1) / per), dim3(kMergeThreads * share), 0, s, true, 1, a);
  };
  // (The parts of a request, on average: 1 + groups / batch.)
  if (2 * a.batch >= a.groups) return merge(mla_merge_kernel<2, 1>, 4, 1);
  if (8 * a.batch <= a.groups && a.batch * rows <= 64) return merge(mla_merge_kernel<8, 4>, 1, 4);
  return merge(mla_merge_kernel<8, 1>, 1, 1);
}

}  // namespace dsa
