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
// Bound by the matrix pipe: 640 flop a visible pair against ~5 bytes of
// exponentials' operands in registers.  One CTA = 256 queries of one head, as
// two query tiles of 128 (M = 128): while one tile's scores are in the softmax,
// the matrix pipe works on the other's.
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
// Warps 0-3 and 4-7: softmax and epilogue of query tile 0 and 1, a row a
// thread.  Warp 8: copies.  Warp 9: MMAs, issued from uniform control flow.
// The running maximum is raised lazily (by 2^8 at least), by the row's own
// thread, which then rescales its row of O.  P is rounded to bf16 for the
// matrix pipe, its sum kept unrounded in fp32.
//
// Keys behind a request's end (the next request's rows in the packed tensors)
// get probability zero, and their rows of V are cleared in shared memory: they
// may hold anything.
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
constexpr int kNumBars = 17;
constexpr int kOffSlot = kOffBar + kNumBars * 8;
constexpr int kSmemBytes = kOffSlot + 16 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory");
constexpr int kThreads = 384;                  // two softmax warpgroups; copies, MMAs and two idle warps
// Registers: launched with 168 a thread (384 x 168 = 64512); the softmax holds a
// row of 128 scores and takes 208, the third warpgroup keeps 88 (256 x 208 +
// 128 x 88 = 64512).
constexpr int kSoftRegs = 208, kOtherRegs = 88;
static_assert(256 * kSoftRegs + 128 * kOtherRegs <= 384 * 168, "registers");
constexpr int kColS = 0, kColO = 256, kTmemCols = 512;
constexpr float kRaiseLog2 = 8.0f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// Keys a query row sees: its own token and those before it, or all.
__device__ __forceinline__ int key_limit(int row, int qlen, int klen, int causal) {
  return causal ? max(0, klen - qlen + row + 1) : klen;
}

__global__ void __launch_bounds__(kThreads, 1)
    mla_prefill_kernel(const __grid_constant__ CUtensorMap tmap_q,
                       const __grid_constant__ CUtensorMap tmap_kv,
                       const __grid_constant__ CUtensorMap tmap_rope, const MlaPrefillLaunch p) {
  extern __shared__ uint8_t smem_raw[];
  const int head = blockIdx.y, req = blockIdx.z;
  // Late queries see the most keys: they start first.
  const int row0 = static_cast<int>(gridDim.x - 1 - blockIdx.x) * kCtaRows;
  const int q0 = __ldg(p.cu_q + req), k0 = __ldg(p.cu_k + req);
  const int qlen = __ldg(p.cu_q + req + 1) - q0, klen = max(0, __ldg(p.cu_k + req + 1) - k0);
  // Offsets outside the packed tensors, or a length above max_q, are reported;
  // the request's rows are left as they were, or not all of them written.
  const bool bad = q0 < 0 || k0 < 0 || qlen < 0 || q0 + qlen > p.total_q || k0 + klen > p.total_k;
  if (bad || qlen > static_cast<int>(gridDim.x) * kCtaRows) {
    if (threadIdx.x == 0) raise_error(kErrCheck);
    if (bad) return;
  }
  if (row0 >= qlen) return;
  // Key tiles of the two query tiles.
  auto tiles_from = [&](int first) {
    if (first >= qlen) return 0;
    return (key_limit(min(first + kTile, qlen) - 1, qlen, klen, p.causal) + kTile - 1) / kTile;
  };
  const int nt0 = tiles_from(row0), nt1 = tiles_from(row0 + kTile), ntmax = max(nt0, nt1);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const float ninf = __int_as_float(0xff800000);

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffSlot);
  const uint32_t bar0 = sbase + kOffBar;
// K / V of key tile j (at most two of each are in the ring): landed, and read.
#define K_FULL(j) (bar0 + 8u * ((j) & 1))
#define V_FULL(j) (bar0 + 16u + 8u * ((j) & 1))
#define K_EMPTY(j) (bar0 + 32u + 8u * ((j) & 1))
#define V_EMPTY(j) (bar0 + 48u + 8u * ((j) & 1))
#define PARITY(j) (((j) >> 1) & 1)
#define Q_FULL(q) (bar0 + 64u + 8u * (q))
#define S_FULL(q) (bar0 + 80u + 8u * (q))
#define P_FULL(q) (bar0 + 96u + 8u * (q))
#define O_FULL(q) (bar0 + 112u + 8u * (q))
#define DRAIN (bar0 + 128u)

  if (warp == 8 && lane == 0) {
    for (int q = 0; q < 2; ++q) {
      mbar_init(K_FULL(q), 1);
      mbar_init(V_FULL(q), 1);
      mbar_init(K_EMPTY(q), 1);
      mbar_init(V_EMPTY(q), 1);
      mbar_init(Q_FULL(q), 1);
      mbar_init(S_FULL(q), 1);
      mbar_init(P_FULL(q), kTile);
      mbar_init(O_FULL(q), 1);
    }
    mbar_init(DRAIN, 1);
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

  if (warp >= 8) {
  setmaxnreg_dec<kOtherRegs>();
  if (warp == 8) {
    // ------------------------------------------------------------- copies
    if (lane == 0) {
      bool ok = true;
      int n = 0;
      const uint64_t pol_rope = policy_evict_last();      // every head reads it
      for (int j = 0; ok && j < ntmax; ++j) {
        for (int g = 0; g < kPerTile; ++g, ++n) {
          // The granule's slot held granule n - kRing, of an earlier tile.
          const int old = n - kRing, oj = old / kPerTile;
          if (old >= 0 &&
              !(ok = mbar_wait(old % kPerTile < kKGranules ? K_EMPTY(oj) : V_EMPTY(oj), PARITY(oj))))
            break;
          const uint32_t bar = g < kKGranules ? K_FULL(j) : V_FULL(j);
          if (g == 0) mbar_expect_tx(bar, kKGranules * kAtomBytes);
          if (g == kKGranules) mbar_expect_tx(bar, (kPerTile - kKGranules) * kAtomBytes);
          const uint32_t dst = sbase + kOffRing + (n % kRing) * kAtomBytes;
          const int row = k0 + j * kTile;
          if (g == 2) tma_load_2d(dst, &tmap_rope, 0, row, bar, pol_rope);
          else tma_load_4d(dst, &tmap_kv, 0, row, g < 2 ? g : g - 1, head, bar);
          if (j == 0 && g < 2 && (g == 0 ? nt0 : nt1) > 0) {
            mbar_expect_tx(Q_FULL(g), kQAtoms * kAtomBytes);
            tma_load_4d(sbase + kOffQ + g * kQAtoms * kAtomBytes, &tmap_q, 0, q0 + row0 + g * kTile, 0,
                        head, Q_FULL(g));
          }
        }
      }
      if (!ok) raise_error(kErrTimeout);
      // No copy is in flight when the CTA ends.
      if (ok)
        for (int j = max(0, ntmax - 2); j < ntmax; ++j) {
          mbar_wait(K_FULL(j), PARITY(j));
          mbar_wait(V_FULL(j), PARITY(j));
        }
      for (int q = 0; q < 2; ++q)
        if (ntmax > 0 && (q == 0 ? nt0 : nt1) > 0) mbar_wait(Q_FULL(q), 0);
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
      if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) {
        done_bar = bar;
        done_parity = parity;
      }
    };
    // (A phase that completed stays the barrier's latest until its data has
    // been used, so a remembered answer does not go stale before that; it is
    // dropped after a use.)
    // What the step after the current one waits for: K, V or P.
    auto qk = [&](int q, int j, uint32_t next_bar, uint32_t next_parity) {
#pragma unroll
      for (int a = 0; a < kQAtoms; ++a) {
        const uint64_t dk = dr0 + static_cast<uint64_t>((((j * kPerTile + a) % kRing) * kAtomBytes) >> 4);
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
    auto pv = [&](int q, int j, uint32_t next_bar, uint32_t next_parity) {
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const uint64_t dv = dr0 + static_cast<uint64_t>((((j * kPerTile + 3 + a) % kRing) * kAtomBytes) >> 4);
        if (a == 1) peek(next_bar, next_parity);
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          mma_f16_ts_uni(tmem + kColO + kHeadDim * q + 64 * a, tmem + kColS + kTile * q + 8 * k,
                         dv + static_cast<uint64_t>((2048 * k) >> 4), idesc_pv, (j > 0 || k > 0) ? 1u : 0u,
                         el);
      }
      if (j == (q == 0 ? nt0 : nt1) - 1) {
        if (el) tc_commit(O_FULL(q));
        __syncwarp();
      }
    };
    auto commit = [&](uint32_t bar) {
      if (el) tc_commit(bar);
      __syncwarp();
    };
    for (int j = 0; ok && j <= ntmax; ++j) {
      if (j < nt0) {
        if (j == 0) ok = warp_wait(Q_FULL(0), 0);
        want(K_FULL(j), PARITY(j));
        tc_fence_after();
        if (ok) qk(0, j, P_FULL(1), (j - 1) & 1);
      }
      if (ok && j >= 1) {
        if (j - 1 < nt1) {
          if (j - 1 >= nt0) ok = ok && warp_wait(V_FULL(j - 1), PARITY(j - 1));
          want(P_FULL(1), (j - 1) & 1);
          tc_fence_after();
          if (ok) pv(1, j - 1, K_FULL(j), PARITY(j));
        }
        commit(V_EMPTY(j - 1));
      }
      if (!ok || j == ntmax) break;
      if (j < nt1) {
        if (j == 0) ok = warp_wait(Q_FULL(1), 0);
        if (j >= nt0) want(K_FULL(j), PARITY(j));
        tc_fence_after();
        if (ok) qk(1, j, P_FULL(0), j & 1);
      }
      commit(K_EMPTY(j));
      if (j < nt0) {
        want(P_FULL(0), j & 1);
        ok = ok && warp_wait(V_FULL(j), PARITY(j));
        tc_fence_after();
        if (ok) pv(0, j, K_FULL(j + 1), PARITY(j + 1));
      }
    }
    if (!ok && el) raise_error(kErrTimeout);
    if (el) tc_commit(DRAIN);      // every MMA is done before TMEM is freed
    __syncwarp();
    mbar_wait(DRAIN, 0);
  }
  } else {
    // ---------------------------------------------- softmax and epilogue
    setmaxnreg_inc<kSoftRegs>();
    const int q = warp >> 2, w4 = warp & 3;
    const int n = (q == 0 ? nt0 : nt1);
    const int row = row0 + q * kTile + w4 * 32 + lane;     // of the request
    const bool live = row < qlen;
    const uint32_t tS = tmem + (static_cast<uint32_t>(w4 * 32) << 16) + kColS + kTile * q;
    const uint32_t tO = tmem + (static_cast<uint32_t>(w4 * 32) << 16) + kColO + kHeadDim * q;
    const int lim = live ? min(klen, key_limit(row, qlen, klen, p.causal)) : 0;
    const float sc = p.sm_scale * kLog2e;
    float mrun = ninf, lrun = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      if (ok && !mbar_wait(S_FULL(q), j & 1)) ok = false;
      tc_fence_after();
      uint32_t s[128];
      tmem_ld128(tS, s);
      const int seen = lim - j * kTile;
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
      float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t pk[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float2 x = fma2(make_float2(__uint_as_float(s[64 * c + 2 * e]),
                                            __uint_as_float(s[64 * c + 2 * e + 1])),
                                make_float2(sc, sc), make_float2(-mref, -mref));
          const float2 w = make_float2(ex2(x.x), ex2(x.y));
          ls[e & 1] = add2(ls[e & 1], w);
          pk[e] = pack_bf16x2(w.x, w.y);
        }
        tmem_st32(tS + 32 * c, pk);
      }
      lrun += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
      // Rows of V behind the request's end are cleared, by the first query
      // tile that reads them.
      const int vlive = klen - j * kTile;
      if (vlive < kTile && (q == 0 || j >= nt0)) {
        if (ok && !mbar_wait(V_FULL(j), PARITY(j))) ok = false;
#pragma unroll 1
        for (int a = 0; a < 2; ++a) {
          uint4* v = reinterpret_cast<uint4*>(smem + kOffRing + ((j * kPerTile + 3 + a) % kRing) * kAtomBytes);
          for (int e = (threadIdx.x & 127) + vlive * 8; e < kAtomBytes / 16; e += 128)
            v[e] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();
      mbar_arrive(P_FULL(q));
    }
    if (n > 0) {
      if (ok && !mbar_wait(O_FULL(q), 0)) ok = false;
      tc_fence_after();
    }
    if (!ok && lane == 0) raise_error(kErrTimeout);
    const bool any = lrun > 0.f || lrun != lrun;
    const float inv = any ? 1.f / lrun : 0.f;
    const long long orow = (static_cast<long long>(q0) + row) * p.heads + head;
    uint4* dst = reinterpret_cast<uint4*>(p.out + orow * kHeadDim);
    if (row0 + q * kTile < qlen) {
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        if (n > 0) tmem_ld32(tO + 32 * c, o);
        if (!live) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = any ? pack_bf16x2(__uint_as_float(o[8 * e + 2 * i]) * inv,
                                     __uint_as_float(o[8 * e + 2 * i + 1]) * inv)
                       : 0u;
          dst[4 * c + e] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (live && p.lse) p.lse[orow] = any ? (mrun + log2f(lrun)) * kLn2 : ninf;
    }
    tc_fence_before();
  }
  __syncthreads();
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
#undef DRAIN
}

}  // namespace

cudaError_t launch_mla_prefill(const MlaPrefillLaunch& a, cudaStream_t s) {
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
  const dim3 grid((a.max_q + kCtaRows - 1) / kCtaRows, a.heads, a.batch);
  return launch_kernel(mla_prefill_kernel, grid, dim3(kThreads), kSmemBytes, s, false, 1, tq, tk, tr, a);
}

}  // namespace dsa
