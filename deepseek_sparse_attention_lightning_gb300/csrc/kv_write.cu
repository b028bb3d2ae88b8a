// kv_write.cu -- the keys and values of packed tokens into the paged caches of a
// layer with grouped heads, at the rows of a slot map (a page of a head is
// contiguous: [num_pages, heads, 64, dim]), copied as bf16 or quantised to FP8
// E4M3 with one fp32 scale for a token and head.
//
//   scale = amax / 448 (1 for zeros),  code = E4M3(x / scale), to nearest even.
//
// Bound by HBM: each value is read and written once.  A thread takes 16 bytes (FP8:
// 32) of a token's keys and the same of its values, so that a warp reads
// consecutive bytes of a row and writes whole segments of a head; a block is as
// wide as a token (or 256).  32767 tokens of 8 heads of 128 dims: bf16 40 us (6.7
// TB/s, 98 % of the measured copy rate), FP8 36 us (5.6 TB/s; the quantisation's
// instructions beside the copies).
#include <cuda_fp8.h>

#include <algorithm>

#include "dsa_ptx.cuh"
#include "dsa_internal.h"

DSA_DEFINE_ERROR_WORD(kv_write)

namespace dsa {
namespace {

constexpr int kThreads = 256;
// Blocks of an SM that registers are kept for (FP8; without it 86 a thread, 58 us for
// 32767 tokens of 8 heads; 4 blocks 37.8, 5 36.3, 6 36.7; two tokens a thread 35.3 to
// 36.3, and slower where there are few).
constexpr int kBlocksFp8 = 5;

// Cache row of a token, or -1 (none, or outside the cache: reported).
__device__ __forceinline__ int slot_of(const KvWriteLaunch& p, int t) {
  const int s = __ldg(p.slots + t);
  if (s < -1 || s >= p.num_pages * kPage) {
    raise_error(kErrCheck);
    return -1;
  }
  return s;
}

// x / b to nearest from y, the reciprocal of b: the product, corrected by its
// remainder (Markstein's division).  Not where remainders leave fp32's range.
__device__ __forceinline__ float2 divide2(float2 x, float b, float y) {
  const float2 q = mul2(x, make_float2(y, y));
  return fma2(fma2(q, make_float2(-b, -b), x), make_float2(y, y), q);
}

// amax / 448, or 1 for zeros.
__device__ __forceinline__ float scale_of(float amax) {
  if (amax < 0x1p-90f) return amax > 0.f ? amax / 448.f : 1.f;
  return divide2(make_float2(amax, 0.f), 448.f, 1.f / 448.f).x;
}

// 16 values over `scale`, as E4M3 codes.  Both are moved into the middle of the range
// by a power of two where they lie near its ends.  (A branch to the compiler's
// division there: 51 us for 32767 tokens of 8 heads, instead of 36.)
__device__ __forceinline__ uint4 encode16(const float2 (&x)[8], float scale) {
  const float f = scale < 0x1p-60f ? 0x1p64f : scale > 0x1p60f ? 0x1p-64f : 1.f;
  const float b = scale * f;
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(b));
#pragma unroll
  for (int i = 0; i < 2; ++i) y = fmaf(fmaf(-b, y, 1.f), y, y);      // Newton's steps
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 q = divide2(mul2(x[e], make_float2(f, f)), b, y);
    const uint32_t c = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
    if (e & 1) o[e >> 1] |= c << 16;
    else o[e >> 1] = c;
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ void unpack16(const uint4 a, const uint4 b, float2 (&x)[8]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = make_float2(bf16lo_to_f32(w[e]), bf16hi_to_f32(w[e]));
}

__device__ __forceinline__ float amax16(const float2 (&x)[8]) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max3(m, fabsf(x[e].x), fabsf(x[e].y));
  return m;
}

// Tokens of a thread.
template <bool kFp8>
constexpr int unroll() {
  return kFp8 ? 1 : 2;
}

// Block: x = pieces of a token (8 values, FP8: 16, of its keys and its values), y =
// tokens.  kShift: log2 of a head's pieces.
template <bool kFp8, int kShift>
__global__ void __launch_bounds__(kThreads, kFp8 ? kBlocksFp8 : 1) kv_write_kernel(const KvWriteLaunch p) {
  constexpr int kValues = kFp8 ? 16 : 8, kUnroll = unroll<kFp8>();
  const int per_token = p.kv_heads << kShift;
  const long long t0 = static_cast<long long>(blockIdx.x) * (kUnroll * blockDim.y) + threadIdx.y;
  int slot[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long t = t0 + u * blockDim.y;
    slot[u] = t < p.tokens ? slot_of(p, static_cast<int>(t)) : -1;
  }
  // (FP8: the lanes of a head stay together: blockDim.x and per_token are multiples
  // of 8.  A warp's lanes may be of several tokens.)
  for (int c = threadIdx.x; c < per_token; c += blockDim.x) {
    const int head = c >> kShift, piece = c & ((1 << kShift) - 1);
    uint4 k[kUnroll][2], v[kUnroll][2];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
#pragma unroll
      for (int e = 0; e < 2; ++e) k[u][e] = v[u][e] = make_uint4(0u, 0u, 0u, 0u);
      if (slot[u] < 0) continue;
      const long long t = t0 + u * blockDim.y;
      const uint4* ks = reinterpret_cast<const uint4*>(p.k + t * p.ld_k + c * kValues);
      const uint4* vs = reinterpret_cast<const uint4*>(p.v + t * p.ld_v + c * kValues);
#pragma unroll
      for (int e = 0; e < kValues / 8; ++e) {
        k[u][e] = __ldg(ks + e);
        v[u][e] = __ldg(vs + e);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      // The row of the caches: its scale's index, and its first piece's >> kShift.
      const long long row = (static_cast<long long>(slot[u] / kPage) * p.kv_heads + head) * kPage + slot[u] % kPage;
      if constexpr (kFp8) {
        float2 xk[8], xv[8];
        unpack16(k[u][0], k[u][1], xk);
        unpack16(v[u][0], v[u][1], xv);
        float mk = amax16(xk), mv = amax16(xv);
        const uint32_t lanes = 0xffu << (threadIdx.y * blockDim.x + threadIdx.x & 24);      // of this head
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) {
          mk = fmaxf(mk, __shfl_xor_sync(lanes, mk, o));
          mv = fmaxf(mv, __shfl_xor_sync(lanes, mv, o));
        }
        if (slot[u] < 0) continue;
        const float sk = scale_of(mk), sv = scale_of(mv);
        reinterpret_cast<uint4*>(p.k_cache)[(row << kShift) + piece] = encode16(xk, sk);
        reinterpret_cast<uint4*>(p.v_cache)[(row << kShift) + piece] = encode16(xv, sv);
        if (piece == 0) {
          p.k_scale[row] = sk;
          p.v_scale[row] = sv;
        }
      } else {
        if (slot[u] < 0) continue;
        reinterpret_cast<uint4*>(p.k_cache)[(row << kShift) + piece] = k[u][0];
        reinterpret_cast<uint4*>(p.v_cache)[(row << kShift) + piece] = v[u][0];
      }
    }
  }
}

template <bool kFp8, int kShift>
cudaError_t launch(const KvWriteLaunch& a, cudaStream_t s) {
  const int per_token = a.kv_heads << kShift;
  const int wide = std::min(per_token, kThreads), tall = kThreads / wide;
  constexpr int kUnroll = unroll<kFp8>();
  const long long grid = (a.tokens + static_cast<long long>(kUnroll) * tall - 1) / (kUnroll * tall);
  return launch_kernel(kv_write_kernel<kFp8, kShift>, dim3(static_cast<unsigned>(grid)), dim3(wide, tall), 0, s, false, 1, a);
}

}  // namespace

cudaError_t launch_kv_write(const KvWriteLaunch& a, cudaStream_t s) {
  if (a.k_scale) return launch<true, 3>(a, s);
  return a.dim == 128 ? launch<false, 4>(a, s) : launch<false, 3>(a, s);
}

}  // namespace dsa
