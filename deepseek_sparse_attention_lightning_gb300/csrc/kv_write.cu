// kv_write.cu -- the keys and values of packed tokens into the paged caches of a
// layer with grouped heads, at the rows of a slot map (a page of a head is
// contiguous: [num_pages, heads, 64, dim]), copied as bf16 or quantised to FP8
// E4M3 with one fp32 scale for a token and head.
//
//   scale = amax / 448 (1 for zeros),  code = E4M3(x / scale), to nearest even.
//
// Bound by HBM: each value is read and written once.  A thread takes 16 bytes (FP8:
// 32) of a token's keys and the same of its values, so that a warp reads
// consecutive bytes of a row and writes whole segments of a head; several tokens
// a thread keep enough loads under way.
#include <cuda_fp8.h>

#include <algorithm>

#include "dsa_ptx.cuh"
#include "dsa_internal.h"

DSA_DEFINE_ERROR_WORD(kv_write)

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;      // pieces of a thread under way

// Cache row of a token, or -1 (none, or outside the cache: reported).
__device__ __forceinline__ int slot_of(const KvWriteLaunch& p, int t) {
  const int s = __ldg(p.slots + t);
  if (s < -1 || s >= p.num_pages * kPage) {
    raise_error(kErrCheck);
    return -1;
  }
  return s;
}

// 16 values over `scale`, as E4M3 codes.  The quotient: x * (1 / scale), corrected
// once by its remainder (Markstein's division), which gives the correctly rounded
// one but for a few borders; a scale near the end of the range, where the
// remainder would be lost, takes the division itself.
__device__ __forceinline__ uint4 encode16(const float2 (&x)[8], float scale) {
  uint32_t o[4];
  const float inv = 1.f / scale;
  const bool safe = scale > 0x1p-90f && scale < 0x1p90f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float2 q;
    if (safe) {
      q = mul2(x[e], make_float2(inv, inv));
      const float2 rem = fma2(q, make_float2(-scale, -scale), x[e]);
      q = fma2(rem, make_float2(inv, inv), q);
    } else {
      q = make_float2(x[e].x / scale, x[e].y / scale);
    }
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

// Piece i of the call: piece c of token t's keys (and values), 8 values (FP8: 16)
// each.  A piece's index in a cache: that of its row, head and place.
template <bool kFp8>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvWriteLaunch p) {
  constexpr int kValues = kFp8 ? 16 : 8;
  const int per_head = p.dim / kValues, per_token = p.kv_heads * per_head;      // pieces
  const long long total = static_cast<long long>(p.tokens) * per_token;
  const long long step = static_cast<long long>(gridDim.x) * kThreads;
  // (FP8: a whole warp stays together, its lanes reduce over a head's pieces.)
  for (long long i0 = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; (kFp8 ? i0 - (threadIdx.x & 31) : i0) < total;
       i0 += kUnroll * step) {
    uint4 k[kUnroll][2], v[kUnroll][2];
    long long at[kUnroll];      // piece of the cache, or -1
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const long long i = i0 + u * step;
      at[u] = -1;
#pragma unroll
      for (int e = 0; e < 2; ++e) k[u][e] = v[u][e] = make_uint4(0u, 0u, 0u, 0u);
      if (i >= total) continue;
      const int t = static_cast<int>(i / per_token), c = static_cast<int>(i - static_cast<long long>(t) * per_token);
      const int slot = slot_of(p, t);
      if (slot < 0) continue;
      const int head = c / per_head;
      at[u] = ((static_cast<long long>(slot / kPage) * p.kv_heads + head) * kPage + slot % kPage) * per_head + (c - head * per_head);
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
      if constexpr (kFp8) {
        float2 xk[8], xv[8];
        unpack16(k[u][0], k[u][1], xk);
        unpack16(v[u][0], v[u][1], xv);
        float mk = amax16(xk), mv = amax16(xv);
        // (per_head lanes, a power of two, hold a head's values; a head's pieces
        // start at a multiple of that, and are together in or out of range.)
        for (int o = per_head >> 1; o > 0; o >>= 1) {
          mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
          mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
        }
        if (at[u] < 0) continue;
        const float sk = mk > 0.f ? mk / 448.f : 1.f, sv = mv > 0.f ? mv / 448.f : 1.f;
        reinterpret_cast<uint4*>(p.k_cache)[at[u]] = encode16(xk, sk);
        reinterpret_cast<uint4*>(p.v_cache)[at[u]] = encode16(xv, sv);
        if (at[u] % per_head == 0) {
          p.k_scale[at[u] / per_head] = sk;
          p.v_scale[at[u] / per_head] = sv;
        }
      } else {
        if (at[u] < 0) continue;
        reinterpret_cast<uint4*>(p.k_cache)[at[u]] = k[u][0];
        reinterpret_cast<uint4*>(p.v_cache)[at[u]] = v[u][0];
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_write(const KvWriteLaunch& a, cudaStream_t s) {
  const bool fp8 = a.k_scale != nullptr;
  const long long pieces = static_cast<long long>(a.tokens) * a.kv_heads * (a.dim / (fp8 ? 16 : 8));
  const long long most = (pieces + kThreads - 1) / kThreads;
  const int grid = static_cast<int>(std::min<long long>(most, 16LL * device_sm_count()));
  return launch_kernel(fp8 ? kv_write_kernel<true> : kv_write_kernel<false>, dim3(grid), dim3(kThreads), 0, s, false, 1, a);
}

}  // namespace dsa
