// rmsnorm.cu -- the norm in front of a layer's projections (and of the cached
// latent): residual addition, root-mean-square norm, and the output in bf16
// and/or FP8 E4M3 with fp32 scales.
//
//   h = x + residual,  y = h / sqrt(mean(h^2) + eps) * weight,
//   scale = amax(|y| over a tile) / 448 (1 for a tile of zeros),
//   code = E4M3(y / scale), rounded to nearest even and saturated.
//
// Everything between the loads and the outputs is fp32: h is rounded only where
// it is stored as the next residual, y only where it is stored in bf16.  The
// codes come from t = h * weight: y = t / rms, so y / scale = t / (amax |t| /
// 448), without the roundings of the reciprocal root and of y (each moves a
// few codes that lie near a border).  A tile is 128 columns (the 1 x 128 tiles of
// "Deepseek Details", section "FP8 Training"; the last may be shorter) or the
// whole row, the two granularities of the library's other quantisers.
//
// Each value is read once, kept in registers across the row's reduction and
// written once.  The threads of a row (as many warps as it takes, with V vectors
// of 8 values each) load 16 bytes each, so that a warp's load is 512 consecutive
// bytes and 16 neighbouring lanes hold one 128-column tile.  Rows of few warps
// share a block: one row of 2048 columns a block of 128 threads took 111 us for
// 32768 rows, codes alone, against 61; one of 640, 96 against 29.
//
// With a residual bound by HBM: 16384 x 8192, both outputs, 177 us (6.8 TB/s of
// the measured 6.79).  Without one by the arithmetic and the latency of a row's
// phases: codes alone 113 us (53 %), bf16 as well 123 us (81 %); fewer registers
// and more rows at a time (V = 2, 3), more vectors a thread (V = 8), the next
// row's loads under way in blocks that stay: all the same or slower.
#include <cuda_fp8.h>

#include "dsa_ptx.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kNormBlock = 256;   // threads of a block of several rows

// Sum (or maximum) over the warps of a row (threadIdx.y of the block); every
// thread gets it.  `buf`: a float a warp, for one call of a kernel.
template <bool kMax, bool kWarp>
__device__ __forceinline__ float row_reduce(float v, float* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? fmaxf(v, u) : v + u;
  }
  const int warps = kWarp ? 1 : blockDim.x >> 5;
  if (warps > 1) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) buf[threadIdx.x >> 5] = v;
    // (An id that is not a constant reserves all sixteen barriers, and those of
    // the SM then admit four blocks: 168 us instead of 135 for 32704 x 4104.)
    switch (threadIdx.y) {
      case 0: named_bar_sync(1, blockDim.x); break;
      case 1: named_bar_sync(2, blockDim.x); break;
      case 2: named_bar_sync(3, blockDim.x); break;
      default: named_bar_sync(4, blockDim.x); break;
    }
    v = lane < warps ? buf[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float u = __shfl_xor_sync(0xffffffffu, v, o);
      v = kMax ? fmaxf(v, u) : v + u;
    }
  }
  return v;
}

__device__ __forceinline__ void unpack8(const uint4 v, float2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = make_float2(bf16lo_to_f32(w[e]), bf16hi_to_f32(w[e]));
}

__device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
  return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                    pack_bf16x2(f[3].x, f[3].y));
}

// Block: x = threads of a row, y = rows.
template <int V, bool kWarp>
__global__ void __launch_bounds__(kWarp ? kNormBlock : 1024, V == 2 ? 6 : 1) rmsnorm_kernel(const RmsNormLaunch p) {
  __shared__ float red[2][32];
  const int tid = threadIdx.x, tpr = kWarp ? 32 : blockDim.x;
  const long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (row >= p.rows) return;   // all threads of a row
  float* buf = red[0] + threadIdx.y * (tpr >> 5);
  const int nvec = p.dim >> 3;
  // Plain loads: an output may be the input it replaces (every thread writes
  // only the vectors it read).
  const uint4* x = reinterpret_cast<const uint4*>(p.x + row * p.ld_x);
  const uint4* res = p.residual ? reinterpret_cast<const uint4*>(p.residual + row * p.dim) : nullptr;

  uint4 xv[V], rv[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = tid + k * tpr;
    xv[k] = c < nvec ? x[c] : make_uint4(0u, 0u, 0u, 0u);
    rv[k] = (res && c < nvec) ? res[c] : make_uint4(0u, 0u, 0u, 0u);
  }
  float2 h[V][4];
  float2 ss2 = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    float2 r[4];
    unpack8(xv[k], h[k]);
    unpack8(rv[k], r);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      h[k][e] = add2(h[k][e], r[e]);
      ss2 = fma2(h[k][e], h[k][e], ss2);
    }
  }
  const float ss = row_reduce<false, kWarp>(ss2.x + ss2.y, buf);
  const float rstd = 1.f / sqrtf(ss / static_cast<float>(p.dim) + p.eps);

  const uint4* wt = reinterpret_cast<const uint4*>(p.weight);
  uint4* hout = p.residual_out ? reinterpret_cast<uint4*>(p.residual_out + row * p.dim) : nullptr;
  uint4* yout = p.y ? reinterpret_cast<uint4*>(p.y + row * p.dim) : nullptr;
  float amax[V];         // of |t| of a vector
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = tid + k * tpr;
    amax[k] = 0.f;
    if (c < nvec) {
      if (hout) hout[c] = pack8(h[k]);
      float2 w[4];
      unpack8(__ldg(wt + c), w);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[k][e] = mul2(h[k][e], w[e]);                   // t
        amax[k] = max3(amax[k], fabsf(h[k][e].x), fabsf(h[k][e].y));
      }
      if (yout) {
        float2 y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = mul2(h[k][e], make_float2(rstd, rstd));
        yout[c] = pack8(y);
      }
    }
  }
  if (!p.y8) return;

  uint2* codes = reinterpret_cast<uint2*>(p.y8 + row * p.dim);
  float a = 0.f;
  if (p.group == 0) {
#pragma unroll
    for (int k = 0; k < V; ++k) a = fmaxf(a, amax[k]);
    a = row_reduce<true, kWarp>(a, buf + 32);
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = tid + k * tpr;
    if (p.group != 0) {
      // 16 lanes hold the vectors of one 128-column tile (past the row's end
      // they hold zeros).
      a = amax[k];
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    }
    if (c >= nvec) continue;
    // amax |y|.  A tile of zeros has scale 1 and codes 0, also where y is zero
    // because the row's sum of squares overflowed (rstd = 0) or amax |t| / rms
    // rounds to zero.  (A row whose rms is zero or not a number keeps its NaN in
    // the scale.)
    const float ymax = a * rstd;
    if (p.group != 0 ? (c & 15) == 0 : c == 0) {
      const float scale = ymax == 0.f ? 1.f : ymax / 448.f;
      if (p.group != 0) p.y_scale[row * ((p.dim + 127) >> 7) + (c >> 4)] = scale;
      else p.y_scale[row] = scale;
    }
    // t / (a / 448) as the product t * (448 / a): as many roundings, and a
    // division a tile instead of one a value (16384 x 8192, codes alone: 139
    // against 113 us; 8388608 codes: 20 to 80 more of them off by one, beside
    // ~700 ties).  Refining the product by its residual gave the division's
    // codes for 121 us.  (The reciprocal of the smallest tiles would overflow.)
    float top = a;
    if (top < 0x1p-96f) {
      top *= 0x1p64f;
#pragma unroll
      for (int e = 0; e < 4; ++e) h[k][e] = mul2(h[k][e], make_float2(0x1p64f, 0x1p64f));
    }
    const float inv = ymax == 0.f ? 0.f : top > 0.f ? 448.f / top : 1.f;
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 q = mul2(h[k][e], make_float2(inv, inv));
      o[e] = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
    }
    codes[c] = make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
  }
}

template <int V, bool kWarp>
cudaError_t launch(const RmsNormLaunch& a, cudaStream_t s) {
  const int tpr = ((a.dim >> 3) + 32 * V - 1) / (32 * V) * 32;      // threads of a row
  const int per = tpr < kNormBlock ? kNormBlock / tpr : 1;
  const long long grid = (a.rows + per - 1) / per;
  return launch_kernel(rmsnorm_kernel<V, kWarp>, dim3(static_cast<unsigned>(grid)), dim3(tpr, per), 0, s, false, 1,
                       a);
}

}  // namespace

cudaError_t launch_rmsnorm(const RmsNormLaunch& a, cudaStream_t s) {
  const int nvec = a.dim >> 3;
  // A row a warp: no barrier.  (Two vectors a thread: 40 registers, six blocks an
  // SM: 32768 x 512 to bf16 in 14.5 us; with 44 registers, five blocks, 16.3.)
  if (nvec <= 64) return launch<2, true>(a, s);
  if (nvec <= 128) return launch<4, true>(a, s);
  return launch<4, false>(a, s);
}

}  // namespace dsa
