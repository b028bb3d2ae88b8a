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
// Memory bound: each value is read once, kept in registers across the row's
// reduction and written once.  TPR threads share a row, each with V vectors of
// 8 values (16-byte loads, TPR apart, so that a warp's load is 512 consecutive
// bytes and 16 neighbouring lanes hold one 128-column tile).
#include <cuda_fp8.h>

#include "dsa_ptx.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kNormBlock = 256;   // threads of a block of several rows

// Sum (or maximum) over the TPR threads of a row; every thread gets it.  `buf`
// (one float per warp) serves one call of a kernel.
template <int TPR, bool kMax>
__device__ __forceinline__ float row_reduce(float v, float* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? fmaxf(v, u) : v + u;
  }
  if constexpr (TPR > 32) {
    constexpr int kW = TPR / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) buf[warp] = v;
    __syncthreads();
    v = lane < kW ? buf[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float u = __shfl_xor_sync(0xffffffffu, v, o);
      v = kMax ? fmaxf(v, u) : v + u;
    }
  }
  return v;
}

__device__ __forceinline__ void unpack8(const uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = bf16lo_to_f32(w[e]);
    f[2 * e + 1] = bf16hi_to_f32(w[e]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

template <int TPR, int V>
__global__ void __launch_bounds__(TPR > kNormBlock ? TPR : kNormBlock)
    rmsnorm_kernel(const RmsNormLaunch p) {
  __shared__ float red[2][32];
  const int tid = TPR > 32 ? threadIdx.x : (threadIdx.x & 31);
  const long long row = TPR > 32 ? static_cast<long long>(blockIdx.x)
                                 : static_cast<long long>(blockIdx.x) * (kNormBlock / 32) +
                                       (threadIdx.x >> 5);
  if (row >= p.rows) return;   // a whole warp (TPR = 32) or never
  const int nvec = p.dim >> 3;
  // Plain loads: an output may be the input it replaces (every thread writes
  // only the vectors it read).
  const uint4* x = reinterpret_cast<const uint4*>(p.x + row * p.ld_x);
  const uint4* res = p.residual ? reinterpret_cast<const uint4*>(p.residual + row * p.dim) : nullptr;

  uint4 xv[V], rv[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = tid + k * TPR;
    xv[k] = c < nvec ? x[c] : make_uint4(0u, 0u, 0u, 0u);
    rv[k] = (res && c < nvec) ? res[c] : make_uint4(0u, 0u, 0u, 0u);
  }
  float h[V][8];
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    float r[8];
    unpack8(xv[k], h[k]);
    unpack8(rv[k], r);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[k][e] += r[e];
      ss = fmaf(h[k][e], h[k][e], ss);
    }
  }
  ss = row_reduce<TPR, false>(ss, red[0]);
  const float rstd = 1.f / sqrtf(ss / static_cast<float>(p.dim) + p.eps);

  const uint4* wt = reinterpret_cast<const uint4*>(p.weight);
  uint4* hout = p.residual_out ? reinterpret_cast<uint4*>(p.residual_out + row * p.dim) : nullptr;
  uint4* yout = p.y ? reinterpret_cast<uint4*>(p.y + row * p.dim) : nullptr;
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = tid + k * TPR;
    if (c < nvec) {
      if (hout) hout[c] = pack8(h[k]);
      float w[8];
      unpack8(__ldg(wt + c), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[k][e] *= w[e];                   // t
        amax = fmaxf(amax, fabsf(h[k][e]));
      }
      if (yout) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = h[k][e] * rstd;
        yout[c] = pack8(y);
      }
    }
  }
  if (!p.y8) return;

  uint2* codes = reinterpret_cast<uint2*>(p.y8 + row * p.dim);
  float step = 1.f;      // scale / rstd
  if (p.group == 0) {
    amax = row_reduce<TPR, true>(amax, red[1]);
    step = amax > 0.f ? amax / 448.f : 1.f;
    if (tid == 0) p.y_scale[row] = amax > 0.f ? step * rstd : 1.f;
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = tid + k * TPR;
    if (p.group != 0) {
      // 16 lanes hold the vectors of one 128-column tile (past the row's end
      // they hold zeros).
      float a = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(h[k][e]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      step = a > 0.f ? a / 448.f : 1.f;
      if (c < nvec && (c & 15) == 0)
        p.y_scale[row * ((p.dim + 127) >> 7) + (c >> 4)] = a > 0.f ? step * rstd : 1.f;
    }
    if (c < nvec) {
      uint32_t o[2] = {0u, 0u};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        o[e >> 2] |= static_cast<uint32_t>(
                         __nv_cvt_float_to_fp8(h[k][e] / step, __NV_SATFINITE, __NV_E4M3))
                     << (8 * (e & 3));
      codes[c] = make_uint2(o[0], o[1]);
    }
  }
}

template <int TPR, int V>
cudaError_t launch(const RmsNormLaunch& a, cudaStream_t s) {
  constexpr int threads = TPR > 32 ? TPR : kNormBlock;
  const long long per = TPR > 32 ? 1 : kNormBlock / 32;
  const long long grid = (a.rows + per - 1) / per;
  return launch_kernel(rmsnorm_kernel<TPR, V>, dim3(static_cast<unsigned>(grid)), dim3(threads), 0, s,
                       false, 1, a);
}

}  // namespace

cudaError_t launch_rmsnorm(const RmsNormLaunch& a, cudaStream_t s) {
  const int nvec = a.dim >> 3;
  if (nvec <= 64) return launch<32, 2>(a, s);
  if (nvec <= 512) return launch<128, 4>(a, s);
  if (nvec <= 1024) return launch<256, 4>(a, s);
  if (nvec <= 2048) return launch<512, 4>(a, s);
  return launch<1024, 4>(a, s);
}

}  // namespace dsa
