// The norms around a block in one pass over the rows: the norm of the block's output, its gate and
// the residual update, and the norm that feeds the next block.
//
// One row per group of threads, the row in registers: each thread owns 8-element chunks of h, y
// and the gate, all loaded before the first sum.  mean(y^2) is one reduction over the group, h'
// follows in registers, mean(h'^2) is a second one, so h and y are read once and h' and xn written
// once (against a pass per norm and one for the residual).  Bound by memory: 8192 x 4096 with a gate
// per token 81.6 us one after the other in a graph (81.9 at the measured copy rate; 85 to 90 called from
// the host; 85.4 in a graph with two chunks on half the threads); with a gate per channel 73 us (84%).
// Rows of 8192 on 512 threads 83 us for 4096 tokens (on 1024: 113, on 256: 98); rows of 16384 leave one
// or two rows per SM and wait for their sums: 61%.  The next kernel is not let start early (tcgen05.cuh);
// its CTAs would only take the place of rows: 512 rows of 2048, one call after the other, 3.6 us, 4.8
// with the trigger.
#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace csffn {
namespace {

constexpr int kNormRowThreads = 128;  // threads of a CTA, when a row takes fewer

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void load8(const bf16* p, float (&f)[8]) { unpack(*reinterpret_cast<const uint4*>(p), f); }
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(bf16* p, const float (&f)[8]) {
  __nv_bfloat162 b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<uint4*>(b);
}

// Sum over the TPR threads of a row (whole warps).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* part, int row_in_cta) {
  v = warp_sum(v);
  if constexpr (TPR > kWarp) {
    constexpr int W = TPR / kWarp;
    const int w = (threadIdx.x >> 5) % W;
    if ((threadIdx.x & 31) == 0) part[row_in_cta * W + w] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) v += part[row_in_cta * W + i];
  }
  return v;
}

template <typename Y, typename X, int TPR, int C>  // TPR threads per row, C chunks of 8 per thread
__global__ void __launch_bounds__(TPR < kNormRowThreads ? kNormRowThreads : TPR) block_norm_kernel(const BlockNormArgs a) {
  constexpr int kRows = TPR < kNormRowThreads ? kNormRowThreads / TPR : 1;
  __shared__ float part[2][kRows * (TPR / kWarp)];
  pdl_wait_prior();  // and no trigger: xn and h_out may be weights of the call that follows
  const int r = threadIdx.x / TPR, i = threadIdx.x % TPR;
  const int t = blockIdx.x * kRows + r;
  const bool live = t < a.T;
  const int d = a.d, chunks = d / 8;
  const size_t row = (size_t)t * d;
  float h[C][8], u[C][8], g[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int q = i + c * TPR;
    if (live && q < chunks) {
      load8(a.h + row + q * 8, h[c]);
      if (a.y) load8(reinterpret_cast<const Y*>(a.y) + row + q * 8, u[c]);
      if (a.gate) load8(a.gate + (a.gate_per_token ? row : 0) + q * 8, g[c]);
    }
  }
  float ry = 1.f;
  if (a.g_post) {  // uniform over the grid
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (live && i + c * TPR < chunks) {
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(u[c][e], u[c][e], ss);
      }
    ry = 1.0f / sqrtf(row_sum<TPR>(ss, part[0], r) / (float)d + a.eps);
  }
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int q = i + c * TPR;
    if (live && q < chunks) {
      if (a.y) {
        if (a.g_post) {
          float p[8];
          load8(a.g_post + q * 8, p);
#pragma unroll
          for (int e = 0; e < 8; ++e) u[c][e] = u[c][e] * ry * p[e];
        }
        if (a.gate) {
#pragma unroll
          for (int e = 0; e < 8; ++e) u[c][e] *= g[c][e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) h[c][e] = fmaf(a.out_scale, u[c][e], a.res_scale * h[c][e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[c][e] *= a.res_scale;
      }
      if (a.h_out) store8(a.h_out + row + q * 8, h[c]);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(h[c][e], h[c][e], ss);
    }
  }
  if (!a.xn) return;
  const float rh = 1.0f / sqrtf(row_sum<TPR>(ss, part[1], r) / (float)d + a.eps);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int q = i + c * TPR;
    if (live && q < chunks) {
      float p[8];
      if (a.g_pre) load8(a.g_pre + q * 8, p);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[c][e] = a.g_pre ? h[c][e] * rh * p[e] : h[c][e] * rh;
      store8(reinterpret_cast<X*>(a.xn) + row + q * 8, h[c]);
    }
  }
}

template <typename Y, typename X, int TPR, int C>
cudaError_t launch_norm_t(const BlockNormArgs& a, cudaStream_t s) {
  constexpr int kRows = TPR < kNormRowThreads ? kNormRowThreads / TPR : 1;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.T + kRows - 1) / kRows));
  cfg.blockDim = dim3(TPR < kNormRowThreads ? kNormRowThreads : TPR);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_norm_kernel<Y, X, TPR, C>, a);
}

template <typename Y, typename X>
cudaError_t launch_norm_d(const BlockNormArgs& a, cudaStream_t s) {
  const int chunks = a.d / 8;
  if (chunks <= 32) return launch_norm_t<Y, X, 32, 1>(a, s);
  if (chunks <= 64) return launch_norm_t<Y, X, 64, 1>(a, s);
  if (chunks <= 128) return launch_norm_t<Y, X, 128, 1>(a, s);
  if (chunks <= 256) return launch_norm_t<Y, X, 256, 1>(a, s);
  if (chunks <= 512) return launch_norm_t<Y, X, 512, 1>(a, s);
  if (chunks <= 1024) return launch_norm_t<Y, X, 512, 2>(a, s);
  return launch_norm_t<Y, X, 1024, 2>(a, s);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& a, int ydtype, int xdtype, cudaStream_t s) {
  if (ydtype == CSFFN_BF16)
    return xdtype == CSFFN_BF16 ? launch_norm_d<bf16, bf16>(a, s) : launch_norm_d<bf16, float>(a, s);
  return xdtype == CSFFN_BF16 ? launch_norm_d<float, bf16>(a, s) : launch_norm_d<float, float>(a, s);
}

}  // namespace csffn
