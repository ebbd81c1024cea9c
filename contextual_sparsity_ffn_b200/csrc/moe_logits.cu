// Router projection.
//
// Plain tiled kernels: a CTA of 256 threads computes a tile of 64 rows x 64 outputs of one expert,
// 4 x 4 outputs per thread, the contraction in steps of 32 through shared memory, fp32 FMA.
#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace csffn {
namespace {

constexpr int kT = 64, kK = 32, kThreads = 256;

enum { kGateUp = 0, kDown = 1, kLogits = 2 };

struct TileArgs {
  const bf16* a;        // rows [n, K]
  const bf16* w0;       // [E, N, K] (gate, router) or [E, K, N] (down)
  const bf16* w1;       // up
  const int32_t* offsets;  // NULL: one group of n rows
  int n, N, K, E, act;
  void* out;            // [n, N]
};

template <int MODE>
__global__ void __launch_bounds__(kThreads) tile_kernel(const TileArgs p) {
  __shared__ float sa[kT][kK + 1], s0[kT][kK + 1], s1[MODE == kGateUp ? kT : 1][kK + 1];
  pdl_trigger();
  pdl_wait_prior();
  // this row tile's expert and rows
  int e = 0, r0 = 0, r1 = 0, left = blockIdx.y;
  bool found = false;
  int lo = 0;
  for (e = 0; e < p.E; ++e) {
    int hi = p.n;
    if (p.offsets) {
      if (e == 0) lo = min(max(p.offsets[0], 0), p.n);
      hi = max(lo, min(max(p.offsets[e + 1], 0), p.n));
    }
    const int tiles = (hi - lo + kT - 1) / kT;
    if (left < tiles) {
      r0 = lo + left * kT;
      r1 = min(hi, r0 + kT);
      found = true;
      break;
    }
    left -= tiles;
    lo = hi;
  }
  if (!found) return;
  const int c0 = blockIdx.x * kT;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const size_t wbase = (size_t)e * p.N * p.K;
  float acc0[4][4] = {}, acc1[4][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += kK) {
    for (int i = threadIdx.x; i < kT * kK; i += kThreads) {
      const int r = i / kK, k = i % kK;
      sa[r][k] = r0 + r < r1 && k0 + k < p.K ? __bfloat162float(p.a[(size_t)(r0 + r) * p.K + k0 + k]) : 0.f;
      if (MODE == kDown) {
        const int kk = i / kT, c = i % kT;
        s0[c][kk] = c0 + c < p.N && k0 + kk < p.K ? __bfloat162float(p.w0[wbase + (size_t)(k0 + kk) * p.N + c0 + c]) : 0.f;
      } else {
        const bool in = c0 + r < p.N && k0 + k < p.K;
        s0[r][k] = in ? __bfloat162float(p.w0[wbase + (size_t)(c0 + r) * p.K + k0 + k]) : 0.f;
        if (MODE == kGateUp) s1[r][k] = in ? __bfloat162float(p.w1[wbase + (size_t)(c0 + r) * p.K + k0 + k]) : 0.f;
      }
    }
    __syncthreads();
#pragma unroll 8
    for (int k = 0; k < kK; ++k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = sa[ty + 16 * i][k];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc0[i][j] = fmaf(x, s0[tx + 16 * j][k], acc0[i][j]);
          if (MODE == kGateUp) acc1[i][j] = fmaf(x, s1[tx + 16 * j][k], acc1[i][j]);
        }
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + ty + 16 * i;
    if (r >= r1) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + tx + 16 * j;
      if (c >= p.N) continue;
      const size_t o = (size_t)r * p.N + c;
      if (MODE == kLogits)
        reinterpret_cast<float*>(p.out)[o] = acc0[i][j];
      else if (MODE == kDown)
        reinterpret_cast<bf16*>(p.out)[o] = __float2bfloat16_rn(acc0[i][j]);
      else
        reinterpret_cast<bf16*>(p.out)[o] = __float2bfloat16_rn(gate_act(acc0[i][j], p.act) * acc1[i][j]);
    }
  }
}

template <int MODE>
cudaError_t launch_tiles(const TileArgs& p, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // an expert's last tile may be ragged: at most one tile more per expert that has rows
  const int row_tiles = (p.n + kT - 1) / kT + (p.offsets ? (p.E < p.n ? p.E : p.n) : 0);
  cfg.gridDim = dim3((unsigned)((p.N + kT - 1) / kT), (unsigned)row_tiles);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tile_kernel<MODE>, p);
}

}  // namespace

cudaError_t launch_moe_logits(const void* x, const void* w, int T, int E, int d, float* logits, cudaStream_t s) {
  const TileArgs p{static_cast<const bf16*>(x), static_cast<const bf16*>(w), nullptr, nullptr, T, E, d, 1, 0, logits};
  return launch_tiles<kLogits>(p, s);
}

}  // namespace csffn
