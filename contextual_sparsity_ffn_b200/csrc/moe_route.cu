// Router selection: the k experts of every token and their weights.
//
// One warp per token; lane l holds the keys of experts l, l + 32, ... in registers (up to 16 of
// them).  The keys are mapped to 32-bit integers of the same order, so one round of the selection
// is a maximum over the lane's keys, one warp-wide integer maximum (redux) and one warp-wide
// minimum over the lanes' lowest expert that holds it: the largest key, equal keys by the lower
// expert, exactly.  Bound by issuing instructions (the schedulers issue in 75% of the cycles; 16384
// tokens x 160 experts, 6 chosen: 10.9 us; a lane that keeps its own maximum and looks again only
// when it loses it took 11.9).  0 stands for a key that is never selected (-inf, NaN, already taken).
// The weights follow the selected logits: lane j takes slot j, and the softmax's maximum and sum
// are warp reductions in fp32.
#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace csffn {
namespace {

constexpr int kRouteWarps = 4;

__device__ __forceinline__ float load_logit(const float* p, size_t i) { return p[i]; }
__device__ __forceinline__ float load_logit(const bf16* p, size_t i) { return __bfloat162float(p[i]); }

// Order-preserving integer of a key; 0 for -inf and NaN.  Adding +0 turns -0 into +0, so the two
// zeros are equal keys.
__device__ __forceinline__ uint32_t key_order(float key) {
  const uint32_t u = __float_as_uint(key + 0.0f);
  const uint32_t o = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return key > -INFINITY ? o : 0u;  // false for NaN too
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// exp(l - m) with the limits a softmax wants: 1 where l is the maximum (also when both are +inf),
// 0 for -inf and NaN.
__device__ __forceinline__ float softmax_term(float l, float m) {
  return l == m ? 1.f : l > -INFINITY ? expf(l - m) : 0.f;
}

template <typename T, int PER>  // PER keys per lane: E <= 32 * PER
__global__ void __launch_bounds__(kRouteWarps * kWarp) route_kernel(const RouteArgs a) {
  pdl_trigger();
  pdl_wait_prior();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const T* row = reinterpret_cast<const T*>(a.logits) + (size_t)t * a.E;
  float l[PER];
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + kWarp * i;
    l[i] = e < a.E ? load_logit(row, e) : -INFINITY;
    key[i] = e < a.E ? key_order(a.bias ? l[i] + a.bias[e] : l[i]) : 0u;
  }
  int mine = -1;  // lane j: the expert of slot j
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = 0u;
#pragma unroll
    for (int i = 0; i < PER; ++i) best = max(best, key[i]);
    best = __reduce_max_sync(0xffffffffu, best);
    if (best == 0u) break;  // no expert is left
    uint32_t e = 0xffffffffu;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i)
      if (key[i] == best) e = (uint32_t)(lane + kWarp * i);
    e = __reduce_min_sync(0xffffffffu, e);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (e == (uint32_t)(lane + kWarp * i)) key[i] = 0u;
    if (lane == j) mine = (int)e;
  }
  const float sel = mine >= 0 ? load_logit(row, mine) : -INFINITY;
  float w = 0.f;
  if (a.score == CSFFN_ROUTE_SIGMOID) {
    w = mine >= 0 ? 1.f / (1.f + expf(-sel)) : 0.f;
    if (a.renorm) w = w / fmaxf(warp_sum(w), 1e-20f);
  } else if (a.renorm) {
    const float m = warp_max(sel);
    w = mine >= 0 ? softmax_term(sel, m) : 0.f;
    w = w / fmaxf(warp_sum(w), 1e-20f);
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) m = fmaxf(m, l[i]);  // fmaxf drops NaN
    m = warp_max(m);
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) z += l[i] > -INFINITY ? softmax_term(l[i], m) : 0.f;
    z = warp_sum(z);
    w = mine >= 0 ? softmax_term(sel, m) / fmaxf(z, 1e-20f) : 0.f;
  }
  if (lane < a.k) {
    a.ids[(size_t)t * a.k + lane] = mine;
    a.weights[(size_t)t * a.k + lane] = mine >= 0 ? w * a.scale : 0.f;
  }
}

template <typename T, int PER>
cudaError_t launch_route_t(const RouteArgs& a, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.T + kRouteWarps - 1) / kRouteWarps));
  cfg.blockDim = dim3(kRouteWarps * kWarp);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, route_kernel<T, PER>, a);
}

template <typename T>
cudaError_t launch_route_e(const RouteArgs& a, cudaStream_t s) {
  switch ((a.E + kWarp - 1) / kWarp) {
    case 1: return launch_route_t<T, 1>(a, s);
    case 2: return launch_route_t<T, 2>(a, s);
    case 3: return launch_route_t<T, 3>(a, s);
    case 4: return launch_route_t<T, 4>(a, s);
    case 5: return launch_route_t<T, 5>(a, s);
    case 6: return launch_route_t<T, 6>(a, s);
    case 7:
    case 8: return launch_route_t<T, 8>(a, s);
    case 9:
    case 10:
    case 11:
    case 12: return launch_route_t<T, 12>(a, s);
    default: return launch_route_t<T, 16>(a, s);
  }
}

}  // namespace

cudaError_t launch_moe_route(const RouteArgs& a, int ldtype, cudaStream_t s) {
  return ldtype == CSFFN_BF16 ? launch_route_e<bf16>(a, s) : launch_route_e<float>(a, s);
}

}  // namespace csffn
