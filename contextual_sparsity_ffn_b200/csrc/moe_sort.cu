// Tokens sorted by expert, and back.
//
// Sort: a stable counting sort of the R = T k slots by expert.  The slots are cut into chunks; a
// chunk's CTA counts its experts (count kernel), then places its slots (place kernel): a slot's
// position is the number of kept slots of lower experts, plus those of its expert in earlier
// chunks, in earlier warps of the chunk, in earlier rounds of the warp and in lower lanes.  All of
// these are counts, no order of arrival enters, so the result is the stable sort whatever the
// timing.  With one chunk (decode steps) a single kernel does it all: every CTA places the whole
// chunk for itself in shared memory and gathers its own tokens' rows.
//
// Gather: one pass over the tokens: a token's row is read once and written to the positions of its
// slots (d bytes read + k d written, against k d + k d for a gather by position).
//
// Combine: one pass over the tokens: each thread owns 8 columns and adds the token's k rows in slot
// order in fp32, so the sum does not depend on timing (no atomics).
#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace csffn {
namespace {

constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / kWarp;

template <typename... P, typename... A>
cudaError_t launch_chained(void (*kern)(P...), int grid, int block, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// The expert of slot s, or E for slots that are dropped (padding, or past the end).
__device__ __forceinline__ int slot_expert(const DispatchArgs& a, int s, int end) {
  if (s >= end) return a.E;
  const int e = a.ids[s];
  return e >= 0 && e < a.E ? e : a.E;
}

// Slots [lo, hi) of this warp within chunk [c0, c1): contiguous, 32 at a time.
__device__ __forceinline__ void warp_span(int c0, int c1, int warp, int* lo, int* hi) {
  const int per = ((c1 - c0 + kSortWarps - 1) / kSortWarps + kWarp - 1) / kWarp * kWarp;
  *lo = min(c0 + warp * per, c1);
  *hi = min(*lo + per, c1);
}

// whist[w][e] = slots of expert e in warp w's span.
__device__ void count_warps(const DispatchArgs& a, int c0, int c1, int* whist, int warp, int lane) {
  for (int i = threadIdx.x; i < kSortWarps * a.E; i += kSortThreads) whist[i] = 0;
  __syncthreads();
  int lo, hi;
  warp_span(c0, c1, warp, &lo, &hi);
  for (int s0 = lo; s0 < hi; s0 += kWarp) {
    const int e = slot_expert(a, s0 + lane, hi);
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (e < a.E && lane == __ffs(same) - 1) whist[warp * a.E + e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kSortThreads) count_kernel(const DispatchArgs a, int chunk) {
  extern __shared__ int sort_smem[];
  pdl_trigger();
  pdl_wait_prior();
  const int R = a.T * a.k, c0 = blockIdx.x * chunk, c1 = min(R, c0 + chunk);
  count_warps(a, c0, c1, sort_smem, threadIdx.x >> 5, threadIdx.x & 31);
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) n += sort_smem[w * a.E + e];
    a.hist[(size_t)blockIdx.x * a.E + e] = n;
  }
}

// Exclusive prefix sum over experts of tot[0 .. E) in shared memory, in place; returns the sum.
__device__ int scan_experts(int* tot, int E, int* s_sum) {
  __syncthreads();
  if (threadIdx.x < kWarp) {
    int base = 0;
    for (int e0 = 0; e0 < E; e0 += kWarp) {
      const int e = e0 + (int)threadIdx.x;
      const int v = e < E ? tot[e] : 0;
      int x = v;
#pragma unroll
      for (int o = 1; o < kWarp; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if ((int)threadIdx.x >= o) x += y;
      }
      if (e < E) tot[e] = base + x - v;
      base += __shfl_sync(0xffffffffu, x, kWarp - 1);
    }
    if (threadIdx.x == 0) *s_sum = base;
  }
  __syncthreads();
  return *s_sum;
}

// Places this chunk's slots: calls put(slot, position) for every slot, position -1 for a dropped
// one.  `first[e]`: position of the chunk's first slot of expert e.  whist: as count_warps left it.
template <typename Put>
__device__ void place_chunk(const DispatchArgs& a, int c0, int c1, int* whist, const int* first, int warp, int lane,
                            Put put) {
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) {
    int n = first[e];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = whist[w * a.E + e];
      whist[w * a.E + e] = n;
      n += c;
    }
  }
  __syncthreads();
  int lo, hi;
  warp_span(c0, c1, warp, &lo, &hi);
  for (int s0 = lo; s0 < hi; s0 += kWarp) {
    const int s = s0 + lane, e = slot_expert(a, s, hi);
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    const int base = e < a.E ? whist[warp * a.E + e] : 0;
    __syncwarp();
    if (e < a.E && rank == 0) whist[warp * a.E + e] = base + __popc(same);
    __syncwarp();
    if (s < hi) put(s, e < a.E ? base + rank : -1);
  }
}

__global__ void __launch_bounds__(kSortThreads) place_kernel(const DispatchArgs a, int chunk, int n_chunks) {
  extern __shared__ int sort_smem[];
  __shared__ int s_sum;
  int* whist = sort_smem;                // [kSortWarps][E]
  int* tot = whist + kSortWarps * a.E;   // [E] totals, then first positions of the experts
  int* before = tot + a.E;               // [E] slots of the expert in earlier chunks
  pdl_trigger();
  pdl_wait_prior();
  const int R = a.T * a.k, c0 = blockIdx.x * chunk, c1 = min(R, c0 + chunk);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) {
    int all = 0, mine = 0;
    for (int c = 0; c < n_chunks; ++c) {
      if (c == (int)blockIdx.x) mine = all;
      all += __ldcg(a.hist + (size_t)c * a.E + e);
    }
    tot[e] = all;
    before[e] = mine;
  }
  const int kept = scan_experts(tot, a.E, &s_sum);
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e < a.E; e += kSortThreads) a.offsets[e] = tot[e];
    if (threadIdx.x == 0) a.offsets[a.E] = kept;
  }
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) before[e] += tot[e];
  count_warps(a, c0, c1, whist, warp, lane);
  place_chunk(a, c0, c1, whist, before, warp, lane, [&](int s, int p) {
    a.pos[s] = p;
    if (p >= 0) a.order[p] = s;
  });
}

// The rows of token t to its slots' positions, by `n` threads of which this one is number i.
__device__ __forceinline__ void gather_token(const DispatchArgs& a, int t, const int* pos, int i, int n) {
  const uint4* src = reinterpret_cast<const uint4*>(a.x) + (size_t)t * a.row_vecs;
  uint4* dst = reinterpret_cast<uint4*>(a.xs);
  for (int c = i; c < a.row_vecs; c += n) {
    const uint4 v = __ldcg(src + c);
    for (int j = 0; j < a.k; ++j) {
      const int p = pos[j];
      if (p >= 0) dst[(size_t)p * a.row_vecs + c] = v;
    }
  }
}

constexpr int kGatherThreads = 128;

__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const DispatchArgs a, int per_token) {
  __shared__ int s_pos[(kGatherThreads / kWarp) * CSFFN_MAX_TOPK];
  pdl_trigger();
  pdl_wait_prior();
  const int tokens = kGatherThreads / per_token, t0 = blockIdx.x * tokens;
  const int n = min(tokens, a.T - t0) * a.k;
  for (int i = threadIdx.x; i < n; i += kGatherThreads) s_pos[i] = __ldcg(a.pos + (size_t)t0 * a.k + i);
  __syncthreads();
  const int g = threadIdx.x / per_token, t = t0 + g;
  if (t < a.T) gather_token(a, t, s_pos + g * a.k, threadIdx.x % per_token, per_token);
}

// One chunk: every CTA sorts all slots, then gathers its own tokens.
__global__ void __launch_bounds__(kSortThreads) dispatch_small_kernel(const DispatchArgs a, int tokens) {
  extern __shared__ int sort_smem[];
  __shared__ int s_sum;
  __shared__ int s_pos[kMoeChunk];
  int* whist = sort_smem;
  int* tot = whist + kSortWarps * a.E;
  pdl_trigger();
  pdl_wait_prior();
  const int R = a.T * a.k, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  count_warps(a, 0, R, whist, warp, lane);
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) n += whist[w * a.E + e];
    tot[e] = n;
  }
  const int kept = scan_experts(tot, a.E, &s_sum);
  const bool lead = blockIdx.x == 0;
  place_chunk(a, 0, R, whist, tot, warp, lane, [&](int s, int p) {
    s_pos[s] = p;
    if (lead) {
      a.pos[s] = p;
      if (p >= 0) a.order[p] = s;
    }
  });
  if (lead) {
    for (int e = threadIdx.x; e < a.E; e += kSortThreads) a.offsets[e] = tot[e];
    if (threadIdx.x == 0) a.offsets[a.E] = kept;
  }
  __syncthreads();
  const int t0 = blockIdx.x * tokens, t1 = min(a.T, t0 + tokens);
  for (int t = t0; t < t1; ++t) gather_token(a, t, s_pos + t * a.k, threadIdx.x, kSortThreads);
}

// ------------------------------------------------------------------------------------------ back

constexpr int kCombineThreads = 128;

__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const CombineArgs a, int per_token) {
  __shared__ int s_pos[(kCombineThreads / kWarp) * CSFFN_MAX_TOPK];
  __shared__ float s_w[(kCombineThreads / kWarp) * CSFFN_MAX_TOPK];
  pdl_trigger();
  pdl_wait_prior();
  const int tokens = kCombineThreads / per_token, t0 = blockIdx.x * tokens;
  const int n = min(tokens, a.T - t0) * a.k;
  for (int i = threadIdx.x; i < n; i += kCombineThreads) {
    const int p = __ldcg(a.pos + (size_t)t0 * a.k + i);
    s_pos[i] = p >= 0 && p < a.rows ? p : -1;
    s_w[i] = a.weights ? __ldcg(a.weights + (size_t)t0 * a.k + i) : 1.f;
  }
  __syncthreads();
  const int g = threadIdx.x / per_token, t = t0 + g;
  if (t >= a.T) return;
  const int vecs = a.d / 8;
  const uint4* ys = reinterpret_cast<const uint4*>(a.ys);
  for (int c = threadIdx.x % per_token; c < vecs; c += per_token) {
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    for (int j0 = 0; j0 < a.k; j0 += 4) {
      uint4 r[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = j0 + u;
        if (j < a.k && s_pos[g * a.k + j] >= 0)
          r[u] = __ldcg(ys + (size_t)s_pos[g * a.k + j] * vecs + c);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = j0 + u;
        if (j < a.k && s_pos[g * a.k + j] >= 0) {
          const float w = s_w[g * a.k + j];
          float f[8];
          unpack(r[u], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, f[i], acc[i]);
        }
      }
    }
    const size_t o = (size_t)t * a.d + (size_t)c * 8;
    if (a.out_mode == CSFFN_OUT_BF16) {
      __nv_bfloat162 b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = __floats2bfloat162_rn(acc[2 * i], acc[2 * i + 1]);
      *reinterpret_cast<uint4*>(reinterpret_cast<bf16*>(a.out) + o) = *reinterpret_cast<uint4*>(b);
    } else {
      float4* out = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + o);
      float4 lo = make_float4(acc[0], acc[1], acc[2], acc[3]), hi = make_float4(acc[4], acc[5], acc[6], acc[7]);
      if (a.out_mode == CSFFN_OUT_F32_ACCUMULATE) {
        const float4 x = out[0], y = out[1];
        lo = make_float4(x.x + lo.x, x.y + lo.y, x.z + lo.z, x.w + lo.w);
        hi = make_float4(y.x + hi.x, y.y + hi.y, y.z + hi.z, y.w + hi.w);
      }
      out[0] = lo;
      out[1] = hi;
    }
  }
}

// Threads per token: enough for one 16-byte vector each, whole warps, at most `most`.
int token_threads(int vecs, int most) {
  int n = kWarp;
  while (n < vecs && n < most) n *= 2;
  return n;
}

}  // namespace

cudaError_t launch_moe_dispatch(const DispatchArgs& a, cudaStream_t s) {
  const int R = a.T * a.k;
  const int sms = sm_count();
  if (R <= kMoeChunk) {
    const int tokens = (a.T + sms - 1) / sms;
    return launch_chained(dispatch_small_kernel, (a.T + tokens - 1) / tokens, kSortThreads,
                          sizeof(int) * (size_t)(kSortWarps + 1) * a.E, s, a, tokens);
  }
  const int chunk = moe_chunk_slots(R), chunks = moe_chunks(R);
  cudaError_t e = launch_chained(count_kernel, chunks, kSortThreads, sizeof(int) * (size_t)kSortWarps * a.E, s, a, chunk);
  if (e != cudaSuccess) return e;
  e = launch_chained(place_kernel, chunks, kSortThreads, sizeof(int) * (size_t)(kSortWarps + 2) * a.E, s, a, chunk,
                     chunks);
  if (e != cudaSuccess) return e;
  const int per = token_threads(a.row_vecs, kGatherThreads), tokens = kGatherThreads / per;
  return launch_chained(gather_kernel, (a.T + tokens - 1) / tokens, kGatherThreads, 0, s, a, per);
}

cudaError_t launch_moe_combine(const CombineArgs& a, cudaStream_t s) {
  const int per = token_threads(a.d / 8, kCombineThreads), tokens = kCombineThreads / per;
  return launch_chained(combine_kernel, (a.T + tokens - 1) / tokens, kCombineThreads, 0, s, a, per);
}

}  // namespace csffn
