// Tokens sorted by expert, and back.
//
// Sort: a stable counting sort of the R = T k slots by expert.  The slots are cut into chunks; a
// chunk's CTA counts its experts (count kernel), then places its slots (place kernel): a slot's
// position is the number of kept slots of lower experts, plus those of its expert in earlier
// chunks, in earlier warps of the chunk, in earlier rounds of the warp and in lower lanes.  All of
// these are counts, no order of arrival enters, so the result is the stable sort whatever the
// timing.  With one chunk (decode steps) a single kernel does it all: every CTA places the whole
// chunk for itself in shared memory and gathers its own tokens' rows.  With a few chunks one cluster
// does both steps.
//
// Gather: one pass over the tokens: a token's row is read once and written to the positions of its
// slots (d bytes read + k d written, against k d + k d for a gather by position).  8192 tokens x 8 of
// 64 experts, d 2048 bf16: the three kernels 60 us with random experts (46 at the copy rate), 53 where
// every token has the same ones and an eighth has none, of which the gather is 43 (41); 13 tokens in the
// one kernel: 3.4 us, the latency of its chain of loads, counts and stores.
//
// The kernels that write rows (xs, out) do not let the next kernel start early: the rows may be weights
// of the call that follows (tcgen05.cuh).  It costs nothing: combine, 512 tokens, call after call 4.6 us
// (6.2 with the trigger, whose waiting CTAs take the place of working ones).
//
// Combine: one pass over the tokens: each thread owns 8 columns and adds the token's k rows in slot
// order in fp32, so the sum does not depend on timing (no atomics).  Bound by memory: the same
// tokens 49.5 us (46 at the copy rate), with an eighth of none 45 (41).
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

// The functions below work for a CTA of THREADS threads; ROUNDS: rounds of 32 slots per warp and batch.
constexpr int kRounds = kMoeChunk / kSortThreads;

// This warp's slots of chunk [c0, c1) from round r0 on: lane's slot in round r is *first + 32 r, and its
// expert ex[r], or E for slots that are dropped (padding, or past the chunk).  All loads go out at
// once.
template <int THREADS, int ROUNDS>
__device__ __forceinline__ void load_slots(const DispatchArgs& a, int c0, int c1, int warp, int lane, int r0,
                                           int (&ex)[ROUNDS], int* first) {
  const int per = (c1 - c0 + THREADS - 1) / THREADS * kWarp;  // slots of a warp
  const int lo = c0 + warp * per, hi = min(lo + per, c1);
  *first = lo + r0 * kWarp + lane;
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int s = *first + r * kWarp;
    ex[r] = s < hi ? __ldcg(a.ids + s) : -1;
  }
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) ex[r] = ex[r] >= 0 && ex[r] < a.E ? ex[r] : a.E;
}
// Rounds of a chunk: whole batches.
template <int THREADS, int ROUNDS>
__device__ __forceinline__ int chunk_rounds(int c0, int c1) {
  return ((c1 - c0 + THREADS - 1) / THREADS + ROUNDS - 1) / ROUNDS * ROUNDS;
}

// whist[w][e] = slots of expert e in warp w's share of the chunk.  `ex` holds the first batch.
template <int THREADS, int ROUNDS>
__device__ void count_warps(const DispatchArgs& a, int c0, int c1, int* whist, int warp, int lane, int (&ex)[ROUNDS]) {
  for (int i = threadIdx.x; i < THREADS / kWarp * a.E; i += THREADS) whist[i] = 0;
  __syncthreads();
  for (int r0 = 0; r0 < chunk_rounds<THREADS, ROUNDS>(c0, c1); r0 += ROUNDS) {
    int first;
    if (r0 > 0) load_slots<THREADS, ROUNDS>(a, c0, c1, warp, lane, r0, ex, &first);
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      const uint32_t same = __match_any_sync(0xffffffffu, ex[r]);
      if (ex[r] < a.E && lane == __ffs(same) - 1) whist[warp * a.E + ex[r]] += __popc(same);
      __syncwarp();
    }
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kSortThreads) count_kernel(const DispatchArgs a, int chunk) {
  extern __shared__ int sort_smem[];
  pdl_trigger();
  pdl_wait_prior();
  const int R = a.T * a.k, c0 = blockIdx.x * chunk, c1 = min(R, c0 + chunk);
  int ex[kRounds], first;
  load_slots<kSortThreads, kRounds>(a, c0, c1, threadIdx.x >> 5, threadIdx.x & 31, 0, ex, &first);
  count_warps<kSortThreads, kRounds>(a, c0, c1, sort_smem, threadIdx.x >> 5, threadIdx.x & 31, ex);
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
// one.  `start[e]`: position of the chunk's first slot of expert e.  whist: as count_warps left it;
// `ex`: the batch that it read last.
template <int THREADS, int ROUNDS, typename Put>
__device__ void place_chunk(const DispatchArgs& a, int c0, int c1, int* whist, const int* start, int warp, int lane,
                            int (&ex)[ROUNDS], Put put) {
  for (int e = threadIdx.x; e < a.E; e += THREADS) {
    int n = start[e];
#pragma unroll 8
    for (int w = 0; w < THREADS / kWarp; ++w) {
      const int c = whist[w * a.E + e];
      whist[w * a.E + e] = n;
      n += c;
    }
  }
  __syncthreads();
  const int per = (c1 - c0 + THREADS - 1) / THREADS * kWarp;
  const int hi = min(c0 + (warp + 1) * per, c1);
  const int rounds = chunk_rounds<THREADS, ROUNDS>(c0, c1);
  for (int r0 = 0; r0 < rounds; r0 += ROUNDS) {
    int first = c0 + warp * per + lane;
    if (rounds > ROUNDS) load_slots<THREADS, ROUNDS>(a, c0, c1, warp, lane, r0, ex, &first);
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      const int s = first + r * kWarp, e = ex[r];
      const uint32_t same = __match_any_sync(0xffffffffu, e);
      const int rank = __popc(same & ((1u << lane) - 1u));
      const int base = e < a.E ? whist[warp * a.E + e] : 0;
      __syncwarp();
      if (e < a.E && rank == 0) whist[warp * a.E + e] = base + __popc(same);
      __syncwarp();
      if (s < hi) put(s, e < a.E ? base + rank : -1);
    }
  }
}

// Up to 16384 slots one cluster of 8 CTAs plans them in one kernel, a chunk each; the CTAs read each
// other's counts from shared memory.  4000 slots: 7.8 us with the gather (9.5 with the two kernels),
// 16384 slots 20.9 (21.1); 65536 slots would take 25.7 (15.5), too few CTAs.
constexpr int kPlanCtas = 8, kPlanThreads = 1024, kPlanRounds = 2;
constexpr int kPlanMaxSlots = kPlanCtas * kPlanThreads * kPlanRounds;

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const DispatchArgs a) {
  extern __shared__ int sort_smem[];
  __shared__ int s_sum;
  int* whist = sort_smem;                            // [warps][E]
  int* tot = whist + kPlanThreads / kWarp * a.E;     // [E] totals, then first positions of the experts
  int* before = tot + a.E;                           // [E] slots of the expert in earlier chunks
  int* mine = before + a.E;                          // [E] slots of the expert in this chunk
  pdl_trigger();
  pdl_wait_prior();
  const int R = a.T * a.k, chunk = (R + kPlanCtas - 1) / kPlanCtas, rank = (int)cluster_rank();
  const int c0 = min(R, rank * chunk), c1 = min(R, c0 + chunk);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int ex[kPlanRounds], first;
  load_slots<kPlanThreads, kPlanRounds>(a, c0, c1, warp, lane, 0, ex, &first);
  count_warps<kPlanThreads, kPlanRounds>(a, c0, c1, whist, warp, lane, ex);
  for (int e = threadIdx.x; e < a.E; e += kPlanThreads) {
    int n = 0;
#pragma unroll 8
    for (int w = 0; w < kPlanThreads / kWarp; ++w) n += whist[w * a.E + e];
    mine[e] = n;
  }
  cluster_sync_all();
  for (int e = threadIdx.x; e < a.E; e += kPlanThreads) {
    int all = 0, low = 0;
#pragma unroll
    for (int q = 0; q < kPlanCtas; ++q) {
      int n;
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(n) : "r"(map_to_rank(mine + e, (uint32_t)q)) : "memory");
      all += n;
      if (q < rank) low += n;
    }
    tot[e] = all;
    before[e] = low;
  }
  cluster_arrive_all();  // done with the other CTAs' shared memory
  const int kept = scan_experts(tot, a.E, &s_sum);
  if (rank == 0) {
    for (int e = threadIdx.x; e < a.E; e += kPlanThreads) a.offsets[e] = tot[e];
    if (threadIdx.x == 0) a.offsets[a.E] = kept;
  }
  for (int e = threadIdx.x; e < a.E; e += kPlanThreads) before[e] += tot[e];
  __syncthreads();
  place_chunk<kPlanThreads, kPlanRounds>(a, c0, c1, whist, before, warp, lane, ex, [&](int s, int p) {
    a.pos[s] = p;
    if (p >= 0) a.order[p] = s;
  });
  cluster_wait_all();
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
  int ex[kRounds], first;
  load_slots<kSortThreads, kRounds>(a, c0, c1, warp, lane, 0, ex, &first);
  for (int e = threadIdx.x; e < 2 * a.E; e += kSortThreads) tot[e] = 0;  // and `before`
  __syncthreads();
  // The chunks' counts, added by groups of threads with a share of the chunks each (integers: the
  // order of the additions does not matter).
  const int wide = min(a.E, kSortThreads), groups = kSortThreads / wide, g = threadIdx.x / wide;
  if (g < groups) {
    const int lo = g * n_chunks / groups, hi = (g + 1) * n_chunks / groups;
    for (int e = threadIdx.x % wide; e < a.E; e += wide) {
      int all = 0, mine = 0;
      for (int q = lo; q < hi; q += 8) {
        int n[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) n[u] = q + u < hi ? __ldcg(a.hist + (size_t)(q + u) * a.E + e) : 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          all += n[u];
          if (q + u < (int)blockIdx.x) mine += n[u];
        }
      }
      atomicAdd(&tot[e], all);
      atomicAdd(&before[e], mine);
    }
  }
  const int kept = scan_experts(tot, a.E, &s_sum);
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e < a.E; e += kSortThreads) a.offsets[e] = tot[e];
    if (threadIdx.x == 0) a.offsets[a.E] = kept;
  }
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) before[e] += tot[e];
  count_warps<kSortThreads, kRounds>(a, c0, c1, whist, warp, lane, ex);
  place_chunk<kSortThreads, kRounds>(a, c0, c1, whist, before, warp, lane, ex, [&](int s, int p) {
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
  pdl_wait_prior();
  const int R = a.T * a.k, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int ex[kRounds], first;
  load_slots<kSortThreads, kRounds>(a, 0, R, warp, lane, 0, ex, &first);
  count_warps<kSortThreads, kRounds>(a, 0, R, whist, warp, lane, ex);
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) n += whist[w * a.E + e];
    tot[e] = n;
  }
  const int kept = scan_experts(tot, a.E, &s_sum);
  const bool lead = blockIdx.x == 0;
  place_chunk<kSortThreads, kRounds>(a, 0, R, whist, tot, warp, lane, ex, [&](int s, int p) {
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

cudaError_t launch_plan(const DispatchArgs& a, cudaStream_t s) {
  const size_t smem = sizeof(int) * (size_t)(kPlanThreads / kWarp + 3) * a.E;
  cudaError_t e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kPlanCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPlanCtas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, plan_kernel, a);
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
  cudaError_t e;
  if (R <= kPlanMaxSlots) {
    if ((e = launch_plan(a, s)) != cudaSuccess) return e;
  } else {
    const int chunk = moe_chunk_slots(R), chunks = moe_chunks(R);
    e = launch_chained(count_kernel, chunks, kSortThreads, sizeof(int) * (size_t)kSortWarps * a.E, s, a, chunk);
    if (e != cudaSuccess) return e;
    e = launch_chained(place_kernel, chunks, kSortThreads, sizeof(int) * (size_t)(kSortWarps + 2) * a.E, s, a, chunk, chunks);
    if (e != cudaSuccess) return e;
  }
  const int per = token_threads(a.row_vecs, kGatherThreads), tokens = kGatherThreads / per;
  return launch_chained(gather_kernel, (a.T + tokens - 1) / tokens, kGatherThreads, 0, s, a, per);
}

cudaError_t launch_moe_combine(const CombineArgs& a, cudaStream_t s) {
  const int per = token_threads(a.d / 8, kCombineThreads), tokens = kCombineThreads / per;
  return launch_chained(combine_kernel, (a.T + tokens - 1) / tokens, kCombineThreads, 0, s, a, per);
}

}  // namespace csffn
