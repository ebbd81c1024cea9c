// Router projection: logits[t, e] = sum_c x[t, c] w_router[e, c].
//
// Few tokens (row_kernel): a CTA per expert and group of 8 tokens.  Its 8 warps share the row of the
// weights, each lane a few 16-byte vectors of it, and multiply them with the tokens' vectors in fp32
// FMA; one sum over the warp and one over the CTA.  Bound by latency: one round of loads.
//
// More tokens (tile_kernel), on the tensor cores: a tile is 128 tokens (M) x up to 128 experts (N),
// and a cluster of S CTAs shares it along the contraction, so that a prompt of any length puts a CTA
// or two on every SM and the weights are read S times less often per SM.  Operands by TMA (128-byte
// swizzle, 64 contraction elements a stage), fp32 accumulators in TMEM; the k-steps alternate between
// two accumulators, and each CTA has 1/S of the steps: the tensor core cuts the running sum after
// every step, so short chains keep the fp32 result.  The CTAs put their parts into shared memory,
// and each adds one S-th of the tokens over the cluster, in the CTAs' order, and writes it.  8192
// tokens x 128 experts, d 4096: 20 us, 11 at the copy rate; the operands' way through L2 (each CTA
// reads its share of the weights, as many bytes as of x) and the cluster's sum are the rest.  Every
// wait is bounded (one second); there is no workspace to record one that ran out, so its tile's
// logits become NaN.
//
// Both kernels read the router weights after the dependency wait only, as they do x: the weights may
// be another call's output (a router normalised per call by csffn_block_norm).  Fetching them before it
// would gain next to nothing: 16 tokens x 128 experts 4.0 us against 4.1, 8192 tokens the same.
#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace csffn {
namespace {

// ------------------------------------------------------------------------------------ few tokens

constexpr int kRowThreads = 256, kRowTokens = 8;

__global__ void __launch_bounds__(kRowThreads) row_kernel(const bf16* x, const bf16* w, int T, int E, int d,
                                                          float* logits) {
  __shared__ float part[kRowThreads / kWarp][kRowTokens];
  pdl_trigger();
  const int e = blockIdx.x, t0 = blockIdx.y * kRowTokens, n = min(kRowTokens, T - t0);
  const int vecs = d / 8;
  const uint4* wr = reinterpret_cast<const uint4*>(w) + (size_t)e * vecs;
  const uint4* xr = reinterpret_cast<const uint4*>(x) + (size_t)t0 * vecs;
  float acc[kRowTokens] = {};
  uint4 wv = make_uint4(0u, 0u, 0u, 0u);
  pdl_wait_prior();
  if ((int)threadIdx.x < vecs) wv = __ldcg(wr + threadIdx.x);
  for (int v = threadIdx.x; v < vecs; v += kRowThreads) {
    const uint4 cur = wv;
    if (v + kRowThreads < vecs) wv = __ldcg(wr + v + kRowThreads);
    uint4 xv[kRowTokens];
#pragma unroll
    for (int t = 0; t < kRowTokens; ++t)
      if (t < n) xv[t] = __ldcg(xr + (size_t)t * vecs + v);
    float wf[8];
    unpack(cur, wf);
#pragma unroll
    for (int t = 0; t < kRowTokens; ++t) {
      if (t < n) {
        float xf[8];
        unpack(xv[t], xf);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[t] = fmaf(wf[i], xf[i], acc[t]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < kRowTokens; ++t) acc[t] = warp_sum(acc[t]);
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int t = 0; t < kRowTokens; ++t) part[threadIdx.x >> 5][t] = acc[t];
  }
  __syncthreads();
  if ((int)threadIdx.x < n) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kRowThreads / kWarp; ++i) s += part[i][threadIdx.x];
    logits[(size_t)(t0 + threadIdx.x) * E + e] = s;
  }
}

// ------------------------------------------------------------------------------------ more tokens

constexpr int kThreads = 192;
constexpr int kM = 128, kMaxN = 128, kKB = 64;
constexpr int kStages = 3;
constexpr uint32_t kXBytes = kM * kKB * 2, kWBytes = kMaxN * kKB * 2, kStage = kXBytes + kWBytes;
constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
constexpr int kMaxSplit = 8;
static_assert(kM * (kMaxN + 4) * 4 <= kStages * kStage, "a tile's part fits where the stages were");

__device__ __forceinline__ float4 load_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__global__ void __launch_bounds__(kThreads)
    tile_kernel(int T, int E, int d, float* logits, int split,
                const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w) {
  extern __shared__ __align__(1024) unsigned char lg_raw[];
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], accf;
  __shared__ uint32_t s_tmem, s_err;
  __shared__ int s_abort;
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(lg_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank(), t0 = (int)(blockIdx.x / split) * kM, e0 = (int)blockIdx.y * kMaxN;
  const int n = (min(kMaxN, E - e0) + 15) / 16 * 16;
  const int n_kb = (d + kKB - 1) / kKB;
  const int kb0 = rank * n_kb / split, kb1 = (rank + 1) * n_kb / split;

  pdl_trigger();
  if (threadIdx.x == 0) {
    s_abort = 0;
    s_err = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&accf, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, 2 * kMaxN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // Before anything is read (and written: the logits may still be read by what came before), and before
  // a bounded wait could count the time of the kernels before this one.
  pdl_wait_prior();

  if (warp == 0) {
    if (lane == 0) {
      // ---- producer
      int issued = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++issued) {
        const int slot = issued % kStages;
        unsigned char* st = smem + (size_t)slot * kStage;
        if (issued >= kStages && !mbar_wait(&empty[slot], (uint32_t)(issued / kStages - 1) & 1, &s_err, &s_abort)) break;
        mbar_arrive_expect_tx(&full[slot], kStage);
        tma_load_2d_plain(st + kXBytes, &tm_w, kb * kKB, e0, &full[slot]);
        tma_load_2d_plain(st, &tm_x, kb * kKB, t0, &full[slot]);
      }
      for (int q = issued > kStages ? issued - kStages : 0; q < issued; ++q)
        mbar_wait_drain(&full[q % kStages], (uint32_t)(q / kStages) & 1, &s_err);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---- MMA issuer
      const uint32_t idesc = umma_idesc_bf16(kM, n, false);
      for (int kb = kb0, i = 0; kb < kb1; ++kb, ++i) {
        const int slot = i % kStages;
        if (!mbar_wait(&full[slot], (uint32_t)(i / kStages) & 1, &s_err, &s_abort)) break;
        tc_fence_after();
        const uint32_t sb = smem_u32(smem + (size_t)slot * kStage);
#pragma unroll
        for (int k = 0; k < kKB / 16; ++k)
          umma_bf16(tmem + (uint32_t)(kMaxN * (k & 1)), umma_desc_k(sb + 32u * k), umma_desc_k(sb + kXBytes + 32u * k),
                    idesc, (i > 0 || k > 1) ? 1u : 0u);
        umma_commit(&empty[slot]);
      }
      umma_commit(&accf);
      mbar_wait_drain(&accf, 0, &s_err);
    }
  }
  __syncthreads();  // every copy has landed and every MMA is done: the stages' memory is free
  tc_fence_after();
  const int stride = n + 4;  // floats per token: vectors of 32 lanes' rows fall on different banks
  if (warp >= 2) {
    const int row = 32 * (warp & 3) + lane;
    const uint32_t acc = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    float* mine = reinterpret_cast<float*>(smem) + row * stride;
    for (int c = 0; c < n; c += 16) {
      float a[16], b[16];
      __syncwarp();
      tmem_ld16(acc + (uint32_t)c, a);
      tmem_ld16(acc + (uint32_t)(kMaxN + c), b);
      tmem_ld_wait(a);
      tmem_ld_wait(b);
      if (s_err) {  // a wait ran out: no logits
#pragma unroll
        for (int k = 0; k < 16; ++k) a[k] = __int_as_float(0x7fc00000);
      }
#pragma unroll
      for (int k = 0; k < 16; k += 4)
        *reinterpret_cast<float4*>(mine + c + k) =
            make_float4(a[k] + b[k], a[k + 1] + b[k + 1], a[k + 2] + b[k + 2], a[k + 3] + b[k + 3]);
    }
    tc_fence_before();
  }
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * kMaxN);
  }
  // this CTA's share of the tokens
  const int r0 = rank * kM / split, r1 = (rank + 1) * kM / split, vecs = n / 4, width = min(kMaxN, E - e0);
  uint32_t base[kMaxSplit];
#pragma unroll
  for (int q = 0; q < kMaxSplit; ++q) base[q] = map_to_rank(smem, (uint32_t)min(q, split - 1));
  for (int i = threadIdx.x; i < (r1 - r0) * vecs; i += kThreads) {
    const int row = r0 + i / vecs, c = i % vecs * 4;
    const uint32_t off = (uint32_t)(row * stride + c) * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int q = 0; q < kMaxSplit; ++q) {
      if (q < split) {
        const float4 v = load_cluster(base[q] + off);
        s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
      }
    }
    if (t0 + row < T) {
      float* out = logits + (size_t)(t0 + row) * E + e0 + c;
      const float f[4] = {s.x, s.y, s.z, s.w};
      if ((E & 3) == 0 && (reinterpret_cast<uintptr_t>(logits) & 15) == 0) {
        if (c < width) *reinterpret_cast<float4*>(out) = s;
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (c + k < width) out[k] = f[k];
      }
    }
  }
  cluster_sync_all();  // no CTA leaves while another reads its part
}

bool encode_rows(CUtensorMap* tm, const void* base, int rows, int width, cuuint32_t high) {
  TensorMapEncodeFn fn = tensor_map_encoder();
  const cuuint64_t dim[2] = {(cuuint64_t)width, (cuuint64_t)rows};
  const cuuint64_t stride[1] = {(cuuint64_t)width * 2};
  const cuuint32_t box[2] = {kKB, high};
  const cuuint32_t ones[2] = {1, 1};
  return fn && fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dim, stride, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// Tokens up to which the row kernel runs: 32 tokens x 128 experts of d 4096 5.7 us (8 experts 2.9),
// the tile kernel 7.9 (5.9).
constexpr int kRowMaxTokens = 32;

cudaError_t launch_moe_logits(const void* x, const void* w, int T, int E, int d, float* logits, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (T <= kRowMaxTokens) {
    cfg.gridDim = dim3((unsigned)E, (unsigned)((T + kRowTokens - 1) / kRowTokens));
    cfg.blockDim = dim3(kRowThreads);
    return cudaLaunchKernelEx(&cfg, row_kernel, static_cast<const bf16*>(x), static_cast<const bf16*>(w), T, E, d, logits);
  }
  CUtensorMap tm_x, tm_w;
  if (!encode_rows(&tm_x, x, T, d, kM) || !encode_rows(&tm_w, w, E, d, kMaxN)) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  // As many CTAs per tile as two per SM allow, each with at least two stages of work; and enough that
  // no accumulator takes more than 44 steps (d / split <= 1408) where 8 CTAs can do that.  Relative
  // error at d 4096: 2.4e-7 with 16 steps, 4.7e-7 with 32, 1.0e-6 with 64, 2.1e-6 with 128.
  const long long token_tiles = (T + kM - 1) / kM, tiles = token_tiles * ((E + kMaxN - 1) / kMaxN);
  const int n_kb = (d + kKB - 1) / kKB;
  int split = 1;
  while (split < kMaxSplit && tiles * split * 2 <= 2 * sm_count() && n_kb >= 4 * split) split *= 2;
  // Clusters of 1, 2, 3, 4 and 8 fill the chip: 10000 tokens x 128 experts 22.6 us with 3 (32.1 with 4,
  // more than fit at once); 5000 tokens 17.6 with 4 (24.5 with 7).
  const int need = (n_kb + 21) / 22;
  if (split < need) split = need <= 4 ? need : kMaxSplit;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(token_tiles * split), (unsigned)((E + kMaxN - 1) / kMaxN));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, tile_kernel, T, E, d, logits, split, tm_x, tm_w);
}

}  // namespace csffn
