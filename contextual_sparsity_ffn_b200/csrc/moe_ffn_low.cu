// The experts' gated FFNs where experts have few rows (decode steps): the weights' stream.
//
// The same products as moe_ffn.cu, D[output, row] with the weights as M = 128 and up to 32 rows of one
// expert as N, one CTA per tile.  A gate/up tile is 64 neurons: its A operand is their W_gate rows over
// their W_up rows, so one MMA yields both, gate in the lower 64 TMEM lanes and up in the upper 64; the
// epilogue hands up over to the gate's warps through shared memory.  A down tile is 128 columns.  Tiles
// this small go round the 148 SMs evenly without being cut: one token through 8 of 64 experts of 1024
// neurons is 128 tiles of each kind.
//
// v is kept as a bf16 high part and a bf16 low part (v - high), the two halves of the down product's
// N side: about 16 bits of v reach the product at no cost in time.  The k-steps alternate between two
// accumulators, so that consecutive MMAs do not wait on one another's sums.
//
// Work split as in moe_ffn.cu, by CTAs: whole tiles in rounds, then the tiles left over, cut along the
// contraction where that saves enough k-blocks; more than half as many as CTAs, as one run of k-blocks
// divided evenly (a CTA holds parts of at most two tiles).
//
// Warp roles (320 threads): warp 0 issues the TMA copies, warp 1 owns TMEM and issues the MMAs, warps
// 2-9 run the epilogue: two per TMEM lane quarter, 16 of the 32 rows each.  Every wait is bounded (one
// second) and records the timeout.
#include "moe_ffn.cuh"

namespace csffn {
namespace {

using namespace moe;

constexpr int kThreads = 320, kEpiWarps = 8;
constexpr int kN = kMoeLowTile;                       // rows per tile
constexpr uint32_t kWBytes = 128 * kRowBytes;         // weights of a stage: 16 KB
constexpr uint32_t kRowsBytes = kN * kRowBytes;       // rows of a stage (of one part of v): 4 KB

// What rounding v to its high part left.  Nothing where the high part is infinite: v itself, or a v
// past bf16's range; inf - inf would make the row NaN.
__device__ __forceinline__ float rest(float v, float high) { return fabsf(high) < INFINITY ? v - high : 0.f; }

template <bool kDown>
struct Cfg {
  static constexpr int kTileOut = kDown ? 128 : 64;
  static constexpr int kParts = kDown ? 2 : 1;  // high and low part of v
  static constexpr uint32_t kStage = kWBytes + kParts * kRowsBytes;
  static constexpr int kStages = kDown ? 8 : 10;
  static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
  // columns: two buffers of two accumulators (even and odd k-steps)
  static constexpr uint32_t kAcc = kParts * kN, kBuffer = 2 * kAcc, kColumns = 2 * kBuffer;
};

template <bool kDown>
__global__ void __launch_bounds__(kThreads, 1)
    low_kernel(const Args a, const __grid_constant__ CUtensorMap tm_w0, const __grid_constant__ CUtensorMap tm_w1,
               const __grid_constant__ CUtensorMap tm_r) {
  using C = Cfg<kDown>;
  constexpr int kStages = C::kStages;
  extern __shared__ __align__(1024) unsigned char low_raw[];
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], accf[2], acce[2], drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ bool s_last;
  __shared__ Plan s_plan;
  __shared__ float s_up[kDown ? 1 : 2][kDown ? 1 : kN][64];  // up values on their way to the gate's warps
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(low_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mb = (a.N + C::kTileOut - 1) / C::kTileOut, n_kb = (a.K + kKB - 1) / kKB;

  if (threadIdx.x == 0) {
    tma_prefetch_map(&tm_w0);
    if (!kDown) tma_prefetch_map(&tm_w1);
    tma_prefetch_map(&tm_r);
    s_abort = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&accf[i], 1);
      mbar_init(&acce[i], kEpiWarps);
    }
    mbar_init(&drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, C::kColumns);
    tmem_relinquish();
  }
  // As in moe_ffn.cu: the down kernel starts after the gate/up kernel's wait, so it may read the offsets
  // and the weights before its own, and v after it; and it lets nothing start early.
  if (!kDown) {
    pdl_wait_prior();
    pdl_trigger();
  }
  for (int e = threadIdx.x; e <= a.E; e += kThreads) s_plan.lo[e] = __ldcg(a.offsets + e);
  __syncthreads();
  if (warp == 0) make_plan<kN>(a, &s_plan);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int n_tiles = s_plan.tp[a.E] * mb;

  if (warp == 0) {
    if (lane == 0) {
      // ---- producer
      Ring r;
      long long issued = 0;
      bool ok = true;
      // weights that one tile alone reads make way first in L2 (1% on the stream of 2.8 GB)
      const uint64_t first_out = l2_evict_first_policy(), normal = l2_evict_normal_policy();
      auto weights = [&](const Tile& t, int kb, int slot) {
        unsigned char* st = smem + (size_t)slot * C::kStage;
        const uint64_t pol = t.once ? first_out : normal;
        mbar_arrive_expect_tx(&full[slot], C::kStage);
        if constexpr (kDown) {
          tma_load_3d_hint(st, &tm_w0, t.m * 128, kb * kKB, t.e, &full[slot], pol);
          tma_load_3d_hint(st + kWBytes / 2, &tm_w0, t.m * 128 + 64, kb * kKB, t.e, &full[slot], pol);
        } else {
          tma_load_3d_hint(st, &tm_w0, kb * kKB, t.m * 64, t.e, &full[slot], pol);
          tma_load_3d_hint(st + kWBytes / 2, &tm_w1, kb * kKB, t.m * 64, t.e, &full[slot], pol);
        }
      };
      Items w(blockIdx.x, gridDim.x, n_kb, n_tiles, true);
      bool more = w.advance();
      int first = 0;  // stages of the first item whose weights went out before the wait
      if (kDown && more) {
        const Tile t = find_tile(s_plan, a.E, mb, w.tile);
        first = min(kStages, w.kb1 - w.kb0);
        for (int q = 0; q < first; ++q) weights(t, w.kb0 + q, q);
      }
      if (kDown) pdl_wait_prior();
      for (; ok && more; more = w.advance()) {
        const Tile t = find_tile(s_plan, a.E, mb, w.tile);
        for (int kb = w.kb0; kb < w.kb1; ++kb, ++issued) {
          if (issued >= first) {
            if (r.round > 0 && !mbar_wait(&empty[r.slot], (r.round - 1) & 1, a.err, &s_abort)) {
              ok = false;
              break;
            }
            weights(t, kb, r.slot);
          }
          unsigned char* st = smem + (size_t)r.slot * C::kStage + kWBytes;
          tma_load_2d_plain(st, &tm_r, kb * kKB, t.row0, &full[r.slot]);
          if constexpr (kDown) tma_load_2d_plain(st + kRowsBytes, &tm_r, kb * kKB, a.rows + t.row0, &full[r.slot]);
          r.next(kStages);
        }
      }
      // the copies in flight land before the CTA's shared memory is released
      for (long long q = issued > kStages ? issued - kStages : 0; q < issued; ++q)
        mbar_wait_drain(&full[q % kStages], (uint32_t)(q / kStages) & 1, a.err);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---- MMA issuer
      const uint32_t idesc = umma_idesc_bf16(128, C::kAcc, kDown);
      Ring r;
      int m = 0;
      bool ok = true;
      Items w(blockIdx.x, gridDim.x, n_kb, n_tiles, true);
      while (ok && w.advance()) {
        const int b = m & 1;
        if (m >= 2 && !mbar_wait(&acce[b], ((m >> 1) - 1) & 1, a.err, &s_abort)) break;
        tc_fence_after();
        const uint32_t d0 = tmem + C::kBuffer * b;
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!mbar_wait(&full[r.slot], r.round & 1, a.err, &s_abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sb = smem_u32(smem + (size_t)r.slot * C::kStage);
#pragma unroll
          for (int k = 0; k < kKB / 16; ++k) {
            const uint64_t aw = kDown ? umma_desc_mn(sb + 2048u * k, kWBytes / 2) : umma_desc_k(sb + 32u * k);
            umma_bf16(d0 + C::kAcc * (k & 1), aw, umma_desc_k(sb + kWBytes + 32u * k), idesc,
                      (kb > w.kb0 || k > 1) ? 1u : 0u);
          }
          umma_commit(&empty[r.slot]);
          r.next(kStages);
        }
        if (!ok) break;
        umma_commit(&accf[b]);
        ++m;
      }
      umma_commit(&drain);
      mbar_wait_drain(&drain, 0, a.err);
    }
  } else {
    // ---- epilogue
    if (kDown) pdl_wait_prior();  // the parts and counters are the gate/up kernel's until it is done
    const int quarter = warp & 3, c0 = ((warp - 2) >> 2) * 16;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16);
    const bool odd = lane & 1, high = lane & 2;
    int m = 0, turn = 0;
    Items w(blockIdx.x, gridDim.x, n_kb, n_tiles, true);
    for (; w.advance(); ++m) {
      const Tile t = find_tile(s_plan, a.E, mb, w.tile);
      const int b = m & 1;
      // every epilogue warp leaves together (they meet at named barriers)
      if (!named_all(1, kEpiWarps * kWarp, mbar_wait(&accf[b], (m >> 1) & 1, a.err, &s_abort))) break;
      tc_fence_after();
      const uint32_t acc = lane_base + C::kBuffer * b + (uint32_t)c0;
      float g[16], x[16];
      tmem_ld16(acc, g);
      tmem_ld16(acc + C::kAcc, x);
      tmem_ld_wait(g);
      tmem_ld_wait(x);
#pragma unroll
      for (int k = 0; k < 16; ++k) g[k] += x[k];
      if constexpr (kDown) {  // the low part of v's share
        float y[16];
        tmem_ld16(acc + kN, x);
        tmem_ld16(acc + C::kAcc + kN, y);
        tmem_ld_wait(x);
        tmem_ld_wait(y);
#pragma unroll
        for (int k = 0; k < 16; ++k) g[k] += x[k] + y[k];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acce[b]);

      if (!w.whole()) {
        // a part: into its place, [32 / 4 columns][128 lanes][4]
        auto part_at = [&](int place) {
          return reinterpret_cast<float4*>(a.part) + ((size_t)place * (kN / 4) + c0 / 4) * 128 + 32 * quarter + lane;
        };
        float4* mine = part_at(w.my_place());
#pragma unroll
        for (int k = 0; k < 4; ++k)
          __stcg(mine + k * 128, make_float4(g[4 * k], g[4 * k + 1], g[4 * k + 2], g[4 * k + 3]));
        const int parts = w.parts();
        // the barriers order the CTA's stores and loads around one thread's fences
        named_sync(2, kEpiWarps * kWarp);
        if (threadIdx.x == 2 * kWarp) {
          uint32_t* ctr = a.ctr + w.left_tile();
          __threadfence();
          s_last = atomicAdd(ctr, 1u) + 1u == (uint32_t)parts;
          if (s_last) *ctr = 0u;
          __threadfence();
        }
        named_sync(2, kEpiWarps * kWarp);
        const bool last = s_last;
        named_sync(2, kEpiWarps * kWarp);  // s_last is written again by the next part
        if (!last) continue;
#pragma unroll
        for (int k = 0; k < 16; ++k) g[k] = 0.f;
#pragma unroll 4
        for (int r = 0; r < parts; ++r) {
          const float4* from = part_at(w.place(r));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 v = __ldcg(from + k * 128);
            g[4 * k] += v.x, g[4 * k + 1] += v.y, g[4 * k + 2] += v.z, g[4 * k + 3] += v.w;
          }
        }
      }

      if constexpr (!kDown) {
        // Up to the gate's warps.  Two buffers and one barrier a tile: a buffer is written again only after
        // the next tile's barrier, which the gate's warps reach when they are done with it.
        if (quarter >= 2) {
#pragma unroll
          for (int k = 0; k < 16; ++k) s_up[turn][c0 + k][32 * (quarter - 2) + lane] = g[k];
        }
        named_sync(3, kEpiWarps * kWarp);
        if (quarter < 2) {
#pragma unroll
          for (int k = 0; k < 16; ++k) g[k] = act_fast(g[k], a.act) * s_up[turn][c0 + k][32 * quarter + lane];
        }
        turn ^= 1;
        if (quarter >= 2) continue;
      }
      // As in moe_ffn.cu, 4 outputs x 4 rows turned around among neighbouring lanes; gate/up: the high
      // part, then what its rounding left.
      const int out = t.m * C::kTileOut + 32 * quarter + (lane & ~3);  // N is a multiple of 8
      bf16* base = a.out;
#pragma unroll
      for (int pass = 0; pass < (kDown ? 1 : 2); ++pass) {
        uint32_t p[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(g[2 * k], g[2 * k + 1]);
          p[k] = reinterpret_cast<const uint32_t&>(v);
          g[2 * k] = rest(g[2 * k], bf16lo(p[k]));
          g[2 * k + 1] = rest(g[2 * k + 1], bf16hi(p[k]));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t got = __shfl_xor_sync(0xffffffffu, __byte_perm(p[2 * j], p[2 * j + 1], odd ? 0x5410 : 0x7632), 1);
          const uint32_t a0 = __byte_perm(p[2 * j], got, odd ? 0x3254 : 0x5410);
          const uint32_t a1 = __byte_perm(p[2 * j + 1], got, odd ? 0x3276 : 0x7610);
          const uint32_t back = __shfl_xor_sync(0xffffffffu, high ? a0 : a1, 2);
          const int row = t.row0 + c0 + 4 * j + (lane & 3);
          if (row < t.row1 && out < a.N)
            *reinterpret_cast<uint2*>(base + (size_t)row * a.N + out) = high ? make_uint2(back, a1) : make_uint2(a0, back);
        }
        base += (size_t)a.rows * a.N;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kColumns);
  }
}

template <bool kDown>
cudaError_t launch_low(const Args& p, const CUtensorMap& w0, const CUtensorMap& w1, const CUtensorMap& r, cudaStream_t s) {
  using C = Cfg<kDown>;
  cudaError_t e = cudaFuncSetAttribute(low_kernel<kDown>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (e != cudaSuccess) return e;
  // one CTA per SM; no more than k-blocks there can be (every tile has a row, an expert at most one
  // ragged tile)
  const long long row_tiles = (long long)(p.rows + kN - 1) / kN + (p.E < p.rows ? p.E : p.rows);
  const long long blocks = row_tiles * ((p.N + C::kTileOut - 1) / C::kTileOut) * ((p.K + kKB - 1) / kKB);
  int ctas = sm_count() < 2 * kMoeMaxPairs ? sm_count() : 2 * kMoeMaxPairs;
  if (blocks < ctas) ctas = (int)blocks;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, low_kernel<kDown>, p, w0, w1, r);
}

}  // namespace

cudaError_t launch_moe_ffn_low(const MoeFfnArgs& a, cudaStream_t s) {
  CUtensorMap tm_g, tm_u, tm_x, tm_d, tm_v;
  if (!encode_weights(&tm_g, a.W_gate, a, 64) || !encode_weights(&tm_u, a.W_up, a, 64) ||
      !encode_weights(&tm_d, a.W_down_t, a, 64) || !encode_rows(&tm_x, a.xs, a.rows, a.d, kN) ||
      !encode_rows(&tm_v, a.v, 2 * a.rows, a.h, kN))
    return cudaErrorInvalidValue;
  const Args gu{a.offsets, a.rows, a.E, a.h, a.d, a.act, static_cast<bf16*>(a.v), a.part, kN, a.ctr, a.err};
  cudaError_t e = launch_low<false>(gu, tm_g, tm_u, tm_x, s);
  if (e != cudaSuccess) return e;
  const Args dn{a.offsets, a.rows, a.E, a.d, a.h, a.act, static_cast<bf16*>(a.ys), a.part, kN,
                a.ctr + 2 * kMoeMaxPairs, a.err};
  return launch_low<true>(dn, tm_d, tm_d, tm_v, s);
}

}  // namespace csffn
