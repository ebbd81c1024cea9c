// The experts' gated FFNs on rows sorted by expert, on the fifth-generation tensor cores.
//
//   gate/up: v[p, i] = act(xs_p . W_gate[e, i]) * (xs_p . W_up[e, i])      (bf16 into the workspace)
//   down:    ys[p, c] = sum_i v[p, i] W_down^T[e, i, c]
//
// For experts with many rows each; moe_ffn_low.cu is for few.
//
// v is rounded once to bf16, the operands' type.  The result's error against 64 bits is 2.3e-3 (relative L2),
// 1.7e-3 where v reaches the down product in two parts as in moe_ffn_low.cu: that is the rounding of ys
// alone.  There the second part comes for nothing, the weights' stream is the time; here the
// multiplications are, and it would double the down product's, a third more of all.
//
// Both kernels compute D[output, row] with the weights as the M side: a tile is 256 outputs
// (neurons, or columns of ys) x up to 256 rows of one expert, and a pair of CTAs works on it
// (cta_group::2, M = 256: 128 outputs each).  The rows are the N side because an expert's row count
// is whatever the router made it: N is any multiple of 32 up to 256 chosen per tile, so a ragged
// expert wastes at most 31 rows of multiplication and none of the weight traffic.
//
// The down kernel's tiles are 512 columns wide where there are enough of them (kWide): two blocks of
// 256 that share the rows, as gate and up do.  What bounds these tiles with many rows is the operands'
// way from L2 to the SMs: 64 bytes a cycle and SM for 256 x 256 at the tensor cores' full rate, 48 for
// 512 x 256.
//
// Work split: whole tiles go round the pairs as long as there is one for every pair.  The R tiles
// left over would leave pairs idle, so they are cut along the
// contraction where that pays: up to half as many tiles as pairs, each into S = pairs / R parts (at
// most kMaxPartsTall), one part per pair.  A pair with a part stores its fp32 accumulators in the
// workspace and counts up the tile's counter; the last one adds the parts in their order (the same
// bits whoever is last), writes the tile and clears the counter.  No pair waits for another.
//
// Row split: an expert with n rows takes ceil(n / 256) tiles of equal height (rounded up to 32).
// Tiles are numbered expert by expert, output block by output block, row tiles innermost, so the
// pairs at work at one time share weight blocks and an expert's rows through L2.
//
// Operands come by TMA tensor copies with the 128-byte swizzle, 64 contraction elements per stage:
// W_gate and W_up 128 x 64 each (gate/up, K-major) or W_down^T as two boxes of 64 columns x 64
// neurons per block (down, MN-major), and half the tile's rows in each CTA.  All copies of a stage
// complete on one barrier of the pair's even CTA, whose MMA warp issues for both.  Accumulators: two
// buffers, one drained while the next tile accumulates: 256 TMEM columns each, or 128 columns of each
// of two accumulators (gate and up, the blocks of a wide tile); a tile of more than 128 rows with two
// accumulators takes both buffers.
//
// Warp roles: warp 0 issues the copies, warp 1 owns TMEM and (even CTA) issues the MMAs, the other
// 8 run the epilogue: TMEM lane = output, column = row, two warps per lane quarter, each half of the
// columns.  While a tile with two accumulators is drained no MMA runs, so the epilogue keeps the next
// columns' TMEM loads under way and stores 8 bytes a lane.
//
// Row bounds come from the device: `offsets` is clamped to 0 .. rows and to ascending order when it is
// read, so no offsets can lead an access outside the buffers.  Every wait is bounded (one second)
// and records the timeout.
//
// One B200, balanced routing: 4096 tokens x 2 of 8 experts (d 4096, h 14336) 2.0 to 2.2 ms with the clock
// that the power limit leaves, 1310 to 1440 TFLOP/s; 4096 x 8 of 64 (d 2048, h 1024) 373 us, where a
// tile's epilogue (7 of 40 thousand cycles) shows.
#include "moe_ffn.cuh"

namespace csffn {
namespace {

using namespace moe;

constexpr uint32_t kWBox = 128 * kRowBytes;  // one CTA's 128 outputs x 64: 16 KB

template <bool kDown, bool kWide>
struct Cfg {
  static constexpr int kTileOut = kWide ? 512 : 256;                   // outputs per tile
  static constexpr int kAccs = kDown && !kWide ? 1 : 2;                // gate and up, or two blocks of 256 columns
  static constexpr int kEpiWarps = 8;
  static constexpr int kSides = kEpiWarps / 4;         // shares of a tile's columns
  static constexpr int kThreads = (2 + kEpiWarps) * kWarp;
  static constexpr uint32_t kW = kAccs * kWBox;
  static constexpr uint32_t kStage = kW + (uint32_t)(kMoeTileRows / 2) * kRowBytes;
  static constexpr int kStages = kAccs == 1 ? 6 : 4;
  static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
  // Accumulator columns: two buffers; the second accumulator is kUp columns behind the first.  With two
  // accumulators a tile of more than 128 rows takes both buffers.
  static constexpr uint32_t kBuffer = kAccs == 1 ? 256u : 128u;
  static constexpr uint32_t kUp = 2 * kBuffer;
  static constexpr uint32_t kColumns = 512;
};

// Which accumulator buffers an item takes, and how often each was taken before: every role counts the
// same items, so they agree on the barriers' phases.
template <bool kDown, bool kWide>
struct Buffers {
  int turn = 0;
  uint32_t used0 = 0, used1 = 0;
  int b;      // first buffer of the item
  bool both;  // it takes both
  __device__ uint32_t used() const { return b ? used1 : used0; }
  __device__ void take(int n) {
    both = Cfg<kDown, kWide>::kAccs == 2 && n > 128;
    b = both ? 0 : turn;
    if (!both) turn ^= 1;
  }
  __device__ void done() {
    if (b == 0) ++used0;
    if (b == 1 || both) ++used1;
  }
  __device__ uint32_t column() const { return Cfg<kDown, kWide>::kBuffer * b; }
};

template <bool kDown, bool kWide>
__global__ void __launch_bounds__(Cfg<kDown, kWide>::kThreads, 1)
    pair_kernel(const Args a, const __grid_constant__ CUtensorMap tm_w0, const __grid_constant__ CUtensorMap tm_w1,
                const __grid_constant__ CUtensorMap tm_r64, const __grid_constant__ CUtensorMap tm_r16) {
  using C = Cfg<kDown, kWide>;
  constexpr int kStages = C::kStages, kEpiWarps = C::kEpiWarps, kChunk = 16;
  extern __shared__ __align__(1024) unsigned char moe_raw[];
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], accf[2], acce[2], drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ bool s_last;
  __shared__ Plan s_plan;
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(moe_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int mb = (a.N + C::kTileOut - 1) / C::kTileOut, n_kb = (a.K + kKB - 1) / kKB;

  if (threadIdx.x == 0) {
    tma_prefetch_map(&tm_w0);
    if (!kDown) tma_prefetch_map(&tm_w1);
    tma_prefetch_map(&tm_r64);
    tma_prefetch_map(&tm_r16);
    s_abort = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&accf[i], 1);
      mbar_init(&acce[i], 2 * kEpiWarps);
    }
    mbar_init(&drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&s_tmem, C::kColumns);
    tmem_relinquish_pair();
  }
  // The gate/up kernel lets the down kernel start only after its own wait, so what came before the
  // gate/up kernel is complete when the down kernel starts: the offsets (and the weights) may be read
  // before the down kernel's wait, v after it.  The down kernel lets nothing start early: ys may be weights
  // of the call that follows.
  if (!kDown) {
    pdl_wait_prior();
    pdl_trigger();
  }
  for (int e = threadIdx.x; e <= a.E; e += C::kThreads) s_plan.lo[e] = __ldcg(a.offsets + e);
  tc_fence_before();
  __syncthreads();
  cluster_arrive_all();
  if (warp == 0) make_plan<kMoeTileRows>(a, &s_plan);
  __syncthreads();
  cluster_wait_all();  // both CTAs' barriers and TMEM are set up
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int n_tiles = s_plan.tp[a.E] * mb;

  if (warp == 0) {
    if (lane == 0) {
      // ---- producer
      Ring r;
      long long issued = 0;
      bool ok = true;
      auto weights = [&](const Tile& t, int kb, unsigned char* st, uint32_t bar) {
        const int out0 = t.m * C::kTileOut + (int)rank * 128;
        if constexpr (kDown) {
#pragma unroll
          for (int b = 0; b < C::kAccs; ++b) {
            tma_load_3d_pair(st + b * kWBox, &tm_w0, out0 + 256 * b, kb * kKB, t.e, bar);
            tma_load_3d_pair(st + b * kWBox + kWBox / 2, &tm_w0, out0 + 256 * b + 64, kb * kKB, t.e, bar);
          }
        } else {
          tma_load_3d_pair(st, &tm_w0, kb * kKB, out0, t.e, bar);
          tma_load_3d_pair(st + kWBox, &tm_w1, kb * kKB, out0, t.e, bar);
        }
      };
      auto rows = [&](const Tile& t, int kb, unsigned char* st, uint32_t bar) {
        const int half = t.n / 2, row0 = t.row0 + (int)rank * half;
        int n = 0;
        for (; n + 64 <= half; n += 64) tma_load_2d_pair(st + C::kW + n * kRowBytes, &tm_r64, kb * kKB, row0 + n, bar);
        for (; n < half; n += 16) tma_load_2d_pair(st + C::kW + n * kRowBytes, &tm_r16, kb * kKB, row0 + n, bar);
      };
      auto expect = [&](const Tile& t, int slot) {
        if (rank == 0) mbar_arrive_expect_tx(&full[slot], 2 * (C::kW + (uint32_t)(t.n / 2) * kRowBytes));
      };
      Items w(pair, pairs, n_kb, n_tiles, false);
      bool more = w.advance();
      int first = 0;  // stages of the first item whose weights went out before the wait
      if (kDown && more) {
        const Tile t = find_tile(s_plan, a.E, mb, w.tile);
        first = min(kStages, w.kb1 - w.kb0);
        for (int q = 0; q < first; ++q) {
          expect(t, q);
          weights(t, w.kb0 + q, smem + (size_t)q * C::kStage, map_to_rank(&full[q], 0));
        }
      }
      if (kDown) pdl_wait_prior();
      for (; ok && more; more = w.advance()) {
        const Tile t = find_tile(s_plan, a.E, mb, w.tile);
        for (int kb = w.kb0; kb < w.kb1; ++kb, ++issued) {
          unsigned char* st = smem + (size_t)r.slot * C::kStage;
          const uint32_t bar = map_to_rank(&full[r.slot], 0);
          if (issued >= first) {
            if (r.round > 0 && !mbar_wait(&empty[r.slot], (r.round - 1) & 1, a.err, &s_abort)) {
              ok = false;
              break;
            }
            expect(t, r.slot);
            weights(t, kb, st, bar);
          }
          rows(t, kb, st, bar);
          r.next(kStages);
        }
      }
      // the copies in flight land before the pair's shared memory is released
      if (rank == 0) {
        for (long long q = issued > kStages ? issued - kStages : 0; q < issued; ++q)
          mbar_wait_drain(&full[q % kStages], (uint32_t)(q / kStages) & 1, a.err);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ---- MMA issuer
      Ring r;
      bool ok = true;
      Buffers<kDown, kWide> buf;
      Items w(pair, pairs, n_kb, n_tiles, false);
      while (ok && w.advance()) {
        const int n = find_tile(s_plan, a.E, mb, w.tile).n;
        const uint32_t idesc = umma_idesc_bf16(256, n, kDown);
        buf.take(n);
        if (buf.used() && !mbar_wait(&acce[buf.b], (buf.used() - 1) & 1, a.err, &s_abort)) break;
        if (buf.both && buf.used1 && !mbar_wait(&acce[1], (buf.used1 - 1) & 1, a.err, &s_abort)) break;
        tc_fence_after();
        const uint32_t d0 = tmem + buf.column(), d1 = d0 + C::kUp;
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!mbar_wait(&full[r.slot], r.round & 1, a.err, &s_abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sb = smem_u32(smem + (size_t)r.slot * C::kStage);
#pragma unroll
          for (int k = 0; k < kKB / 16; ++k) {
            const uint32_t acc = (kb > w.kb0 || k) ? 1u : 0u;
            const uint64_t br = umma_desc_k(sb + C::kW + 32u * k);
            if constexpr (kDown) {
              umma_bf16_pair(d0, umma_desc_mn(sb + 2048u * k, kWBox / 2), br, idesc, acc);
              if constexpr (kWide) umma_bf16_pair(d1, umma_desc_mn(sb + kWBox + 2048u * k, kWBox / 2), br, idesc, acc);
            } else {
              umma_bf16_pair(d0, umma_desc_k(sb + 32u * k), br, idesc, acc);
              umma_bf16_pair(d1, umma_desc_k(sb + kWBox + 32u * k), br, idesc, acc);
            }
          }
          umma_commit_pair(&empty[r.slot]);
          r.next(kStages);
        }
        if (!ok) break;
        umma_commit_pair(&accf[buf.b]);
        if (buf.both) umma_commit_pair(&accf[1]);
        buf.done();
      }
      umma_commit_pair(&drain);
      mbar_wait_drain(&drain, 0, a.err);
    } else if (lane == 0) {
      mbar_wait_drain(&drain, 0, a.err);  // the even CTA's last commit has arrived here too
    }
  } else {
    // ---- epilogue: warps 2..9, TMEM lane quarter warp % 4, share (warp - 2) / 4 of the columns
    if (kDown) pdl_wait_prior();  // the parts and counters are the gate/up kernel's until it is done
    const int quarter = warp & 3, side = (warp - 2) >> 2;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16);
    const int out_lane = 32 * quarter + lane;
    const bool odd = lane & 1, high = lane & 2;
    const size_t part_acc = (size_t)a.part_n / 4 * 128, part_place = C::kAccs * part_acc * 4;  // float4s, floats
    Buffers<kDown, kWide> buf;
    Items w(pair, pairs, n_kb, n_tiles, false);
    while (w.advance()) {
      const Tile t = find_tile(s_plan, a.E, mb, w.tile);
      buf.take(t.n);
      bool got = mbar_wait(&accf[buf.b], buf.used() & 1, a.err, &s_abort);
      if (got && buf.both) got = mbar_wait(&accf[1], buf.used1 & 1, a.err, &s_abort);
      // every epilogue warp leaves together (split tiles meet at a named barrier)
      if (!named_all(1, kEpiWarps * kWarp, got)) break;
      tc_fence_after();
      const uint32_t acc = lane_base + buf.column();
      const int o = t.m * C::kTileOut + (int)rank * 128 + (out_lane & ~3);  // N is a multiple of 8
      const int c0 = side * (t.n / C::kSides), c1 = c0 + t.n / C::kSides;

      // A chunk of columns' results to memory.  `p`: column pairs of this lane's output.  Two exchanges
      // turn 4 outputs x 4 columns of neighbouring lanes around, so that a lane stores 4 adjacent
      // outputs (8 bytes) of column 4 j + lane % 4.
      auto store = [&](int c, const uint32_t (&p)[kChunk / 2], int out, bf16* base) {
#pragma unroll
        for (int j = 0; j < kChunk / 4; ++j) {
          const uint32_t got = __shfl_xor_sync(0xffffffffu, __byte_perm(p[2 * j], p[2 * j + 1], odd ? 0x5410 : 0x7632), 1);
          const uint32_t a0 = __byte_perm(p[2 * j], got, odd ? 0x3254 : 0x5410);
          const uint32_t a1 = __byte_perm(p[2 * j + 1], got, odd ? 0x3276 : 0x7610);
          const uint32_t back = __shfl_xor_sync(0xffffffffu, high ? a0 : a1, 2);
          const int row = t.row0 + c + 4 * j + (lane & 3);
          if (row < t.row1 && out < a.N)
            *reinterpret_cast<uint2*>(base + (size_t)row * a.N + out) = high ? make_uint2(back, a1) : make_uint2(a0, back);
        }
      };
      auto put16 = [&](int c, const float (&g)[kChunk], int out) {
        uint32_t p[kChunk / 2];
#pragma unroll
        for (int k = 0; k < kChunk / 2; ++k) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(g[2 * k], g[2 * k + 1]);
          p[k] = reinterpret_cast<const uint32_t&>(v);
        }
        store(c, p, out, a.out);
      };
      auto put = [&](int c, float (&g)[kChunk], const float (&u)[kChunk]) {
        if constexpr (!kDown) {
#pragma unroll
          for (int k = 0; k < kChunk; ++k) g[k] = act_fast(g[k], a.act) * u[k];
        }
        put16(c, g, o);
        if constexpr (kWide) put16(c, u, o + 256);
      };
      const bool whole = w.whole();
      // this thread's 4-column vectors of the part kept at a place
      auto part_at = [&](int place) {
        return reinterpret_cast<float4*>(a.part + (size_t)(place * 2 + (int)rank) * part_place) + out_lane;
      };
      float4* mine = whole ? nullptr : part_at(w.my_place());
      auto load = [&](int c, float (&g)[kChunk], float (&u)[kChunk]) {
        __syncwarp();
        tmem_ld16(acc + (uint32_t)c, g);
        if constexpr (C::kAccs == 2) tmem_ld16(acc + C::kUp + (uint32_t)c, u);
      };
      auto take = [&](int c, float (&g)[kChunk], float (&u)[kChunk]) {
        if (whole) {
          put(c, g, u);
        } else {
#pragma unroll
          for (int k = 0; k < kChunk / 4; ++k) {
            __stcg(mine + (size_t)(c / 4 + k) * 128, make_float4(g[4 * k], g[4 * k + 1], g[4 * k + 2], g[4 * k + 3]));
            if constexpr (C::kAccs == 2)
              __stcg(mine + part_acc + (size_t)(c / 4 + k) * 128,
                     make_float4(u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]));
          }
        }
      };
      auto ready = [&](float (&g)[kChunk], float (&u)[kChunk]) {
        tmem_ld_wait(g);
        if constexpr (C::kAccs == 2) tmem_ld_wait(u);
      };
      // A tile that holds both buffers gives them up as soon as its last columns are in registers: the
      // next tile's MMAs wait for that.
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_cluster(map_to_rank(&acce[buf.b], 0));
          if (buf.both) mbar_arrive_cluster(map_to_rank(&acce[1], 0));
        }
      };
      // the next chunk's loads are under way while one is worked on
      float g0[kChunk], u0[kChunk], g1[kChunk], u1[kChunk];
      load(c0, g0, u0);
      for (int c = c0; c < c1; c += 2 * kChunk) {
        const bool two = c + kChunk < c1, more = c + 2 * kChunk < c1;
        ready(g0, u0);
        if (two) load(c + kChunk, g1, u1);
        if (!more && buf.both) {
          if (two) ready(g1, u1);
          release();
        }
        take(c, g0, u0);
        if (two) {
          if (more || !buf.both) ready(g1, u1);
          if (more) load(c + 2 * kChunk, g0, u0);
          take(c + kChunk, g1, u1);
        }
      }
      if (!buf.both) release();
      buf.done();
      if (whole) continue;

      const int parts = w.parts();
      uint32_t* ctr = a.ctr + 2 * w.left_tile() + rank;
      // the barriers order the CTA's stores and loads around one thread's fences
      named_sync(2, kEpiWarps * kWarp);
      if (threadIdx.x == 2 * kWarp) {
        __threadfence();
        s_last = atomicAdd(ctr, 1u) + 1u == (uint32_t)parts;
        if (s_last) *ctr = 0u;
        __threadfence();
      }
      named_sync(2, kEpiWarps * kWarp);
      if (!s_last) {
        named_sync(2, kEpiWarps * kWarp);  // s_last is written again by the next part
        continue;
      }
      for (int c = c0; c < c1; c += kChunk) {
        float g[kChunk], u[kChunk];
#pragma unroll
        for (int k = 0; k < kChunk; ++k) g[k] = u[k] = 0.f;
#pragma unroll 2
        for (int r = 0; r < parts; ++r) {
          const float4* from = part_at(w.place(r)) + (size_t)(c / 4) * 128;
#pragma unroll
          for (int k = 0; k < kChunk / 4; ++k) {
            const float4 x = __ldcg(from + (size_t)k * 128);
            g[4 * k] += x.x, g[4 * k + 1] += x.y, g[4 * k + 2] += x.z, g[4 * k + 3] += x.w;
            if constexpr (C::kAccs == 2) {
              const float4 y = __ldcg(from + part_acc + (size_t)k * 128);
              u[4 * k] += y.x, u[4 * k + 1] += y.y, u[4 * k + 2] += y.z, u[4 * k + 3] += y.w;
            }
          }
        }
        put(c, g, u);
      }
      named_sync(2, kEpiWarps * kWarp);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA's shared memory or TMEM goes while the pair still uses it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, C::kColumns);
  }
}

// Pairs of CTAs to launch: as many as fit on the device at once (a static split over more would
// wait for the first ones to finish), looked up once per device and kernel.
template <bool kDown, bool kWide>
cudaError_t resident_pairs(const cudaLaunchConfig_t& cfg, int* out) {
  static int cached[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int n = dev >= 0 && dev < 64 ? cached[dev] : 0;
  if (n == 0) {
    e = cudaOccupancyMaxActiveClusters(&n, pair_kernel<kDown, kWide>, &cfg);
    if (e != cudaSuccess) return e;
    if (n > kMoeMaxPairs) n = kMoeMaxPairs;
    if (n < 1) return cudaErrorInvalidConfiguration;
    if (dev >= 0 && dev < 64) cached[dev] = n;
  }
  *out = n;
  return cudaSuccess;
}

template <bool kDown, bool kWide>
cudaError_t launch_pair(const Args& p, const CUtensorMap& w0, const CUtensorMap& w1, const CUtensorMap& r64,
                        const CUtensorMap& r16, cudaStream_t s) {
  using C = Cfg<kDown, kWide>;
  cudaError_t e = cudaFuncSetAttribute(pair_kernel<kDown, kWide>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sm_count() / 2 * 2));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;  // the cluster; the dependent launch is no part of the query
  int pairs = 0;
  if ((e = resident_pairs<kDown, kWide>(cfg, &pairs)) != cudaSuccess) return e;
  // no more pairs than k-blocks there can be: every tile has a row, an expert at most one ragged tile
  const long long row_tiles = (long long)(p.rows + kMoeTileRows - 1) / kMoeTileRows + (p.E < p.rows ? p.E : p.rows);
  const long long blocks = row_tiles * ((p.N + C::kTileOut - 1) / C::kTileOut) * ((p.K + kKB - 1) / kKB);
  if (blocks < pairs) pairs = (int)blocks;
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, pair_kernel<kDown, kWide>, p, w0, w1, r64, r16);
}

}  // namespace

cudaError_t launch_moe_ffn(const MoeFfnArgs& a, cudaStream_t s) {
  if (moe_low(a.rows, a.E)) return launch_moe_ffn_low(a, s);
  CUtensorMap tm_g, tm_u, tm_x64, tm_x16, tm_d, tm_v64, tm_v16;
  if (!encode_weights(&tm_g, a.W_gate, a, 128) || !encode_weights(&tm_u, a.W_up, a, 128) ||
      !encode_weights(&tm_d, a.W_down_t, a, 64) || !encode_rows(&tm_x64, a.xs, a.rows, a.d, 64) ||
      !encode_rows(&tm_x16, a.xs, a.rows, a.d, 16) || !encode_rows(&tm_v64, a.v, a.rows, a.h, 64) ||
      !encode_rows(&tm_v16, a.v, a.rows, a.h, 16))
    return cudaErrorInvalidValue;
  const int part_n = moe_part_rows(a.rows);
  const Args gu{a.offsets, a.rows, a.E, a.h, a.d, a.act, static_cast<bf16*>(a.v), a.part, part_n, a.ctr, a.err};
  cudaError_t e = launch_pair<false, false>(gu, tm_g, tm_u, tm_x64, tm_x16, s);
  if (e != cudaSuccess) return e;
  const Args dn{a.offsets, a.rows, a.E,    a.d,    a.h, a.act, static_cast<bf16*>(a.ys), a.part,
                part_n,    a.ctr + 2 * kMoeMaxPairs, a.err};
  // Half as many tiles twice as wide, as long as they go round half the pairs when the rows spread
  // over the experts.  8 experts, d 4096, h 14336: 256 rows 459 us (256 columns: 499), 8192 rows 2073
  // (2335); 16 wide tiles (8 experts of 128 rows, d 1024, h 1024) 41 us (37).
  const int spread = a.E < a.rows ? a.E : a.rows, high = (a.rows + kMoeTileRows - 1) / kMoeTileRows;
  const long long wide = (long long)(spread > high ? spread : high) * ((a.d + 511) / 512);
  return wide * 4 >= sm_count() ? launch_pair<true, true>(dn, tm_d, tm_d, tm_v64, tm_v16, s)
                                : launch_pair<true, false>(dn, tm_d, tm_d, tm_v64, tm_v16, s);
}

}  // namespace csffn
