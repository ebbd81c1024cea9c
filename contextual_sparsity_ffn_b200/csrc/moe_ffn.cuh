// What the two forms of the experts' FFN share (moe_ffn.cu: many rows, moe_ffn_low.cu: few): the tiles
// worked out from the offsets, their split over the CTAs, and the activation.
#pragma once

#include "common.cuh"
#include "fused_end.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace csffn {
namespace moe {

constexpr int kKB = 64;                            // contraction elements per stage
constexpr uint32_t kRowBytes = kKB * 2;            // one row of a stage's tile
constexpr int kMaxParts = 8, kMaxPartsTall = 4;                       // parts of a tile
constexpr int kMinSaved = 16, kMinSavedRun = 24, kMinSavedTall = 24;  // k-blocks

struct Args {
  const int32_t* offsets;
  int rows, E, N, K, act;  // N outputs per expert, K contraction
  bf16* out;               // [rows, N]; gate/up with few rows: [2][rows, N], high and low parts
  float* part;             // split tiles' parts
  int part_n;              // most rows of a tile of this call
  uint32_t* ctr;           // parts done of the split tiles
  uint32_t* err;
};

// Every expert's rows and tiles, worked out once per CTA: lo[e] .. lo[e + 1] are expert e's rows,
// tp[e] the row tiles of the experts before it.
struct Plan {
  int lo[CSFFN_MAX_EXPERTS + 1];
  int tp[CSFFN_MAX_EXPERTS + 1];
};

// By one warp, from the raw offsets in p->lo: each lane takes a few consecutive entries.
template <int kTileRows>
__device__ inline void make_plan(const Args& a, Plan* p) {
  const int lane = threadIdx.x & 31, per = (a.E + kWarp) / kWarp;  // E + 1 entries
  const int e0 = min(lane * per, a.E + 1), e1 = min(e0 + per, a.E + 1);
  int top = 0;  // the largest offset up to here: ascending order
  for (int e = e0; e < e1; ++e) {
    top = max(top, min(p->lo[e], a.rows));
    p->lo[e] = top;
  }
#pragma unroll
  for (int o = 1; o < kWarp; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, top, o);
    if (lane >= o) top = max(top, u);
  }
  int before = __shfl_up_sync(0xffffffffu, top, 1);  // of the entries of lower lanes
  if (lane == 0) before = 0;
  // entry e closes expert e - 1
  int tiles = 0, prev = before;
  for (int e = e0; e < e1; ++e) {
    const int v = max(p->lo[e], before);
    p->lo[e] = v;
    if (e > 0) tiles += (v - prev + kTileRows - 1) / kTileRows;
    p->tp[e] = tiles;
    prev = v;
  }
  int sum = tiles;
#pragma unroll
  for (int o = 1; o < kWarp; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += u;
  }
  for (int e = e0; e < e1; ++e) p->tp[e] += sum - tiles;
}

struct Tile {
  int e, m;        // expert, output block
  int row0, row1;  // rows
  int n;           // N of its MMAs: the rows rounded up to 32
  bool once;       // no other tile reads its weights
};

__device__ __forceinline__ Tile find_tile(const Plan& p, int E, int mb, int i) {
  const int q = i / mb;
  int a = 0, b = E;  // tp[a] <= q < tp[b]
  while (b - a > 1) {
    const int c = (a + b) >> 1;
    if (p.tp[c] <= q)
      a = c;
    else
      b = c;
  }
  const int nt = p.tp[a + 1] - p.tp[a], r = i - p.tp[a] * mb;
  const int cnt = p.lo[a + 1] - p.lo[a];
  const int height = ((cnt + nt - 1) / nt + 31) / 32 * 32;
  Tile t;
  t.e = a;
  t.m = r / nt;
  t.row0 = p.lo[a] + (r % nt) * height;
  t.row1 = min(t.row0 + height, p.lo[a + 1]);
  t.n = (t.row1 - t.row0 + 31) / 32 * 32;
  t.once = nt == 1;
  return t;
}

// The work of one pair of CTAs (few rows: of one CTA) in order: (tile, k-blocks [kb0, kb1)).
struct Items {
  int pair, pairs, n_kb, n_whole, left;  // tiles [0, n_whole) go round whole, `left` after them
  int split;                             // parts of a left-over tile, or 0: one run for all of them
  int next;                              // next whole tile
  int it, it1;                           // this pair's k-blocks of the run
  int tile, kb0, kb1;                    // the current item
  __device__ Items(int pair_, int pairs_, int n_kb_, int n_tiles, bool low)
      : pair(pair_), pairs(pairs_), n_kb(n_kb_) {
    n_whole = n_tiles / pairs * pairs;
    left = n_tiles - n_whole;
    // A part costs its accumulators' way through L2 and about 4 us at the end, so tiles are cut only where
    // enough k-blocks less are to be done.  us, as it stands / never cut / cut wherever that is possible:
    //   low, parts, 16: one token, d 2048, h 1024, 1 expert 21.7 / 25.0 / 22.6, 4 experts 24.7 / 25.5 / 27.0;
    //   low, a run, 24: one expert, d 4096, h 5376 (28 saved) 40.6 / 43.4 / 40.6, 8 experts, d 2048, h 1024
    //     (5 saved) 30.7 / 30.7 / 39.5;
    //   tall, 24: 300 rows, d 8192, h 1024 48.1 / 80.4 / 48.0, 1024 rows of 8 experts, d 1024, h 1024
    //     (8 saved) 28.9 / 28.9 / 37.7.  At the border it is not exact: 512 rows, d 2048, h 2048 (24 saved)
    //     56.7 / 46.5 / 56.7.
    split = left ? min(min(pairs / left, low ? kMaxParts : kMaxPartsTall), n_kb) : 1;
    if (n_kb - n_kb / split < (low ? kMinSaved : kMinSavedTall)) split = 1;
    if (low && left && pairs / left == 1 && n_kb - (int)((long long)n_kb * left / pairs) >= kMinSavedRun) split = 0;
    next = pair;
    it = split == 0 ? run_start(pair) : 0;
    it1 = split == 0 ? run_start(pair + 1) : 0;
  }
  // the run: left * n_kb k-blocks, more than half as many tiles as pairs, so no pair's share is empty
  __device__ int run_start(int q) const { return (int)((long long)q * left * n_kb / pairs); }
  __device__ int run_owner(int j) const { return (int)(((long long)(j + 1) * pairs - 1) / (left * n_kb)); }
  __device__ bool advance() {
    kb0 = 0;
    kb1 = n_kb;
    tile = next;
    if (next < n_whole) {
      next += pairs;
      return true;
    }
    if (split == 0) {
      if (it >= it1) return false;
      tile = n_whole + it / n_kb;
      kb0 = it % n_kb;
      kb1 = min(n_kb, kb0 + (it1 - it));
      it += kb1 - kb0;
      return true;
    }
    const int q = next - n_whole;  // this pair's number, until its last item is out
    if (q >= left * split) return false;
    next = 0x7fffffff;
    tile = n_whole + q % left;
    kb0 = (q / left) * n_kb / split;
    kb1 = (q / left + 1) * n_kb / split;
    return true;
  }
  __device__ bool whole() const { return kb1 - kb0 == n_kb; }
  __device__ int left_tile() const { return tile - n_whole; }
  // the parts of the current tile, and where part r is kept (at most 2 * pairs places)
  __device__ int first_pair() const { return run_owner(left_tile() * n_kb); }
  __device__ int parts() const { return split ? split : run_owner(left_tile() * n_kb + n_kb - 1) - first_pair() + 1; }
  __device__ int place(int r) const {
    if (split) return left_tile() * split + r;
    const int q = first_pair() + r;
    return 2 * q + (run_start(q) >= left_tile() * n_kb ? 0 : 1);
  }
  __device__ int my_place() const {
    if (split) return left_tile() * split + pair / left;
    return 2 * pair + (run_start(pair) >= left_tile() * n_kb ? 0 : 1);
  }
};

struct Ring {
  int slot = 0;
  uint32_t round = 0;
  __device__ void next(int n) {
    if (++slot == n) {
      slot = 0;
      ++round;
    }
  }
};

// The activation of a value that goes on in bf16.  SiLU as z * 1 / (1 + 2^(-z log2 e)) on the
// approximate exponential and reciprocal instructions: a few fp32 steps, far below the rounding, and
// with 4 other operations per value the least the epilogue can do (it is bound by these two: 16
// cycles per warp and value of the special-function units).
__device__ __forceinline__ float act_fast(float z, int act) {
  if (act != CSFFN_ACT_SILU) return fmaxf(z, 0.0f);
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.44269504f * z));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return z * r;
}

inline bool encode(CUtensorMap* tm, const void* base, int rank, const cuuint64_t* dim, const cuuint64_t* stride,
            const cuuint32_t* box) {
  TensorMapEncodeFn fn = tensor_map_encoder();
  const cuuint32_t ones[3] = {1, 1, 1};
  return fn && fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), dim, stride, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Weights [E, h, d], boxes of 64 x `high`.
inline bool encode_weights(CUtensorMap* tm, const void* base, const MoeFfnArgs& a, cuuint32_t high) {
  const cuuint64_t dim[3] = {(cuuint64_t)a.d, (cuuint64_t)a.h, (cuuint64_t)a.E};
  const cuuint64_t stride[2] = {(cuuint64_t)a.d * 2, (cuuint64_t)a.h * a.d * 2};
  const cuuint32_t box[3] = {64, high, 1};
  return encode(tm, base, 3, dim, stride, box);
}

// Rows [rows, width], boxes of 64 x `high`.
inline bool encode_rows(CUtensorMap* tm, const void* base, int rows, int width, cuuint32_t high) {
  const cuuint64_t dim[2] = {(cuuint64_t)width, (cuuint64_t)rows};
  const cuuint64_t stride[1] = {(cuuint64_t)width * 2};
  const cuuint32_t box[2] = {64, high};
  return encode(tm, base, 2, dim, stride, box);
}

}  // namespace moe
}  // namespace csffn
