// C entry points of the routed FFN and of the norms around a block: argument validation and
// dispatch.  Nothing here touches the data.
#include <cmath>

#include "common.cuh"
#include "kernels.h"

using namespace csffn;

namespace csffn {

MoeWs moe_ws_layout(int rows, int E, int h) {
  MoeWs L;
  L.err = ws_layout(8, 1, 1, 0).err;
  L.ctr = 1024;  // fixed: calls of fewer rows must not write where the counters of larger ones are
  size_t o = L.ctr + align_up(sizeof(uint32_t) * 2 * kMoeMaxPairs * 2, 256);
  L.hist = o;
  L.v = o;  // the dispatch's counts and the experts' v are never live at once
  // the most chunks any call of up to `rows` slots has
  const int chunks = (rows + kMoeChunk - 1) / kMoeChunk;
  const size_t hist = sizeof(int32_t) * (size_t)(chunks < kMoeMaxChunks ? chunks : kMoeMaxChunks) * E;
  const size_t v = sizeof(bf16) * moe_v_rows(rows, E) * h;
  o += align_up(hist > v ? hist : v, 256);
  L.part = o;
  if (h > 0) o += sizeof(float) * moe_part_floats(rows);
  L.total = o;
  return L;
}

}  // namespace csffn

namespace {

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
inline bool known_dtype(int t) { return t == CSFFN_BF16 || t == CSFFN_F32; }
inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline csffn_status cuda_status(cudaError_t e) { return e == cudaSuccess ? CSFFN_OK : CSFFN_ERR_CUDA; }
template <typename T>
T* at(void* ws, size_t off) { return reinterpret_cast<T*>(reinterpret_cast<char*>(ws) + off); }

// Whether two buffers share a byte.
struct Span {
  const void* p;
  size_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return x < y + b.bytes && y < x + a.bytes;
}

csffn_status check_width(int d, int multiple = 8) {
  if (d < 8 || d > CSFFN_MAX_D) return CSFFN_ERR_UNSUPPORTED_SHAPE;
  return d % multiple ? CSFFN_ERR_ALIGNMENT : CSFFN_OK;
}

bool known_out_mode(int m) {
  return m == CSFFN_OUT_BF16 || m == CSFFN_OUT_F32 || m == CSFFN_OUT_F32_ACCUMULATE;
}

// T tokens of k slots each: an argument error, or too many rows.
csffn_status check_slots(int T, int k) {
  if (T < 0 || k < 1 || k > CSFFN_MAX_TOPK) return CSFFN_ERR_INVALID_ARG;
  return (long long)T * k > CSFFN_MAX_MOE_ROWS ? CSFFN_ERR_UNSUPPORTED_SHAPE : CSFFN_OK;
}

csffn_status check_moe_layer(const csffn_moe_layer* L) {
  if (!L) return CSFFN_ERR_INVALID_ARG;
  if (L->act != CSFFN_ACT_SILU && L->act != CSFFN_ACT_RELU) return CSFFN_ERR_INVALID_ARG;
  if (L->n_experts < 1 || L->n_experts > CSFFN_MAX_EXPERTS) return CSFFN_ERR_INVALID_ARG;
  if (L->h < 8 || (long long)L->h * L->n_experts > CSFFN_MAX_H) return CSFFN_ERR_UNSUPPORTED_SHAPE;
  if (L->h % 8) return CSFFN_ERR_ALIGNMENT;
  return check_width(L->d);
}

}  // namespace

extern "C" {

csffn_status csffn_moe_logits(const void* x, const void* w_router, int T, int E, int d, float* logits, void* stream) {
  if (T < 0 || E < 1 || E > CSFFN_MAX_EXPERTS) return CSFFN_ERR_INVALID_ARG;
  csffn_status st = check_width(d);
  if (st != CSFFN_OK) return st;
  if (T > CSFFN_MAX_MOE_ROWS) return CSFFN_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return CSFFN_OK;
  if (!x || !w_router || !logits) return CSFFN_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_router) || !aligned4(logits)) return CSFFN_ERR_ALIGNMENT;
  return cuda_status(launch_moe_logits(x, w_router, T, E, d, logits, as_stream(stream)));
}

csffn_status csffn_moe_route(const void* logits, int ldtype, const float* sel_bias, int T, int E, int k, int score,
                             int renormalize, float scale, int32_t* ids, float* weights, void* stream) {
  if (!known_dtype(ldtype) || E < 1 || E > CSFFN_MAX_EXPERTS || std::isnan(scale)) return CSFFN_ERR_INVALID_ARG;
  if (score != CSFFN_ROUTE_SOFTMAX && score != CSFFN_ROUTE_SIGMOID) return CSFFN_ERR_INVALID_ARG;
  csffn_status st = check_slots(T, k);
  if (st != CSFFN_OK) return st;
  if (k > E) return CSFFN_ERR_INVALID_ARG;
  if (T == 0) return CSFFN_OK;
  if (!logits || !ids || !weights) return CSFFN_ERR_INVALID_ARG;
  if (((uintptr_t)logits & (ldtype == CSFFN_BF16 ? 1u : 3u)) || !aligned4(sel_bias) || !aligned4(ids) ||
      !aligned4(weights))
    return CSFFN_ERR_ALIGNMENT;
  const RouteArgs a{logits, sel_bias, T, E, k, score, renormalize != 0, scale, ids, weights};
  return cuda_status(launch_moe_route(a, ldtype, as_stream(stream)));
}

size_t csffn_moe_dispatch_workspace_size(int max_rows, int n_experts) {
  if (max_rows < 1 || max_rows > CSFFN_MAX_MOE_ROWS || n_experts < 1 || n_experts > CSFFN_MAX_EXPERTS) return 0;
  return moe_ws_layout(max_rows, n_experts, 0).total;
}

csffn_status csffn_moe_dispatch(const void* x, int xdtype, const int32_t* ids, int T, int k, int E, int d,
                                int32_t* offsets, int32_t* order, int32_t* pos, void* xs, void* ws,
                                size_t ws_bytes, void* stream) {
  if (!known_dtype(xdtype) || E < 1 || E > CSFFN_MAX_EXPERTS) return CSFFN_ERR_INVALID_ARG;
  csffn_status st = check_slots(T, k);
  if (st != CSFFN_OK) return st;
  if ((st = check_width(d, xdtype == CSFFN_BF16 ? 8 : 4)) != CSFFN_OK) return st;  // rows of whole 16-byte vectors
  if (!offsets) return CSFFN_ERR_INVALID_ARG;
  if (!aligned4(offsets)) return CSFFN_ERR_ALIGNMENT;
  if (T == 0) return cuda_status(cudaMemsetAsync(offsets, 0, sizeof(int32_t) * (E + 1), as_stream(stream)));
  if (!x || !ids || !order || !pos || !xs) return CSFFN_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(xs) || !aligned4(ids) || !aligned4(order) || !aligned4(pos))
    return CSFFN_ERR_ALIGNMENT;
  const MoeWs L = moe_ws_layout(T * k, E, 0);
  if (!ws || ws_bytes < L.total || !aligned16(ws)) return CSFFN_ERR_WORKSPACE;
  // The CTAs write while others still read, so no output may lie on an input, or on another output:
  // pos in the place of ids, of the same shape and type, is the one that invites it.
  const size_t R = (size_t)T * k, row = (size_t)d * (xdtype == CSFFN_BF16 ? 2 : 4);
  const Span in[2] = {{x, T * row}, {ids, 4 * R}};
  const Span out[4] = {{offsets, 4 * ((size_t)E + 1)}, {order, 4 * R}, {pos, 4 * R}, {xs, R * row}};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return CSFFN_ERR_INVALID_ARG;
    if (overlap(out[i], in[0]) || overlap(out[i], in[1])) return CSFFN_ERR_INVALID_ARG;
  }
  DispatchArgs a{};
  a.x = x;
  a.ids = ids;
  a.T = T;
  a.k = k;
  a.E = E;
  a.row_vecs = d / (xdtype == CSFFN_BF16 ? 8 : 4);
  a.offsets = offsets;
  a.order = order;
  a.pos = pos;
  a.xs = xs;
  a.hist = at<int32_t>(ws, L.hist);
  return cuda_status(launch_moe_dispatch(a, as_stream(stream)));
}

size_t csffn_moe_workspace_size(const csffn_moe_layer* layer, int max_rows) {
  if (check_moe_layer(layer) != CSFFN_OK || max_rows < 1 || max_rows > CSFFN_MAX_MOE_ROWS) return 0;
  return moe_ws_layout(max_rows, layer->n_experts, layer->h).total;
}

csffn_status csffn_moe_ffn_forward(const csffn_moe_layer* layer, const void* xs, const int32_t* offsets, int rows,
                                   void* ys, void* ws, size_t ws_bytes, void* stream) {
  csffn_status st = check_moe_layer(layer);
  if (st != CSFFN_OK) return st;
  if (rows < 0) return CSFFN_ERR_INVALID_ARG;
  if (rows > CSFFN_MAX_MOE_ROWS) return CSFFN_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return CSFFN_OK;
  if (!xs || !offsets || !ys || !layer->w_gate || !layer->w_up || !layer->w_down_t) return CSFFN_ERR_INVALID_ARG;
  if (!aligned16(xs) || !aligned16(ys) || !aligned4(offsets) || !aligned16(layer->w_gate) ||
      !aligned16(layer->w_up) || !aligned16(layer->w_down_t))
    return CSFFN_ERR_ALIGNMENT;
  const MoeWs L = moe_ws_layout(rows, layer->n_experts, layer->h);
  if (!ws || ws_bytes < L.total || !aligned16(ws)) return CSFFN_ERR_WORKSPACE;
  MoeFfnArgs a{};
  a.W_gate = layer->w_gate;
  a.W_up = layer->w_up;
  a.W_down_t = layer->w_down_t;
  a.xs = xs;
  a.offsets = offsets;
  a.d = layer->d;
  a.h = layer->h;
  a.E = layer->n_experts;
  a.act = layer->act;
  a.rows = rows;
  a.v = at<void>(ws, L.v);
  a.part = at<float>(ws, L.part);
  a.ctr = at<uint32_t>(ws, L.ctr);
  a.ys = ys;
  a.err = at<uint32_t>(ws, L.err);
  return cuda_status(launch_moe_ffn(a, as_stream(stream)));
}

csffn_status csffn_moe_combine(const void* ys, const int32_t* pos, const float* weights, int T, int k, int rows, int d,
                               void* out, int out_mode, void* stream) {
  if (!known_out_mode(out_mode) || rows < 0) return CSFFN_ERR_INVALID_ARG;
  csffn_status st = check_slots(T, k);
  if (st != CSFFN_OK) return st;
  if ((st = check_width(d)) != CSFFN_OK) return st;
  if (rows > CSFFN_MAX_MOE_ROWS) return CSFFN_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return CSFFN_OK;
  if ((!ys && rows > 0) || !pos || !out) return CSFFN_ERR_INVALID_ARG;
  if (!aligned16(ys) || !aligned16(out) || !aligned4(pos) || !aligned4(weights)) return CSFFN_ERR_ALIGNMENT;
  const CombineArgs a{ys, pos, weights, T, k, rows, d, out, out_mode};
  return cuda_status(launch_moe_combine(a, as_stream(stream)));
}

csffn_status csffn_block_norm(const float* h, const void* y, int ydtype, const float* g_post, const float* gate,
                              int gate_rows, const float* g_pre, float res_scale, float out_scale, float eps, int T,
                              int d, float* h_out, void* xn, int xdtype, void* stream) {
  if (T < 0 || !known_dtype(ydtype) || !known_dtype(xdtype)) return CSFFN_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || std::isnan(res_scale) || std::isnan(out_scale)) return CSFFN_ERR_INVALID_ARG;
  csffn_status st = check_width(d);
  if (st != CSFFN_OK) return st;
  if (T > CSFFN_MAX_MOE_ROWS) return CSFFN_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return CSFFN_OK;
  if (!h || (!h_out && !xn)) return CSFFN_ERR_INVALID_ARG;
  if (!y && (g_post || gate)) return CSFFN_ERR_INVALID_ARG;  // nothing to scale
  if (gate && gate_rows != 1 && gate_rows != T) return CSFFN_ERR_INVALID_ARG;
  if (xn && (xn == h || xn == h_out)) return CSFFN_ERR_INVALID_ARG;
  if (!aligned16(h) || !aligned16(y) || !aligned16(g_post) || !aligned16(gate) || !aligned16(g_pre) ||
      !aligned16(h_out) || !aligned16(xn))
    return CSFFN_ERR_ALIGNMENT;
  BlockNormArgs a{};
  a.h = h;
  a.y = y;
  a.g_post = g_post;
  a.gate = gate;
  a.g_pre = g_pre;
  a.h_out = h_out;
  a.xn = xn;
  a.T = T;
  a.d = d;
  a.gate_per_token = gate && gate_rows != 1;
  a.res_scale = res_scale;
  a.out_scale = out_scale;
  a.eps = eps;
  return cuda_status(launch_block_norm(a, ydtype, xdtype, as_stream(stream)));
}

}  // extern "C"
