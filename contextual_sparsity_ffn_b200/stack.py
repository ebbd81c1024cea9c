"""Compositions of the library's entry points: a residual stack of sparse FFN layers, a Sirius
round (sparse drafts, then the dense verify of the chunk) and a residual stack of routed FFN layers.

These only sequence C-ABI calls (csffn_rmsnorm_bf16, csffn_calibrate_threshold,
csffn_dense_ffn_forward, csffn_cats_ffn_forward, csffn_block_norm, csffn_moe_*); every step of the
arithmetic runs in the library.

Stack ("SVD Contextual Sparsity Predictors for Fast LLM Inference", Table 12: the LLaMA-3-8B FFN
shape; the block structure is the plain reading): h <- h + FFN(bf16(RMSNorm(h))) per layer, the
residual h in fp32, the FFN output added in place (CSFFN_OUT_F32_ACCUMULATE).  Each layer's CATS
threshold is calibrated on the calibration vectors carried through the DENSE stack, RMSNorm'd at
that layer.

Sirius round ("SIRIUS : Contexual Sparisty with Correction for Efficient LLMs", "Approach"): the
sparse FFN drafts the chunk's tokens one at a time, then the full FFN (same weights) runs on the
whole chunk at once.

Routed stack (moe_stack): h <- res_scale h + out_scale gate * (rms(y) g_post) per layer, y the routed
FFN of rms(h) g_pre: the router picks k of the layer's experts for each token, the tokens are sorted
by expert, each expert's gated FFN runs on its rows, and the results come back weighted.  Any number
of tokens (a decode step or a prompt); nothing leaves the device, so a step can be captured.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import List, Optional

import torch

from . import _abi
from . import binding as cs

RMS_EPS = 1e-6
DENSE_CHUNK = 16  # tokens per csffn_dense_ffn_forward call (its batch limit)


def calibrate_stack(layers: List[cs.FFNLayer], h_cal: torch.Tensor, sparsity: float,
                    ws: torch.Tensor, keep_inputs: Optional[dict] = None) -> List[float]:
    """Per-layer CATS thresholds: h_cal [n, d] fp32 (device, updated in place) is carried through the
    dense stack; layer l's threshold is calibrated on bf16(RMSNorm(h_cal)) at that layer.  ws: a
    workspace of the layers' shape for batch 16.  ``keep_inputs``: a dict whose keys are layer
    numbers; each gets that layer's calibration input (bf16 bits on the host), for checks."""
    n, d = h_cal.shape
    xn = torch.empty(n, d, dtype=torch.bfloat16, device=h_cal.device)
    t_dev = torch.zeros(1, device=h_cal.device)
    ts = []
    for layer in layers:
        cs.rmsnorm_bf16(h_cal, RMS_EPS, xn)
        if keep_inputs is not None and len(ts) in keep_inputs:
            keep_inputs[len(ts)] = cs.to_numpy_bits(xn)
        cs.calibrate_threshold(layer, xn, sparsity, _abi.CAL_GLOBAL_ABS_ACT, t_dev)
        ts.append(float(t_dev.item()))
        for b0 in range(0, n, DENSE_CHUNK):
            b1 = min(n, b0 + DENSE_CHUNK)
            cs.dense_ffn_forward(layer, xn[b0:b1], h_cal[b0:b1], ws, out_mode=_abi.OUT_F32_ACCUMULATE)
    return ts


@dataclass
class StackBuffers:
    xn: torch.Tensor        # bf16 [B, d]: the current layer's input
    buf: cs.DecodeBuffers   # idx / count / a_val / workspace of one step


def stack_buffers(layer: cs.FFNLayer, B: int) -> StackBuffers:
    return StackBuffers(xn=torch.empty(B, layer.d, dtype=torch.bfloat16, device="cuda"),
                        buf=cs.DecodeBuffers.new(layer, B))


def sparse_stack(layers: List[cs.FFNLayer], ts: List[float], h: torch.Tensor, sb: StackBuffers,
                 record: Optional[list] = None, counts: Optional[list] = None) -> None:
    """One decode step through the stack: for each layer, xn = bf16(RMSNorm(h)), then
    h += CATS-FFN(xn) by csffn_cats_ffn_forward (accumulate mode).  With ``record`` (a list), each
    layer appends (xn, idx, a_val, h before, h after) copies on the host, for checks; with
    ``counts``, each layer appends the size of its active list (both synchronise every layer)."""
    for layer, t in zip(layers, ts):
        cs.rmsnorm_bf16(h, RMS_EPS, sb.xn)
        before = h.clone() if record is not None else None
        cs.cats_ffn_forward(layer, sb.xn, t, sb.buf.idx, sb.buf.count, sb.buf.a_val, h, sb.buf.ws,
                            out_mode=_abi.OUT_F32_ACCUMULATE)
        if record is not None:
            n = int(sb.buf.count.item())
            B = h.shape[0]
            record.append((cs.to_numpy_bits(sb.xn), sb.buf.idx[:n].cpu().numpy(),
                           sb.buf.a_val[:B, :n].cpu().numpy(), before.cpu().numpy(), h.cpu().numpy()))
        if counts is not None:
            counts.append(int(sb.buf.count.item()))


def dense_stack(layers: List[cs.FFNLayer], h: torch.Tensor, xn: torch.Tensor, ws: torch.Tensor) -> None:
    """The same step with every layer dense: xn = bf16(RMSNorm(h)), h += FFN(xn) by
    csffn_dense_ffn_forward (accumulate mode), batch <= 16."""
    for layer in layers:
        cs.rmsnorm_bf16(h, RMS_EPS, xn)
        cs.dense_ffn_forward(layer, xn, h, ws, out_mode=_abi.OUT_F32_ACCUMULATE)


def sirius_round(layer: cs.FFNLayer, x: torch.Tensor, t: float, sparse_out: torch.Tensor, dense_out: torch.Tensor,
                 buf: cs.DecodeBuffers, ws_dense: torch.Tensor, record: Optional[list] = None) -> None:
    """The FFN work of one Sirius round on a chunk x [T, d]: T one-token sparse steps
    (csffn_cats_ffn_forward, batch 1) into sparse_out [T, d], then one dense forward of the whole
    chunk (csffn_dense_ffn_forward, batch T <= 16) into dense_out [T, d].  With ``record``, each
    draft appends its (idx, a_val) on the host."""
    T = x.shape[0]
    for k in range(T):
        cs.cats_ffn_forward(layer, x[k:k + 1], t, buf.idx, buf.count, buf.a_val, sparse_out[k:k + 1], buf.ws)
        if record is not None:
            n = int(buf.count.item())
            record.append((buf.idx[:n].cpu().numpy(), buf.a_val[:1, :n].cpu().numpy()))
    cs.dense_ffn_forward(layer, x, dense_out, ws_dense)


def round_effective_density(counts, h: int) -> float:
    """Weight rows one Sirius round reads over the rows T dense decode steps read (FFN weights): each
    one-token draft reads all h rows of W_gate and the W_up and W_down^T rows of its n_t kept
    neurons, the verify reads the 3 h rows once for the chunk, and every draft counts as accepted.
    ``counts``: the drafts' n_t.  (sum_t (h + 2 n_t) + 3 h) / (3 h T)."""
    T = len(counts)
    return (sum(h + 2.0 * n for n in counts) + 3.0 * h) / (3.0 * h * T)


# ------------------------------------------------------------------------------ routed FFN stack

@dataclass
class MoEBlock:
    """One routed FFN layer of the stack: experts, router, and the norms around it (fp32 vectors)."""

    experts: cs.MoELayer
    w_router: torch.Tensor                      # bf16 [n_experts, d]
    k: int                                      # experts per token
    g_pre: Optional[torch.Tensor] = None        # [d] gain of the norm before the block
    g_post: Optional[torch.Tensor] = None       # [d] gain of the norm of its output; None: no such norm
    gate: Optional[torch.Tensor] = None         # [d] or [T, d] gate of its output
    sel_bias: Optional[torch.Tensor] = None     # [n_experts] added to the logits for the choice alone
    score: int = _abi.ROUTE_SOFTMAX
    renormalize: bool = True
    route_scale: float = 1.0
    res_scale: float = 1.0
    out_scale: float = 1.0


@dataclass
class MoEBuffers:
    """Device buffers of routed layers of one shape for T tokens (T may be 0)."""

    xn: torch.Tensor        # bf16 [T, d]: the layer's input
    logits: torch.Tensor    # fp32 [T, n_experts]
    ids: torch.Tensor       # int32 [T, k]
    weights: torch.Tensor   # fp32 [T, k]
    offsets: torch.Tensor   # int32 [n_experts + 1]
    order: torch.Tensor     # int32 [T * k]
    pos: torch.Tensor       # int32 [T, k]
    xs: torch.Tensor        # bf16 [T * k, d]: the rows by expert
    ys: torch.Tensor        # bf16 [T * k, d]: the experts' outputs
    y: torch.Tensor         # bf16 [T, d]: the layer's output
    ws: torch.Tensor

    @classmethod
    def new(cls, block: MoEBlock, T: int) -> "MoEBuffers":
        L, k, dev = block.experts, block.k, block.w_router.device

        def empty(*shape, dtype):
            return torch.empty(*shape, dtype=dtype, device=dev)
        bf, i32 = torch.bfloat16, torch.int32
        return cls(xn=empty(T, L.d, dtype=bf), logits=empty(T, L.n_experts, dtype=torch.float32),
                   ids=empty(T, k, dtype=i32), weights=empty(T, k, dtype=torch.float32),
                   offsets=empty(L.n_experts + 1, dtype=i32), order=empty(T * k, dtype=i32), pos=empty(T, k, dtype=i32),
                   xs=empty(T * k, L.d, dtype=bf), ys=empty(T * k, L.d, dtype=bf), y=empty(T, L.d, dtype=bf),
                   ws=cs.new_moe_workspace(L, max(1, T * k)))  # an empty batch takes the least


def moe_layer(block: MoEBlock, x: torch.Tensor, y: torch.Tensor, buf: MoEBuffers) -> None:
    """y [T, d] = the routed FFN of x [T, d] (bf16): router, sort, experts, weighted sum."""
    cs.moe_logits(x, block.w_router, buf.logits)
    cs.moe_route(buf.logits, buf.ids, buf.weights, bias=block.sel_bias, score=block.score,
                 renormalize=block.renormalize, scale=block.route_scale)
    cs.moe_dispatch(x, buf.ids, buf.offsets, buf.order, buf.pos, buf.xs, buf.ws)
    cs.moe_ffn_forward(block.experts, buf.xs, buf.offsets, buf.ys, buf.ws)
    cs.moe_combine(buf.ys, buf.pos, buf.weights, y)


def moe_stack(blocks: List[MoEBlock], h: torch.Tensor, buf: MoEBuffers) -> None:
    """One pass of h [T, d] (fp32, updated in place) through routed layers of one shape: the norm
    before the first layer, then for each layer its routed FFN and one pass that norms its output,
    updates h and norms the next layer's input."""
    cs.block_norm(h, None, None, buf.xn, g_pre=blocks[0].g_pre, eps=RMS_EPS)
    for i, b in enumerate(blocks):
        moe_layer(b, buf.xn, buf.y, buf)
        last = i + 1 == len(blocks)
        cs.block_norm(h, buf.y, h, None if last else buf.xn, g_post=b.g_post, gate=b.gate,
                      g_pre=None if last else blocks[i + 1].g_pre, res_scale=b.res_scale, out_scale=b.out_scale,
                      eps=RMS_EPS)
