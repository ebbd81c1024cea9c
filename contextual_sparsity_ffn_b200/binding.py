"""Thin torch-facing binding of libcsffn: argument marshalling only.

Every function takes CUDA tensors, passes their device pointers and the
current CUDA stream to the C entry point of the same name, and raises
``CsffnError`` on a non-zero status.  No arithmetic of the method happens
here; PyTorch only provides device memory and streams.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass, field
from typing import Optional

import numpy as np
import torch

from . import _abi
from ._abi import CsffnError, check, load  # noqa: F401

TORCH_DTYPE = {_abi.BF16: torch.bfloat16, _abi.F32: torch.float32}


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("csffn takes CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("csffn takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


@dataclass
class FFNLayer:
    """Device copy of one gated FFN layer plus the csffn_layer struct pointing at it."""

    w_gate: torch.Tensor
    w_up: torch.Tensor
    w_down_t: torch.Tensor
    act: int
    bias: Optional[torch.Tensor] = None
    c: _abi.Layer = field(default=None, repr=False)

    def __post_init__(self):
        h, d = self.w_gate.shape
        wdtype = _abi.BF16 if self.w_gate.dtype == torch.bfloat16 else _abi.F32
        self.c = _abi.Layer(d, h, wdtype, self.act, self.w_gate.data_ptr(), self.w_up.data_ptr(),
                            self.w_down_t.data_ptr(), self.bias.data_ptr() if self.bias is not None else None)

    @property
    def d(self) -> int:
        return self.c.d

    @property
    def h(self) -> int:
        return self.c.h

    @property
    def wdtype(self) -> int:
        return self.c.wdtype

    @property
    def dtype(self) -> torch.dtype:
        return TORCH_DTYPE[self.c.wdtype]

    @classmethod
    def from_spec(cls, spec, device="cuda") -> "FFNLayer":
        """Upload a synth.LayerSpec (bf16 bits as uint16, or float32) to the device."""
        def up(a):
            return to_device(a, device)
        act = _abi.ACT_SILU if spec.act == "silu" else _abi.ACT_RELU
        bias = torch.from_numpy(np.ascontiguousarray(spec.bias)).to(device) if spec.bias is not None else None
        return cls(up(spec.w_gate), up(spec.w_up), up(spec.w_down_t), act, bias)

    def ref(self):
        return ctypes.byref(self.c)


def to_device(a: np.ndarray, device="cuda") -> torch.Tensor:
    """numpy operand -> device tensor: uint16 arrays are bf16 bit patterns."""
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).to(device).view(torch.bfloat16)
    return torch.from_numpy(a).to(device)


def to_numpy_bits(t: torch.Tensor) -> np.ndarray:
    """device tensor -> numpy (bf16 as uint16 bit patterns)."""
    t = t.detach().cpu().contiguous()
    if t.dtype == torch.bfloat16:
        return t.view(torch.int16).numpy().view(np.uint16)
    return t.numpy()


# ------------------------------------------------------------------------------ workspace

def workspace_size(layer: FFNLayer, max_batch: int, max_rank: int = 0) -> int:
    n = load().csffn_workspace_size(layer.ref(), max_batch, max_rank)
    if n == 0:
        raise CsffnError(_abi.ERR_INVALID_ARG, "csffn_workspace_size")
    return int(n)


def workspace_init(ws: torch.Tensor, stream=None) -> None:
    check(load().csffn_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
          "csffn_workspace_init")


def new_workspace(layer: FFNLayer, max_batch: int, max_rank: int = 0, device="cuda") -> torch.Tensor:
    ws = torch.empty(workspace_size(layer, max_batch, max_rank), dtype=torch.uint8, device=device)
    workspace_init(ws)
    return ws


def check_status(ws: torch.Tensor, stream=None) -> int:
    """Synchronise and return the device-side status (0 = ok, 6 = a bounded wait timed out)."""
    return int(load().csffn_check_status(_ptr(ws), _stream(stream)))


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


# ------------------------------------------------------------------------------ decode path

def gate_mask(layer: FFNLayer, x: torch.Tensor, t: float, idx: torch.Tensor, count: torch.Tensor,
              a_val: torch.Tensor, ws: torch.Tensor, cand_idx: Optional[torch.Tensor] = None,
              cand_count: Optional[torch.Tensor] = None, stream=None) -> None:
    B = x.shape[0] if x.dim() == 2 else 1
    check(load().csffn_gate_mask(layer.ref(), _ptr(x), B, float(t), _ptr(cand_idx), _ptr(cand_count),
                                 _ptr(idx), _ptr(count), _ptr(a_val), _ptr(ws), _nbytes(ws), _stream(stream)),
          "csffn_gate_mask")


def sparse_ffn_forward(layer: FFNLayer, x: torch.Tensor, idx: torch.Tensor, count: torch.Tensor,
                       a_val: torch.Tensor, out: torch.Tensor, ws: torch.Tensor,
                       out_mode: Optional[int] = None, stream=None) -> None:
    B = x.shape[0] if x.dim() == 2 else 1
    if out_mode is None:
        out_mode = _abi.OUT_BF16 if out.dtype == torch.bfloat16 else _abi.OUT_F32
    check(load().csffn_sparse_ffn_forward(layer.ref(), _ptr(x), B, _ptr(idx), _ptr(count), _ptr(a_val),
                                          _ptr(out), out_mode, _ptr(ws), _nbytes(ws), _stream(stream)),
          "csffn_sparse_ffn_forward")


def cats_ffn_forward(layer: FFNLayer, x: torch.Tensor, t: float, idx: torch.Tensor, count: torch.Tensor,
                     a_val: torch.Tensor, out: torch.Tensor, ws: torch.Tensor, out_mode: Optional[int] = None,
                     cand_idx: Optional[torch.Tensor] = None, cand_count: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    B = x.shape[0] if x.dim() == 2 else 1
    if out_mode is None:
        out_mode = _abi.OUT_BF16 if out.dtype == torch.bfloat16 else _abi.OUT_F32
    check(load().csffn_cats_ffn_forward(layer.ref(), _ptr(x), B, float(t), _ptr(cand_idx), _ptr(cand_count),
                                        _ptr(idx), _ptr(count), _ptr(a_val), _ptr(out), out_mode, _ptr(ws),
                                        _nbytes(ws), _stream(stream)),
          "csffn_cats_ffn_forward")


def _host_ptr(t: torch.Tensor):
    if t.is_cuda:
        raise ValueError("csffn host entry points take CPU tensors (pinned for asynchronous copies)")
    if not t.is_contiguous():
        raise ValueError("csffn takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def cats_ffn_forward_host(layer: FFNLayer, x_host: torch.Tensor, t: float, idx: torch.Tensor,
                          count: torch.Tensor, a_val: torch.Tensor, out_host: torch.Tensor, ws: torch.Tensor,
                          stream=None) -> None:
    """csffn_cats_ffn_forward_host: x_host and out_host are CPU tensors.  Pinned (page-locked)
    tensors are read and written by the step itself over the host link; pageable ones are staged
    through the workspace by copies.  The result is in out_host once the step has completed on the
    stream, and x_host must stay unchanged until then."""
    B = x_host.shape[0] if x_host.dim() == 2 else 1
    out_mode = _abi.OUT_BF16 if out_host.dtype == torch.bfloat16 else _abi.OUT_F32
    check(load().csffn_cats_ffn_forward_host(layer.ref(), _host_ptr(x_host), B, float(t), _ptr(idx), _ptr(count),
                                             _ptr(a_val), _host_ptr(out_host), out_mode, _ptr(ws), _nbytes(ws),
                                             _stream(stream)),
          "csffn_cats_ffn_forward_host")


def dense_ffn_forward(layer: FFNLayer, x: torch.Tensor, out: torch.Tensor, ws: torch.Tensor,
                      out_mode: Optional[int] = None, stream=None) -> None:
    B = x.shape[0] if x.dim() == 2 else 1
    if out_mode is None:
        out_mode = _abi.OUT_BF16 if out.dtype == torch.bfloat16 else _abi.OUT_F32
    check(load().csffn_dense_ffn_forward(layer.ref(), _ptr(x), B, _ptr(out), out_mode, _ptr(ws),
                                         _nbytes(ws), _stream(stream)),
          "csffn_dense_ffn_forward")


def predict_lowrank(layer: FFNLayer, x: torch.Tensor, u_rt: torch.Tensor, v_r: torch.Tensor,
                    tau: torch.Tensor, cand_idx: torch.Tensor, cand_count: torch.Tensor,
                    ws: torch.Tensor, stream=None) -> None:
    B = x.shape[0] if x.dim() == 2 else 1
    rank = u_rt.shape[0]
    check(load().csffn_predict_lowrank(layer.ref(), _ptr(x), B, rank, _ptr(u_rt), _ptr(v_r), _ptr(tau),
                                       _ptr(cand_idx), _ptr(cand_count), _ptr(ws), _nbytes(ws),
                                       _stream(stream)),
          "csffn_predict_lowrank")


def svd_ffn_forward(layer: FFNLayer, x: torch.Tensor, u_rt: torch.Tensor, v_r: torch.Tensor, tau: torch.Tensor,
                    t: float, idx: torch.Tensor, count: torch.Tensor, a_val: torch.Tensor, out: torch.Tensor,
                    ws: torch.Tensor, out_mode: Optional[int] = None, stream=None, parallel: bool = False) -> None:
    """csffn_svd_ffn_forward, or with parallel=True csffn_svd_ffn_forward_parallel (same outputs)."""
    B = x.shape[0] if x.dim() == 2 else 1
    rank = u_rt.shape[0]
    if out_mode is None:
        out_mode = _abi.OUT_BF16 if out.dtype == torch.bfloat16 else _abi.OUT_F32
    name = "csffn_svd_ffn_forward_parallel" if parallel else "csffn_svd_ffn_forward"
    check(getattr(load(), name)(layer.ref(), _ptr(x), B, rank, _ptr(u_rt), _ptr(v_r), _ptr(tau), float(t),
                                _ptr(idx), _ptr(count), _ptr(a_val), _ptr(out), out_mode, _ptr(ws), _nbytes(ws),
                                _stream(stream)),
          name)


def calibrate_workspace_size(layer: FFNLayer, n: int, mode: int, rank: int = 0) -> int:
    s = load().csffn_calibrate_workspace_size(layer.ref(), n, mode, rank)
    if s == 0:
        raise CsffnError(_abi.ERR_INVALID_ARG, "csffn_calibrate_workspace_size")
    return int(s)


def calibrate_threshold(layer: FFNLayer, x_cal: torch.Tensor, target_sparsity: float, mode: int,
                        t_out: torch.Tensor, u_rt: Optional[torch.Tensor] = None,
                        v_r: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                        stream=None) -> None:
    n = x_cal.shape[0]
    rank = u_rt.shape[0] if u_rt is not None else 0
    if ws is None:
        ws = torch.empty(calibrate_workspace_size(layer, n, mode, rank), dtype=torch.uint8, device=x_cal.device)
    check(load().csffn_calibrate_threshold(layer.ref(), _ptr(x_cal), n, float(target_sparsity), mode,
                                           _ptr(u_rt), _ptr(v_r), rank, _ptr(t_out), _ptr(ws), _nbytes(ws),
                                           _stream(stream)),
          "csffn_calibrate_threshold")


def kth_smallest(values: torch.Tensor, k: int, out: torch.Tensor, ws: Optional[torch.Tensor] = None,
                 stream=None) -> None:
    if ws is None:
        ws = torch.empty(int(load().csffn_kth_workspace_size()), dtype=torch.uint8, device=values.device)
    check(load().csffn_kth_smallest(_ptr(values), values.numel(), int(k), _ptr(out), _ptr(ws), _nbytes(ws),
                                    _stream(stream)),
          "csffn_kth_smallest")


def rmsnorm_bf16(h: torch.Tensor, eps: float, xn: torch.Tensor, stream=None) -> None:
    B, d = h.shape
    check(load().csffn_rmsnorm_bf16(_ptr(h), B, d, float(eps), _ptr(xn), _stream(stream)), "csffn_rmsnorm_bf16")


def selftest_timeout(ws: torch.Tensor, spin_limit: int, stream=None) -> None:
    check(load().csffn_selftest_timeout(_ptr(ws), _nbytes(ws), int(spin_limit), _stream(stream)),
          "csffn_selftest_timeout")


# ------------------------------------------------------------------------------ routed FFN, block norm

# A decode step makes one of these calls every few microseconds, so each argument is checked by one
# expression and explained only when that fails.

_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_CODE = {_BF16: _abi.BF16, _F32: _abi.F32}


def _device(t: torch.Tensor) -> int:
    if not t.is_cuda:
        raise ValueError("csffn takes CUDA tensors")
    return t.get_device()


def _code(t: torch.Tensor, name: str) -> int:
    code = _CODE.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, not {t.dtype}")
    return code


def _arg(t: Optional[torch.Tensor], name: str, shape, dtype: torch.dtype, dev: int):
    """Pointer of a contiguous tensor of this shape and dtype on device `dev`; None stays None."""
    if t is None:
        return None
    if t.shape == shape and t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError("csffn takes contiguous tensors")
    raise ValueError(f"{name} must be on the device of the call's other tensors (cuda:{dev})")


def _run(name: str, dev: int, stream, *args) -> None:
    """Calls the entry point on `stream`, or on the current stream of device `dev`, which is made
    current for the call (kernels launch on the current device)."""
    s = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev)
    fn = getattr(load(), name)
    if torch._C._cuda_getDevice() == dev:
        status = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, s)
    if status != _abi.OK:
        raise CsffnError(status, name)


def _matrix(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, not {t.dim()}")
    return t.shape


@dataclass
class MoELayer:
    """Device copy of one routed FFN layer (bf16 [E, h, d] matrices) plus the csffn_moe_layer struct."""

    w_gate: torch.Tensor
    w_up: torch.Tensor
    w_down_t: torch.Tensor
    act: int
    c: _abi.MoELayer = field(default=None, repr=False)

    def __post_init__(self):
        if self.w_gate.dim() != 3:
            raise ValueError("w_gate must be [n_experts, h, d]")
        dev = _device(self.w_gate)
        E, h, d = self.w_gate.shape
        ptrs = [_arg(w, n, self.w_gate.shape, _BF16, dev)
                for w, n in ((self.w_gate, "w_gate"), (self.w_up, "w_up"), (self.w_down_t, "w_down_t"))]
        self.c = _abi.MoELayer(d, h, E, self.act, *ptrs)

    @property
    def d(self) -> int:
        return self.c.d

    @property
    def h(self) -> int:
        return self.c.h

    @property
    def n_experts(self) -> int:
        return self.c.n_experts

    def ref(self):
        return ctypes.byref(self.c)


def moe_workspace_size(layer: MoELayer, max_rows: int) -> int:
    n = load().csffn_moe_workspace_size(layer.ref(), max_rows)
    if n == 0:
        raise CsffnError(_abi.ERR_INVALID_ARG, "csffn_moe_workspace_size")
    return int(n)


def moe_dispatch_workspace_size(max_rows: int, n_experts: int) -> int:
    n = load().csffn_moe_dispatch_workspace_size(max_rows, n_experts)
    if n == 0:
        raise CsffnError(_abi.ERR_INVALID_ARG, "csffn_moe_dispatch_workspace_size")
    return int(n)


def new_moe_workspace(layer: MoELayer, max_rows: int) -> torch.Tensor:
    """An initialised workspace for moe_ffn_forward and moe_dispatch of up to max_rows = T * k rows."""
    ws = torch.empty(moe_workspace_size(layer, max_rows), dtype=torch.uint8, device=layer.w_gate.device)
    with torch.cuda.device(ws.device):
        workspace_init(ws)
    return ws


def new_moe_dispatch_workspace(max_rows: int, n_experts: int, device="cuda") -> torch.Tensor:
    """A workspace for moe_dispatch alone (it needs no initialisation)."""
    return torch.empty(moe_dispatch_workspace_size(max_rows, n_experts), dtype=torch.uint8, device=device)


def moe_logits(x: torch.Tensor, w_router: torch.Tensor, logits: torch.Tensor, stream=None) -> None:
    """logits [T, E] fp32 = x [T, d] . w_router [E, d]^T (bf16 operands, fp32 sums)."""
    (T, d), (E, _) = _matrix(x, "x"), _matrix(w_router, "w_router")
    dev = _device(x)
    _run("csffn_moe_logits", dev, stream, _arg(x, "x", (T, d), _BF16, dev), _arg(w_router, "w_router", (E, d), _BF16, dev),
         T, E, d, _arg(logits, "logits", (T, E), _F32, dev))


def moe_route(logits: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, bias: Optional[torch.Tensor] = None,
              score: int = _abi.ROUTE_SOFTMAX, renormalize: bool = True, scale: float = 1.0, stream=None) -> None:
    """The k = ids.shape[1] experts of every token, by logits [T, E] (plus bias [E] for the choice
    alone), and their weights; see csffn_moe_route."""
    (T, E), (_, k) = _matrix(logits, "logits"), _matrix(ids, "ids")
    dev = _device(logits)
    code = _code(logits, "logits")
    _run("csffn_moe_route", dev, stream, _arg(logits, "logits", (T, E), logits.dtype, dev), code,
         _arg(bias, "bias", (E,), _F32, dev), T, E, k, score, renormalize, scale, _arg(ids, "ids", (T, k), _I32, dev),
         _arg(weights, "weights", (T, k), _F32, dev))


def moe_dispatch(x: torch.Tensor, ids: torch.Tensor, offsets: torch.Tensor, order: torch.Tensor, pos: torch.Tensor,
                 xs: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """Sorts the token slots by expert and gathers the tokens' rows into xs [T * k, d]; the number of
    experts is offsets.shape[0] - 1.  See csffn_moe_dispatch."""
    (T, d), (_, k) = _matrix(x, "x"), _matrix(ids, "ids")
    E, n = offsets.numel() - 1, ws.numel()
    dev = _device(x)
    code = _code(x, "x")
    _run("csffn_moe_dispatch", dev, stream, _arg(x, "x", (T, d), x.dtype, dev), code, _arg(ids, "ids", (T, k), _I32, dev),
         T, k, E, d, _arg(offsets, "offsets", (E + 1,), _I32, dev), _arg(order, "order", (T * k,), _I32, dev),
         _arg(pos, "pos", (T, k), _I32, dev), _arg(xs, "xs", (T * k, d), x.dtype, dev), _arg(ws, "ws", (n,), _U8, dev), n)


def moe_ffn_forward(layer: MoELayer, xs: torch.Tensor, offsets: torch.Tensor, ys: torch.Tensor, ws: torch.Tensor,
                    stream=None) -> None:
    """The experts' gated FFNs on the sorted rows xs [rows, d] -> ys [rows, d] (bf16); see
    csffn_moe_ffn_forward.  ws: new_moe_workspace(layer, rows or more)."""
    rows, _ = _matrix(xs, "xs")
    dev, n = _device(xs), ws.numel()
    if layer.w_gate.get_device() != dev:
        raise ValueError("the layer must be on the device of the rows")
    _run("csffn_moe_ffn_forward", dev, stream, layer.ref(), _arg(xs, "xs", (rows, layer.d), _BF16, dev),
         _arg(offsets, "offsets", (layer.n_experts + 1,), _I32, dev), rows, _arg(ys, "ys", (rows, layer.d), _BF16, dev),
         _arg(ws, "ws", (n,), _U8, dev), n)


def moe_combine(ys: torch.Tensor, pos: torch.Tensor, weights: Optional[torch.Tensor], out: torch.Tensor,
                out_mode: Optional[int] = None, stream=None) -> None:
    """out [T, d] = sum over the token's slots of weights * ys[pos]; see csffn_moe_combine."""
    (rows, d), (T, k) = _matrix(ys, "ys"), _matrix(pos, "pos")
    if out_mode is None:
        out_mode = _abi.OUT_BF16 if out.dtype == _BF16 else _abi.OUT_F32
    dev = _device(out)
    _run("csffn_moe_combine", dev, stream, _arg(ys, "ys", (rows, d), _BF16, dev), _arg(pos, "pos", (T, k), _I32, dev),
         _arg(weights, "weights", (T, k), _F32, dev), T, k, rows, d,
         _arg(out, "out", (T, d), _BF16 if out_mode == _abi.OUT_BF16 else _F32, dev), out_mode)


def block_norm(h: torch.Tensor, y: Optional[torch.Tensor], h_out: Optional[torch.Tensor],
               xn: Optional[torch.Tensor], g_post: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
               g_pre: Optional[torch.Tensor] = None, res_scale: float = 1.0, out_scale: float = 1.0,
               eps: float = 1e-6, stream=None) -> None:
    """h_out = res_scale * h + out_scale * gate * rms(y) * g_post, xn = rms(h_out) * g_pre; see
    csffn_block_norm.  gate: [d] (per channel) or [T, d] (per token)."""
    T, d = _matrix(h, "h")
    dev = _device(h)
    rows, row = (T, d), (d,)
    per_token = gate is not None and gate.dim() == 2
    ycode = _abi.BF16 if y is None else _code(y, "y")
    xcode = _abi.BF16 if xn is None else _code(xn, "xn")
    _run("csffn_block_norm", dev, stream, _arg(h, "h", rows, _F32, dev),
         None if y is None else _arg(y, "y", rows, y.dtype, dev), ycode, _arg(g_post, "g_post", row, _F32, dev),
         _arg(gate, "gate", rows if per_token else row, _F32, dev), T if per_token else 1,
         _arg(g_pre, "g_pre", row, _F32, dev), res_scale, out_scale, eps, T, d, _arg(h_out, "h_out", rows, _F32, dev),
         None if xn is None else _arg(xn, "xn", rows, xn.dtype, dev), xcode)


# ------------------------------------------------------------------------------ buffers

@dataclass
class DecodeBuffers:
    """Per-layer-shape device buffers of one CATS decode step (batch <= max_batch)."""

    idx: torch.Tensor
    count: torch.Tensor
    a_val: torch.Tensor
    ws: torch.Tensor

    @classmethod
    def new(cls, layer: FFNLayer, max_batch: int, max_rank: int = 0, device="cuda") -> "DecodeBuffers":
        return cls(idx=torch.zeros(layer.h, dtype=torch.int32, device=device),
                   count=torch.zeros(1, dtype=torch.int32, device=device),
                   a_val=torch.zeros(max_batch, layer.h, dtype=torch.float32, device=device),
                   ws=new_workspace(layer, max_batch, max_rank, device))


def cats_decode(layer: FFNLayer, x: torch.Tensor, t: float, out: torch.Tensor, buf: DecodeBuffers,
                out_mode: Optional[int] = None, stream=None, one_launch: bool = True) -> None:
    """One CATS sparse FFN step: the single-launch csffn_cats_ffn_forward, or with
    one_launch=False csffn_gate_mask then csffn_sparse_ffn_forward (same outputs)."""
    if one_launch:
        cats_ffn_forward(layer, x, t, buf.idx, buf.count, buf.a_val, out, buf.ws, out_mode=out_mode, stream=stream)
        return
    gate_mask(layer, x, t, buf.idx, buf.count, buf.a_val, buf.ws, stream=stream)
    sparse_ffn_forward(layer, x, buf.idx, buf.count, buf.a_val, out, buf.ws, out_mode=out_mode, stream=stream)
