"""CPU oracle of the routed FFN and of the norms around a block: the plain definitions in float64
with numpy, on the operand values the GPU receives (already decoded).  Test infrastructure only."""
from __future__ import annotations

import math

import numpy as np


def moe_logits(x: np.ndarray, w_router: np.ndarray) -> np.ndarray:
    """logits[t, e] = sum_c x[t, c] w_router[e, c]."""
    return x @ w_router.T


def moe_route(logits: np.ndarray, k: int, bias=None, score: str = "softmax", renormalize: bool = True,
              scale: float = 1.0) -> tuple:
    """(ids [T, k], weights [T, k]): the experts of the k largest keys, one token and one choice at a
    time.  The keys are fp32 by definition: the logit, or one fp32 addition of the bias."""
    logits = np.asarray(logits, dtype=np.float32)
    T, E = logits.shape
    ids = np.full((T, k), -1, dtype=np.int64)
    weights = np.zeros((T, k))
    for t in range(T):
        with np.errstate(invalid="ignore"):
            key = logits[t] if bias is None else (logits[t] + np.asarray(bias, dtype=np.float32)).astype(np.float32)
        left = [e for e in range(E) if key[e] > -np.inf]
        for j in range(min(k, len(left))):
            best = max(key[e] for e in left)
            ids[t, j] = next(e for e in left if key[e] == best)
            left.remove(ids[t, j])
        sel = [float(logits[t, e]) for e in ids[t] if e >= 0]
        if not sel:
            continue
        if score == "sigmoid":
            w = [1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0 for v in sel]
            z = max(sum(w), 1e-20) if renormalize else 1.0
        else:
            among = sel if renormalize else [float(v) for v in logits[t] if v > -np.inf]
            m = max(among)
            term = (lambda v: 1.0 if v == m else 0.0 if m == np.inf else math.exp(v - m))  # noqa: E731
            w, z = [term(v) for v in sel], sum(term(v) for v in among)
        weights[t, :len(sel)] = [scale * v / z for v in w]
    return ids, weights


def moe_sort(ids: np.ndarray, n_experts: int) -> tuple:
    """(offsets [E + 1], order [kept], pos [T, k]) of the stable sort of the kept slots by expert."""
    flat = np.asarray(ids).reshape(-1)
    order = [s for e in range(n_experts) for s in range(flat.size) if flat[s] == e] if flat.size * n_experts < 20000 \
        else [int(s) for e in range(n_experts) for s in np.nonzero(flat == e)[0]]
    pos = np.full(flat.size, -1, dtype=np.int64)
    for p, s in enumerate(order):
        pos[s] = p
    offsets = np.array([int(np.sum((flat >= 0) & (flat < e))) for e in range(n_experts + 1)])
    return offsets, np.array(order, dtype=np.int64), pos.reshape(np.asarray(ids).shape)


def moe_ffn(xs: np.ndarray, offsets, w_gate: np.ndarray, w_up: np.ndarray, w_down_t: np.ndarray, act: str) -> tuple:
    """(ys, size) on the sorted rows; size[p, c] = sum_i |v_i W_down^T[i, c]|, what a relative error
    of v can move ys by.  Rows of no expert are NaN."""
    ys = np.full((xs.shape[0], w_gate.shape[2]), np.nan)
    size = np.full_like(ys, np.nan)
    for e in range(w_gate.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            z = xs[lo:hi] @ w_gate[e].T
            a = z / (1.0 + np.exp(-np.clip(z, -700, None))) if act == "silu" else np.maximum(z, 0.0)
            v = a * (xs[lo:hi] @ w_up[e].T)
            ys[lo:hi] = v @ w_down_t[e]
            size[lo:hi] = np.abs(v) @ np.abs(w_down_t[e])
    return ys, size


def moe_combine(ys: np.ndarray, pos: np.ndarray, weights) -> np.ndarray:
    """out[t] = sum_j weights[t, j] ys[pos[t, j]], entries outside the rows skipped."""
    T, k = pos.shape
    out = np.zeros((T, ys.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < ys.shape[0]:
                out[t] += (1.0 if weights is None else weights[t, j]) * ys[pos[t, j]]
    return out


def block_norm(h: np.ndarray, y=None, g_post=None, gate=None, g_pre=None, res_scale: float = 1.0,
               out_scale: float = 1.0, eps: float = 1e-6) -> tuple:
    """(h', xn): h' = res_scale h + out_scale gate rms(y) g_post, xn = rms(h') g_pre."""
    def rms(r):
        return r / np.sqrt((r * r).mean(axis=1, keepdims=True) + eps)
    hn = res_scale * h
    if y is not None:
        u = y if g_post is None else rms(y) * g_post
        hn = hn + out_scale * (u if gate is None else gate * u)
    return hn, rms(hn) * (1.0 if g_pre is None else g_pre)


def moe_ffn_parts(xs: np.ndarray, offsets, w_gate: np.ndarray, w_up: np.ndarray, act: str) -> tuple:
    """(v, slip) on the sorted rows: v[p, i] = act(z) u, and how far v in fp32 may be from it.  An MMA adds
    16 products and may cut the running sum by an fp32 step of 2^-23, so z and u are off by at most
    (d / 16 + 16) 2^-23 of their sums of absolute products; the activation's slope is at most 1.1, its own
    error (|z| + 8) 2^-22 relative (the rounded exponent, the approximate exponential and reciprocal), the
    product's 2^-23."""
    E, h, d = w_gate.shape
    v, slip = np.zeros((xs.shape[0], h)), np.zeros((xs.shape[0], h))
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            x, step = xs[lo:hi], (d / 16 + 16) * 2.0 ** -23
            z, u = x @ w_gate[e].T, x @ w_up[e].T
            dz, du = step * (np.abs(x) @ np.abs(w_gate[e]).T), step * (np.abs(x) @ np.abs(w_up[e]).T)
            a = z / (1.0 + np.exp(-np.clip(z, -700, None))) if act == "silu" else np.maximum(z, 0.0)
            v[lo:hi] = a * u
            da = 1.1 * dz + (np.abs(z) + 8) * 2.0 ** -22 * np.abs(a)
            slip[lo:hi] = da * (np.abs(u) + du) + np.abs(a) * du + 2.0 ** -23 * np.abs(a * u)
    return v, slip


def moe_ffn_tol_two_parts(v: np.ndarray, slip: np.ndarray, offsets, w_down_t: np.ndarray, want: np.ndarray) -> np.ndarray:
    """How far ys may be from `want` where v reaches the down product as a bf16 high part and a bf16 low
    part: each rounding is off by at most 2^-8 of what it rounds, so both together leave 2^-16 of v; the sum
    over h neurons of two parts in fp32 is off by (h / 8 + 32) 2^-23 of its absolute products; ys is rounded
    once, by 2^-8 of itself."""
    E, h, _ = w_down_t.shape
    b = np.zeros(want.shape)
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            off = slip[lo:hi] * (1 + 2.0 ** -16) + (2.0 ** -16 + (h / 8 + 32) * 2.0 ** -23) * np.abs(v[lo:hi])
            b[lo:hi] = off @ np.abs(w_down_t[e])
    return b + 2.0 ** -8 * (np.abs(want) + b)
