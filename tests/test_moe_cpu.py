"""Routed FFN and block norm without a GPU: the oracle against values worked out by hand, and the
refusals of the C ABI and of the binding (fake, never-dereferenced pointers)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from contextual_sparsity_ffn_b200 import _abi
from contextual_sparsity_ffn_b200 import binding as cs
from contextual_sparsity_ffn_b200.build import build

FAKE = 0x7F0000000000
BIG = 1 << 40
ERR = _abi.ERR_INVALID_ARG, _abi.ERR_UNSUPPORTED_SHAPE, _abi.ERR_ALIGNMENT, _abi.ERR_WORKSPACE
ARG, SHAPE, ALIGN, WS = ERR


@pytest.fixture(scope="module")
def lib():
    build()
    return _abi.load()


# ------------------------------------------------------------------------------ oracle, by hand

def test_route_by_hand():
    lg = np.array([[1.0, 3.0, 3.0, -np.inf], [-np.inf, -np.inf, 2.0, -np.inf], [-np.inf] * 4,
                   [np.nan, 0.0, -0.0, np.inf]], dtype=np.float32)
    ids, w = oracle.moe_route(lg, 2)
    assert ids.tolist() == [[1, 2], [2, -1], [-1, -1], [3, 1]]  # ties by the lower expert, also 0 and -0
    np.testing.assert_allclose(w, [[0.5, 0.5], [1, 0], [0, 0], [1, 0]])
    ids, w = oracle.moe_route(lg[:1], 2, renormalize=False)
    e = np.exp([1.0, 3.0])
    np.testing.assert_allclose(w, [[e[1] / (e[0] + 2 * e[1])] * 2])
    ids, w = oracle.moe_route(lg[:1], 2, bias=[5, 0, 0, 0], score="sigmoid", scale=2.0)
    assert ids.tolist() == [[0, 1]]  # the bias moves the choice, not the weights
    s = 1 / (1 + np.exp(-np.array([1.0, 3.0])))
    np.testing.assert_allclose(w, [2 * s / s.sum()])


def test_sort_by_hand():
    off, order, pos = oracle.moe_sort(np.array([[2, 0], [-1, 2], [0, 7]]), 3)
    assert off.tolist() == [0, 2, 2, 4] and order.tolist() == [1, 4, 0, 3]
    assert pos.tolist() == [[2, 0], [-1, 3], [1, -1]]


def test_ffn_combine_norm_by_hand():
    xs = np.array([[1.0, 0.0], [0.0, 2.0], [5.0, 5.0]])
    wg = np.array([[[2.0, 0.0]], [[0.0, -1.0]]])  # two experts of one neuron
    wu, wd = np.ones((2, 1, 2)), np.array([[[1.0, -1.0]], [[3.0, 0.0]]])
    ys, size = oracle.moe_ffn(xs, [0, 1, 2], wg, wu, wd, "relu")
    assert ys[0].tolist() == [2.0, -2.0] and ys[1].tolist() == [0.0, 0.0] and np.isnan(ys[2]).all()
    assert size[0].tolist() == [2.0, 2.0]
    out = oracle.moe_combine(ys, np.array([[0, -1], [0, 1]]), np.array([[0.5, np.nan], [1.0, 2.0]]))
    assert out.tolist() == [[1.0, -1.0], [2.0, -2.0]]
    hn, xn = oracle.block_norm(np.array([[3.0, 4.0]]), np.array([[1.0, 1.0]]), gate=np.array([2.0, 0.0]), res_scale=2,
                               out_scale=0.5, eps=0.0)
    assert hn.tolist() == [[7.0, 8.0]]
    np.testing.assert_allclose(xn, hn / np.sqrt((49 + 64) / 2))


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("act", ["silu", "relu"])
@pytest.mark.parametrize("d,h,counts", [(64, 64, [20, 44]), (72, 136, [3, 5, 0, 30]), (256, 200, [0, 31, 33]),
                                        (64, 2048, [40]), (64, 64, [1] * 40)])
def test_two_part_tolerance_sees_a_lost_part(d, h, counts, act):
    """The tolerance of a v in two bf16 parts holds for such a v, and does not hold when the low part is
    lost, taken from the row before, or added twice."""
    rng = np.random.default_rng(d + h)
    off = np.concatenate([[0], np.cumsum(counts)])
    E, n = len(counts), off[-1]
    xs, wg, wu, wd = (bf16(rng.standard_normal(s) * f) for s, f in (((n, d), 1), ((E, h, d), d ** -0.5), ((E, h, d), d ** -0.5),
                                                                    ((E, h, d), h ** -0.5)))
    v, slip = oracle.moe_ffn_parts(xs, off, wg, wu, act)
    want, _ = oracle.moe_ffn(xs, off, wg, wu, wd, act)
    tol = oracle.moe_ffn_tol_two_parts(v, slip, off, wd, want)
    high = bf16(v)
    low = bf16(v - high)

    def outside(p):
        ys = bf16(np.concatenate([p[off[e]:off[e + 1]] @ wd[e] for e in range(E)]))
        return int((~(np.abs(ys - want) <= tol)).sum())
    assert outside(high + low) == 0
    assert min(outside(high), outside(high + np.roll(low, 1, axis=0)), outside(high + 2 * low)) > 0


# ------------------------------------------------------------------------------ refusals of the C ABI

def moe_layer(d=256, h=128, E=4, act=_abi.ACT_SILU, w=FAKE):
    return _abi.MoELayer(d, h, E, act, w, w and w + 0x1000, w and w + 0x2000)


def test_logits_refusals(lib):
    def f(x=FAKE, w=FAKE, T=4, E=8, d=256, out=FAKE):
        return lib.csffn_moe_logits(x, w, T, E, d, out, None)
    assert f(T=0) == _abi.OK
    assert f(T=-1) == f(E=0) == f(E=513) == f(x=0) == f(w=0) == f(out=0) == ARG
    assert f(d=0) == f(d=16392) == f(T=(1 << 22) + 1) == SHAPE
    assert f(d=260) == f(x=FAKE + 8) == f(w=FAKE + 2) == f(out=FAKE + 2) == ALIGN


def test_route_refusals(lib):
    def f(lg=FAKE, dt=_abi.F32, bias=None, T=4, E=8, k=2, score=0, scale=1.0, ids=FAKE, w=FAKE):
        return lib.csffn_moe_route(lg, dt, bias, T, E, k, score, 1, scale, ids, w, None)
    assert f(T=0) == _abi.OK
    assert f(dt=2) == f(E=0) == f(E=513, k=1) == f(k=0) == f(k=9) == f(k=17, E=64) == f(score=2) == f(T=-1) == ARG
    assert f(scale=float("nan")) == f(lg=0) == f(ids=0) == f(w=0) == ARG
    assert f(T=1 << 22) == SHAPE
    assert f(lg=FAKE + 2) == f(bias=FAKE + 2) == f(ids=FAKE + 1) == f(w=FAKE + 2) == ALIGN
    assert f(lg=FAKE + 1, dt=_abi.BF16) == ALIGN


def test_dispatch_refusals(lib):
    def f(x=FAKE, dt=_abi.BF16, ids=FAKE, T=4, k=2, E=8, d=256, off=FAKE, order=FAKE, pos=FAKE, xs=FAKE, ws=FAKE, n=BIG):
        return lib.csffn_moe_dispatch(x, dt, ids, T, k, E, d, off, order, pos, xs, ws, n, None)
    assert f(dt=2) == f(T=-1) == f(k=0) == f(k=17) == f(E=0) == f(E=513) == ARG
    assert f(x=0) == f(ids=0) == f(off=0) == f(order=0) == f(pos=0) == f(xs=0) == ARG
    assert f(T=1 << 22) == f(d=0) == f(d=16392) == SHAPE
    assert f(d=260) == f(x=FAKE + 8) == f(xs=FAKE + 4) == f(ids=FAKE + 2) == f(off=FAKE + 1) == ALIGN
    assert f(ws=0) == f(ws=FAKE + 4) == f(n=100) == WS
    need = lib.csffn_moe_dispatch_workspace_size(8, 8)
    assert need > 0 and f(n=need - 1) == WS
    assert lib.csffn_moe_dispatch_workspace_size(0, 8) == lib.csffn_moe_dispatch_workspace_size(8, 0) == 0
    assert lib.csffn_moe_dispatch_workspace_size((1 << 22) + 1, 8) == lib.csffn_moe_dispatch_workspace_size(8, 513) == 0


def test_dispatch_widths_by_type(lib):
    """Rows are whole 16-byte vectors: multiples of 8 in bf16, of 4 in fp32 (then the workspace is refused)."""
    def f(dt, d):
        return lib.csffn_moe_dispatch(FAKE, dt, FAKE, 4, 2, 8, d, FAKE, FAKE, FAKE, FAKE, FAKE, 100, None)
    assert f(_abi.F32, 260) == f(_abi.F32, 12) == f(_abi.BF16, 264) == WS
    assert f(_abi.F32, 258) == f(_abi.BF16, 260) == ALIGN
    assert f(_abi.F32, 4) == f(_abi.F32, 16388) == SHAPE


def test_dispatch_refuses_overlapping_buffers(lib):
    """T = 4, k = 2, E = 8, rows of 512 bytes: every buffer at an address of its own, then one output moved
    onto another buffer, onto its last word, or to where the two share one word."""
    size = dict(x=4 * 512, ids=32, off=36, order=32, pos=32, xs=8 * 512)
    base = {n: FAKE + 0x10000 * i for i, n in enumerate(size)}

    def f(n=BIG, **at):
        p = {**base, **at}
        return lib.csffn_moe_dispatch(p["x"], _abi.BF16, p["ids"], 4, 2, 8, 256, p["off"], p["order"], p["pos"], p["xs"],
                                      FAKE, n, None)
    assert f(n=8) == WS
    for a, b in (("pos", "ids"), ("order", "ids"), ("off", "ids"), ("xs", "ids"), ("xs", "x"), ("pos", "x"), ("order", "x"),
                 ("off", "x"), ("order", "off"), ("pos", "off"), ("pos", "order"), ("xs", "order"), ("xs", "pos"), ("xs", "off")):
        assert f(**{a: base[b]}) == ARG
        last = base[b] + size[b] - 4
        if a != "xs" or last % 16 == 0:
            assert f(**{a: last}) == ARG
        below = base[b] - size[a] + 4
        if a != "xs" or below % 16 == 0:
            assert f(**{a: below}) == ARG


def test_ffn_refusals(lib):
    def f(L=None, xs=FAKE, off=FAKE, rows=8, ys=FAKE + 0x10000, ws=FAKE, n=BIG):
        L = moe_layer() if L is None else L
        return lib.csffn_moe_ffn_forward(ctypes.byref(L) if L else None, xs, off, rows, ys, ws, n, None)
    assert f(rows=0) == _abi.OK
    assert f(L=False) == f(moe_layer(E=0)) == f(moe_layer(E=513)) == f(moe_layer(act=5)) == f(rows=-1) == ARG
    assert f(xs=0) == f(off=0) == f(ys=0) == f(moe_layer(w=0)) == ARG
    assert f(moe_layer(d=0)) == f(moe_layer(d=16392)) == f(moe_layer(h=0)) == SHAPE
    assert f(moe_layer(h=1 << 23, E=4)) == f(rows=(1 << 22) + 1) == SHAPE
    assert f(moe_layer(d=260)) == f(moe_layer(h=100)) == f(moe_layer(w=FAKE + 8)) == ALIGN
    assert f(xs=FAKE + 8) == f(ys=FAKE + 8) == f(off=FAKE + 2) == ALIGN
    need = lib.csffn_moe_workspace_size(ctypes.byref(moe_layer()), 8)
    assert f(ws=0) == f(ws=FAKE + 8) == f(n=need - 1) == WS
    assert lib.csffn_moe_workspace_size(ctypes.byref(moe_layer(d=260)), 8) == 0
    assert lib.csffn_moe_workspace_size(ctypes.byref(moe_layer()), 0) == lib.csffn_moe_workspace_size(None, 8) == 0
    assert need >= lib.csffn_moe_dispatch_workspace_size(8, 4)


def test_workspace_for_more_rows_serves_fewer(lib):
    """The queried sizes never fall as the rows grow."""
    rows = sorted({r + d for b in range(1, 23) for r in (1 << b, 3 << b >> 1) for d in (-1, 0, 1)} - {0})
    for L in (moe_layer(h=8), moe_layer(h=1024, E=64)):
        sizes = [lib.csffn_moe_workspace_size(ctypes.byref(L), r) for r in rows if r <= 1 << 22]
        assert sizes == sorted(sizes) and sizes[0] > 0
    sizes = [lib.csffn_moe_dispatch_workspace_size(r, 512) for r in rows if r <= 1 << 22]
    assert sizes == sorted(sizes) and sizes[0] > 0


def test_combine_refusals(lib):
    def f(ys=FAKE, pos=FAKE, w=FAKE, T=4, k=2, rows=8, d=256, out=FAKE, mode=_abi.OUT_F32):
        return lib.csffn_moe_combine(ys, pos, w, T, k, rows, d, out, mode, None)
    assert f(T=0) == _abi.OK
    assert f(mode=3) == f(rows=-1) == f(T=-1) == f(k=0) == f(k=17) == f(ys=0) == f(pos=0) == f(out=0) == ARG
    assert f(d=0) == f(T=1 << 22) == f(rows=(1 << 22) + 1) == SHAPE
    assert f(d=260) == f(ys=FAKE + 8) == f(out=FAKE + 8) == f(pos=FAKE + 2) == f(w=FAKE + 2) == ALIGN


def test_block_norm_refusals(lib):
    def f(h=FAKE, y=FAKE, yd=0, gp=None, gate=None, gr=1, gn=None, a=1.0, b=1.0, eps=1e-6, T=4, d=256,
          ho=FAKE, xn=FAKE + 0x1000, xd=0):
        return lib.csffn_block_norm(h, y, yd, gp, gate, gr, gn, a, b, eps, T, d, ho, xn, xd, None)
    nan = float("nan")
    assert f(T=0) == _abi.OK
    assert f(T=-1) == f(yd=2) == f(xd=2) == f(eps=-1.0) == f(eps=nan) == f(a=nan) == f(b=nan) == f(h=0) == ARG
    assert f(ho=None, xn=None) == f(y=None, gp=FAKE) == f(y=None, gate=FAKE) == f(gate=FAKE, gr=3) == ARG
    assert f(xn=FAKE) == f(h=FAKE + 0x4000, ho=FAKE + 0x1000) == ARG
    assert f(d=0) == f(d=16392) == f(T=(1 << 22) + 1) == SHAPE
    assert f(d=260) == f(h=FAKE + 8) == f(y=FAKE + 4) == f(gp=FAKE + 4) == f(gate=FAKE + 4) == f(gn=FAKE + 4) == ALIGN
    assert f(ho=FAKE + 4) == f(xn=FAKE + 4) == ALIGN


# ------------------------------------------------------------------------------ refusals of the binding

def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    ids = torch.zeros(2, 1, dtype=torch.int32)
    for call in (lambda: cs.moe_logits(x, x, torch.zeros(2, 2)),
                 lambda: cs.moe_route(torch.zeros(2, 8), ids, torch.zeros(2, 1)),
                 lambda: cs.moe_dispatch(x, ids, torch.zeros(3, dtype=torch.int32), ids[:, 0], ids, x, x),
                 lambda: cs.moe_combine(x, ids, None, x), lambda: cs.block_norm(x.float(), x, None, x),
                 lambda: cs.MoELayer(x[None], x[None], x[None], _abi.ACT_SILU)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
