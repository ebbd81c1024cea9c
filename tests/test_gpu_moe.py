"""Routed FFN and block norm on the GPU against the 64-bit oracle: router projection and selection,
tokens sorted by expert and back, the experts' gated FFNs, the norms around a block, and a stack.

Tolerances follow from the roundings (half a step: bf16 2^-8, fp32 2^-24 relative):
  logits   fp32 sums of exact products: an MMA adds 16 products and may cut the running sum by one
           fp32 step (2^-23), so the relative L2 error stays below (d / 16 + 16) 2^-23.
  weights  exp(l - m): the rounded difference moves it by |l - m| 2^-24, expf itself by 2 steps,
           the sum of n terms by n 2^-24, the division by one: (64 + n) 2^-23 relative for |l - m| < 64.
  ffn      v carries one bf16 rounding (2^-8 of each |v_i W_i|, summed: `size`) and ys another; gate
           and up in fp32 add (d / 16 + 16) 2^-23 of their own sums, for which 2^-10 of `size` is
           ample at these widths.  Element by element: 2^-8 (size + |ys|) + 2^-10 size.  In L2 both
           roundings are at most 2^-8 / sqrt(3) each and independent: below 2^-8 together.
  combine  k products and sums in fp32: (k + 2) 2^-24 of sum |w y|; a bf16 result adds 2^-8 |out|.
  norm     a mean of squares in fp32 by threads, warps and CTA: at most 64 additions deep, so
           32 2^-24 relative on the root, and 16 more steps for the products: 48 2^-24, of h' for each
           of its two terms and again for xn; a bf16 result adds 2^-8 |xn|.
"""
import numpy as np
import pytest
import torch

import oracle
from contextual_sparsity_ffn_b200 import _abi
from contextual_sparsity_ffn_b200 import binding as cs
from contextual_sparsity_ffn_b200 import stack

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
U32, U16 = 2.0 ** -24, 2.0 ** -8


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, *shape, std=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def np64(t):
    return t.detach().double().cpu().numpy()


def within(got, want, tol):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outside, worst "
                           f"{np.nanmax(np.abs(got - want) - tol):.3e} over, first {np.argwhere(bad)[0]}")


# ------------------------------------------------------------------------------ logits

@pytest.mark.parametrize("T,E,d", [(1, 1, 8), (1, 64, 2048), (3, 5, 72), (16, 128, 4096), (17, 8, 256), (31, 33, 520),
                                   (64, 64, 1024), (65, 129, 640), (130, 512, 128), (257, 160, 2056), (1000, 7, 64),
                                   (2049, 128, 4096), (33, 300, 16384)])
def test_logits(T, E, d):
    g = gen(T + E + d)
    x, w = rnd(g, T, d), rnd(g, E, d, std=d ** -0.5)
    out = torch.full((T, E), float("nan"), device="cuda")
    cs.moe_logits(x, w, out)
    want = oracle.moe_logits(np64(x), np64(w))
    assert oracle.rel_l2(np64(out), want) <= (d / 16 + 16) * 2.0 ** -23
    within(np64(out), want, (d / 16 + 16) * 2.0 ** -23 * (np.abs(np64(x)) @ np.abs(np64(w)).T))
    again = torch.empty_like(out)
    cs.moe_logits(x, w, again)
    assert torch.equal(out, again)


def test_logits_nan_rows_stay_apart():
    g = gen(5)
    x, w = rnd(g, 70, 256), rnd(g, 40, 256)
    x[3], x[40] = float("nan"), float("inf")
    out = torch.empty(70, 40, device="cuda")
    cs.moe_logits(x, w, out)
    clean = [t for t in range(70) if t not in (3, 40)]
    assert torch.isfinite(out[clean]).all() and torch.isnan(out[3]).all()


# ------------------------------------------------------------------------------ route

def run_route(lg, k, bias=None, score="softmax", renorm=True, scale=1.0):
    T = lg.shape[0]
    ids = torch.full((T, k), 77, dtype=I32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    cs.moe_route(lg, ids, w, bias=bias, score=_abi.ROUTE_SOFTMAX if score == "softmax" else _abi.ROUTE_SIGMOID,
                 renormalize=renorm, scale=scale)
    want_ids, want_w = oracle.moe_route(lg.float().cpu().numpy(), k, None if bias is None else bias.cpu().numpy(), score,
                                        renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    within(np64(w), want_w, (64 + lg.shape[1]) * 2.0 ** -23 * want_w + 1e-37)
    return ids, w


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("T,E,k,dtype,biased", [(1, 1, 1, F32, False), (5, 2, 2, BF, False), (3, 31, 16, F32, True),
                                                (64, 64, 8, BF, True), (33, 65, 6, F32, False), (7, 160, 6, BF, True),
                                                (4, 257, 16, BF, False), (9, 512, 8, F32, True)])
def test_route(T, E, k, dtype, biased, score, renorm):
    g = gen(E * k + T)
    lg = rnd(g, T, E, std=2.0, dtype=dtype)
    lg[torch.rand(T, E, generator=g, device="cuda") < 0.3] = float("-inf")
    run_route(lg, k, rnd(g, E, std=0.5, dtype=F32) if biased else None, score, renorm, 2.5)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_special_values(score, renorm):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(F32).min
    lg = torch.tensor([[0.0, -0.0, 0.0, -0.0], [-inf] * 4, [nan] * 4, [nan, 1, -inf, 2], [inf, inf, 1, -inf],
                       [low, low, low, -inf], [-200.0, -300.0, -inf, nan], [50.0, -50.0, 0.0, 1e-40]], device="cuda")
    run_route(lg, 3, None, score, renorm)
    run_route(lg, 1, torch.tensor([0.0, 3.0, -inf, nan], device="cuda"), score, renorm)


# ------------------------------------------------------------------------------ dispatch, combine

def random_ids(g, T, E, k, drop):
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=I32)  # repeats within a token too
    ids[torch.rand(T, k, generator=g, device="cuda") < drop] = -1
    return ids


def run_dispatch(x, ids, E, ws=None):
    T, k = ids.shape
    out = dict(offsets=torch.full((E + 1,), -9, dtype=I32, device="cuda"),
               order=torch.full((T * k,), -9, dtype=I32, device="cuda"),
               pos=torch.full((T, k), -9, dtype=I32, device="cuda"),
               xs=torch.full((T * k, x.shape[1]), 7.0, dtype=x.dtype, device="cuda"))
    ws = cs.new_moe_dispatch_workspace(max(1, T * k), E) if ws is None else ws
    cs.moe_dispatch(x, ids, out["offsets"], out["order"], out["pos"], out["xs"], ws)
    return out


def check_dispatch(x, ids, E, got):
    T, k = ids.shape
    off, order, pos = oracle.moe_sort(ids.cpu().numpy(), E)
    n = off[-1]
    assert np.array_equal(got["offsets"].cpu().numpy(), off)
    assert np.array_equal(got["order"][:n].cpu().numpy(), order)
    assert np.array_equal(got["pos"].cpu().numpy(), pos)
    rows = torch.from_numpy(order // k).cuda()
    assert torch.equal(got["xs"][:n], x[rows])
    assert (got["order"][n:] == -9).all() and (got["xs"][n:] == 7.0).all()  # left as they were


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,E,k,d,drop", [(1, 1, 1, 8, 0), (1, 64, 8, 2048, 0), (13, 64, 8, 264, 0.2), (128, 8, 8, 64, 0.5),
                                          (129, 8, 8, 64, 0.5), (5, 512, 16, 4096, 0.1), (700, 3, 2, 1032, 0.9),
                                          (1025, 160, 6, 128, 0.05), (4100, 512, 1, 24, 0.3), (40, 5, 3, 16384, 0),
                                          (20000, 64, 16, 8, 0.1), (300, 7, 4, 256, 1.0)])
def test_dispatch(T, E, k, d, drop, dtype):
    g = gen(T * k + E)
    x, ids = rnd(g, T, d, dtype=dtype), random_ids(g, T, E, k, drop)
    ids[ids == E - 1] = E + 3 if T > 100 else E - 1  # ids past the experts are dropped too
    check_dispatch(x, ids, E, run_dispatch(x, ids, E))


@pytest.mark.parametrize("T,k", [(1023, 1), (1024, 1), (1025, 1), (341, 3), (2048, 8), (16385, 1), (1023, 16), (8192, 8),
                                 (16384, 16), (16385, 16), (131072, 2)])
def test_dispatch_sizes_of_its_forms(T, k):
    """Slot counts around those where one kernel, one cluster or many CTAs plan the sort."""
    g = gen(T + k)
    x, ids = rnd(g, T, 16), random_ids(g, T, 37, k, 0.05)
    got = run_dispatch(x, ids, 37)
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, 37, flat)
    want = torch.sort(key, stable=True).indices
    n = int((flat >= 0).sum())
    assert torch.equal(got["order"][:n].long(), want[:n]) and (got["order"][n:] == -9).all()
    assert got["offsets"].tolist() == [int((key < e).sum()) for e in range(38)]
    pos = torch.full_like(flat, -1)
    pos[want[:n]] = torch.arange(n, device="cuda")
    assert torch.equal(got["pos"].reshape(-1).long(), pos)
    assert torch.equal(got["xs"][:n], x[want[:n] // k]) and (got["xs"][n:] == 7.0).all()


@pytest.mark.parametrize("T,d", [(5, 12), (700, 260), (9000, 20)])
def test_dispatch_fp32_rows_of_odd_multiples_of_four(T, d):
    g = gen(T + d)
    x, ids = rnd(g, T, d, dtype=F32), random_ids(g, T, 6, 2, 0.1)
    check_dispatch(x, ids, 6, run_dispatch(x, ids, 6))
    with pytest.raises(cs.CsffnError) as e:
        run_dispatch(x.bfloat16(), ids, 6)
    assert e.value.status == _abi.ERR_ALIGNMENT


def test_dispatch_one_expert_takes_all():
    x, ids = rnd(gen(1), 2000, 32), torch.full((2000, 2), 5, dtype=I32, device="cuda")
    check_dispatch(x, ids, 9, run_dispatch(x, ids, 9))


def test_dispatch_no_tokens():
    got = run_dispatch(torch.empty(0, 64, dtype=BF, device="cuda"), torch.empty(0, 2, dtype=I32, device="cuda"), 4)
    assert (got["offsets"] == 0).all()


@pytest.mark.parametrize("mode", [_abi.OUT_BF16, _abi.OUT_F32, _abi.OUT_F32_ACCUMULATE])
@pytest.mark.parametrize("T,k,d,rows,drop", [(1, 1, 8, 1, 0), (13, 8, 264, 90, 0.3), (300, 2, 4096, 600, 0), (7, 16, 72, 100, 0.6),
                                             (5, 5, 16384, 25, 0), (1000, 6, 256, 6000, 1.0), (3, 4, 2048, 0, 0)])
def test_combine(T, k, d, rows, drop, mode):
    g = gen(T + d)
    ys = rnd(g, rows, d)
    pos = torch.randint(-2, rows + 2, (T, k), generator=g, device="cuda", dtype=I32)
    pos[torch.rand(T, k, generator=g, device="cuda") < drop] = -1
    for w in (rnd(g, T, k, dtype=F32), None):
        if w is not None:
            w[(pos < 0) | (pos >= rows)] = float("nan")  # skipped whatever the weight
        start = rnd(g, T, d, dtype=BF if mode == _abi.OUT_BF16 else F32)
        out = start.clone()
        cs.moe_combine(ys, pos, w, out, out_mode=mode)
        wn = np.ones((T, k)) if w is None else np.nan_to_num(np64(w))
        want = oracle.moe_combine(np64(ys), pos.cpu().numpy(), wn)
        size = oracle.moe_combine(np.abs(np64(ys)), pos.cpu().numpy(), np.abs(wn))
        if mode == _abi.OUT_F32_ACCUMULATE:
            want, size = want + np64(start), size + np.abs(np64(start))
        within(np64(out), want, (k + 2) * U32 * size + (U16 * np.abs(want) if mode == _abi.OUT_BF16 else 0))


# ------------------------------------------------------------------------------ experts

def make_experts(g, E, d, h, act="silu"):
    return cs.MoELayer(rnd(g, E, h, d, std=d ** -0.5), rnd(g, E, h, d, std=d ** -0.5), rnd(g, E, h, d, std=h ** -0.5),
                       _abi.ACT_SILU if act == "silu" else _abi.ACT_RELU)


def check_ffn(layer, xs, counts, act="silu", spare=0, ws=None):
    """counts: rows per expert; `spare` rows behind the last expert's hold NaN and stay as they were."""
    E, n = len(counts), int(sum(counts))
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=I32, device="cuda")
    xs = torch.cat([xs[:n], torch.full((spare, layer.d), float("nan"), dtype=BF, device="cuda")])
    ys = torch.full((n + spare, layer.d), 3.0, dtype=BF, device="cuda")
    ws = cs.new_moe_workspace(layer, max(1, n + spare)) if ws is None else ws
    cs.moe_ffn_forward(layer, xs, offsets, ys, ws)
    assert cs.check_status(ws) == 0
    assert (ys[n:] == 3.0).all()
    want, size = oracle.moe_ffn(np64(xs[:n]), offsets.cpu().numpy(), np64(layer.w_gate), np64(layer.w_up),
                                np64(layer.w_down_t), act)
    got = np64(ys[:n])
    within(got, want, U16 * (size + np.abs(want)) + 2.0 ** -10 * size)
    if n * layer.d >= 1000:
        assert oracle.rel_l2(got, want) <= U16
    again = torch.full_like(ys, 3.0)
    cs.moe_ffn_forward(layer, xs, offsets, again, ws)
    assert torch.equal(ys[:n], again[:n])  # bit for bit
    return ys


@pytest.mark.parametrize("act", ["silu", "relu"])
@pytest.mark.parametrize("d,h,counts,spare", [
    (8, 8, [1], 0), (64, 128, [1, 0, 2], 0), (72, 136, [3, 5], 2), (256, 200, [0, 0, 0, 1], 5), (520, 264, [17, 16, 33], 0),
    (256, 512, [1] * 40, 0), (1024, 256, [0, 31, 32, 0, 1, 65], 3), (2048, 1024, [8, 0, 1, 2, 0, 0, 0, 4], 0),
    (128, 1000, [200, 0, 7], 9), (640, 384, [255, 256, 257, 0, 1], 0), (264, 1032, [129, 500], 11),
    (4096, 512, [40, 3], 0), (512, 2048, [700, 300], 0), (192, 320, [0, 0, 1500, 2], 1), (256, 128, [0, 0], 4)])
def test_ffn(d, h, counts, spare, act):
    g = gen(d + h)
    check_ffn(make_experts(g, len(counts), d, h, act), rnd(g, sum(counts), d), counts, act, spare)


# Tiles left over and cut along the contraction: into parts (few rows; many rows), as one run over the
# pairs; whole rounds before them; wide down tiles with a ragged last block.
@pytest.mark.parametrize("d,h,counts", [
    (4096, 512, [40]), (4096, 512, [300, 40]), (1024, 4096, [5, 0, 9]), (4096, 2560, [2, 1, 30, 0, 8, 4]),
    (2048, 4104, [33, 1]), (512, 2048, [600, 900, 10, 1300]), (1032, 264, [70, 3, 0, 300, 1, 8, 257, 31, 64, 5, 9, 2, 128, 40]),
    (264, 520, [10 + 3 * i for i in range(45)]), (8200, 128, [90, 200, 33]), (64, 8200, [400]),
    (4096, 5376, [3]), (10240, 3584, [7])])
def test_ffn_split_tiles(d, h, counts):
    g = gen(d + h)
    check_ffn(make_experts(g, len(counts), d, h), rnd(g, sum(counts), d), counts)


def test_ffn_many_experts():
    g = gen(3)
    counts = [int(c) for c in torch.randint(0, 4, (512,), generator=torch.Generator().manual_seed(1))]
    check_ffn(make_experts(g, 512, 64, 64), rnd(g, sum(counts), 64), counts)


def test_ffn_workspace_serves_smaller_calls():
    """One workspace for the largest call: larger and smaller ones in turn, and a dispatch between."""
    g = gen(4)
    layer = make_experts(g, 4, 256, 384)
    ws = cs.new_moe_workspace(layer, 1024)
    xs = rnd(g, 1024, 256)
    for counts in ([300, 400, 0, 324], [1, 0, 2, 0], [0, 9, 9, 9], [256] * 4, [0, 0, 0, 1]):
        check_ffn(layer, xs, counts, ws=ws)
        ids = random_ids(g, 64, 4, 2, 0.1)
        check_dispatch(xs[:64], ids, 4, run_dispatch(xs[:64], ids, 4, ws=ws))


def test_ffn_offsets_are_clamped():
    """Offsets outside 0 .. rows or descending are brought into range: no access outside the buffers."""
    g = gen(6)
    layer = make_experts(g, 4, 64, 64)
    xs = rnd(g, 50, 64)
    ws = cs.new_moe_workspace(layer, 50)
    for off in ([-5, 10, 5, 1000, 20], [60, 70, 80, 90, 100], [0, 50, 0, 50, 50], [-1] * 5):
        ys = torch.full((50, 64), 3.0, dtype=BF, device="cuda")
        cs.moe_ffn_forward(layer, xs, torch.tensor(off, dtype=I32, device="cuda"), ys, ws)
        assert cs.check_status(ws) == 0
        lo = np.maximum.accumulate(np.clip(off, 0, 50))
        want, size = oracle.moe_ffn(np64(xs), lo, np64(layer.w_gate), np64(layer.w_up), np64(layer.w_down_t), "silu")
        live = ~np.isnan(want)
        within(np64(ys)[live], want[live], U16 * (size + np.abs(want))[live] + 2.0 ** -10 * size[live])
        assert (np64(ys)[~live] == 3.0).all()


# ------------------------------------------------------------------------------ block norm

@pytest.mark.parametrize("ydt,xdt", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("T,d,gate", [(1, 8, "channel"), (3, 264, "token"), (5, 512, "none"), (2, 1032, "channel"),
                                      (9, 2056, "token"), (16, 4096, "channel"), (4, 8192, "none"), (3, 16384, "token"),
                                      (1000, 64, "channel"), (7, 8200, "token")])
def test_block_norm(T, d, gate, ydt, xdt):
    g = gen(T + d)
    h, y = rnd(g, T, d, std=2.0, dtype=F32), rnd(g, T, d, dtype=ydt)
    gv = {"none": None, "channel": rnd(g, d, dtype=F32), "token": rnd(g, T, d, dtype=F32)}[gate]
    for post in (rnd(g, d, dtype=F32), None):
        for pre in (rnd(g, d, dtype=F32), None):
            want_h, want_x = oracle.block_norm(np64(h), np64(y), None if post is None else np64(post),
                                               None if gv is None else np64(gv), None if pre is None else np64(pre),
                                               0.9, 0.7)
            term = np.abs(want_h - 0.9 * np64(h)) + np.abs(0.9 * np64(h))
            ho = torch.full_like(h, float("nan"))
            xn = torch.full((T, d), float("nan"), dtype=xdt, device="cuda")
            cs.block_norm(h, y, ho, xn, post, gv, pre, 0.9, 0.7)
            within(np64(ho), want_h, 48 * U32 * term)
            size = np.abs(want_x) + 48 * U32 * term * np.abs(want_x / np.where(want_h == 0, 1, want_h))
            slip = 48 * U32 * term * np.abs(want_x) / np.maximum(np.abs(want_h), 1e-30)
            within(np64(xn), want_x, 48 * U32 * size + slip + (U16 * 1.01 * np.abs(want_x) if xdt == BF else 0))
            only_x, only_h = torch.empty_like(xn), torch.empty_like(ho)
            cs.block_norm(h, y, None, only_x, post, gv, pre, 0.9, 0.7)
            cs.block_norm(h, y, only_h, None, post, gv, None, 0.9, 0.7)
            assert torch.equal(only_x, xn) and torch.equal(only_h, ho)
            h2 = h.clone()
            cs.block_norm(h2, y, h2, xn, post, gv, pre, 0.9, 0.7)  # in place
            assert torch.equal(h2, ho) and torch.equal(only_x, xn)


def test_block_norm_first_and_zero_rows():
    g = gen(9)
    h = rnd(g, 6, 256, dtype=F32)
    h[2] = 0
    xn = torch.empty(6, 256, dtype=F32, device="cuda")
    cs.block_norm(h, None, None, xn)
    _, want = oracle.block_norm(np64(h))
    within(np64(xn), want, 48 * U32 * np.abs(want))
    assert (xn[2] == 0).all()
    y = torch.zeros(6, 256, dtype=BF, device="cuda")
    cs.block_norm(h, y, None, xn, g_post=torch.ones(256, device="cuda"))
    within(np64(xn), want, 96 * U32 * np.abs(want))


# ------------------------------------------------------------------------------ refusals with real tensors

def test_binding_refusals():
    g = gen(2)
    x, w = rnd(g, 4, 64), rnd(g, 8, 64)
    lg = torch.empty(4, 8, device="cuda")
    ids, wt = torch.zeros(4, 2, dtype=I32, device="cuda"), torch.zeros(4, 2, device="cuda")
    for call, word in ((lambda: cs.moe_logits(x.float(), w, lg), "x must be"),
                       (lambda: cs.moe_logits(x, w[:, :32], lg), "shape"),
                       (lambda: cs.moe_logits(x, w, lg.T), "shape"),
                       (lambda: cs.moe_logits(x.T.contiguous().T, w, lg), "contiguous"),
                       (lambda: cs.moe_logits(x, w.cpu(), lg), "device"),
                       (lambda: cs.moe_route(lg, ids.long(), wt), "ids must be"),
                       (lambda: cs.moe_route(lg, ids, wt[:, :1]), "shape"),
                       (lambda: cs.moe_route(lg, ids, wt, bias=wt), "shape"),
                       (lambda: cs.moe_combine(x, ids, wt, x.float(), out_mode=_abi.OUT_BF16), "out must be"),
                       (lambda: cs.block_norm(lg, None, None, lg.bfloat16()[:2]), "shape"),
                       (lambda: cs.block_norm(lg, None, lg.cpu(), None), "device")):
        with pytest.raises(ValueError, match=word):
            call()
    with pytest.raises(cs.CsffnError) as e:
        cs.moe_route(lg, torch.zeros(4, 9, dtype=I32, device="cuda"), torch.zeros(4, 9, device="cuda"))
    assert e.value.status == _abi.ERR_INVALID_ARG
    with pytest.raises(cs.CsffnError) as e:
        cs.moe_logits(x[:, :60].contiguous(), w[:, :60].contiguous(), lg)
    assert e.value.status == _abi.ERR_ALIGNMENT


# ------------------------------------------------------------------------------ a run of them together

def make_block(g, E, d, h, k, **more):
    return stack.MoEBlock(make_experts(g, E, d, h), rnd(g, E, d, std=2 * d ** -0.5), k, g_pre=1 + rnd(g, d, std=0.1, dtype=F32),
                          **more)


def stack_blocks(g, E, d, h, k):
    return [make_block(g, E, d, h, k, g_post=1 + rnd(g, d, std=0.1, dtype=F32), out_scale=0.5),
            make_block(g, E, d, h, k, gate=rnd(g, d, dtype=F32), score=_abi.ROUTE_SIGMOID, route_scale=1.5,
                       sel_bias=rnd(g, E, std=0.1, dtype=F32)),
            make_block(g, E, d, h, k, renormalize=False, res_scale=0.9)]


def check_stack_layerwise(blocks, h, buf):
    """Each layer of the stack against the oracle fed with that layer's own inputs on the device."""
    before = h.clone()
    stack.moe_stack(blocks[:1], h, buf)
    b, x = blocks[0], np64(buf.xn)
    d = x.shape[1]
    lg = oracle.moe_logits(x, np64(b.w_router))
    assert oracle.rel_l2(np64(buf.logits), lg) <= (d / 16 + 16) * 2.0 ** -23
    ids, w = oracle.moe_route(np64(buf.logits), b.k, None, "softmax", b.renormalize)
    assert np.array_equal(buf.ids.cpu().numpy(), ids)
    off, order, pos = oracle.moe_sort(ids, b.experts.n_experts)
    ys, _ = oracle.moe_ffn(x[order // b.k], off, np64(b.experts.w_gate), np64(b.experts.w_up), np64(b.experts.w_down_t), "silu")
    y = oracle.moe_combine(ys, pos, w)
    assert oracle.rel_l2(np64(buf.y), y) <= 2 * U16  # ys' two roundings and y's own
    want, _ = oracle.block_norm(np64(before), np64(buf.y), None if b.g_post is None else np64(b.g_post), None, None,
                                b.res_scale, b.out_scale)
    assert oracle.rel_l2(np64(h), want) <= 96 * U32


@pytest.mark.parametrize("T", [1, 5, 64, 500])
def test_stack(T):
    g = gen(T)
    blocks = stack_blocks(g, 8, 256, 192, 2)
    buf = stack.MoEBuffers.new(blocks[0], T)
    h0 = rnd(g, T, 256, dtype=F32)
    check_stack_layerwise(blocks, h0.clone(), buf)
    h = h0.clone()
    stack.moe_stack(blocks, h, buf)
    assert cs.check_status(buf.ws) == 0 and torch.isfinite(h).all()
    # captured and replayed, the inputs changed in between; on a side stream; twice the same bits
    hg = h0.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            stack.moe_stack(blocks, hg, buf)
    torch.cuda.current_stream().wait_stream(side)
    for start in (h0, rnd(g, T, 256, dtype=F32), h0):
        hg.copy_(start)
        graph.replay()
        he = start.clone()
        torch.cuda.synchronize()
        stack.moe_stack(blocks, he, buf)
        assert torch.equal(hg, he)
    assert torch.equal(hg, h)


def test_stack_two_streams():
    """Two stacks with buffers of their own on two streams at once give the bits of one at a time."""
    g = gen(11)
    blocks = stack_blocks(g, 16, 512, 256, 4)
    starts = [rnd(g, T, 512, dtype=F32) for T in (96, 40)]
    bufs = [stack.MoEBuffers.new(blocks[0], s.shape[0]) for s in starts]
    want = []
    for s, b in zip(starts, bufs):
        want.append(s.clone())
        stack.moe_stack(blocks, want[-1], b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in starts]
    for _ in range(3):
        got = [s.clone() for s in starts]
        torch.cuda.synchronize()
        for h, b, st in zip(got, bufs, streams):
            with torch.cuda.stream(st):
                for _ in range(1):
                    stack.moe_stack(blocks, h, b)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------------------ sizes and uses at the edge

def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the last rows are right in every row-wise operator."""
    g = gen(21)
    T, k, d, E = 66000, 2, 16384, 2
    x = torch.empty(T, d, dtype=BF, device="cuda").normal_(generator=g)
    ids = torch.stack([torch.zeros(T), torch.ones(T)], 1).to(device="cuda", dtype=I32)
    got = run_dispatch(x, ids, E)
    n = T * k
    assert got["xs"].numel() > 2 ** 31 and got["offsets"].tolist() == [0, T, n]
    for p in (0, T - 1, T, n - 2, n - 1):
        assert torch.equal(got["xs"][p], x[p % T])
    layer = make_experts(g, E, d, 8)
    ys = torch.zeros_like(got["xs"])
    ws = cs.new_moe_workspace(layer, n)
    cs.moe_ffn_forward(layer, got["xs"], got["offsets"], ys, ws)
    assert cs.check_status(ws) == 0
    last = slice(n - 70, n)
    want, size = oracle.moe_ffn(np64(got["xs"][last]), [0, 0, 70], np64(layer.w_gate), np64(layer.w_up), np64(layer.w_down_t), "silu")
    within(np64(ys[last]), want, U16 * (size + np.abs(want)) + 2.0 ** -10 * size)
    del x
    w = torch.rand(T, k, generator=g, device="cuda")
    out = torch.empty(T, d, device="cuda")
    cs.moe_combine(ys, got["pos"], w, out)
    t = slice(T - 3, T)
    y2 = torch.stack([ys[T - 3:T], ys[n - 3:n]], 1)
    want = (np64(y2) * np64(w[t])[:, :, None]).sum(1)
    within(np64(out[t]), want, (k + 2) * U32 * (np.abs(np64(y2)) * np64(w[t])[:, :, None]).sum(1))
    del got, out, y2
    h = torch.empty(n, d, device="cuda").normal_(generator=g)
    xn = torch.empty(n, d, dtype=BF, device="cuda")
    cs.block_norm(h, ys, h, xn, out_scale=0.0, res_scale=2.0)
    assert h.numel() > 2 ** 31
    _, want = oracle.block_norm(np64(h[last]))
    within(np64(xn[last]), want, 48 * U32 * np.abs(want) + U16 * 1.01 * np.abs(want))


def test_many_tokens_router():
    """The most tokens: projection and selection of the first and the last rows."""
    g = gen(22)
    T, E, d = 1 << 22, 40, 16
    x, w = rnd(g, T, d), rnd(g, E, d)
    lg = torch.empty(T, E, device="cuda")
    cs.moe_logits(x, w, lg)
    ids, wt = torch.empty(T, 1, dtype=I32, device="cuda"), torch.empty(T, 1, device="cuda")
    cs.moe_route(lg, ids, wt)
    for t in (slice(0, 200), slice(T - 200, T)):
        want = oracle.moe_logits(np64(x[t]), np64(w))
        within(np64(lg[t]), want, (d / 16 + 16) * 2.0 ** -23 * (np.abs(np64(x[t])) @ np.abs(np64(w)).T))
        assert torch.equal(ids[t, 0].long(), lg[t].argmax(1)) and (wt[t] == 1).all()
    offsets, order = torch.empty(E + 1, dtype=I32, device="cuda"), torch.empty(T, dtype=I32, device="cuda")
    pos, xs = torch.empty(T, 1, dtype=I32, device="cuda"), torch.empty(T, d, dtype=BF, device="cuda")
    cs.moe_dispatch(x, ids, offsets, order, pos, xs, cs.new_moe_dispatch_workspace(T, E))
    want = torch.sort(ids[:, 0], stable=True).indices
    assert torch.equal(order.long(), want) and torch.equal(xs, x[want])
    assert torch.equal(offsets[1:].long(), torch.cumsum(torch.bincount(ids[:, 0], minlength=E), 0))


def test_layer_in_a_graph_between_eager_calls():
    """One workspace for a captured layer and for eager calls of other row counts, in turn on one stream."""
    g = gen(23)
    layer = make_experts(g, 8, 256, 512)
    ws = cs.new_moe_workspace(layer, 600)
    xs = rnd(g, 600, 256)
    off = {n: torch.tensor([n * i // 8 for i in range(9)], dtype=I32, device="cuda") for n in (24, 600)}
    ys = torch.zeros(600, 256, dtype=BF, device="cuda")
    want = {}
    for n in (24, 600):
        cs.moe_ffn_forward(layer, xs[:n], off[n], ys[:n], ws)
        want[n] = ys[:n].clone()
    graph = torch.cuda.CUDAGraph()
    yg = torch.zeros(24, 256, dtype=BF, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        cs.moe_ffn_forward(layer, xs[:24], off[24], yg, ws)
    for _ in range(3):
        yg.zero_()
        ys.zero_()
        cs.moe_ffn_forward(layer, xs, off[600], ys, ws)
        graph.replay()
        assert torch.equal(yg, want[24]) and torch.equal(ys, want[600])
    assert cs.check_status(ws) == 0


def test_workspace_too_small_for_the_rows():
    layer = make_experts(gen(24), 4, 64, 64)
    ws = cs.new_moe_dispatch_workspace(64, 4)
    xs = torch.zeros(64, 64, dtype=BF, device="cuda")
    with pytest.raises(cs.CsffnError) as e:
        cs.moe_ffn_forward(layer, xs, torch.zeros(5, dtype=I32, device="cuda"), xs.clone(), ws)
    assert e.value.status == _abi.ERR_WORKSPACE


# ------------------------------------------------------------------------------ weights made in the stream

@pytest.mark.parametrize("chained", [False, True])
@pytest.mark.parametrize("T,E,d", [(4, 64, 2048), (4, 512, 16384), (256, 128, 8192), (256, 512, 4096)])
def test_logits_of_weights_made_just_before(T, E, d, chained):
    """A router whose weights block_norm makes in the stream just before the projection, with and without
    a chained kernel between the two: the projection sees all of them.  Replayed, so that the kernels
    follow one another without a gap, on weights that are NaN until they are made."""
    g = gen(E + T)
    x, w32 = rnd(g, T, d), rnd(g, E, d, dtype=F32)
    w16, want, out = torch.empty(E, d, dtype=BF, device="cuda"), torch.empty(T, E, device="cuda"), torch.empty(T, E, device="cuda")
    cs.block_norm(w32, None, None, w16)
    torch.cuda.synchronize()
    cs.moe_logits(x, w16, want)
    lg, ids, wt = rnd(g, 8, 16, dtype=F32), torch.empty(8, 2, dtype=I32, device="cuda"), torch.empty(8, 2, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w16.fill_(float("nan"))
        cs.block_norm(w32, None, None, w16)
        if chained:
            cs.moe_route(lg, ids, wt)
        cs.moe_logits(x, w16, out)
    for _ in range(5):
        out.fill_(float("nan"))
        graph.replay()
        assert torch.equal(out, want)


# ------------------------------------------------------------------------------ values past the range of bf16

@pytest.mark.parametrize("act", ["silu", "relu"])
@pytest.mark.parametrize("rows", [3, 64, 65, 300])
def test_ffn_overflowing_row(rows, act):
    """One neuron of one row overflows (in fp32, or only when it is rounded to bf16): that row is +-inf by
    the signs of the neuron's down weights, with few rows and with many, and the other rows keep their bits."""
    g = gen(rows)
    d, h = 72, 136
    wg, wu, wd = (rnd(g, 1, h, d, std=s) for s in (d ** -0.5, d ** -0.5, h ** -0.5))
    wg[0, :, :2] = wu[0, :, :2] = 0
    wg[0, 5], wu[0, 5] = 0, 0
    wg[0, 5, 0] = wu[0, 5, 1] = 1  # neuron 5: z = x[0], u = x[1]
    wd[0, 5] = torch.where(wd[0, 5] == 0, torch.ones_like(wd[0, 5]), wd[0, 5])
    layer = cs.MoELayer(wg, wu, wd, _abi.ACT_SILU if act == "silu" else _abi.ACT_RELU)
    xs = rnd(g, rows, d)
    xs[:, :2] = 0
    offsets = torch.tensor([0, rows], dtype=I32, device="cuda")
    ws = cs.new_moe_workspace(layer, rows)
    clean = torch.zeros(rows, d, dtype=BF, device="cuda")
    cs.moe_ffn_forward(layer, xs, offsets, clean, ws)
    edge = 181 / 128  # its square, times 2^127, is below fp32's largest value and rounds past bf16's
    for z, u in ((1e20, 1e25), (1e20, -1e25), (edge * 2.0 ** 63, edge * 2.0 ** 64)):
        bad = xs.clone()
        bad[1, 0], bad[1, 1] = z, u
        ys = torch.zeros_like(clean)
        cs.moe_ffn_forward(layer, bad, offsets, ys, ws)
        assert cs.check_status(ws) == 0
        want = torch.where((wd[0, 5] > 0) == (u > 0), float("inf"), float("-inf")).to(BF)
        assert torch.equal(ys[1], want)
        keep = [r for r in range(rows) if r != 1]
        assert torch.equal(ys[keep], clean[keep])


# ------------------------------------------------------------------------------ no tokens

def test_stack_of_no_tokens():
    """An empty batch goes through the layer and the stack as it goes through every call, captured too."""
    g = gen(31)
    blocks = stack_blocks(g, 8, 64, 64, 2)
    buf = stack.MoEBuffers.new(blocks[0], 0)
    h = torch.empty(0, 64, device="cuda")
    buf.offsets.fill_(-1)
    stack.moe_layer(blocks[0], buf.xn, buf.y, buf)
    assert (buf.offsets == 0).all()
    stack.moe_stack(blocks, h, buf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stack.moe_stack(blocks, h, buf)
    buf.offsets.fill_(-1)
    graph.replay()
    assert (buf.offsets == 0).all() and cs.check_status(buf.ws) == 0


# ------------------------------------------------------------------------------ the two parts of v

@pytest.mark.parametrize("act", ["silu", "relu"])
@pytest.mark.parametrize("d,h,counts,spare", [
    (64, 64, [20, 44], 0), (72, 136, [3, 5, 0, 30], 2), (256, 200, [0, 31, 33], 0), (64, 2048, [40], 0), (64, 64, [1] * 40, 7),
    (64, 64, [0] * 20 + [70, 0, 9], 1), (128, 1000, [33, 0, 7], 24), (264, 72, [1], 0), (1032, 64, [8] * 8, 0)])
def test_ffn_few_rows_keep_both_parts_of_v(d, h, counts, spare, act):
    """Up to max(64, 4 n_experts) rows v reaches the down product as a high and a low part: the tolerance
    has no bf16 rounding of v in it, and does not hold without the low part."""
    g = gen(d + h)
    n = sum(counts)
    assert n + spare <= max(64, 4 * len(counts))
    layer = make_experts(g, len(counts), d, h, act)
    xs = rnd(g, n, d)
    ys = check_ffn(layer, xs, counts, act, spare)
    off = np.concatenate([[0], np.cumsum(counts)])
    wg, wu, wd = np64(layer.w_gate), np64(layer.w_up), np64(layer.w_down_t)
    v, slip = oracle.moe_ffn_parts(np64(xs), off, wg, wu, act)
    want, _ = oracle.moe_ffn(np64(xs), off, wg, wu, wd, act)
    within(np64(ys[:n]), want, oracle.moe_ffn_tol_two_parts(v, slip, off, wd, want))


@pytest.mark.parametrize("E,rows", [(1, 64), (1, 65), (16, 64), (16, 65), (17, 68), (17, 69), (40, 160), (40, 161)])
def test_ffn_around_the_limit_of_few_rows(E, rows):
    """Row counts at the limit and one above it."""
    g = gen(E + rows)
    counts = [rows // E + (1 if e < rows % E else 0) for e in range(E)]
    layer = make_experts(g, E, 64, 64)
    xs = rnd(g, rows, 64)
    ys = check_ffn(layer, xs, counts)
    if rows <= max(64, 4 * E):
        off = np.concatenate([[0], np.cumsum(counts)])
        wd = np64(layer.w_down_t)
        v, slip = oracle.moe_ffn_parts(np64(xs), off, np64(layer.w_gate), np64(layer.w_up), "silu")
        want, _ = oracle.moe_ffn(np64(xs), off, np64(layer.w_gate), np64(layer.w_up), wd, "silu")
        within(np64(ys), want, oracle.moe_ffn_tol_two_parts(v, slip, off, wd, want))


@pytest.mark.parametrize("chained", [False, True])
@pytest.mark.parametrize("maker", ["block_norm", "dispatch", "ffn", "ffn few rows", "combine"])
def test_ffn_layer_of_weights_made_just_before(maker, chained):
    """The weights of a csffn_layer, whose decode steps read them before they wait, made in the stream just
    before by the calls that write rows, with and without a chained kernel in between; replayed, on weights
    that are NaN until they are made."""
    g = gen(77)
    d, h = (512, 5000) if maker != "ffn few rows" else (4096, 2048)
    fixed = [rnd(g, h, d, std=d ** -0.5) for _ in range(3)]
    w = torch.empty(h, d, dtype=BF, device="cuda")
    tokens = {1: rnd(g, 1, d), 16: rnd(g, 16, d)}
    src, src32 = rnd(g, h, d), rnd(g, h, d, dtype=F32)
    ids = torch.zeros(h, 1, dtype=I32, device="cuda")
    pos = torch.randperm(h, generator=g, device="cuda").to(I32)[:, None].contiguous()
    off, order, back = (torch.empty(n, dtype=I32, device="cuda") for n in (2, h, h))
    E = 1 if maker != "ffn few rows" else 512
    experts = make_experts(g, E, d, 64)
    bounds = torch.tensor([h * e // E for e in range(E + 1)], dtype=I32, device="cuda")
    ews, dws = cs.new_moe_workspace(experts, h), cs.new_moe_dispatch_workspace(h, 1)

    def make():
        if maker == "block_norm":
            cs.block_norm(src32, None, None, w)
        elif maker == "dispatch":
            cs.moe_dispatch(src, ids, off, order, back[:, None], w, dws)
        elif maker == "combine":
            cs.moe_combine(src, pos, None, w)
        else:
            cs.moe_ffn_forward(experts, src, bounds, w, ews)

    lg, ri, rw = rnd(g, 8, 16, dtype=F32), torch.empty(8, 2, dtype=I32, device="cuda"), torch.empty(8, 2, device="cuda")
    for place in range(3):  # as gate, up or down weights
        layer = cs.FFNLayer(*[w if i == place else fixed[i] for i in range(3)], _abi.ACT_SILU)
        buf = cs.DecodeBuffers.new(layer, 16)
        for step in ("sparse", "dense", "verify"):
            x = tokens[16 if step == "verify" else 1]
            out = torch.empty(x.shape[0], d, device="cuda")

            def use():
                if step == "sparse":
                    cs.cats_decode(layer, x, 0.05, out, buf)
                else:
                    cs.dense_ffn_forward(layer, x, out, buf.ws)
            make()
            torch.cuda.synchronize()
            use()
            want = out.double()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                w.fill_(float("nan"))
                make()
                if chained:
                    cs.moe_route(lg, ri, rw)
                use()
            for _ in range(3):
                out.fill_(float("nan"))
                graph.replay()
                # the sparse step adds its kept neurons' shares in the order they come: at most h fp32
                # additions of terms whose absolute sum is taken as 100 times the result's norm
                assert (out.double() - want).norm() <= 100 * h * U32 * want.norm()
            assert cs.check_status(buf.ws) == 0
