"""The routed FFN's operators and the block norm, as they are measured: cases, inputs, plain forms, 64-bit values.

A routed (mixture-of-experts) FFN layer of the residual stack runs, per layer: the block norm, the
router's projection and selection, the tokens sorted by expert, the experts' gated FFNs, and the
tokens back in order with their weights.  Each is a case family here ("op"):

  logits    router projection        l = x Wr^T                                (fp32 out)
  route     router selection         top-k experts of each token and their weights
  dispatch  tokens sorted by expert  offsets, order, inverse order, gathered rows
  ffn       the experts' gated FFN   ys = (act(xs Wg^T) * (xs Wu^T)) Wd        per expert, ragged rows
  combine   tokens back in order     out[t] = sum_j w[t, j] ys[pos[t, j]]
  norm      norms around a block     h' = a h + b gate * (rms(y) g_post), xn = rms(h') g_pre
"""
import math

import torch

own = False

EPS = 1e-6
NEG = float("-inf")
BF16 = torch.bfloat16


def listed():
    return [
        # one decode step of a few requests through the router's projection: latency
        {"name": "logits decode", "op": "logits", "T": 4, "E": 64, "d": 2048},
        # a long prompt through a wide router
        {"name": "logits prompt", "op": "logits", "T": 8192, "E": 128, "d": 4096},
        # selection for one decode step: softmax over all experts, the selected weights renormalised
        {"name": "route decode", "op": "route", "T": 16, "E": 64, "k": 8, "score": "softmax", "renorm": True,
         "bias": False, "dtype": "f32", "masked": 0.0},
        # selection for a long prompt from bf16 logits (ties), a balancing bias on the keys, some experts masked
        {"name": "route prompt", "op": "route", "T": 16384, "E": 160, "k": 6, "score": "sigmoid", "renorm": True,
         "bias": True, "dtype": "bf16", "masked": 0.05},
        # 13 requests' tokens to their experts: latency, odd count
        {"name": "dispatch decode", "op": "dispatch", "T": 13, "E": 64, "k": 8, "d": 2048, "dtype": "bf16", "drop": 0.0},
        # a padded prompt batch: an eighth of the tokens are padding (expert -1), skewed load
        {"name": "dispatch prompt", "op": "dispatch", "T": 8192, "E": 64, "k": 8, "d": 2048, "dtype": "bf16", "drop": 0.125},
        # the same prompt's expert outputs back to token order
        {"name": "combine prompt", "op": "combine", "T": 8192, "E": 64, "k": 8, "d": 2048, "dtype": "bf16", "drop": 0.125},
        # one token through 8 of 64 small experts: the weights' stream and the launches
        {"name": "ffn one token", "op": "ffn", "T": 1, "E": 64, "k": 8, "d": 2048, "h": 1024, "act": "silu", "drop": 0.0},
        # 16 requests through 2 of 8 large experts (the 8B stack's FFN shape): the weights' stream
        {"name": "ffn decode batch", "op": "ffn", "T": 16, "E": 8, "k": 2, "d": 4096, "h": 14336, "act": "silu", "drop": 0.0},
        # a prompt through the same experts: the tensor cores
        {"name": "ffn prompt", "op": "ffn", "T": 4096, "E": 8, "k": 2, "d": 4096, "h": 14336, "act": "silu", "drop": 0.03},
        # the norms around a block at decode: 16 tokens
        {"name": "norm decode", "op": "norm", "T": 16, "d": 4096, "y": "bf16", "post": True, "gate": "channel", "pre": True},
        # the same for a prompt batch, with a gate of each token's own
        {"name": "norm prompt", "op": "norm", "T": 8192, "d": 4096, "y": "bf16", "post": True, "gate": "token", "pre": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logits", "route", "dispatch", "ffn", "combine", "norm"])
    if op == "logits":
        return {"op": op, "T": _log(rng, 1, 8192), "E": rng.randint(4, 128), "d": 8 * _log(rng, 32, 512)}
    if op == "route":
        E = rng.randint(2, 160)
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(E, 8)),
                "score": rng.choice(["softmax", "sigmoid"]), "renorm": rng.random() < 0.6, "bias": rng.random() < 0.4,
                "dtype": rng.choice(["f32", "bf16"]), "masked": rng.choice([0.0, 0.1, 0.9])}
    if op in ("dispatch", "combine"):
        E = rng.randint(2, 128)
        return {"op": op, "T": _log(rng, 1, 8192), "E": E, "k": rng.randint(1, min(E, 8)), "d": 8 * _log(rng, 32, 256),
                "dtype": rng.choice(["bf16", "f32"]) if op == "dispatch" else "bf16", "drop": rng.choice([0.0, 0.1, 0.6])}
    if op == "ffn":
        E = rng.choice([2, 5, 8, 16, 32, 64])
        # the experts' weights together stay within the largest listed case's
        d, h = 8 * _log(rng, 32, 512), 8 * _log(rng, 16, 1792)
        while E * d * h > 8 * 4096 * 14336:
            h = max(8, h // 16 * 8)
        k = rng.randint(1, min(E, 8))
        rows = _log(rng, 1, 8192)
        return {"op": op, "T": max(1, rows // k), "E": E, "k": k, "d": d, "h": h, "act": rng.choice(["silu", "relu"]),
                "drop": rng.choice([0.0, 0.1, 0.5])}
    return {"op": op, "T": _log(rng, 1, 8192), "d": 8 * _log(rng, 16, 512), "y": rng.choice(["bf16", "f32"]),
            "post": rng.random() < 0.7, "gate": rng.choice(["none", "channel", "token"]), "pre": rng.random() < 0.8}


# ---------------------------------------------------------------------------- inputs

def _dtype(name):
    return BF16 if name == "bf16" else torch.float32


def _routing(case, g):
    """Expert ids [T, k] of a skewed router (distinct per token), whole tokens dropped as padding, and weights."""
    T, E, k = case["T"], case["E"], case["k"]
    skew = torch.randn(E, device="cuda", generator=g) * 0.7
    noise = torch.rand(T, E, device="cuda", generator=g).clamp_min(1e-12)
    score = skew - torch.log(-torch.log(noise).clamp_min(1e-12))
    top = torch.sort(score, dim=1, descending=True, stable=True)
    ids = top.indices[:, :k].to(torch.int32).contiguous()
    pad = torch.rand(T, 1, device="cuda", generator=g) < case["drop"]
    ids = torch.where(pad, torch.full_like(ids, -1), ids).contiguous()
    w = torch.rand(T, k, device="cuda", generator=g) + 0.05
    w = (w / w.sum(1, keepdim=True)).contiguous()
    return ids, w


def _plan(ids, E):
    """offsets [E + 1], order, pos of the stable sort by expert, in elementary operations (int32)."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.sort(key, stable=True).indices
    edges = torch.arange(E + 1, device=ids.device)
    offsets = (key[None, :] < edges[:, None]).sum(1) if n * (E + 1) < (1 << 24) else torch.cumsum(
        torch.zeros(E + 1, dtype=torch.long, device=ids.device).scatter_add_(0, (key + 1).clamp_max(E), (key < E).long()), 0)
    rank = torch.empty_like(order).scatter_(0, order, torch.arange(n, device=ids.device))
    keep = torch.arange(n, device=ids.device) < offsets[E]
    pos = torch.where(key < E, rank, torch.full_like(rank, -1))
    order = torch.where(keep, order, torch.full_like(order, -1))
    return offsets.to(torch.int32), order.to(torch.int32), pos.to(torch.int32).reshape(ids.shape), keep


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, device="cuda", generator=g, dtype=dtype) * std

    s = {"case": case}
    if op == "logits":
        T, E, d = case["T"], case["E"], case["d"]
        s["x"] = normal(T, d, dtype=BF16)
        s["w"] = normal(E, d, std=d ** -0.5, dtype=BF16)
        s["out"] = torch.zeros(T, E, device="cuda")
    elif op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        logits = normal(T, E, std=1.5).to(_dtype(case["dtype"]))
        logits[torch.rand(T, E, device="cuda", generator=g) < case["masked"]] = NEG
        s["logits"] = logits
        s["bias"] = normal(E, std=0.1) if case["bias"] else None
        s["ids"] = torch.zeros(T, k, dtype=torch.int32, device="cuda")
        s["weights"] = torch.zeros(T, k, device="cuda")
    elif op == "dispatch":
        T, E, k, d = case["T"], case["E"], case["k"], case["d"]
        s["ids"], _ = _routing(case, g)
        s["x"] = normal(T, d).to(_dtype(case["dtype"]))
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        s["order"] = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
        s["pos"] = torch.zeros(T, k, dtype=torch.int32, device="cuda")
        s["xs"] = torch.zeros(T * k, d, dtype=s["x"].dtype, device="cuda")
        if own:
            from contextual_sparsity_ffn_b200 import binding as cs
            s["ws"] = cs.new_moe_dispatch_workspace(T * k, E)
    elif op == "combine":
        T, E, k, d = case["T"], case["E"], case["k"], case["d"]
        ids, s["weights"] = _routing(case, g)
        _, _, s["pos"], _ = _plan(ids, E)
        s["ys"] = normal(T * k, d).to(BF16)
        s["out"] = torch.zeros(T, d, dtype=BF16, device="cuda")
    elif op == "ffn":
        T, E, k, d, h = case["T"], case["E"], case["k"], case["d"], case["h"]
        ids, _ = _routing(case, g)
        s["offsets"], _, _, _ = _plan(ids, E)
        s["bounds"] = s["offsets"].tolist()
        s["xs"] = normal(T * k, d, dtype=BF16)
        s["wg"] = torch.empty(E, h, d, dtype=BF16, device="cuda").normal_(0, d ** -0.5, generator=g)
        s["wu"] = torch.empty(E, h, d, dtype=BF16, device="cuda").normal_(0, d ** -0.5, generator=g)
        s["wd"] = torch.empty(E, h, d, dtype=BF16, device="cuda").normal_(0, h ** -0.5, generator=g)
        s["ys"] = torch.zeros(T * k, d, dtype=BF16, device="cuda")
        if own:
            from contextual_sparsity_ffn_b200 import binding as cs
            s["layer"] = cs.MoELayer(s["wg"], s["wu"], s["wd"], cs._abi.ACT_SILU if case["act"] == "silu" else cs._abi.ACT_RELU)
            s["ws"] = cs.new_moe_workspace(s["layer"], T * k)
    else:
        T, d = case["T"], case["d"]
        s["h"] = normal(T, d, std=2.0)
        s["y"] = normal(T, d).to(_dtype(case["y"]))
        s["g_post"] = 1 + normal(d, std=0.1) if case["post"] else None
        s["gate"] = None if case["gate"] == "none" else normal(d) if case["gate"] == "channel" else normal(T, d)
        s["g_pre"] = 1 + normal(d, std=0.1) if case["pre"] else None
        s["h_out"] = torch.zeros(T, d, device="cuda")
        s["xn"] = torch.zeros(T, d, dtype=BF16, device="cuda") if case["pre"] else None
        s["a"], s["b"] = 1.0, 0.7
    return s


# ---------------------------------------------------------------------------- one pass

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from contextual_sparsity_ffn_b200 import binding as cs
    c = s["case"]
    op = c["op"]
    if op == "logits":
        cs.moe_logits(s["x"], s["w"], s["out"])
        return s["out"]
    if op == "route":
        cs.moe_route(s["logits"], s["ids"], s["weights"], bias=s["bias"],
                     score=cs._abi.ROUTE_SOFTMAX if c["score"] == "softmax" else cs._abi.ROUTE_SIGMOID,
                     renormalize=c["renorm"])
        return s["ids"], s["weights"]
    if op == "dispatch":
        cs.moe_dispatch(s["x"], s["ids"], s["offsets"], s["order"], s["pos"], s["xs"], s["ws"])
        return s["offsets"], s["order"], s["pos"], s["xs"]
    if op == "combine":
        cs.moe_combine(s["ys"], s["pos"], s["weights"], s["out"])
        return s["out"]
    if op == "ffn":
        cs.moe_ffn_forward(s["layer"], s["xs"], s["offsets"], s["ys"], s["ws"])
        return s["ys"]
    cs.block_norm(s["h"], s["y"], s["h_out"], s["xn"], g_post=s["g_post"], gate=s["gate"], g_pre=s["g_pre"],
                  res_scale=s["a"], out_scale=s["b"], eps=EPS)
    return (s["h_out"], s["xn"]) if c["pre"] else s["h_out"]


def _act(z, name):
    return z / (1 + torch.exp(-z)) if name == "silu" else torch.clamp_min(z, 0)


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "logits":
        return s["x"].float() @ s["w"].float().T
    if op == "route":
        logits = s["logits"].float()
        key = logits if s["bias"] is None else logits + s["bias"]
        key = torch.where(torch.isnan(key), torch.full_like(key, NEG), key)
        top = torch.sort(key, dim=1, descending=True, stable=True)
        k = c["k"]
        ok = top.values[:, :k] > NEG
        ids = top.indices[:, :k]
        sel = torch.gather(logits, 1, ids)
        if c["score"] == "sigmoid":
            w = torch.where(ok, 1 / (1 + torch.exp(-sel)), torch.zeros_like(sel))
            if c["renorm"]:
                w = w / w.sum(1, keepdim=True).clamp_min(1e-20)
        else:
            among = torch.where(ok, sel, torch.full_like(sel, NEG)) if c["renorm"] else logits
            top_l = among.amax(1, keepdim=True).clamp_min(-3e38)
            w = torch.where(ok, torch.exp(sel - top_l), torch.zeros_like(sel))
            w = w / torch.exp(among - top_l).sum(1, keepdim=True).clamp_min(1e-20)
        return torch.where(ok, ids, torch.full_like(ids, -1)).to(torch.int32), w
    if op == "dispatch":
        offsets, order, pos, keep = _plan(s["ids"], c["E"])
        rows = s["x"][torch.where(keep, order.long() // c["k"], torch.zeros_like(order, dtype=torch.long))]
        return offsets, order, pos, torch.where(keep[:, None], rows, torch.zeros_like(rows))
    if op == "combine":
        pos = s["pos"].long()
        w = torch.where(pos >= 0, s["weights"], torch.zeros_like(s["weights"]))
        rows = s["ys"][pos.clamp_min(0).reshape(-1)].reshape(*pos.shape, -1).float()
        return (rows * w[:, :, None]).sum(1).to(BF16)
    if op == "ffn":
        ys = torch.zeros_like(s["xs"])
        b = s["bounds"]
        for e in range(c["E"]):  # the experts that got rows, one after the other
            if b[e + 1] > b[e]:
                x = s["xs"][b[e]:b[e + 1]].float()
                v = _act(x @ s["wg"][e].float().T, c["act"]) * (x @ s["wu"][e].float().T)
                ys[b[e]:b[e + 1]] = (v @ s["wd"][e].float()).to(BF16)
        return ys
    y = s["y"].float()
    if s["g_post"] is not None:
        y = y / torch.sqrt((y * y).mean(1, keepdim=True) + EPS) * s["g_post"]
    if s["gate"] is not None:
        y = y * s["gate"]
    h = s["a"] * s["h"] + s["b"] * y
    if s["g_pre"] is None:
        return h
    return h, (h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * s["g_pre"]).to(BF16)


# ---------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, T = case["op"], case["T"]
    es = 2 if case.get("dtype") == "bf16" else 4
    if op == "logits":
        E, d = case["E"], case["d"]
        return {"bytes": 2 * (T + E) * d + 4 * T * E, "flops": 2 * T * E * d}
    if op == "route":
        return {"bytes": T * case["E"] * es + 8 * T * case["k"], "flops": T * case["E"] * 4}
    k = case.get("k", 1)
    n = T * k * (1 - case.get("drop", 0.0))
    if op == "dispatch":
        return {"bytes": T * case["d"] * es + n * case["d"] * es + 12 * T * k, "flops": T * k}
    if op == "combine":
        return {"bytes": n * case["d"] * 2 + 2 * T * case["d"] + 8 * T * k, "flops": 2 * n * case["d"]}
    if op == "ffn":
        d, h, E = case["d"], case["h"], case["E"]
        active = E * (1 - (1 - k / E) ** max(1.0, T * (1 - case["drop"])))  # experts a uniform router reaches
        return {"bytes": active * 6 * d * h + 4 * n * d, "flops": 6 * n * d * h}
    d, ys = case["d"], 2 if case["y"] == "bf16" else 4
    per = 8 + ys + (4 if case["gate"] == "token" else 0) + (2 if case["pre"] else 0)
    return {"bytes": T * d * per + 4 * d * 3, "flops": 10 * T * d}


# ---------------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "logits":
        return torch.einsum("td,ed->te", s["x"].to(f64), s["w"].to(f64))
    if op == "route":
        lg = s["logits"].to(f64)
        key = s["logits"].float() + (0.0 if s["bias"] is None else s["bias"][None, :])  # the keys are fp32 sums by definition
        T, E = lg.shape
        ids = torch.full((T, case["k"]), -1, dtype=torch.int64, device="cuda")
        left = key.clone()
        for j in range(case["k"]):  # the best of those left, the lowest of equals
            best = left.amax(1, keepdim=True)
            first = torch.where(left == best, torch.arange(E, device="cuda")[None, :], E).amin(1)
            found = best[:, 0] > NEG
            ids[:, j] = torch.where(found, first, -1)
            left[torch.arange(T, device="cuda"), first.clamp_max(E - 1)] = NEG
        ok = ids >= 0
        sel = torch.gather(lg, 1, ids.clamp_min(0))
        if case["score"] == "sigmoid":
            w = torch.sigmoid(sel) * ok
            w = w / w.sum(1, keepdim=True).clamp_min(1e-20) if case["renorm"] else w
        elif case["renorm"]:
            w = torch.nan_to_num(torch.softmax(sel.masked_fill(~ok, NEG), 1), nan=0.0)
        else:
            w = torch.gather(torch.nan_to_num(torch.softmax(lg, 1), nan=0.0), 1, ids.clamp_min(0)) * ok
        return ids.to(torch.int32), w
    if op == "dispatch":
        return None
    if op == "combine":
        out = torch.zeros(case["T"], case["d"], dtype=f64, device="cuda")
        for j in range(case["k"]):
            p = s["pos"][:, j].long()
            t = torch.nonzero(p >= 0)[:, 0]
            out[t] += s["weights"][t, j, None].to(f64) * s["ys"][p[t]].to(f64)
        return out
    if op == "ffn":
        ys = torch.zeros(s["xs"].shape, dtype=f64, device="cuda")
        b = s["bounds"]
        for e in range(case["E"]):
            x = s["xs"][b[e]:b[e + 1]].to(f64)
            if x.shape[0]:
                z = torch.einsum("nd,hd->nh", x, s["wg"][e].to(f64))
                z = z * torch.sigmoid(z) if case["act"] == "silu" else torch.relu(z)
                ys[b[e]:b[e + 1]] = torch.einsum("nh,hd->nd", z * torch.einsum("nd,hd->nh", x, s["wu"][e].to(f64)), s["wd"][e].to(f64))
        return ys
    h, y = s["h"].to(f64), s["y"].to(f64)
    if case["post"]:
        y = y * torch.rsqrt(y.square().mean(1, keepdim=True) + EPS) * s["g_post"].to(f64)
    if case["gate"] != "none":
        y = y * s["gate"].to(f64)
    h = s["a"] * h + s["b"] * y
    if not case["pre"]:
        return h
    return h, h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["g_pre"].to(f64)
