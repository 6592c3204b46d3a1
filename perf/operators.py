"""Timed cases of the operators on either side of the compressed exchange.

In data-parallel training of mixture-of-experts models the exchanged tensors
are expert chunks (all-to-all), gradients (reduce-scatter) and parameters
(all-gather).  The operators here make and use them: ``moe_route`` chooses
each token's experts, ``moe_plan`` lays the chosen pairs out as one chunk per
expert, ``moe_dispatch`` fills the chunks, ``moe_combine`` brings the experts'
rows back to their tokens, and ``adamw_step`` turns a reduced gradient shard
into new parameters.

Each case runs either way: ``own`` false, the operator in its plain form
(elementary torch operations in 32 bits, rounded once at the end); ``own``
true, the package's own calls.  ``exact`` gives the same answers from the
definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 256                    # values that share one scale of an 8-bit optimizer state
F8_MAX = 448.0                 # largest value of torch.float8_e4m3fn
F8_MIN = 2.0 ** -9             # smallest positive one
SCALE_MIN = 2.0 ** -126        # smallest scale: an all-zero block has a scale too
ADAMW = {"lr": 3e-4, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1, "step": 1000}
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# One rank's eighth of four layers of the 4096-wide, 14336-deep weight stack
# that the package's parameter workload has: q, k, v, o, gate, up, down.
SHARD = [4096 * 4096, 1024 * 4096, 1024 * 4096, 4096 * 4096, 14336 * 4096, 14336 * 4096, 14336 * 4096]
SHARD = [n // 8 for n in SHARD] * 4


def listed():
    return [
        # one new token while generating: what counts is the latency of the call
        {"name": "route, one token", "op": "route", "tokens": 1, "experts": 64, "top_k": 2, "type": "bf16",
         "score": "softmax", "bias": False, "groups": 1, "kept": 1, "group_score": "max", "renorm": True,
         "scale": 1.0, "masked": 0.0, "train": False},
        # a batch of prompts: sigmoid scores with balance bias, experts in groups
        {"name": "route, prompts in groups", "op": "route", "tokens": 8192, "experts": 256, "top_k": 8,
         "type": "f32", "score": "sigmoid", "bias": True, "groups": 8, "kept": 4, "group_score": "top2",
         "renorm": True, "scale": 2.5, "masked": 0.0, "train": False},
        # the training batch of the package's all-to-all workload, forward and backward
        {"name": "route, training batch", "op": "route", "tokens": 16384, "experts": 64, "top_k": 2, "type": "f32",
         "score": "softmax", "bias": False, "groups": 1, "kept": 1, "group_score": "max", "renorm": True,
         "scale": 1.0, "masked": 0.02, "train": True},
        # a few tokens of several generating requests
        {"name": "plan, few tokens", "op": "plan", "tokens": 61, "experts": 64, "top_k": 2, "dropped": 0.0},
        # a long training batch over many experts, padding among it
        {"name": "plan, long batch", "op": "plan", "tokens": 65536, "experts": 256, "top_k": 8, "dropped": 0.03},
        # the package's all-to-all workload: 16,384 tokens of 4,096, two experts each, forward and backward
        {"name": "dispatch, training batch", "op": "dispatch", "tokens": 16384, "hidden": 4096, "experts": 64,
         "top_k": 2, "type": "bf16", "dropped": 0.0, "strided": False, "train": True},
        # an odd width, rows that are a slice of wider ones, padding tokens
        {"name": "dispatch, odd width", "op": "dispatch", "tokens": 1021, "hidden": 2055, "experts": 48,
         "top_k": 6, "type": "bf16", "dropped": 0.05, "strided": True, "train": False},
        # generating: a handful of tokens, the residual added on the way
        {"name": "combine, few tokens", "op": "combine", "tokens": 7, "hidden": 4096, "experts": 64, "top_k": 2,
         "type": "bf16", "dropped": 0.0, "residual": True, "train": False},
        # the training batch again, forward and backward
        {"name": "combine, training batch", "op": "combine", "tokens": 16384, "hidden": 4096, "experts": 64,
         "top_k": 2, "type": "bf16", "dropped": 0.02, "residual": False, "train": True},
        # norms and biases of odd sizes, packed without padding
        {"name": "adamw, small odd tensors", "op": "adamw", "sizes": "odd", "tensors": 9, "values": 40000,
         "bits": 32, "param": "f32", "grad": "f32", "copy": False, "clip": True},
        # one rank's shard of the parameter workload: 28 tensors, 109,051,904 values
        {"name": "adamw, shard", "op": "adamw", "sizes": "shard", "tensors": 28, "values": sum(SHARD), "bits": 32,
         "param": "f32", "grad": "bf16", "copy": True, "clip": False},
        # the same shard with its states held in 8 bits
        {"name": "adamw, shard, 8-bit states", "op": "adamw", "sizes": "shard", "tensors": 28,
         "values": sum(SHARD), "bits": 8, "param": "f32", "grad": "bf16", "copy": True, "clip": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "plan", "dispatch", "combine", "adamw", "adamw"])
    if op == "route":
        groups = rng.choice([1, 1, 1, 2, 4, 5, 8])
        experts = groups * rng.randint(2, 384 // groups)
        kept = rng.randint(1, groups)
        top_k = rng.randint(1, min(10, kept * (experts // groups)))
        return {"op": op, "tokens": _log(rng, 1, 32768), "experts": experts, "top_k": top_k,
                "type": rng.choice(["bf16", "f32", "f16"]), "score": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.5, "groups": groups, "kept": kept,
                "group_score": rng.choice(["max", "top2"]), "renorm": rng.random() < 0.7,
                "scale": rng.choice([1.0, 2.5]), "masked": rng.choice([0.0, 0.04]), "train": rng.random() < 0.5}
    if op == "plan":
        top_k = rng.randint(1, 10)
        return {"op": op, "tokens": _log(rng, 1, 524288 // top_k), "experts": rng.randint(max(4, top_k), 384),
                "top_k": top_k, "dropped": rng.choice([0.0, 0.05])}
    if op in ("dispatch", "combine"):
        top_k = rng.randint(1, 8)
        hidden = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            hidden = max(64, hidden // 64 * 64)
        case = {"op": op, "tokens": _log(rng, 1, max(2, min(16384, 100_000_000 // (hidden * top_k)))), "hidden": hidden,
                "experts": rng.randint(max(4, top_k), 256), "top_k": top_k, "type": rng.choice(["bf16", "bf16", "f16", "f32"]),
                "dropped": rng.choice([0.0, 0.05]), "train": rng.random() < 0.5}
        case["strided" if op == "dispatch" else "residual"] = rng.random() < 0.4
        return case
    param = rng.choice(["f32", "f32", "bf16"])
    return {"op": op, "sizes": rng.choice(["odd", "even"]), "tensors": rng.randint(1, 40),
            "values": _log(rng, 2000, 60_000_000), "bits": rng.choice([32, 8]), "param": param,
            "grad": rng.choice(["bf16", "f32"]), "copy": param == "f32" and rng.random() < 0.6,
            "clip": rng.random() < 0.4}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _scores64(case, logits, bias):
    """What the experts are chosen by, in 64 bits: the score with the balance bias."""
    l = logits.double()
    s = l.softmax(-1) if case["score"] == "softmax" else l.sigmoid()
    return s if bias is None else s + bias.double()


def _undecided(case, logits, bias):
    """Tokens whose choice hangs on the last bits of a score: two different
    scores nearer to each other than 32-bit arithmetic tells apart."""
    T, E = logits.shape
    c = _scores64(case, logits, bias)
    if case["groups"] > 1:
        g = c.view(T, case["groups"], -1)
        n = 2 if case["group_score"] == "top2" and g.shape[-1] > 1 else 1
        score = g.topk(n, -1).values.sum(-1)
        order = score.sort(dim=-1, descending=True, stable=True)
        keep = torch.zeros_like(score, dtype=torch.bool).scatter_(1, order.indices[:, :case["kept"]], True)
        c = c.masked_fill(~keep.repeat_interleave(E // case["groups"], 1), -1.0)
        edge = order.values[:, case["kept"] - 1:case["kept"] + 1]
        near = ((edge[:, :1] - edge[:, 1:]) > 0) & ((edge[:, :1] - edge[:, 1:]) < 3e-6)
        bad = near.any(-1)
    else:
        bad = torch.zeros(T, dtype=torch.bool, device=logits.device)
    top = c.topk(min(E, case["top_k"] + 1), -1).values
    gap = top[:, :-1] - top[:, 1:]
    return bad | ((gap > 0) & (gap < 3e-6 * top[:, :1].abs().clamp(max=1.0))).any(-1)


def _logits(case, gen):
    T, E = case["tokens"], case["experts"]
    dt = TYPES[case["type"]]
    bias = None
    if case["bias"]:  # as balance rules leave it: a whole number of steps of 0.001
        bias = torch.randint(-20, 21, (E,), generator=gen, device="cuda").float() * 1e-3
    logits = (1.5 * torch.randn(T, E, generator=gen, device="cuda")).to(dt)
    if case["score"] == "softmax" and bias is None and (case["groups"] == 1 or case["group_score"] == "max"):
        return logits, bias  # chosen by the logits themselves: nothing is rounded
    for _ in range(6):
        bad = _undecided(case, logits, bias)
        again = (1.5 * torch.randn(T, E, generator=gen, device="cuda")).to(dt)
        logits = torch.where(bad[:, None], again, logits)
    bad = _undecided(case, logits, bias)
    steps = 2.0 - 5.0 * torch.arange(E, device="cuda") / E
    return torch.where(bad[:, None], steps.to(dt), logits), bias


def _ids(case, gen):
    """Expert ids as a router leaves them: distinct for a token, uneven over the
    experts; a dropped (masked) token has -1 throughout."""
    T, E, K = case["tokens"], case["experts"], case["top_k"]
    pull = 0.5 * torch.randn(E, generator=gen, device="cuda")
    ids = (torch.randn(T, E, generator=gen, device="cuda") + pull).topk(K, -1).indices
    gone = torch.rand(T, generator=gen, device="cuda") < case["dropped"]
    return torch.where(gone[:, None], torch.full_like(ids, -1), ids).to(torch.int32).contiguous()


def _sizes(case):
    if case["sizes"] == "shard":
        return list(SHARD)
    n, total = case["tensors"], case["values"]
    g = torch.Generator()
    g.manual_seed(total)
    parts = (torch.rand(n, generator=g) + 0.1).tolist()
    sizes = [max(1, int(total * p / sum(parts))) for p in parts]
    if case["sizes"] == "even":
        return [max(1024, s // 1024 * 1024) for s in sizes]
    return [s | 1 for s in sizes]


def _quantize(x, raise_small):
    """8-bit form of blocks of 256 values: codes and one scale for each block."""
    x = x.view(-1, BLOCK)
    scale = (x.abs().amax(-1) * (1.0 / F8_MAX)).clamp(min=SCALE_MIN)
    y = x * (1.0 / scale)[:, None]
    if raise_small:
        y = torch.where(x > 0, y.clamp(min=F8_MIN), y)
    return y.to(torch.float8_e4m3fn).view(-1), scale


def _pieces(flat, starts, sizes):
    return [flat[a:a + n] for a, n in zip(starts, sizes)]


def prepare(case, seed):
    gen = _generator(seed)
    op = case["op"]
    if op == "route":
        logits, bias = _logits(case, gen)
        T = case["tokens"]
        mask = None
        if case["masked"]:
            mask = torch.rand(T, generator=gen, device="cuda") >= case["masked"]
        grad = torch.randn(T, case["top_k"], generator=gen, device="cuda") if case["train"] else None
        return {"case": case, "logits": logits, "bias": bias, "mask": mask, "grad": grad}
    if op == "plan":
        return {"case": case, "ids": _ids(case, gen)}
    if op in ("dispatch", "combine"):
        T, H, K = case["tokens"], case["hidden"], case["top_k"]
        dt = TYPES[case["type"]]
        slots = _plan(_ids(case, gen), case["experts"])[2]
        state = {"case": case, "slots": slots}
        if op == "dispatch":
            wide = torch.randn(T, H + (41 if case["strided"] else 0), generator=gen, device="cuda").to(dt)
            state["x"] = wide[:, :H]
            if case["train"]:
                state["grad"] = torch.randn(T * K, H, generator=gen, device="cuda").to(dt)
            return state
        state["rows"] = torch.randn(T * K, H, generator=gen, device="cuda").to(dt)
        w = torch.rand(T, K, generator=gen, device="cuda") + 0.05
        state["weights"] = w / w.sum(-1, keepdim=True)
        state["residual"] = torch.randn(T, H, generator=gen, device="cuda").to(dt) if case["residual"] else None
        if case["train"]:
            state["grad"] = torch.randn(T, H, generator=gen, device="cuda").to(dt)
        return state
    # optimizer: every tensor is a piece of a flat buffer, as sharded training keeps them
    sizes = _sizes(case)
    pad = BLOCK if case["bits"] == 8 else 1
    starts, total = [], 0
    for n in sizes:
        starts.append(total)
        total += -(-n // pad) * pad
    live = torch.zeros(total, device="cuda")
    for piece in _pieces(live, starts, sizes):
        piece.fill_(1.0)

    def normal(sigma):
        return torch.randn(total, generator=gen, device="cuda").mul_(sigma).mul_(live)

    dt = TYPES[case["param"]]
    flat = {"param": normal(0.02).to(dt), "grad": normal(1e-3).to(TYPES[case["grad"]])}
    m, r = normal(3e-4), normal(1e-3).abs_().add_(live, alpha=1e-4)
    if case["bits"] == 8:
        flat["avg"], flat["avg_scale"] = _quantize(m, False)
        flat["rms"], flat["rms_scale"] = _quantize(r, True)
    else:
        flat["avg"], flat["sq"] = m, r.square_()
    if case["copy"]:
        flat["copy"] = flat["param"].to(torch.bfloat16)
    lists = {k: _pieces(v, starts, sizes) for k, v in flat.items() if not k.endswith("_scale")}
    blocks = [(a // BLOCK, -(-n // BLOCK)) for a, n in zip(starts, sizes)]
    lists |= {k: [v[a:a + n] for a, n in blocks] for k, v in flat.items() if k.endswith("_scale")}
    clip = torch.full((1,), 0.37, device="cuda") if case["clip"] else None
    return {"case": case, "flat": flat, "lists": lists, "clip": clip}


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    return (_run_own if own else _run_plain)(case, state)


def _run_own(case, state):
    import lossless_bf16_tensor_zipccl_gb300 as zc
    op = case["op"]
    if op == "route":
        how = {"score": case["score"], "renormalize": case["renorm"], "scale": case["scale"]}
        weights, ids = zc.moe_route(state["logits"], case["top_k"], bias=state["bias"], groups=case["groups"],
                                    groups_kept=case["kept"], group_score=case["group_score"], mask=state["mask"],
                                    **how)
        out = {"weights": weights, "ids": ids}
        if case["train"]:
            out["grad_logits"] = zc.moe_route_backward(state["grad"], state["logits"], ids, **how)
        return out
    if op == "plan":
        counts, offsets, slots = zc.moe_plan(state["ids"], case["experts"])
        return {"counts": counts, "offsets": offsets, "slots": slots}
    if op == "dispatch":
        out = {"rows": zc.moe_dispatch(state["x"], state["slots"])}
        if case["train"]:
            out["grad_x"] = zc.moe_dispatch_backward(state["grad"], state["slots"])
        return out
    if op == "combine":
        out = {"y": zc.moe_combine(state["rows"], state["slots"], state["weights"], residual=state["residual"])}
        if case["train"]:
            out["grad_rows"], out["grad_weights"] = zc.moe_combine_backward(state["grad"], state["rows"],
                                                                            state["slots"], state["weights"])
        return out
    l = state["lists"]
    zc.adamw_step(l["param"], l["grad"], l["avg"], l["rms"] if case["bits"] == 8 else l["sq"],
                  scales=(l["avg_scale"], l["rms_scale"]) if case["bits"] == 8 else None, copies=l.get("copy"),
                  grad_scale=state["clip"], step=ADAMW["step"], lr=ADAMW["lr"],
                  betas=(ADAMW["beta1"], ADAMW["beta2"]), eps=ADAMW["eps"], weight_decay=ADAMW["weight_decay"])
    return {k: v for k, v in state["flat"].items() if k != "grad"}


def _run_plain(case, state):
    op = case["op"]
    if op == "route":
        return _route(case, state)
    if op == "plan":
        return dict(zip(("counts", "offsets", "slots"), _plan(state["ids"], case["experts"])))
    if op == "dispatch":
        x, slots = state["x"], state["slots"]
        out = {"rows": _rows_of(x.float(), slots).to(x.dtype)}
        if case["train"]:
            g = state["grad"]
            out["grad_x"] = _gathered(g.float(), slots).sum(1).to(g.dtype)
        return out
    if op == "combine":
        rows, slots, w = state["rows"], state["slots"], state["weights"]
        picked = _gathered(rows.float(), slots)
        y = (picked * w[:, :, None]).sum(1)
        if state["residual"] is not None:
            y = y + state["residual"].float()
        out = {"y": y.to(rows.dtype)}
        if case["train"]:
            g = state["grad"].float()
            back = torch.zeros_like(rows)
            flat = slots.view(-1).long()
            back[torch.where(flat < 0, -1 - flat, flat)] = (torch.where((slots < 0)[:, :, None], 0.0, w[:, :, None] * g[:, None, :])
                                                           .view(-1, rows.shape[1]).to(rows.dtype))
            out["grad_rows"] = back
            out["grad_weights"] = (picked * g[:, None, :]).sum(-1)
        return out
    return _adamw(case, state)


def _route(case, state):
    logits = state["logits"].float()
    T, E = logits.shape
    K, G = case["top_k"], case["groups"]
    l = logits.clamp(max=torch.finfo(torch.float32).max)
    fit = l > -math.inf
    if state["mask"] is not None:
        fit = fit & state["mask"][:, None]
    soft = case["score"] == "softmax"
    if soft:
        e = torch.where(fit, torch.exp(l - torch.where(fit, l, -math.inf).amax(-1, keepdim=True)), 0.0)
        s = e / e.sum(-1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-l))
    by_logit = soft and state["bias"] is None and (G == 1 or case["group_score"] == "max")
    c = l if by_logit else s if state["bias"] is None else s + state["bias"]
    c = torch.where(fit, c, -math.inf)
    if G > 1:
        g = c.view(T, G, E // G)
        score = g.amax(-1)
        if case["group_score"] == "top2" and E // G > 1:
            pair = g.topk(2, -1).values
            score = torch.where(pair[..., 1] > -math.inf, pair.sum(-1), score)
        best = score.sort(dim=-1, descending=True, stable=True).indices[:, :case["kept"]]
        keep = torch.zeros_like(score, dtype=torch.bool).scatter(1, best, True)
        c = torch.where(keep[:, :, None], g, -math.inf).view(T, E)
    order = c.sort(dim=-1, descending=True, stable=True)
    ids = order.indices[:, :K]
    there = order.values[:, :K] > -math.inf
    w = torch.where(there, s.gather(1, ids), 0.0)
    if case["renorm"]:
        if soft:  # the same quotient, taken over the chosen logits alone
            top = torch.where(there, l.gather(1, ids), -math.inf)
            w = torch.where(there, torch.exp(top - top.amax(-1, keepdim=True)), 0.0)
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    out = {"weights": w * case["scale"], "ids": torch.where(there, ids, -1).to(torch.int32)}
    if case["train"]:
        d = torch.where(there, state["grad"], 0.0) * case["scale"]
        if case["renorm"]:
            u = w * (d - (w * d).sum(-1, keepdim=True))  # s times the derivative by s
        else:
            u = w * d
        if soft:
            back = torch.zeros_like(s).scatter_add(1, ids, u)
            if not case["renorm"]:
                back = back - torch.where(fit, s, 0.0) * u.sum(-1, keepdim=True)
        else:
            back = torch.zeros_like(s).scatter_add(1, ids, u * (1.0 - torch.where(there, s.gather(1, ids), 0.0)))
        out["grad_logits"] = back.to(state["logits"].dtype)
    return out


def _plan(ids, experts):
    """Counts and offsets of the experts' chunks and each pair's row: pairs in
    expert order, token order within an expert; a dropped pair has -1 - row,
    its row after the last expert's."""
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    held, order = key.sort(stable=True)
    offsets = torch.searchsorted(held, torch.arange(experts + 1, device=ids.device, dtype=torch.int32))
    row = torch.empty_like(flat)
    row[order] = torch.arange(flat.numel(), device=ids.device, dtype=torch.int32)
    slots = torch.where(key < experts, row, -1 - row).view(ids.shape)
    return (offsets[1:] - offsets[:-1]).to(torch.int32), offsets.to(torch.int32), slots


def _rows_of(x, slots):
    """Every pair's copy of its token's row, at the pair's place; zeros for a dropped pair."""
    T, K = slots.shape
    rows = torch.empty(T * K, x.shape[1], dtype=x.dtype, device=x.device)
    flat = slots.view(-1).long()
    rows[torch.where(flat < 0, -1 - flat, flat)] = torch.where((slots < 0)[:, :, None], 0.0, x[:, None, :]).view(T * K, -1)
    return rows


def _gathered(rows, slots):
    """[tokens, k, hidden]: the rows of each token's pairs; zeros for a dropped pair."""
    flat = slots.view(-1).long()
    got = rows[flat.clamp(min=0)].view(*slots.shape, -1)
    return torch.where((slots < 0)[:, :, None], 0.0, got)


def _adamw(case, state):
    f, a = state["flat"], ADAMW
    c1, c2 = 1.0 - a["beta1"] ** a["step"], 1.0 - a["beta2"] ** a["step"]
    g = f["grad"].float()
    if state["clip"] is not None:
        g = g * state["clip"]
    if case["bits"] == 8:
        m = (f["avg"].float().view(-1, BLOCK) * f["avg_scale"][:, None]).view(-1)
        r = (f["rms"].float().view(-1, BLOCK) * f["rms_scale"][:, None]).view(-1)
        v = r * r
    else:
        m, v = f["avg"], f["sq"]
    m = m * a["beta1"] + g * (1.0 - a["beta1"])
    v = v * a["beta2"] + (g * g) * (1.0 - a["beta2"])
    r = v.sqrt()
    step = m / (r * (1.0 / math.sqrt(c2)) + a["eps"]) * (a["lr"] / c1)
    p = f["param"].float() * (1.0 - a["lr"] * a["weight_decay"]) - step
    f["param"].copy_(p)
    if case["copy"]:
        f["copy"].copy_(p)
    if case["bits"] == 8:
        for name, x in (("avg", m), ("rms", r)):
            code, scale = _quantize(x, name == "rms")
            f[name].copy_(code)
            f[name + "_scale"].copy_(scale)
    else:
        f["avg"].copy_(m)
        f["sq"].copy_(v)
    return {k: v for k, v in f.items() if k != "grad"}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    return {"route": _route64, "plan": _plan64, "dispatch": _dispatch64, "combine": _combine64,
            "adamw": _adamw64}[case["op"]](case, state)


def _route64(case, state):
    l = state["logits"].double()
    T, E = l.shape
    K, G = case["top_k"], case["groups"]
    s = l.softmax(-1) if case["score"] == "softmax" else l.sigmoid()
    c = s if state["bias"] is None else s + state["bias"].double()
    allowed = torch.ones(T, E, dtype=torch.bool, device=l.device)
    if G > 1:
        parts = c.reshape(T, G, E // G)
        n = min(2 if case["group_score"] == "top2" else 1, E // G)
        rank = parts.sort(dim=-1, descending=True).values[..., :n].sum(-1).argsort(dim=-1, descending=True, stable=True)
        allowed = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, rank[:, :case["kept"]], True)
        allowed = allowed.repeat_interleave(E // G, 1)
    ids = torch.where(allowed, c, -torch.inf).argsort(dim=-1, descending=True, stable=True)[:, :K]
    live = torch.ones(T, 1, dtype=torch.float64, device=l.device) if state["mask"] is None else state["mask"].double()[:, None]
    chosen = torch.zeros(T, E, dtype=torch.float64, device=l.device).scatter_(1, ids, 1.0) * live
    raw = s * chosen
    total = raw.sum(-1, keepdim=True)
    full = raw / torch.where(total > 0, total, 1.0) if case["renorm"] else raw
    out = {"weights": full.gather(1, ids) * case["scale"], "ids": None}
    if case["train"]:
        # the whole Jacobian's product: weights by scores, then scores by logits
        gw = torch.zeros_like(full).scatter_(1, ids, state["grad"].double()) * chosen * case["scale"]
        if case["renorm"]:
            gs = chosen * (gw - (gw * full).sum(-1, keepdim=True)) / torch.where(total > 0, total, 1.0)
        else:
            gs = gw
        out["grad_logits"] = s * (gs - (gs * s).sum(-1, keepdim=True)) if case["score"] == "softmax" else gs * s * (1 - s)
    return out


def _plan64(case, state):
    return None  # whole numbers throughout


def _dispatch64(case, state):
    slots = state["slots"].long()
    T, K = slots.shape
    x = state["x"].double()
    rows = torch.zeros(T * K, x.shape[1], dtype=torch.float64, device="cuda")
    for k in range(K):
        live = slots[:, k] >= 0
        rows[slots[live, k]] = x[live]
    out = {"rows": rows}
    if case["train"]:
        gx = torch.zeros_like(x)
        for k in range(K):
            live = slots[:, k] >= 0
            gx[live] += state["grad"][slots[live, k]].double()
        out["grad_x"] = gx
    return out


def _combine64(case, state):
    slots, rows = state["slots"].long(), state["rows"]
    T, K = slots.shape
    y = torch.zeros(T, rows.shape[1], dtype=torch.float64, device="cuda")
    if state["residual"] is not None:
        y += state["residual"].double()
    grad = state["grad"].double() if case["train"] else None
    back = torch.zeros(rows.shape, dtype=torch.float64, device="cuda") if case["train"] else None
    gw = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    for k in range(K):
        live = slots[:, k] >= 0
        at, w = slots[live, k], state["weights"][live, k].double()[:, None]
        y[live] += w * rows[at].double()
        if case["train"]:
            back[at] = w * grad[live]
            gw[live, k] = (grad[live] * rows[at].double()).sum(-1)
    return {"y": y, "grad_rows": back, "grad_weights": gw} if case["train"] else {"y": y}


def _round8(x, up):
    """Blocks of 256 values in 64 bits: the nearest 8-bit value of each after
    scaling (3 bits after the point, exponents from -6), and the scales."""
    x = x.view(-1, BLOCK)
    scale = (x.abs().amax(-1) / F8_MAX).clamp(min=SCALE_MIN)
    y = x / scale[:, None]
    unit = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    y = torch.round(y / unit) * unit
    if up:
        y = torch.where((x > 0) & (y < F8_MIN), F8_MIN, y)
    return y.view(-1), scale


def _adamw64(case, state):
    f, a = state["flat"], ADAMW
    g = f["grad"].double()
    if state["clip"] is not None:
        g *= state["clip"].double()
    if case["bits"] == 8:
        m = (f["avg"].to(torch.float32).double().view(-1, BLOCK) * f["avg_scale"].double()[:, None]).view(-1)
        v = (f["rms"].to(torch.float32).double().view(-1, BLOCK) * f["rms_scale"].double()[:, None]).view(-1).square_()
    else:
        m, v = f["avg"].double(), f["sq"].double()
    m = m.mul_(a["beta1"]).add_(g, alpha=1.0 - a["beta1"])
    v = v.mul_(a["beta2"]).add_(g.square_(), alpha=1.0 - a["beta2"])
    mhat = m / (1.0 - a["beta1"] ** a["step"])
    rhat = (v / (1.0 - a["beta2"] ** a["step"])).sqrt_().add_(a["eps"])
    p = f["param"].double()
    p = p - a["lr"] * (mhat / rhat + a["weight_decay"] * p)
    out = {"param": p}
    if case["bits"] == 8:
        out["avg"], out["avg_scale"] = _round8(m, False)
        out["rms"], out["rms_scale"] = _round8(v.sqrt(), True)
    else:
        out["avg"], out["sq"] = m, v
    if case["copy"]:
        out["copy"] = p
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if op == "route":
        T, E, K = case["tokens"], case["experts"], case["top_k"]
        b = T * E * size[case["type"]] + T * K * 8 + (4 * E if case["bias"] else 0) + (T if case["masked"] else 0)
        f = 4 * T * E
        if case["train"]:
            b += T * E * size[case["type"]] + 4 * T * K
            f += 4 * T * E
        return {"bytes": b, "flops": f}
    if op == "plan":
        n = case["tokens"] * case["top_k"]
        return {"bytes": 8 * n + 8 * case["experts"] + 4, "flops": n}
    if op in ("dispatch", "combine"):
        T, H, K, z = case["tokens"], case["hidden"], case["top_k"], size[case["type"]]
        live = 1.0 - case["dropped"]
        if op == "dispatch":
            b = T * H * z * live + T * K * H * z + 4 * T * K
            f = 0
            if case["train"]:
                b += T * K * H * z * live + T * H * z
                f = T * K * H
            return {"bytes": b, "flops": f}
        b = T * K * H * z * live + T * H * z * (2 if case["residual"] else 1) + 8 * T * K
        f = 2 * T * K * H
        if case["train"]:  # the rows are read once for both directions
            b += T * H * z + T * K * H * z + 4 * T * K
            f += 3 * T * K * H
        return {"bytes": b, "flops": f}
    n = sum(_sizes(case))
    p, g = size[case["param"]], size[case["grad"]]
    states = 2 * (4 if case["bits"] == 32 else 1 + 4 / BLOCK)
    return {"bytes": n * (2 * p + g + 2 * states + (2 if case["copy"] else 0)), "flops": 14 * n}
