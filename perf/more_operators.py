"""Timed cases of what the experts compute between dispatch and combine.

``moe_quantize`` and its kin turn rows and weights into 8-bit floating point
with a power-of-two scale for each block of 128 values, ``moe_matmul`` and its
gradients multiply them chunk by chunk, and ``moe_layer`` is the whole layer
for a few tokens: router, choice of experts, their products and the weighted
sum.

Each case runs either way: ``own`` false, the operator in its plain form
(elementary torch operations in 32 bits, rounded once at the end); ``own``
true, the package's own calls.  ``exact`` gives the same answers from the
definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 128                    # values, rows or both that share a scale
F8_MAX = 448.0                 # largest value of torch.float8_e4m3fn
LOWEST = -127                  # smallest exponent of a scale: that of an all-zero block
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "f8": 1}


def listed():
    return [
        # both operands of the training step's products from the rows that dispatch fills: 16,384 tokens
        # of 4,096, two of 64 experts each (the package's all-to-all workload)
        {"name": "quantize, training batch", "op": "quantize", "form": "both", "rows": 32768, "cols": 4096,
         "experts": 64, "type": "bf16", "dropped": 0.02},
        # an odd width in full precision, rows alone: inference
        {"name": "quantize, odd rows", "op": "quantize", "form": "rows", "rows": 6126, "cols": 2055, "experts": 48,
         "type": "f32", "dropped": 0.0},
        # the experts' weights, every step of training
        {"name": "quantize, weights", "op": "quantize", "form": "weights", "rows": 2048, "cols": 4096, "experts": 32,
         "type": "bf16", "dropped": 0.0},
        # 61 tokens of several generating requests, two experts each: every expert's weights for a row or two
        {"name": "product, few tokens", "op": "product", "rows": 122, "inner": 4096, "outer": 2048, "experts": 64,
         "type": "bf16", "dropped": 0.0, "train": False},
        # odd widths, uneven chunks, padding tokens among the rows
        {"name": "product, odd widths", "op": "product", "rows": 6126, "inner": 2055, "outer": 1021, "experts": 48,
         "type": "f16", "dropped": 0.05, "train": False},
        # prompts: 8,192 tokens, six of 128 small experts each
        {"name": "product, prompts", "op": "product", "rows": 49152, "inner": 2048, "outer": 1536, "experts": 128,
         "type": "bf16", "dropped": 0.0, "train": False},
        # the training batch: forward, gradient by the rows, gradient by the weights
        {"name": "product, training batch", "op": "product", "rows": 32768, "inner": 4096, "outer": 2048,
         "experts": 64, "type": "bf16", "dropped": 0.02, "train": True},
        # one dense matrix of the weight stack that the package's parameter workload has, forward and backward
        {"name": "product, one matrix", "op": "product", "rows": 8192, "inner": 4096, "outer": 14336, "experts": 1,
         "type": "bf16", "dropped": 0.0, "train": True},
        # one new token through a layer of large experts
        {"name": "layer, one token", "op": "layer", "tokens": 1, "hidden": 4096, "inner": 14336, "experts": 8,
         "top_k": 2, "type": "bf16", "weights": "same", "gated": True, "activation": "silu", "score": "softmax",
         "bias": False, "renorm": True, "scale": 1.0, "residual": True},
        # a handful of generating requests, weights in 8 bits
        {"name": "layer, few tokens, 8 bits", "op": "layer", "tokens": 7, "hidden": 4096, "inner": 2048,
         "experts": 64, "top_k": 2, "type": "bf16", "weights": "f8", "gated": True, "activation": "silu",
         "score": "softmax", "bias": False, "renorm": True, "scale": 1.0, "residual": True},
        # many requests over many small experts, sigmoid scores with balance bias
        {"name": "layer, many requests", "op": "layer", "tokens": 32, "hidden": 2048, "inner": 768, "experts": 128,
         "top_k": 8, "type": "bf16", "weights": "same", "gated": True, "activation": "silu", "score": "sigmoid",
         "bias": True, "renorm": True, "scale": 2.5, "residual": False},
        # a small model of odd sizes, without a gate: latency
        {"name": "layer, small and odd", "op": "layer", "tokens": 3, "hidden": 520, "inner": 201, "experts": 6,
         "top_k": 2, "type": "f16", "weights": "same", "gated": False, "activation": "gelu", "score": "softmax",
         "bias": False, "renorm": False, "scale": 1.0, "residual": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: two thirds of them multiples of 64, as models have them."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.33 else max(64, n // 64 * 64)


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "layer", "layer"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "quantize":
        form = rng.choice(["rows", "both", "columns", "weights"])
        cols = _width(rng, 16, 8192)
        if form == "weights":
            experts = _log(rng, 1, 64)
            rows = _width(rng, 16, min(8192, max(64, 250_000_000 // (cols * experts))))
        else:
            experts = rng.randint(1, 128)
            rows = _log(rng, 1, min(65536, 130_000_000 // cols))
        return {"op": op, "form": form, "rows": rows, "cols": cols, "experts": experts, "type": kind,
                "dropped": 0.0 if form == "weights" else rng.choice([0.0, 0.05])}
    if op == "product":
        inner, outer = _width(rng, 24, 8192), _width(rng, 24, 8192)
        train = rng.random() < 0.5
        experts = _log(rng, 1, max(1, min(128, 500_000_000 // (inner * outer))))
        most = int(1.2e12 / (2.0 * inner * outer * (3 if train else 1)))
        rows = _log(rng, 1, max(2, min(65536, most, 250_000_000 // max(inner, outer))))
        return {"op": op, "rows": rows, "inner": inner, "outer": outer, "experts": experts, "type": kind,
                "dropped": rng.choice([0.0, 0.05]), "train": train}
    top_k = rng.randint(1, 8)
    tokens, hidden = _log(rng, 1, 32), _width(rng, 64, 8192)
    inner = _width(rng, 16, max(64, min(8192, 500_000_000 // (2 * hidden * tokens * top_k))))
    experts = rng.randint(max(2, top_k), max(top_k, 2, min(256, 800_000_000 // (3 * hidden * inner))))
    return {"op": op, "tokens": tokens, "hidden": hidden, "inner": inner, "experts": experts, "top_k": top_k,
            "type": kind, "weights": rng.choice(["same", "f8"]), "gated": rng.random() < 0.7,
            "activation": rng.choice(["silu", "gelu", "relu"]), "score": rng.choice(["softmax", "sigmoid"]),
            "bias": rng.random() < 0.4, "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5]),
            "residual": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _offsets(case, gen):
    """First row of each expert's chunk and the rows in all: uneven chunks, some
    empty where there are few rows, as a router leaves them."""
    pull = 0.5 * torch.randn(case["experts"], generator=gen, device="cuda")
    live = case["rows"] - int(case["rows"] * case["dropped"])
    share = torch.softmax(pull, 0)
    who = torch.multinomial(share, live, replacement=True, generator=gen)
    counts = torch.bincount(who, minlength=case["experts"])
    offsets = torch.zeros(case["experts"] + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return offsets, int(counts.max()), live


def _activations(rows, cols, live, kind, gen, sigma=1.0):
    """Rows of normal values, columns of uneven size among them; behind the last chunk zeros."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x *= sigma * torch.exp(0.7 * torch.randn(cols, generator=gen, device="cuda"))
    x[live:] = 0
    return x.to(TYPES[kind])


def _stored(codes):
    """Codes as the package keeps them: rows from multiples of 16 bytes on."""
    cols = codes.shape[-1]
    held = torch.zeros(*codes.shape[:-1], -(-cols // 16) * 16, dtype=torch.uint8, device=codes.device)
    held[..., :cols] = codes.view(torch.uint8)
    return held.view(torch.float8_e4m3fn)[..., :cols]


def _weights8(experts, rows, cols, gen):
    """Experts' matrices [experts, rows, cols] in 8 bits, made one by one."""
    codes = torch.empty(experts, rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(experts, -(-rows // BLOCK), -(-cols // BLOCK), dtype=torch.uint8, device="cuda")
    for e in range(experts):
        w = torch.randn(1, rows, cols, generator=gen, device="cuda") * cols ** -0.5
        c, s = _quantize_weights(w)
        codes[e], scales[e] = c[0], s[0].view(torch.uint8)
    return _stored(codes), scales.view(torch.float8_e8m0fnu)


def _undecided(case, x, router, bias):
    """Tokens whose choice hangs on the last bits of a logit."""
    l = x.double() @ router.double().T
    c = l
    if bias is not None:
        s = l.softmax(-1) if case["score"] == "softmax" else l.sigmoid()
        c = s + bias.double()
    top = c.topk(min(case["experts"], case["top_k"] + 1), -1).values
    return ((top[:, :-1] - top[:, 1:]) < 2e-5).any(-1)


def prepare(case, seed):
    gen = _generator(seed)
    op = case["op"]
    if op == "quantize":
        if case["form"] == "weights":
            w = torch.randn(case["experts"], case["rows"], case["cols"], generator=gen, device="cuda")
            return {"case": case, "x": w.mul_(case["cols"] ** -0.5).to(TYPES[case["type"]])}
        offsets, _, live = _offsets(case, gen)
        return {"case": case, "offsets": offsets,
                "x": _activations(case["rows"], case["cols"], live, case["type"], gen)}
    if op == "product":
        M, K, N, E = case["rows"], case["inner"], case["outer"], case["experts"]
        offsets, most, live = _offsets(case, gen)
        state = {"case": case, "offsets": offsets, "most": most, "x": _activations(M, K, live, case["type"], gen),
                 "w": _weights8(E, N, K, gen)}
        if case["train"]:
            state["g"] = _activations(M, N, live, case["type"], gen, 1e-3)
        return state
    T, H, I, E = case["tokens"], case["hidden"], case["inner"], case["experts"]
    dt = TYPES[case["type"]]
    bias = None
    if case["bias"]:  # as balance rules leave it: a whole number of steps of 0.001
        bias = torch.randint(-20, 21, (E,), generator=gen, device="cuda").float() * 1e-3
    router = (1.5 * H ** -0.5 * torch.randn(E, H, generator=gen, device="cuda")).to(dt)
    x = torch.randn(T, H, generator=gen, device="cuda").to(dt)
    for _ in range(8):
        bad = _undecided(case, x, router, bias)
        x = torch.where(bad[:, None], torch.randn(T, H, generator=gen, device="cuda").to(dt), x)
    shape = (E, I * (2 if case["gated"] else 1), H), (E, H, I)
    if case["weights"] == "f8":
        up, down = (_weights8(*s, gen) for s in shape)
    else:
        up, down = (torch.empty(s, dtype=dt, device="cuda") for s in shape)
        for w in (up, down):
            for e in range(E):
                w[e] = torch.randn(w.shape[1:], generator=gen, device="cuda") * w.shape[2] ** -0.5
    residual = torch.randn(T, H, generator=gen, device="cuda").to(dt) if case["residual"] else None
    return {"case": case, "x": x, "router": router, "bias": bias, "up": up, "down": down, "residual": residual}


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    return (_run_own if own else _run_plain)(case, state)


def _run_own(case, state):
    import lossless_bf16_tensor_zipccl_gb300 as zc
    op = case["op"]
    if op == "quantize":
        x, form = state["x"], case["form"]
        if form == "weights":
            return zc.moe_quantize_weights(x)
        if form == "rows":
            return zc.moe_quantize(x)
        return zc.moe_quantize_columns(x, state["offsets"], by_rows=form == "both")
    if op == "product":
        at, w = state["offsets"], state["w"]
        if not case["train"]:
            return {"y": zc.moe_matmul(zc.moe_quantize(state["x"]), w, at)}
        x, x_columns = zc.moe_quantize_columns(state["x"], at, by_rows=True)
        out = {"y": zc.moe_matmul(x, w, at)}
        g, g_columns = zc.moe_quantize_columns(state["g"], at, by_rows=True)
        out["grad_x"] = zc.moe_matmul_backward(g, w, at)
        out["grad_w"] = zc.moe_matmul_backward_weights(g_columns, x_columns, at)
        return out
    y, weights, ids = zc.moe_layer(state["x"], state["router"], state["up"], state["down"], case["top_k"],
                                   score=case["score"], bias=state["bias"], renormalize=case["renorm"],
                                   scale=case["scale"], activation=case["activation"], residual=state["residual"])
    return {"y": y, "weights": weights, "ids": ids}


def _run_plain(case, state):
    op = case["op"]
    if op == "quantize":
        x, form = state["x"].float(), case["form"]
        if form == "weights":
            return _quantize_weights(x)
        if form == "rows":
            return _quantize_rows(x)
        columns = _quantize_columns(x, state["offsets"])
        return (_quantize_rows(x), columns) if form == "both" else columns
    if op == "product":
        return _product(case, state)
    return _layer(case, state)


def _exponents(top):
    """Of the smallest power of two that brings `top` to 448 at most."""
    m, e = torch.frexp(top)
    return torch.where(top > 0, e - 9 + (m > 0.875), LOWEST).clamp(min=LOWEST)


def _scaled(x, e):
    """x * 2^-e as 8-bit codes."""
    return (x * ((127 - e) << 23).to(torch.int32).view(torch.float32)).to(torch.float8_e4m3fn)


def _bytes(e):
    return (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _factors(scales):
    b = scales.view(torch.uint8).to(torch.int32)
    return torch.where(b > 0, (b << 23).view(torch.float32), 2.0 ** LOWEST)


def _spread(t, dim, size):
    """One value of a block for each of its places."""
    return t.repeat_interleave(BLOCK, dim).narrow(dim, 0, size)


def _quantize_rows(x):
    M, K = x.shape
    whole = torch.nn.functional.pad(x, (0, -K % BLOCK)).view(M, -1, BLOCK)
    e = _exponents(whole.abs().amax(-1))
    return _scaled(x, _spread(e, 1, K)), _bytes(e)


def _places(offsets, M):
    """Of each row: its expert (the number of experts where it is in no chunk),
    its place in the chunk and its block of 128 rows."""
    E = offsets.numel() - 1
    m = torch.arange(M, dtype=torch.int32, device=offsets.device)
    expert = torch.searchsorted(offsets[1:].contiguous(), m, right=True)
    blocks = (offsets[1:] - offsets[:-1] + BLOCK - 1) // BLOCK
    first = torch.cat([torch.zeros_like(blocks[:1]), blocks.cumsum(0).to(torch.int32)])
    place = m - offsets[expert]
    return expert, place, first[expert] + place // BLOCK


def _quantize_columns(x, offsets):
    M, K = x.shape
    E = offsets.numel() - 1
    expert, place, block = _places(offsets, M)
    inside = expert < E
    count = M // BLOCK + E
    held = torch.full(((count + 1) * BLOCK,), M, device=x.device)
    held[torch.where(inside, block * BLOCK + place % BLOCK, count * BLOCK)] = torch.arange(M, device=x.device)
    rows = torch.cat([x, torch.zeros_like(x[:1])])[held[:count * BLOCK]]
    e = _exponents(rows.view(count, BLOCK, K).abs().amax(1))
    codes = _scaled(x, e[block.clamp(max=count - 1)])
    return torch.where(inside[:, None], codes.view(torch.uint8), 0).view(torch.float8_e4m3fn), _bytes(e)


def _quantize_weights(w):
    E, N, K = w.shape
    whole = torch.nn.functional.pad(w, (0, -K % BLOCK, 0, -N % BLOCK))
    e = _exponents(whole.view(E, whole.shape[1] // BLOCK, BLOCK, -1, BLOCK).abs().amax((2, 4)))
    return _scaled(w, _spread(_spread(e, 1, N), 2, K)), _bytes(e)


def _values_of_weights(w):
    codes, scales = w
    return codes.float() * _spread(_spread(_factors(scales), 1, codes.shape[1]), 2, codes.shape[2])


def _product(case, state):
    x, at, M, E = state["x"].float(), state["offsets"], case["rows"], case["experts"]
    w = _values_of_weights(state["w"])
    expert, place, block = _places(at, M)
    inside = expert < E
    # the chunks side by side, each as long as the longest
    held = at[:-1, None] + torch.arange(state["most"], dtype=torch.int32, device="cuda")
    held = torch.where(held < at[1:, None], held, M)

    def chunks(rows):
        return torch.cat([rows, torch.zeros_like(rows[:1])])[held]

    def back(parts):
        got = parts[expert.clamp(max=E - 1), place.clamp(max=state["most"] - 1)]
        return torch.where(inside[:, None], got, 0.0).to(torch.bfloat16)

    def by_rows(t):
        codes, scales = _quantize_rows(t)
        return codes.float() * _spread(_factors(scales), 1, t.shape[1])

    def by_columns(t):
        codes, scales = _quantize_columns(t, at)
        return codes.float() * _factors(scales)[block.clamp(max=scales.shape[0] - 1)]

    out = {"y": back(torch.bmm(chunks(by_rows(x)), w.mT))}
    if case["train"]:
        g = state["g"].float()
        out["grad_x"] = back(torch.bmm(chunks(by_rows(g)), w))
        out["grad_w"] = torch.bmm(chunks(by_columns(g)).mT, chunks(by_columns(x))).to(torch.bfloat16)
    return out


def _layer(case, state):
    x, T, k = state["x"].float(), case["tokens"], case["top_k"]
    logits = x @ state["router"].float().T
    soft = case["score"] == "softmax"
    s = torch.exp(logits - logits.amax(-1, keepdim=True))
    s = s / s.sum(-1, keepdim=True) if soft else 1.0 / (1.0 + torch.exp(-logits))
    c = logits if state["bias"] is None else s + state["bias"]
    ids = c.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    weights = s.gather(1, ids)
    if case["renorm"]:
        weights = weights / weights.sum(-1, keepdim=True)
    weights = weights * case["scale"]

    def chosen(w):  # the chosen experts' matrices, [pairs, rows, cols]
        flat = ids.reshape(-1)
        if case["weights"] != "f8":
            return w[flat].float()
        return _values_of_weights((w[0].view(torch.uint8)[flat].view(torch.float8_e4m3fn),
                                   w[1].view(torch.uint8)[flat].view(torch.float8_e8m0fnu)))

    pairs = x.repeat_interleave(k, 0)
    h = torch.bmm(chosen(state["up"]), pairs[:, :, None])[:, :, 0]
    gate = h[:, :case["inner"]]
    if case["activation"] == "silu":
        a = gate / (1.0 + torch.exp(-gate))
    elif case["activation"] == "gelu":
        a = 0.5 * gate * (1.0 + torch.erf(gate * math.sqrt(0.5)))
    else:
        a = gate.clamp(min=0.0)
    if case["gated"]:
        a = a * h[:, case["inner"]:]
    y = torch.bmm(chosen(state["down"]), a[:, :, None])[:, :, 0]
    y = (y * weights.reshape(-1, 1)).view(T, k, -1).sum(1)
    if state["residual"] is not None:
        y = y + state["residual"].float()
    return {"y": y.to(state["x"].dtype), "weights": weights, "ids": ids.to(torch.int32)}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    return {"quantize": _quantize64, "product": _product64, "layer": _layer64}[case["op"]](case, state)


def _scale64(top):
    """2^e, e the smallest whole number from -127 on with top <= 448 * 2^e."""
    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / F8_MAX))
    e = torch.where(top > F8_MAX * torch.exp2(e), e + 1, torch.where(top <= F8_MAX * torch.exp2(e - 1), e - 1, e))
    return torch.exp2(torch.where(top > 0, e.clamp(min=-127.0), -127.0))


def _round64(y):
    """The nearest value with 3 bits after the point, exponents from -6 on; ties to even."""
    unit = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / unit) * unit


def _rows64(x):
    codes, scales = torch.empty_like(x), []
    for k in range(0, x.shape[1], BLOCK):
        part = x[:, k:k + BLOCK]
        s = _scale64(part.abs().amax(1))
        codes[:, k:k + BLOCK] = _round64(part / s[:, None])
        scales.append(s)
    return codes, torch.stack(scales, 1)


def _columns64(x, offsets):
    at = offsets.tolist()
    codes = torch.zeros_like(x)
    scales = torch.full((x.shape[0] // BLOCK + len(at) - 1, x.shape[1]), 2.0 ** -127, dtype=torch.float64, device="cuda")
    values, n = torch.zeros_like(x), 0
    for a, b in zip(at, at[1:]):
        for m in range(a, b, BLOCK):
            part = x[m:min(b, m + BLOCK)]
            scales[n] = _scale64(part.abs().amax(0))
            codes[m:min(b, m + BLOCK)] = _round64(part / scales[n])
            values[m:min(b, m + BLOCK)] = codes[m:min(b, m + BLOCK)] * scales[n]
            n += 1
    return codes, scales, values


def _quantize64(case, state):
    x, form = state["x"].double(), case["form"]
    if form == "weights":
        E, N, K = x.shape
        codes = torch.empty_like(x)
        scales = torch.empty(E, -(-N // BLOCK), -(-K // BLOCK), dtype=torch.float64, device="cuda")
        for i in range(scales.shape[1]):
            for j in range(scales.shape[2]):
                part = x[:, i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
                scales[:, i, j] = _scale64(part.abs().amax((1, 2)))
                codes[:, i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] = _round64(part / scales[:, i, j, None, None])
        return codes, scales
    if form == "rows":
        return _rows64(x)
    columns = _columns64(x, state["offsets"])[:2]
    return (_rows64(x), columns) if form == "both" else columns


def _weight64(w, e):
    codes, scales = w[0][e].double(), torch.exp2(w[1][e].view(torch.uint8).double() - 127)
    N, K = codes.shape
    return codes * scales.repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]


def _product64(case, state):
    def values(x):
        codes, scales = _rows64(x.double())
        return codes * scales.repeat_interleave(BLOCK, 1)[:, :x.shape[1]]

    at, E = state["offsets"].tolist(), case["experts"]
    x = values(state["x"])
    out = {"y": torch.zeros(case["rows"], case["outer"], dtype=torch.float64, device="cuda")}
    if case["train"]:
        g, gc, xc = values(state["g"]), _columns64(state["g"].double(), state["offsets"])[2], _columns64(state["x"].double(), state["offsets"])[2]
        out["grad_x"] = torch.zeros_like(x)
        out["grad_w"] = torch.zeros(E, case["outer"], case["inner"], dtype=torch.float64, device="cuda")
    for e, (a, b) in enumerate(zip(at, at[1:])):
        if a == b:
            continue
        w = _weight64(state["w"], e)
        out["y"][a:b] = x[a:b] @ w.T
        if case["train"]:
            out["grad_x"][a:b] = g[a:b] @ w
            out["grad_w"][e] = gc[a:b].T @ xc[a:b]
    return out


def _layer64(case, state):
    x, k, I = state["x"].double(), case["top_k"], case["inner"]
    logits = x @ state["router"].double().T
    s = logits.softmax(-1) if case["score"] == "softmax" else logits.sigmoid()
    c = s if state["bias"] is None else s + state["bias"].double()
    if state["bias"] is None:
        c = logits
    ids = c.argsort(dim=-1, descending=True, stable=True)[:, :k]
    w = s.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    w = w * case["scale"]
    y = torch.zeros_like(x) if state["residual"] is None else state["residual"].double()
    act = {"silu": lambda v: v * v.sigmoid(), "gelu": lambda v: v * 0.5 * torch.erfc(-v * math.sqrt(0.5)),
           "relu": lambda v: v.clamp(min=0.0)}[case["activation"]]
    f8 = case["weights"] == "f8"
    for e in ids.unique().tolist():
        up, down = ((_weight64(state[n], e) if f8 else state[n][e].double()) for n in ("up", "down"))
        t, j = (ids == e).nonzero(as_tuple=True)
        h = x[t] @ up.T
        h = act(h[:, :I]) * (h[:, I:] if case["gated"] else 1.0)
        y[t] += w[t, j, None] * (h @ down.T)
    return {"y": y, "weights": w, "ids": None}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "quantize":
        n, z = case["rows"] * case["cols"], SIZE[case["type"]]
        if case["form"] == "weights":
            n *= case["experts"]
            return {"bytes": n * (z + 1 + 1 / BLOCK ** 2), "flops": 2 * n}
        forms = 2 if case["form"] == "both" else 1
        return {"bytes": n * (z + forms * (1 + 1 / BLOCK)), "flops": 2 * n * forms}
    if op == "product":
        M, K, N, E, z = case["rows"], case["inner"], case["outer"], case["experts"], SIZE[case["type"]]
        live = M * (1 - case["dropped"])
        used = E * (1 - (1 - 1 / E) ** live)  # experts with rows
        b, f = M * K * z + used * N * K + 2 * M * N, 2 * live * N * K
        if case["train"]:  # the weights are read once for both directions
            b += M * N * z + 2 * M * K + 2 * E * N * K
            f *= 3
        return {"bytes": b, "flops": f}
    T, H, I, E, k = case["tokens"], case["hidden"], case["inner"], case["experts"], case["top_k"]
    z = SIZE[case["type"]]
    used = E * (1 - (1 - k / E) ** T)
    matrices = (3 if case["gated"] else 2) * I * H
    b = used * matrices * (1 if case["weights"] == "f8" else z) + E * H * z + T * H * z * (3 if case["residual"] else 2) + 8 * T * k
    return {"bytes": b, "flops": 2 * T * (k * matrices + E * H)}
