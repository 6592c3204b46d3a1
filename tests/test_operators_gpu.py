"""The operators around the exchange on the GPU against their definitions in
64 bits (operator_reference).

Tolerances.  u = 2^-24 is half a unit in the last place of a float.
 - Route: a weight is a quotient of an exponential (2 units at most, its
   argument off by u times the logits' spread, below 40 here: 40 u) and a sum
   of at most 1,024 such terms added in runs of at most 32 and a tree of 5
   (37 u): about 120 u = 7e-6 of the weight; 1e-5 is asked.  The gradient adds
   a difference of products of that accuracy: 2e-5 of the largest |grad| the
   token gets (times the scale).  A 16-bit result is rounded once more.
 - Combine: up to 33 terms, each product and sum rounded: 40 u of the sum of
   magnitudes, and one rounding to the type.  Its weight gradient: runs of
   hidden / 256 products and a tree: (hidden / 256 + 20) u of the magnitudes.
 - AdamW: m, v: 4 roundings of terms no larger than what they add up to in
   magnitude; the update: 10 roundings relative; p: 2 more of itself.
"""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import lossless_bf16_tensor_zipccl_gb300 as zc  # noqa: E402
import operator_reference as ref  # noqa: E402

U = 2.0 ** -24
TYPES = [torch.float32, torch.bfloat16, torch.float16]
ROUND = {torch.float32: U, torch.bfloat16: 2.0 ** -9, torch.float16: 2.0 ** -12}  # half a unit, relative (doubled below)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    zc.load()
    yield


def host(t):
    return t.double().cpu().numpy()


def near(got, want, tol):
    """|got - want| <= tol everywhere; equal where the wanted value is not finite."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape
    odd = ~np.isfinite(want)
    assert np.array_equal(got[odd], want[odd], equal_nan=True)
    off = np.abs(got - want)[~odd] - np.broadcast_to(tol, want.shape)[~odd]
    assert off.size == 0 or off.max() <= 0, f"{off.max():.3g} over the tolerance"


def near_rounded(got, want, tol, dtype):
    """near() for a result that is rounded to `dtype` at the end: in its normal
    range by one part in its precision, below that (float16) by half of the
    smallest step, 2^-24."""
    want = np.asarray(want, np.float64)
    small = np.abs(want) < float(torch.finfo(dtype).tiny)
    once = np.where(small, 2.0 ** -25 if dtype == torch.float16 else 0.0, 2 * ROUND[dtype] * np.abs(want))
    near(got, want, tol + once * (dtype != torch.float32))


# ------------------------------------------------------------------ route
def draw_logits(rng, T, E, dtype, **how):
    """Logits whose choice does not hang on the last bits: tokens where two
    different scores come nearer than 1e-6 are drawn again."""
    l = torch.from_numpy(rng.normal(0, 1.5, (T, E))).to(dtype)
    for _ in range(60):
        bad = []
        for t in range(T):
            _, gap = ref.choose(host(l[t]), how["k"], how["score"], how["bias"], how["groups"], how["kept"], how["group_score"])
            if gap < 1e-6:
                bad.append(t)
        if not bad:
            return l.cuda()
        l[bad] = torch.from_numpy(rng.normal(0, 1.5, (len(bad), E))).to(dtype)
    raise AssertionError("no settled draw")


ROUTES = [
    # T, E, k, score, bias, groups, kept, group score, renormalize, scale
    (1, 64, 2, "softmax", False, 1, 1, "max", True, 1.0),
    (37, 64, 2, "softmax", False, 1, 1, "max", False, 1.0),
    (33, 8, 8, "softmax", True, 1, 1, "max", True, 1.0),
    (5, 1, 1, "sigmoid", False, 1, 1, "max", True, 2.5),
    (19, 65, 7, "sigmoid", True, 5, 2, "top2", True, 2.5),
    (50, 256, 8, "sigmoid", True, 8, 4, "top2", True, 2.5),
    (21, 256, 8, "softmax", False, 8, 3, "max", False, 16.0),
    (18, 160, 6, "softmax", True, 8, 3, "max", True, 1.0),
    (9, 128, 32, "sigmoid", False, 32, 32, "top2", False, 1.0),
    (10, 300, 10, "softmax", False, 3, 1, "top2", True, 1.0),
    (7, 513, 5, "sigmoid", True, 27, 3, "max", True, 1.0),
    (6, 1024, 32, "softmax", False, 1, 1, "max", False, 1.0),
    (4, 1000, 9, "softmax", True, 10, 4, "top2", True, 1.0),
    (300, 30, 4, "softmax", False, 15, 5, "top2", True, 1.0),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", ROUTES, ids=lambda c: f"T{c[0]}-E{c[1]}-k{c[2]}-{c[3]}-g{c[5]}")
def test_route_and_gradient(case, dtype):
    T, E, k, score, with_bias, groups, kept, gs, renorm, scale = case
    rng = np.random.default_rng(T * 1000 + E)
    bias = rng.integers(-20, 21, E) * 1e-3 if with_bias else None
    b = torch.from_numpy(bias).float().cuda() if with_bias else None
    bias = host(b) if with_bias else None
    logits = draw_logits(rng, T, E, dtype, k=k, score=score, bias=bias, groups=groups, kept=kept, group_score=gs)
    mask = rng.random(T) > 0.2
    w, ids = zc.moe_route(logits, k, score=score, bias=b, groups=groups, groups_kept=kept, group_score=gs,
                          renormalize=renorm, scale=scale, mask=torch.from_numpy(mask).cuda())
    rw, rids, _ = ref.route(host(logits), k, score, bias, groups, kept, gs, renorm, scale, mask)
    assert np.array_equal(ids.cpu().numpy(), rids)
    near(host(w), rw, 1e-5 * np.abs(rw))
    g = torch.from_numpy(rng.standard_normal((T, k))).float().cuda()
    dl = zc.moe_route_backward(g, logits, ids, score=score, renormalize=renorm, scale=scale)
    assert dl.dtype == dtype
    want = ref.route_grad(host(g), host(logits), rids, score, renorm, scale)
    top = np.abs(host(g)).max(1, keepdims=True) * scale
    near(host(dl), want, 2e-5 * top + (0 if dtype == torch.float32 else 2 * ROUND[dtype] * np.abs(want) + 2.0 ** -24))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_gradient_agrees_with_differences(score):
    # differences of the 64-bit weights at the float logits: 2e-9 from the
    # differences (h = 1e-4), 2e-5 from the kernel
    rng = np.random.default_rng(3)
    logits = torch.from_numpy(rng.standard_normal((4, 20))).float().cuda()
    for renorm in (True, False):
        _, ids = zc.moe_route(logits, 5, score=score, renormalize=renorm)
        g = torch.from_numpy(rng.standard_normal((4, 5))).float().cuda()
        dl = host(zc.moe_route_backward(g, logits, ids, score=score, renormalize=renorm))
        for t in range(4):
            for e in range(20):
                row = host(logits[t])
                up, down = row.copy(), row.copy()
                up[e] += 1e-4
                down[e] -= 1e-4
                at = ids[t].tolist()
                d = (ref.weigh(up, at, score, renorm, 1.0) - ref.weigh(down, at, score, renorm, 1.0)) / 2e-4
                assert abs((d * host(g[t])).sum() - dl[t, e]) < 3e-5 * host(g[t]).__abs__().max()


@pytest.mark.parametrize("E", [64, 100, 256, 700])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties_go_to_the_lowest_expert(E, score):
    l = torch.zeros(3, E, device="cuda")
    l[1, E // 2:] = 1.0                      # a tied upper half
    l[2] = -0.0
    l[2, 5::7] = 0.0                         # both zeros are one value
    _, ids = zc.moe_route(l, 4, score=score)
    assert ids.tolist() == [[0, 1, 2, 3], [E // 2 + i for i in range(4)], [0, 1, 2, 3]]
    g = 4 if E % 4 == 0 else 1
    _, ids = zc.moe_route(l, 4, score=score, groups=g, groups_kept=1, group_score="top2")
    assert ids[0].tolist() == [0, 1, 2, 3]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_special_logits(dtype, score, renorm):
    """Rows with nothing left, the type's lowest value, infinities and NaN."""
    E, k = 16, 4
    low = torch.finfo(dtype).min
    inf, nan = float("inf"), float("nan")
    l = torch.full((8, E), -inf, dtype=dtype)
    l[1, 3] = 1.0                            # one eligible expert
    l[2] = low                               # a mask of the type's lowest value throughout
    l[3] = low
    l[3, [2, 9]] = torch.tensor([0.5, 1.5], dtype=dtype)
    l[4] = nan
    l[4, 7] = 0.25
    l[5] = 0.0
    l[5, [4, 11]] = inf                      # two infinities share the token
    l[6] = torch.linspace(-1, 1, E).to(dtype)
    l[6, 15] = -inf                          # a closed expert, NaN beside it
    l[6, 14] = nan
    d = l.cuda()
    w, ids = zc.moe_route(d, k, score=score, renormalize=renorm)
    rw, rids, _ = ref.route(host(l), k, score, renormalize=renorm)
    assert np.array_equal(ids.cpu().numpy(), rids)
    assert ids[0].tolist() == [-1] * 4 and ids[1].tolist() == [3, -1, -1, -1] and ids[7].tolist() == [-1] * 4
    # a softmax over logits of 3e38 has no spread to lose: the tolerance of the weights holds
    near(host(w), rw, 1e-5 * np.abs(rw) + 1e-37)
    g = torch.ones(8, k, device="cuda")
    g[:, 1] = -2.0
    dl = host(zc.moe_route_backward(g, d, ids, score=score, renormalize=renorm))
    assert np.isfinite(dl).all()
    want = ref.route_grad(host(g), host(l), rids, score, renorm, 1.0)
    near(dl, want, 4e-5 + 2 * ROUND[dtype] * np.abs(want))
    assert not dl[0].any() and not dl[7].any()


def test_route_strides_streams_and_given_outputs():
    rng = np.random.default_rng(11)
    wide = torch.from_numpy(rng.permutation(40 * 101).reshape(40, 101) * 1e-3).float().cuda()
    for first, E in ((0, 64), (1, 64), (3, 90), (37, 61)):
        part = wide[:, first:first + E]
        w0, i0 = zc.moe_route(part.contiguous(), 6)
        w = torch.full((40, 6), 7.0, device="cuda")
        ids = torch.full((40, 6), 7, dtype=torch.int32, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        w1, i1 = zc.moe_route(part, 6, weights=w, ids=ids, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert w1 is w and torch.equal(w0, w1) and torch.equal(i0, i1)
        g = torch.from_numpy(rng.standard_normal((40, 6))).float().cuda()
        assert torch.equal(zc.moe_route_backward(g, part, ids), zc.moe_route_backward(g, part.contiguous(), ids))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups", [(20011, 64, 2, 1), (9001, 64, 12, 4), (12345, 256, 8, 8), (3000, 384, 6, 6)])
def test_route_many_tokens(T, E, k, groups, score):
    """Every token's logits are the same well separated values in an order of
    its own (0.02 apart at least: scores 4e-6 of themselves or more), against 64 bits on the GPU."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    order = torch.rand(T, E, generator=gen, device="cuda").argsort(1)
    l = torch.linspace(-4, 4, E, device="cuda")[order]
    kept = max(1, groups // 2)
    w, ids = zc.moe_route(l, k, score=score, groups=groups, groups_kept=kept, scale=2.0)
    d = l.double()
    best = d.view(T, groups, -1).amax(-1).topk(kept, 1).indices
    open_ = torch.zeros(T, groups, dtype=torch.bool, device="cuda").scatter(1, best, True).repeat_interleave(E // groups, 1)
    want = torch.where(open_, d, -torch.inf).topk(k, 1).indices
    assert torch.equal(ids.long(), want)
    s = (d.softmax(1) if score == "softmax" else d.sigmoid()).gather(1, want)
    s = s / s.sum(1, keepdim=True)
    near(host(w), host(2 * s), 1e-5 * host(2 * s))
    g = torch.randn(T, k, generator=gen, device="cuda")
    u = s * (g.double() - (s * g.double()).sum(1, keepdim=True)) * 2
    if score == "sigmoid":
        u = u * (1 - d.gather(1, want).sigmoid())
    dl = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter(1, want, u)
    near(host(zc.moe_route_backward(g, l, ids, score=score, scale=2.0)), host(dl), 2e-5 * 2 * np.abs(host(g)).max(1, keepdims=True))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [5, 64, 128, 256])
def test_route_of_one_renormalised_pair_is_exact(score, E):
    torch.manual_seed(E)
    l = torch.randn(500, E, device="cuda")
    w, ids = zc.moe_route(l, 1, score=score, scale=2.5)
    assert (w == 2.5).all() and torch.equal(ids[:, 0].long(), l.argmax(1))
    assert not zc.moe_route_backward(torch.randn(500, 1, device="cuda"), l, ids, score=score, scale=2.5).any()


def test_route_no_tokens():
    w, ids = zc.moe_route(torch.zeros(0, 64, device="cuda"), 2)
    assert w.shape == ids.shape == (0, 2)
    assert zc.moe_route_backward(w, torch.zeros(0, 64, device="cuda"), ids).shape == (0, 64)


# ------------------------------------------------------------------ plan
@pytest.mark.parametrize("T,k,E", [(0, 2, 64), (1, 1, 1), (1, 8, 256), (61, 2, 64), (513, 8, 7), (512, 8, 1024),
                                   (1025, 4, 33), (4097, 1, 300), (9001, 6, 160), (70000, 2, 64), (40000, 8, 1000)])
def test_plan(T, k, E):
    rng = np.random.default_rng(T + k + E)
    ids = rng.integers(-1, E + 1, (T, k)).astype(np.int32)   # some outside on either side
    if T:
        ids[rng.integers(0, T, max(1, T // 10))] = rng.integers(0, E)   # and an expert with many
    ids[:1] = np.int32(-2 ** 31)
    counts, offsets, slots = zc.moe_plan(torch.from_numpy(ids).cuda(), E)
    rc, ro, rs = ref.plan(ids, E)
    assert np.array_equal(counts.cpu().numpy(), rc)
    assert np.array_equal(offsets.cpu().numpy(), ro)
    assert np.array_equal(slots.cpu().numpy(), rs)


def test_plan_all_dropped_and_all_on_one():
    for value, n in ((-1, 0), (5, 10000)):
        p = zc.moe_plan(torch.full((5000, 2), value, dtype=torch.int32, device="cuda"), 8)
        assert p.offsets[-1].item() == n and p.counts.sum().item() == n
        line = torch.arange(10000, dtype=torch.int32, device="cuda").view(5000, 2)
        assert torch.equal(p.slots, line if n else -1 - line)


# ------------------------------------------------------------------ dispatch and combine
def random_slots(rng, T, k, E, dropped=0.15):
    ids = np.stack([rng.permutation(max(E, k))[:k] for _ in range(T)]) if T else np.zeros((0, k), int)
    ids = np.where(rng.random((T, k)) < dropped, -1, ids)
    if T > 2:
        ids[1] = -1                           # a token without experts
    return ref.plan(ids, max(E, k))[2]


ROWS = [(1, 1, 1), (1, 2, 4096), (3, 2, 7), (17, 8, 64), (33, 3, 129), (9, 32, 40), (65, 4, 1000), (5, 2, 8192),
        (12, 6, 2055), (40, 5, 776), (2, 1, 20000)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,H", ROWS)
def test_dispatch_combine_and_gradients(T, k, H, dtype):
    rng = np.random.default_rng(T * 100 + k * 10 + H)
    slots = random_slots(rng, T, k, 2 * k)
    ds = torch.from_numpy(slots.astype(np.int32)).cuda()
    new = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(dtype).cuda()  # noqa: E731
    x = new(T, H)
    rows = zc.moe_dispatch(x, ds)
    assert np.array_equal(host(rows), ref.dispatch(host(x), slots))
    r, res, gy = new(T * k, H), new(T, H), new(T, H)
    w = torch.from_numpy(rng.random((T, k)) - 0.3).float().cuda()
    for weights, residual in ((w, None), (None, res), (w, res)):
        y = zc.moe_combine(r, ds, weights, residual=residual)
        want, size = ref.combine(host(r), slots, None if weights is None else host(w), None if residual is None else host(res))
        near_rounded(host(y), want, 40 * U * size, dtype)
    want, size = ref.combine(host(r), slots)
    near_rounded(host(zc.moe_dispatch_backward(r, ds)), want, 40 * U * size, dtype)
    for weights in (w, None):
        gr, gw = zc.moe_combine_backward(gy, r, ds, weights)
        wr, ww, size = ref.combine_grad(host(gy), host(r), slots, None if weights is None else host(w))
        near(host(gr), wr, 2 * ROUND[dtype] * np.abs(wr) + 2.0 ** -25 * (dtype == torch.float16))
        near(host(gw), ww, (H / 256 + 20) * U * size)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,first,gap", [(64, 0, 64), (64, 8, 24), (64, 1, 1), (63, 0, 1), (130, 2, 6), (4096, 16, 48)])
def test_dispatch_strided_and_unaligned_rows(H, first, gap, dtype):
    rng = np.random.default_rng(H + first)
    wide = torch.from_numpy(rng.standard_normal((21, first + H + gap))).to(dtype).cuda()
    x = wide[:, first:first + H]
    ds = torch.from_numpy(random_slots(rng, 21, 3, 9).astype(np.int32)).cuda()
    assert torch.equal(zc.moe_dispatch(x, ds), zc.moe_dispatch(x.contiguous(), ds))
    same = wide[:1, first:first + H].expand(21, H)             # one row for every token
    assert torch.equal(zc.moe_dispatch(same, ds), zc.moe_dispatch(same.contiguous(), ds))
    # results and operands that start at an odd place
    flat = torch.zeros(63 * H + 3, dtype=dtype, device="cuda")
    out = flat[3:].view(63, H)
    assert torch.equal(zc.moe_dispatch(x, ds, out=out), zc.moe_dispatch(x, ds))
    w = torch.rand(21, 3, device="cuda")
    assert torch.equal(zc.moe_combine(out, ds, w), zc.moe_combine(out.clone(), ds, w))
    a, b = zc.moe_combine_backward(x.contiguous(), out, ds, w), zc.moe_combine_backward(x.contiguous(), out.clone(), ds, w)
    assert torch.equal(a[0], b[0])
    # the two forms may add the products in another order
    size = (host(x)[:, None, :] * host(out)[np.maximum(ds.cpu().numpy(), 0)])
    near(host(a[1]), host(b[1]), 2 * (H / 32 + 20) * U * np.abs(size).sum(-1))


def test_dropped_rows_never_leak_and_slots_out_of_range_take_no_part():
    T, k, H = 6, 2, 96
    ids = torch.tensor([[0, 1], [-1, 2], [-1, -1], [2, 0], [1, -1], [9, 0]], dtype=torch.int32, device="cuda")
    p = zc.moe_plan(ids, 3)
    rows = torch.ones(T * k, H, device="cuda", dtype=torch.bfloat16)
    n = p.offsets[-1].item()
    rows[n:] = float("nan")
    rows[n] = float("inf")
    w = torch.full((T, k), 0.5, device="cuda")
    w[2] = float("nan")                                        # weights of dropped pairs are not looked at
    y = zc.moe_combine(rows, p.slots, w)
    assert torch.isfinite(y).all() and not y[2].any()
    x = torch.full((T, H), float("nan"), device="cuda", dtype=torch.bfloat16)
    x[3] = 1.0
    d = zc.moe_dispatch(x, p.slots)
    assert not d[n:].any()
    gy = torch.ones(T, H, device="cuda", dtype=torch.bfloat16)
    gr, gw = zc.moe_combine_backward(gy, rows, p.slots, w)
    assert not gr[n:].any() and torch.isfinite(gw).all() and not gw[2].any()
    # out of range: skipped, the neighbours untouched
    bad = p.slots.clone()
    bad[0, 0], bad[3, 1] = T * k, 2 ** 31 - 1
    bad[4, 0] = -2 ** 31
    guard = torch.full((T * k, H), 3.0, device="cuda", dtype=torch.bfloat16)
    zc.moe_dispatch(torch.ones_like(gy), bad, out=guard)
    untouched = [int(p.slots[0, 0]), int(p.slots[3, 1]), int(p.slots[4, 0])]
    assert all((guard[i] == 3.0).all() for i in untouched)
    assert torch.isfinite(zc.moe_combine(rows, bad, w)).all()
    _, gw = zc.moe_combine_backward(gy, rows, bad, w, grad_rows=guard)
    assert gw[0, 0] == 0 and gw[3, 1] == 0 and gw[4, 0] == 0


def test_rows_empty():
    s = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    assert zc.moe_dispatch(torch.zeros(0, 64, device="cuda"), s).shape == (0, 64)
    assert zc.moe_combine(torch.zeros(0, 64, device="cuda"), s).shape == (0, 64)
    s = zc.moe_plan(torch.zeros(3, 2, dtype=torch.int32, device="cuda"), 2).slots
    assert zc.moe_dispatch(torch.zeros(3, 0, device="cuda"), s).shape == (6, 0)
    gr, gw = zc.moe_combine_backward(torch.zeros(3, 0, device="cuda"), torch.zeros(6, 0, device="cuda"), s)
    assert gr.shape == (6, 0) and not gw.any()


def test_combine_residual_in_place():
    rng = np.random.default_rng(5)
    ds = torch.from_numpy(random_slots(rng, 30, 2, 8).astype(np.int32)).cuda()
    r = torch.randn(60, 520, device="cuda").bfloat16()
    y = torch.randn(30, 520, device="cuda").bfloat16()
    want = zc.moe_combine(r, ds, residual=y)
    assert torch.equal(zc.moe_combine(r, ds, residual=y, out=y), want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,H", [(30000, 3, 24), (20011, 2, 300), (6000, 5, 768), (5000, 3, 1030), (4100, 2, 1536),
                                   (3000, 7, 2055), (3001, 2, 4096), (900, 9, 3333), (40, 20, 10007)])
def test_many_tokens(T, k, H, dtype):
    """Several turns of every warp, and rows of one piece to many, against sums in 64 bits on the GPU."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T + H)
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    ids = torch.rand(T, 3 * k, generator=gen, device="cuda").topk(k, -1).indices.int()
    ids[torch.rand(T, k, generator=gen, device="cuda") < 0.1] = -1
    slots = zc.moe_plan(ids, 3 * k).slots
    gone = (slots < 0)[:, :, None]
    at = torch.where(slots < 0, -1 - slots, slots).long()
    assert torch.equal(at.view(-1).sort().values, torch.arange(T * k, device="cuda"))
    x, r, res, gy = new(T, H), new(T * k, H), new(T, H), new(T, H)
    w = torch.rand(T, k, generator=gen, device="cuda") - 0.3
    rows = zc.moe_dispatch(x, slots)
    assert torch.equal(rows[at.view(-1)].view(T, k, H), torch.where(gone, torch.zeros((), dtype=dtype, device="cuda"), x[:, None, :].expand(T, k, H)))
    picked = torch.where(gone, 0.0, r[at.view(-1)].view(T, k, H).double())
    terms = picked * w.double()[:, :, None]
    for weights, want, size in ((w, terms.sum(1) + res.double(), terms.abs().sum(1) + res.double().abs()),
                                (None, picked.sum(1), picked.abs().sum(1))):
        y = zc.moe_combine(r, slots, weights, residual=res) if weights is not None else zc.moe_dispatch_backward(r, slots)
        near_rounded(host(y), host(want), 40 * U * host(size), dtype)
    gr, gw = zc.moe_combine_backward(gy, r, slots, w)
    want = torch.where(gone, 0.0, w.double()[:, :, None] * gy.double()[:, None, :])
    near_rounded(host(gr[at.view(-1)]), host(want.view(T * k, H)), 2 * U * np.abs(host(want.view(T * k, H))), dtype)
    products = picked * gy.double()[:, None, :]
    near(host(gw), host(products.sum(-1)), (H / 32 + 20) * U * host(products.abs().sum(-1)))


def test_offsets_past_32_bits():
    """More than 2^31 values (4.3 GB) in the rows: the last rows are where they belong."""
    T, k, H = 66000, 8, 4104
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    ids = torch.rand(T, 16, generator=gen, device="cuda").topk(k, -1).indices.int()
    p = zc.moe_plan(ids, 16)
    x = torch.randn(T, H, generator=gen, device="cuda").bfloat16()
    rows = zc.moe_dispatch(x, p.slots)
    assert rows.numel() > 2 ** 31
    pick = torch.randint(0, T, (200,), generator=gen, device="cuda")
    for j in range(k):
        assert torch.equal(rows[p.slots[pick, j].long()], x[pick])
    back = zc.moe_dispatch_backward(rows, p.slots)
    assert torch.equal(back, (x.float() * k).bfloat16())        # sums of equal values, exact
    gr, gw = zc.moe_combine_backward(x, rows, p.slots)
    assert torch.equal(gr[p.slots[pick, 3].long()], x[pick])
    want = (x[pick].double() ** 2).sum(-1, keepdim=True).expand(-1, k)
    assert ((gw[pick].double() - want).abs() <= (H / 256 + 20) * U * want).all()


# ------------------------------------------------------------------ AdamW
STEP = dict(step=3, lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


def adamw_inputs(rng, sizes, ptype, gtype, first=0):
    """Parameters and gradients as pieces of flat buffers that start `first` values in."""
    def pieces(sigma, dtype):
        flat = torch.from_numpy(rng.standard_normal(first + sum(sizes)) * sigma).to(dtype).cuda()
        return list(flat[first:].split(sizes))
    return pieces(0.02, ptype), pieces(1e-3, gtype)


def check_params(p, p0, change, want, dtype):
    # 10 roundings of the change, 2 of the sum, one to the type
    near(host(p), want, 10 * U * np.abs(change) + 3 * U * np.abs(host(p0)) + 2 * ROUND[dtype] * np.abs(want) * (dtype != torch.float32))


@pytest.mark.parametrize("ptype", TYPES[:2])
@pytest.mark.parametrize("gtype", TYPES[:2])
@pytest.mark.parametrize("sizes,first", [([1], 0), ([4096, 0, 2048, 8], 0), ([1, 7, 2049, 300, 4097, 255, 3], 0),
                                         ([20000, 511], 3), ([5] * 900, 1)])
def test_adamw_32_bit_states(sizes, first, ptype, gtype):
    rng = np.random.default_rng(len(sizes) + first)
    p, g = adamw_inputs(rng, sizes, ptype, gtype, first)
    m = [torch.from_numpy(rng.standard_normal(n) * 3e-4).float().cuda() for n in sizes]
    v = [torch.from_numpy(rng.random(n) * 1e-6).float().cuda() for n in sizes]
    copies = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in sizes] if ptype == torch.float32 else None
    scale = torch.tensor([0.37], device="cuda")
    p0, m0, v0 = ([host(t) for t in ts] for ts in (p, m, v))
    p00 = [t.clone() for t in p]
    zc.adamw_step(p, g, m, v, copies=copies, grad_scale=scale, **STEP)
    gs = float(host(scale)[0])
    for i in range(len(sizes)):
        _, wm, wv, _ = ref.adamw(p0[i], host(g[i]), m0[i], v0[i], STEP["step"], STEP["lr"], STEP["betas"],
                                 STEP["eps"], STEP["weight_decay"], gs)
        # the parameters from the states as they came out: a cancelling m keeps its own error
        c1, c2 = (1 - b ** STEP["step"] for b in STEP["betas"])
        change = STEP["lr"] / c1 * host(m[i]) / (np.sqrt(host(v[i]) / c2) + STEP["eps"])
        check_params(p[i], p00[i], change, p0[i] * (1 - STEP["lr"] * STEP["weight_decay"]) - change, ptype)
        near(host(m[i]), wm, 4 * U * (np.abs(m0[i]) + np.abs(host(g[i]) * gs)))
        near(host(v[i]), wv, 6 * U * wv + 1e-45)
        if copies is not None:
            assert torch.equal(copies[i], p[i].bfloat16())


def check_state8(code, scale, want, root):
    """Each code is the value nearest to what it holds, and each scale is the block's maximum over 448."""
    n = want.size
    blocks = -(-n // 256)
    full = np.zeros(blocks * 256)
    full[:n] = want
    top = np.abs(full.reshape(blocks, 256)).max(1)
    ws = np.maximum(top / 448.0, 2.0 ** -126)
    near(host(scale), ws, 8 * U * ws)
    s = np.repeat(host(scale), 256)[:n]
    y = want / s
    half = ref.e4m3_step(y) / 2 * (1 + 2e-6)
    got = code.float().cpu().numpy().astype(np.float64)
    if root:
        assert ((got > 0) == (want > 0)).all()
        half = np.where((y > 0) & (y < 2.0 ** -9), 2.0 ** -9, half)   # raised to the smallest value
    # what it holds is itself 8 roundings off
    near(got, np.clip(y, -448, 448), half + 8 * U * np.abs(y))


@pytest.mark.parametrize("ptype", TYPES[:2])
@pytest.mark.parametrize("gtype", TYPES[:2])
@pytest.mark.parametrize("sizes,first", [([1], 0), ([256, 0, 2048, 512], 0), ([257, 7, 2049, 300, 4097, 255, 3], 0),
                                         ([20000, 511], 3), ([300] * 500, 1)])
def test_adamw_8_bit_states(sizes, first, ptype, gtype):
    rng = np.random.default_rng(len(sizes) + first + 50)
    p, g = adamw_inputs(rng, sizes, ptype, gtype, first)
    state = [zc.adamw_state(t, bits=8) for t in p]
    m, v, ms, vs = ([s[j] for s in state] for j in range(4))
    copies = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in sizes] if ptype == torch.float32 else None
    for turn in range(3):
        p0, m0, r0 = [host(t) for t in p], [], []
        p00 = [t.clone() for t in p]
        for i, n in enumerate(sizes):
            spread = lambda s: np.repeat(host(s[i]), 256)[:n]  # noqa: E731
            m0.append(m[i].float().cpu().numpy() * spread(ms))
            r0.append(v[i].float().cpu().numpy() * spread(vs))
        how = dict(STEP, step=turn + 1)
        zc.adamw_step(p, g, m, v, scales=(ms, vs), copies=copies, **how)
        for i in range(len(sizes)):
            want, wm, wv, change = ref.adamw(p0[i], host(g[i]), m0[i], r0[i] ** 2, how["step"], how["lr"], how["betas"],
                                             how["eps"], how["weight_decay"])
            # the states are sums of two terms of either sign: the change is as exact as m
            size = np.abs(m0[i]) * 0.9 + np.abs(host(g[i])) * 0.1
            with np.errstate(divide="ignore", invalid="ignore"):
                worst = np.where(wm != 0, np.abs(change / wm) * size, 0.0)
            check_params(p[i], p00[i], worst, want, ptype)
            sure = np.abs(wm) > 1e-3 * size   # m's own rounding is relative to its terms
            if sure.all():
                check_state8(m[i], ms[i], wm, False)
            check_state8(v[i], vs[i], np.sqrt(wv), True)
            if copies is not None:
                assert torch.equal(copies[i], p[i].bfloat16())


def test_adamw_8_bit_small_roots_zero_blocks_and_what_is_not_finite():
    n = 256 * 4
    p = torch.zeros(n, device="cuda")
    g = torch.zeros(n, device="cuda")
    g[:256] = 1e-9                             # far below the block's largest
    g[7] = 1.0
    g[512:768] = 1e-3
    g[600], g[601] = float("inf"), float("nan")
    g[768:] = 1e-30                            # its square is below the smallest float
    m, v, ms, vs = zc.adamw_state(p, bits=8)
    zc.adamw_step([p], [g], [m], [v], scales=([ms], [vs]), step=1, lr=1e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.0)
    mf, vf = m.float(), v.float()
    assert (vf[:256] > 0).all() and vf[8].item() == 2.0 ** -9   # raised, not lost
    assert not mf[256:512].any() and not vf[256:512].any() and ms[1].item() == 2.0 ** -126
    odd = torch.zeros(n, dtype=torch.bool, device="cuda")
    odd[600:602] = True
    assert torch.isnan(mf[odd]).all() and torch.isnan(vf[odd]).all()
    assert torch.isfinite(mf[~odd]).all() and torch.isfinite(vf[~odd]).all()
    assert torch.isfinite(p[~odd]).all() and torch.isfinite(ms).all() and torch.isfinite(vs).all()
    assert (p[512:600] < 0).all()


def test_adamw_streams_and_agreement_of_the_two_forms_of_a_tensor():
    """The same values at aligned and at odd places, and on another stream, give the same bits."""
    torch.manual_seed(4)
    n = 256 * 9 + 100
    for bits in (32, 8):
        for ptype in TYPES[:2]:
            results = []
            for first in (0, 1):
                def piece(t, off=first):
                    flat = torch.zeros(n + 8, dtype=t.dtype, device="cuda") if t.dtype != torch.float8_e4m3fn else \
                        torch.zeros(n + 8, dtype=torch.uint8, device="cuda").view(t.dtype)
                    flat[off:off + n].copy_(t)
                    return flat[off:off + n]
                torch.manual_seed(9)
                p, g = piece((torch.randn(n, device="cuda") * 0.02).to(ptype)), piece(torch.randn(n, device="cuda") * 1e-3)
                s = zc.adamw_state(p, bits)
                m, v = piece(s[0]), piece(s[1])
                side = torch.cuda.Stream() if first else torch.cuda.current_stream()
                side.wait_stream(torch.cuda.current_stream())
                for step in (1, 2, 3):
                    zc.adamw_step([p], [g], [m], [v], step=step, lr=1e-3, stream=side,
                                  scales=([s[2]], [s[3]]) if bits == 8 else None)
                torch.cuda.current_stream().wait_stream(side)
                torch.cuda.synchronize()
                results.append([p.clone(), m.clone().view(torch.uint8), v.clone().view(torch.uint8), *s[2:]])
            assert all(torch.equal(a, b) for a, b in zip(*results))


def test_adamw_past_32_bits():
    """A tensor of more than 2^31 values: its last part equals the same part stepped alone."""
    n, tail = 2 ** 31 + 256 * 5 + 77, 256 * 3 + 77
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    torch.manual_seed(2)
    p[-tail:], g[-tail:] = torch.randn(tail, device="cuda") * 0.02, torch.randn(tail, device="cuda") * 1e-3
    pt, gt = p[-tail:].clone(), g[-tail:].clone()
    m, v, ms, vs = zc.adamw_state(p, bits=8)
    st = zc.adamw_state(pt, bits=8)
    zc.adamw_step([p], [g], [m], [v], scales=([ms], [vs]), step=1, lr=1e-2)
    zc.adamw_step([pt], [gt], [st[0]], [st[1]], scales=([st[2]], [st[3]]), step=1, lr=1e-2)
    assert torch.equal(p[-tail:], pt) and not torch.equal(pt, torch.zeros_like(pt))
    assert torch.equal(m.view(torch.uint8)[-tail:], st[0].view(torch.uint8))
    assert torch.equal(vs[-4:], st[3]) and not p[:256].any()


# ------------------------------------------------------------------ graphs, the pointer-level calls
def test_calls_capture_into_a_cuda_graph_and_replay():
    """Captured once, replayed with new values in the same buffers: what the
    calls give outside a graph."""
    T, E, k, H = 3000, 64, 4, 264
    torch.manual_seed(6)
    logits, x = torch.randn(T, E, device="cuda"), torch.randn(T, H, device="cuda").bfloat16()
    p, g = torch.randn(5000, device="cuda"), torch.randn(5000, device="cuda").bfloat16()
    m, v, ms, vs = zc.adamw_state(p, bits=8)

    def step():
        w, ids = zc.moe_route(logits, k, score="sigmoid")
        plan = zc.moe_plan(ids, E)
        rows = zc.moe_dispatch(x, plan.slots)
        y = zc.moe_combine(rows, plan.slots, w)
        gr, gw = zc.moe_combine_backward(y, rows, plan.slots, w)
        gx = zc.moe_dispatch_backward(gr, plan.slots)
        gl = zc.moe_route_backward(gw, logits, ids, score="sigmoid")
        zc.adamw_step([p], [g], [m], [v], scales=([ms], [vs]), step=2, lr=1e-2)
        return [w, ids, *plan, rows, y, gr, gw, gx, gl]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                # each call once before capturing
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in (1, 2):
        torch.manual_seed(seed)
        logits.copy_(torch.randn(T, E, device="cuda"))
        x.copy_(torch.randn(T, H, device="cuda"))
        g.copy_(torch.randn(5000, device="cuda"))
        before = [t.clone() if t.dtype != torch.float8_e4m3fn else t.view(torch.uint8).clone() for t in (p, m, v, ms, vs)]
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured] + [p.clone(), m.view(torch.uint8).clone(), ms.clone()]
        for t, b in zip((p, m, v, ms, vs), before):
            (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t).copy_(b)
        want = step() + [p, m.view(torch.uint8), ms]
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_pointer_level_calls_match_the_tensor_level():
    T, E, k, H = 200, 32, 2, 96
    torch.manual_seed(8)
    s = torch.cuda.current_stream().cuda_stream
    logits, x = torch.randn(T, E, device="cuda"), torch.randn(T, H, device="cuda").bfloat16()
    w, ids = torch.empty(T, k, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
    opt = zc.RouteOptions(k, 0, 1, 1.0, 1, 1, 0)
    assert zc.zipccl_moe_route(logits.data_ptr(), zc.TYPE_F32, E, T, E, opt, 0, 0, w.data_ptr(), ids.data_ptr(), s) == zc.OK
    w2, ids2 = zc.moe_route(logits, k)
    assert torch.equal(w, w2) and torch.equal(ids, ids2)
    counts, offsets = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E, E + 1))
    slots = torch.empty_like(ids)
    assert zc.zipccl_moe_plan(ids.data_ptr(), T * k, E, counts.data_ptr(), offsets.data_ptr(), slots.data_ptr(), 0, 0, s) == zc.OK
    assert all(torch.equal(a, b) for a, b in zip(zc.moe_plan(ids, E), (counts, offsets, slots)))
    rows, y = torch.empty(T * k, H, dtype=x.dtype, device="cuda"), torch.empty_like(x)
    assert zc.zipccl_moe_dispatch(x.data_ptr(), zc.TYPE_BF16, H, T, k, H, slots.data_ptr(), rows.data_ptr(), s) == zc.OK
    assert torch.equal(rows, zc.moe_dispatch(x, slots))
    assert zc.zipccl_moe_combine(rows.data_ptr(), zc.TYPE_BF16, T, k, H, slots.data_ptr(), w.data_ptr(), x.data_ptr(),
                                 y.data_ptr(), s) == zc.OK
    assert torch.equal(y, zc.moe_combine(rows, slots, w, residual=x))
    gr, gw, gx, gl = torch.empty_like(rows), torch.empty_like(w), torch.empty_like(x), torch.empty_like(logits)
    assert zc.zipccl_moe_combine_backward(y.data_ptr(), rows.data_ptr(), zc.TYPE_BF16, T, k, H, slots.data_ptr(),
                                          w.data_ptr(), gr.data_ptr(), gw.data_ptr(), s) == zc.OK
    assert zc.zipccl_moe_dispatch_backward(gr.data_ptr(), zc.TYPE_BF16, T, k, H, slots.data_ptr(), gx.data_ptr(), s) == zc.OK
    assert zc.zipccl_moe_route_backward(gw.data_ptr(), logits.data_ptr(), zc.TYPE_F32, E, T, E, opt, ids.data_ptr(),
                                        gl.data_ptr(), s) == zc.OK
    a, b = zc.moe_combine_backward(y, rows, slots, w)
    assert torch.equal(gr, a) and torch.equal(gw, b) and torch.equal(gx, zc.moe_dispatch_backward(gr, slots))
    assert torch.equal(gl, zc.moe_route_backward(gw, logits, ids))
    p = torch.randn(700, device="cuda")
    q, m, v = p.clone(), torch.zeros(700, device="cuda"), torch.zeros(700, device="cuda")
    g = p.clone()
    record = (zc.AdamWTensor * 1)(zc.AdamWTensor(d_param=p.data_ptr(), d_grad=g.data_ptr(), d_exp_avg=m.data_ptr(),
                                                 d_exp_avg_sq=v.data_ptr(), n=700))
    assert zc.zipccl_adamw_step(record, 1, zc.TYPE_F32, zc.TYPE_F32, 32, zc.AdamWOptions(1e-3, 0.9, 0.99, 1e-8, 0.1, 1), 0, s) == zc.OK
    zc.adamw_step([q], [g], [torch.zeros_like(m)], [torch.zeros_like(v)], step=1, lr=1e-3, betas=(0.9, 0.99), weight_decay=0.1)
    assert torch.equal(p, q) and m.any()
