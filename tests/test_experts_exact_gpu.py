"""The layer for a few tokens where its answers are known exactly, or to a few
units of 32 bits: what a tolerance by the magnitudes of all terms would let pass.
"""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import experts_norms as norms  # noqa: E402
import lossless_bf16_tensor_zipccl_gb300 as zc  # noqa: E402
from experts_norms import ex  # noqa: E402
from test_experts_gpu import LAYERS  # noqa: E402

TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    zc.load()
    yield
    torch.cuda.synchronize()
    zc.moe_status()          # no wait inside a kernel has run out


@pytest.mark.parametrize("blocks", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("inner", [200, 1100])
def test_layer_holds_21_bits_of_h(inner, dtype, blocks):
    """h = 1 + 2^-9 + m 2^-20, m from 0 to 15, and results that are differences of two of them: (m - n) 2^-20,
    exact in every type.  16 bits of h, in two parts of 8, leave 0."""
    torch.manual_seed(1)
    hidden, tokens = 160, 5
    m = torch.randint(0, 16, (inner,), device="cuda").double()
    up = torch.zeros(1, inner, hidden, dtype=torch.float64, device="cuda")
    up[0, :, 0], up[0, :, 1], up[0, :, 2] = 1, m * 2.0 ** -12, 0.5
    x = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda")
    x[:, 0], x[:, 1], x[:, 2] = 1, 2.0 ** -8, 2.0 ** -8
    down = torch.zeros(1, hidden, inner, dtype=torch.float64, device="cuda")
    row = torch.arange(hidden, device="cuda")
    plus, minus = row % inner, (row * 7 + inner // 2) % inner
    down[0, row, plus] += 1
    down[0, row, minus] -= 1
    matrices = [w.to(dtype) for w in (up, down)]
    if blocks:
        matrices = [zc.moe_quantize_weights(w) for w in matrices]
    y, weights, _ = zc.moe_layer(x.to(dtype), torch.ones(1, hidden, dtype=dtype, device="cuda"), *matrices, 1, activation="relu")
    assert (weights == 1).all()
    assert torch.equal(y.double(), ((m[plus] - m[minus]) * 2.0 ** -20).expand(tokens, hidden))


@pytest.mark.parametrize("float_router", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hidden", [64, 256, 1030, 2048, 2050, 7168])
def test_layer_of_infinite_tokens(hidden, dtype, float_router):
    """An infinite value makes every logit infinite, by the sign of the router's weight there: experts and weights as
    moe_route gives for these logits, and nothing of that token's result is finite.  The other tokens do not change."""
    torch.manual_seed(hidden)
    experts, inner, tokens = 6, 24, 11
    router = torch.randn(experts, hidden, device="cuda")
    router = ((router + router.sign()) * hidden ** -0.5).to(torch.float32 if float_router else dtype)  # none near 0
    up, down = torch.randn(experts, 2 * inner, hidden, device="cuda").to(dtype), torch.randn(experts, hidden, inner, device="cuda").to(dtype)
    residual, good = torch.randn(tokens, hidden, device="cuda").to(dtype), torch.randn(tokens, hidden, device="cuda").to(dtype)
    want = zc.moe_layer(good, router, up, down, 2, residual=residual)
    for i, at in enumerate(sorted({*range(0, hidden, hidden // 19), 1, hidden // 2 - 1, hidden - 1})):
        hit = i % tokens
        x = good.clone()
        x[hit, at] = float("inf") if i % 2 else float("-inf")
        logits = x.double() @ router.double().T
        assert logits[hit].isinf().all()
        w, ids = zc.moe_route(logits.float(), 2)
        got = zc.moe_layer(x, router, up, down, 2, residual=residual)
        assert torch.equal(got[2][hit], ids[hit]) and torch.equal(got[1][hit], w[hit])
        some = ids[hit, 0] >= 0
        assert not got[0][hit].isfinite().any() if some else torch.equal(got[0][hit], residual[hit])
        rest = torch.arange(tokens, device="cuda") != hit
        assert all(torch.equal(a[rest], b[rest]) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", TYPES)
def test_layer_of_a_token_that_is_not_a_number_and_of_an_infinite_router(dtype):
    torch.manual_seed(4)
    router = torch.randn(6, 300, device="cuda").to(dtype)
    up, down = torch.randn(6, 40, 300, device="cuda").to(dtype), torch.randn(6, 300, 20, device="cuda").to(dtype)
    x, residual = (torch.randn(3, 300, device="cuda").to(dtype) for _ in range(2))
    x[1, 77] = float("nan")
    y, w, ids = zc.moe_layer(x, router, up, down, 2, residual=residual)
    assert (ids[1] == -1).all() and not w[1].any() and torch.equal(y[1], residual[1]) and y.isfinite().all()
    x[1, 77] = 1
    router[3, 200], router[4, 211] = float("inf"), float("-inf")
    y, w, ids = zc.moe_layer(x, router, up, down, 2)
    want = zc.moe_route((x.double() @ router.double().T).float(), 2)
    assert torch.equal(ids, want[1]) and y.isfinite().all()


def _through(gates, factors, activation):
    """act(gate) * factor for each pair, through a gated layer of one expert: a token's only value is 1, `down` is the unit matrix."""
    n = gates.numel()
    x = torch.zeros(1, n, device="cuda")
    x[0, 0] = 1
    up = torch.zeros(1, 2 * n, n, device="cuda")
    up[0, :n, 0], up[0, n:, 0] = gates, factors
    y, _, _ = zc.moe_layer(x, torch.ones(1, n, device="cuda"), up, torch.eye(n, device="cuda")[None].contiguous(), 1, activation=activation)
    return y[0].double()


def test_gelu_of_negative_gates_is_relatively_near():
    """erfc's argument is off by 2^-23 of itself at most (the gate's second part 2^-22, the constant and the product
    2^-24 each): e^(-v^2/2) by v^2 of that.  erfc itself is off by 4 units (CUDA's bound), the products, h and the
    factor by 2^-21 together."""
    gates = torch.cat([-torch.linspace(0.01, 12, 500), torch.linspace(0.01, 12, 100)]).cuda()
    factors = torch.where(torch.arange(600, device="cuda") % 2 > 0, 1e6, 1.0)
    got = _through(gates, factors, "gelu")
    v = gates.double()
    want = 0.5 * v * torch.erfc(-v * 0.5 ** 0.5) * factors.double()
    assert ((got - want).abs() <= (2.0 ** -20 + v * v * 2.0 ** -21) * want.abs()).all()


def test_silu_keeps_its_value_down_to_the_smallest_floats():
    """e^v is off by v times the gate's 2^-22 and 2^-21 of itself, or by a unit of the smallest floats; factor, product
    and h by 2^-21 together."""
    gates = torch.linspace(-103, 20, 800, device="cuda")
    factors = torch.full((800,), 2.0 ** 100, device="cuda")
    got = _through(gates, factors, "silu")
    v = gates.double()
    want = v * v.sigmoid() * factors.double()
    assert ((got - want).abs() <= (2.0 ** -20 + v.abs() * 2.0 ** -22) * want.abs() + v.abs() * 2.0 ** (100 - 149)).all()


def test_gradient_of_the_weights_of_a_chunk_that_takes_longer_than_a_wait():
    """One chunk of 900 million rows, whose only tile takes longer than the 2 s that a wait has: whole
    numbers in a few rows, the first and the last among them, zeros in the others."""
    rows, cols = 900_000_013, 16
    codes = torch.zeros(rows, cols, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows // 128 + 1, cols), 127, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    at = torch.cat([torch.tensor([0, 127, 128, rows - 14, rows - 13, rows - 1], device="cuda"), torch.randperm(rows // 1000, device="cuda")[:300] * 997])
    at = at.unique()
    some = torch.randint(-7, 8, (at.numel(), cols), device="cuda").float()
    codes[at] = some.to(torch.float8_e4m3fn).view(torch.uint8)
    blocks = zc.Fp8Blocks(codes.view(torch.float8_e4m3fn), scales)
    got = zc.moe_matmul_backward_weights(blocks, blocks, dtype=torch.float32)
    zc.moe_status()
    assert torch.equal(got, some.T @ some)


@pytest.mark.parametrize("float_router", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", LAYERS, ids=lambda c: "-".join(map(str, c[:5])) + f"-{c[6]}")
def test_layer_is_near_in_the_norm(case, dtype, float_router):
    """Plain weights and 8-bit ones, with and without a residual (see experts_norms for the bound)."""
    rng = np.random.default_rng(sum(case[:5]) + 1)
    x, router, up, down, residual = norms.draw(rng, case, dtype, torch.float32 if float_router else None)
    k, act = case[4], case[6]
    blocks = [zc.moe_quantize_weights(w.cuda()) for w in (up, down)]
    in_blocks = [ex.weights_values(*ex.quantize_weights(norms.values(w))) for w in (up, down)]
    for matrices, wv in (([up.cuda(), down.cuda()], [norms.values(w) for w in (up, down)]), (blocks, in_blocks)):
        for r in (residual, None):
            got = zc.moe_layer(x.cuda(), router.cuda(), *matrices, k, activation=act, residual=None if r is None else r.cuda())
            rv = None if r is None else norms.values(r)
            y, w, ids, _, _ = ex.layer(norms.values(x), norms.values(router), *wv, k, act, rv)
            assert np.array_equal(got[2].cpu().numpy(), ids)
            assert norms.weights_off(norms.values(got[1]), w) < 1
            assert norms.off(norms.values(got[0]), y, rv, dtype) < 1


@pytest.mark.parametrize("part", ["x", "up", "down"])
def test_a_32_bit_layer_takes_second_parts(part):
    """Values 1 + m 2^-20 whose ones cancel in the sum: what is left is exact, and 0 where an operand has 11 bits."""
    n = 130
    m = torch.arange(n, device="cuda").double() % 16
    x = torch.zeros(2, n, dtype=torch.float64, device="cuda")
    up, down = (torch.zeros(1, n, n, dtype=torch.float64, device="cuda") for _ in range(2))
    i = torch.arange(n, device="cuda")
    if part == "x":        # h = x[i] - x[16]: m[16] is 0, so none is below 0
        x[:] = 1 + m * 2.0 ** -20
        up[0, i, i] += 1
        up[0, :, 16] -= 1
        down[0, i, i] = 1
        want = m * 2.0 ** -20
    elif part == "up":     # (1 + m 2^-20) x[0] - x[1]
        x[:, :2] = 1
        up[0, :, 0], up[0, :, 1] = 1 + m * 2.0 ** -20, -1
        down[0, i, i] = 1
        want = m * 2.0 ** -20
    else:                  # (1 + m 2^-20) h[0] - h[1]
        x[:, 0] = 1
        up[0, :2, 0] = 1
        down[0, :, 0], down[0, :, 1] = 1 + m * 2.0 ** -20, -1
        want = m * 2.0 ** -20
    y, _, _ = zc.moe_layer(x.float(), torch.ones(1, n, device="cuda"), up.float(), down.float(), 1, activation="relu")
    assert torch.equal(y.double(), want.expand(2, n))


@pytest.mark.parametrize("dtype", TYPES)
def test_layer_of_one_row_for_all_tokens(dtype):
    torch.manual_seed(5)
    router, up, down = (torch.randn(s, device="cuda").to(dtype) for s in ((6, 200), (6, 80, 200), (6, 200, 40)))
    mask = torch.tensor([True] * 5 + [False] + [True] * 5, device="cuda")
    x = torch.randn(1, 200, device="cuda").to(dtype).expand(11, 200)
    assert x.stride(0) == 0
    want = zc.moe_layer(x.contiguous(), router, up, down, 2, mask=mask)
    assert all(torch.equal(a, b) for a, b in zip(zc.moe_layer(x, router, up, down, 2, mask=mask), want))


@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("inner,outer", [(0, 40), (40, 0), (0, 0)])
def test_products_of_no_places_are_zeros(inner, outer, side):
    """What the quantizing calls give for widths of 0, multiplied: sums of nothing, or nothing."""
    at = torch.tensor([0, 3, 9], dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream() if side else None
    x, g, w = torch.ones(10, inner, device="cuda"), torch.ones(10, outer, device="cuda"), torch.ones(2, outer, inner, device="cuda")
    for offsets, matrices in ((at, w), (None, w[0])):
        (xr, xc), (gr, gc) = (zc.moe_quantize_columns(t, offsets, by_rows=True) for t in (x, g))
        wq = zc.moe_quantize_weights(matrices)
        out = torch.full((10, outer), 5.0, device="cuda")
        if side:
            stream.wait_stream(torch.cuda.current_stream())
        y = zc.moe_matmul(xr, wq, offsets, dtype=torch.float32, out=out, stream=stream)
        gx = zc.moe_matmul_backward(gr, wq, offsets, stream=stream)
        gw = zc.moe_matmul_backward_weights(gc, xc, offsets, stream=stream)
        if side:
            torch.cuda.current_stream().wait_stream(stream)
        assert y is out or y.data_ptr() == out.data_ptr()
        assert y.shape == (10, outer) and not y.any() and gx.shape == (10, inner) and not gx.any()
        assert gw.shape == matrices.shape


@pytest.mark.parametrize("terms", [4096, 16384, 131072])
def test_long_sums_of_one_sign(terms):
    """Every instruction cuts less than a unit, 2^-23, of a sum that grows evenly from 0: half of terms / 32 units
    of the whole, terms 2^-29 (and a hundredth, and the last rounding's 2^-23).  Forward and by the weights."""
    torch.manual_seed(terms)
    a, b = (torch.rand(terms, 128, device="cuda") for _ in range(2))

    def spread(scales, *dims):  # of each block, for its places
        s = torch.exp2(scales.view(torch.uint8).double() - 127)
        for d in dims:
            s = s.repeat_interleave(128, d)
        return s

    ac, bc = (zc.moe_quantize_columns(t) for t in (a, b))
    values = [q.codes.double() * spread(q.scales, 0)[:terms] for q in (ac, bc)]
    got = [zc.moe_matmul_backward_weights(ac, bc, dtype=torch.float32)]
    want = [values[0].T @ values[1]]
    ar, bw = zc.moe_quantize(a.T.contiguous()), zc.moe_quantize_weights(b.T.contiguous())
    got.append(zc.moe_matmul(ar, bw, dtype=torch.float32))
    want.append((ar.codes.double() * spread(ar.scales, 1)) @ (bw.codes.double() * spread(bw.scales, 0, 1)).T)
    for g, w in zip(got, want):
        off = (w - g.double()) / w
        assert off.abs().max() <= terms * 2.0 ** -29 * 1.01 + 2.0 ** -23
        assert off.mean() > 0 or terms < 16384   # cut, not rounded: a sum of one sign comes out small


@pytest.mark.parametrize("experts,groups,k", [(6, 1, 2), (8, 4, 3), (40, 1, 4), (40, 5, 8), (40, 20, 4), (63, 9, 2), (64, 1, 9), (64, 8, 8), (100, 1, 4), (300, 1, 6)])
def test_layer_has_the_routing_calls_bits(experts, groups, k):
    """Weights and ids for logits that are whole sixteenths, exact in any order: softmax over all experts, added to a
    bias or as it is, sums its terms in the order of the routing call."""
    torch.manual_seed(experts + k)
    for seed in range(6):
        x, router = torch.randint(-3, 4, (32, 96), device="cuda").bfloat16(), (torch.randint(-2, 3, (experts, 96), device="cuda") / 16).bfloat16()
        up, down = torch.zeros(experts, 16, 96, device="cuda").bfloat16(), torch.zeros(experts, 96, 16, device="cuda").bfloat16()
        bias = torch.randint(-9, 10, (experts,), device="cuda") * 1e-2
        mask = torch.rand(32, device="cuda") < 0.9
        for how in (dict(), dict(renormalize=False), dict(score="sigmoid", renormalize=False, scale=2.5), dict(bias=bias),
                    dict(bias=bias, renormalize=False, mask=mask), dict(bias=bias, score="sigmoid")):
            how.update(groups=groups, groups_kept=max(1, (groups + 1) // 2), group_score="top2" if seed % 2 else "max")
            got = zc.moe_layer(x, router, up, down, k, **how)
            w, ids = zc.moe_route(x.float() @ router.float().T, k, **how)
            assert torch.equal(got[2], ids) and torch.equal(got[1], w)
