"""What the experts compute, on the GPU against its definition in 64 bits
(experts_reference).

Tolerances.
 - 8-bit blocks: none.  Scaling by a power of two is exact and the code is one
   rounding, so codes and scales are equal.
 - Products: codes have 4 significant bits and scales are powers of two, so every
   term is exact.  An instruction adds 32 terms to a 32-bit sum and cuts what is
   below its last places: 2 units of 2^-23 of the magnitudes in play at most, which
   the sum of all magnitudes S bounds.  (terms / 32 + 1) 2^-22 S, and the result's
   own rounding: half a step, 2^-8 of a bfloat16 value, 2^-11 of a float16 one
   (2^-25 where that is subnormal), 2^-24 of a float.
 - Layer: each of its three sums, of n terms, is off by (n / 32 + 10) 2^-22 of its
   magnitudes by the same count (chunks are added in ordinary floats, 2^-24 each);
   a 32-bit operand of two parts is off by 2^-22 more.  An activation's slope is at
   most 1.13, a weight's relative change twice that of a logit.  With S the
   magnitudes carried through (experts_reference.layer): 4 ((H + I) / 32 + 40) 2^-22 S.
"""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import experts_reference as ex  # noqa: E402
import lossless_bf16_tensor_zipccl_gb300 as zc  # noqa: E402
from test_operators_gpu import host, near  # noqa: E402

TYPES = [torch.float32, torch.bfloat16, torch.float16]
HALF = {t: torch.finfo(t).eps / 2 for t in TYPES}   # half a step relative to the value: eps is a step at 1, the least of its binade
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    zc.load()
    yield
    torch.cuda.synchronize()
    zc.moe_status()          # no wait inside a kernel has run out


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def exponents(scales):
    return bits(scales).astype(np.int64) - 127


def values(rng, shape, dtype, odd=False):
    """Rows and columns of uneven size; odd: what is not finite, zeros, the smallest and largest values among them."""
    x = rng.normal(size=shape) * np.exp2(rng.integers(-6, 7, shape[-1])) * np.exp2(rng.integers(-3, 4, shape[:-1] + (1,)))
    t = torch.from_numpy(x).to(dtype)
    if odd:
        f = torch.finfo(dtype)
        picks = torch.tensor([np.inf, -np.inf, np.nan, 0.0, -0.0, f.max, f.min, f.tiny, f.tiny / 4, 448.0, 449.0, 1.75, 1.8125]).to(dtype)
        at = torch.from_numpy(rng.integers(0, 60, shape))
        t = torch.where(at < len(picks), picks[at.clamp(max=len(picks) - 1)], t)
    return t.cuda()


def placed(t, how):
    """The same values aligned, as a slice of wider rows, or from an odd place on."""
    if how == "whole":
        return t
    if how == "slice":
        wide = torch.zeros(t.shape[0], t.shape[1] + 19, dtype=t.dtype, device="cuda")
        wide[:, 3:3 + t.shape[1]] = t
        return wide[:, 3:3 + t.shape[1]]
    flat = torch.zeros(t.numel() + 8, dtype=t.dtype, device="cuda")
    flat[1:1 + t.numel()] = t.reshape(-1)
    return flat[1:1 + t.numel()].view(t.shape)


def same_codes(blocks, want):
    codes, scales = want
    assert np.array_equal(exponents(blocks.scales), scales)
    assert np.array_equal(host(blocks.codes), codes, equal_nan=True)


SHAPES = [(1, 1), (1, 16), (3, 127), (5, 129), (130, 128), (257, 640), (40, 1000), (129, 17)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("how", ["whole", "slice", "odd place"])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_rows(shape, how, dtype):
    rng = np.random.default_rng(shape[0] * 7 + shape[1])
    for odd in (False, True):
        x = values(rng, shape, dtype, odd)
        q = zc.moe_quantize(placed(x, how))
        assert q.codes.shape == shape and q.scales.shape == (shape[0], -(-shape[1] // 128))
        same_codes(q, ex.quantize_rows(host(x)))


CHUNKS = {
    "one": None, "several": [0, 1, 1, 130, 386], "to the end": [0, 127, 255, 400], "none": [0, 0, 0],
    "falling and outside": [7, 50, 20, 1000000, -5, 300], "many": [0] + [3 * i for i in range(1, 101)],
}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("chunks", CHUNKS)
@pytest.mark.parametrize("cols,how", [(1, "whole"), (256, "whole"), (200, "slice"), (131, "odd place")])
def test_quantize_columns(cols, how, chunks, dtype):
    rng = np.random.default_rng(cols)
    offsets = CHUNKS[chunks]
    at = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    x = values(rng, (400, cols), dtype, odd=cols != 256)
    rows, columns = zc.moe_quantize_columns(placed(x, how), at, by_rows=True)
    same_codes(columns, ex.quantize_columns(host(x), offsets))
    same_codes(rows, ex.quantize_rows(host(x)))
    alone = zc.moe_quantize_columns(placed(x, how), at)
    assert np.array_equal(bits(alone.codes), bits(columns.codes)) and np.array_equal(bits(alone.scales), bits(columns.scales))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 128, 128), (3, 130, 257), (1, 40, 1000), (5, 16, 16)])
def test_quantize_weights(shape, dtype):
    rng = np.random.default_rng(sum(shape))
    for odd in (False, True):
        w = values(rng, shape, dtype, odd)
        same_codes(zc.moe_quantize_weights(w), ex.quantize_weights(host(w)))
    alone = zc.moe_quantize_weights(w[0])
    assert alone.scales.dim() == 2
    same_codes(zc.Fp8Blocks(alone.codes[None], alone.scales[None]), ex.quantize_weights(host(w[:1])))


def test_no_rows_and_given_results():
    for shape in ((0, 256), (4, 0)):
        q = zc.moe_quantize(torch.zeros(shape, device="cuda"))
        assert q.codes.shape == shape
        assert zc.moe_quantize(torch.zeros(shape, device="cuda").as_strided(shape, (0, 0))).codes.shape == shape
    at = torch.zeros(4, dtype=torch.int32, device="cuda")
    q = zc.moe_quantize_columns(torch.zeros(0, 64, device="cuda"), at)
    assert not bits(q.scales).any() and q.scales.shape == (3, 64)
    x = torch.randn(70, 200, device="cuda")
    held = torch.full((70, 256), 7, dtype=torch.uint8, device="cuda")
    out = zc.Fp8Blocks(held.view(F8)[:, :200], torch.empty(70, 2, dtype=torch.float8_e8m0fnu, device="cuda"))
    got = zc.moe_quantize(x, out=out)
    assert got.codes.data_ptr() == out.codes.data_ptr() and (held[:, 200:] == 7).all()   # nothing behind the rows is written
    same_codes(out, ex.quantize_rows(host(x)))
    for bad in (zc.Fp8Blocks(held.view(F8)[:, :128], out.scales), zc.Fp8Blocks(held.view(F8)[:, 1:201], out.scales),
                zc.Fp8Blocks(torch.empty(70, 200, dtype=F8, device="cuda"), out.scales)):
        with pytest.raises((ValueError, zc.ZipcclError)):
            zc.moe_quantize(x, out=bad)


def test_quantize_past_32_bits():
    """More than 2^31 values: the last rows equal the same rows alone."""
    n, cols = (1 << 21) + 5, 1040
    x = torch.zeros(n, cols, dtype=torch.bfloat16, device="cuda")
    x[-300:] = torch.randn(300, cols, device="cuda")
    at = torch.tensor([0, n - 300, n], dtype=torch.int32, device="cuda")
    rows, columns = zc.moe_quantize_columns(x, at, by_rows=True)
    tail, tail_columns = zc.moe_quantize_columns(x[-300:], by_rows=True)
    plain = zc.moe_quantize(x)
    for big in (rows, plain):
        assert torch.equal(big.codes[-300:].view(torch.uint8), tail.codes.view(torch.uint8))
        assert torch.equal(big.scales[-300:].view(torch.uint8), tail.scales.view(torch.uint8))
    assert torch.equal(columns.codes[-300:].view(torch.uint8), tail_columns.codes.view(torch.uint8))
    first = -(-(n - 300) // 128)
    assert torch.equal(columns.scales[first:first + 3].view(torch.uint8), tail_columns.scales[:3].view(torch.uint8))


# ------------------------------------------------------------------ products
def tolerance(terms, size, want, dtype):
    once = HALF[dtype] * np.abs(want)
    if dtype == torch.float16:
        once = np.maximum(once, 2.0 ** -25)
    return (terms / 32 + 1) * 2.0 ** -22 * size + once * 1.001


def product_case(rng, rows, inner, outer, experts, offsets):
    x = torch.from_numpy(rng.normal(size=(rows, inner)) * np.exp2(rng.integers(-4, 5, (rows, 1)))).bfloat16().cuda()
    g = torch.from_numpy(rng.normal(size=(rows, outer)) * np.exp2(rng.integers(-4, 5, (rows, 1)))).bfloat16().cuda()
    w = torch.from_numpy(rng.normal(size=(experts, outer, inner)) * np.exp2(rng.integers(-3, 4, (experts, outer, 1)))).bfloat16().cuda()
    at = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    return x, g, w, at


PRODUCTS = [
    # rows, inner, outer, offsets (None: one matrix)
    (1, 16, 16, None), (1, 1, 1, None), (33, 100, 70, None), (300, 640, 256, None), (513, 128, 513, None), (256, 1024, 130, None),
    (1, 256, 256, [0, 0, 1]), (40, 130, 77, [0, 1, 1, 32, 40]), (700, 256, 384, [0, 257, 257, 512, 545, 700]),
    (600, 333, 129, [0, 300, 600]), (130, 512, 256, [0, 31, 64, 128]), (64, 384, 200, [0] * 9), (90, 257, 300, [0] + [3 * i for i in range(1, 31)]),
    (1000, 200, 260, [5, 200, 100, 5000, -3, 900]), (2049, 64, 48, [0, 2049]),
]


@pytest.mark.parametrize("case", PRODUCTS, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}-{'one' if c[3] is None else len(c[3]) - 1}")
def test_products_and_gradients(case):
    rows, inner, outer, offsets = case
    rng = np.random.default_rng(rows + inner)
    experts = 1 if offsets is None else len(offsets) - 1
    x, g, w, at = product_case(rng, rows, inner, outer, experts, offsets)
    (xr, xc), (gr, gc) = (zc.moe_quantize_columns(t, at, by_rows=True) for t in (x, g))
    wq = zc.moe_quantize_weights(w if offsets is not None else w[0])
    xv, gv, wv = (ex.rows_values(*ex.quantize_rows(host(x))), ex.rows_values(*ex.quantize_rows(host(g))),
                  ex.weights_values(*ex.quantize_weights(host(w))))
    xcv, gcv = (ex.columns_values(*ex.quantize_columns(host(t), offsets), offsets) for t in (x, g))
    forward, backward = ex.matmul(xv, wv, offsets), ex.matmul(gv, wv.transpose(0, 2, 1), offsets)
    by_weights = [t if offsets is not None else t[0] for t in ex.matmul_weights(gcv, xcv, offsets)]
    most = max(b - a for a, b in ex.chunks(offsets, rows))
    for dtype in TYPES:
        near(host(zc.moe_matmul(xr, wq, at, dtype=dtype)), forward[0], tolerance(inner, forward[1], forward[0], dtype))
        near(host(zc.moe_matmul_backward(gr, wq, at, dtype=dtype)), backward[0], tolerance(outer, backward[1], backward[0], dtype))
        near(host(zc.moe_matmul_backward_weights(gc, xc, at, dtype=dtype)), by_weights[0],
             tolerance(most, by_weights[1], by_weights[0], dtype))


def test_products_of_a_thousand_chunks():
    """As many experts as a call takes, most of them without rows."""
    torch.manual_seed(11)
    counts = torch.zeros(1024, dtype=torch.int32)
    counts[[0, 5, 6, 500, 1023]] = torch.tensor([40, 1, 130, 300, 29], dtype=torch.int32)
    at = torch.cat([torch.zeros(1, dtype=torch.int32), counts.cumsum(0).int()]).cuda()
    rows = int(counts.sum())
    x, w = torch.randint(-7, 8, (rows, 128), device="cuda").float(), torch.randint(-7, 8, (1024, 32, 128), device="cuda").float()
    x[:, 0], w[:, 0, 0] = 7, 7
    y = zc.moe_matmul(zc.moe_quantize(x), zc.moe_quantize_weights(w), at, dtype=torch.float32)
    expert = torch.arange(1024).repeat_interleave(counts.long()).cuda()
    assert torch.equal(y, torch.einsum("mk,mnk->mn", x.double(), w[expert].double()).float())
    g = torch.randint(-7, 8, (rows, 32), device="cuda").float()
    gw = zc.moe_matmul_backward_weights(zc.moe_quantize_columns(g, at), zc.moe_quantize_columns(x, at), at, dtype=torch.float32)
    want = torch.zeros(1024, 32, 128, dtype=torch.float64, device="cuda").index_add_(0, expert, torch.einsum("mn,mk->mnk", g.double(), x.double()))
    assert torch.equal(gw, want.float())              # whole numbers up to 7 are exact in every block's scale
    assert not gw[1:5].any() and not gw[7:500].any()


def test_layer_of_the_most_tokens_pairs_and_experts():
    """32 tokens of 32 pairs each, all of 1,024 experts or all of 32: entries of 8 tokens, of 1, and of none."""
    rng = np.random.default_rng(12)
    for E in (1024, 32):
        case = (32, 64, 24, E, 32, True, "silu")
        x, router, up, down, residual = layer_case(rng, case, torch.float32)
        got = zc.moe_layer(x, router, up, down, 32, residual=residual)
        layer_near(got, case, torch.float32, ex.layer(*map(host, (x, router, up, down)), 32, "silu", host(residual)))


def test_products_of_whole_numbers_are_exact():
    """Sums below 2^24 of whole numbers: no rounding anywhere, long sums and large chunks among them."""
    torch.manual_seed(1)
    rows, inner, outer = 1500, 4100, 300
    at = torch.tensor([0, 700, 1450], dtype=torch.int32, device="cuda")
    x = torch.randint(-7, 8, (rows, inner), device="cuda").float()
    w = torch.randint(-7, 8, (2, outer, inner), device="cuda").float()
    g = torch.randint(-7, 8, (rows, outer), device="cuda").float()
    x[:, ::128], g[:, ::128], w[..., ::128] = 7, 7, 7     # every block has the same scale
    x[::128], g[::128] = 7, 7
    (xr, xc), (gr, gc) = (zc.moe_quantize_columns(t, at, by_rows=True) for t in (x, g))
    wq = zc.moe_quantize_weights(w)
    assert torch.equal(wq.codes.float() * wq.scales.float().repeat_interleave(128, 1)[:, :outer].repeat_interleave(128, 2)[..., :inner], w)
    y, gx, gw = (f(a, b, at, dtype=torch.float32) for f, a, b in ((zc.moe_matmul, xr, wq), (zc.moe_matmul_backward, gr, wq),
                                                                  (zc.moe_matmul_backward_weights, gc, xc)))
    for e, (a, b) in enumerate(((0, 700), (700, 1450))):
        assert torch.equal(y[a:b].double(), x[a:b].double() @ w[e].double().T)
        assert torch.equal(gx[a:b].double(), g[a:b].double() @ w[e].double())
        assert torch.equal(gw[e].double(), g[a:b].double().T @ x[a:b].double())
    assert not y[1450:].any() and not gx[1450:].any()


def test_what_is_not_a_number_stays_in_its_rows_and_chunks():
    torch.manual_seed(2)
    x, g = torch.randn(200, 300, device="cuda"), torch.randn(200, 260, device="cuda")
    w = torch.randn(3, 260, 300, device="cuda")
    at = torch.tensor([0, 37, 101, 190], dtype=torch.int32, device="cuda")
    x[60, 5], x[195] = float("nan"), float("inf")          # in the second chunk, and behind the last
    g[60, 7] = float("inf")
    (xr, xc), (gr, gc) = (zc.moe_quantize_columns(t, at, by_rows=True) for t in (x, g))
    wq = zc.moe_quantize_weights(w)
    y, gx = zc.moe_matmul(xr, wq, at), zc.moe_matmul_backward(gr, wq, at)
    gw = zc.moe_matmul_backward_weights(gc, xc, at)
    odd = torch.zeros(200, dtype=torch.bool, device="cuda")
    odd[60] = True
    for t in (y, gx):
        assert t[odd].isnan().all() and t[~odd].isfinite().all()
    assert gw[0].isfinite().all() and gw[2].isfinite().all()
    assert gw[1][:, 5].isnan().all() and gw[1][7].isnan().all()
    rest = gw[1].clone()
    rest[:, 5] = 0
    rest[7] = 0
    assert rest.isfinite().all()
    assert not y[190:].any() and not gx[190:].any()
    scales = wq.scales.view(torch.uint8).clone()
    scales[2, 0, 0] = 255                                  # a block's scale that is no number
    y = zc.moe_matmul(xr, zc.Fp8Blocks(wq.codes, scales.view(torch.float8_e8m0fnu)), at)
    assert y[101:190, :128].isnan().all() and y[101:190, 128:].isfinite().all() and y[:37].isfinite().all()


def test_smallest_and_largest_scales():
    """Scales of 2^-127 and 2^120: products of both ends, and a result past the range of floats."""
    x = torch.full((3, 128), 2.0 ** -140, device="cuda")
    w = torch.full((130, 128), 2.0 ** 120, device="cuda")
    y = zc.moe_matmul(zc.moe_quantize(x), zc.moe_quantize_weights(w), dtype=torch.float32)
    xv, wv = ex.rows_values(*ex.quantize_rows(host(x))), ex.weights_values(*ex.quantize_weights(host(w[None])))
    near(host(y), ex.matmul(xv, wv)[0], 0.0)
    y = zc.moe_matmul(zc.moe_quantize(torch.full((3, 128), 2.0 ** 100, device="cuda")), zc.moe_quantize_weights(w), dtype=torch.float32)
    assert torch.isinf(y).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_results_given_apart_and_at_odd_places(dtype):
    torch.manual_seed(3)
    x, w = torch.randn(150, 256, device="cuda"), torch.randn(2, 136, 256, device="cuda")
    at = torch.tensor([0, 70, 140], dtype=torch.int32, device="cuda")
    xq, wq = zc.moe_quantize(x), zc.moe_quantize_weights(w)
    want = zc.moe_matmul(xq, wq, at, dtype=dtype)
    out = torch.empty_like(want)
    assert zc.moe_matmul(xq, wq, at, dtype=dtype, out=out) is not None and torch.equal(out, want)
    flat = torch.full((150 * 136 + 9,), 5.0, dtype=dtype, device="cuda")
    odd = flat[1:1 + 150 * 136].view(150, 136)
    zc.moe_matmul(xq, wq, at, dtype=dtype, out=odd)
    assert torch.equal(odd, want) and flat[0] == 5 and (flat[-8:] == 5).all()
    a, b = zc.Fp8BlocksArg(xq.codes.data_ptr(), xq.scales.data_ptr(), 256), zc.Fp8BlocksArg(wq.codes.data_ptr(), wq.scales.data_ptr(), 256)
    apart = torch.full((150, 147), 5.0, dtype=dtype, device="cuda")
    type_ = {torch.float32: zc.TYPE_F32, torch.bfloat16: zc.TYPE_BF16, torch.float16: zc.TYPE_F16}[dtype]
    stream = torch.cuda.current_stream().cuda_stream
    assert zc.zipccl_moe_matmul(0, a, b, 150, 256, 136, at.data_ptr(), 2, apart.data_ptr(), type_, 147, stream) == zc.OK
    assert torch.equal(apart[:, :136], want) and (apart[:, 136:] == 5).all()


def test_products_past_32_bits():
    """A result of more than 2^31 values: its last rows equal the same rows alone."""
    rows, inner, outer = (1 << 16) + 3000, 64, 32784
    torch.manual_seed(4)
    x, w = torch.randn(rows, inner, device="cuda"), torch.randn(1, outer, inner, device="cuda")
    wq = zc.moe_quantize_weights(w[0])
    y = zc.moe_matmul(zc.moe_quantize(x), wq)
    assert y.numel() > 2 ** 31
    alone = zc.moe_matmul(zc.moe_quantize(x[-1000:].contiguous()), wq)
    assert torch.equal(y[-1000:], alone) and alone.any()


# ------------------------------------------------------------------ layer
LAYERS = [
    # tokens, hidden, inner, experts, top_k, gated, activation
    (1, 256, 128, 8, 2, True, "silu"), (1, 1, 1, 1, 1, True, "silu"), (2, 5, 3, 4, 2, False, "relu"), (3, 520, 201, 6, 2, False, "gelu"),
    (7, 130, 65, 70, 3, True, "gelu"), (8, 64, 300, 33, 8, True, "relu"), (9, 257, 64, 12, 4, True, "silu"), (16, 1030, 40, 300, 5, False, "silu"),
    (32, 192, 96, 16, 2, True, "silu"), (32, 100, 260, 4, 4, True, "silu"), (5, 2050, 129, 9, 3, True, "silu"), (17, 48, 33, 1024, 32, True, "silu"),
]


def layer_case(rng, case, dtype, **how):
    """Inputs whose choice does not hang on the last bits: drawn again until the nearest logits are 1e-4 apart."""
    T, H, I, E, k, gated, act = case
    up = torch.from_numpy(rng.normal(size=(E, I * (2 if gated else 1), H)) * H ** -0.5).to(dtype).cuda()
    down = torch.from_numpy(rng.normal(size=(E, H, I)) * I ** -0.5).to(dtype).cuda()
    residual = torch.from_numpy(rng.normal(size=(T, H))).to(dtype).cuda()
    router = torch.from_numpy(rng.normal(size=(E, H)) * 2 * H ** -0.5).to(dtype).cuda()
    x = torch.from_numpy(rng.normal(size=(T, H))).to(dtype)
    for _ in range(200):
        l = np.sort(host(x) @ host(router).T, 1)[:, ::-1][:, :k + 1]
        bad = (l[:, :-1] - l[:, 1:] < 1e-4).any(1)
        if not bad.any():
            return x.cuda(), router, up, down, residual
        x[bad] = torch.from_numpy(rng.normal(size=(int(bad.sum()), H))).to(dtype)
    raise AssertionError("no settled draw")


def layer_near(got, case, dtype, want):
    y, w, ids, _, size = want
    T, H, I, E, k = case[:5]
    assert np.array_equal(got[2].cpu().numpy(), ids)
    near(host(got[1]), w, 4 * (H / 32 + 40) * 2.0 ** -22 * (np.abs(w) + 1e-30) * 40)
    once = HALF[dtype] * np.abs(y)
    if dtype == torch.float16:
        once = np.maximum(once, 2.0 ** -25)
    near(host(got[0]), y, 4 * ((H + I) / 32 + 40) * 2.0 ** -22 * size + 1.001 * once)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", LAYERS, ids=lambda c: "-".join(map(str, c[:5])) + f"-{c[6]}")
def test_layer(case, dtype):
    rng = np.random.default_rng(sum(case[:5]))
    x, router, up, down, residual = layer_case(rng, case, dtype)
    k, act = case[4], case[6]
    got = zc.moe_layer(x, router, up, down, k, activation=act, residual=residual)
    assert got[0].dtype == dtype and got[1].dtype == torch.float32 and got[2].dtype == torch.int32
    layer_near(got, case, dtype, ex.layer(*map(host, (x, router, up, down)), k, act, host(residual)))
    if up.numel() > 200:   # the same with weights in 8-bit blocks
        uq, dq = zc.moe_quantize_weights(up), zc.moe_quantize_weights(down)
        uv, dv = (ex.weights_values(*ex.quantize_weights(host(t))) for t in (up, down))
        got = zc.moe_layer(x, router, uq, dq, k, activation=act)
        layer_near(got, case, dtype, ex.layer(host(x), host(router), uv, dv, k, act))


@pytest.mark.parametrize("how", [
    dict(score="sigmoid", scale=2.5), dict(renormalize=False), dict(score="sigmoid", renormalize=False, scale=0.5),
    dict(groups=8, groups_kept=3), dict(groups=5, groups_kept=2, group_score="top2", score="sigmoid"), dict(bias=True, score="sigmoid")])
def test_layer_chooses_as_the_routing_call_does(how):
    """Its weights and ids are those of moe_route for its logits: whole numbers, so that both have the same bits."""
    rng = np.random.default_rng(5)
    T, H, I, E, k = 13, 96, 40, 40, 4
    x = torch.from_numpy(rng.integers(-3, 4, (T, H))).bfloat16().cuda()
    router = torch.from_numpy(rng.integers(-2, 3, (E, H)) / 16).bfloat16().cuda()
    up, down = torch.randn(E, 2 * I, H, device="cuda").bfloat16(), torch.randn(E, H, I, device="cuda").bfloat16()
    mask = torch.from_numpy(rng.random(T) > 0.3).cuda()
    how = dict(how)
    if how.pop("bias", False):
        how["bias"] = torch.from_numpy(rng.integers(-9, 10, E) * 1e-2).float().cuda()
    y, weights, ids = zc.moe_layer(x, router, up, down, k, mask=mask, **how)
    w, i = zc.moe_route(x.float() @ router.float().T, k, mask=mask, **how)
    assert torch.equal(ids, i) and torch.equal(weights, w)
    assert not y[~mask].any() and y[mask].any()


@pytest.mark.parametrize("dtype", TYPES)
def test_layer_operands_at_any_place(dtype):
    """Rows apart, buffers from odd places on, a float router, the residual in place: the same answers."""
    rng = np.random.default_rng(6)
    case = (6, 130, 70, 5, 2, True, "silu")
    x, router, up, down, residual = layer_case(rng, case, dtype)
    want = ex.layer(*map(host, (x, router, up, down)), 2, "silu", host(residual))
    wide = torch.full((6, 150), float("nan"), dtype=dtype, device="cuda")
    wide[:, 11:141] = x
    shifted = [placed(t.reshape(1, -1), "odd place").view(t.shape) for t in (router, up, down)]
    y = residual.clone()
    w, ids = torch.empty(6, 2, device="cuda"), torch.empty(6, 2, dtype=torch.int32, device="cuda")
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    got = zc.moe_layer(wide[:, 11:141], shifted[0], shifted[1], shifted[2], 2, residual=y, out=y, weights=w, ids=ids, ws=ws)
    assert got[0].data_ptr() == y.data_ptr() and got[1].data_ptr() == w.data_ptr()
    layer_near(got, case, dtype, want)
    layer_near(zc.moe_layer(x, router.float(), up, down, 2, residual=residual), case, dtype, want)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")   # too small: another is taken
    layer_near(zc.moe_layer(x, router, up, down, 2, residual=residual, ws=small), case, dtype, want)


@pytest.mark.parametrize("tokens", [3, 12])
def test_layer_what_is_not_a_number_reaches_only_its_tokens(tokens):
    torch.manual_seed(7)
    H, I, E = 256, 96, 6
    x = torch.zeros(tokens, H, device="cuda").bfloat16()
    router = torch.zeros(E, H, device="cuda").bfloat16()
    for e in range(E):
        router[e, e] = 4
    for t in range(tokens):                                     # token t: experts t and t + 1
        x[t] = torch.randn(H, device="cuda") * 0.1
        x[t, :E] = 0
        x[t, t % E], x[t, (t + 1) % E] = 2, 1
    up, down = torch.randn(E, 2 * I, H, device="cuda").bfloat16(), torch.randn(E, H, I, device="cuda").bfloat16()
    good = zc.moe_layer(x, router, up, down, 2)[0]
    up[2, 5, 7], down[2, 9, 3] = float("nan"), float("inf")     # an expert of tokens 1 and 2 (and 7, 8)
    y = zc.moe_layer(x, router, up, down, 2)[0]
    hit = torch.tensor([t % E in (1, 2) for t in range(tokens)], device="cuda")
    assert torch.equal(y[~hit], good[~hit]) and y[hit].isnan().any(1).all()
    x[0, 100] = float("inf")
    y = zc.moe_layer(x, router, up, down, 2)[0]
    assert torch.equal(y[~hit][1:], good[~hit][1:])


def test_layer_of_no_tokens_and_of_masked_ones():
    up, down, router = torch.randn(4, 64, 32, device="cuda"), torch.randn(4, 32, 32, device="cuda"), torch.randn(4, 32, device="cuda")
    y, w, ids = zc.moe_layer(torch.randn(0, 32, device="cuda"), router, up, down, 2)
    assert y.shape == (0, 32) and w.shape == (0, 2) and ids.shape == (0, 2)
    x, residual = torch.randn(5, 32, device="cuda"), torch.randn(5, 32, device="cuda")
    y, w, ids = zc.moe_layer(x, router, up, down, 2, mask=torch.zeros(5, dtype=torch.bool, device="cuda"), residual=residual)
    assert torch.equal(y, residual) and not w.any() and (ids == -1).all()


# ------------------------------------------------------------------ together
def expert_step(x, logits, w, g, k, experts):
    """Forward and backward of an expert layer in 8 bits, as training runs it."""
    weights, ids = zc.moe_route(logits, k)
    plan = zc.moe_plan(ids, experts)
    rows, columns = zc.moe_quantize_columns(zc.moe_dispatch(x, plan.slots), plan.offsets, by_rows=True)
    wq = zc.moe_quantize_weights(w)
    out = zc.moe_matmul(rows, wq, plan.offsets)
    y = zc.moe_combine(out, plan.slots, weights, residual=x)
    grad_out, grad_weights = zc.moe_combine_backward(g, out, plan.slots, weights)
    grad_rows, grad_columns = zc.moe_quantize_columns(grad_out, plan.offsets, by_rows=True)
    grad_x = zc.moe_dispatch_backward(zc.moe_matmul_backward(grad_rows, wq, plan.offsets), plan.slots)
    grad_w = zc.moe_matmul_backward_weights(grad_columns, columns, plan.offsets)
    return y, grad_x, grad_w, grad_weights, zc.moe_route_backward(grad_weights, logits, ids)


def step_inputs(seed, T=700, E=6, H=320, N=320):
    torch.manual_seed(seed)
    return (torch.randn(T, H, device="cuda").bfloat16(), torch.randn(T, E, device="cuda"),
            (torch.randn(E, N, H, device="cuda") * H ** -0.5).bfloat16(), torch.randn(T, N, device="cuda").bfloat16())


def test_a_training_step_in_8_bits_is_near_the_step_in_64():
    """Every operand is rounded to 3 bits after the point, off by at most 2^-4 of itself (2^-10 of its block's
    largest where that is more): a product by 2 * 2^-4 + 2^-8 of its magnitudes at most, and, errors being of
    either sign, by a few hundredths of its size in the mean."""
    x, logits, w, g = step_inputs(1)
    y, grad_x, grad_w, grad_weights, grad_logits = expert_step(x, logits, w, g, 2, 6)
    xd, ld, wd = (t.double().requires_grad_() for t in (x, logits, w))
    top = ld.softmax(1).topk(2, 1)
    share = top.values / top.values.sum(1, keepdim=True)
    out = xd + sum(share[:, j, None] * torch.einsum("tnh,th->tn", wd[top.indices[:, j]], xd) for j in range(2))
    (out * g.double()).sum().backward()
    for got, want in ((y, out), (grad_x, xd.grad - g.double()), (grad_w, wd.grad), (grad_logits, ld.grad)):
        want = want.detach()
        assert (got.double() - want).norm() < 2 * 2.0 ** -4 * want.norm()


def test_steps_capture_replay_and_repeat():
    """Captured in two graphs that share inputs, replayed in turn with new values: the bits of calls outside a graph."""
    x, logits, w, g = step_inputs(2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    few = (torch.randn(6, 320, device="cuda") * 0.05).bfloat16()
    down = torch.randn(6, 320, 160, device="cuda").bfloat16()

    def step():
        return [*expert_step(x, logits, w, g, 2, 6), *zc.moe_layer(x[:4], few, w, down, 2)]

    with torch.cuda.stream(side):
        first = step()                        # each call once before capturing
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, step()))
            assert graphs[-1][0] is graph
    for seed in (3, 4):
        for a, b in zip((x, logits, w, g), step_inputs(seed)):
            a.copy_(b)
        for graph, captured in graphs:
            graph.replay()
            got = [t.clone() for t in captured]
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_calls_on_another_stream_give_the_same_bits():
    x, logits, w, g = step_inputs(5)
    at = torch.tensor([0, 100, 300, 301, 650, 650, 700], dtype=torch.int32, device="cuda")
    down, router = torch.randn(6, 320, 160, device="cuda").bfloat16(), torch.randn(6, 320, device="cuda").bfloat16()
    side = torch.cuda.Stream()

    def calls(stream):
        rows, columns = zc.moe_quantize_columns(x, at, by_rows=True, stream=stream)
        grad_rows, grad_columns = zc.moe_quantize_columns(g, at, by_rows=True, stream=stream)
        wq = zc.moe_quantize_weights(w, stream=stream)
        return [zc.moe_quantize(x, stream=stream).codes.view(torch.uint8), zc.moe_matmul(rows, wq, at, stream=stream),
                zc.moe_matmul_backward(grad_rows, wq, at, stream=stream),
                zc.moe_matmul_backward_weights(grad_columns, columns, at, stream=stream),
                *zc.moe_layer(x[:5], router, w, down, 2, stream=stream)]

    want = calls(None)
    torch.cuda.synchronize()
    for _ in range(5):
        got = calls(side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        side.wait_stream(torch.cuda.current_stream())


def test_layer_agrees_with_the_calls_for_many_tokens():
    """The layer in 8-bit blocks, and route, plan, dispatch, quantize, products, combine: the second rounds rows and h
    to 8 bits, off by 2^-4 of themselves at most each, and the results of three products to bfloat16."""
    torch.manual_seed(8)
    T, H, I, E, k = 20, 512, 256, 8, 2
    x, router = torch.randn(T, H, device="cuda").bfloat16(), torch.randn(E, H, device="cuda").bfloat16() * 0.1
    up, down = torch.randn(E, 2 * I, H, device="cuda").bfloat16() * 0.05, torch.randn(E, H, I, device="cuda").bfloat16() * 0.06
    uq, dq = zc.moe_quantize_weights(up), zc.moe_quantize_weights(down)
    y, weights, ids = zc.moe_layer(x, router, uq, dq, k, residual=x)
    plan = zc.moe_plan(ids, E)
    rows = zc.moe_matmul(zc.moe_quantize(zc.moe_dispatch(x, plan.slots)), uq, plan.offsets)
    h = (torch.nn.functional.silu(rows[:, :I].float()) * rows[:, I:].float()).bfloat16()
    z = zc.moe_combine(zc.moe_matmul(zc.moe_quantize(h), dq, plan.offsets), plan.slots, weights, residual=x)
    part = (y - x).double()
    assert ((z - x).double() - part).norm() < 3 * 2.0 ** -4 * part.norm()


def test_example_runs_in_8_bits_and_its_gradients_are_near_those_of_16():
    """The example's step with its products in 8 bits: gradients off by the rounding of both operands, 2^-4 of each at
    most, so by less than 2 * 2^-4 of their norm."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_training_step.py")
    spec = importlib.util.spec_from_file_location("moe_training_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    torch.manual_seed(10)
    x, target = torch.randn(500, 192, device="cuda").bfloat16(), torch.randn(500, 192, device="cuda")
    grads = [example.Layer(192, 5, 8, fp8=fp8).forward_backward(x, target, 2)[1].double() for fp8 in (False, True)]
    assert (grads[0] - grads[1]).norm() < 2 * 2.0 ** -4 * grads[0].norm()
    losses, ratio = example.train(steps=2, ranks=2, tokens=300, hidden=200, experts=4, fp8=True)
    assert all(np.isfinite(losses)) and ratio < 1


def test_pointer_level_calls_match_the_tensor_level():
    torch.manual_seed(9)
    s = torch.cuda.current_stream().cuda_stream
    x, w = torch.randn(90, 200, device="cuda").bfloat16(), torch.randn(2, 70, 200, device="cuda").bfloat16()
    at = torch.tensor([0, 30, 90], dtype=torch.int32, device="cuda")
    byte = lambda *n: torch.zeros(*n, dtype=torch.uint8, device="cuda")  # noqa: E731
    codes, scales, wide, column_scales = byte(90, 208), byte(90, 2), byte(90, 208), byte(2, 200)
    assert zc.zipccl_moe_quantize(x.data_ptr(), zc.TYPE_BF16, 200, 90, 200, codes.data_ptr(), 208, scales.data_ptr(), s) == zc.OK
    q = zc.moe_quantize(x)
    assert np.array_equal(bits(q.codes), codes[:, :200].cpu().numpy()) and np.array_equal(bits(q.scales), scales.cpu().numpy())
    assert zc.zipccl_moe_quantize_columns(x.data_ptr(), zc.TYPE_BF16, 200, 90, 200, at.data_ptr(), 2, wide.data_ptr(), 208,
                                          column_scales.data_ptr(), 0, 0, 0, s) == zc.OK
    c = zc.moe_quantize_columns(x, at)
    assert np.array_equal(bits(c.codes), wide[:, :200].cpu().numpy()) and np.array_equal(bits(c.scales), column_scales.cpu().numpy())
    wcodes, wscales = byte(2, 70, 208), byte(2, 1, 2)
    assert zc.zipccl_moe_quantize_weights(w.data_ptr(), zc.TYPE_BF16, 2, 70, 200, wcodes.data_ptr(), 208, wscales.data_ptr(), s) == zc.OK
    wq = zc.moe_quantize_weights(w)
    assert np.array_equal(bits(wq.scales), wscales.cpu().numpy())
    y = torch.empty(90, 70, dtype=torch.bfloat16, device="cuda")
    a, b = zc.Fp8BlocksArg(codes.data_ptr(), scales.data_ptr(), 208), zc.Fp8BlocksArg(wcodes.data_ptr(), wscales.data_ptr(), 208)
    assert zc.zipccl_moe_matmul(zc.MATMUL_FORWARD, a, b, 90, 200, 70, at.data_ptr(), 2, y.data_ptr(), zc.TYPE_BF16, 70, s) == zc.OK
    assert torch.equal(y, zc.moe_matmul(q, wq, at))
    up, down, router = torch.randn(4, 60, 200, device="cuda"), torch.randn(4, 200, 30, device="cuda"), torch.randn(4, 200, device="cuda")
    t = torch.randn(3, 200, device="cuda")
    got = [torch.empty(3, 200, device="cuda"), torch.empty(3, 2, device="cuda"), torch.empty(3, 2, dtype=torch.int32, device="cuda")]
    need = zc.zipccl_moe_layer_workspace_bytes(3, 2, 30)
    ws = byte(need)
    args = zc.MoeLayerArgs(d_x=t.data_ptr(), d_router=router.data_ptr(), d_up=up.data_ptr(), d_down=down.data_ptr(), d_y=got[0].data_ptr(),
                           d_weights=got[1].data_ptr(), d_ids=got[2].data_ptr(), tokens=3, hidden=200, inner=30, x_stride=200, up_stride=200,
                           down_stride=30, experts=4, type=zc.TYPE_F32, router_type=zc.TYPE_F32, weight_bits=32, gated=1, activation=0)
    assert zc.zipccl_moe_layer(args, zc.RouteOptions(2, 0, 1, 1.0, 1, 1, 0), ws.data_ptr(), need, s) == zc.OK
    assert all(torch.equal(a, b) for a, b in zip(got, zc.moe_layer(t, router, up, down, 2)))
    assert zc.zipccl_moe_status(s) == zc.OK


def test_operands_that_require_a_gradient_are_warned_of_and_what_is_written_counts_as_changed():
    x = torch.randn(4, 64, device="cuda", requires_grad=True)
    w = torch.randn(2, 64, 64, device="cuda", requires_grad=True)
    router, down = torch.randn(2, 64, device="cuda"), torch.randn(2, 64, 32, device="cuda")
    for call in (lambda: zc.moe_quantize(x), lambda: zc.moe_quantize_columns(x), lambda: zc.moe_quantize_weights(w),
                 lambda: zc.moe_layer(x, router, w, down, 1)):
        with pytest.warns(UserWarning, match="requires a gradient"):
            call()
    y = torch.empty(4, 64, device="cuda")
    before = y._version
    zc.moe_layer(x.detach(), router, w.detach(), down, 1, out=y)
    out = torch.empty(4, 64, device="cuda", dtype=torch.bfloat16)
    zc.moe_matmul(zc.moe_quantize(x.detach()), zc.moe_quantize_weights(w.detach()[0]), out=out)
    assert y._version > before and out._version > 0
