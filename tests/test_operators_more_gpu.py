"""The operators around the exchange on the GPU: values, streams, threads and
kinds of arguments beside those of test_operators_gpu.  Tolerances are derived
at each test; u = 2^-24 is half a unit in the last place of a float."""
from __future__ import annotations

import threading
import warnings

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import lossless_bf16_tensor_zipccl_gb300 as zc  # noqa: E402

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    zc.load()
    yield


# ------------------------------------------------------------------ AdamW, what is not finite
@pytest.mark.parametrize("ptype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("first", [0, 1])
def test_adamw_8_bit_root_that_overflowed_makes_its_parameter_nan(ptype, first):
    """A finite gradient whose square is infinite: the first step divides by
    infinity, the second moment's code is then NaN and the first one's is not,
    and the next step's parameter is NaN there and nowhere else."""
    n = 256 * 3 + 40
    at = torch.tensor([3, 300, n - 1], device="cuda")
    flat = lambda dtype: torch.zeros(n + 8, dtype=dtype, device="cuda")[first:first + n]  # noqa: E731
    p, g = flat(ptype), flat(torch.float32)
    p += 0.5
    g += 1e-3
    g[at] = torch.tensor([1e20, -3e19, 1e20], device="cuda")
    m, v, ms, vs = zc.adamw_state(p, bits=8)
    how = dict(scales=([ms], [vs]), lr=3e-4, betas=(0.9, 0.95), weight_decay=0.0)
    zc.adamw_step([p], [g], [m], [v], step=1, **how)
    odd = torch.zeros(n, dtype=torch.bool, device="cuda")
    odd[at] = True
    assert torch.isfinite(p).all() and (p[odd] == 0.5).all()
    assert torch.isfinite(m.float()).all() and torch.equal(torch.isnan(v.float()), odd)
    g.zero_()
    zc.adamw_step([p], [g], [m], [v], step=2, **how)
    assert torch.equal(torch.isnan(p), odd) and torch.isfinite(p[~odd]).all()


@pytest.mark.parametrize("ptype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("first", [0, 1])
def test_adamw_32_bit_second_moment_that_is_not_a_number(ptype, first):
    """NaN, or negative and so without a root, as a damaged checkpoint has them;
    an infinite one divides: no change but the decay."""
    n = 256 + 30
    flat = lambda dtype, x: torch.full((n + 8,), x, dtype=dtype, device="cuda")[first:first + n]  # noqa: E731
    p, g, m, v = flat(ptype, 0.5), flat(torch.float32, 1e-3), flat(torch.float32, 1e-3), flat(torch.float32, 1e-6)
    v[5], v[n - 1], v[17] = float("nan"), -1.0, float("inf")
    m[6] = 0.0
    v[6] = float("nan")
    odd = torch.zeros(n, dtype=torch.bool, device="cuda")
    odd[[5, 6, n - 1]] = True
    zc.adamw_step([p], [g], [m], [v], step=4, lr=3e-4, weight_decay=0.0)
    assert torch.equal(torch.isnan(p), odd) and torch.isfinite(p[~odd]).all() and p[17].item() == 0.5
    assert (p[~odd][:5] < 0.5).all() if ptype == torch.float32 else True


# ------------------------------------------------------------------ devices and streams
class Elsewhere(torch.Tensor):
    """A tensor that says it is on a second GPU, and has no memory."""
    @staticmethod
    def __new__(cls, *shape, dtype):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device="cuda:1")

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise AssertionError(f"{func} on a tensor without memory")


def test_given_results_on_another_device_are_refused():
    f32, i32, u8 = torch.float32, torch.int32, torch.uint8
    l, g = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 2, device="cuda")
    ids, r = torch.zeros(4, 2, dtype=i32, device="cuda"), torch.zeros(8, 8, device="cuda")
    many = torch.zeros(1 << 16, dtype=i32, device="cuda")
    need = zc.zipccl_moe_plan_workspace_bytes(1 << 16, 8)
    for call in (lambda: zc.moe_route(l, 2, weights=Elsewhere(4, 2, dtype=f32)),
                 lambda: zc.moe_route(l, 2, ids=Elsewhere(4, 2, dtype=i32)),
                 lambda: zc.moe_route_backward(g, l, ids, grad_logits=Elsewhere(4, 8, dtype=f32)),
                 lambda: zc.moe_plan(ids, 8, counts=Elsewhere(8, dtype=i32)),
                 lambda: zc.moe_plan(ids, 8, offsets=Elsewhere(9, dtype=i32)),
                 lambda: zc.moe_plan(ids, 8, slots=Elsewhere(4, 2, dtype=i32)),
                 lambda: zc.moe_plan(many, 8, ws=Elsewhere(need, dtype=u8)),
                 lambda: zc.moe_dispatch(l, ids, out=Elsewhere(8, 8, dtype=f32)),
                 lambda: zc.moe_dispatch_backward(r, ids, out=Elsewhere(4, 8, dtype=f32)),
                 lambda: zc.moe_combine(r, ids, out=Elsewhere(4, 8, dtype=f32)),
                 lambda: zc.moe_combine_backward(l, r, ids, grad_rows=Elsewhere(8, 8, dtype=f32)),
                 lambda: zc.moe_combine_backward(l, r, ids, grad_weights=Elsewhere(4, 2, dtype=f32))):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ host threads
def test_plans_of_two_threads_with_different_expert_counts():
    """400 experts (54 KB of shared memory) and 1,024 (139 KB) at once, through
    the calls that leave Python's lock: every call succeeds and has its answer."""
    def work(experts, turns, out):
        torch.cuda.set_device(0)
        gen = torch.Generator().manual_seed(experts)
        ids = torch.randint(-1, experts, (1500,), generator=gen, dtype=torch.int32).cuda()
        counts, offsets, slots = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (experts, experts + 1, 1500))
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        at = [t.data_ptr() for t in (ids, counts, offsets, slots)]
        bad = 0
        for _ in range(turns):
            bad += zc.zipccl_moe_plan(at[0], 1500, experts, *at[1:], 0, 0, stream.cuda_stream) != zc.OK
        stream.synchronize()
        want = torch.bincount(ids[ids >= 0].long(), minlength=experts)
        key = torch.where(ids < 0, experts, ids)
        row = torch.empty_like(ids)
        row[key.sort(stable=True).indices] = torch.arange(1500, dtype=torch.int32, device="cuda")
        out.append((experts, bad, torch.equal(counts.long(), want), torch.equal(slots, torch.where(ids < 0, -1 - row, row))))

    out = []
    threads = [threading.Thread(target=work, args=(e, 4000, out)) for e in (400, 1024, 400, 1024)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert sorted(out) == [(400, 0, True, True)] * 2 + [(1024, 0, True, True)] * 2


def test_results_on_another_stream_do_not_take_memory_that_the_current_one_still_reads():
    """A tensor freed while the current stream's queue still holds its readers:
    its memory is that stream's to use again, and no other's."""
    T, k, E, H = 4096, 4, 64, 128
    logits, x = torch.randn(T, E, device="cuda"), torch.randn(T, H, device="cuda").bfloat16()
    w, ids = zc.moe_route(logits, k)
    plan = zc.moe_plan(ids, E)
    rows = zc.moe_dispatch(x, plan.slots)
    gy, gw = torch.randn_like(x), torch.randn_like(w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    calls = (lambda: zc.moe_route(logits, k, stream=side), lambda: [zc.moe_route_backward(gw, logits, ids, stream=side)],
             lambda: zc.moe_plan(ids, E, stream=side), lambda: [zc.moe_dispatch(x, plan.slots, stream=side)],
             lambda: [zc.moe_dispatch_backward(rows, plan.slots, stream=side)],
             lambda: [zc.moe_combine(rows, plan.slots, w, stream=side)],
             lambda: zc.moe_combine_backward(gy, rows, plan.slots, w, stream=side))
    for call in calls:
        sizes = [t.nbytes for t in call()]
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        freed = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
        held = {t.untyped_storage().data_ptr(): t.nbytes for t in freed}
        del freed
        got = call()
        for t in got:
            assert not any(a <= t.data_ptr() < a + n for a, n in held.items())
        # and on the current stream they are used again, as ever
        at = torch.empty(sizes[0], dtype=torch.uint8, device="cuda").data_ptr()
        assert at in held
        torch.cuda.synchronize()


def test_results_freed_while_the_current_stream_reads_them_are_not_written_by_the_other():
    """A result read by the current stream, freed, and the same call again: the
    first one's readers are still queued, so the second's memory is another."""
    logits = torch.randn(4096, 64, device="cuda")
    other = -logits                           # every kernel is loaded before: loading one may wait for all
    want = zc.moe_route(logits, 4)[0].double().sum()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    w, ids = zc.moe_route(logits, 4, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    first = {w.data_ptr(), ids.data_ptr()}
    torch.cuda._sleep(200_000_000)            # a tenth of a second: kernels queued before the reader
    read = w.double().sum()
    done = torch.cuda.Event()
    done.record()
    del w, ids
    w, ids = zc.moe_route(other, 4, stream=side)
    assert not done.query()
    assert not first & {w.data_ptr(), ids.data_ptr()}
    assert torch.equal(read, want)




# ------------------------------------------------------------------ scores far below and above 0
def sigmoid64(l):
    l = l.double()
    return torch.where(l < 0, l.exp() / (1 + l.exp()), 1 / (1 + (-l).exp()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(6, 4), (64, 9), (256, 8)])
def test_route_sigmoid_scores_down_to_the_smallest_float(E, k, dtype):
    """Logits from -85 to -100, where scores leave the normal floats (-87.3) and
    e^-l the finite ones (-88.7): each keeps its rank and its value.  A score is
    off by two units in the last place of the exponential (4 u of itself, or two
    steps of 2^-149 among the subnormal ones), the sum's and the quotient's
    rounding (2 u, or half a step): 7 u and 3 steps.  Neighbours are 18 steps
    apart or more."""
    step = 1.0 if dtype == torch.bfloat16 else 0.5
    far = -85.0 - step * torch.arange(round(15 / step) + 1)
    gen = torch.Generator().manual_seed(E)
    rows = [torch.cat([far[torch.randperm(len(far), generator=gen)][:k], torch.full((E - k,), -200.0)])
            [torch.randperm(E, generator=gen)] for _ in range(30)]
    l = torch.stack(rows).to(dtype).cuda()
    s = sigmoid64(l)
    want = s.argsort(dim=1, descending=True, stable=True)[:, :k]
    bias = torch.zeros(E, device="cuda")
    ws = s.gather(1, want)
    tol = 7 * U * ws + 3 * 2.0 ** -149
    for b in (bias, None):
        w, ids = zc.moe_route(l, k, score="sigmoid", bias=b, renormalize=False)
        assert torch.equal(ids.long(), want)
        assert ((w.double() - ws).abs() <= tol).all()
        # the quotient: its terms' errors, k additions and a division
        w, ids = zc.moe_route(l, k, score="sigmoid", bias=b)
        total = ws.sum(1, keepdim=True)
        q = ws / total
        assert torch.equal(ids.long(), want)
        assert ((w.double() - q).abs() <= tol / total + q * (tol.sum(1, keepdim=True) / total) * 1.01 + (k + 2) * U * q).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4, 5])
def test_route_without_bias_tells_apart_what_scores_alike(score, groups, dtype):
    """Logits whose 32-bit scores are all 1, or all 0: the largest logits are
    chosen, in order, not the lowest experts."""
    E, k = 20 * groups, 6
    gen = torch.Generator().manual_seed(groups)
    for lo, step in ((20.0, 0.5), (-300.0, 1.0)):
        values = lo + step * torch.arange(E)
        l = torch.stack([values[torch.randperm(E, generator=gen)] for _ in range(40)]).to(dtype)
        kept = max(1, groups - 2)
        best = l.view(40, groups, -1).amax(-1).argsort(dim=1, descending=True, stable=True)[:, :kept]
        allowed = torch.zeros(40, groups, dtype=torch.bool).scatter(1, best, True).repeat_interleave(20, 1)
        want = torch.where(allowed, l.double(), -torch.inf).argsort(dim=1, descending=True, stable=True)[:, :k]
        w, ids = zc.moe_route(l.cuda(), k, score=score, groups=groups, groups_kept=kept)
        assert torch.equal(ids.cpu().long(), want)
        if score == "sigmoid":
            # u of the quotient of equal scores, for each of 1 / k and the sum
            assert torch.allclose(w.cpu(), torch.full((40, k), 1 / k if lo > 0 else 0.0), rtol=4 * U, atol=0)


# ------------------------------------------------------------------ AdamW, its lists
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_takes_iterators(bits):
    """model.parameters() is one: each list is read once."""
    torch.manual_seed(3)
    sizes = (1, 300, 4096)
    p = [torch.randn(n, device="cuda") for n in sizes]
    g = [torch.randn(n, device="cuda") for n in sizes]
    results = []
    for form in (list, iter, lambda x: (t for t in x), tuple):
        q = [t.clone() for t in p]
        states = list(zip(*(zc.adamw_state(t, bits) for t in q)))
        copies = [torch.empty_like(t, dtype=torch.bfloat16) for t in q]
        scales = None if bits == 32 else (form(states[2]), form(states[3]))
        zc.adamw_step(form(q), form(g), form(states[0]), form(states[1]), scales=scales, copies=form(copies), step=1, lr=1e-2)
        results.append(torch.cat(q))
        assert torch.equal(torch.cat(copies), results[-1].bfloat16())
    assert all(torch.equal(r, results[0]) for r in results) and not torch.equal(results[0], torch.cat(p))


# ------------------------------------------------------------------ autograd
def test_what_a_call_writes_counts_as_changed():
    """The version that autograd compares for a tensor it has saved."""
    T, k, E, H = 6, 2, 8, 16
    x, l = torch.randn(T, H, device="cuda"), torch.randn(T, E, device="cuda")
    new = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    i32 = lambda *s: new(*s, dtype=torch.int32)  # noqa: E731
    w, ids, counts, offsets, slots = new(T, k), i32(T, k), i32(E), i32(E + 1), i32(T, k)
    gl, rows, gx, y, gr, gw = new(T, E), new(T * k, H), new(T, H), new(T, H), new(T * k, H), new(T, k)

    def changed(call, *tensors):
        before = [t._version for t in tensors]
        call()
        assert all(t._version > b for t, b in zip(tensors, before))

    changed(lambda: zc.moe_route(l, k, weights=w, ids=ids), w, ids)
    changed(lambda: zc.moe_plan(ids, E, counts=counts, offsets=offsets, slots=slots), counts, offsets, slots)
    changed(lambda: zc.moe_dispatch(x, slots, out=rows), rows)
    changed(lambda: zc.moe_combine(rows, slots, w, out=y), y)
    changed(lambda: zc.moe_combine_backward(y, rows, slots, w, grad_rows=gr, grad_weights=gw), gr, gw)
    changed(lambda: zc.moe_dispatch_backward(gr, slots, out=gx), gx)
    changed(lambda: zc.moe_route_backward(gw, l, ids, grad_logits=gl), gl)
    for bits in (32, 8):
        p = torch.nn.Parameter(torch.randn(300, device="cuda"))
        copy = torch.empty(300, dtype=torch.bfloat16, device="cuda")
        s = zc.adamw_state(p, bits)
        changed(lambda: zc.adamw_step([p], [x.new_ones(300)], [s[0]], [s[1]], copies=[copy], step=1, lr=1e-2,
                                      scales=None if bits == 32 else ([s[2]], [s[3]])), p, copy, *s)
    a = torch.ones(T, H, device="cuda", requires_grad=True)
    loss = (a * y).sum()                      # saves y
    zc.moe_combine(rows, slots, w, out=y)
    with pytest.raises(RuntimeError):
        loss.backward()
    with torch.inference_mode():
        z = torch.empty(T, H, device="cuda")
        assert torch.equal(zc.moe_combine(rows, slots, w, out=z), zc.moe_combine(rows, slots, w))
    zc.moe_combine(rows, slots, w, out=z)     # an inference tensor has no version


def test_operands_that_require_a_gradient_are_warned_of():
    T, k, E, H = 6, 2, 8, 16
    l, x = torch.randn(T, E, device="cuda"), torch.randn(T, H, device="cuda")
    w, ids = zc.moe_route(l, k)
    slots = zc.moe_plan(ids, E).slots
    rows = zc.moe_dispatch(x, slots)
    need = lambda t: t.clone().requires_grad_()  # noqa: E731
    calls = {"moe_route:": lambda f: zc.moe_route(f(l), k), "moe_route_backward:": lambda f: zc.moe_route_backward(f(w), l, ids),
             "moe_dispatch:": lambda f: zc.moe_dispatch(f(x), slots),
             "moe_dispatch_backward:": lambda f: zc.moe_dispatch_backward(f(rows), slots),
             "moe_combine:": lambda f: zc.moe_combine(rows, slots, f(w)),
             "moe_combine_backward:": lambda f: zc.moe_combine_backward(f(x), rows, slots, w)}
    for name, call in calls.items():
        with pytest.warns(UserWarning, match=name) as caught:
            call(need)
        assert caught[0].filename == __file__
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            call(lambda t: t.clone())
            call(lambda t: need(t).detach())
            with torch.no_grad():
                call(need)
            p = torch.nn.Parameter(torch.randn(50, device="cuda"))     # a step is no part of a graph
            zc.adamw_step([p], [torch.ones(50, device="cuda")], *([t] for t in zc.adamw_state(p)), step=1, lr=1e-2)
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            with pytest.raises(UserWarning):
                call(need)


# ------------------------------------------------------------------ AdamW, states that cancel
def e4m3_half_step(y):
    y = y.abs().clamp(min=2.0 ** -6)
    return torch.exp2(torch.floor(torch.log2(y)) - 4)


@pytest.mark.parametrize("first", [0, 3])
@pytest.mark.parametrize("sizes", [[257, 7, 4097], [20000, 511]])
def test_adamw_8_bit_first_moments_of_changing_gradients(sizes, first):
    """Gradients of a new draw each step, so that first moments cancel and change
    sign; every code and scale is checked.  m is off by 4 roundings of its two
    terms' magnitudes (5 u with what is left of them squared); a scale by that of its block's largest value and 2
    roundings; a code is the value nearest to m over the scale, which is off by
    another 3 u."""
    torch.manual_seed(len(sizes) + first)
    flat = lambda s: list((torch.randn(first + sum(sizes), device="cuda") * s)[first:].split(sizes))  # noqa: E731
    p = flat(0.02)
    m, v, ms, vs = (list(x) for x in zip(*(zc.adamw_state(t, bits=8) for t in p)))
    spread = lambda t, s, n: t.double() * s.double().repeat_interleave(256)[:n]  # noqa: E731
    flips = 0
    for step in range(1, 5):
        g = flat(1e-3)
        m0 = [spread(a.float(), s, a.numel()) for a, s in zip(m, ms)]
        zc.adamw_step(p, g, m, v, scales=(ms, vs), step=step, lr=1e-2, betas=(0.9, 0.95))
        for i, n in enumerate(sizes):
            want = 0.9 * m0[i] + 0.1 * g[i].double()
            size = 0.9 * m0[i].abs() + 0.1 * g[i].double().abs()
            off = 5 * U * size
            blocks = torch.nn.functional.pad(torch.stack([want.abs(), off]), (0, -n % 256)).view(2, -1, 256)
            top, slack = blocks[0].amax(1), blocks[1].amax(1)
            s = ms[i].double()
            assert ((s - top / 448).abs() <= (slack + 3 * U * top) / 448 + 2.0 ** -126).all()
            sv = s.repeat_interleave(256)[:n]
            y = (want / sv).clamp(-448, 448)
            code = m[i].float().double()
            tol = (e4m3_half_step(y) + off / sv + 3 * U * y.abs()) * 1.0001
            # where y and its rounding lie on either side of a power of two the coarser step counts
            tol = torch.maximum(tol, (e4m3_half_step(code) + off / sv + 3 * U * y.abs()) * 1.0001)
            assert ((code - y).abs() <= tol).all()
            flips += int(((want * m0[i]) < 0).sum())
    assert flips > 100                            # the draw does what the test is for


# ------------------------------------------------------------------ rows that start anywhere
def pairs(T, k, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    ids = torch.rand(T, 3 * k, generator=gen, device="cuda").topk(k, -1).indices.int()
    ids[torch.rand(T, k, generator=gen, device="cuda") < 0.1] = -1
    slots = zc.moe_plan(ids, 3 * k).slots
    return slots, gen


ROUND = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,k,H", [(3, 2, 1), (40, 2, 7), (900, 3, 64), (300, 2, 1030), (1500, 2, 2055), (61, 4, 10007)])
@pytest.mark.parametrize("start", [0, 1, 5])
def test_residual_in_place_and_operands_at_any_place(T, k, H, dtype, start):
    """Combine with the residual as its result, and both gradients, with every
    row buffer `start` values into its memory, against 64 bits: up to 5 products
    and sums, 2 roundings each (10 u of the magnitudes), and one to the type
    (half a step of 2^-24 below float16's normal range)."""
    slots, gen = pairs(T, k, T + H)

    def new(n):
        flat = torch.randn(n * H + start, generator=gen, device="cuda").to(dtype)
        return flat[start:].view(n, H)
    rows, y, gy = new(T * k), new(T), new(T)
    w = torch.rand(T, k, generator=gen, device="cuda") - 0.3
    gone = (slots < 0)[:, :, None]
    at = torch.where(slots < 0, -1 - slots, slots).long()
    picked = torch.where(gone, 0.0, rows[at.view(-1)].view(T, k, H).double())

    def near(got, want, size):
        tol = 10 * U * size + (0 if dtype == torch.float32 else ROUND[dtype] * want.abs() + 2.0 ** -25)
        assert ((got.double() - want).abs() <= tol).all()
    terms = picked * w.double()[:, :, None]
    want, size = terms.sum(1) + y.double(), terms.abs().sum(1) + y.double().abs()
    got = zc.moe_combine(rows, slots, w, residual=y, out=y)
    assert got.data_ptr() == y.data_ptr()
    near(y, want, size)
    gx = new(T)
    zc.moe_dispatch_backward(rows, slots, out=gx)
    near(gx, picked.sum(1), picked.abs().sum(1))
    gr = new(T * k)
    _, gw = zc.moe_combine_backward(gy, rows, slots, w, grad_rows=gr)
    back = torch.where(gone, 0.0, w.double()[:, :, None] * gy.double()[:, None, :])
    near(gr[at.view(-1)].view(T, k, H), back, back.abs())
    # a lane sums H / 32 products at most, or the 8 of one vector; then a tree
    products = picked * gy.double()[:, None, :]
    runs = max(H / 32, min(H, 8))
    assert ((gw.double() - products.sum(-1)).abs() <= (runs + 20) * U * products.abs().sum(-1)).all()
