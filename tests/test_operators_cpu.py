"""The operators around the exchange without a GPU: what their calls refuse
(before anything is launched), their workspace sizes, and the reference that
the GPU tests compare with (its gradients against differences)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

import lossless_bf16_tensor_zipccl_gb300 as zc
import operator_reference as ref

FAKE = 1 << 20  # aligned non-null "device" address: never dereferenced, every call below fails validation first


def options(**change):
    o = dict(top_k=2, score=0, renormalize=1, scale=1.0, groups=1, groups_kept=1, group_score=0)
    o.update(change)
    return zc.RouteOptions(**o)


def call_route(opt=None, logits=FAKE, type=0, stride=64, tokens=4, experts=64, bias=None, mask=None, weights=FAKE,
               ids=FAKE):
    return zc.zipccl_moe_route(logits, type, stride, tokens, experts, opt or options(), bias, mask, weights, ids, 0)


@pytest.mark.parametrize("change", [
    dict(type=3), dict(type=-1), dict(experts=0), dict(experts=1025, stride=1025), dict(stride=63), dict(logits=0),
    dict(logits=FAKE + 2), dict(weights=0), dict(weights=FAKE + 2), dict(ids=0), dict(ids=FAKE + 1),
    dict(bias=FAKE + 2), dict(tokens=1 << 30), dict(opt=options(top_k=0)), dict(opt=options(top_k=33)),
    dict(opt=options(top_k=3), experts=2, stride=2), dict(opt=options(score=2)), dict(opt=options(group_score=2)),
    dict(opt=options(groups=0)), dict(opt=options(groups=33), experts=66, stride=66), dict(opt=options(groups=3)),
    dict(opt=options(groups=4, groups_kept=0)), dict(opt=options(groups=4, groups_kept=5)),
    dict(opt=options(groups=64, groups_kept=1)), dict(opt=options(groups=32, groups_kept=1, top_k=3)),
    dict(opt=options(scale=float("nan"))), dict(opt=options(scale=float("inf")))])
def test_route_refusals(change):
    assert call_route(**change) == zc.ERR_INVALID_ARG


def test_route_backward_refusals():
    def call(grad=FAKE, logits=FAKE, ids=FAKE, out=FAKE, opt=None):
        return zc.zipccl_moe_route_backward(grad, logits, 1, 64, 4, 64, opt or options(), ids, out, 0)
    assert call(grad=0) == call(logits=0) == call(ids=0) == call(out=0) == zc.ERR_INVALID_ARG
    assert call(out=FAKE + 1) == call(grad=FAKE + 2) == call(logits=FAKE + 1) == zc.ERR_INVALID_ARG
    assert call(opt=options(top_k=40)) == zc.ERR_INVALID_ARG


def test_empty_calls_need_no_pointers_and_launch_nothing():
    assert call_route(tokens=0, logits=0, weights=0, ids=0) == zc.OK
    assert zc.zipccl_moe_dispatch(0, 1, 0, 0, 2, 64, 0, 0, 0) == zc.OK
    assert zc.zipccl_moe_combine(0, 1, 0, 2, 64, 0, 0, 0, 0, 0) == zc.OK
    assert zc.zipccl_adamw_step(None, 0, 0, 0, 32, zc.AdamWOptions(1e-3, 0.9, 0.99, 1e-8, 0.1, 1), 0, 0) == zc.OK
    empty = (zc.AdamWTensor * 2)()
    assert zc.zipccl_adamw_step(empty, 2, 0, 1, 8, zc.AdamWOptions(1e-3, 0.9, 0.99, 1e-8, 0.1, 1), 0, 0) == zc.OK


def test_plan_refusals_and_workspace():
    assert zc.zipccl_moe_plan_workspace_bytes(100, 64) == 0
    big = zc.zipccl_moe_plan_workspace_bytes(1 << 19, 256)
    assert big > 0
    for pairs, experts in ((1 << 31, 64), (10, 0), (10, 1025)):
        with pytest.raises(zc.ZipcclError) as e:
            zc.zipccl_moe_plan_workspace_bytes(pairs, experts)
        assert e.value.status == zc.ERR_INVALID_ARG

    def call(ids=FAKE, pairs=1 << 19, experts=256, counts=FAKE, offsets=FAKE, slots=FAKE, ws=FAKE, ws_bytes=big):
        return zc.zipccl_moe_plan(ids, pairs, experts, counts, offsets, slots, ws, ws_bytes, 0)
    assert call(ids=0) == call(counts=0) == call(offsets=0) == call(slots=0) == call(ws=0) == zc.ERR_INVALID_ARG
    assert call(ids=FAKE + 2) == call(slots=FAKE + 1) == call(ws=FAKE + 16) == zc.ERR_INVALID_ARG
    assert call(experts=0) == call(pairs=1 << 31) == zc.ERR_INVALID_ARG
    assert call(ws_bytes=big - 1) == zc.ERR_CAPACITY


def test_row_refusals():
    def dispatch(x=FAKE, type=1, stride=64, tokens=4, k=2, hidden=64, slots=FAKE, rows=FAKE):
        return zc.zipccl_moe_dispatch(x, type, stride, tokens, k, hidden, slots, rows, 0)
    bad = [dict(x=0), dict(x=FAKE + 1), dict(type=7), dict(stride=63), dict(k=0), dict(k=33), dict(slots=0),
           dict(slots=FAKE + 2), dict(rows=0), dict(rows=FAKE + 1), dict(tokens=1 << 30), dict(hidden=1 << 31)]
    for b in bad:
        assert dispatch(**b) == zc.ERR_INVALID_ARG, b

    def combine(rows=FAKE, type=1, tokens=4, k=2, hidden=64, slots=FAKE, w=FAKE, res=FAKE, y=FAKE):
        return zc.zipccl_moe_combine(rows, type, tokens, k, hidden, slots, w, res, y, 0)
    for b in [dict(rows=0), dict(type=-1), dict(k=0), dict(slots=0), dict(w=FAKE + 1), dict(res=FAKE + 1), dict(y=0),
              dict(y=FAKE + 1), dict(tokens=1 << 31)]:
        assert combine(**b) == zc.ERR_INVALID_ARG, b
    assert zc.zipccl_moe_dispatch_backward(0, 1, 4, 2, 64, FAKE, FAKE, 0) == zc.ERR_INVALID_ARG

    def back(gy=FAKE, rows=FAKE, gr=FAKE, gw=FAKE, slots=FAKE):
        return zc.zipccl_moe_combine_backward(gy, rows, 0, 4, 2, 64, slots, None, gr, gw, 0)
    assert back(gy=0) == back(rows=0) == back(gr=0) == back(slots=0) == zc.ERR_INVALID_ARG
    assert back(gy=FAKE + 2) == back(gw=FAKE + 2) == zc.ERR_INVALID_ARG


def adamw_options(**change):
    o = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, step=1)
    o.update(change)
    return zc.AdamWOptions(**o)


def adamw_record(**change):
    r = dict(d_param=FAKE, d_grad=FAKE, d_exp_avg=FAKE, d_exp_avg_sq=FAKE, d_avg_scale=FAKE, d_sq_scale=FAKE, n=100)
    r.update(change)
    return (zc.AdamWTensor * 1)(zc.AdamWTensor(**r))


def test_adamw_refusals():
    def call(record=None, n=1, p=0, g=0, bits=8, opt=None, scale=None):
        return zc.zipccl_adamw_step(adamw_record() if record is None else record, n, p, g, bits,
                                    opt or adamw_options(), scale, 0)
    for b in [dict(p=2), dict(g=2), dict(bits=16), dict(scale=FAKE + 2)]:
        assert call(**b) == zc.ERR_INVALID_ARG, b
    for b in [dict(d_param=None), dict(d_grad=None), dict(d_exp_avg=None), dict(d_exp_avg_sq=None),
              dict(d_avg_scale=None), dict(d_sq_scale=None), dict(d_param=FAKE + 2), dict(d_grad=FAKE + 2),
              dict(d_copy=FAKE + 1), dict(d_avg_scale=FAKE + 2), dict(n=(1 << 40) + 1)]:
        assert call(adamw_record(**b)) == zc.ERR_INVALID_ARG, b
    assert call(adamw_record(d_exp_avg=FAKE + 1), bits=32) == zc.ERR_INVALID_ARG
    for b in [dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=-1e-8),
              dict(eps=float("inf")), dict(lr=-1.0), dict(lr=float("inf")), dict(weight_decay=-0.1), dict(step=0)]:
        assert call(opt=adamw_options(**b)) == zc.ERR_INVALID_ARG, b


def test_tensor_refusals():
    torch = pytest.importorskip("torch")
    f, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        zc.moe_route(f, 2)                                        # not on the GPU
    with pytest.raises(TypeError):
        zc.moe_route(f.double(), 2)
    with pytest.raises(ValueError):
        zc.moe_route(f, 2, score="relu")
    with pytest.raises(ValueError):
        zc.moe_route(f, 2, group_score="mean")
    with pytest.raises(ValueError):
        zc.moe_route(f, 0)
    with pytest.raises(TypeError):
        zc.moe_plan(i.long(), 8)
    with pytest.raises(ValueError):
        zc.moe_plan(i, 8)
    with pytest.raises(ValueError):
        zc.moe_dispatch(f, i)
    with pytest.raises(TypeError):
        zc.moe_combine(f.double(), i)
    with pytest.raises(TypeError):
        zc.adamw_step([f.double()], [f], [f], [f], step=1, lr=1e-3)
    with pytest.raises(ValueError):
        zc.adamw_step([f], [f], [f], [f], step=1, lr=1e-3)
    with pytest.raises(ValueError):
        zc.adamw_state(f, bits=4)
    zc.adamw_step([], [], [], [], step=1, lr=1e-3)
    m, v, ms, vs = zc.adamw_state(torch.zeros(300), bits=8)
    assert m.dtype == v.dtype == torch.float8_e4m3fn and ms.numel() == vs.numel() == 2


def test_record_layouts_match_the_header():
    assert ctypes.sizeof(zc.RouteOptions) == 28
    assert ctypes.sizeof(zc.AdamWTensor) == 64
    assert ctypes.sizeof(zc.AdamWOptions) == 48


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_reference_gradient_agrees_with_differences(score, renormalize):
    # central differences of a smooth function in 64 bits: h^2 f'''/6 with
    # h = 1e-4 and derivatives of order 1 is 2e-9, rounding 1e-16 / h = 1e-12
    rng = np.random.default_rng(7)
    logits, g = rng.standard_normal((3, 9)), rng.standard_normal((3, 4))
    w, ids, _ = ref.route(logits, 4, score, renormalize=renormalize, scale=1.7)
    grad = ref.route_grad(g, logits, ids, score, renormalize, 1.7)
    h = 1e-4
    for t in range(3):
        for e in range(9):
            up, down = logits[t].copy(), logits[t].copy()
            up[e] += h
            down[e] -= h
            d = (ref.weigh(up, ids[t], score, renormalize, 1.7) - ref.weigh(down, ids[t], score, renormalize, 1.7)) / (2 * h)
            assert abs((d * g[t]).sum() - grad[t, e]) < 1e-7


def test_reference_combine_gradient_agrees_with_differences():
    # y is linear in the rows and in the weights: differences are exact up to rounding
    rng = np.random.default_rng(8)
    ids = np.array([[0, 2], [1, -1], [-1, -1], [2, 0]])
    _, _, slots = ref.plan(ids, 3)
    rows, w, g = rng.standard_normal((8, 5)), rng.random((4, 2)), rng.standard_normal((4, 5))
    gr, gw, _ = ref.combine_grad(g, rows, slots, w)
    f = lambda r, q: (ref.combine(r, slots, q)[0] * g).sum()  # noqa: E731
    for i in np.ndindex(rows.shape):
        up = rows.copy()
        up[i] += 1.0
        assert abs(f(up, w) - f(rows, w) - gr[i]) < 1e-12
    for i in np.ndindex(w.shape):
        up = w.copy()
        up[i] += 1.0
        assert abs(f(rows, up) - f(rows, w) - gw[i]) < 1e-12
