"""What the experts' calls refuse before anything is launched, and the reference
that the GPU tests compare with."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

import experts_reference as ex
import lossless_bf16_tensor_zipccl_gb300 as zc

torch = pytest.importorskip("torch")
from test_operators_tensors_cpu import here, there  # noqa: E402

FAKE = 1 << 20  # aligned non-null "device" address: never dereferenced, every call below fails validation first
F8, E8, I32, BF16 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.int32, torch.bfloat16


def quantize(x=FAKE, type=1, stride=256, rows=4, cols=256, codes=FAKE, code_stride=256, scales=FAKE):
    return zc.zipccl_moe_quantize(x, type, stride, rows, cols, codes, code_stride, scales, 0)


def columns(x=FAKE, type=1, stride=256, rows=4, cols=256, offsets=FAKE, experts=3, codes=FAKE, code_stride=256, scales=FAKE,
            row_codes=0, row_stride=0, row_scales=0):
    return zc.zipccl_moe_quantize_columns(x, type, stride, rows, cols, offsets, experts, codes, code_stride, scales,
                                          row_codes, row_stride, row_scales, 0)


def weights(w=FAKE, type=1, experts=2, rows=64, cols=256, codes=FAKE, code_stride=256, scales=FAKE):
    return zc.zipccl_moe_quantize_weights(w, type, experts, rows, cols, codes, code_stride, scales, 0)


COMMON = [dict(type=3), dict(type=-1), dict(rows=1 << 31), dict(cols=(1 << 22) + 1, code_stride=1 << 23), dict(codes=0),
          dict(codes=FAKE + 8), dict(code_stride=240), dict(code_stride=264), dict(scales=0)]


@pytest.mark.parametrize("change", COMMON + [dict(x=0), dict(x=FAKE + 1)])
def test_quantize_refusals(change):
    assert quantize(**change) == zc.ERR_INVALID_ARG


@pytest.mark.parametrize("change", COMMON + [dict(x=0), dict(experts=0), dict(experts=1025), dict(offsets=0), dict(offsets=FAKE + 2),
                                             dict(row_codes=FAKE, row_stride=256), dict(row_codes=FAKE + 4, row_stride=256, row_scales=FAKE),
                                             dict(row_codes=FAKE, row_stride=255, row_scales=FAKE)])
def test_quantize_columns_refusals(change):
    assert columns(**change) == zc.ERR_INVALID_ARG


@pytest.mark.parametrize("change", COMMON + [dict(w=0), dict(w=FAKE + 1)])
def test_quantize_weights_refusals(change):
    assert weights(**change) == zc.ERR_INVALID_ARG


def matmul(form=0, a=FAKE, a_scales=FAKE, a_stride=4096, b=FAKE, b_scales=FAKE, b_stride=4096, rows=100, inner=256, outer=512,
           offsets=FAKE, experts=4, out=FAKE, type=1, stride=512):
    return zc.zipccl_moe_matmul(form, zc.Fp8BlocksArg(a, a_scales, a_stride), zc.Fp8BlocksArg(b, b_scales, b_stride), rows, inner,
                                outer, offsets, experts, out, type, stride, 0)


@pytest.mark.parametrize("change", [
    dict(form=3), dict(form=-1), dict(type=4), dict(a=0), dict(a=FAKE + 8), dict(a_scales=0), dict(a_stride=250), dict(a_stride=200),
    dict(b=0), dict(b=FAKE + 1), dict(b_scales=0), dict(b_stride=128), dict(rows=1 << 31), dict(inner=0), dict(outer=0),
    dict(inner=(1 << 22) + 1), dict(outer=(1 << 22) + 1, stride=1 << 23), dict(experts=0), dict(experts=1025), dict(offsets=0),
    dict(offsets=FAKE + 1), dict(out=0), dict(out=FAKE + 1), dict(stride=511), dict(form=1, a_stride=496), dict(form=2, stride=255)])
def test_matmul_refusals(change):
    assert matmul(**change) == zc.ERR_INVALID_ARG


def layer(ws=FAKE, ws_bytes=1 << 30, options=None, **change):
    a = dict(d_x=FAKE, d_router=FAKE, d_up=FAKE, d_down=FAKE, d_residual=0, d_up_scales=0, d_down_scales=0, d_bias=0, d_mask=0, d_y=FAKE,
             d_weights=FAKE, d_ids=FAKE, tokens=4, hidden=256, inner=128, x_stride=256, up_stride=256, down_stride=128, experts=8, type=1,
             router_type=1, weight_bits=16, gated=1, activation=0)
    a.update(change)
    o = dict(top_k=2, score=0, renormalize=1, scale=1.0, groups=1, groups_kept=1, group_score=0)
    o.update(options or {})
    return zc.zipccl_moe_layer(zc.MoeLayerArgs(**a), zc.RouteOptions(**o), ws, ws_bytes, 0)


@pytest.mark.parametrize("change", [
    dict(d_x=0), dict(d_router=0), dict(d_up=0), dict(d_down=0), dict(d_y=0), dict(d_weights=0), dict(d_ids=0), dict(d_x=FAKE + 1),
    dict(d_up=FAKE + 1), dict(d_down=FAKE + 1), dict(d_y=FAKE + 1), dict(d_weights=FAKE + 2), dict(d_ids=FAKE + 2), dict(d_bias=FAKE + 2),
    dict(d_residual=FAKE + 1), dict(tokens=33), dict(hidden=0), dict(inner=0), dict(hidden=1 << 22, x_stride=1 << 23, up_stride=1 << 23),
    dict(x_stride=255), dict(up_stride=255), dict(down_stride=127), dict(experts=0), dict(experts=1025), dict(type=3), dict(router_type=2),
    dict(weight_bits=32), dict(weight_bits=8), dict(weight_bits=8, d_up_scales=FAKE, d_down_scales=FAKE, up_stride=264),
    dict(weight_bits=8, d_up_scales=FAKE, d_down_scales=FAKE, d_down=FAKE + 8), dict(activation=3), dict(activation=-1), dict(ws=0),
    dict(ws=FAKE + 16), dict(options=dict(top_k=0)), dict(options=dict(top_k=9)), dict(options=dict(score=2)),
    dict(options=dict(groups=3)), dict(options=dict(groups=4, groups_kept=0)), dict(options=dict(groups=8, groups_kept=1)),
    dict(options=dict(scale=float("nan")))])
def test_layer_refusals(change):
    assert layer(**change) == zc.ERR_INVALID_ARG


def test_layer_workspace():
    need = zc.zipccl_moe_layer_workspace_bytes(32, 8, 1000)
    assert need >= 32 * 8 * 1000 * 8 and need % 256 == 0
    assert layer(tokens=32, inner=1000, down_stride=1000, options=dict(top_k=8), ws_bytes=need - 1) == zc.ERR_CAPACITY
    for bad in ((33, 2, 64), (4, 0, 64), (4, 33, 64), (4, 2, 1 << 22)):
        with pytest.raises(zc.ZipcclError):
            zc.zipccl_moe_layer_workspace_bytes(*bad)


def test_empty_calls_launch_nothing():
    assert quantize(rows=0, x=0, codes=0, scales=0) == quantize(cols=0) == zc.OK
    assert columns(cols=0, x=0, codes=0, scales=0) == zc.OK
    assert weights(experts=0, w=0) == weights(rows=0) == weights(cols=0) == zc.OK
    assert matmul(rows=0, a=0, b=0, out=0) == matmul(form=1, rows=0, stride=256) == zc.OK
    assert layer(tokens=0, d_x=0, d_y=0, ws=0, ws_bytes=0) == zc.OK


def test_null_records_are_refused():
    one = zc.Fp8BlocksArg(FAKE, FAKE, 4096)
    lib = zc.load()
    assert lib.zipccl_moe_matmul(0, None, ctypes.byref(one), 4, 16, 16, None, 1, FAKE, 1, 16, None) == zc.ERR_INVALID_ARG
    assert lib.zipccl_moe_matmul(0, ctypes.byref(one), None, 4, 16, 16, None, 1, FAKE, 1, 16, None) == zc.ERR_INVALID_ARG
    assert lib.zipccl_moe_layer(None, None, None, 0, None) == zc.ERR_INVALID_ARG


# ------------------------------------------------------------------ calls on tensors
def blocks(rows, cols, lead=(), place=here):
    return zc.Fp8Blocks(place(*lead, rows, cols, dtype=F8), place(*lead, rows, -(-cols // 128), dtype=E8))


def matrices(experts, rows, cols, place=here):
    return zc.Fp8Blocks(place(experts, rows, cols, dtype=F8), place(experts, -(-rows // 128), -(-cols // 128), dtype=E8))


OFFSETS = dict(dtype=I32)
REFUSED = {
    "quantize, a vector": lambda: zc.moe_quantize(here(8)),
    "columns, offsets on another device": lambda: zc.moe_quantize_columns(here(4, 256), there(3, dtype=I32)),
    "columns, a single offset": lambda: zc.moe_quantize_columns(here(4, 256), here(1, dtype=I32)),
    "columns, rows_out without by_rows": lambda: zc.moe_quantize_columns(here(4, 256), here(3, dtype=I32), rows_out=blocks(4, 256)),
    "weights, one dimension": lambda: zc.moe_quantize_weights(here(256)),
    "matmul, weights for other chunks": lambda: zc.moe_matmul(blocks(4, 256), matrices(3, 128, 256), here(3, dtype=I32)),
    "matmul, another inner size": lambda: zc.moe_matmul(blocks(4, 128), matrices(2, 128, 256), here(3, dtype=I32)),
    "matmul, one matrix and offsets": lambda: zc.moe_matmul(blocks(4, 256), blocks(128, 256), here(3, dtype=I32)),
    "matmul, offsets on another device": lambda: zc.moe_matmul(blocks(4, 256), matrices(2, 128, 256), there(3, dtype=I32)),
    "matmul, weights on another device": lambda: zc.moe_matmul(blocks(4, 256), matrices(2, 128, 256, there), here(3, dtype=I32)),
    "matmul, scales of another shape": lambda: zc.moe_matmul(zc.Fp8Blocks(here(4, 256, dtype=F8), here(4, 1, dtype=E8)),
                                                             matrices(2, 128, 256), here(3, dtype=I32)),
    "backward, another outer size": lambda: zc.moe_matmul_backward(blocks(4, 256), matrices(2, 128, 256), here(3, dtype=I32)),
    "backward by weights, other rows": lambda: zc.moe_matmul_backward_weights(
        zc.Fp8Blocks(here(4, 256, dtype=F8), here(2, 256, dtype=E8)), zc.Fp8Blocks(here(5, 128, dtype=F8), here(2, 128, dtype=E8)),
        here(3, dtype=I32)),
    "layer, router of other experts": lambda: zc.moe_layer(here(4, 256), here(3, 256), here(2, 64, 256), here(2, 256, 32), 2),
    "layer, router on another device": lambda: zc.moe_layer(here(4, 256), there(2, 256), here(2, 64, 256), here(2, 256, 32), 2),
    "layer, up of a third of the rows": lambda: zc.moe_layer(here(4, 256), here(2, 256), here(2, 96, 256), here(2, 256, 32), 2),
    "layer, down on another device": lambda: zc.moe_layer(here(4, 256), here(2, 256), here(2, 64, 256), there(2, 256, 32), 2),
    "layer, mask of other tokens": lambda: zc.moe_layer(here(4, 256), here(2, 256), here(2, 64, 256), here(2, 256, 32), 2,
                                                        mask=here(5, dtype=torch.bool)),
    "layer, residual of another shape": lambda: zc.moe_layer(here(4, 256), here(2, 256), here(2, 64, 256), here(2, 256, 32), 2,
                                                             residual=here(4, 255)),
    "layer, an unknown activation": lambda: zc.moe_layer(here(4, 256), here(2, 256), here(2, 64, 256), here(2, 256, 32), 2,
                                                         activation="tanh"),
}
WRONG_TYPES = {
    "quantize, whole numbers": lambda: zc.moe_quantize(here(4, 256, dtype=I32)),
    "quantize, not a tensor": lambda: zc.moe_quantize([1.0]),
    "matmul, plain rows": lambda: zc.moe_matmul(here(4, 256), matrices(2, 128, 256), here(3, dtype=I32)),
    "matmul, codes of another type": lambda: zc.moe_matmul(zc.Fp8Blocks(here(4, 256, dtype=torch.float8_e5m2), here(4, 2, dtype=E8)),
                                                           matrices(2, 128, 256), here(3, dtype=I32)),
    "matmul, scales as floats": lambda: zc.moe_matmul(zc.Fp8Blocks(here(4, 256, dtype=F8), here(4, 2)), matrices(2, 128, 256),
                                                      here(3, dtype=I32)),
    "matmul, offsets of 64 bits": lambda: zc.moe_matmul(blocks(4, 256), matrices(2, 128, 256), here(3, dtype=torch.int64)),
    "matmul, an 8-bit result": lambda: zc.moe_matmul(blocks(4, 256), matrices(2, 128, 256), here(3, dtype=I32), dtype=F8),
    "layer, weights of another type": lambda: zc.moe_layer(here(4, 256), here(2, 256), here(2, 64, 256, dtype=BF16), here(2, 256, 32), 2),
    "layer, one matrix in blocks": lambda: zc.moe_layer(here(4, 256), here(2, 256), matrices(2, 64, 256), here(2, 256, 32), 2),
    "layer, router of another type": lambda: zc.moe_layer(here(4, 256, dtype=BF16), here(2, 256, dtype=torch.float16),
                                                          here(2, 64, 256, dtype=BF16), here(2, 256, 32, dtype=BF16), 2),
}


@pytest.mark.parametrize("what", REFUSED)
def test_tensors_that_do_not_fit_are_refused(what):
    with pytest.raises(ValueError):
        REFUSED[what]()


@pytest.mark.parametrize("what", WRONG_TYPES)
def test_tensors_of_other_types_are_refused(what):
    with pytest.raises(TypeError):
        WRONG_TYPES[what]()


def test_sizes_past_the_limits_are_the_librarys_refusals():
    wide = (1 << 22) + 16
    calls = [lambda: zc.moe_quantize(here(1, wide)), lambda: zc.moe_quantize_columns(here(1, wide)),
             lambda: zc.moe_quantize_columns(here(1, 16), here(1026, dtype=I32)),
             lambda: zc.moe_quantize_weights(here(1025, 16, 16)),
             lambda: zc.moe_layer(here(33, 16), here(2, 16), here(2, 16, 16), here(2, 16, 16), 2),
             lambda: zc.moe_layer(here(3, 16), here(2, 16), here(2, 16, 16), here(2, 16, 16), 33)]
    for call in calls:
        with pytest.raises(zc.ZipcclError) as e:
            call()
        assert e.value.status == zc.ERR_INVALID_ARG


# ------------------------------------------------------------------ the reference itself
def test_reference_rounds_as_the_type_does():
    rng = np.random.default_rng(1)
    y = np.concatenate([rng.uniform(-448, 448, 4000), rng.normal(0, 0.02, 4000), [0.0, 448.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0]])
    y = y.astype(np.float32).astype(np.float64)
    t = torch.from_numpy(y).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ex.e4m3(y), t)


def test_reference_exponents_are_the_smallest():
    rng = np.random.default_rng(2)
    top = np.concatenate([np.exp2(rng.uniform(-140, 127.9, 500)), 448 * np.exp2(np.arange(-130.0, 119)), [0.0]])
    e = ex.exponents(top)
    assert (top <= 448 * np.exp2(e.astype(float))).all() and (e >= -127).all()
    assert ((e == -127) | (top > 448 * np.exp2(e - 1.0))).all()


def test_reference_gradients_agree_with_differences():
    rng = np.random.default_rng(3)
    x, w, g = rng.normal(size=(9, 5)), rng.normal(size=(3, 4, 5)), rng.normal(size=(9, 4))
    offsets = [0, 4, 4, 8]
    gx = np.zeros_like(x)
    for e, (a, b) in enumerate(ex.chunks(offsets, 9)):
        gx[a:b] = g[a:b] @ w[e]
    gw = ex.matmul_weights(g, x, offsets)[0]
    at = lambda x, w: (g * ex.matmul(x, w, offsets)[0]).sum()  # noqa: E731
    for target, grad in ((x, gx), (w, gw)):
        for i in np.ndindex(target.shape):
            old = target[i]
            target[i] = old + 1e-4
            up = at(x, w)
            target[i] = old - 1e-4
            down = at(x, w)
            target[i] = old
            assert abs((up - down) / 2e-4 - grad[i]) < 1e-8
