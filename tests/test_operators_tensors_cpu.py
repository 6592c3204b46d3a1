"""What the operators' calls on tensors refuse before they touch a device:
operands are stand-ins that carry a device, a type and a shape, and no memory."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import lossless_bf16_tensor_zipccl_gb300 as zc  # noqa: E402


class StandIn(torch.Tensor):
    @staticmethod
    def __new__(cls, *shape, dtype=torch.float32, device="cuda:0"):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device=device)

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise AssertionError(f"{func} on a tensor without memory")


def here(*shape, dtype=torch.float32):
    return StandIn(*shape, dtype=dtype)


def there(*shape, dtype=torch.float32):
    return StandIn(*shape, dtype=dtype, device="cuda:1")


I32, F8 = torch.int32, torch.float8_e4m3fn
ADAMW = dict(step=1, lr=1e-3)
OTHER_DEVICE = {
    "route, bias": lambda: zc.moe_route(here(4, 8), 2, bias=there(8)),
    "route, mask": lambda: zc.moe_route(here(4, 8), 2, mask=there(4, dtype=torch.bool)),
    "route backward, grad": lambda: zc.moe_route_backward(there(4, 2), here(4, 8), here(4, 2, dtype=I32)),
    "route backward, ids": lambda: zc.moe_route_backward(here(4, 2), here(4, 8), there(4, 2, dtype=I32)),
    "dispatch, slots": lambda: zc.moe_dispatch(here(4, 8), there(4, 2, dtype=I32)),
    "dispatch backward, slots": lambda: zc.moe_dispatch_backward(here(8, 8), there(4, 2, dtype=I32)),
    "combine, slots": lambda: zc.moe_combine(here(8, 8), there(4, 2, dtype=I32)),
    "combine, weights": lambda: zc.moe_combine(here(8, 8), here(4, 2, dtype=I32), there(4, 2)),
    "combine, residual": lambda: zc.moe_combine(here(8, 8), here(4, 2, dtype=I32), residual=there(4, 8)),
    "combine, residual on the host": lambda: zc.moe_combine(here(8, 8), here(4, 2, dtype=I32), residual=torch.zeros(4, 8)),
    "combine backward, grad": lambda: zc.moe_combine_backward(there(4, 8), here(8, 8), here(4, 2, dtype=I32)),
    "combine backward, weights": lambda: zc.moe_combine_backward(here(4, 8), here(8, 8), here(4, 2, dtype=I32), there(4, 2)),
    "adamw, a later parameter": lambda: zc.adamw_step([here(5), there(5)], [here(5)] * 2, [here(5)] * 2, [here(5)] * 2, **ADAMW),
    "adamw, grads": lambda: zc.adamw_step([here(5)], [there(5)], [here(5)], [here(5)], **ADAMW),
    "adamw, exp_avgs": lambda: zc.adamw_step([here(5)], [here(5)], [there(5)], [here(5)], **ADAMW),
    "adamw, exp_avg_sqs": lambda: zc.adamw_step([here(5)], [here(5)], [here(5)], [there(5)], **ADAMW),
    "adamw, scales": lambda: zc.adamw_step([here(5)], [here(5)], [here(5, dtype=F8)], [here(5, dtype=F8)],
                                           scales=([here(1)], [there(1)]), **ADAMW),
    "adamw, copies": lambda: zc.adamw_step([here(5)], [here(5)], [here(5)], [here(5)],
                                           copies=[there(5, dtype=torch.bfloat16)], **ADAMW),
    "adamw, grad_scale": lambda: zc.adamw_step([here(5)], [here(5)], [here(5)], [here(5)], grad_scale=there(1), **ADAMW),
}


@pytest.mark.parametrize("what", OTHER_DEVICE)
def test_operands_on_another_device_are_refused_before_anything_runs(what):
    with pytest.raises(ValueError):
        OTHER_DEVICE[what]()


@pytest.mark.parametrize("k", [0, 33, 1 << 31, (1 << 32) + 2])
def test_pairs_of_a_token_that_no_call_takes_are_refused_before_anything_is_allocated(k):
    """The library's own refusal, however many: a count past 32 bits is not cut, and no
    result of that size is asked for."""
    T, H = 3, 1
    ids, slots, w = here(T, k, dtype=I32), here(T, k, dtype=I32), here(T, k)
    calls = [lambda: zc.moe_route_backward(w, here(T, 8), ids), lambda: zc.moe_dispatch(here(T, H), slots),
             lambda: zc.moe_dispatch_backward(here(T * k, H), slots), lambda: zc.moe_combine(here(T * k, H), slots),
             lambda: zc.moe_combine_backward(here(T, H), here(T * k, H), slots)]
    if k:
        calls.append(lambda: zc.moe_route(here(T, 8), k))
    for call in calls:
        with pytest.raises(zc.ZipcclError) as e:
            call()
        assert e.value.status == zc.ERR_INVALID_ARG
