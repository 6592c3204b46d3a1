"""The exchange's calls on tensors with stream=: their results and workspaces
are not memory that the current stream may still be reading."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import lossless_bf16_tensor_zipccl_gb300 as zc  # noqa: E402


def test_results_on_another_stream_do_not_take_memory_that_the_current_one_still_reads():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    n = 100_000
    x = torch.randn(n, device="cuda").bfloat16()
    packed = zc.compress(x)
    chunk = packed.chunk(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def compress():
        c = zc.compress(x, stream=side)
        return [c.data, c.offsets]
    for call in (compress, lambda: [zc.decompress(packed, stream=side)],
                 lambda: [zc.decompress_reduce([chunk, chunk], n, stream=side)]):
        sizes = [t.untyped_storage().nbytes() for t in call()]
        torch.cuda.synchronize()
        freed = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in sizes]
        held = {t.data_ptr(): t.nbytes for t in freed}
        del freed
        for t in call():
            assert not any(a <= t.data_ptr() < a + s for a, s in held.items())
        # memory that the current stream has freed is still its own to use again
        assert torch.empty(sizes[0], dtype=torch.uint8, device="cuda").data_ptr() in held
        torch.cuda.synchronize()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(zc.decompress(zc.compress(x, stream=None)).view(torch.int16), x.view(torch.int16))
