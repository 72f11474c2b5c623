"""The 4-bit calls on a stream that is not the current one: outputs that a call allocates come from that
stream's memory, since what the current stream has freed may still be in use there."""

import pytest
import torch

from compressed_sparse_kv_compress_b200 import api

pytestmark = pytest.mark.gpu


def _calls():
    x = torch.randn(512, 1024, device="cuda")
    rows = torch.randn(3000, 256, device="cuda")
    c, s = api.mxfp4_quantize(x)
    cache = api.kv_quantize_fp4(rows)
    return {
        "mxfp4_quantize": lambda **k: api.mxfp4_quantize(x, **k),
        "mxfp4_dequantize": lambda **k: (api.mxfp4_dequantize(c, s, **k),),
        "mxfp4_matmul": lambda **k: (api.mxfp4_matmul(c, s, c, s, **k),),
        "kv_quantize_fp4": lambda **k: (api.kv_quantize_fp4(rows, **k),),
        "kv_dequantize_fp4": lambda **k: (api.kv_dequantize_fp4(cache, **k),),
        "kv_quantize_fp8": lambda **k: (api.kv_quantize_fp8(rows, **k),),
    }


@pytest.mark.parametrize("name", ["mxfp4_quantize", "mxfp4_dequantize", "mxfp4_matmul", "kv_quantize_fp4",
                                  "kv_dequantize_fp4", "kv_quantize_fp8"])
def test_outputs_belong_to_the_stream_of_the_call(name):
    call = _calls()[name]
    torch.cuda.synchronize()
    ref = call()
    freed = [torch.empty_like(o) for o in ref for _ in range(4)]
    torch.cuda.synchronize()
    places = {o.data_ptr() for o in freed}
    del freed                                     # the current stream's, to be had again on it
    side = torch.cuda.Stream()
    got = call(stream=side)
    assert not places & {o.data_ptr() for o in got}
    # one of them had again on the current stream, and written there, while the call runs on its own
    more = [call(stream=side) for _ in range(10)]
    for _ in range(10):
        for o in ref:
            torch.full_like(o, 1)
    torch.cuda.current_stream().wait_stream(side)
    for outs in [got] + more:
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(outs, ref))
