"""The `stream` argument on the GPU: a call runs on the stream that the handle names."""
import pytest
import torch

import dense_gemm_13_gb300 as g13

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_gemm_13_gb300 import _build
    _build.build()
    g13.load()


@pytest.mark.parametrize("current", ["default", "side"])
def test_handle_of_the_default_stream(monkeypatch, current):
    # 0 is the default stream, also where another one is current: each call enqueues there
    t = g13._t()
    x = torch.randn(20, 128, device="cuda")
    w = g13.fp4_quantize(torch.randn(40, 128, device="cuda"), "nvfp4")
    g = torch.Generator(device="cuda").manual_seed(1)
    moe = [torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((4, 64), (6, 64), (6, 32, 64), (6, 64, 16))]
    want = (g13.fp4_matmul(g13.fp4_quantize(x, "nvfp4"), w), g13.moe_layer(*moe, 2))
    handle = torch.cuda.current_stream().cuda_stream
    assert handle == 0
    torch.cuda.synchronize()
    used, raw = [], t.raw_stream
    monkeypatch.setattr(t, "raw_stream", lambda i: used.append(raw(i)) or used[-1])
    with torch.cuda.stream(torch.cuda.default_stream() if current == "default" else torch.cuda.Stream()):
        q = g13.fp4_quantize(x, "nvfp4", stream=handle)
        y = g13.fp4_matmul(q, w, stream=handle)
        v = g13.fp4_dequantize(q, stream=handle)
        m = g13.moe_layer(*moe, 2, stream=handle)
    torch.cuda.synchronize()
    assert used == [0] * 4
    assert torch.equal(y, want[0]) and torch.equal(m, want[1]) and torch.equal(v, g13.fp4_dequantize(q))
