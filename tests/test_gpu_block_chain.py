"""A decoder block's linear parts as they are used together: norm, 8-bit or 4-bit products, routing, experts; eagerly and as
one captured graph."""
import numpy as np
import pytest
import torch

import dense_gemm_13_gb300 as g13
from tests import blocks_ref as ref
from tests import test_gpu_fp8 as fp8
from tests import test_gpu_norm as norm
from tests import test_gpu_route as routes
from tests import test_gpu_w4 as w4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_gemm_13_gb300 import _build
    _build.build()
    g13.load()


def randn(seed, *shape, std=1.0):
    return torch.randn(*shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)) * std


def test_prompt_in_8_bits():
    # norm -> 8-bit product with bias and GELU -> 8-bit product added to the FP32 stream
    T, H, F = 300, 520, 1000
    x, r, g = randn(1, T, H).bfloat16(), randn(2, T, H, std=3.0), (1 + 0.1 * randn(3, H)).bfloat16()
    up, down, bias = g13.fp8_quantize(randn(4, F, H, std=H ** -0.5)), g13.fp8_quantize(randn(5, H, F, std=F ** -0.5)), randn(6, F)
    a, h = g13.rms_norm(x, g, residual=r, out_dtype="mxfp8")
    want, h64 = norm.stream_of(x, r)
    assert torch.equal(h, want)
    norm.check_fp8(a, h64, g, 1e-6, 0.0)
    y = g13.fp8_matmul(a, up, bias=bias, act="gelu", out_dtype="bf16")
    fp8.check_product(y, *(g13.fp8_dequantize(t).double().cpu().numpy() for t in (a, up)), "bf16", bias.double().cpu().numpy(), "gelu")
    b = g13.fp8_quantize(y)
    fp8.check_quantised(b, y.float().cpu().numpy())
    z = g13.fp8_matmul(b, down, residual=h)
    fp8.check_product(z, *(g13.fp8_dequantize(t).double().cpu().numpy() for t in (b, down)), "f32", R=h.double().cpu().numpy())


@pytest.mark.parametrize("T", [1, 6, 40])
def test_tokens_through_4_bit_weights_and_experts(T):
    # norm -> 4-bit product -> norm -> logits -> routing -> experts
    H, E, I, k = 512, 24, 64, 4
    x, r, g = randn(1, T, H).bfloat16(), randn(2, T, H).bfloat16(), (1 + 0.1 * randn(3, H)).bfloat16()
    W = g13.w4_quantize(randn(4, H, H, std=H ** -0.5), 64)
    router = randn(5, E, H, std=H ** -0.5)
    w1, w2 = randn(6, E, 2 * I, H, std=H ** -0.5).bfloat16(), randn(7, E, H, I, std=I ** -0.5).bfloat16()
    balance = randn(8, E, std=0.1)
    kw = dict(scores="sigmoid", bias=balance, groups=4, top_groups=2, group_score="top2", scale=2.5)

    def block(x, r):
        y, h = g13.rms_norm(x, g, residual=r)
        o = g13.w4_matmul(y, W)
        y2, h2 = g13.rms_norm(o, g, residual=h)
        z = g13.matmul(y2, router.bfloat16(), b_layout="nk")
        ids, wts = g13.route(z, k, **kw)
        return y, h, o, y2, h2, z, ids, wts, g13.moe_experts(y2, w1, w2, ids, wts)

    def check(got, x, r):
        y, h, o, y2, h2, z, ids, wts, out = got
        want, h64 = norm.stream_of(x, r)
        assert torch.equal(h, want)
        norm.check_values(y, h64, g, 1e-6, 0.0, "bf16")
        w = g13.w4_dequantize(W).double().cpu().numpy()
        w4.check_product(o, y, (w, np.abs(w) + 30 * float(W.scales.max())), "bf16")
        want, h64 = norm.stream_of(o, h)
        assert torch.equal(h2, want)
        norm.check_values(y2, h64, g, 1e-6, 0.0, "bf16")
        rid, rw = ref.route(z.double().cpu().numpy(), k, **dict(kw, bias=balance.double().cpu().numpy()))
        assert np.array_equal(ids.cpu().numpy(), rid) and np.allclose(wts.cpu().numpy(), rw, rtol=1e-5)
        routes.check_experts(out, y2, w1, w2, ids, wts, "swiglu")

    got = block(x, r)
    check(got, x, r)
    # as one graph, replayed on other tokens
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        kept = block(x, r)
    x.copy_(randn(9, T, H))
    r.copy_(randn(10, T, H))
    for _ in range(3):
        gr.replay()
    torch.cuda.synchronize()
    check(kept, x, r)
    for a, b in zip(kept, block(x, r)):
        assert torch.equal(a, b)
    assert g13.gemm_kept_status() == 0


def test_plans_that_go_during_a_capture():
    # (as the garbage collector may have it)
    x = randn(1, 8, 64).bfloat16()
    y = g13.rms_norm(x)
    plans = [g13.gemm_plan("bf16", 8, 8, 64, 64, 64, 8, g13.Epilogue(b_layout="nk")), g13.gemm_fp4_plan("mxfp4", 8, 8, 64, 8),
             g13.gemm_fp8_plan(8, 8, 64, 8), g13.gemm_moe_plan("bf16", 8, 4, 2, 64, 64, "gelu")]
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        a = g13.rms_norm(x)
        for p in plans:
            p.destroy()
        b = g13.rms_norm(a)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, y) and torch.equal(b, g13.rms_norm(y))


def test_two_streams_at_once():
    # two requests at a time, on streams of their own
    H = 640
    W8, W4 = g13.fp8_quantize(randn(1, 900, H)), g13.w4_quantize(randn(2, 900, H), 128)
    xs = [randn(i, n, H).bfloat16() for i, n in ((3, 1), (4, 30))]

    def one(x):
        a = g13.rms_norm(x, out_dtype="mxfp8")
        y = g13.rms_norm(x)
        return g13.fp8_matmul(a, W8), g13.w4_matmul(y, W4), *g13.route(g13.w4_matmul(y, W4, out_dtype="f32")[:, :256], 8)

    want = [one(x) for x in xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = one(xs[i])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for u, v in zip(a, b):
            assert torch.equal(u, v)
