"""The plans that fp4_matmul and moe_layer keep: a wait that runs out is told."""
import pytest
import torch

import dense_gemm_13_gb300 as g13

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_gemm_13_gb300 import _build
    _build.build()
    g13.load()


def moe_inputs():
    g = torch.Generator(device="cuda").manual_seed(3)
    return [torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((3, 72), (5, 72), (5, 48, 72), (5, 72, 24))]


def test_moe_layer_that_timed_out(monkeypatch):
    moe = moe_inputs()
    monkeypatch.setattr(g13, "_moe_plans", {})
    want = g13.moe_layer(*moe, 2)
    assert g13.gemm_kept_status() == 0
    make = g13.gemm_moe_plan
    monkeypatch.setattr(g13, "_moe_plans", {})
    monkeypatch.setattr(g13, "gemm_moe_plan",
                        lambda *a, **k: make(*a, **k, flags=g13.FLAG_TEST_STALL, timeout_ms=50))
    g13.moe_layer(*moe, 2)
    assert g13.gemm_kept_status() == -5
    monkeypatch.undo()
    assert torch.equal(g13.moe_layer(*moe, 2), want)


def test_fp4_matmul_that_timed_out(monkeypatch):
    A, B = (g13.fp4_quantize(torch.randn(n, 96, device="cuda"), "mxfp4") for n in (6, 40))
    monkeypatch.setattr(g13, "_fp4_plans", {})
    want = g13.fp4_matmul(A, B)
    assert g13.gemm_kept_status() == 0
    make = g13.gemm_fp4_plan

    def stalled(format, M, N, K, ldc, ep):
        ep.flags, ep.timeout_ms = g13.FLAG_TEST_STALL, 50
        return make(format, M, N, K, ldc, ep)

    monkeypatch.setattr(g13, "_fp4_plans", {})
    monkeypatch.setattr(g13, "gemm_fp4_plan", stalled)
    g13.fp4_matmul(A, B)
    assert g13.gemm_kept_status() == -5
    monkeypatch.undo()
    assert torch.equal(g13.fp4_matmul(A, B), want)
