"""The plans that fp4_matmul and moe_layer keep: a wait that runs out is told."""
import threading
import time

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


@pytest.mark.parametrize("call", ["matmul", "fp4_matmul", "moe_layer"])
def test_first_calls_of_two_threads_make_one_plan(monkeypatch, call):
    A, B = (torch.randn(n, 88, device="cuda").bfloat16() for n in (5, 48))
    run, kept, maker = {
        "matmul": (lambda: g13.matmul(A, B, b_layout="nk"), "_plans", "gemm_plan"),
        "fp4_matmul": (lambda: g13.fp4_matmul(g13.fp4_quantize(A), g13.fp4_quantize(B)), "_fp4_plans", "gemm_fp4_plan"),
        "moe_layer": (lambda m=moe_inputs(): g13.moe_layer(*m, 2), "_moe_plans", "gemm_moe_plan")}[call]
    want = run()
    torch.cuda.synchronize()
    make, made, got = getattr(g13, maker), [], []

    def slowly(*a, **k):
        made.append(1)
        time.sleep(0.2)
        return make(*a, **k)

    def work():
        got.append(run())
        torch.cuda.synchronize()

    monkeypatch.setattr(g13, kept, {})
    monkeypatch.setattr(g13, maker, slowly)
    both = [threading.Thread(target=work) for _ in range(2)]
    for t in both:
        t.start()
    for t in both:
        t.join()
    assert len(made) == 1 and len(got) == 2 and all(torch.equal(y, want) for y in got)
