"""CPU tests of the plans that matmul, fp4_matmul and moe_layer keep, with stand-ins for the library's calls."""
import contextlib
from types import SimpleNamespace

import pytest

import dense_gemm_13_gb300 as g13

KEPT = {"_plans": "gemm_plan_status", "_fp4_plans": "gemm_fp4_status", "_moe_plans": "gemm_moe_status"}


@pytest.mark.parametrize("which", list(KEPT))
def test_a_timeout_of_any_kept_plan_is_told(monkeypatch, which):
    pytest.importorskip("torch")
    on = []  # the device that is current when a plan's status is read: the status synchronises that one
    monkeypatch.setattr(g13._t(), "torch", SimpleNamespace(cuda=SimpleNamespace(
        device=lambda i: on.append(i) or contextlib.nullcontext())))
    for plans, status in KEPT.items():
        monkeypatch.setattr(g13, plans, {("shape", n, 3): (plans, n) for n in range(2)})
        monkeypatch.setattr(g13, status, lambda plan: 0)
    assert g13.gemm_kept_status() == 0 and on == [3] * 6
    monkeypatch.setattr(g13, KEPT[which], lambda plan: -5 if plan == (which, 1) else 0)
    assert g13.gemm_kept_status() == -5


def test_no_plans(monkeypatch):
    for plans in KEPT:
        monkeypatch.setattr(g13, plans, {})
    assert g13.gemm_kept_status() == 0
