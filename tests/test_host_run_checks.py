"""CPU tests of gemm_fp4_run and gemm_moe_run: tensors that the GPU must not be given are refused first."""
from types import SimpleNamespace

import pytest

import dense_gemm_13_gb300 as g13
from dense_gemm_13_gb300 import _build

BAD_PLAN = -6  # what the library says to a call that got past the checks: no plan is made here


class Tensor:
    def __init__(self, device, nbytes=1 << 20):
        self.device, self.nbytes = device, nbytes

    def get_device(self):
        return self.device

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        return self.nbytes // 2

    def element_size(self):
        return 2


@pytest.fixture
def current(monkeypatch):
    """Device 1 is the current one."""
    pytest.importorskip("torch")
    _build.build()
    monkeypatch.setattr(g13._t(), "device_index", lambda: 1)
    monkeypatch.setattr(g13._t(), "raw_stream", lambda i: 0)


def fp4(index, rows):
    q = g13.Fp4Tensor.__new__(g13.Fp4Tensor)
    q._codes, q._scales, q._both, q._g = Tensor(index), Tensor(index), None, None
    q._rows, q._cols, q._format, q._index = rows, 64, "nvfp4", index
    return q


@pytest.mark.parametrize("bad", ["A", "B", "C", "bias", "residual"])
@pytest.mark.parametrize("device", [0, -1])
def test_fp4_run_off_the_current_device(current, bad, device):
    plan = SimpleNamespace(handle=None, M=2, N=3, K=64, format="nvfp4")
    args = dict(A=fp4(1, 2), B=fp4(1, 3), C=Tensor(1), bias=Tensor(1), residual=Tensor(1))
    with pytest.raises(g13.GemmError) as e:
        g13.gemm_fp4_run(plan, **args)
    assert e.value.status == BAD_PLAN
    args[bad] = fp4(device, args[bad]._rows) if bad in "AB" else Tensor(device)
    with pytest.raises(g13.GemmError, match="current device"):
        g13.gemm_fp4_run(plan, **args)


NAMES = ["X", "router", "W1", "W2", "Y", "workspace", "expert_ids", "expert_weights"]


@pytest.mark.parametrize("bad", NAMES)
def test_moe_run_off_the_current_device(current, bad):
    plan = SimpleNamespace(handle=None, workspace_bytes=4096)
    args = {n: Tensor(1) for n in NAMES}
    with pytest.raises(g13.GemmError) as e:
        g13.gemm_moe_run(plan, **args)
    assert e.value.status == BAD_PLAN
    for device in (0, -1):
        with pytest.raises(g13.GemmError, match="current device"):
            g13.gemm_moe_run(plan, **dict(args, **{bad: Tensor(device)}))


def test_moe_run_short_workspace(current):
    plan = SimpleNamespace(handle=None, workspace_bytes=4096)
    args = {n: Tensor(1) for n in NAMES}
    for nbytes, short in ((4096, False), (4094, True), (0, True)):
        with pytest.raises(g13.GemmError) as e:
            g13.gemm_moe_run(plan, **dict(args, workspace=Tensor(1, nbytes)))
        assert (e.value.status == BAD_PLAN) is not short
        assert ("4096 bytes" in str(e.value)) is short
    with pytest.raises(g13.GemmError) as e:  # an address is taken as it is
        g13.gemm_moe_run(plan, **dict(args, workspace=1 << 20))
    assert e.value.status == BAD_PLAN


def test_objects_that_only_have_an_address(current):
    # taken as they are, like an address
    thing = SimpleNamespace(data_ptr=lambda: 1 << 20)
    with pytest.raises(g13.GemmError) as e:
        g13.gemm_fp4_run(SimpleNamespace(handle=None, M=2, N=3, K=64, format="nvfp4"), fp4(1, 2), fp4(1, 3), thing, thing)
    assert e.value.status == BAD_PLAN
    with pytest.raises(g13.GemmError) as e:
        g13.gemm_moe_run(SimpleNamespace(handle=None, workspace_bytes=4096), **{n: thing for n in NAMES})
    assert e.value.status == BAD_PLAN
