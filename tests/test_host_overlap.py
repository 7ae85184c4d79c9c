"""CPU tests of the overlap refusals: the calls run as far as the library on CPU tensors that say they are on device 0."""
import pytest

import dense_gemm_13_gb300 as g13
from dense_gemm_13_gb300 import _build

torch = pytest.importorskip("torch")
INVALID = -1


class On0(torch.Tensor):
    def get_device(self):
        return 0


def on0(t):
    return t.as_subclass(On0)


@pytest.fixture
def called(monkeypatch):
    """Device 0 is the current one; what gets past the checks is counted instead of called."""
    _build.build()
    L, calls = g13.load(), []
    monkeypatch.setattr(g13._t(), "device_index", lambda: 0)
    monkeypatch.setattr(g13._t(), "raw_stream", lambda i: 0)
    monkeypatch.setattr(L, "gemm_w4_run", lambda *a: calls.append(a) or 0)
    return calls


def refused(call):
    with pytest.raises(g13.GemmError) as e:
        call()
    assert e.value.status == INVALID and "overlap" in str(e.value)


@pytest.mark.parametrize("which", ["x", "bias", "residual", "codes", "scales", "zeros"])
def test_w4_matmul_out_overlaps_no_input(called, which):
    M, N, K = 3, 32, 64
    pool = on0(torch.zeros(1 << 16, dtype=torch.uint8))
    at = 0

    def take(shape, dtype):
        nonlocal at
        n = torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()
        t = pool[at: at + n].view(dtype).view(shape)
        at += (n + 255) // 256 * 256
        return t
    a = dict(x=take((M, K), torch.bfloat16), bias=take((N,), torch.float32), residual=take((M, N), torch.float32),
             codes=take((2 * 512,), torch.uint8), scales=take((32,), torch.bfloat16), zeros=take((32,), torch.uint8))
    W = g13.W4Tensor(a["codes"], a["scales"], a["zeros"], N, K)
    call = lambda out: g13.w4_matmul(a["x"], W, bias=a["bias"], residual=a["residual"], out=out)  # noqa: E731
    free = take((M, N), torch.bfloat16)
    assert call(free) is free and len(called) == 1
    # an output of which only a first or last byte lies in the array
    start = a[which].data_ptr() - pool.data_ptr()
    end = start + a[which].numel() * a[which].element_size()
    for first in (start - 2 * M * N + 2, end - 2):
        if first >= 0:
            refused(lambda: call(pool[first: first + 2 * M * N].view(torch.bfloat16).view(M, N)))
    assert len(called) == 1
