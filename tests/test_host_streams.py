"""CPU tests of the `stream` argument: which stream a handle stands for."""
from types import SimpleNamespace

import pytest

import dense_gemm_13_gb300 as g13


@pytest.fixture
def torch_of(monkeypatch):
    """The library's view of torch, with a stand-in for torch.cuda that notes how each stream is made."""
    pytest.importorskip("torch")
    cuda = SimpleNamespace(
        ExternalStream=lambda handle, device: ("pool" if handle == 0 else "external", handle, device),
        default_stream=lambda device: ("default", device),
        stream=lambda s: s)
    t = g13._t()
    monkeypatch.setattr(t, "torch", SimpleNamespace(cuda=cuda))
    return t


@pytest.mark.parametrize("handle", [0, 1])
def test_the_default_streams_handle(torch_of, handle):
    # torch takes a stream pointer of 0 as none given and hands out a stream of its pool
    assert torch_of.on(handle, 3) == ("default", 3)


def test_other_handles_and_streams(torch_of):
    assert torch_of.on(0x7F0012340000, 1) == ("external", 0x7F0012340000, 1)
    s = SimpleNamespace(device=SimpleNamespace(index=1))
    assert torch_of.on(s, 1) is s
    with pytest.raises(g13.GemmError, match="another device"):
        torch_of.on(s, 0)
