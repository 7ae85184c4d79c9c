"""CPU tests of the overlap refusals: the calls run as far as the library on CPU tensors that say they are on device 0."""
import pytest

import dense_gemm_13_gb300 as g13
from dense_gemm_13_gb300 import _build, blocks

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
    for name in ("gemm_w4_run", "gemm_moe_run_routed"):
        monkeypatch.setattr(L, name, lambda *a: calls.append(a) or 0)
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


@pytest.mark.parametrize("which", ["x", "w1", "w2", "ids", "weights"])
def test_moe_experts_out_overlaps_no_input(called, monkeypatch, which):
    T, E, k, H, I = 3, 4, 2, 32, 16
    monkeypatch.setattr(blocks, "_no_capture", lambda *a: None)
    monkeypatch.setattr(blocks, "_keep", lambda plans, key, make: type("P", (), dict(workspace_bytes=256, handle=0)))
    pool = on0(torch.zeros(1 << 16, dtype=torch.uint8))
    at = 0

    def take(shape, dtype):
        nonlocal at
        n = torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()
        t = pool[at: at + n].view(dtype).view(shape)
        at += (n + 255) // 256 * 256
        return t
    bf = torch.bfloat16
    a = dict(x=take((T, H), bf), w1=take((E, 2 * I, H), bf), w2=take((E, H, I), bf), ids=take((T, k), torch.int32),
             weights=take((T, k), torch.float32))
    call = lambda out: g13.moe_experts(a["x"], a["w1"], a["w2"], a["ids"], a["weights"], out=out)  # noqa: E731
    free = take((T, H), bf)
    assert call(free) is free and len(called) == 1
    start = a[which].data_ptr() - pool.data_ptr()
    end = start + a[which].numel() * a[which].element_size()
    for first in (start - 2 * T * H + 2, end - 2):
        if first >= 0:
            refused(lambda: call(pool[first: first + 2 * T * H].view(bf).view(T, H)))
    assert len(called) == 1


def views(r, pool):
    """Rows of a random stride, in one of a few types, somewhere in the pool."""
    t = pool.view((torch.uint8, torch.bfloat16, torch.float32)[r.integers(3)])
    rows, cols = int(r.integers(1, 5)), int(r.integers(1, 7))
    ld = int(r.choice([cols, cols + 1, 8, 12])) if r.random() < 0.9 else cols + int(r.integers(0, 9))
    ld = max(ld, cols)
    left = t.numel() - (rows - 1) * ld - cols
    return None if left < 0 else t.as_strided((rows, cols), (ld, 1), int(r.integers(0, left + 1)))


def own_bytes(x, pool):
    size, first = x.element_size(), x.data_ptr() - pool.data_ptr()
    return {first + (i * x.stride(0) + j) * size + b for i in range(x.shape[0]) for j in range(x.shape[1]) for b in range(size)}


def test_bytes_overlap_against_the_bytes_themselves():
    np = pytest.importorskip("numpy")
    r, pool = np.random.default_rng(5), torch.zeros(256, dtype=torch.uint8)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        a, b = views(r, pool), views(r, pool)
        if a is None or b is None:
            continue
        want, got = bool(own_bytes(a, pool) & own_bytes(b, pool)), blocks._bytes_overlap(a, b)
        assert got == blocks._bytes_overlap(b, a)
        gaps = [x.stride(0) * x.element_size() for x in (a, b) if x.shape[0] > 1 and x.stride(0) > x.shape[1]]
        if len(set(gaps)) <= 1:
            assert got == want, (a.shape, a.stride(), a.dtype, b.shape, b.stride(), b.dtype, b.data_ptr() - a.data_ptr())
            seen[want] += 1
        else:
            assert got or not want
    assert min(seen.values()) > 300


def test_columns_of_one_buffer_do_not_overlap():
    buf = torch.zeros(4, 96, dtype=torch.bfloat16)
    q, k, v = buf[:, :32], buf[:, 32:64], buf[:, 64:]
    w = torch.ones(32, dtype=torch.bfloat16)
    blocks._check_norm_overlap("rms_norm", q, w, k, k, v)
    blocks._check_norm_overlap("rms_norm", q, buf[2, 40:72], None, None, v[:, 8:])
    for out in (buf[:, 31:63], buf[:, 1:33], buf[1:, :32]):
        with pytest.raises(g13.GemmError):
            blocks._check_norm_overlap("rms_norm", q, w, None, None, out)
    with pytest.raises(g13.GemmError):
        blocks._check_norm_overlap("rms_norm", q, buf[2, 40:72], None, None, k)


def test_w4_matmul_into_the_columns_beside_x(called):
    buf = on0(torch.zeros(5, 64 + 32, dtype=torch.bfloat16))
    W = g13.W4Tensor(*(on0(t) for t in (torch.zeros(1024, dtype=torch.uint8), torch.zeros(32, dtype=torch.bfloat16),
                                        torch.zeros(32, dtype=torch.uint8))), 32, 64)
    g13.w4_matmul(buf[:, :64], W, out=buf[:, 64:])
    assert len(called) == 1
    refused(lambda: g13.w4_matmul(buf[:, :64], W, out=buf[:, 63:95]))


def test_moe_experts_into_the_columns_beside_x(called, monkeypatch):
    monkeypatch.setattr(blocks, "_no_capture", lambda *a: None)
    monkeypatch.setattr(blocks, "_keep", lambda plans, key, make: type("P", (), dict(workspace_bytes=256, handle=0)))
    buf, bf = on0(torch.zeros(3, 64, dtype=torch.bfloat16)), torch.bfloat16
    w1, w2 = on0(torch.zeros(4, 32, 32, dtype=bf)), on0(torch.zeros(4, 32, 16, dtype=bf))
    ids, weights = on0(torch.zeros(3, 2, dtype=torch.int32)), on0(torch.zeros(3, 2))
    g13.moe_experts(buf[:, :32], w1, w2, ids, weights, out=buf[:, 32:])
    assert len(called) == 1
    refused(lambda: g13.moe_experts(buf[:, :32], w1, w2, ids, weights, out=buf[:, 31:63]))
