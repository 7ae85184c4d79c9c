"""A wait that runs out in the 4-bit-weight product, without faulting the GPU.

With GEMM_FLAG_TEST_STALL the first CTA issues no tensor-core product, so its producers wait for stages that are never
freed and its sums for products that never come.  With a 50 ms limit each wait gives up, the CTA's copies land, it frees its TMEM
and stores NaN; the call has no status, so that has to show with every activation.
The other tiles are as ever, and so is the next call.
"""
import ctypes

import pytest
import torch

import dense_gemm_13_gb300 as g13
from dense_gemm_13_gb300 import blocks
from tests.test_gpu_w4 import DT, rng, weight

pytestmark = pytest.mark.gpu
TYPE = {"f32": 0, "f16": 1, "bf16": 2}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_gemm_13_gb300 import _build
    _build.build()
    g13.load()


def run(x, W, out, act, R, flags):
    M, K = x.shape
    y = torch.full((M, W.rows), 7.0, dtype=DT[out], device="cuda")
    L, d = g13.load(), blocks._W4Desc()
    L.gemm_w4_desc_init(ctypes.byref(d))
    d.dtype, d.out_dtype, d.M, d.N, d.K, d.group = TYPE[W.dtype], TYPE[out], M, W.rows, K, W.group
    d.has_zeros, d.act, d.has_residual, d.flags, d.timeout_ms = 1, g13.ACTS[act], R is not None, flags, 50
    rc = L.gemm_w4_run(ctypes.byref(d), x.data_ptr(), W.codes.data_ptr(), W.scales.data_ptr(), W.zeros.data_ptr(),
                       y.data_ptr(), None, None if R is None else R.data_ptr(), 1.0, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    return y


# both numbers of tokens that a tile has; one step, fewer than the ring holds, more; K on one CTA and on a cluster
@pytest.mark.parametrize("M", [20, 64])
@pytest.mark.parametrize("N,K", [(300, 128), (300, 256), (300, 8192), (30000, 2048)])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_wait_that_runs_out_gives_nan(M, N, K, group, dtype):
    r = rng("stall", M, N, K)
    W = weight(r, N, K, group, dtype)[0]
    x = torch.randn(M, K, device="cuda").to(DT[dtype])
    R = torch.randn(M, N, device="cuda")
    for out, act, res in (("f32", "none", None), ("bf16", "relu", None), ("f16", "relu", R), ("f32", "gelu", None)):
        want = run(x, W, out, act, res, 0)
        assert bool(torch.isfinite(want).all())
        got = run(x, W, out, act, res, g13.FLAG_TEST_STALL)
        assert bool(got[:, :128].isnan().all())
        assert torch.equal(got[:, 128:], want[:, 128:])
        assert torch.equal(run(x, W, out, act, res, 0), want)
