"""GELU in the epilogue of the 4-bit product: a grid of values goes in through the bias, the product is zero.

The bound follows the computation max(y, 0) - z Q(z), z = |y|, Q(z) = erfc(z / sqrt 2) / 2, with u = 2^-24.
z Q(z) is off, relative to itself, by: the fit of the tail's polynomial with rounded coefficients 2.5 u, its steps 3.1 u,
the argument 1 / (1 + c z) by (1 + 2) u with a sensitivity of 2.66, its product with that 1 u, the exponential by 4 u
and its exponent by three roundings of 0.5 z^2, a further product 1 u: (20 + 1.5 z^2) u in all.
The subtraction rounds its result (u), the output's cast by half a step of its type; below 2^-120 results are flushed.
"""
import numpy as np
import pytest
import torch
from scipy.special import erfc

import dense_gemm_13_gb300 as g13

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_gemm_13_gb300 import _build
    _build.build()
    g13.load()


def zeros(rows, cols, fmt):
    return g13.fp4_quantize(torch.zeros(rows, cols, device="cuda"), fmt)


@pytest.mark.parametrize("out", list(DT))
# one row, K cut over a cluster; rows of two tiles; CTA pairs
@pytest.mark.parametrize("M,N,K", [(1, 300001, 64), (1, 2000, 4096), (200, 3001, 64), (600, 20001, 2048)])
def test_gelu_on_a_grid(out, M, N, K):
    if M == 600:
        assert g13.gemm_fp4_select_config(M, N, K).bn == 256
    y = np.linspace(-8, 8, N).astype(np.float32)
    y[: N // 8] = -np.geomspace(1e-6, 12, N // 8)
    got = g13.fp4_matmul(zeros(M, K, "mxfp4"), zeros(N, K, "mxfp4"), bias=torch.from_numpy(y).cuda(), act="gelu",
                         out_dtype=out)
    assert torch.equal(got, got[:1].expand(M, N))
    y = y.astype(np.float64)
    z, u = np.abs(y), 2.0 ** -24
    tail = z * erfc(z / np.sqrt(2)) / 2
    want = np.maximum(y, 0) - tail
    tol = u * np.abs(want) + (20 + 1.5 * z * z) * u * tail + 2.0 ** -120
    f = torch.finfo(DT[out])
    tol += f.eps / 2 * (np.abs(want) + tol) + (f.smallest_normal * f.eps / 2 if out == "f16" else 0)
    err = np.abs(got[0].double().cpu().numpy() - want)
    assert (err <= tol).all(), f"max err/tol {np.max(err / tol):.3g} at {y[np.argmax(err / tol)]}"


def test_gelu_of_extremes():
    y = torch.tensor([float("inf"), float("-inf"), float("nan"), 0.0, -0.0, 3e38, -3e38, 1e-38, -1e-38, 40.0, -40.0])
    N = y.numel()
    got = g13.fp4_matmul(zeros(3, 32, "nvfp4"), zeros(N, 32, "nvfp4"), bias=y.cuda(), act="gelu").cpu()
    want = torch.tensor([float("inf"), 0.0, float("nan"), 0.0, 0.0, 3e38, 0.0, 0.5e-38, -0.5e-38, 40.0, 0.0])
    assert torch.equal(got.isnan(), want.isnan().expand(3, N))
    assert torch.allclose(got, want.expand(3, N), rtol=2.0 ** -22, atol=2.0 ** -126, equal_nan=True)
