"""Inputs and outputs that are column ranges of one buffer; bounds as in test_gpu_norm.py and test_gpu_w4.py (where rows
begin decides how sums are cut, so bits may differ from those of tensors of their own)."""
import pytest
import torch

import dense_gemm_13_gb300 as g13
from tests.test_gpu_norm import check_values, stream_of
from tests.test_gpu_w4 import check_product, rng, weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_gemm_13_gb300 import _build
    _build.build()
    g13.load()


@pytest.mark.parametrize("H", [8, 64, 100, 333, 1024, 2049, 4097, 17000])
@pytest.mark.parametrize("gap", [0, 1, 8])
def test_norm_of_columns(H, gap):
    T = 300
    buf = torch.randn(T, 4 * (H + gap), device="cuda").bfloat16()
    part = [buf[:, i * (H + gap): i * (H + gap) + H] for i in range(4)]
    w = torch.randn(H, device="cuda").bfloat16()
    x, r = part[0].clone(), part[2].clone()
    before = buf.clone()
    h, h64 = stream_of(x, r)
    g13.rms_norm(part[0], w, residual=part[2], out=part[1], residual_out=part[3])
    assert torch.equal(part[3], h)
    check_values(part[1], h64, w, 1e-6, 0.0, "bf16")
    part[1].copy_(before[:, H + gap: 2 * H + gap])
    part[3].copy_(before[:, 3 * (H + gap): 3 * (H + gap) + H])
    assert torch.equal(buf, before)


@pytest.mark.parametrize("M,K,N", [(1, 64, 32), (5, 100, 40), (16, 512, 96), (40, 256, 300), (40, 333, 77)])
def test_w4_matmul_into_columns(M, K, N):
    W, _, _, _, w = weight(rng("columns", M, K, N), N, K, 64, "bf16")
    buf = torch.randn(M, K + N + 3, device="cuda").bfloat16()
    x = buf[:, :K].clone()
    out = buf[:, K: K + N]
    behind = buf[:, K + N:].clone()
    g13.w4_matmul(buf[:, :K], W, out=out)
    check_product(out, x, w, "bf16")
    assert torch.equal(buf[:, :K], x) and torch.equal(buf[:, K + N:], behind)
