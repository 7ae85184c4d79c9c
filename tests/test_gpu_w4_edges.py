"""4-bit weights on the GPU where values leave the ordinary range: NaN and infinities behind an activation, GELU's
left tail, activations near the top of BF16's range.  The bound of a product is that of test_gpu_w4.py."""
import numpy as np
import pytest
import torch

import dense_gemm_13_gb300 as g13
from tests import blocks_ref as ref
from tests.test_gpu_w4 import DT, check_product, rng, weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_gemm_13_gb300 import _build
    _build.build()
    g13.load()


def rows_of(x, aligned):
    """x with rows on 16 bytes, or off them."""
    M, K = x.shape
    big = torch.zeros((M, K // 8 * 8 + 24), dtype=x.dtype, device="cuda")
    rows = big[:, :K] if aligned else big[:, 1: 1 + K]
    rows.copy_(x)
    return rows


# one row, 2 to 16 (mma.sync), 17 to 64 (tcgen05, and mma.sync where rows are off 16 bytes)
@pytest.mark.parametrize("M", [1, 5, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_activations_keep_a_nan(M, aligned, dtype):
    N, K = 150, 600
    r = rng("nan act", M, dtype)
    W = weight(r, N, K, 64, dtype)[0]
    x = torch.from_numpy(r.standard_normal((M, K)).astype(np.float32)).to(DT[dtype])
    x[0, 7] = float("nan")
    if M > 4:
        x[2, 99], x[4, 599] = float("inf"), float("-inf")
    x = rows_of(x, aligned)
    bias = torch.zeros(N, device="cuda")
    bias[3] = float("nan")
    R = torch.zeros(M, N, device="cuda")
    R[-1, 5] = float("nan")
    for out in DT:
        plain = g13.w4_matmul(x, W, bias=bias, out_dtype=out)
        assert bool(plain[0].isnan().all()) and bool(plain[:, 3].isnan().all())
        if M > 4:
            assert not bool(torch.isfinite(plain[[2, 4]]).any())
        relu = g13.w4_matmul(x, W, bias=bias, act="relu", out_dtype=out)
        # (rounding keeps signs, so ReLU may come after it)
        assert torch.equal(relu.nan_to_num(7, 8, 9), plain.clamp(min=0).nan_to_num(7, 8, 9))
        gelu = g13.w4_matmul(x, W, bias=bias, act="gelu", out_dtype=out)
        finite = torch.isfinite(plain)
        assert bool(gelu[plain.isnan()].isnan().all()) and bool(torch.isfinite(gelu[finite]).all())
        assert bool((gelu[plain == float("inf")] == float("inf")).all())
        last = g13.w4_matmul(x, W, act="relu", residual=R, out_dtype=out)
        assert bool(last[-1, 5].isnan()) and bool(last[0].isnan().all())


@pytest.mark.parametrize("M", [1, 16, 17, 64])
@pytest.mark.parametrize("out", list(DT))
def test_gelu_keeps_its_digits(M, out):
    # a grid of values through the bias, the product zero; the bound is that of test_gpu_fp4_gelu.py, whose GELU this is
    from scipy.special import erfc
    N = 20001
    y = np.linspace(-8, 8, N).astype(np.float32)
    y[: N // 4] = -np.geomspace(1e-6, 12, N // 4)
    W = weight(rng("gelu"), N, 64, 64, "bf16")[0]
    x = torch.zeros(M, 64, dtype=torch.bfloat16, device="cuda")
    got = g13.w4_matmul(x, W, bias=torch.from_numpy(y).cuda(), act="gelu", out_dtype=out)
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
    ends = torch.tensor([float("inf"), float("-inf"), float("nan"), 0.0, 3e38, -3e38, 40.0, -40.0])
    got = g13.w4_matmul(x, weight(rng("ends"), 8, 64, 64, "bf16")[0], bias=ends.cuda(), act="gelu", out_dtype="f32").cpu()
    want = torch.tensor([float("inf"), 0.0, float("nan"), 0.0, 3e38, 0.0, 40.0, 0.0])
    assert torch.allclose(got, want.expand(M, 8), rtol=2.0 ** -22, atol=2.0 ** -126, equal_nan=True)


def given(q, s, z, group, dtype="bf16"):
    """A weight of these codes, scales and zeros, as test_gpu_w4.weight gives it."""
    s = torch.from_numpy(s.astype(np.float32)).to(DT[dtype])
    W = g13.w4_pack(torch.from_numpy(q).cuda(), s.cuda(), None if z is None else torch.from_numpy(z).cuda(), group)
    s64 = s.double().numpy()
    z64 = np.full(s64.shape, 8.0) if z is None else z
    return W, (ref.w4_values(q, s64, z, group), ref.w4_values(q, s64, -z64.astype(float), group))


@pytest.mark.parametrize("M", [1, 7, 16])
@pytest.mark.parametrize("group", [32, 64, 128, 192])
@pytest.mark.parametrize("aligned", [True, False])
def test_activations_near_the_top_of_the_range(M, group, aligned):
    # neighbours whose plain sum is beyond FP32, under scales that bring the products back
    N, K = 100, 700
    r = rng("top", M, group)
    G = -(-K // group)
    q = r.integers(0, 16, (N, K)).astype(np.uint8)
    s = 2.0 ** -20 * (1 + r.random((N, G)))
    x = r.standard_normal((M, K)).astype(np.float32) * 1e37
    x[:, 5:9] = 3.0e38
    x[-1] = -np.abs(x[-1])
    x = rows_of(torch.from_numpy(x).bfloat16(), aligned)
    for z in (None, np.zeros((N, G), np.uint8), r.integers(0, 16, (N, G)).astype(np.uint8)):
        W, w = given(q, s, z, group)
        check_product(g13.w4_matmul(x, W, out_dtype="f32"), x, w, "f32")


@pytest.mark.parametrize("M", [1, 7, 16])
@pytest.mark.parametrize("group", [32, 64, 96])
def test_a_large_scale_beside_large_activations(M, group):
    # 128 columns with a group of large activations and small scales, and one of small activations and scales
    # above one: the product of the largest activation and the largest scale is beyond FP32, no result is
    N, K = 50, 384
    r = rng("beside", M, group)
    G = -(-K // group)
    q = r.integers(0, 16, (N, K)).astype(np.uint8)
    z = r.integers(1, 16, (N, G)).astype(np.uint8)
    s, x = np.full((N, G), 2.0 ** -40), np.full((M, K), 2.0 ** 126)
    s[:, 1::2] = 2.0 ** r.integers(3, 20, (N, G // 2))
    for c in range(1, G, 2):
        x[:, c * group: (c + 1) * group] = r.standard_normal((M, len(range(c * group, min(K, (c + 1) * group)))))
    x *= np.where(r.random((M, K)) < 0.5, -1, 1)
    W, w = given(q, s, z, group)
    x = torch.from_numpy(x.astype(np.float32)).bfloat16().cuda()
    check_product(g13.w4_matmul(x, W, out_dtype="f32"), x, w, "f32")
    # weights of zero under a large scale, on large activations
    q[:] = np.repeat(z, group, 1)[:, :K]
    W, w = given(q, np.full((N, G), 64.0), z, group)
    x = torch.full((M, K), 3e38, device="cuda").bfloat16()
    y = g13.w4_matmul(x, W, out_dtype="f32")
    assert bool(torch.isfinite(y).all())
    check_product(y, x, w, "f32")


@pytest.mark.parametrize("M", [1, 5, 16, 17, 64])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_fp32_results_are_as_exact_as_fp32_sums(M, dtype):
    # With u = 2^-24: an FP32 sum over n = K / 128 groups of random signs, each addition off by u / sqrt(3) of a partial
    # sum that grows like a random walk, is off by u sqrt(n / 6), 3.3 u at K = 8192; a group's own sum, the scale and the
    # joins are allowed 1.2 u more.
    N = 1024
    for K in (512, 4096, 8192):
        for group in (32, 64, 128, 256):
            for zeros in (True, False):
                r = rng("exact", M, K, group, zeros)
                W, _, _, _, (w, _) = weight(r, N, K, group, dtype, zeros)
                x = torch.from_numpy(r.standard_normal((M, K)).astype(np.float32)).to(DT[dtype])
                want = x.double().numpy() @ w.T
                got = g13.w4_matmul(x.cuda(), W, out_dtype="f32").double().cpu().numpy()
                off = np.linalg.norm(got - want) / np.linalg.norm(want)
                assert off <= ((K / 128 / 6) ** 0.5 + 1.2) * 2.0 ** -24, (K, group, zeros, off)
