"""The 4-bit product on CTA pairs (256 x 256 tiles, overlapping accumulators): three tiles a pair and more, so that
both accumulators are used again, ragged in every direction, in both formats and with every epilogue.

Each test asserts that its shape is one that the library sends to pairs.  Tolerances are those of
tests/test_gpu_fp4.py (check_product), sums of integers are exact.
"""
import numpy as np
import pytest
import torch

import dense_gemm_13_gb300 as g13
from tests import fp4_ref as ref
from tests.test_gpu_fp4 import DT, FMTS, check_product, operand, rng

pytestmark = pytest.mark.gpu
SMS = 152


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_gemm_13_gb300 import _build
    _build.build()
    g13.load()


def on_pairs(M, N, K, tiles_a_pair=3):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert sms == SMS, "the shapes are chosen for this many SMs"
    assert g13.gemm_fp4_select_config(M, N, K, sms).bn == 256
    assert -(-M // 256) * -(-N // 256) > (tiles_a_pair - 1) * (sms // 2)


# the last tiles hold 20, 188, 2, 1 and 160 tokens and 88, 20, 136, 65 and 40 weight rows: some leave a pair's second
# CTA no token, or no row, of its own
SHAPES = [(1300, 7000, 2900), (700, 14100, 3001), (2050, 5000, 2600), (257, 40001, 2700), (4000, 2600, 2305)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_pairs_exact_integers(fmt, shape):
    M, N, K = shape
    on_pairs(*shape)
    r = rng("pairs", fmt, shape)
    (A, a), (B, b) = operand(r, M, K, fmt, ints=True), operand(r, N, K, fmt, ints=True)
    assert 144 * K < 2 ** 24  # every partial sum is exact in FP32
    want = torch.from_numpy(a @ b.T)
    big = torch.full((M + 2, N + 3), 7.0, device="cuda")
    for _ in range(2):
        g13.fp4_matmul(A, B, out=big[1:-1, 1: N + 1])
        got = big[1:-1, 1: N + 1].cpu().double()
        assert torch.equal(got, want), f"{int((got != want).sum())} of {got.numel()} differ"
    big[1:-1, 1: N + 1] = 7
    assert bool((big == 7).all()), "store outside the M x N window"


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out", list(DT))
def test_pairs_epilogue(fmt, out):
    M, N, K = 1300, 7001, 2881
    on_pairs(M, N, K)
    r = rng("pairs epi", fmt, out)
    ga, gb = (None, None) if fmt == "mxfp4" else (0.0123, 0.004)
    (A, a), (B, b) = operand(r, M, K, fmt, ga), operand(r, N, K, fmt, gb)
    al = np.float32(1.0 / np.abs(a @ b.T).max())
    bias, R = r.standard_normal(N).astype(np.float32), r.standard_normal((M, N)).astype(np.float32)
    tb, tR = torch.from_numpy(bias).cuda(), torch.from_numpy(R).cuda()
    check_product(g13.fp4_matmul(A, B, alpha=al, out_dtype=out), a, b, out, alpha=float(al))
    check_product(g13.fp4_matmul(A, B, alpha=4 * al, out_dtype=out, bias=tb, act="gelu"), a, b, out, bias, "gelu",
                  alpha=4 * float(al))
    check_product(g13.fp4_matmul(A, B, alpha=al, out_dtype=out, bias=tb, act="relu", residual=tR, beta=-0.5), a, b,
                  out, bias, "relu", R, float(al), -0.5)


@pytest.mark.parametrize("fmt", FMTS)
def test_pairs_nan_scale_stays_in_its_row(fmt):
    M, N, K = 1300, 7000, 2900
    on_pairs(M, N, K)
    g = torch.Generator(device="cuda").manual_seed(5)
    x, w = (torch.randn(n, K, generator=g, device="cuda") for n in (M, N))
    x[1200, 2899] = float("inf")
    w[6999, 0] = float("nan")
    C = g13.fp4_matmul(g13.fp4_quantize(x, fmt), g13.fp4_quantize(w, fmt)).isnan()
    assert bool(C[1200].all()) and bool(C[:, 6999].all()) and int(C.sum()) == M + N - 1


@pytest.mark.parametrize("fmt", FMTS)
def test_pairs_linear_captured(fmt):
    # quantise, then multiply, as it is served: captured, replayed, and beside an eager call on another stream
    M, N, K = 2050, 5000, 2600
    on_pairs(M, N, K)
    r = rng("pairs lin", fmt)
    x, w = (torch.from_numpy(r.standard_normal((n, K)).astype(np.float32)).bfloat16().cuda() for n in (M, N))
    W = g13.fp4_quantize(w, fmt)
    want = g13.fp4_matmul(g13.fp4_quantize(x, fmt), W)
    a, b = (ref.values(*ref.quantise(v.float().cpu().numpy(), fmt), fmt) for v in (x, w))
    check_product(want, a, b, "f32")
    out, gr, side = torch.zeros_like(want), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(gr):
        g13.fp4_matmul(g13.fp4_quantize(x, fmt), W, out=out)
    torch.cuda.synchronize()
    for _ in range(5):
        gr.replay()
        with torch.cuda.stream(side):
            y = g13.fp4_matmul(g13.fp4_quantize(x, fmt), W)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(y, want)
