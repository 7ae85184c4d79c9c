"""Calls of the norm, 4-bit weights, routing and experts that the other files do not make: the largest sizes, in place
without a residual, many tokens off 16 bytes against a long K, biases that are not finite, no tokens, two threads.
Bounds as in the files of the operators."""
import threading

import numpy as np
import pytest
import torch

import dense_gemm_13_gb300 as g13
from tests import blocks_ref as ref
from tests.test_gpu_norm import check_fp8, check_values, stream_of, tensor
from tests.test_gpu_norm_exact import check_exact
from tests.test_gpu_w4 import DT, check_product, rng, weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_gemm_13_gb300 import _build
    _build.build()
    g13.load()


@pytest.mark.parametrize("M,N,K,group", [(64, 40, 65001, 64), (17, 33, 65535, 65536), (64, 200, 20001, 128), (33, 50, 30001, 32),
                                         (24, 20, 65001, 96)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_w4_many_tokens_off_16_bytes_against_a_long_k(M, N, K, group, dtype):
    r = rng("long", M, K)
    for ints in (True, False):
        W, _, _, _, w = weight(r, N, K, group, dtype, ints=ints)
        v = r.integers(-1, 2, (M, K)) if ints else r.standard_normal((M, K))
        x = torch.from_numpy(v.astype(np.float32)).to(DT[dtype]).cuda()
        y = g13.w4_matmul(x, W, out_dtype="f32")
        if ints:
            assert np.array_equal(y.cpu().numpy(), v.astype(np.float64) @ w[0].T)
        else:
            check_product(y, x, w, "f32")


@pytest.mark.parametrize("M", [1, 20])
def test_w4_many_rows(M):
    N, K = 700001, 70
    r = rng("rows", M)
    W, _, _, _, (w, _) = weight(r, N, K, 32, "bf16", ints=True)
    v = r.integers(-1, 2, (M, K))
    x = torch.from_numpy(v.astype(np.float32)).bfloat16().cuda()
    assert np.array_equal(g13.w4_matmul(x, W, out_dtype="f32").cpu().numpy(), v.astype(np.float64) @ w.T)


@pytest.mark.parametrize("H", [5, 64, 333, 2049, 4096, 16384, 16399, 40000])
@pytest.mark.parametrize("dtype", list(DT))
def test_norm_in_place_of_x(H, dtype):
    r = rng("alone", H, dtype)
    for T in (1, 3, 500):
        x, w = tensor(r, dtype, T, H), tensor(r, dtype, H)
        _, h64 = stream_of(x, None)
        y = g13.rms_norm(x, w, out=x)
        assert y is x
        check_values(y, h64, w, 1e-6, 0.0, dtype)


@pytest.mark.parametrize("H", [(1 << 22) - 3, 1 << 22])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_of_the_longest_rows(H, dtype):
    r = rng("longest", H, dtype)
    x, rs, w = tensor(r, dtype, 2, H), tensor(r, "f32", 2, H), tensor(r, "bf16", H)
    h, h64 = stream_of(x, rs)
    y, h2 = g13.rms_norm(x, w, residual=rs, out_dtype="f32")
    assert torch.equal(h2, h)
    check_values(y, h64, w, 1e-6, 0.0, "f32")
    q = g13.rms_norm(x, w, residual=rs, out_dtype="mxfp8")[0]
    check_fp8(q, h64, w, 1e-6, 0.0)
    # (a thread adds 4096 squares in each of two sums: 4096 times 4096 products of two roundings at most)
    check_exact(q, h64, w, float(np.float32(1e-6)), d=2.0 ** -24)


def test_route_with_biases_that_are_not_finite():
    inf, nan = float("inf"), float("nan")
    r = rng("bias")
    z = torch.from_numpy(r.standard_normal((300, 48)).astype(np.float32)).cuda()
    for places in ({3: inf}, {3: inf, 20: inf, 21: inf}, {3: nan}, {0: nan, 47: inf, 5: -inf}, {i: -inf for i in range(44)}):
        bias = (r.standard_normal(48) * 0.1).astype(np.float32)
        for i, v in places.items():
            bias[i] = v
        for kw in (dict(), dict(groups=6, top_groups=2), dict(groups=6, top_groups=2, group_score="top2")):
            for scores in ("sigmoid", "softmax"):
                ids, w = g13.route(z, 4, bias=torch.from_numpy(bias).cuda(), scores=scores, normalize=False, **kw)
                rid, rw = ref.route(z.double().cpu().numpy(), 4, bias=bias.astype(np.float64), scores=scores, normalize=False, **kw)
                assert np.array_equal(ids.cpu().numpy(), rid), (places, kw, scores)
                assert np.allclose(w.cpu().numpy(), rw, rtol=2.0 ** -17, atol=1e-37)


def test_no_tokens():
    bf, dev = torch.bfloat16, "cuda"
    x = torch.zeros(0, 64, dtype=bf, device=dev)
    ids, w = g13.route(torch.zeros(0, 8, device=dev), 2, bias=torch.zeros(8, device=dev), groups=2, top_groups=1)
    assert tuple(ids.shape) == tuple(w.shape) == (0, 2)
    y = g13.moe_experts(x, torch.zeros(8, 32, 64, dtype=bf, device=dev), torch.zeros(8, 64, 16, dtype=bf, device=dev), ids, w)
    assert tuple(y.shape) == (0, 64)
    q, h = g13.rms_norm(x, residual=x, out_dtype="mxfp8")
    assert (q.rows, q.cols, tuple(h.shape)) == (0, 64, (0, 64))
    W = g13.fp8_quantize(torch.randn(10, 64, device=dev))
    assert tuple(g13.fp8_matmul(q, W).shape) == (0, 10) and tuple(g13.fp8_dequantize(q).shape) == (0, 64)


def test_two_threads():
    # each on a stream of its own, the same shapes and the same weight
    r = rng("threads")
    W, _, _, _, _ = weight(r, 300, 1000, 64, "bf16")
    xs = [torch.from_numpy(r.standard_normal((20, 1000)).astype(np.float32)).bfloat16().cuda() for _ in range(2)]
    wn, z = torch.ones(1000, device="cuda"), torch.randn(20, 64, device="cuda")

    def calls(x):
        n = g13.rms_norm(x, wn)
        q = g13.rms_norm(x, wn, out_dtype="mxfp8")
        return [n, g13.w4_matmul(n, W), g13.fp8_dequantize(q), *g13.route(z, 4, groups=4, top_groups=2)]
    want = [calls(x) for x in xs]
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(2)

    def work(i):
        s = torch.cuda.Stream()
        start.wait()
        with torch.cuda.stream(s):
            for _ in range(200):
                got = calls(xs[i])
            s.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                bad.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("M,N,K", [(1, 300, 1000), (40, 129, 333), (300, 400, 520), (600, 1100, 2048)])
@pytest.mark.parametrize("power", [30, 70, 110, 118, -30, -70, -110])
def test_fp8_scales_over_their_whole_range(M, N, K, power):
    # a power of two more on one side and less on the other leaves every bit of the product; blocks of zeros (the least
    # scale) beside the largest ones
    r = rng("fp8 range", M, N, K)
    a, b = (torch.from_numpy(r.standard_normal((n, K)).astype(np.float32)) for n in (M, N))
    a[:, K // 3: K // 3 + 64], b[:, : 40] = 0, 0
    a, b = a.cuda(), b.cuda()
    want = g13.fp8_matmul(g13.fp8_quantize(a), g13.fp8_quantize(b))
    qa, qb = g13.fp8_quantize(a * 2.0 ** power), g13.fp8_quantize(b * 2.0 ** -power)
    assert torch.equal(g13.fp8_dequantize(qa), g13.fp8_dequantize(g13.fp8_quantize(a)) * 2.0 ** power)
    got = g13.fp8_matmul(qa, qb)
    assert bool(torch.isfinite(got).all()) and torch.equal(got, want)


@pytest.mark.parametrize("M", [1, 300])
def test_fp8_products_at_the_ends_of_the_range(M):
    # scales of 2^-127 whose codes are kept, and terms that leave FP32
    N, K = 200, 256
    r = rng("fp8 ends", M)
    a = torch.from_numpy(r.integers(-7, 8, (M, K)).astype(np.float32)).cuda()
    b = torch.from_numpy(r.integers(-7, 8, (N, K)).astype(np.float32)).cuda()
    want = a.double() @ b.double().T
    qa, qb = g13.fp8_quantize(a * 2.0 ** -126), g13.fp8_quantize(b * 2.0 ** 100)
    assert bool((qa.scales <= 5).all()) and torch.equal(g13.fp8_dequantize(qa), a * 2.0 ** -126)
    assert torch.equal(g13.fp8_matmul(qa, qb).double(), want * 2.0 ** -26)
    big = g13.fp8_matmul(g13.fp8_quantize(a * 2.0 ** 100), qb)
    assert not bool(torch.isfinite(big).any())  # (terms of both signs beyond FP32: infinities or NaN)
