"""4-bit weights with group scales on the GPU: layout and quantisation element for element, products against 64-bit sums.

Tolerance of a product, with S = sum |x| (q + z) s of an element and u = 2^-24.  Up to sixteen tokens (or rows that are
not aligned): a group's products q x come in two chains of at most four tensor-core steps (each adds 16 exact products, off by at
most 2^-22 of the magnitudes so far if it truncates: 4 * 2^-22); its sum of x has at most eight additions; taking off z times
it, joining the chains and multiplying by the scale into a running sum round once each.  More tokens: products (q - z) x, |q - z|
<= q + z, in one chain of at most eight such steps (8 * 2^-22 = 2^-19), times the scale into the running sum.  A warp adds one such sum
for every 32 columns of its share of K at most, then at most eight warps' and eight CTAs' sums are added; alpha rounds once.  Up
to sixteen tokens activations are brought to FP16 by a power of two per 128 columns that puts the largest of them into [2^14, 2^15),
half of them by a 16th more, so [2^10, 2^11); half a step of FP16's lowest range, 2^-25, is 2^-35 of that at most:
    |Y - ref| <= (2^-19 + (K / 32 + 28) u) S + 2^-35 sum_b max_b|x| sum_b (q + z) s      before the epilogue (b: 128 columns).
GELU (erff) is off by at most 4 units of |y|; each FP32 step of the epilogue rounds its result; the cast adds half a
step of its type.
"""
import zlib

import numpy as np
import pytest
import torch

import dense_gemm_13_gb300 as g13
from tests import blocks_ref as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_gemm_13_gb300 import _build
    _build.build()
    g13.load()


def rng(*key):
    return np.random.default_rng(zlib.crc32(repr(key).encode()))


def weight(r, N, K, group, dtype, zeros=True, ints=False):
    """(W4Tensor made by w4_pack, codes, scales, zeros, (64-bit values, (q + z) s))."""
    G = -(-K // group)
    q = r.integers(0, 16, (N, K)).astype(np.uint8)
    s = torch.from_numpy((2.0 ** r.integers(-1, 2, (N, G)) if ints else r.random((N, G)) * 0.1 + 0.01).astype(np.float32))
    s = s.to(DT[dtype])
    z = r.integers(0, 16, (N, G)).astype(np.uint8) if zeros else None
    W = g13.w4_pack(torch.from_numpy(q).cuda(), s.cuda(), None if z is None else torch.from_numpy(z).cuda(), group)
    s64 = s.double().numpy()
    z64 = np.full(s64.shape, 8.0) if z is None else z
    return W, q, s, z, (ref.w4_values(q, s64, z, group), ref.w4_values(q, s64, -z64.astype(float), group))


LAYOUTS = [(1, 1, 32), (16, 64, 64), (17, 65, 32), (40, 130, 128), (100, 1000, 96), (33, 300, 256), (5, 64, 65536)]


@pytest.mark.parametrize("shape", LAYOUTS, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("zeros", [True, False])
def test_pack_and_read_back(shape, dtype, zeros):
    N, K, group = shape
    W, q, s, z, values = weight(rng("pack", shape, zeros), N, K, group, dtype, zeros)
    values = values[0]
    assert np.array_equal(W.codes.cpu().numpy(), ref.w4_words(q))
    bits = s.view(torch.int16).numpy()
    assert np.array_equal(W.scales.view(torch.int16).cpu().numpy(), ref.w4_entries(bits))
    assert (W.zeros is None) == (not zeros)
    if zeros:
        assert np.array_equal(W.zeros.cpu().numpy(), ref.w4_entries(z))
    for out in DT:
        assert torch.equal(g13.w4_dequantize(W, out).cpu(), torch.from_numpy(values.astype(np.float32)).to(DT[out]))
    again = g13.W4Tensor(W.codes, W.scales, W.zeros, N, K, group)
    big = torch.full((N + 2, K + 5), 7.0, device="cuda")
    g13.w4_dequantize(again, out=big[1:-1, 2: 2 + K])
    assert torch.equal(big[1:-1, 2: 2 + K], g13.w4_dequantize(W))
    big[1:-1, 2: 2 + K] = 7
    assert bool((big == 7).all())


@pytest.mark.parametrize("shape", LAYOUTS, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("symmetric", [True, False])
def test_quantise(shape, dtype, symmetric):
    N, K, group = shape
    r = rng("quant", shape, dtype, symmetric)
    w = torch.from_numpy(r.standard_normal((N, K)).astype(np.float32) * 0.2)
    w[0, : K // 2] = 0
    if N > 3:
        w[2] = w[2].abs()
        w[3] = -w[3].abs() - 1
    w = w.to(DT[dtype])
    sdt = "f16" if dtype == "f16" else "bf16"
    W = g13.w4_quantize(w.cuda(), group, symmetric=symmetric, dtype=sdt)
    assert W.dtype == sdt and (W.zeros is None) == symmetric
    G = -(-K // group)
    x = np.zeros((N, G * group))
    x[:, :K] = w.double().numpy()
    x = x.reshape(N, G, group)
    lo, hi = np.minimum(x.min(2), 0), np.maximum(x.max(2), 0)
    step = np.maximum(hi, -lo) / 7.5 if symmetric else (hi - lo) / 15
    nt = -(-N // 16) * 16
    rr, cc = np.meshgrid(np.arange(N), np.arange(G), indexing="ij")
    at = (rr // 16 * G + cc) * 16 + rr % 8 * 2 + rr % 16 // 8
    assert W.scales.numel() == nt * G
    s = W.scales.double().cpu().numpy()[at]
    u = torch.finfo(DT[sdt]).eps / 2
    assert (np.abs(s - step) <= step * (u + 2.0 ** -21) + torch.finfo(DT[sdt]).tiny).all()
    z = np.full((N, G), 8.0) if symmetric else W.zeros.cpu().numpy()[at].astype(float)
    v = g13.w4_dequantize(W).double().cpu().numpy()
    full = np.zeros((N, G * group))
    full[:, :K] = v
    q = np.round(full.reshape(N, G, group) / np.where(s > 0, s, 1)[..., None] + z[..., None])
    assert ((q >= 0) & (q <= 15)).all()
    # nearest code: off by half a step, and where a range's end was cut by what the scale's and the zero's
    # rounding leave beyond it
    cut = np.maximum(np.maximum(hi - (15 - z) * s, -lo - z * s), 0)
    err = np.abs(full.reshape(N, G, group) - x)
    assert (err <= (0.5 * s + cut)[..., None] * (1 + 2.0 ** -20)).all()
    assert (cut <= (0.5 + 16 * u) * s + 1e-30).all()
    assert (v[0, : K // 2 // group * group] == 0).all()
    # zero is a value of its own with zeros; strided sources
    view = torch.zeros(N, K + 3, dtype=DT[dtype], device="cuda")
    view[:, 1: 1 + K] = w.cuda()
    V = g13.w4_quantize(view[:, 1: 1 + K], group, symmetric=symmetric, dtype=sdt)
    assert torch.equal(V.codes, W.codes) and torch.equal(V.scales, W.scales)


def test_quantise_not_finite():
    w = torch.ones(4, 128, device="cuda")
    w[1, 3], w[2, 100] = float("inf"), float("nan")
    for symmetric in (True, False):
        v = g13.w4_dequantize(g13.w4_quantize(w, 64, symmetric=symmetric))
        bad = torch.zeros(4, 128, dtype=torch.bool, device="cuda")
        bad[1, :64] = bad[2, 64:] = True
        assert torch.equal(torch.isnan(v), bad)


def check_product(got, x, w, out, bias=None, act="none", R=None, alpha=1.0, beta=1.0):
    x, K = x.double().cpu().numpy(), x.shape[1]
    w, both = w  # values, (q + z) s
    S, y = np.abs(x) @ both.T * abs(alpha), alpha * (x @ w.T)
    tol = (2.0 ** -19 + (K / 32 + 28) * 2.0 ** -24) * S
    for b in range(0, K, 128):
        tol = tol + 2.0 ** -35 * abs(alpha) * np.abs(x[:, b:b + 128]).max(1)[:, None] * both[:, b:b + 128].sum(1)
    if bias is not None:
        y = y + bias.double().cpu().numpy()
        tol = tol + 2.0 ** -24 * np.abs(y)
    if act == "gelu":
        from scipy.special import erfc
        tol = 1.13 * tol + 2.0 ** -21 * np.abs(y)
        y = 0.5 * y * erfc(-y / np.sqrt(2))
    elif act == "relu":
        y = np.maximum(y, 0)
    if R is not None:
        y = y + beta * R.double().cpu().numpy()
        tol = tol + 2.0 ** -24 * np.abs(y)
    tol = tol + torch.finfo(DT[out]).eps / 2 * (np.abs(y) + tol) + torch.finfo(DT[out]).smallest_normal * 2.0 ** -10
    err = np.abs(got.double().cpu().numpy() - y)
    assert got.dtype == DT[out] and (err <= tol).all(), f"max err/tol {np.max(err / tol):.3g}"


SHAPES = [(1, 1, 1, 32), (1, 16, 64, 64), (1, 6144, 512, 128), (2, 17, 65, 32), (3, 100, 3001, 96), (8, 500, 1000, 128),
          (9, 31, 130, 32), (16, 333, 2000, 64), (17, 40, 4097, 256), (32, 130, 700, 32), (33, 64, 520, 128),
          (64, 200, 1500, 64), (64, 16, 8192, 128), (5, 2500, 64, 64), (1, 48, 65536, 128), (7, 10, 20000, 4096),
          (64, 20, 30000, 96), (40, 33, 65536, 65536), (1, 40000, 200, 32)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_product_exact_integers(shape, dtype):
    # x of -1, 0, 1, weights of 15 steps at most of 1/2, 1 or 2: every sum is a multiple of 1/2 below 2^22
    M, N, K, group = shape
    for zeros in (True, False):
        r = rng("int", shape, zeros)
        W, _, _, _, (w, _) = weight(r, N, K, group, dtype, zeros, ints=True)
        assert 30 * K < 2 ** 22
        x = torch.from_numpy(r.integers(-1, 2, (M, K)).astype(np.float32)).to(DT[dtype]).cuda()
        big = torch.full((M + 2, N + 3), 7.0, device="cuda")
        g13.w4_matmul(x, W, out=big[1:-1, 1: N + 1], out_dtype="f32")
        got, want = big[1:-1, 1: N + 1].cpu().numpy(), x.double().cpu().numpy() @ w.T
        assert np.array_equal(got, want), f"{np.sum(got != want)} of {got.size} differ"
        big[1:-1, 1: N + 1] = 7
        assert bool((big == 7).all()), "store outside the M x N window"


@pytest.mark.parametrize("shape", [(1, 515, 900, 128), (4, 131, 2000, 32), (12, 300, 333, 64), (30, 129, 4000, 96),
                                   (64, 300, 770, 256)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("out", list(DT))
def test_product_epilogue(shape, dtype, out):
    M, N, K, group = shape
    r = rng("epi", shape, dtype, out)
    W, _, _, _, w = weight(r, N, K, group, dtype, zeros=K % 2 == 0)
    x = torch.from_numpy(r.standard_normal((M, K)).astype(np.float32)).to(DT[dtype]).cuda()
    bias = torch.from_numpy(r.standard_normal(N).astype(np.float32)).cuda()
    R = torch.from_numpy(r.standard_normal((M, N)).astype(np.float32)).cuda()
    y = g13.w4_matmul(x, W, out_dtype=out)
    check_product(y, x, w, out)
    for _ in range(3):  # the same bits again: no sum depends on timing
        assert torch.equal(y, g13.w4_matmul(x, W, out_dtype=out))
    check_product(g13.w4_matmul(x, W, out_dtype=out, bias=bias, act="gelu", alpha=0.25), x, w, out, bias, "gelu", alpha=0.25)
    check_product(g13.w4_matmul(x, W, out_dtype=out, bias=bias, act="relu", residual=R, beta=-0.5), x, w, out, bias,
                  "relu", R, 1.0, -0.5)


@pytest.mark.parametrize("M", [9, 16, 17, 32, 33, 48, 64])
@pytest.mark.parametrize("shape", [(1, 1, 32), (130, 127, 128), (128, 129, 64), (300, 1000, 32), (1000, 3001, 96),
                                   (17, 9000, 65536), (2100, 2305, 192), (140, 65500, 256)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_product_of_aligned_rows(M, shape, dtype):
    # rows of x on 16 bytes, with NaN behind their end; integers, so that every sum is exact, and fractions
    N, K, group = shape
    r = rng("aligned", M, shape, dtype)
    for ints in (True, False):
        W, _, _, _, w = weight(r, N, K, group, dtype, zeros=M % 2 == 0, ints=ints)
        v = r.integers(-1, 2, (M, K)) if ints else r.standard_normal((M, K))
        big = torch.full((M, K // 8 * 8 + 16), float("nan"), dtype=DT[dtype], device="cuda")
        x = big[:, :K]
        x.copy_(torch.from_numpy(v.astype(np.float32)))
        room = torch.full((M + 2, N + 3), 7.0, device="cuda")
        y = room[1:-1, 1: N + 1]
        g13.w4_matmul(x, W, out=y, out_dtype="f32")
        if ints:
            assert np.array_equal(y.cpu().numpy(), v.astype(np.float64) @ w[0].T)
        else:
            check_product(y, x, w, "f32")
            assert torch.equal(y, g13.w4_matmul(x, W, out_dtype="f32"))
        y.fill_(7)
        assert bool((room == 7).all()), "store outside the M x N window"


@pytest.mark.parametrize("M", [1, 7, 30])
def test_strides(M):
    # x inside larger rows at every alignment, a strided residual
    r = rng("strides", M)
    N, K = 77, 520
    W, _, _, _, w = weight(r, N, K, 128, "bf16")
    for left, right in ((0, 8), (8, 0), (1, 2), (3, 3)):
        big = torch.from_numpy(r.standard_normal((M, K + left + right)).astype(np.float32)).bfloat16().cuda()
        x = big[:, left: left + K]
        R = torch.from_numpy(r.standard_normal((M, N + 3)).astype(np.float32)).cuda()[:, 1: N + 1]
        check_product(g13.w4_matmul(x, W, residual=R, out_dtype="f32"), x, w, "f32", R=R)


def test_not_finite_values_stay_in_their_row():
    r = rng("nan")
    W, _, _, _, w = weight(r, 40, 300, 64, "bf16")
    x = torch.randn(5, 300, device="cuda").bfloat16()
    x[1, 7], x[3, 299] = float("nan"), float("inf")
    for t in (torch.bfloat16, torch.float16):
        V = W if t is torch.bfloat16 else g13.W4Tensor(W.codes, W.scales.half(), W.zeros, 40, 300, 64)
        y = g13.w4_matmul(x.to(t), V, out_dtype="f32")
        assert bool(torch.isnan(y[1]).all()) and not bool(torch.isfinite(y[3]).any())
    y = g13.w4_matmul(x, W, out_dtype="f32")
    rest = [0, 2, 4]
    check_product(y[rest], x[rest], w, "f32")


def test_magnitudes_far_apart():
    # BF16's whole range, between tokens and within one; tokens of zeros
    r = rng("range")
    W, _, _, _, w = weight(r, 60, 1000, 128, "bf16")
    x = r.standard_normal((8, 1000)).astype(np.float32)
    x *= np.exp2(np.array([0, 100, -100, -120, 60, -60, 0, 0]))[:, None].astype(np.float32)
    x[4] *= np.exp2(r.integers(-28, 1, 1000)).astype(np.float32)
    x[5, ::7] = 0
    x[6] = 0
    x[7], x[7, 500:] = 1e-38, 0
    x = torch.from_numpy(x).bfloat16().cuda()
    y = g13.w4_matmul(x, W, out_dtype="f32")
    check_product(y, x, w, "f32")
    assert bool((y[6] == 0).all())
    for i in range(8):  # (a token's neighbours do not count)
        check_product(g13.w4_matmul(x[i: i + 1], W, out_dtype="f32"), x[i: i + 1], w, "f32")


def test_large_codes():
    # code offsets beyond 2^31 bytes
    N, K = 140000, 32768
    tiles, blocks = N // 16, K // 64
    codes = torch.zeros(tiles * blocks * 512, dtype=torch.uint8, device="cuda")
    assert codes.numel() > 2 ** 31
    scales = torch.ones(N, dtype=torch.bfloat16, device="cuda")
    W = g13.W4Tensor(codes, scales, torch.zeros(N, dtype=torch.uint8, device="cuda"), N, K, 65536)
    codes.view(torch.int32)[-1] = 0x11111111  # the last row's last eight columns: 1
    x = torch.ones(1, K, dtype=torch.bfloat16, device="cuda")
    y = g13.w4_matmul(x, W, out_dtype="f32")
    assert float(y[0, -1]) == 8 and float(y[0, :-1].abs().max()) == 0


def test_empty_and_refusals():
    r = rng("refuse")
    W = weight(r, 20, 100, 32, "bf16")[0]
    x = torch.randn(3, 100, device="cuda").bfloat16()
    assert tuple(g13.w4_matmul(x[:0], W).shape) == (0, 20)
    empty = g13.w4_quantize(torch.zeros(0, 64, device="cuda"))
    assert tuple(g13.w4_matmul(torch.zeros(2, 64, device="cuda").bfloat16(), empty).shape) == (2, 0)
    E = g13.GemmError
    f = torch.zeros(3, 20, device="cuda")
    for args, kw in (((x.half(), W), {}), ((x.cpu(), W), {}), ((x[:, :99], W), {}), ((x[0], W), {}), ((x, x), {}),
                     ((x.t().contiguous().t(), W), {}), ((x[:1].expand(3, 100), W), {}),
                     ((torch.zeros(65, 100, device="cuda").bfloat16(), W), {}), ((x, W), dict(act="softmax")),
                     ((x, W), dict(out_dtype="e4m3")), ((x, W), dict(bias=f[0, :19])), ((x, W), dict(bias=f[0].bfloat16())),
                     ((x, W), dict(residual=f[:2])), ((x, W), dict(residual=f.bfloat16())), ((x, W), dict(out=f)),
                     ((x, W), dict(out=f.bfloat16()[:2])), ((torch.tensor(1.0, device="cuda"), W), dict(bias=f[0])),
                     ((x, W), dict(residual=f, out=f, out_dtype="f32")), ((x, W), dict(out=x[:, :20]))):
        with pytest.raises(E):
            g13.w4_matmul(*args, **kw)
    for args in ((W.codes[:-1], W.scales, W.zeros, 20, 100, 32), (W.codes, W.scales.float(), W.zeros, 20, 100, 32),
                 (W.codes, W.scales[:-1], W.zeros, 20, 100, 32), (W.codes, W.scales, W.zeros.int(), 20, 100, 32),
                 (W.codes, W.scales, W.zeros[:-1], 20, 100, 32), (W.codes, W.scales, W.zeros, 20, 100, 33),
                 (W.codes.cpu(), W.scales, W.zeros, 20, 100, 32), (W.codes, W.scales, W.zeros, 20, 0, 32),
                 (W.codes, W.scales, W.zeros, -1, 100, 32)):
        with pytest.raises(E):
            g13.W4Tensor(*args)
    q = torch.zeros(20, 100, dtype=torch.uint8, device="cuda")
    s = torch.zeros(20, 4, dtype=torch.bfloat16, device="cuda")
    for args in ((q.int(), s, None, 32), (q, s[:, :3], None, 32), (q, s.float(), None, 32), (q, s, s, 32),
                 (q, s, None, 64), (q, s.cpu(), None, 32), (q[0], s, None, 32)):
        with pytest.raises(E):
            g13.w4_pack(*args)
    for args, kw in (((x[0],), {}), ((x.double(),), {}), ((x, 48), {}), ((x,), dict(dtype="f32")), ((x.cpu(),), {})):
        with pytest.raises(E):
            g13.w4_quantize(*args, **kw)
    with pytest.raises(E):
        g13.w4_dequantize(x)
    with pytest.raises(E):
        g13.w4_dequantize(W, "f64")


@pytest.mark.parametrize("M,N", [(1, 600), (20, 64)])
def test_streams_and_graphs(M, N):
    r = rng("graph", M)
    W = weight(r, N, 2000, 128, "bf16")[0]
    x = torch.randn(M, 2000, device="cuda").bfloat16()
    want = g13.w4_matmul(x, W)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        y = g13.w4_matmul(x, W, stream=s)
        v = g13.w4_dequantize(W, "bf16", stream=s)
        W2 = g13.w4_quantize(v, 128, stream=s)
        side.synchronize()
        assert torch.equal(y, want) and W2.rows == N
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(g13.w4_matmul(x, W))
        graphs.append(gr)
    x.copy_(torch.randn(M, 2000, device="cuda"))
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(s[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    want = g13.w4_matmul(x, W)
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
