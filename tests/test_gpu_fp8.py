"""8-bit floats on the GPU: quantisation byte for byte against the definition, products against 64-bit sums.

Tolerance of a product, with S = sum |a b| of an element: the tensor core adds K / 32 partial sums in FP32 (each
addition off by at most 2^-22 of a running value <= S if it truncates, and one partial sum of 32 products by as
much), and alpha rounds twice (2^-24 each):
    |C - ref| <= ((K / 32 + 2) 2^-22 + 2 2^-24) S      before the epilogue.
GELU's slope is below 1.13 and its own error below 1e-6 (1 + |y|); each FP32 step of the epilogue rounds its
result (2^-24); the output cast adds half a step of its type.
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


def matrix(r, rows, cols):
    """Normal values with blocks of zeros, tiny and large magnitudes."""
    x = r.standard_normal((rows, cols)).astype(np.float32)
    x *= np.exp2(r.integers(-12, 12, (rows, -(-cols // 16)))).astype(np.float32).repeat(16, 1)[:, :cols]
    x[r.random((rows, cols)) < 0.05] = 0
    x[:, cols // 2: cols // 2 + 32] *= r.random((rows, 1)) < 0.7
    return x


def check_quantised(q, x):
    code, byte = ref.mxfp8(x.astype(np.float64))
    assert np.array_equal(q.scales.cpu().numpy(), ref.tiles(byte)), "scales"
    got, want = q.codes.cpu().numpy(), ref.mxfp8_rows(code)
    fine = np.repeat(byte != 255, 32, 1)  # codes under a NaN scale mean nothing
    assert np.array_equal(got[fine], want[fine]), f"{np.sum(got[fine] != want[fine])} codes differ"


SHAPES = [(1, 1), (1, 16), (3, 17), (1, 4096), (5, 31), (127, 33), (128, 64), (129, 100), (300, 257), (33, 1000),
          (257, 520), (2, 300007), (70003, 17)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_quantise_bytes(dtype, shape):
    x = torch.from_numpy(matrix(rng(dtype, shape), *shape)).to(DT[dtype])
    q = g13.fp8_quantize(x.cuda())
    check_quantised(q, x.float().numpy())
    v = torch.from_numpy(ref.mxfp8_values(*ref.mxfp8(x.double().numpy()))).float()
    for out in DT:
        assert torch.equal(g13.fp8_dequantize(q, out).cpu(), v.to(DT[out])), out


def test_quantise_every_tie_and_border():
    # every midpoint between codes and its neighbours, under several scales; blocks whose largest lies at a border of the scales
    mid = (ref.E4M3[1:] + ref.E4M3[:-1]) / 2
    m = mid.astype(np.float32)
    base = np.concatenate([m, np.nextafter(m, np.float32(1e9)), np.nextafter(m, np.float32(0)), ref.E4M3.astype(np.float32)])
    base = base[: len(base) // 31 * 31].reshape(-1, 31)
    rows = []
    for s in (1.0, 2.0 ** -20, 2.0 ** 30):
        x = np.full((len(base), 32), 448.0, np.float32)
        x[:, :31] = base * np.where(np.arange(31) % 2, -1, 1)
        rows.append(np.minimum(np.abs(x), 448) * np.sign(x) * np.float32(s))
    x = np.concatenate(rows).reshape(-1, 32)
    check_quantised(g13.fp8_quantize(torch.from_numpy(x).cuda()), x)
    tops = np.array([448, np.nextafter(np.float32(448), np.float32(449)), 447.9, 1.75, 1.75 + 2.0 ** -23, 2 - 2.0 ** -23,
                     1.0, 2.0 ** -118 * 1.75, 2.0 ** -120, 2.0 ** -126, 2.0 ** -149, 3.4e38, 0.0], np.float32)
    y = np.zeros((len(tops), 96), np.float32)
    y[:, 5], y[:, 40], y[:, 64:] = tops, -tops, tops[:, None] * np.linspace(0, 1, 32).astype(np.float32)
    check_quantised(g13.fp8_quantize(torch.from_numpy(y).cuda()), y)


def test_quantise_not_finite():
    x = np.ones((4, 100), np.float32)
    x[1, 40], x[2, 99], x[3, 0] = np.inf, np.nan, -np.inf
    q = g13.fp8_quantize(torch.from_numpy(x).cuda())
    check_quantised(q, x)
    v = g13.fp8_dequantize(q).cpu().numpy()
    assert np.isnan(v[1, 32:64]).all() and np.isnan(v[2, 96:]).all() and np.isnan(v[3, :32]).all()
    assert np.isfinite(v[0]).all() and np.isfinite(v[1, 64:]).all()


@pytest.mark.parametrize("dtype", list(DT))
def test_strides_and_offsets(dtype):
    x = torch.from_numpy(matrix(rng("s", dtype), 70, 203)).to(DT[dtype]).cuda()
    for view in (x[1:, 3:150], x[:, 1:], x[::2, 8:40], x.t()[:, :60]):
        q = g13.fp8_quantize(view)
        check_quantised(q, view.float().cpu().numpy())
        big = torch.full((view.shape[0] + 2, view.shape[1] + 5), 7.0, dtype=DT[dtype], device="cuda")
        g13.fp8_dequantize(q, dtype, out=big[1:-1, 3: 3 + view.shape[1]])
        assert torch.equal(big[1:-1, 3: 3 + view.shape[1]], g13.fp8_dequantize(q, dtype))
        big[1:-1, 3: 3 + view.shape[1]] = 7
        assert bool((big == 7).all())


# ------------------------------------------------------------------ products
def operand(r, rows, cols, ints=False):
    """(Fp8Tensor, 64-bit values)."""
    nb = -(-cols // 32)
    if ints:  # 0, +-1, +-2, +-3, scales 1 or 2
        code = np.array([0, 0x38, 0x40, 0x44, 0xB8, 0xC0, 0xC4], np.uint8)[r.integers(0, 7, (rows, cols))]
        byte = r.integers(127, 129, (rows, nb)).astype(np.uint8)
    else:
        code = r.integers(0, 256, (rows, cols)).astype(np.uint8)
        code[(code & 127) == 127] = 5
        byte = r.integers(120, 134, (rows, nb)).astype(np.uint8)
    t = g13.Fp8Tensor(torch.from_numpy(ref.mxfp8_rows(code)).cuda(), torch.from_numpy(ref.tiles(byte)).cuda(), rows, cols)
    return t, ref.mxfp8_values(code, byte)


P_SHAPES = [(1, 1, 1), (1, 128, 32), (1, 300, 1000), (7, 129, 33), (16, 128, 128), (17, 200, 257), (32, 64, 512),
            (33, 500, 96), (64, 130, 300), (65, 257, 700), (127, 384, 1030), (128, 128, 2048), (129, 130, 31),
            (300, 515, 520), (257, 1000, 64), (3, 100001, 70), (100001, 3, 70), (5, 130, 60000),
            # CTA pairs: several tiles per pair, ragged in every direction
            (257, 19700, 320), (1030, 5000, 1100), (2100, 2700, 31), (2050, 5000, 161)]


@pytest.mark.parametrize("shape", P_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_product_exact_integers(shape):
    # products are integers up to 36 and every partial sum stays below 2^24: FP32 is exact in any order
    M, N, K = shape
    r = rng("int", shape)
    (A, a), (B, b) = operand(r, M, K, ints=True), operand(r, N, K, ints=True)
    assert 36 * K < 2 ** 24
    big = torch.full((M + 2, N + 3), 7.0, device="cuda")
    g13.fp8_matmul(A, B, out=big[1:-1, 1: N + 1])
    got, want = big[1:-1, 1: N + 1].cpu().numpy(), a @ b.T
    assert np.array_equal(got, want), f"{np.sum(got != want)} of {got.size} differ"
    big[1:-1, 1: N + 1] = 7
    assert bool((big == 7).all()), "store outside the M x N window"


def check_product(got, a, b, out, bias=None, act="none", R=None, alpha=1.0, beta=1.0):
    K = a.shape[1]
    S = np.abs(a) @ np.abs(b).T * abs(alpha)
    y = alpha * (a @ b.T)
    tol = ((K / 32 + 2) * 2.0 ** -22 + 2 * 2.0 ** -24) * S
    if bias is not None:
        y = y + bias
        tol = tol + 2.0 ** -24 * np.abs(y)
    if act == "gelu":
        from scipy.special import erfc
        tol = 1.13 * tol + 1e-6 * (1 + np.abs(y))
        y = 0.5 * y * erfc(-y / np.sqrt(2))
    elif act == "relu":
        y = np.maximum(y, 0)
    if R is not None:
        y = y + beta * R
        tol = tol + 2.0 ** -24 * np.abs(y)
    tol = tol + torch.finfo(DT[out]).eps / 2 * (np.abs(y) + tol) + torch.finfo(DT[out]).smallest_normal * 2.0 ** -10
    err = np.abs(got.double().cpu().numpy() - y)
    assert (err <= tol).all(), f"max err/tol {np.max(err / tol):.3g}"


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("shape", [(1, 515, 900), (20, 131, 2000), (50, 300, 333), (100, 129, 4000),
                                   (200, 300, 770), (600, 9800, 128), (1300, 3900, 700)], ids=lambda s: "x".join(map(str, s)))
def test_product_epilogue(out, shape):
    M, N, K = shape
    r = rng("epi", out, shape)
    (A, a), (B, b) = operand(r, M, K), operand(r, N, K)
    al = np.float32(1.0 / np.abs(a @ b.T).max())
    bias, R = r.standard_normal(N).astype(np.float32), r.standard_normal((M, N)).astype(np.float32)
    tb, tR = torch.from_numpy(bias).cuda(), torch.from_numpy(R).cuda()
    check_product(g13.fp8_matmul(A, B, alpha=al, out_dtype=out), a, b, out, alpha=float(al))
    check_product(g13.fp8_matmul(A, B, alpha=4 * al, out_dtype=out, bias=tb, act="gelu"), a, b, out, bias, "gelu",
                  alpha=4 * float(al))
    check_product(g13.fp8_matmul(A, B, alpha=al, out_dtype=out, bias=tb, act="relu", residual=tR, beta=-0.5), a, b,
                  out, bias, "relu", R, float(al), -0.5)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_nan_scale_stays_in_its_row(M):
    r = rng("nan", M)
    x = r.standard_normal((M, 700)).astype(np.float32)
    x[M // 2, 600] = np.inf
    w = r.standard_normal((200, 700)).astype(np.float32)
    w[7, 0] = np.nan
    C = g13.fp8_matmul(g13.fp8_quantize(torch.from_numpy(x).cuda()), g13.fp8_quantize(torch.from_numpy(w).cuda())).cpu().numpy()
    bad = np.zeros(C.shape, bool)
    bad[M // 2, :] = bad[:, 7] = True
    assert np.array_equal(np.isnan(C), bad)


def test_empty():
    for shape in ((0, 5), (4, 0)):
        assert tuple(g13.fp8_dequantize(g13.fp8_quantize(torch.zeros(shape, device="cuda"))).shape) == shape
    A, B = (g13.fp8_quantize(torch.zeros((n, 0), device="cuda")) for n in (3, 40))
    bias = torch.arange(40.0, device="cuda")
    assert torch.equal(g13.fp8_matmul(A, B, bias=bias), bias.expand(3, 40))  # K = 0: the epilogue of zero


@pytest.mark.parametrize("M", [1, 100, 400])
def test_graphs_and_streams(M):
    r = rng("graph", M)
    ops = [(operand(r, M, 1500), operand(r, 800, 1500)) for _ in range(2)]
    want = [g13.fp8_matmul(A, B) for (A, _), (B, _) in ops]
    graphs, outs = [], []
    for (A, _), (B, _) in ops:
        out, gr = torch.zeros(M, 800, device="cuda"), torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            g13.fp8_matmul(A, B, out=out)
        graphs.append(gr)
        outs.append(out)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(s[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], want[i])
    (A, _), (B, _) = ops[0]
    s[0].wait_stream(torch.cuda.current_stream())
    for st in (s[0], s[0].cuda_stream):
        y = g13.fp8_matmul(A, B, stream=st)
        s[0].synchronize()
        assert torch.equal(y, want[0])


def test_no_plan_while_capturing():
    A, B = (g13.fp8_quantize(torch.randn(n, 77, device="cuda")) for n in (3, 41))
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        with pytest.raises(g13.GemmError, match="capturing"):
            g13.fp8_matmul(A, B)
        torch.zeros(1, device="cuda")


@pytest.mark.parametrize("flag", [g13.FLAG_TEST_STALL, g13.FLAG_TEST_STALL_PEER])
@pytest.mark.parametrize("M,N", [(1, 300), (200, 300), (1200, 4100)])
def test_timeout_is_reported(M, N, flag):
    # one CTA withholds one stage: the waits run out, the plan says so, and a new plan works
    r = rng("stall", M)
    (A, a), (B, b) = operand(r, M, 1000, ints=True), operand(r, N, 1000, ints=True)
    C = torch.zeros(M, N, device="cuda")
    plan = g13.gemm_fp8_plan(M, N, 1000, N, g13.Epilogue(b_layout="nk", flags=flag, timeout_ms=50))
    g13.gemm_fp8_run(plan, A, B, C)
    assert g13.gemm_fp8_status(plan) == -5
    plan2 = g13.gemm_fp8_plan(M, N, 1000, N)
    g13.gemm_fp8_run(plan2, A, B, C)
    assert g13.gemm_fp8_status(plan2) == 0
    assert np.array_equal(C.cpu().numpy(), a @ b.T)


def test_python_refusals():
    x = torch.randn(5, 70, device="cuda")
    q, f4 = g13.fp8_quantize(x), g13.fp4_quantize(x, "mxfp4")
    assert tuple(q.codes.shape) == (5, 96) and q.scales.numel() == 512 and q.format == "mxfp8"
    same = g13.Fp8Tensor(q.codes, q.scales, 5, 70)
    assert torch.equal(g13.fp8_dequantize(same), g13.fp8_dequantize(q))
    E = g13.GemmError
    for args in ((q.codes, q.scales[:256], 5, 70), (q.codes, q.scales, 6, 70), (q.codes[:, :64], q.scales, 5, 70),
                 (q.codes.int(), q.scales, 5, 70), (q.codes, q.scales, -5, 70), (q.codes.cpu(), q.scales, 5, 70)):
        with pytest.raises(E):
            g13.Fp8Tensor(*args)
    for kw in (dict(B=f4), dict(A=f4, B=f4), dict(A=x), dict(B=g13.fp8_quantize(x[:, :60])), dict(act="softmax"),
               dict(out_dtype="f64"), dict(bias=torch.zeros(4, device="cuda")), dict(bias=torch.zeros(5)),
               dict(residual=torch.zeros(5, 6, device="cuda")), dict(residual=torch.zeros(1, 5, device="cuda").expand(5, 5)),
               dict(out=torch.zeros(5, 5, device="cuda", dtype=torch.float16))):
        c = dict(dict(A=q, B=q), **kw)
        with pytest.raises(E):
            g13.fp8_matmul(c.pop("A"), c.pop("B"), **c)
    for bad in (x, f4):
        with pytest.raises(E):
            g13.fp8_dequantize(bad)
    with pytest.raises(E):
        g13.fp4_dequantize(q)
    with pytest.raises(E):
        g13.fp4_matmul(q, q)
    with pytest.raises(E):
        g13.fp8_dequantize(q, out=torch.zeros(5, 71, device="cuda"))
    with pytest.raises(E):
        g13.gemm_fp8_run(g13.gemm_fp8_plan(5, 5, 64, 5), q, q, x)
