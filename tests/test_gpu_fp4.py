"""Microscaled 4-bit floats on the GPU: quantisation byte for byte against the
definition, products against 64-bit sums, the epilogue, and how calls share a GPU.

Tolerance of a product, with S = sum |a b| of an element: the tensor core adds
K / 64 partial sums in FP32 (each addition off by at most 2^-22 of a running
value <= S if it truncates, and one partial sum of 64 products by as much), the
scales s g of both operands and alpha gA gB round 5 times (2^-24 each):
    |C - ref| <= ((K / 64 + 2) 2^-22 + 5 2^-24) S      before the epilogue.
GELU's slope is below 1.13 and its own error below 1e-6 (1 + |y|); each FP32
step of the epilogue rounds its result (2^-24); the output cast adds half a
step of its type.
"""
import zlib

import numpy as np
import pytest
import torch

import dense_gemm_13_gb300 as g13
from tests import fp4_ref as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FMTS = ["mxfp4", "nvfp4"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_gemm_13_gb300 import _build
    _build.build()
    g13.load()


def rng(*key):
    return np.random.default_rng([zlib.crc32(str(k).encode()) for k in key])


def matrix(r, rows, cols):
    """Normal values with blocks of zeros, tiny and large magnitudes."""
    x = r.standard_normal((rows, cols)).astype(np.float32)
    x *= np.exp2(r.integers(-12, 12, (rows, -(-cols // 16)))).astype(np.float32).repeat(16, 1)[:, :cols]
    x[r.random((rows, cols)) < 0.05] = 0
    x[:, cols // 2: cols // 2 + 32] *= r.random((rows, 1)) < 0.7
    return x


def check_quantised(q, x32, fmt, g):
    code, byte = ref.quantise(x32, fmt, g)
    got_s = q.scales.cpu().numpy()
    want_s = ref.tiles(byte)
    assert np.array_equal(got_s, want_s), f"{np.sum(got_s != want_s)} scale bytes differ"
    got, want = q.codes.cpu().numpy(), ref.pack(code)
    bad = ref.pack(np.broadcast_to((byte == (255 if fmt == "mxfp4" else 127))[..., None] * np.uint8(15),
                                   byte.shape + (ref.BLOCK[fmt],)).reshape(byte.shape[0], -1)[:, : code.shape[1]])
    assert np.array_equal(got & ~bad, want & ~bad), f"{np.sum((got ^ want) & ~bad != 0)} code bytes differ"


SHAPES = [(1, 1), (1, 16), (3, 17), (1, 4096), (5, 31), (127, 33), (128, 64), (129, 100), (300, 257), (33, 1000),
          (257, 520)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_quantise_bytes(fmt, dtype, shape):
    x = torch.from_numpy(matrix(rng(fmt, dtype, shape), *shape)).to(DT[dtype])
    x32 = x.float().numpy()
    g = None
    if fmt == "nvfp4" and shape[0] != 128:
        g = np.float32(np.abs(x32).max() / np.float32(6 * 448))
        g = g if g > 0 else np.float32(1)
    tg = None if g is None else torch.tensor([g], device="cuda")
    q = g13.fp4_quantize(x.cuda(), fmt, tensor_scale=tg)
    check_quantised(q, x32, fmt, 1.0 if g is None else g)
    # back: FP32 products of code and scale, cast once
    for out in DT:
        v = torch.from_numpy(ref.values(*ref.quantise(x32, fmt, 1.0 if g is None else g), fmt,
                                        1.0 if g is None else g)).float()
        assert torch.equal(g13.fp4_dequantize(q, out).cpu(), v.to(DT[out])), out


@pytest.mark.parametrize("fmt", FMTS)
def test_quantise_every_tie(fmt):
    # every midpoint, its neighbours and every magnitude up to 8, under scales whose quotients are exact
    # and under ones that are not
    base = np.concatenate([ref.MID, np.nextafter(ref.MID.astype(np.float32), np.float32(9)),
                           np.nextafter(ref.MID.astype(np.float32), np.float32(0)), ref.E2M1[:8], [7.0, 5.5]])
    rows = []
    for s in (1.0, 0.5, 448.0, 2.0 ** -9, 0.4375, 1.875, 3e-3, 26.0):
        x = np.zeros(32 * len(base), np.float32)
        x[0::2] = np.repeat(base, 16) * s * np.tile([1, -1], 8 * len(base))
        x[1::32] = 6 * s  # the block's largest
        x[17::32] = 6 * s
        rows.append(x)
    x = np.stack(rows)
    check_quantised(g13.fp4_quantize(torch.from_numpy(x).cuda(), fmt), x, fmt, 1.0)
    if fmt == "nvfp4":
        for g in (np.float32(0.1), np.float32(3e-39), np.float32(1.7e-30), np.float32(2.0 ** 70)):
            y = (x * g).astype(np.float32)
            check_quantised(g13.fp4_quantize(torch.from_numpy(y).cuda(), fmt,
                                             tensor_scale=torch.tensor([g], device="cuda")), y, fmt, g)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantise_extremes(fmt):
    x = np.zeros((6, 100), np.float32)
    x[0, 3] = 1e-45
    x[1, :] = np.float32(3.4e38)
    x[2, 40] = np.inf
    x[3, 99] = np.nan
    x[4, :] = np.float32(1.2e-38)
    x[5, ::3] = -0.0
    q = g13.fp4_quantize(torch.from_numpy(x).cuda(), fmt)
    check_quantised(q, x, fmt, 1.0)
    v = g13.fp4_dequantize(q).cpu().numpy()
    b = ref.BLOCK[fmt]
    assert np.isnan(v[2, 40 // b * b: 40 // b * b + b]).all() and np.isnan(v[3, 96:]).all()
    assert np.isfinite(np.delete(v, [2, 3], 0)).all() and np.isfinite(v[2, : 40 // b * b]).all()


@pytest.mark.parametrize("g", [1e-15, 3e-19])
def test_quantise_saturates_with_its_sign(g):
    # quotients past FP32's range, next to ordinary ones: the scale of the whole tensor is far too small
    x = np.zeros((4, 64), np.float32)
    x[0], x[1, ::2], x[1, 1::2] = -1e30, 3e38, -3e38
    x[2] = np.linspace(-1, 1, 64) * np.float32(g) * 2000
    x[3, :16], x[3, 16:] = -1e30, np.linspace(-3, 3, 48) * np.float32(g)
    q = g13.fp4_quantize(torch.from_numpy(x).cuda(), "nvfp4", tensor_scale=torch.tensor([g], device="cuda"))
    with np.errstate(over="ignore"):
        check_quantised(q, x, "nvfp4", np.float32(g))
    v = g13.fp4_dequantize(q).cpu().numpy()
    assert np.array_equal(np.sign(v[:2]), np.sign(x[:2]))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", list(DT))
def test_strides_and_offsets(fmt, dtype):
    # rows and bases that are not 16-byte aligned; a destination inside a larger one keeps its surroundings
    x = torch.from_numpy(matrix(rng("s", fmt, dtype), 70, 203)).to(DT[dtype]).cuda()
    for view in (x[1:, 3:150], x[:, 1:], x[::2, 8:40], x.t()[:, :60]):
        q = g13.fp4_quantize(view, fmt)
        check_quantised(q, view.float().cpu().numpy(), fmt, 1.0)
        big = torch.full((view.shape[0] + 2, view.shape[1] + 5), 7.0, dtype=DT[dtype], device="cuda")
        g13.fp4_dequantize(q, dtype, out=big[1:-1, 3: 3 + view.shape[1]])
        assert torch.equal(big[1:-1, 3: 3 + view.shape[1]], g13.fp4_dequantize(q, dtype))
        big[1:-1, 3: 3 + view.shape[1]] = 7
        assert bool((big == 7).all())


def test_empty():
    for shape in ((0, 5), (4, 0)):
        q = g13.fp4_quantize(torch.zeros(shape, device="cuda"), "mxfp4")
        assert tuple(g13.fp4_dequantize(q).shape) == shape
    A, B = (g13.fp4_quantize(torch.zeros((n, 0), device="cuda"), "mxfp4") for n in (3, 40))
    bias = torch.arange(40.0, device="cuda")
    C = torch.full((3, 40), 5.0, device="cuda")
    g13.fp4_matmul(A, B, bias=bias, out=C)  # K = 0: the epilogue of zero
    assert torch.equal(C, bias.expand(3, 40))
    E = g13.fp4_quantize(torch.zeros((0, 64), device="cuda"), "nvfp4")
    assert tuple(g13.fp4_matmul(E, E).shape) == (0, 0)


# ------------------------------------------------------------------ products
def operand(r, rows, cols, fmt, g=None, ints=False):
    """(Fp4Tensor, 64-bit values)."""
    code = r.integers(0, 16, (rows, cols)).astype(np.uint8)
    nb = -(-cols // ref.BLOCK[fmt])
    if ints:
        code = np.array([0, 2, 4, 5, 6, 7, 8, 10, 12, 13, 14, 15], np.uint8)[r.integers(0, 12, (rows, cols))]
        byte = np.full((rows, nb), 127 if fmt == "mxfp4" else 0x38, np.uint8)
        byte += r.integers(0, 2, byte.shape).astype(np.uint8) * (1 if fmt == "mxfp4" else 8)  # 1 or 2
    elif fmt == "mxfp4":
        byte = r.integers(120, 134, (rows, nb)).astype(np.uint8)
    else:
        byte = r.integers(0, 127, (rows, nb)).astype(np.uint8)
    t = g13.Fp4Tensor(torch.from_numpy(ref.pack(code)).cuda(), torch.from_numpy(ref.tiles(byte)).cuda(), rows,
                      cols, fmt, None if g is None else torch.tensor([g], dtype=torch.float32, device="cuda"))
    return t, ref.values(code, byte, fmt, 1.0 if g is None else g)


P_SHAPES = [(1, 1, 1), (1, 128, 64), (1, 300, 1000), (7, 129, 65), (16, 128, 256), (17, 200, 257), (32, 64, 512),
            (33, 500, 96), (64, 130, 300), (65, 257, 700), (127, 384, 1030), (128, 128, 2048), (129, 130, 31),
            (300, 515, 520), (257, 1000, 64),
            # CTA pairs: several tiles per pair, ragged in every direction
            (257, 19700, 320), (1030, 5000, 1100), (2100, 2700, 31)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("shape", P_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_product_exact_integers(fmt, shape):
    # products are multiples of 1 up to 144 and every partial sum stays below 2^24: FP32 is exact in any order
    M, N, K = shape
    r = rng("int", fmt, shape)
    (A, a), (B, b) = operand(r, M, K, fmt, ints=True), operand(r, N, K, fmt, ints=True)
    want = a @ b.T
    assert (np.abs(a) @ np.abs(b).T).max() < 2 ** 24
    big = torch.full((M + 2, N + 3), 7.0, device="cuda")
    g13.fp4_matmul(A, B, out=big[1:-1, 1: N + 1])
    got = big[1:-1, 1: N + 1].cpu().numpy()
    assert np.array_equal(got, want), f"{np.sum(got != want)} of {got.size} differ"
    big[1:-1, 1: N + 1] = 7
    assert bool((big == 7).all()), "store outside the M x N window"


@pytest.mark.parametrize("shape", [(100001, 3, 70), (3, 100001, 70), (5, 130, 70000), (130, 130, 20000)],
                         ids=lambda s: "x".join(map(str, s)))
def test_product_long_sides(shape):
    M, N, K = shape
    r = rng("long", shape)
    (A, a), (B, b) = operand(r, M, K, "nvfp4", ints=True), operand(r, N, K, "nvfp4", ints=True)
    assert 144 * K < 2 ** 24
    assert np.array_equal(g13.fp4_matmul(A, B).cpu().numpy(), a @ b.T)


def test_scales_whose_partial_product_overflows():
    r = rng("range")
    (A, a), (B, b) = operand(r, 20, 64, "nvfp4", ints=True), operand(r, 40, 64, "nvfp4", ints=True)

    def scaled(q, g):
        return g13.Fp4Tensor(q.codes, q.scales, q.rows, q.cols, "nvfp4", torch.tensor([g], device="cuda"))

    # alpha gB lies beyond FP32, alpha gA gB does not: powers of two, so the result is exact
    y = g13.fp4_matmul(scaled(A, 2.0 ** -100), scaled(B, 2.0 ** 90), alpha=2.0 ** 60)
    assert np.array_equal(y.cpu().numpy(), (a @ b.T * 2.0 ** 50).astype(np.float32))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("shape", [(200003, 17), (2, 300007)], ids=lambda s: f"{s[0]}x{s[1]}")
def test_quantise_long_sides(fmt, shape):
    x = matrix(rng("ql", fmt, shape), *shape)
    check_quantised(g13.fp4_quantize(torch.from_numpy(x).cuda(), fmt), x, fmt, 1.0)


def check_product(got, A, B, out, bias=None, act="none", R=None, alpha=1.0, beta=1.0):
    K = A.shape[1]
    S = np.abs(A) @ np.abs(B).T * abs(alpha)
    y = alpha * (A @ B.T)
    tol = ((K / 64 + 2) * 2.0 ** -22 + 5 * 2.0 ** -24) * S
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


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("shape", [(1, 515, 900), (20, 131, 2000), (50, 300, 333), (100, 129, 4000),
                                   (200, 300, 770), (600, 9800, 128), (1300, 3900, 700)], ids=lambda s: "x".join(map(str, s)))
def test_product_epilogue(fmt, out, shape):
    M, N, K = shape
    r = rng("epi", fmt, out, shape)
    ga, gb = (None, None) if fmt == "mxfp4" else (0.0123, 0.004)
    (A, a), (B, b) = operand(r, M, K, fmt, ga), operand(r, N, K, fmt, gb)
    alpha = 1.0 / np.abs(a @ b.T).max()
    bias, R = r.standard_normal(N).astype(np.float32), r.standard_normal((M, N)).astype(np.float32)
    tb, tR = torch.from_numpy(bias).cuda(), torch.from_numpy(R).cuda()
    al = np.float32(alpha)
    check_product(g13.fp4_matmul(A, B, alpha=al, out_dtype=out), a, b, out, alpha=float(al))
    check_product(g13.fp4_matmul(A, B, alpha=4 * al, out_dtype=out, bias=tb, act="gelu"), a, b, out, bias, "gelu",
                  alpha=4 * float(al))
    check_product(g13.fp4_matmul(A, B, alpha=al, out_dtype=out, bias=tb, act="relu", residual=tR, beta=-0.5), a, b,
                  out, bias, "relu", R, float(al), -0.5)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 40, 300])
def test_nan_scale_stays_in_its_row(fmt, M):
    r = rng("nan", fmt, M)
    x = r.standard_normal((M, 700)).astype(np.float32)
    x[M // 2, 600] = np.inf
    A = g13.fp4_quantize(torch.from_numpy(x).cuda(), fmt)
    w = r.standard_normal((200, 700)).astype(np.float32)
    w[7, 0] = np.nan
    C = g13.fp4_matmul(A, g13.fp4_quantize(torch.from_numpy(w).cuda(), fmt)).cpu().numpy()
    bad = np.zeros(C.shape, bool)
    bad[M // 2, :] = bad[:, 7] = True
    assert np.array_equal(np.isnan(C), bad)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_linear_layer(fmt, dtype):
    # quantise the activations, multiply by a 4-bit weight: as used, on a side stream, repeated
    r = rng("lin", fmt, dtype)
    x = torch.from_numpy(r.standard_normal((45, 640)).astype(np.float32)).to(DT[dtype]).cuda()
    w = torch.from_numpy(r.standard_normal((333, 640)).astype(np.float32)).cuda()
    g = None if fmt == "mxfp4" else (x.float().abs().max() / (6 * 448)).reshape(1)
    W = g13.fp4_quantize(w, fmt)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        ys = [g13.fp4_matmul(g13.fp4_quantize(x, fmt, tensor_scale=g), W) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(st)
    gv = 1.0 if g is None else np.float32(g.item())
    a = ref.values(*ref.quantise(x.float().cpu().numpy(), fmt, gv), fmt, gv)
    b = ref.values(*ref.quantise(w.cpu().numpy(), fmt), fmt)
    for y in ys:
        check_product(y, a, b, "f32")
        assert torch.equal(y, ys[0])


@pytest.mark.parametrize("M", [1, 100, 400])
def test_graph_and_two_streams(M):
    r = rng("graph", M)
    ops = [(operand(r, M, 1500, "nvfp4", 0.5), operand(r, 800, 1500, "nvfp4", 0.25)) for _ in range(2)]
    want = [g13.fp4_matmul(A, B) for (A, _), (B, _) in ops]
    graphs, outs = [], []
    for (A, _), (B, _) in ops:
        out = torch.zeros(M, 800, device="cuda")
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            g13.fp4_matmul(A, B, out=out)
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


@pytest.mark.parametrize("flag", [g13.FLAG_TEST_STALL, g13.FLAG_TEST_STALL_PEER])
@pytest.mark.parametrize("M,N", [(1, 300), (200, 300), (1200, 4100)])
def test_timeout_is_reported(M, N, flag):
    # one CTA withholds one stage: the waits run out, the plan says so, and a new plan works
    r = rng("stall", M)
    (A, a), (B, b) = operand(r, M, 2000, "mxfp4", ints=True), operand(r, N, 2000, "mxfp4", ints=True)
    C = torch.zeros(M, N, device="cuda")
    ep = g13.Epilogue(b_layout="nk", flags=flag, timeout_ms=50)
    plan = g13.gemm_fp4_plan("mxfp4", M, N, 2000, N, ep)
    g13.gemm_fp4_run(plan, A, B, C)
    assert g13.gemm_fp4_status(plan) == -5
    plan2 = g13.gemm_fp4_plan("mxfp4", M, N, 2000, N)
    g13.gemm_fp4_run(plan2, A, B, C)
    assert g13.gemm_fp4_status(plan2) == 0
    assert np.array_equal(C.cpu().numpy(), a @ b.T)


def test_python_refusals():
    x = torch.randn(5, 70, device="cuda")
    q = g13.fp4_quantize(x, "nvfp4")
    p = g13.fp4_quantize(x, "mxfp4")
    assert tuple(q.codes.shape) == (5, 48) and q.scales.numel() == 1024
    g = torch.ones(1, device="cuda")
    same = g13.Fp4Tensor(q.codes, q.scales, 5, 70, "nvfp4", None)
    assert torch.equal(g13.fp4_dequantize(same), g13.fp4_dequantize(q))
    with pytest.raises(AttributeError):
        q.codes = x
    E = g13.GemmError
    for args in ((q.codes, q.scales[:512], 5, 70, "nvfp4"), (q.codes, q.scales, 6, 70, "nvfp4"),
                 (q.codes, q.scales, 5, 70, "mxfp4"), (q.codes[:, :32], q.scales, 5, 70, "nvfp4"),
                 (q.codes.int(), q.scales, 5, 70, "nvfp4"), (q.codes, q.scales, -5, 70, "nvfp4"),
                 (q.codes, q.scales, 5, 70, "nvfp4", g.double()), (q.codes, q.scales, 5, 70, "nvfp4", g.cpu()),
                 (p.codes, p.scales, 5, 70, "mxfp4", g)):
        with pytest.raises(E):
            g13.Fp4Tensor(*args)
    with pytest.raises(E):
        g13.fp4_quantize(x, "mxfp4", tensor_scale=g)
    bad = dict(A=q, B=q)
    for kw in (dict(B=p), dict(B=g13.fp4_quantize(x[:, :60], "nvfp4")), dict(act="softmax"), dict(out_dtype="f64"),
               dict(bias=torch.zeros(4, device="cuda")), dict(bias=torch.zeros(5)), dict(bias=g.bfloat16().expand(5)),
               dict(residual=torch.zeros(5, 5)), dict(residual=torch.zeros(5, 6, device="cuda")),
               dict(residual=torch.zeros(1, 5, device="cuda").expand(5, 5)),
               dict(out=torch.zeros(5, 5, device="cuda").t()[:, :4]),
               dict(out=torch.zeros(5, 5, device="cuda", dtype=torch.float16))):
        with pytest.raises(E):
            c = dict(bad, **kw)
            g13.fp4_matmul(c.pop("A"), c.pop("B"), **c)
    with pytest.raises(E):
        g13.fp4_dequantize(q, out=torch.zeros(5, 71, device="cuda"))
    plan = g13.gemm_fp4_plan("nvfp4", 5, 5, 64, 5)
    with pytest.raises(E):
        g13.gemm_fp4_run(plan, q, q, x)


def test_stream_argument():
    # a stream or its handle: the same results, in order on that stream, whatever the current one does
    x = torch.randn(300, 640, device="cuda")
    w = g13.fp4_quantize(torch.randn(500, 640, device="cuda"), "nvfp4")
    want = g13.fp4_matmul(g13.fp4_quantize(x, "nvfp4"), w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        for _ in range(4):
            torch.randn(300, 500, device="cuda")  # allocations of the current stream in between
            q = g13.fp4_quantize(x, "nvfp4", stream=s)
            y = g13.fp4_matmul(q, w, stream=s)
            v = g13.fp4_dequantize(q, "bf16", stream=s)
        side.synchronize()
        assert torch.equal(y, want) and torch.equal(v, g13.fp4_dequantize(g13.fp4_quantize(x, "nvfp4"), "bf16"))


def test_misaligned_arrays_are_refused():
    # an address off its type is refused before anything is enqueued
    lib, M, N, K = g13.load(), 2, 32, 64
    q = [g13.fp4_quantize(torch.ones(r, K, device="cuda"), "nvfp4", tensor_scale=torch.ones(1, device="cuda"))
         for r in (M, N)]
    f = torch.zeros(M * N + 8, device="cuda").data_ptr()
    for out, size in (("f32", 4), ("bf16", 2)):
        pl = g13.gemm_fp4_plan("nvfp4", M, N, K, N, g13.Epilogue(b_layout="nk", out_dtype=out, bias=True,
                                                                residual=True, ldr=N))
        (ac, as_, ag), (bc, bs, bg) = q[0]._ptrs(), q[1]._ptrs()
        C = torch.empty(M * N + 8, dtype=DT[out], device="cuda")
        good = dict(ac=ac, as_=as_, ag=ag, bc=bc, bs=bs, bg=bg, C=C.data_ptr(), bias=f, res=f)
        off = dict(ac=8, as_=8, ag=2, bc=8, bs=4, bg=1, C=size // 2, bias=2, res=1)
        for k, d in off.items():
            a = dict(good, **{k: good[k] + d})
            assert lib.gemm_fp4_run(pl.handle, *a.values(), 1.0, None) == -3, k


@pytest.mark.parametrize("M", [1, 200])
def test_relu_of_nan_is_nan(M):
    A, B = (g13.fp4_quantize(torch.zeros(n, 64, device="cuda"), "nvfp4") for n in (M, 5))
    bias = torch.tensor([float("nan"), -1.0, 2.0, float("inf"), float("-inf")], device="cuda")
    want = torch.tensor([float("nan"), 0.0, 2.0, float("inf"), 0.0], device="cuda").expand(M, 5)
    assert torch.equal(g13.fp4_matmul(A, B, bias=bias, act="relu").nan_to_num(-7), want.nan_to_num(-7))
