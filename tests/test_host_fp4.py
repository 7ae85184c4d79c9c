"""CPU tests of the 4-bit entry points: sizes, refusals, the choice of tile, and the numpy reference itself."""
import ctypes

import numpy as np
import pytest

import dense_gemm_13_gb300 as g13
from dense_gemm_13_gb300 import _build
from tests import fp4_ref as ref

INVALID, UNSUPPORTED, MISALIGNED = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return g13.load()


def test_sizes(lib):
    for cols in (0, 1, 31, 32, 33, 64, 1000):
        assert lib.gemm_fp4_row_bytes(cols) == -(-cols // 32) * 16
    assert lib.gemm_fp4_row_bytes(-1) == 0
    for fmt, f in g13.FP4_FORMATS.items():
        for rows, cols in ((0, 5), (1, 1), (128, 64), (129, 65), (1000, 3001)):
            nb = -(-cols // ref.BLOCK[fmt])
            assert lib.gemm_fp4_scales_bytes(f, rows, cols) == -(-rows // 128) * -(-nb // 4) * 512
    assert lib.gemm_fp4_scales_bytes(7, 10, 10) == 0
    assert lib.gemm_fp4_scales_bytes(0, -1, 10) == 0
    assert lib.gemm_fp4_scales_bytes(0, 2 ** 62, 2 ** 62) == 0 and lib.gemm_fp4_row_bytes(2 ** 63 - 1) == 0


P = 1 << 20  # an aligned address that no refused call reads


@pytest.mark.parametrize("fn", ["gemm_fp4_quantize", "gemm_fp4_dequantize"])
def test_convert_refusals(lib, fn):
    def call(fmt=1, dtype=2, rows=4, cols=40, matrix=P, ld=40, g=P, codes=P, scales=P):
        if fn == "gemm_fp4_quantize":
            return lib.gemm_fp4_quantize(fmt, dtype, rows, cols, matrix, ld, g, codes, scales, None)
        return lib.gemm_fp4_dequantize(fmt, dtype, rows, cols, codes, scales, g, matrix, ld, None)

    for kw in (dict(fmt=2), dict(fmt=-1), dict(dtype=3), dict(rows=-1), dict(cols=-1), dict(ld=39), dict(matrix=None),
               dict(codes=None), dict(scales=None), dict(fmt=0, g=P)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(codes=P + 8), dict(scales=P + 1), dict(matrix=P + 1), dict(dtype=0, matrix=P + 2), dict(g=P + 2)):
        assert call(**kw) == MISALIGNED, kw
    assert call(rows=1 << 31) == UNSUPPORTED
    assert call(cols=1 << 31, ld=1 << 31) == UNSUPPORTED
    assert call(rows=1 << 26, cols=1 << 26, ld=1 << 26) == UNSUPPORTED
    assert call(rows=0, matrix=None, codes=None, scales=None) == 0
    assert call(cols=0, matrix=None, codes=None, scales=None) == 0


def test_plan_refusals(lib):
    def plan(fmt=1, M=4, N=40, K=64, ldc=40, ep=None):
        h = ctypes.c_void_p()
        e = (ep or g13.Epilogue(b_layout="nk"))._c()
        return lib.gemm_fp4_plan(fmt, M, N, K, ldc, ctypes.byref(e), ctypes.byref(h))

    E = g13.Epilogue
    for kw in (dict(fmt=2), dict(M=-1), dict(N=-1), dict(K=-1), dict(ldc=39),
               dict(ep=E(b_layout="nk", residual=True, ldr=39)), dict(ep=E(b_layout="nk", batch=-1))):
        assert plan(**kw) == INVALID, kw
    for kw in (dict(ep=E(b_layout="kn")), dict(ep=E(b_layout="nk", act="softmax")), dict(ep=E(b_layout="nk", batch=2)),
               dict(M=1 << 31), dict(K=1 << 31), dict(M=1 << 30, N=1 << 30, ldc=1 << 30)):
        assert plan(**kw) == UNSUPPORTED, kw
    assert lib.gemm_fp4_plan(1, 4, 40, 64, 40, None, None) == INVALID
    assert plan() in (0, -7)
    assert plan(M=0) in (0, -7)


def test_bad_plans(lib):
    for h in (None, 12345):
        assert lib.gemm_fp4_run(h, P, P, None, P, P, None, P, None, None, 1.0, None) == -6
        assert lib.gemm_fp4_status(h) == -6
        lib.gemm_fp4_destroy(h)


def test_tile_choice(lib):
    c = g13.gemm_fp4_select_config
    # tokens per tile: the narrowest that holds them, and both sides of each border
    for M, bn in ((1, 16), (16, 16), (17, 32), (32, 32), (33, 64), (64, 64), (65, 128), (128, 128)):
        assert c(M, 6144, 6144).bn == bn, M
    for M, N, K in ((1, 128, 64), (1, 1, 256), (0, 5, 1000), (5, 0, 1000), (5, 5, 0)):
        assert c(M, N, K).split_k == 1, (M, N, K)
    held = {1: 152, 2: 76, 4: 36, 8: 15}  # clusters that run at a time
    for M in (1, 20, 60, 100):
        for N in (1, 128, 1000, 6144, 152 * 128, 153 * 128):
            for K in (300, 600, 6144):
                f = c(M, N, K)
                tiles = -(-N // 128) * -(-M // f.bn)
                s = f.split_k
                assert s in held and s <= -(-K // 256), (M, N, K)
                assert s == 1 or tiles <= held[s], (M, N, K)
                if M <= 64 and s < 8 and 2 * s <= -(-K // 256):
                    assert tiles > held[2 * s], (M, N, K)
    # pairs where one wave of them replaces two of 128 x 128, or fills the GPU; not where they leave most of it idle
    assert c(8192, 8192, 8192).bn == 256 and c(8192, 8192, 8192).variant == 2 and c(8192, 8192, 8192).bm == 256
    assert c(1000, 3001, 4097).bn == 256 and c(512, 6144, 6144).bn == 256
    assert c(200, 300, 770).bn == 128 and c(128, 6144, 6144).bn == 128
    with pytest.raises(g13.GemmError):
        c(-1, 1, 1)


def test_python_refusals(lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64)
    for bad in (x, x[0], x.double()):  # on the CPU, 1-D, FP64
        with pytest.raises(g13.GemmError, match="fp4_quantize"):
            g13.fp4_quantize(bad)
    with pytest.raises(g13.GemmError, match="unknown format"):
        g13.fp4_quantize(x, "fp4")
    codes, scales = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    with pytest.raises(g13.GemmError, match="on the GPU"):
        g13.Fp4Tensor(codes, scales, 4, 64, "nvfp4")
    with pytest.raises(g13.GemmError, match="unknown format"):
        g13.Fp4Tensor(codes, scales, 4, 64, "int4")


# ------------------------------------------------------------------ the reference
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_reference_brute_force(fmt):
    r = np.random.default_rng(3)
    x = (r.standard_normal((9, 50)) * np.exp2(r.integers(-6, 6, (9, 50)))).astype(np.float32)
    code, byte = ref.quantise(x, fmt)
    d = np.repeat(ref.scale_value(byte, fmt, 1.0), ref.BLOCK[fmt], 1)[:, :50]
    # no other code is nearer
    dist = np.abs(x[..., None] / d[..., None] - ref.E2M1)
    near = np.take_along_axis(dist, code[..., None].astype(int), 2)[..., 0]
    # (the quotient is rounded to FP32 first: both distances are off by at most 2^-24 |x / d|)
    assert (near <= dist.min(-1) + 2 * 2.0 ** -24 * np.abs(x / d)).all()
    # the scale leaves the block's largest inside the format: below twice its largest value (mxfp4), or
    # half a step of E4M3 beyond it, 2^-4 of a normal scale (nvfp4)
    top = np.abs(x / d)
    if fmt == "mxfp4":
        assert top.max() < 8
    else:
        assert top[np.repeat(byte >= 8, 16, 1)[:, :50]].max() <= 6 / (1 - 2.0 ** -4)


def test_reference_layout():
    byte = np.arange(130 * 5, dtype=np.uint32).reshape(130, 5).astype(np.uint8)
    t = ref.tiles(byte)
    assert t.size == 2 * 2 * 512
    assert t[0] == byte[0, 0] and t[1] == byte[0, 1] and t[16] == byte[1, 0] and t[4] == byte[32, 0]
    assert t[512] == byte[0, 4] and t[1024 + 16] == byte[129, 0] and t[513] == 0
    assert ref.pack(np.array([[1, 2, 3]], np.uint8)).tolist() == [[0x21, 3] + [0] * 14]


@pytest.mark.parametrize("M,N,K", [(1 << 31, 40, 64), (4, 1 << 30, 64), (4, 40, 1 << 31), (1 << 29, 1 << 29, 64),
                                   (1 << 62, 1 << 62, 1 << 62), ((1 << 63) - 1, 1, 1)])
def test_tile_choice_of_sizes_that_no_plan_takes(lib, M, N, K):
    # refused with the plan's code, before any of them is multiplied
    c, h = g13._Config(), ctypes.c_void_p()
    assert lib.gemm_fp4_select_config(M, N, K, 152, ctypes.byref(c)) == UNSUPPORTED
    assert lib.gemm_fp4_plan(1, M, N, K, N, None, ctypes.byref(h)) == UNSUPPORTED
