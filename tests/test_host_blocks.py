"""CPU tests of the norm, 8-bit, 4-bit-weight and routing entry points: sizes, defaults, refusals, and the numpy references."""
import ctypes

import numpy as np
import pytest

import dense_gemm_13_gb300 as g13
from dense_gemm_13_gb300 import _build, blocks
from tests import blocks_ref as ref

OK, INVALID, UNSUPPORTED, MISALIGNED, BAD_PLAN, NO_DEVICE = 0, -1, -2, -3, -6, -7
P = 1 << 20  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return g13.load()


def no_gpu():
    import torch
    return not torch.cuda.is_available()


def test_exported_names():
    for name in blocks.__all__:
        assert name in g13.__all__ and getattr(g13, name) is getattr(blocks, name)


# ------------------------------------------------------------------ norm
def norm(lib, X=P, residual=P + (1 << 30), weight=P + (2 << 30), H=P + (3 << 30), Y=P + (4 << 30), scales=None, **kw):
    d = blocks._NormDesc()
    lib.gemm_norm_desc_init(ctypes.byref(d))
    for k, v in dict(dict(rows=4, cols=64, has_residual=1), **kw).items():
        setattr(d, k, v)
    return lib.gemm_rms_norm(ctypes.byref(d), X, residual, weight, H, Y, scales, None)


def test_norm_defaults(lib):
    d = blocks._NormDesc()
    lib.gemm_norm_desc_init(ctypes.byref(d))
    assert (d.dtype, d.residual_dtype, d.weight_dtype, d.out_dtype) == (2, 2, 2, 2)
    assert (d.has_residual, d.mxfp8, d.rows, d.ldx, d.weight_offset) == (0, 0, 0, 0, 0.0)
    assert d.eps == np.float32(1e-6)
    lib.gemm_norm_desc_init(None)


R = P + (1 << 30)


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(residual_dtype=-1), dict(weight_dtype=9), dict(out_dtype=4), dict(has_residual=2),
    dict(mxfp8=2), dict(rows=-1), dict(cols=0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(weight_offset=float("inf")), dict(residual_dtype=1), dict(dtype=0, residual_dtype=2), dict(ldx=63),
    dict(ldr=1), dict(ldh=63), dict(ldy=63), dict(scales=P), dict(mxfp8=1), dict(has_residual=0),
    dict(has_residual=0, residual=None), dict(X=None), dict(residual=None), dict(Y=None),
    # in place only with the same type and stride, and not both outputs at once
    dict(H=P, dtype=2, residual_dtype=0), dict(H=R, ldh=72), dict(H=P, ldx=72), dict(Y=P, out_dtype=0),
    dict(Y=R, ldy=80), dict(H=R, Y=R), dict(Y=P + (2 << 30)), dict(H=P + (2 << 30)),
    dict(mxfp8=1, scales=P + (5 << 30), Y=P), dict(mxfp8=1, scales=R), dict(mxfp8=1, scales=P + (4 << 30))], ids=str)
def test_norm_invalid(lib, kw):
    assert norm(lib, **kw) == INVALID


@pytest.mark.parametrize("kw,want", [
    (dict(cols=(1 << 22) + 1), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED), (dict(ldx=(1 << 40) + 1), UNSUPPORTED),
    (dict(mxfp8=1, scales=P, rows=1 << 30, cols=1 << 20), UNSUPPORTED), (dict(X=P + 1), MISALIGNED),
    (dict(residual=R + 1), MISALIGNED), (dict(weight=P + 1), MISALIGNED), (dict(H=P + 3), MISALIGNED),
    (dict(Y=P + 7), MISALIGNED), (dict(mxfp8=1, scales=P + 8, Y=P + 64), MISALIGNED),
    (dict(mxfp8=1, scales=P + 16, Y=P + 72), MISALIGNED),
    (dict(rows=0, X=None, residual=None, Y=None), OK)], ids=str)
def test_norm_other_refusals(lib, kw, want):
    assert norm(lib, **kw) == want


@pytest.mark.skipif(not no_gpu(), reason="would run")
def test_norm_valid_needs_a_device(lib):
    for kw in (dict(), dict(H=None), dict(H=R), dict(H=P), dict(Y=P), dict(weight=None), dict(cols=1 << 22),
               dict(mxfp8=1, scales=P + (5 << 30)), dict(has_residual=0, residual=None, H=None),
               dict(dtype=0, residual_dtype=0, weight_dtype=1, out_dtype=2), dict(rows=1, H=R, ldh=72)):
        assert norm(lib, **kw) == NO_DEVICE, kw
    assert lib.gemm_rms_norm(None, *[P] * 6, None) == INVALID


# ------------------------------------------------------------------ 8-bit floats
def test_fp8_sizes(lib):
    for cols in (0, 1, 31, 32, 33, 1000):
        assert lib.gemm_fp8_row_bytes(cols) == -(-cols // 32) * 32
    assert lib.gemm_fp8_row_bytes(-1) == lib.gemm_fp8_row_bytes(2 ** 63 - 1) == 0
    for rows, cols in ((0, 5), (1, 1), (128, 128), (129, 129), (1000, 3001)):
        assert lib.gemm_fp8_scales_bytes(rows, cols) == -(-rows // 128) * -(-cols // 128) * 512
        assert blocks._fp8_sizes(rows, cols) == (rows * lib.gemm_fp8_row_bytes(cols), lib.gemm_fp8_scales_bytes(rows, cols))
    assert lib.gemm_fp8_scales_bytes(-1, 10) == lib.gemm_fp8_scales_bytes(2 ** 62, 2 ** 62) == 0


@pytest.mark.parametrize("fn", ["gemm_fp8_quantize", "gemm_fp8_dequantize"])
def test_fp8_convert_refusals(lib, fn):
    def call(dtype=2, rows=4, cols=40, matrix=P, ld=40, codes=P, scales=P):
        if fn == "gemm_fp8_quantize":
            return lib.gemm_fp8_quantize(dtype, rows, cols, matrix, ld, codes, scales, None)
        return lib.gemm_fp8_dequantize(dtype, rows, cols, codes, scales, matrix, ld, None)

    for kw in (dict(dtype=3), dict(rows=-1), dict(cols=-1), dict(ld=39), dict(matrix=None), dict(codes=None),
               dict(scales=None)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(codes=P + 8), dict(scales=P + 1), dict(matrix=P + 1), dict(dtype=0, matrix=P + 2)):
        assert call(**kw) == MISALIGNED, kw
    assert call(rows=1 << 31) == call(cols=1 << 31, ld=1 << 31) == UNSUPPORTED
    assert call(rows=0, matrix=None, codes=None, scales=None) == OK
    assert call(cols=0, matrix=None, codes=None, scales=None) == OK


def test_fp8_plans(lib):
    def plan(M=4, N=40, K=64, ldc=40, **ep):
        h, e = ctypes.c_void_p(), g13.Epilogue(**dict(dict(b_layout="nk"), **ep))._c()
        return lib.gemm_fp8_plan(M, N, K, ldc, ctypes.byref(e), ctypes.byref(h))

    assert plan(M=-1) == plan(N=-1) == plan(K=-1) == plan(ldc=39) == INVALID
    assert plan(b_layout="kn") == plan(act="softmax") == plan(batch=2, stride_c=400) == UNSUPPORTED
    assert plan(N=1 << 30, ldc=1 << 30) == plan(M=1 << 31) == UNSUPPORTED
    assert lib.gemm_fp8_plan(4, 40, 64, 40, None, None) == INVALID
    h = ctypes.c_void_p()
    assert lib.gemm_fp8_plan(4, 40, 64, 40, None, ctypes.byref(h)) in (OK, NO_DEVICE)
    for bad in (None, 4096):
        assert lib.gemm_fp8_run(bad, P, P, P, P, P, None, None, 1.0, None) == BAD_PLAN
        assert lib.gemm_fp8_status(bad) == BAD_PLAN
        lib.gemm_fp8_destroy(bad)


def test_fp8_select_config():
    # the tile of the 4-bit product with the same number of stages: half the K
    for M, N, K in ((1, 6144, 6144), (20, 300, 1000), (1000, 3001, 4097), (8192, 8192, 8192)):
        a, b = g13.gemm_fp8_select_config(M, N, K), g13.gemm_fp4_select_config(M, N, 2 * K)
        assert (a.bn, a.split_k, a.bk) == (b.bn, b.split_k, 128)
    with pytest.raises(g13.GemmError):
        g13.gemm_fp8_select_config(-1, 1, 1)


# ------------------------------------------------------------------ 4-bit weights
def test_w4_sizes(lib):
    for n, k, g in ((0, 64, 32), (1, 1, 32), (16, 64, 64), (17, 65, 128), (1000, 3001, 96)):
        assert lib.gemm_w4_codes_bytes(n, k) == -(-n // 16) * -(-k // 64) * 512
        assert lib.gemm_w4_scales_count(n, k, g) == -(-n // 16) * 16 * -(-k // g)
        assert blocks._w4_sizes("", n, k, g) == (lib.gemm_w4_codes_bytes(n, k), lib.gemm_w4_scales_count(n, k, g))
    for n, k, g in ((-1, 64, 32), (4, 0, 32), (4, 64, 16), (4, 64, 33), (4, 65537, 32), ((1 << 28) + 1, 64, 32)):
        assert lib.gemm_w4_scales_count(n, k, g) == 0


def test_w4_convert_refusals(lib):
    def quant(dtype=2, sdt=2, N=4, K=40, g=32, src=P, ld=40, codes=P, scales=P, zeros=P):
        return lib.gemm_w4_quantize(dtype, sdt, N, K, g, src, ld, codes, scales, zeros, None)

    def deq(dtype=2, sdt=2, N=4, K=40, g=32, src=P, ld=40, codes=P, scales=P, zeros=P):
        return lib.gemm_w4_dequantize(dtype, sdt, N, K, g, codes, scales, zeros, src, ld, None)

    for call in (quant, deq):
        for kw in (dict(dtype=3), dict(sdt=0), dict(N=-1), dict(K=0), dict(g=0), dict(g=16), dict(g=48), dict(ld=39),
                   dict(src=None), dict(codes=None), dict(scales=None)):
            assert call(**kw) == INVALID, kw
        for kw in (dict(src=P + 1), dict(codes=P + 8), dict(scales=P + 2), dict(zeros=P + 1)):
            assert call(**kw) == MISALIGNED, kw
        assert call(K=65537, ld=65537) == call(N=1 << 29) == call(g=65568) == call(N=1 << 28, K=65536, ld=65536) \
            == UNSUPPORTED
        assert call(N=0, src=None, codes=None, scales=None) == OK

    def pack(N=4, K=40, g=32, q=P, ldq=40, s=P, lds=2, z=P, ldz=2, codes=P, scales=P, zeros=P):
        return lib.gemm_w4_pack(N, K, g, q, ldq, s, lds, z, ldz, codes, scales, zeros, None)

    for kw in (dict(ldq=39), dict(lds=1), dict(ldz=1), dict(z=None), dict(zeros=None), dict(q=None), dict(s=None),
               dict(codes=None), dict(scales=None)):
        assert pack(**kw) == INVALID, kw
    for kw in (dict(s=P + 1), dict(codes=P + 4), dict(scales=P + 2), dict(zeros=P + 8)):
        assert pack(**kw) == MISALIGNED, kw


def w4(lib, X=P, codes=P, scales=P, zeros=None, Y=P, bias=None, residual=None, **kw):
    d = blocks._W4Desc()
    lib.gemm_w4_desc_init(ctypes.byref(d))
    for k, v in dict(dict(M=4, N=40, K=64), **kw).items():
        setattr(d, k, v)
    return lib.gemm_w4_run(ctypes.byref(d), X, codes, scales, zeros, Y, bias, residual, 1.0, None)


def test_w4_run_refusals(lib):
    d = blocks._W4Desc()
    lib.gemm_w4_desc_init(ctypes.byref(d))
    assert (d.dtype, d.out_dtype, d.group, d.act, d.beta, d.has_zeros, d.ldx) == (2, 2, 128, 0, 1.0, 0, 0)
    lib.gemm_w4_desc_init(None)
    for kw in (dict(dtype=3), dict(out_dtype=-1), dict(act=7), dict(M=-1), dict(N=-1), dict(K=0), dict(group=40),
               dict(has_zeros=2), dict(has_zeros=1), dict(zeros=P), dict(has_bias=1), dict(bias=P), dict(residual=P),
               dict(has_residual=1), dict(ldx=63), dict(ldy=39), dict(has_residual=1, residual=P, ldr=39),
               dict(X=None), dict(codes=None), dict(scales=None), dict(Y=None)):
        assert w4(lib, **kw) == INVALID, kw
    for kw in (dict(dtype=0), dict(act=3), dict(M=65), dict(K=65537), dict(N=(1 << 28) + 1), dict(ldx=1 << 41)):
        assert w4(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(X=P + 1), dict(codes=P + 8), dict(scales=P + 2), dict(zeros=P + 1, has_zeros=1), dict(Y=P + 1),
               dict(bias=P + 2, has_bias=1), dict(residual=P + 1, has_residual=1)):
        assert w4(lib, **kw) == MISALIGNED, kw
    assert w4(lib, M=0, X=None, codes=None, scales=None, Y=None) == OK
    assert w4(lib, N=0, X=None, codes=None, scales=None, Y=None) == OK
    assert lib.gemm_w4_run(None, P, P, P, None, P, None, None, 1.0, None) == INVALID
    if no_gpu():
        for kw in (dict(), dict(M=64, K=65536, N=1 << 20), dict(zeros=P, has_zeros=1), dict(group=65536)):
            assert w4(lib, **kw) == NO_DEVICE, kw


# ------------------------------------------------------------------ routing
def route(lib, logits=P, bias=None, ids=P, weights=P, **kw):
    d = blocks._RouteDesc()
    lib.gemm_route_desc_init(ctypes.byref(d))
    for k, v in dict(dict(T=4, E=64, top_k=6), **kw).items():
        setattr(d, k, v)
    return lib.gemm_route(ctypes.byref(d), logits, bias, ids, weights, None)


def test_route_refusals(lib):
    d = blocks._RouteDesc()
    lib.gemm_route_desc_init(ctypes.byref(d))
    assert (d.dtype, d.scores, d.groups, d.top_groups, d.group_score, d.normalize, d.scale) == (0, 0, 1, 1, 0, 1, 1.0)
    lib.gemm_route_desc_init(None)
    for kw in (dict(dtype=3), dict(scores=2), dict(group_score=-1), dict(normalize=2), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(T=-1), dict(E=0), dict(top_k=0), dict(top_k=65), dict(groups=0),
               dict(top_groups=0), dict(groups=5, top_groups=2), dict(groups=8, top_groups=9),
               dict(groups=8, top_groups=1, top_k=9), dict(groups=128), dict(ld=63), dict(logits=None), dict(ids=None),
               dict(weights=None)):
        assert route(lib, **kw) == INVALID, kw
    for kw in (dict(E=513), dict(E=512, top_k=33), dict(E=512, groups=64, top_groups=2), dict(T=(1 << 40) + 1),
               dict(ld=(1 << 20) + 1)):
        assert route(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(logits=P + 2), dict(dtype=2, logits=P + 1), dict(bias=P + 1), dict(ids=P + 2), dict(weights=P + 1)):
        assert route(lib, **kw) == MISALIGNED, kw
    assert route(lib, T=0, logits=None, ids=None, weights=None) == OK
    assert lib.gemm_route(None, P, None, P, P, None) == INVALID
    if no_gpu():
        for kw in (dict(), dict(E=512, top_k=32, groups=32, top_groups=32), dict(E=1, top_k=1), dict(bias=P)):
            assert route(lib, **kw) == NO_DEVICE, kw


def test_moe_run_routed_bad_plans(lib):
    for h in (None, 4096):
        assert lib.gemm_moe_run_routed(h, *[256] * 7, None) == BAD_PLAN


# ------------------------------------------------------------------ the references themselves
def test_ref_mxfp8():
    assert ref.E4M3[126] == 448 and ref.E4M3[8] == 2.0 ** -6 and ref.E4M3[1] == 2.0 ** -9
    for top, byte in ((448.0, 127), (np.nextafter(448.0, 449), 128), (896.0, 128), (449.0, 128), (224.0, 126), (0.0, 0),
                      (1.0, 119), (1.75, 119), (1.7500001, 120), (2.0 ** -149, 0)):
        assert ref.mxfp8_scale(np.array([top]))[0] == byte, top
    assert list(ref.e4m3_code(np.array([0, 2.0 ** -10, 1.5 * 2.0 ** -9, 1.0625, 1.1875, 447, 448]))) == \
        [0, 0, 2, 56, 58, 126, 126]
    r = np.random.default_rng(0)
    x = r.standard_normal((5, 70)) * np.exp2(r.integers(-20, 20, (5, 70)))
    code, byte = ref.mxfp8(x)
    v, d = ref.mxfp8_values(code, byte), np.repeat(np.exp2(byte.astype(float) - 127), 32, 1)[:, :70]
    assert (np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, d * 2.0 ** -10)).all()


def test_ref_w4_layout():
    # every element has a place of its own
    n, k = 40, 130
    seen = np.zeros((n, k), int)
    for r in range(0, n, 13):
        for c in range(k):
            q = np.zeros((n, k), np.uint8)
            q[r, c] = 15
            w = ref.w4_words(q)
            at = np.nonzero(w)[0]
            assert len(at) == 1
            seen[r, c] = at[0] * 2 + (w[at[0]] == 0xF0)
    used = seen[::13].reshape(-1)
    assert len(set(used)) == len(used)
    e = ref.w4_entries(np.arange(1, n * 3 + 1).reshape(n, 3))
    assert sorted(e[e > 0]) == list(range(1, n * 3 + 1)) and len(e) == 48 * 3


def test_ref_route():
    z = np.array([[1.0, 3.0, 3.0, np.nan, 2.0, 0.0]])
    assert list(ref.route(z, 5, scores="sigmoid", normalize=False)[0][0]) == [1, 2, 4, 0, 5]
    z = np.array([[0.0, 5.0, 4.0, 4.0, 1.0, 1.0]])
    ids, w = ref.route(z, 2, groups=3, top_groups=1, group_score="max", scale=2.0)
    assert list(ids[0]) == [1, 0] and abs(w.sum() - 2) < 1e-12
    ids, _ = ref.route(z, 2, scores="sigmoid", groups=3, top_groups=1, group_score="top2")
    assert list(ids[0]) == [2, 3]


def test_w4_run_flags(lib):
    # the test flag only
    for flags in (1, g13.FLAG_TEST_STALL_PEER, g13.FLAG_TEST_STALL | 2):
        assert w4(lib, flags=flags) == INVALID
    d = blocks._W4Desc(flags=7, timeout_ms=7)
    lib.gemm_w4_desc_init(ctypes.byref(d))
    assert (d.flags, d.timeout_ms) == (0, 0)
    assert w4(lib, flags=g13.FLAG_TEST_STALL, timeout_ms=5, M=0) == OK
