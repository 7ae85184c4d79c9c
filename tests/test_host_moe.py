"""CPU tests of the mixture-of-experts entry points: refusals, and the numpy reference against a plain loop."""
import ctypes

import numpy as np
import pytest

import dense_gemm_13_gb300 as g13
from dense_gemm_13_gb300 import _build
from tests import moe_ref


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return g13.load()


def plan(lib, **kw):
    d, h = g13._MoeDesc(), ctypes.c_void_p()
    lib.gemm_moe_desc_init(ctypes.byref(d))
    for k, v in dict(dict(T=4, E=8, top_k=2, H=64, I=32), **kw).items():
        setattr(d, k, v)
    return lib.gemm_moe_plan(ctypes.byref(d), ctypes.byref(h))


def test_defaults(lib):
    d = g13._MoeDesc()
    lib.gemm_moe_desc_init(ctypes.byref(d))
    assert (d.dtype, d.act, d.normalize, d.ldx, d.flags, d.timeout_ms) == (2, 2, 1, 0, 0, 0)
    lib.gemm_moe_desc_init(None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(E=0), dict(H=0), dict(I=0), dict(top_k=0), dict(top_k=9),
                                dict(dtype=7), dict(act=3), dict(act=-1), dict(normalize=2), dict(ldx=63),
                                dict(ld_router=63), dict(ld_w1=63), dict(ld_w2=31), dict(ldy=63),
                                dict(stride_w1=-1), dict(stride_w2=-1), dict(ldx=-5)], ids=str)
def test_invalid(lib, kw):
    assert plan(lib, **kw) == -1


@pytest.mark.parametrize("kw", [dict(dtype=0), dict(T=65), dict(E=513), dict(E=512, top_k=33), dict(H=16385),
                                dict(I=(1 << 20) + 1),
                                dict(T=64, E=512, top_k=32, H=16384, I=1 << 20), dict(ldx=(1 << 40) + 1), dict(stride_w1=1 << 53)], ids=str)
def test_unsupported(lib, kw):
    assert plan(lib, **kw) == -2


def test_valid_needs_a_device(lib):
    for kw in (dict(), dict(T=0), dict(T=64, E=512, top_k=32, H=16384, I=1 << 15), dict(dtype=1, act=0, normalize=0)):
        assert plan(lib, **kw) in (0, -7), kw
    assert lib.gemm_moe_plan(None, None) == -1
    h = ctypes.c_void_p()
    assert lib.gemm_moe_plan(None, ctypes.byref(h)) == -1


def test_bad_plans(lib):
    for h in (None, 4096):
        assert lib.gemm_moe_run(h, *[256] * 5, None, None, 256, None) == -6
        assert lib.gemm_moe_status(h) == -6
        assert lib.gemm_moe_workspace_bytes(h) == 0
        lib.gemm_moe_destroy(h)


def test_python_refusals(lib):
    torch = pytest.importorskip("torch")
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    good = (z(2, 8), z(4, 8), z(4, 12, 8), z(4, 8, 6))
    for bad, why in (((z(2, 8, dt=torch.float32),) + good[1:], "FP16 or BF16"),
                     ((z(8),) + good[1:], "are wanted"),
                     (good[:2] + (z(4, 6, 8), good[3]), "do not fit"),
                     ((good[0], z(4, 8, dt=torch.float16)) + good[2:], "dtype on x's device"),
                     (good, "dtype on x's device")):  # on the CPU
        with pytest.raises(g13.GemmError, match=why):
            g13.moe_layer(*bad, 2)
    with pytest.raises(g13.GemmError, match="act"):
        g13.moe_layer(*good, 2, act="tanh")


@pytest.mark.parametrize("act", ["gelu", "relu", "swiglu"])
def test_reference(act):
    from math import erf, exp, sqrt
    r = np.random.default_rng(1)
    T, E, k, H, I = 3, 5, 2, 7, 4
    rows = 2 * I if act == "swiglu" else I
    x, wr, w1, w2 = (r.standard_normal(s) for s in ((T, H), (E, H), (E, rows, H), (E, H, I)))
    y, bound, ids, w, gap = moe_ref.layer(x, wr, w1, w2, k, act, False, 2.0 ** -9)
    for t in range(T):
        z = [sum(x[t, i] * wr[e, i] for i in range(H)) for e in range(E)]
        p = [exp(v) / sum(exp(q) for q in z) for v in z]
        best = sorted(range(E), key=lambda e: (-z[e], e))[:k]
        assert ids[t].tolist() == best
        want = np.zeros(H)
        for e in best:
            a = w1[e] @ x[t]
            if act == "swiglu":
                h = [a[i] / (1 + exp(-a[i])) * a[I + i] for i in range(I)]
            else:
                h = [max(v, 0) if act == "relu" else 0.5 * v * (1 + erf(v / sqrt(2))) for v in a]
            want += p[e] * (w2[e] @ np.array(h))
        assert np.allclose(y[t], want, rtol=1e-12, atol=1e-13)
    assert (bound > 0).all() and gap > 0


@pytest.mark.parametrize("flags", [0x1, 0x2, g13.FLAG_TEST_STALL_PEER, g13.FLAG_TEST_STALL | 0x10, 0x7FFFFFFF])
def test_flags_that_mean_nothing_are_refused(lib, flags):
    assert plan(lib, flags=flags) == -1
    assert plan(lib, flags=g13.FLAG_TEST_STALL) in (0, -7)
