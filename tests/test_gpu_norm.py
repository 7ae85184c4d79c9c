"""The root-mean-square norm on the GPU against 64 bits: 16- and 32-bit outputs, mxfp8, in place, streams, graphs.

Tolerance of y, relative, u = 2^-24: a thread adds at most C squares (32, or a 512th of a long row and eight more)
and the row's join has at most ten further additions, so the sum is off by (C + 11) u and its root by half that; rsqrtf
by 2 units (4 u); sum / cols, + eps, weight + offset and the two products round once each: 5 u and one to spare.  Then
half a step of the output's type.  In mxfp8 y is within 4 u of the formula, and the code has to be that of a value
within that of it.
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


def tensor(r, dtype, *shape, std=1.0):
    return torch.from_numpy((r.standard_normal(shape) * std).astype(np.float32)).to(DT[dtype]).cuda()


def rel_tol(H):
    return (0.5 * (max(32, H / 512 + 8) + 11) + 10) * 2.0 ** -24


def stream_of(x, r):
    """h as the library has to round it, and its 64-bit values."""
    h = x if r is None else (x.float() + r.float()).to(r.dtype)
    return h, h.double().cpu().numpy()


def check_values(y, h64, w, eps, offset, out):
    want = ref.rms_norm(h64, None if w is None else w.double().cpu().numpy(), eps, offset)
    tol = np.abs(want) * (rel_tol(h64.shape[1]) + torch.finfo(DT[out]).eps / 2) + torch.finfo(DT[out]).smallest_normal
    err = np.abs(y.double().cpu().numpy() - want)
    assert y.dtype == DT[out] and (err <= tol).all(), f"max err/tol {np.max(err / tol):.3g}"


def check_fp8(q, h64, w, eps, offset):
    y = ref.rms_norm(h64, None if w is None else w.double().cpu().numpy(), eps, offset)
    rows, cols = y.shape
    d = 2.0 ** -22
    pad = np.zeros((rows, -(-cols // 32) * 32))
    pad[:, :cols] = np.abs(y)
    top = pad.reshape(rows, -1, 32).max(2)
    nb = top.shape[1]
    got_tiles = q.scales.cpu().numpy()
    rr, cc = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    byte = got_tiles[((rr // 128) * -(-nb // 4) + cc // 4) * 512 + (rr % 32) * 16 + (rr % 128) // 32 * 4 + cc % 4]
    assert np.array_equal(got_tiles, ref.tiles(byte)), "padding of the scales"
    lo, hi = ref.mxfp8_scale(top * (1 - d)), ref.mxfp8_scale(top * (1 + d))
    assert ((byte == lo) | (byte == hi)).all()
    codes = q.codes.cpu().numpy()
    assert (codes[:, cols:] == 0).all(), "padding of the codes"
    v = np.abs(y) * np.repeat(np.exp2(127.0 - byte), 32, 1)[:, :cols]
    clo, chi = ref.e4m3_code(np.minimum(v * (1 - d), 448)), ref.e4m3_code(np.minimum(v * (1 + d), 448))
    mag = codes[:, :cols] & 127
    assert ((mag >= clo) & (mag <= chi)).all(), f"{np.sum((mag < clo) | (mag > chi))} codes"
    assert ((codes[:, :cols] >= 128) == np.signbit(y))[mag > 0].all()
    # the values that are read back are the codes'
    assert np.array_equal(g13.fp8_dequantize(q).cpu().numpy(), ref.mxfp8_values(codes[:, :cols], byte).astype(np.float32))


# lengths on either side of every way that a row is split, long rows among them
COLS = [1, 7, 8, 31, 33, 64, 65, 100, 128, 129, 256, 264, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096, 4097, 4104,
        8192, 8200, 16384, 16392, 16385, 40000]
KINDS = [("bf16", "none", "bf16", "bf16"), ("bf16", "bf16", "bf16", "bf16"), ("f16", "f32", "f16", "f16"),
         ("f32", "f32", "f32", "f32"), ("f32", "none", "bf16", "bf16"), ("bf16", "f32", "f32", "f16"),
         ("f16", "f16", "none", "f32")]


@pytest.mark.parametrize("H", COLS)
@pytest.mark.parametrize("T", [1, 5, 400])
def test_norm(T, H):
    for dtype, res, wdt, out in KINDS:
        r = rng(T, H, dtype, res)
        x = tensor(r, dtype, T, H)
        w = None if wdt == "none" else tensor(r, wdt, H)
        rs = None if res == "none" else tensor(r, res, T, H, std=3.0)
        h, h64 = stream_of(x, rs)
        got = g13.rms_norm(x, w, residual=rs, out_dtype=out)
        y = got if rs is None else got[0]
        if rs is not None:
            assert torch.equal(got[1], h), "the residual stream"
        check_values(y, h64, w, 1e-6, 0.0, out)
        if (dtype, res) in (("bf16", "bf16"), ("f16", "f32"), ("f32", "none")):
            got = g13.rms_norm(x, w, residual=rs, out_dtype="mxfp8")
            if rs is not None:
                assert torch.equal(got[1], h)
            check_fp8(got if rs is None else got[0], h64, w, 1e-6, 0.0)


@pytest.mark.parametrize("H", [72, 1000, 5000, 20000])
def test_offset_and_eps(H):
    r = rng("offset", H)
    x, w = tensor(r, "bf16", 9, H, std=1e-3), tensor(r, "bf16", H)
    _, h64 = stream_of(x, None)
    for eps, offset in ((1e-5, 1.0), (0.0, 0.0), (0.5, -2.0)):
        check_values(g13.rms_norm(x, w, eps=eps, weight_offset=offset), h64, w, float(np.float32(eps)), offset, "bf16")
        check_fp8(g13.rms_norm(x, w, eps=eps, weight_offset=offset, out_dtype="mxfp8"), h64, w,
                  float(np.float32(eps)), offset)


@pytest.mark.parametrize("H", [40, 256, 3000, 17000])
def test_strides_and_offsets(H):
    # rows inside larger ones at every kind of alignment; what lies around them stays
    r = rng("strides", H)
    for left, right in ((8, 8), (1, 3), (0, 5), (4, 4)):
        W, T = H + left + right, 6
        x, rs = tensor(r, "bf16", T, W)[:, left: left + H], tensor(r, "f32", T, W)[:, left: left + H]
        w = tensor(r, "bf16", W)[left: left + H]
        room_y, room_h = (torch.full((T + 2, W), 7.0, dtype=d, device="cuda") for d in (torch.bfloat16, torch.float32))
        y, h = room_y[1:-1, left: left + H], room_h[1:-1, left: left + H]
        g13.rms_norm(x, w, residual=rs, out=y, residual_out=h)
        want, h64 = stream_of(x, rs)
        assert torch.equal(h, want)
        check_values(y, h64, w, 1e-6, 0.0, "bf16")
        check_fp8(g13.rms_norm(x, w, residual=rs, out_dtype="mxfp8")[0], h64, w, 1e-6, 0.0)
        y[:], h[:] = 7, 7
        assert bool((room_y == 7).all()) and bool((room_h == 7).all()), "store outside the rows"


@pytest.mark.parametrize("H", [3, 9, 200, 1001, 4097, 8185, 8191, 16377, 16383])
@pytest.mark.parametrize("lds", [(0, 0, 0, 0), (1, 9, 17, 1), (1, 2, 3, 4), (7, 3, 7, 7)])
def test_rows_off_16_bytes(H, lds):
    # row strides that agree modulo eight and some that do not, from an odd first element; every other row, and what
    # lies between the rows, holds NaN, which stays where it is
    T, r = 7, rng("off", H, lds)
    for dtype, res, out, left in (("bf16", "bf16", "bf16", 0), ("f16", "f32", "f16", 5), ("f32", "f32", "f32", 3)):
        def room(name, ld, fill=None):
            flat = torch.full((left + T * (H + ld),), float("nan") if fill is None else fill, device="cuda").to(DT[name])
            rows = torch.as_strided(flat, (T, H), (H + ld, 1), left)
            if fill is None:
                rows[::2] = tensor(r, name, 4, H)
            return flat, rows
        (_, x), (_, rs) = room(dtype, lds[0]), room(res, lds[1])
        (fh, h), (fy, y) = room(res, lds[2], 7.0), room(out, lds[3], 7.0)
        w = tensor(r, dtype, H)
        g13.rms_norm(x, w, residual=rs, out=y, residual_out=h)
        want, h64 = stream_of(x, rs)
        assert torch.equal(h[::2], want[::2]) and bool(torch.isnan(h[1::2]).all()) and bool(torch.isnan(y[1::2]).all())
        check_values(y[::2], h64[::2], w, 1e-6, 0.0, out)
        q = g13.rms_norm(x, w, residual=rs, out_dtype="mxfp8")[0]
        good = g13.rms_norm(x[::2], w, residual=rs[::2], out_dtype="mxfp8")[0]
        assert torch.equal(q.codes[::2], good.codes)
        check_fp8(good, h64[::2], w, 1e-6, 0.0)
        h[:], y[:] = 7, 7
        assert bool((fh == 7).all()) and bool((fy == 7).all()), "store outside the rows"


@pytest.mark.parametrize("H", [96, 4096, 4097, 18000])
def test_in_place(H):
    r = rng("place", H)
    x, rs, w = tensor(r, "bf16", 300, H), tensor(r, "bf16", 300, H), tensor(r, "bf16", H)
    y, h = g13.rms_norm(x, w, residual=rs)
    for _ in range(2):
        a, b = x.clone(), rs.clone()
        y2, h2 = g13.rms_norm(a, w, residual=b, residual_out=b)  # the stream in its own place
        assert h2 is b and torch.equal(h2, h) and torch.equal(y2, y) and torch.equal(a, x)
        a, b = x.clone(), rs.clone()
        y2, h2 = g13.rms_norm(a, w, residual=b, residual_out=b, out=a)  # and y in x's
        assert y2 is a and torch.equal(a, y) and torch.equal(b, h)
        a, b = x.clone(), rs.clone()
        y2, h2 = g13.rms_norm(a, w, residual=b, residual_out=a, out=b)  # crossed
        assert torch.equal(a, h) and torch.equal(b, y)
        a, b = x.clone(), rs.clone()
        q, h2 = g13.rms_norm(a, w, residual=b, residual_out=b, out_dtype="mxfp8")
        assert torch.equal(b, h)
        assert torch.equal(q.codes, g13.rms_norm(x, w, residual=rs, out_dtype="mxfp8")[0].codes)


def test_special_rows():
    H = 200
    x = torch.randn(140, H, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    x[1], x[2, 5], x[3, 7], x[4] = 0, float("nan"), float("inf"), 1e-30
    x[131, 40] = float("-inf")
    bad = [2, 3, 131]
    y = g13.rms_norm(x)
    assert bool((y[1] == 0).all()) and bool(torch.isnan(y[2]).all())
    assert bool(torch.isnan(y[3, 7])) and bool((y[3, :7] == 0).all())
    q = g13.rms_norm(x, out_dtype="mxfp8")
    v = g13.fp8_dequantize(q)
    assert bool(torch.isnan(v[2]).all())
    for row, at in ((3, 7), (131, 40)):
        b = at // 32 * 32
        assert bool(torch.isnan(v[row, b: b + 32]).all())
        assert bool((v[row, :b] == 0).all()) and bool((v[row, b + 32:] == 0).all())
    rest = [i for i in range(140) if i not in bad]
    h64 = x[rest].double().cpu().numpy()
    check_values(y[rest], h64, None, 1e-6, 0.0, "f32")
    assert torch.allclose(v[rest].double(), y[rest].double(), rtol=2 ** -4, atol=float(y[rest].abs().max()) * 2 ** -15)
    assert bool(torch.isfinite(v[rest]).all())
    # eps = 0 and a row of zeros: 0 / 0
    assert bool(torch.isnan(g13.rms_norm(x[1:2], eps=0.0)).all())
    # the padding of a NaN row's codes and scales stays zero
    q = g13.rms_norm(torch.full((3, 40), float("nan"), device="cuda"), out_dtype="mxfp8")
    assert bool((q.codes[:, 40:] == 0).all())
    s = q.scales.view(32, 4, 4)
    assert bool((s[:3, 0, :2] == 255).all()) and int((s != 0).sum()) == 6


def test_rows_far_apart():
    # offsets beyond 2^31 elements
    big = torch.empty(2 ** 31 + 5000, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((2, 1000), (2 ** 31 + 8, 1))
    x.copy_(torch.randn(2, 1000))
    _, h64 = stream_of(x, None)
    check_values(g13.rms_norm(x), h64, None, 1e-6, 0.0, "bf16")


def test_many_rows():
    x = torch.randn(200001, 72, device="cuda", dtype=torch.bfloat16)
    y = g13.rms_norm(x)
    for part in (x[:100], x[99990:100100], x[-100:]):
        at = (part.data_ptr() - x.data_ptr()) // (72 * 2)
        assert torch.equal(y[at: at + len(part)], g13.rms_norm(part.contiguous()))
    q = g13.rms_norm(x, out_dtype="mxfp8")
    assert torch.equal(q.codes[-100:], g13.rms_norm(x[-100:], out_dtype="mxfp8").codes)


def test_empty_and_refusals():
    assert tuple(g13.rms_norm(torch.zeros(0, 8, device="cuda")).shape) == (0, 8)
    assert g13.rms_norm(torch.zeros(0, 8, device="cuda"), out_dtype="mxfp8").rows == 0
    x = torch.randn(4, 64, device="cuda")
    w, b = torch.ones(64, device="cuda"), torch.zeros(8, 64, device="cuda")
    E = g13.GemmError
    for args, kw in (((x.cpu(),), {}), ((x.double(),), {}), ((x[0],), {}), ((x.t(),), {}), ((x[:, :0],), {}),
                     ((x[:1].expand(4, 64),), {}), ((x, w[:60]), {}), ((x, w.cpu()), {}), ((x, w.double()), {}),
                     ((x, b[:, 0]), {}), ((x, w), dict(residual=x.bfloat16())), ((x, w), dict(residual=x[:3])),
                     ((x, w), dict(residual=x.cpu())), ((x, w), dict(residual_out=x.clone())),
                     ((x, w), dict(residual=x.clone(), residual_out=x.bfloat16())), ((x, w), dict(out_dtype="e4m3")),
                     ((x, w), dict(out=x.bfloat16())), ((x, w), dict(out=x[:3])),
                     ((x, w), dict(out_dtype="mxfp8", out=x.clone())), ((x, w), dict(eps=-1.0)),
                     ((x, w), dict(eps=float("nan"))), ((x, w), dict(weight_offset=float("inf"))),
                     # outputs that overlap other than in place
                     ((b[:4], w), dict(out=b[1:5])), ((b[:4], w), dict(residual=x, residual_out=b[2:6])),
                     ((x, w), dict(residual=b[:4], residual_out=b[4:], out=b[4:])),
                     ((x, b[7]), dict(out=b[4:])), ((x, b[7]), dict(residual=x.clone(), residual_out=b[4:])),
                     ((b[:4].bfloat16(), w), dict(residual=b[:4], residual_out=b[1:5]))):
        with pytest.raises(E):
            g13.rms_norm(*args, **kw)


def test_streams_and_graph():
    r = rng("graph")
    x, rs, w = tensor(r, "bf16", 200, 1000), tensor(r, "bf16", 200, 1000), tensor(r, "bf16", 1000)
    want, h = g13.rms_norm(x, w, residual=rs)
    q = g13.rms_norm(x, w, residual=rs, out_dtype="mxfp8")[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        y, h2 = g13.rms_norm(x, w, residual=rs, stream=s)
        q2 = g13.rms_norm(x, w, residual=rs, out_dtype="mxfp8", stream=s)[0]
        side.synchronize()
        assert torch.equal(y, want) and torch.equal(h2, h) and torch.equal(q2.codes, q.codes)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = g13.rms_norm(x, w, residual=rs, out_dtype="mxfp8")
            val = g13.fp8_dequantize(out[0], "bf16")
        graphs.append((g, out, val))
    x.copy_(tensor(r, "bf16", 200, 1000))
    for _ in range(5):
        for g, _, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    again = g13.rms_norm(x, w, residual=rs, out_dtype="mxfp8")
    for _, out, val in graphs:
        assert torch.equal(out[0].codes, again[0].codes) and torch.equal(out[0].scales, again[0].scales)
        assert torch.equal(out[1], again[1]) and torch.equal(val, g13.fp8_dequantize(again[0], "bf16"))
