"""Norm to mxfp8 on rows that are made to lie next to the codes' and the scales' borders.

Codes and scales have to be those of a value within 2^-39 of the formula's: the sum of squares is off by 2^-40 of itself at
most (a thread's two-sums lose 16 times 16 products of two roundings, 2^-40; the joins 2^-47), so its root by 2^-41; Newton's remainder and
the product in two numbers add 2^-46 each.  The reference, in 64 bits, is off by less than 2^-48.
"""
import numpy as np
import pytest
import torch

import dense_gemm_13_gb300 as g13
from tests import blocks_ref as ref
from tests.test_gpu_norm import DT, rng, stream_of, tensor

pytestmark = pytest.mark.gpu
MIDS = (ref.E4M3[:-1] + ref.E4M3[1:]) / 2  # where the nearest code changes


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_gemm_13_gb300 import _build
    _build.build()
    g13.load()


def check_exact(q, h64, w, eps, offset=0.0, d=2.0 ** -39):
    y = ref.rms_norm(h64, None if w is None else w.double().cpu().numpy(), eps, offset)
    rows, cols = y.shape
    pad = np.zeros((rows, -(-cols // 32) * 32))
    pad[:, :cols] = np.abs(y)
    top = pad.reshape(rows, -1, 32).max(2)
    nb = top.shape[1]
    rr, cc = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    byte = q.scales.cpu().numpy()[((rr // 128) * -(-nb // 4) + cc // 4) * 512 + (rr % 32) * 16 + (rr % 128) // 32 * 4 + cc % 4]
    lo, hi = ref.mxfp8_scale(top * (1 - d)), ref.mxfp8_scale(top * (1 + d))
    assert ((byte == lo) | (byte == hi)).all(), f"{np.sum((byte != lo) & (byte != hi))} of {byte.size} scales"
    v = np.abs(y) * np.repeat(np.exp2(127.0 - byte), 32, 1)[:, :cols]
    clo, chi = ref.e4m3_code(np.minimum(v * (1 - d), 448)), ref.e4m3_code(np.minimum(v * (1 + d), 448))
    mag = q.codes.cpu().numpy()[:, :cols] & 127
    bad = (mag < clo) | (mag > chi)
    assert not bad.any(), f"{bad.sum()} of {bad.size} codes"
    return np.sum(clo != chi), mag.size


def border_weight(r, h64, eps, row):
    """FP32 weights that bring a row's values to borders of the codes (and half of the blocks' largest to one of the
    scales), but for the weights' own rounding."""
    H = h64.shape[1]
    target = r.choice(MIDS[MIDS < 380], H)
    first = np.arange(0, H, 32)
    target[first] = np.where(r.random(len(first)) < 0.5, 448.0, 400.0)
    rs = 1 / np.sqrt((h64[row] ** 2).mean() + eps)
    w = target / (np.abs(h64[row]) * rs) * np.exp2(r.integers(-3, 4))
    return torch.from_numpy(w.astype(np.float32)).cuda()


@pytest.mark.parametrize("H", [1, 8, 33, 64, 100, 128, 264, 512, 1000, 1024, 2049, 4096, 4097, 8185, 8192, 16384, 20000, 40000])
@pytest.mark.parametrize("kind", [("bf16", "none"), ("f16", "f16"), ("bf16", "f32"), ("f32", "none")], ids="-".join)
def test_values_next_to_borders(H, kind):
    dtype, res = kind
    r = rng("border", H, kind)
    for T, left in ((1, 0), (3, 0), (3, 1), (2, 4)):  # rows on 16 bytes and off them, all arrays alike or not
        def room(name, std=1.0):
            flat = torch.zeros(left + T * H, device="cuda").to(DT[name])
            rows = flat[left:].view(T, H)
            rows.copy_(tensor(r, name, T, H, std=std))
            # no value close to zero, whose weight would be without bounds
            rows.copy_(torch.where(rows.abs() < 0.05, torch.full_like(rows, 0.5), rows))
            return rows
        x, rs = room(dtype), None if res == "none" else room(res, 3.0)
        h, h64 = stream_of(x, rs)
        if rs is not None:
            h64 = np.where(h64 == 0, 1.0, h64)
        eps = float(np.float32(1e-6))
        for row in range(T):
            w = border_weight(r, h64, eps, row)
            q = g13.rms_norm(x, w, residual=rs, out_dtype="mxfp8")
            q = q if rs is None else q[0]
            check_exact(q, h.double().cpu().numpy(), w, eps)


@pytest.mark.parametrize("H", [64, 72, 1000, 2049, 4096, 4097, 20000])
def test_large_values_and_weights(H):
    # the product of a value and its weight is beyond FP32, neither the row's squares nor any result is
    r = rng("large", H)
    for T, left in ((300, 0), (300, 1), (40, 2)):
        x = torch.zeros(left + T * H, device="cuda")[left:].view(T, H)
        x.copy_(tensor(r, "f32", T, H, std=1e16))
        w = torch.from_numpy((1e23 * (1 + r.random(H))).astype(np.float32)).cuda()
        q = g13.rms_norm(x, w, out_dtype="mxfp8")
        assert not bool((q.scales == 255).any())
        check_exact(q, x.double().cpu().numpy(), w, float(np.float32(1e-6)))


@pytest.mark.parametrize("H", [40, 256, 2049, 5000])
def test_random_rows(H):
    r = rng("random", H)
    x, w = tensor(r, "bf16", 700, H), tensor(r, "bf16", H)
    check_exact(g13.rms_norm(x, w, out_dtype="mxfp8"), x.double().cpu().numpy(), w, float(np.float32(1e-6)))
