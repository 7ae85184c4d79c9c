"""The microscaled 4-bit formats in numpy, element by element from their definition (64 bits)."""
import numpy as np

BLOCK = {"mxfp4": 32, "nvfp4": 16}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
# midpoints between neighbouring magnitudes; a tie goes up where the code above is even
MID = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
UP = np.array([False, True, False, True, False, True, False])

_E4M3 = np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                  for e in range(16) for m in range(8)])[:127]


def e4m3(v):
    """Nearest E4M3 byte (ties to even) of values in [0, 448]."""
    hi = np.clip(np.searchsorted(_E4M3, v, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = v - _E4M3[lo], _E4M3[hi] - v
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)


def scale_value(byte, fmt, g):
    """FP32 value of a stored scale, in 64 bits."""
    if fmt == "mxfp4":
        v = np.exp2(byte.astype(np.float64) - 127)
        return np.where(byte == 255, np.nan, v)
    table = np.append(_E4M3, np.nan)
    return np.float32(table[byte & 127].astype(np.float32) * np.float32(g)).astype(np.float64)


def quantise(x, fmt, g=1.0):
    """(codes 0..15 [rows, cols], scale bytes [rows, blocks]) of a float32 matrix."""
    x = np.asarray(x, dtype=np.float32)
    rows, cols = x.shape
    b = BLOCK[fmt]
    nb = -(-cols // b)
    full = np.zeros((rows, nb * b), np.float32)
    full[:, :cols] = x
    full = full.reshape(rows, nb, b)
    bad = ~np.isfinite(full).all(2)
    full = np.where(bad[..., None], np.float32(0), full)
    top = np.abs(full).max(2)
    if fmt == "mxfp4":
        e = np.frexp(top.astype(np.float64))[1] - 1
        byte = np.where(top > 0, np.clip(e - 2, -127, 127) + 127, 0).astype(np.uint8)
    else:
        byte = e4m3(np.minimum(top / np.float32(np.float32(6) * np.float32(g)), np.float32(448)).astype(np.float64))
    d = scale_value(byte, fmt, g)
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(d[..., None] > 0, (full.astype(np.float64) / d[..., None]).astype(np.float32), np.float32(0))
    a = np.abs(y).astype(np.float64)[..., None]
    code = ((a > MID) | ((a == MID) & UP)).sum(-1).astype(np.uint8) | (np.signbit(full).astype(np.uint8) << 3)
    byte = np.where(bad, 255 if fmt == "mxfp4" else 127, byte).astype(np.uint8)
    return code.reshape(rows, -1)[:, :cols], byte


def values(codes, byte, fmt, g=1.0):
    """64-bit values of codes [rows, cols] with scale bytes [rows, blocks]."""
    d = scale_value(byte, fmt, g)
    return E2M1[codes] * np.repeat(d, BLOCK[fmt], 1)[:, : codes.shape[1]]


def pack(codes):
    """Rows of bytes as they are stored."""
    rows, cols = codes.shape
    out = np.zeros((rows, -(-cols // 32) * 32), np.uint8)
    out[:, :cols] = codes
    return out[:, 0::2] | (out[:, 1::2] << 4)


def tiles(byte):
    """Scale bytes in stored order, by the layout's formula."""
    rows, nb = byte.shape
    ct = -(-nb // 4)
    out = np.zeros(-(-rows // 128) * ct * 512, np.uint8)
    r, c = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    out[((r // 128) * ct + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4] = byte
    return out
