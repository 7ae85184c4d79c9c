"""Norm, mxfp8, 4-bit weights and routing in numpy, element by element from their definitions (64 bits)."""
import numpy as np

# ------------------------------------------------------------------ mxfp8
E4M3 = np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)])[:127]  # values of codes 0..126; 127 is NaN


def mxfp8_scale(top):
    """Scale byte of blocks whose largest magnitudes are `top` (float64)."""
    e = np.zeros(top.shape, int)
    with np.errstate(all="ignore"):
        e[top > 0] = np.ceil(np.log2(top[top > 0] / 448)).astype(int)
    e = np.where((top > 0) & (448 * np.exp2(e - 1.0) >= top), e - 1, e)  # (log2 may round at a border)
    e = np.where(448 * np.exp2(e.astype(float)) < top, e + 1, e)
    return np.where(top > 0, np.clip(e, -127, 127) + 127, 0).astype(np.uint8)


def e4m3_code(v):
    """Nearest code (ties to the even one) of magnitudes in [0, 448]."""
    hi = np.clip(np.searchsorted(E4M3, v, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = v - E4M3[lo], E4M3[hi] - v
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)


def mxfp8(x):
    """(codes [rows, cols], scale bytes [rows, blocks]) of a float64 matrix."""
    rows, cols = x.shape
    full = np.zeros((rows, -(-cols // 32) * 32))
    full[:, :cols] = x
    full = full.reshape(rows, -1, 32)
    bad = ~np.isfinite(full).all(2)
    full = np.where(bad[..., None], 0.0, full)
    byte = mxfp8_scale(np.abs(full).max(2))
    y = full * np.exp2(127.0 - byte)[..., None]
    code = e4m3_code(np.minimum(np.abs(y), 448)) | (np.signbit(full).astype(np.uint8) << 7)
    return code.reshape(rows, -1)[:, :cols], np.where(bad, 255, byte).astype(np.uint8)


def mxfp8_values(code, byte):
    v = np.append(E4M3, np.nan)[code & 127] * np.where(code >= 128, -1.0, 1.0)
    d = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))
    return v * np.repeat(d, 32, 1)[:, : code.shape[1]]


def mxfp8_rows(code):
    """Rows of bytes as they are stored."""
    out = np.zeros((code.shape[0], -(-code.shape[1] // 32) * 32), np.uint8)
    out[:, : code.shape[1]] = code
    return out


def tiles(byte):
    """Scale bytes in stored order, by the layout's formula."""
    rows, nb = byte.shape
    ct = -(-nb // 4)
    out = np.zeros(-(-rows // 128) * ct * 512, np.uint8)
    r, c = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    out[((r // 128) * ct + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4] = byte
    return out


# ------------------------------------------------------------------ norm
def rms_norm(h, w, eps, offset):
    """y of float64 rows h (already the rounded sum)."""
    with np.errstate(all="ignore"):
        y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    return y * ((1.0 if w is None else w) + offset)


# ------------------------------------------------------------------ 4-bit weights
def w4_words(q):
    """Codes [N, K] as bytes in stored order, by the layout's formula."""
    n, k = q.shape
    kb, nt = -(-k // 64), -(-n // 16)
    out = np.zeros(nt * kb * 512, np.uint8)
    r, c = np.meshgrid(np.arange(n), np.arange(k), indexing="ij")
    word = (r // 16 * kb + c // 64) * 128 + ((r % 8) * 4 + c % 32 // 8) * 4 + c % 64 // 32 * 2 + r % 16 // 8
    bit = 4 * (c % 2 * 4 + c % 8 // 2)
    np.bitwise_or.at(out, word * 4 + bit // 8, (q << (bit % 8)).astype(np.uint8))
    return out


def w4_entries(s):
    """Scales or zeros [N, groups] in stored order."""
    n, g = s.shape
    out = np.zeros(-(-n // 16) * 16 * g, s.dtype)
    r, c = np.meshgrid(np.arange(n), np.arange(g), indexing="ij")
    out[((r // 16) * g + c) * 16 + r % 8 * 2 + r % 16 // 8] = s
    return out


def w4_values(q, s, z, group):
    """64-bit weights of codes [N, K], scales and zeros [N, groups] (z None: 8)."""
    k = q.shape[1]
    zero = 8.0 if z is None else np.repeat(z.astype(np.float64), group, 1)[:, :k]
    return (q - zero) * np.repeat(s.astype(np.float64), group, 1)[:, :k]


# ------------------------------------------------------------------ routing
def _before(a):
    """Indices of each row of `a` in falling order, NaN last, equal ones by the lowest index."""
    return np.argsort(np.where(np.isnan(a), np.inf, -a), axis=1, kind="stable")


def route(z, k, scores="softmax", bias=None, groups=1, top_groups=None, group_score="max", normalize=True, scale=1.0):
    """(ids, weights) of float64 logits [T, E]."""
    T, E = z.shape
    top_groups = groups if top_groups is None else top_groups
    with np.errstate(all="ignore"):
        if scores == "softmax":
            s = np.exp(z - z.max(1, keepdims=True))
            s = s / s.sum(1, keepdims=True)
        else:
            s = 1 / (1 + np.exp(-z))
        c = z if bias is None else s + bias
        ids = np.zeros((T, k), np.int64)
        for t in range(T):
            stay = np.arange(E)
            if top_groups < groups:
                per = E // groups
                by_sum = group_score == "top2"
                v = ((s[t] + (0 if bias is None else bias)) if by_sum else c[t]).reshape(groups, per)
                best = np.take_along_axis(v, _before(v), 1)
                score = best[:, 0] + best[:, 1] if by_sum and per > 1 else best[:, 0]
                kept = np.sort(_before(score[None])[0][:top_groups])
                stay = (kept[:, None] * per + np.arange(per)).reshape(-1)
            ids[t] = stay[_before(c[t][stay][None])[0][:k]]
        w = np.take_along_axis(s, ids, 1)
        if normalize:
            w = w / w.sum(1, keepdims=True)
    return ids, w * scale
