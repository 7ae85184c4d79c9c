"""Workloads of what stands around the products of a transformer block when it is served.

Each case is one call, or one chain of calls, of a serving program:

  norm      h = x + r (the residual stream, written back), y = h / rms(h) * weight
  norm8     the same with y in 8 bits with block scales, read back
  linear8   norm8, then the product with 8-bit weights (a linear layer on a prompt)
  product8  C = cast(act(alpha A B^T + bias) + beta R) of two matrices in 8 bits
  w4        Y = cast(act(X W^T + bias)) with 4-bit weights and group scales
  route     the choice of experts and their weights from logits

`run` computes them with elementary torch operations, or, with `own` set,
through the library's entry points.  `exact` gives the same outputs in 64 bits.

8 bits (mxfp8): blocks of 32 along a row; elements E4M3, scale 2^(b - 127) from
a byte b, its exponent the least with max |x| <= 448 * scale, kept in [-127, 127].
Rows of codes are padded with zeros to 32 elements.  Scales lie in tiles of
128 rows x 4 blocks, 512 bytes each, row r and block c of a tile at byte
(r % 32) * 16 + (r // 32) * 4 + c; tiles follow one another along a row of
tiles; padding is zero.

4-bit weights [N][K]: w = (q - z) * s, codes q and zeros z in 0..15 (no zeros
given: 8), a zero and a scale for `group` columns of a row.  Codes lie in blocks
of 16 rows x 64 columns, 512 bytes each, the blocks of 16 rows one after another
along the columns; row r, column k of a block are in the 32-bit word
((r % 8) * 4 + k % 32 // 8) * 4 + k // 32 * 2 + r // 8 (little endian), at bits
4 * (k % 2 * 4 + k % 8 // 2).  Scale and zero of row r, group c are entry
((r // 16) * groups + c) * 16 + r % 8 * 2 + r % 16 // 8 of their arrays.
Padding is zero.
"""
import math

import torch

own = False

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


def listed():
    return [
        # one decoding token between two layers: latency counts
        dict(name="norm_token", op="norm", T=1, H=4096, dtype="bf16", res="bf16", out="bf16"),
        # a long batch of prompts: bytes count
        dict(name="norm_large", op="norm", T=8192, H=8192, dtype="bf16", res="bf16", out="bf16"),
        # a residual stream in 32 bits, odd sizes, activations for the 8-bit product
        dict(name="norm8_ragged", op="norm8", T=1000, H=4097, dtype="f16", res="f32", out="f16"),
        # a prompt of 512 tokens through norm and projection
        dict(name="linear8_prompt", op="linear8", T=512, H=4096, N=6144, dtype="bf16", res="bf16", out="bf16"),
        # sizes that fill no tile, FP32 result added to a residual stream
        dict(name="product8_ragged", op="product8", M=1000, N=3001, K=4097, out="f32", bias=False, act="none",
             residual=True),
        # the large square product of the benchmark
        dict(name="product8_large", op="product8", M=8192, N=8192, K=8192, out="bf16", bias=False, act="none",
             residual=False),
        # one decoding token against a large weight: the weight's bytes are the cost
        dict(name="w4_token", op="w4", M=1, N=6144, K=6144, group=128, zeros=True, dtype="bf16", out="bf16",
             bias=False, act="none"),
        # a few tokens, odd sizes, the smallest groups, an activation behind it
        dict(name="w4_ragged", op="w4", M=5, N=1000, K=3001, group=32, zeros=False, dtype="f16", out="f32",
             bias=True, act="gelu"),
        # a decoding batch against a wide feed-forward weight
        dict(name="w4_batch", op="w4", M=16, N=16384, K=8192, group=64, zeros=True, dtype="bf16", out="bf16",
             bias=False, act="none"),
        # one token's choice: latency counts
        dict(name="route_token", op="route", T=1, E=64, k=6, groups=1, top_groups=1, group_score="max",
             scores="softmax", bias=False, normalize=True, scale=1.0, dtype="bf16"),
        # odd sizes, groups by their best expert, weights as they are
        dict(name="route_ragged", op="route", T=1001, E=160, k=6, groups=8, top_groups=3, group_score="max",
             scores="softmax", bias=False, normalize=False, scale=16.0, dtype="f32"),
        # a batch of prompts, balanced by a bias, groups by the sum of their two best
        dict(name="route_large", op="route", T=16384, E=256, k=8, groups=8, top_groups=4, group_score="top2",
             scores="sigmoid", bias=True, normalize=True, scale=2.5, dtype="f32"),
    ]


def _log(rng, lo, hi):
    """A size whose logarithm is spread evenly over [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm8", "linear8", "product8", "w4", "w4", "route", "route"])
    dtype = rng.choice(["bf16", "f16"])
    if op in ("norm", "norm8", "linear8"):
        H = _log(rng, 64, 16384)
        c = dict(op=op, T=min(_log(rng, 1, 16384), 2 ** 26 // H), H=H, dtype=dtype,
                 res=rng.choice(["none", "f32", dtype]), out=dtype)
        if op == "norm" and rng.random() < 0.3:
            c.update(dtype="f32", res=rng.choice(["none", "f32"]), out=rng.choice(["f32", "bf16"]))
        if op == "linear8":
            c.update(T=min(c["T"], 4096), N=_log(rng, 16, 8192))
        return c
    if op == "product8":
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 16, 8192), K=_log(rng, 32, 8192),
                    out=rng.choice(["f32", "bf16", "f16"]), bias=rng.random() < 0.5,
                    act=rng.choice(["none", "gelu", "relu"]), residual=rng.random() < 0.5)
    if op == "w4":
        return dict(op=op, M=_log(rng, 1, 64), N=_log(rng, 64, 16384), K=_log(rng, 64, 8192),
                    group=rng.choice([32, 64, 128, 256]), zeros=rng.random() < 0.5, dtype=dtype,
                    out=rng.choice(["f32", dtype]), bias=rng.random() < 0.5, act=rng.choice(["none", "gelu", "relu"]))
    groups, per = rng.choice([1, 1, 2, 4, 8]), _log(rng, 4, 64)
    top = rng.randint(1, groups)
    scores = rng.choice(["softmax", "sigmoid"])
    return dict(op=op, T=_log(rng, 1, 16384), E=groups * per, k=rng.randint(1, min(top * per, 16)), groups=groups,
                top_groups=top, group_score=rng.choice(["max", "top2"]), scores=scores, bias=rng.random() < 0.5,
                normalize=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16", "f16"]))


# ------------------------------------------------------------------ 8 bits with block scales
def _tiles(byte):
    """Scale bytes [rows, blocks] in the order in which they are stored."""
    r, c = byte.shape
    t = torch.nn.functional.pad(byte, (0, -c % 4, 0, -r % 128))
    t = t.reshape(t.shape[0] // 128, 4, 32, t.shape[1] // 4, 4)
    return t.permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _untile(flat, rows, blocks):
    rt, ct = -(-rows // 128), -(-blocks // 4)
    t = flat.reshape(rt, ct, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, ct * 4)
    return t[:rows, :blocks]


def _quantise8(x):
    """(codes in padded rows as E4M3, scale bytes [rows, blocks]) of an FP32 matrix."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, -cols % 32)).reshape(rows, -1, 32)
    amax = x.abs().amax(2)
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1): 448 = 0.875 * 2^9
    byte = ((e - 9 + (m > 0.875)).clamp(-127, 127) + 127) * (amax > 0)
    y = x * torch.ldexp(torch.ones_like(amax), 127 - byte)[..., None]
    return y.to(torch.float8_e4m3fn).reshape(rows, -1), byte.to(torch.uint8)


def _values8(codes, byte, cols):
    d = torch.ldexp(torch.ones(byte.shape, device=byte.device), byte.int() - 127)
    return (codes.float().reshape(*byte.shape, 32) * d[..., None]).reshape(byte.shape[0], -1)[:, :cols]


def _operand8(x):
    codes, byte = _quantise8(x)
    return dict(codes=codes.view(torch.uint8).contiguous(), scales=_tiles(byte), rows=x.shape[0], cols=x.shape[1])


def _read8(o):
    byte = _untile(o["scales"], o["rows"], -(-o["cols"] // 32))
    return _values8(o["codes"].view(torch.float8_e4m3fn), byte, o["cols"])


# ------------------------------------------------------------------ 4-bit weights
def _pack4(q):
    """Codes uint8 [N, K] in the order in which they are stored (see above)."""
    q = torch.nn.functional.pad(q, (0, -q.shape[1] % 64, 0, -q.shape[0] % 16))
    b = q.reshape(q.shape[0] // 16, 2, 8, q.shape[1] // 64, 2, 4, 8)  # tile, r/8, r%8, block, k/32, lane, k%8
    b = b.permute(0, 3, 2, 5, 4, 1, 6).reshape(-1, 8)
    return (b[:, [0, 4, 1, 5]] | (b[:, [2, 6, 3, 7]] << 4)).reshape(-1).contiguous()


def _unpack4(codes, N, K):
    kb, nt = -(-K // 64), -(-N // 16)
    b = torch.stack((codes & 15, codes >> 4), 1).reshape(nt, kb, 8, 4, 2, 2, 8)
    b = b[..., [0, 4, 1, 5, 2, 6, 3, 7]]
    return b.permute(0, 5, 2, 1, 4, 3, 6).reshape(nt * 16, kb * 64)[:N, :K]


def _pack_rows(s):
    """[N, groups] in the order of stored scales and zeros."""
    n, g = s.shape
    s = torch.nn.functional.pad(s, (0, 0, 0, -n % 16))
    return s.reshape(-1, 2, 8, g).permute(0, 3, 2, 1).reshape(-1).contiguous()


def _unpack_rows(flat, n, g):
    return flat.reshape(-1, g, 8, 2).permute(0, 3, 2, 1).reshape(-1, g)[:n]


def _act(y, act):
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if act == "relu":
        return y.clamp(min=0)
    return y


# ------------------------------------------------------------------ inputs
def _randn(gen, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda", dtype=dtype) * std).contiguous()


def _stream(gen, T, H, dtype):
    """Normal values, a few columns ten times as large (outlier channels)."""
    x = _randn(gen, T, H)
    x[:, torch.randperm(H, generator=gen, device="cuda")[: max(1, H // 128)]] *= 10
    return x.to(TORCH[dtype])


def prepare(case, seed):
    gen, c = torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFFFFFFFFFF), dict(case)
    if c["op"] in ("norm", "norm8", "linear8"):
        s = dict(case=c, x=_randn(gen, c["T"], c["H"], dtype=TORCH[c["dtype"]]), r=None,
                 weight=(1 + 0.1 * _randn(gen, c["H"])).to(TORCH[c["dtype"]]))
        if c["res"] != "none":
            s["r"] = _stream(gen, c["T"], c["H"], c["res"])
        if c["op"] == "linear8":
            s["B"] = _operand8(_randn(gen, c["N"], c["H"], std=c["H"] ** -0.5))
        return s
    if c["op"] == "product8":
        M, N, K = c["M"], c["N"], c["K"]
        return dict(case=c, A=_operand8(_stream(gen, M, K, "bf16").float()),
                    B=_operand8(_randn(gen, N, K, std=K ** -0.5)), bias=_randn(gen, N) if c["bias"] else None,
                    R=_randn(gen, M, N) if c["residual"] else None)
    if c["op"] == "w4":
        M, N, K, g, dt = c["M"], c["N"], c["K"], c["group"], TORCH[c["dtype"]]
        w = torch.nn.functional.pad(_randn(gen, N, K, std=K ** -0.5), (0, -K % g)).reshape(N, -1, g)
        if c["zeros"]:  # the group's range, zero among it
            lo, hi = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
            scale = ((hi - lo) / 15).to(dt)
            zero = torch.round(-lo / scale.float()).clamp(0, 15)
        else:
            scale = (w.abs().amax(2) / 7.5).to(dt)
            zero = torch.full_like(scale, 8.0, dtype=torch.float32)
        q = torch.round(w / scale.float()[..., None] + zero[..., None]).clamp(0, 15).to(torch.uint8)
        return dict(case=c, x=_randn(gen, M, K, dtype=dt), codes=_pack4(q.reshape(N, -1)[:, :K]),
                    scales=_pack_rows(scale), zeros=_pack_rows(zero.to(torch.uint8)) if c["zeros"] else None,
                    bias=_randn(gen, N) if c["bias"] else None)
    return dict(case=c, logits=_randn(gen, c["T"], c["E"], dtype=TORCH[c["dtype"]]),
                bias=_randn(gen, c["E"], std=0.05) if c["bias"] else None)


# ------------------------------------------------------------------ one pass
def run(state):
    c = state["case"]
    if own:
        return _run_own(c, state)
    if c["op"] in ("norm", "norm8", "linear8"):
        h, r = state["x"].float(), state["r"]
        if r is not None:
            stream = (h + r.float()).to(r.dtype)
            h = stream.float()
        y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * state["weight"].float()
        if c["op"] != "norm":
            y = _values8(*_quantise8(y), c["H"])
        if c["op"] == "linear8":
            y = y @ _read8(state["B"]).T
        y = y.to(TORCH[c["out"]])
        return y if r is None else (y, stream)
    if c["op"] == "product8":
        y = _read8(state["A"]) @ _read8(state["B"]).T
        if state["bias"] is not None:
            y = y + state["bias"]
        y = _act(y, c["act"])
        if state["R"] is not None:
            y = y + state["R"]
        return y.to(TORCH[c["out"]])
    if c["op"] == "w4":
        N, K, g = c["N"], c["K"], c["group"]
        n_groups = -(-K // g)
        w = _unpack4(state["codes"], N, K).float()
        if state["zeros"] is None:
            w = w - 8
        else:
            w = w - _unpack_rows(state["zeros"], N, n_groups).float().repeat_interleave(g, 1)[:, :K]
        w = w * _unpack_rows(state["scales"], N, n_groups).float().repeat_interleave(g, 1)[:, :K]
        y = state["x"].float() @ w.T
        if state["bias"] is not None:
            y = y + state["bias"]
        return _act(y, c["act"]).to(TORCH[c["out"]])
    return _route(c, state["logits"], state["bias"])


def _route(c, logits, bias):
    T, E, G = c["T"], c["E"], c["groups"]
    z = logits.double()  # the choice is next to a border: 64 bits
    if c["scores"] == "softmax":
        s = torch.exp(z - z.amax(1, keepdim=True))
        s = s / s.sum(1, keepdim=True)
    else:
        s = 1 / (1 + torch.exp(-z))
    choice = s if bias is None else s + bias.double()
    if c["top_groups"] < G:
        by_group = choice.reshape(T, G, E // G)
        if c["group_score"] == "max":
            score = by_group.amax(2)
        else:
            score = torch.sort(by_group, dim=2, descending=True).values[:, :, :2].sum(2)
        best = torch.sort(score, dim=1, descending=True, stable=True).indices[:, : c["top_groups"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=z.device).scatter(1, best, True)
        choice = choice.masked_fill(~kept.repeat_interleave(E // G, 1), -math.inf)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, : c["k"]]
    w = torch.gather(s, 1, ids)
    if c["normalize"]:
        w = w / w.sum(1, keepdim=True)
    return ids.int(), (w * c["scale"]).float()


def _run_own(c, state):
    import dense_gemm_13_gb300 as g13

    if c["op"] == "norm":
        return g13.rms_norm(state["x"], state["weight"], residual=state["r"], eps=EPS, out_dtype=c["out"])
    if c["op"] == "norm8":
        y = g13.rms_norm(state["x"], state["weight"], residual=state["r"], eps=EPS, out_dtype="mxfp8")
        if state["r"] is None:
            return g13.fp8_dequantize(y, c["out"])
        return g13.fp8_dequantize(y[0], c["out"]), y[1]
    if c["op"] in ("linear8", "product8"):
        B = state.get("handle")
        if B is None:  # the weight's handle, which a program makes once
            o = state["B"]
            B = state["handle"] = g13.Fp8Tensor(o["codes"], o["scales"], o["rows"], o["cols"])
        if c["op"] == "linear8":
            y = g13.rms_norm(state["x"], state["weight"], residual=state["r"], eps=EPS, out_dtype="mxfp8")
            A, stream = (y, None) if state["r"] is None else y
            y = g13.fp8_matmul(A, B, out_dtype=c["out"])
            return y if stream is None else (y, stream)
        A = state.get("handle_a")
        if A is None:
            o = state["A"]
            A = state["handle_a"] = g13.Fp8Tensor(o["codes"], o["scales"], o["rows"], o["cols"])
        return g13.fp8_matmul(A, B, bias=state["bias"], act=c["act"], residual=state["R"], out_dtype=c["out"])
    if c["op"] == "w4":
        W = state.get("handle")
        if W is None:
            W = state["handle"] = g13.W4Tensor(state["codes"], state["scales"], state["zeros"], c["N"], c["K"],
                                               c["group"])
        return g13.w4_matmul(state["x"], W, bias=state["bias"], act=c["act"], out_dtype=c["out"])
    return g13.route(state["logits"], c["k"], scores=c["scores"], bias=state["bias"], groups=c["groups"],
                     top_groups=c["top_groups"], group_score=c["group_score"], normalize=c["normalize"],
                     scale=c["scale"])


# ------------------------------------------------------------------ cost
_SIZE = {"none": 0, "f32": 4, "f16": 2, "bf16": 2}


def _bytes8(rows, cols):
    return rows * cols + rows * -(-cols // 32)


def work(case):
    c = case
    if c["op"] in ("norm", "norm8", "linear8"):
        # x, the stream read and written, the weight
        b = c["T"] * c["H"] * (_SIZE[c["dtype"]] + 2 * _SIZE[c["res"]]) + c["H"] * _SIZE[c["dtype"]]
        if c["op"] == "linear8":
            return dict(bytes=b + _bytes8(c["N"], c["H"]) + c["T"] * c["N"] * _SIZE[c["out"]],
                        flops=2 * c["T"] * c["N"] * c["H"])
        return dict(bytes=b + c["T"] * c["H"] * _SIZE[c["out"]], flops=4 * c["T"] * c["H"])
    if c["op"] == "product8":
        M, N, K = c["M"], c["N"], c["K"]
        return dict(bytes=_bytes8(M, K) + _bytes8(N, K) + M * N * _SIZE[c["out"]] + 4 * N * c["bias"]
                    + 4 * M * N * c["residual"], flops=2 * M * N * K)
    if c["op"] == "w4":
        M, N, K = c["M"], c["N"], c["K"]
        groups = -(-K // c["group"])
        return dict(bytes=N * K / 2 + N * groups * (2 + c["zeros"]) + 2 * M * K + M * N * _SIZE[c["out"]]
                    + 4 * N * c["bias"], flops=2 * M * N * K)
    return dict(bytes=c["T"] * c["E"] * _SIZE[c["dtype"]] + 4 * c["E"] * c["bias"] + 8 * c["T"] * c["k"],
                flops=4 * c["T"] * c["E"])


# ------------------------------------------------------------------ the definition in 64 bits
def _round8_64(x):
    """The 8-bit values of a 64-bit matrix, from the format's definition."""
    rows, cols = x.shape
    full = torch.zeros(rows, -(-cols // 32) * 32, dtype=torch.float64, device=x.device)
    full[:, :cols] = x
    full = full.view(rows, -1, 32)
    top = full.abs().max(2, keepdim=True).values
    e = torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** -140)))
    e = torch.where(448 * torch.pow(2.0, e - 1) >= top, e - 1, e)  # log2 may round at a border
    e = torch.where(448 * torch.pow(2.0, e) < top, e + 1, e).clamp(-127, 127)
    d = torch.pow(2.0, e)
    y = full / d
    a = y.abs().clamp(min=2.0 ** -6)  # E4M3: 3 mantissa bits, least exponent -6
    k = torch.floor(torch.log2(a))
    k = torch.where(torch.pow(2.0, k + 1) <= a, k + 1, k)
    k = torch.where(torch.pow(2.0, k) > a, k - 1, k)
    step = torch.pow(2.0, k - 3)
    return (torch.round(y / step) * step * d).view(rows, -1)[:, :cols]


def _read8_64(o):
    """Stored codes and scales as 64-bit values, element by element from the layout's formula."""
    rows, cols, dev = o["rows"], o["cols"], o["codes"].device
    r = torch.arange(rows, device=dev)[:, None]
    code = o["codes"][:, :cols].int()
    e, m = code >> 3 & 15, (code & 7).double()
    mag = torch.where(e == 0, m / 8 * 2.0 ** -6, torch.pow(2.0, (e - 7).double()) * (1 + m / 8))
    blk = torch.arange(-(-cols // 32), device=dev)[None, :]
    tiles = (-(-cols // 32) + 3) // 4
    at = ((r // 128) * tiles + blk // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + blk % 4
    d = torch.pow(2.0, (o["scales"][at].int() - 127).double())
    k = torch.arange(cols, device=dev)[None, :]
    return torch.where(code >= 128, -mag, mag) * d.gather(1, (k // 32).expand(rows, -1))


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] in ("norm", "norm8", "linear8"):
        h = s["x"].double()
        stream = None
        if s["r"] is not None:
            stream = (h + s["r"].double()).to(s["r"].dtype)
            h = stream.double()
        y = h / torch.sqrt(torch.einsum("th,th->t", h, h)[:, None] / c["H"] + EPS) * s["weight"].double()
        if c["op"] != "norm":
            y = _round8_64(y)
        if c["op"] == "linear8":
            y = torch.einsum("mk,nk->mn", y, _read8_64(s["B"]))
        return y if stream is None else (y, stream.double())
    if c["op"] == "route":
        T, E, G = c["T"], c["E"], c["groups"]
        z = s["logits"].double()
        if c["scores"] == "softmax":
            p = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
        else:
            p = torch.where(z < 0, torch.exp(z) / (1 + torch.exp(z)), 1 / (1 + torch.exp(-z)))
        a = p if s["bias"] is None else p + s["bias"].double()
        if c["top_groups"] < G:
            v = a.view(T, G, -1)
            score = v.max(2).values
            if c["group_score"] == "top2" and v.shape[2] > 1:
                score = torch.topk(v, 2, dim=2).values.sum(2)
            rank = (score[:, None, :] > score[:, :, None]).sum(2)  # groups that come before each one
            rank += torch.tril(score[:, None, :] == score[:, :, None], -1).sum(2)
            a = torch.where((rank < c["top_groups"]).repeat_interleave(E // G, 1), a, torch.full_like(a, -math.inf))
        ids = torch.argsort(-a, dim=1, stable=True)[:, : c["k"]]
        w = p.gather(1, ids)
        if c["normalize"]:
            w = w / w.sum(1, keepdim=True)
        return ids.int(), w * c["scale"]
    if c["op"] == "w4":
        N, K, g = c["N"], c["K"], c["group"]
        word = s["codes"].view(torch.int32)
        groups, kb = -(-K // g), -(-K // 64)
        k = torch.arange(K, device=word.device)[None, :]
        y = torch.zeros(c["M"], N, dtype=torch.float64, device=word.device)
        for n0 in range(0, N, 2048):
            r = torch.arange(n0, min(N, n0 + 2048), device=word.device)[:, None]
            at = ((r // 16 * kb + k // 64) * 128 + ((r % 8) * 4 + k % 32 // 8) * 4 + k % 64 // 32 * 2 + r % 16 // 8)
            q = (word[at] >> (4 * (k % 2 * 4 + k % 8 // 2)).int()) & 15
            row = (r // 16 * groups + k // g) * 16 + r % 8 * 2 + r % 16 // 8
            z = s["zeros"][row].double() if s["zeros"] is not None else 8.0
            y[:, n0: n0 + 2048] = torch.einsum("mk,nk->mn", s["x"].double(), (q.double() - z) * s["scales"][row].double())
    else:
        y = torch.einsum("mk,nk->mn", _read8_64(s["A"]), _read8_64(s["B"]))
    if s["bias"] is not None:
        y += s["bias"].double()
    if c["act"] == "gelu":
        y = y * 0.5 * torch.erfc(-y / math.sqrt(2))
    elif c["act"] == "relu":
        y = torch.maximum(y, torch.zeros_like(y))
    if s.get("R") is not None:
        y += s["R"].double()
    return y
