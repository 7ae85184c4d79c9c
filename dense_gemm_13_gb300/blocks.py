"""What stands around the products of a transformer block: the root-mean-square norm with the residual's
addition, 8-bit floats (mxfp8) and their product, 4-bit weights with group scales, routing to experts.

Argument checks and marshalling only, as in the package itself, which exports every name below.
"""
from __future__ import annotations

import ctypes
import sys

from . import (ACTS, DTYPES, MOE_ACTS, Config, Epilogue, GemmError, MoePlan, _Config, _keep, _ld, _moe_plans,
               _no_capture, _on_device, _ptr, _refuse, _rows_ok, _stream, _t, gemm_moe_plan, lib)

__all__ = ["rms_norm", "Fp8Tensor", "Fp8Plan", "fp8_quantize", "fp8_dequantize", "gemm_fp8_plan", "gemm_fp8_run",
           "gemm_fp8_status", "gemm_fp8_select_config", "fp8_matmul", "W4Tensor", "w4_quantize", "w4_pack",
           "w4_dequantize", "w4_matmul", "ROUTE_SCORES", "ROUTE_GROUP_SCORES", "route", "gemm_moe_run_routed",
           "moe_experts"]

_package = sys.modules[__package__]

ROUTE_SCORES = {"softmax": 0, "sigmoid": 1}
ROUTE_GROUP_SCORES = {"max": 0, "top2": 1}


class _NormDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("has_residual", ctypes.c_int), ("residual_dtype", ctypes.c_int),
                ("weight_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("mxfp8", ctypes.c_int),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ldx", ctypes.c_int64), ("ldr", ctypes.c_int64),
                ("ldh", ctypes.c_int64), ("ldy", ctypes.c_int64), ("eps", ctypes.c_float),
                ("weight_offset", ctypes.c_float)]


class _W4Desc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("M", ctypes.c_int64), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64), ("group", ctypes.c_int64), ("has_zeros", ctypes.c_int),
                ("has_bias", ctypes.c_int), ("act", ctypes.c_int), ("has_residual", ctypes.c_int),
                ("beta", ctypes.c_float), ("ldx", ctypes.c_int64), ("ldy", ctypes.c_int64), ("ldr", ctypes.c_int64),
                ("flags", ctypes.c_uint32), ("timeout_ms", ctypes.c_uint32)]


class _RouteDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("T", ctypes.c_int64), ("E", ctypes.c_int64), ("top_k", ctypes.c_int64),
                ("scores", ctypes.c_int), ("groups", ctypes.c_int64), ("top_groups", ctypes.c_int64),
                ("group_score", ctypes.c_int), ("normalize", ctypes.c_int), ("scale", ctypes.c_float),
                ("ld", ctypes.c_int64)]


def _lib_of():
    """The library, where it is loaded already."""
    return _package._lib


def prototypes(L) -> None:
    """The C signatures of this module's entry points."""
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    P = ctypes.POINTER
    for name, res, args in (
            ("gemm_norm_desc_init", None, [P(_NormDesc)]),
            ("gemm_rms_norm", i32, [P(_NormDesc)] + [vp] * 7),
            ("gemm_fp8_row_bytes", i64, [i64]), ("gemm_fp8_scales_bytes", i64, [i64, i64]),
            ("gemm_fp8_quantize", i32, [i32, i64, i64, vp, i64, vp, vp, vp]),
            ("gemm_fp8_dequantize", i32, [i32, i64, i64, vp, vp, vp, i64, vp]),
            ("gemm_fp8_plan", i32, [i64, i64, i64, i64, vp, P(vp)]),
            ("gemm_fp8_run", i32, [vp] * 8 + [f32, vp]),
            ("gemm_fp8_status", i32, [vp]), ("gemm_fp8_destroy", None, [vp]),
            ("gemm_fp8_select_config", i32, [i64, i64, i64, ctypes.c_int32, P(_Config)]),
            ("gemm_w4_codes_bytes", i64, [i64, i64]), ("gemm_w4_scales_count", i64, [i64, i64, i64]),
            ("gemm_w4_quantize", i32, [i32, i32, i64, i64, i64, vp, i64, vp, vp, vp, vp]),
            ("gemm_w4_pack", i32, [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp]),
            ("gemm_w4_dequantize", i32, [i32, i32, i64, i64, i64, vp, vp, vp, vp, i64, vp]),
            ("gemm_w4_desc_init", None, [P(_W4Desc)]),
            ("gemm_w4_run", i32, [P(_W4Desc)] + [vp] * 7 + [f32, vp]),
            ("gemm_route_desc_init", None, [P(_RouteDesc)]),
            ("gemm_route", i32, [P(_RouteDesc)] + [vp] * 5),
            ("gemm_moe_run_routed", i32, [vp] * 9)):
        f = getattr(L, name)
        f.restype, f.argtypes = res, args


def _out_ok(t, out, shape, dtype: str, index: int) -> bool:
    return (tuple(out.shape) == shape and t.name.get(out.dtype) == dtype and out.get_device() == index
            and _rows_ok(out))


def _layout(x):
    """(address, bytes of a row, bytes from a row to the next, rows) of a tensor's memory; without gaps it is one row."""
    size = x.element_size()
    if x.dim() == 2:
        (rows, cols), (ld, step) = x.shape, x.stride()
        if rows > 1 and ld > cols and (cols <= 1 or step == 1):
            return x.data_ptr(), cols * size, ld * size, rows
    n = sum((s - 1) * abs(st) for s, st in zip(x.shape, x.stride())) + 1
    return x.data_ptr(), n * size, 0, 1


def _bytes_overlap(a, b) -> bool:
    """Whether two tensors share memory.  (Column ranges of one buffer do not; of rows of different strides, whether the
    memory that they span does.)"""
    if a.numel() == 0 or b.numel() == 0:
        return False
    (p, la, sa, na), (q, lb, sb, nb) = _layout(a), _layout(b)
    if p >= q + (nb - 1) * sb + lb or q >= p + (na - 1) * sa + la:
        return False
    s = sa or sb
    if (sa and sb and sa != sb) or max(la, lb) > s:
        return True
    # row j of b begins r bytes into row k + j of a
    k, r = divmod(q - p, s)
    return (r < la and -nb < k < na) or (r + lb > s and -nb < k + 1 < na)


def _overlaps(out, *inputs) -> bool:
    return any(a is not None and _bytes_overlap(out, a) for a in inputs)


# ------------------------------------------------------------------ root-mean-square norm
_norm_descs: dict = {}


def rms_norm(x, weight=None, *, residual=None, eps: float = 1e-6, weight_offset: float = 0.0, out_dtype=None,
             out=None, residual_out=None, stream=None):
    """y = h / sqrt(mean(h^2) + eps) * (weight + weight_offset) along the last of x's two dimensions, with
    h = x, or with a residual h = x + residual rounded to the residual's dtype (gemm_rms_norm).

    x [T, H]: FP32, FP16 or BF16, rows contiguous; weight [H] of any of these (None: ones); residual [T, H]:
    FP32 or x's dtype.  out_dtype: "f32", "f16", "bf16" (default: x's), or "mxfp8", which gives an Fp8Tensor for
    fp8_matmul.  Returns y, or with a residual (y, h).  residual_out may be residual or x itself and out may be x
    or residual (in place: same dtype and strides); they overlap nothing else.  A row's sum of squares must stay below
    2^128 (beyond it y is 0).  With `stream`, the call runs, and allocates, as if that were the current stream.
    """
    what, t = "rms_norm", _t()
    index = x.get_device()
    if stream is not None or (index != t.device_index() and index >= 0):
        with t.on(stream, index) if stream is not None else t.torch.cuda.device(index):
            return rms_norm(x, weight, residual=residual, eps=eps, weight_offset=weight_offset, out_dtype=out_dtype,
                            out=out, residual_out=residual_out)
    # what the checks below look at, apart from the addresses: arguments that passed them once pass them again
    key = (x.shape, x.stride(), x.dtype, index, eps, weight_offset, out_dtype,
           None if weight is None else (weight.shape, weight.stride(), weight.dtype, weight.get_device()),
           None if residual is None else (residual.shape, residual.stride(), residual.dtype, residual.get_device()),
           None if out is None else (out.shape, out.stride(), out.dtype, out.get_device()),
           None if residual_out is None else (residual_out.shape, residual_out.stride(), residual_out.dtype,
                                              residual_out.get_device()))
    known = _norm_descs.get(key)
    if known is None:
        known = _check_norm(t, what, x, weight, residual, eps, weight_offset, out_dtype, out, residual_out, index)
        if len(_norm_descs) > 4096:
            _norm_descs.clear()
        _norm_descs[key] = known
    d, T, H, odt = known
    if out is not None or residual_out is not None:
        _check_norm_overlap(what, x, weight, residual, residual_out, out)
    h = residual_out
    if residual is not None and h is None:
        h = t.empty((T, H), dtype=residual.dtype, device=x.device)
    if odt is None:
        y = _new_fp8(t, T, H, x.device, index)
        p, ps, _ = y._ptrs()
    else:
        y = t.empty((T, H), dtype=odt, device=x.device) if out is None else out
        p, ps = y.data_ptr(), None
    rc = (_lib_of() or lib()).gemm_rms_norm(d, x.data_ptr(), None if residual is None else residual.data_ptr(),
                                            None if weight is None else weight.data_ptr(),
                                            None if h is None else h.data_ptr(), p, ps, t.raw_stream(index))
    if rc != 0:
        raise GemmError(rc, what)
    return y if residual is None else (y, h)


def _check_norm(t, what, x, weight, residual, eps, weight_offset, out_dtype, out, residual_out, index):
    """(gemm_norm_desc_t, T, H, the output's torch dtype or None for mxfp8), or a refusal."""
    dt = t.name.get(x.dtype)
    if dt is None or x.dim() != 2 or index < 0:
        _refuse(what, "x: a 2-D CUDA tensor in f32, f16 or bf16 is wanted")
    T, H = x.shape
    ldx, step = x.stride()
    if T <= 1:
        ldx = H
    if H < 1 or (H > 1 and step != 1) or ldx < H:
        _refuse(what, "x: at least one column, rows contiguous and not overlapping, are wanted")
    wdt = "f32"
    if weight is not None:
        wdt = t.name.get(weight.dtype)
        if wdt is None or weight.dim() != 1 or weight.shape[0] != H or weight.get_device() != index \
                or (H > 1 and weight.stride(0) != 1):
            _refuse(what, "weight: contiguous [H] in f32, f16 or bf16 on x's device is wanted")
    rdt, ldr, ldh, ldy = dt, 0, 0, 0
    if residual is not None:
        rdt = t.name.get(residual.dtype)
        if rdt not in ("f32", dt) or not _out_ok(t, residual, (T, H), rdt, index):
            _refuse(what, "residual: a row-major [T, H] in f32 or x's dtype on x's device is wanted")
        ldr = _ld(residual) if T > 1 else H
        ldh = H
        if residual_out is not None:
            if not _out_ok(t, residual_out, (T, H), rdt, index):
                _refuse(what, "residual_out: a row-major [T, H] of the residual's dtype on x's device is wanted")
            ldh = _ld(residual_out) if T > 1 else H
    elif residual_out is not None:
        _refuse(what, "residual_out without a residual")
    f8 = out_dtype == "mxfp8"
    odt = dt if out_dtype is None or f8 else out_dtype
    if f8 and out is not None:
        _refuse(what, "out: mxfp8 makes its own arrays")
    if odt not in DTYPES:
        _refuse(what, f"unknown out_dtype {out_dtype!r}")
    if not f8:
        ldy = H
        if out is not None:
            if not _out_ok(t, out, (T, H), odt, index):
                _refuse(what, f"out: a row-major {odt} [T, H] on x's device is wanted")
            ldy = _ld(out) if T > 1 else H
    d = _NormDesc(DTYPES[dt], residual is not None, DTYPES[rdt], DTYPES[wdt], DTYPES[odt], f8, T, H, ldx, ldr, ldh, ldy,
                  eps, weight_offset)
    return ctypes.byref(d), T, H, None if f8 else t.dtype[odt]


def _check_norm_overlap(what, x, weight, residual, h, out):
    """Refuses outputs that overlap an input or one another otherwise than in place."""
    def bad(o, i):
        if i is None or o is None or not _bytes_overlap(o, i):
            return False
        return not (o.data_ptr() == i.data_ptr() and o.dtype is i.dtype and o.shape == i.shape
                    and (o.shape[0] <= 1 or o.stride(0) == i.stride(0)))
    for o in (h, out):
        if o is not None and (bad(o, x) or bad(o, residual) or (weight is not None and _bytes_overlap(o, weight))):
            _refuse(what, "an output overlaps an input (in place: the same tensor, dtype and strides)")
    if h is not None and out is not None and _bytes_overlap(h, out):
        _refuse(what, "out and residual_out overlap")


# ------------------------------------------------------------------ 8-bit floats
class Fp8Tensor:
    """A matrix in mxfp8 (layout: include/gemm13.h, "8-bit floats"); read-only.

    codes: uint8 [rows, row_bytes]; scales: uint8, flat.  Arrays that do not fit the sizes are refused here, once.
    """

    __slots__ = ("_codes", "_scales", "_rows", "_cols", "_index", "_both")

    def __init__(self, codes, scales, rows, cols):
        t = _t()
        n_codes, n_scales = _fp8_sizes(rows, cols)
        index = codes.get_device()
        if (index < 0 or scales.get_device() != index or codes.dtype is not t.u8 or scales.dtype is not t.u8
                or rows < 0 or cols < 0 or codes.numel() != n_codes or scales.numel() != n_scales
                or not codes.is_contiguous() or not scales.is_contiguous()):
            _refuse("Fp8Tensor", f"{rows} x {cols}: codes ({n_codes} bytes) and scales ({n_scales} bytes), contiguous "
                                 "uint8 on the GPU, are wanted")
        self._codes, self._scales, self._rows, self._cols = codes, scales, rows, cols
        self._index, self._both = index, None

    @property
    def codes(self):
        if self._codes is None:
            row = (self._cols + 31) // 32 * 32
            self._codes = self._both[: self._rows * row].view(self._rows, row)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            self._scales = self._both[self._rows * ((self._cols + 31) // 32 * 32):]
        return self._scales

    rows = property(lambda self: self._rows)
    cols = property(lambda self: self._cols)
    format = _format = property(lambda self: "mxfp8")

    def _ptrs(self):
        """Addresses of codes and scales (and None, the tensor scale that this format lacks)."""
        if self._both is not None:
            p = self._both.data_ptr()
            return p, p + self._rows * ((self._cols + 31) // 32 * 32), None
        return self._codes.data_ptr(), self._scales.data_ptr(), None


def _fp8_sizes(rows: int, cols: int) -> tuple[int, int]:
    return rows * ((cols + 31) // 32 * 32), (rows + 127) // 128 * ((cols + 127) // 128) * 512


def _new_fp8(t, rows: int, cols: int, device, index: int) -> Fp8Tensor:
    """An Fp8Tensor to be written, codes and scales in one allocation (codes are a multiple of 32 bytes)."""
    q = Fp8Tensor.__new__(Fp8Tensor)
    n_codes, n_scales = _fp8_sizes(rows, cols)
    q._both = t.empty(n_codes + n_scales, dtype=t.u8, device=device)
    q._codes = q._scales = None
    q._rows, q._cols, q._index = rows, cols, index
    return q


def _is_fp8(what: str, *tensors):
    for q in tensors:
        if type(q) is not Fp8Tensor:
            _refuse(what, "an Fp8Tensor (fp8_quantize, rms_norm) is wanted")


def fp8_quantize(x, stream=None) -> Fp8Tensor:
    """A 2-D CUDA tensor (FP32, FP16 or BF16, any row stride) in mxfp8 (gemm_fp8_quantize)."""
    what, t = "fp8_quantize", _t()
    dt, index = t.name.get(x.dtype), x.get_device()
    if dt is None or x.dim() != 2 or index < 0:
        _refuse(what, "a 2-D CUDA tensor in f32, f16 or bf16 is wanted")
    if stream is not None or index != t.device_index():
        with t.on(stream, index) if stream is not None else t.torch.cuda.device(index):
            return fp8_quantize(x)
    if not _rows_ok(x):
        x = x.contiguous()
    rows, cols = x.shape
    q = _new_fp8(t, rows, cols, x.device, index)
    codes, scales, _ = q._ptrs()
    rc = lib().gemm_fp8_quantize(DTYPES[dt], rows, cols, x.data_ptr(), max(_ld(x), 1), codes, scales,
                                 t.raw_stream(index))
    if rc != 0:
        raise GemmError(rc, what)
    return q


def fp8_dequantize(q: Fp8Tensor, dtype: str = "f32", out=None, stream=None):
    """The values of an mxfp8 matrix as a tensor of `dtype` (gemm_fp8_dequantize)."""
    what, t = "fp8_dequantize", _t()
    code = DTYPES.get(dtype)
    if code is None:
        _refuse(what, f"unknown dtype {dtype!r}")
    _is_fp8(what, q)
    index, rows, cols = q._index, q._rows, q._cols
    if stream is not None or index != t.device_index():
        with t.on(stream, index) if stream is not None else t.torch.cuda.device(index):
            return fp8_dequantize(q, dtype, out)
    if out is None:
        out, ld = t.empty((rows, cols), dtype=t.dtype[dtype], device=t.device(index)), cols or 1
    else:
        if not _out_ok(t, out, (rows, cols), dtype, index):
            _refuse(what, "out: a row-major tensor of the matrix's shape, dtype and device is wanted")
        ld = max(_ld(out), 1)
    codes, scales, _ = q._ptrs()
    rc = lib().gemm_fp8_dequantize(code, rows, cols, codes, scales, out.data_ptr(), ld, t.raw_stream(index))
    if rc != 0:
        raise GemmError(rc, what)
    return out


class Fp8Plan:
    """Owns a gemm_fp8_plan_t; destroyed with the object (or explicitly)."""

    def __init__(self, handle: int, M: int, N: int, K: int, epilogue: Epilogue):
        self.handle = handle
        self.M, self.N, self.K, self.epilogue = M, N, K, epilogue

    def destroy(self):
        if self.handle:
            lib().gemm_fp8_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def gemm_fp8_plan(M: int, N: int, K: int, ldc: int, epilogue: Epilogue | None = None) -> Fp8Plan:
    """gemm_fp8_plan; the epilogue's b_layout must be "nk".  Raises GemmError on a non-OK status."""
    ep = epilogue or Epilogue(b_layout="nk")
    h, ce = ctypes.c_void_p(), ep._c()
    rc = lib().gemm_fp8_plan(M, N, K, ldc, ctypes.byref(ce), ctypes.byref(h))
    if rc != 0:
        raise GemmError(rc, "gemm_fp8_plan")
    return Fp8Plan(h.value, M, N, K, ep)


def gemm_fp8_run(plan: Fp8Plan, A: Fp8Tensor, B: Fp8Tensor, C, bias=None, residual=None, alpha: float = 1.0,
                 stream=None) -> int:
    """Enqueue C = epilogue(A @ B.T) of a plan on `stream` (default: torch's current stream)."""
    what = "gemm_fp8_run"
    _is_fp8(what, A, B)
    if (A._rows, A._cols, B._rows, B._cols) != (plan.M, plan.K, plan.N, plan.K):
        _refuse(what, "the operands do not fit the plan")
    t = _t()
    index = t.device_index()
    if A._index != index or B._index != index:
        _refuse(what, "the operands are not on the current device")
    _on_device(what, index, C, bias, residual)
    (ac, as_, _), (bc, bs, _) = A._ptrs(), B._ptrs()
    rc = lib().gemm_fp8_run(plan.handle, ac, as_, bc, bs, _ptr(C), _ptr(bias), _ptr(residual), alpha,
                            _stream(t, index, stream))
    if rc != 0:
        raise GemmError(rc, what)
    return rc


def gemm_fp8_status(plan: Fp8Plan) -> int:
    """Synchronise and return the plan's sticky device status (0 or a negative code)."""
    return int(lib().gemm_fp8_status(plan.handle))


def gemm_fp8_select_config(M: int, N: int, K: int, num_sms: int = 152) -> Config:
    """Host-only query of the 8-bit product's tile (no GPU needed)."""
    c = _Config()
    rc = lib().gemm_fp8_select_config(M, N, K, num_sms, ctypes.byref(c))
    if rc != 0:
        raise GemmError(rc, "gemm_fp8_select_config")
    return Config._from(c)


_fp8_plans: dict = {}


def fp8_matmul(A: Fp8Tensor, B: Fp8Tensor, *, alpha=1.0, bias=None, act="none", residual=None, beta=1.0,
               out_dtype="f32", out=None, stream=None):
    """C = cast(act(alpha * A @ B.T + bias) + beta * residual) of two mxfp8 matrices.

    A [M, K] (activations: rms_norm, fp8_quantize), B [N, K] (a weight as it lies for x @ W.T); the other arguments,
    the plans that are kept, streams and graph captures as in fp4_matmul.
    """
    what, t = "fp8_matmul", _t()
    _is_fp8(what, A, B)
    index, M, K, N = A._index, A._rows, A._cols, B._rows
    if B._index != index or B._cols != K:
        _refuse(what, "A and B need the same K and device")
    if stream is not None or index != t.device_index():
        with t.on(stream, index) if stream is not None else t.torch.cuda.device(index):
            return fp8_matmul(A, B, alpha=alpha, bias=bias, act=act, residual=residual, beta=beta,
                              out_dtype=out_dtype, out=out)
    if out_dtype not in DTYPES or act not in ("none", "gelu", "relu"):
        _refuse(what, "out_dtype: f32, f16 or bf16; act: none, gelu or relu")
    _check_epilogue(t, what, bias, residual, M, N, index)
    if out is None:
        out, ldc = t.empty((M, N), dtype=t.dtype[out_dtype], device=t.device(index)), N or 1
    else:
        if not _out_ok(t, out, (M, N), out_dtype, index):
            _refuse(what, f"out: a row-major {out_dtype} [M, N] on the operands' device is wanted")
        ldc = _ld(out)
    ldr = 0 if residual is None else _ld(residual)
    key = (M, N, K, ldc, ldr, out_dtype, bias is not None, act, beta, index)
    pl = _fp8_plans.get(key)
    if pl is None:
        _no_capture(t, what)
        ep = Epilogue(b_layout="nk", out_dtype=out_dtype, bias=bias is not None, act=act,
                      residual=residual is not None, beta=beta, ldr=ldr)
        pl = _keep(_fp8_plans, key, lambda: gemm_fp8_plan(M, N, K, ldc, ep))
    (ac, as_, _), (bc, bs, _) = A._ptrs(), B._ptrs()
    rc = (_lib_of() or lib()).gemm_fp8_run(pl.handle, ac, as_, bc, bs, out.data_ptr(), _ptr(bias), _ptr(residual), alpha,
                            t.raw_stream(index))
    if rc != 0:
        raise GemmError(rc, what)
    return out


def _check_epilogue(t, what: str, bias, residual, M: int, N: int, index: int):
    if bias is not None and (bias.dtype is not t.f32 or tuple(bias.shape) != (N,) or bias.get_device() != index
                             or not bias.is_contiguous()):
        _refuse(what, "bias: contiguous FP32 [N] on the operands' device is wanted")
    if residual is not None and (tuple(residual.shape) != (M, N) or residual.dtype is not t.f32
                                 or residual.get_device() != index or not _rows_ok(residual)):
        _refuse(what, "residual: a row-major f32 [M, N] on the operands' device is wanted")


# ------------------------------------------------------------------ 4-bit weights with group scales
class W4Tensor:
    """A weight [rows, cols] in 4 bits with group scales (layout: include/gemm13.h, "4-bit weights"); read-only.

    codes: uint8, flat; scales: FP16 or BF16, flat; zeros: uint8, flat, or None (8).  Arrays that do not fit the
    sizes are refused here, once.
    """

    __slots__ = ("_codes", "_scales", "_zeros", "_rows", "_cols", "_group", "_dtype", "_index", "_descs")

    def __init__(self, codes, scales, zeros, rows, cols, group=128):
        t, what = _t(), "W4Tensor"
        n_codes, n_scales = _w4_sizes(what, rows, cols, group)
        index, dt = codes.get_device(), t.name.get(scales.dtype)
        arrays = [(codes, n_codes), (scales, n_scales)] + ([] if zeros is None else [(zeros, n_scales)])
        if (index < 0 or dt not in ("f16", "bf16") or codes.dtype is not t.u8
                or (zeros is not None and zeros.dtype is not t.u8)
                or any(a.get_device() != index or a.numel() != n or not a.is_contiguous() for a, n in arrays)):
            _refuse(what, f"{rows} x {cols}, groups of {group}: codes ({n_codes} uint8), scales ({n_scales} FP16 or "
                          f"BF16) and zeros (as many uint8, or None), contiguous on the GPU, are wanted")
        self._set(codes, scales, zeros, rows, cols, group, dt, index)

    def _set(self, codes, scales, zeros, rows, cols, group, dt, index):
        self._codes, self._scales, self._zeros = codes, scales, zeros
        self._rows, self._cols, self._group, self._dtype, self._index = rows, cols, group, dt, index
        self._descs = {}
        return self

    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)
    zeros = property(lambda self: self._zeros)
    rows = property(lambda self: self._rows)
    cols = property(lambda self: self._cols)
    group = property(lambda self: self._group)
    dtype = property(lambda self: self._dtype)


def _w4_sizes(what: str, rows: int, cols: int, group: int) -> tuple[int, int]:
    if group < 32 or group % 32 or group > 65536 or cols < 1 or cols > 65536 or rows < 0 or rows > 1 << 28:
        _refuse(what, "rows 0 to 2^28, cols 1 to 65536 and a group that is a multiple of 32 (up to 65536) are wanted")
    tiles = (rows + 15) // 16
    return tiles * ((cols + 63) // 64) * 512, tiles * 16 * ((cols + group - 1) // group)


def _new_w4(t, what, rows, cols, group, dt, zeros: bool, device, index) -> W4Tensor:
    n_codes, n_scales = _w4_sizes(what, rows, cols, group)
    return W4Tensor.__new__(W4Tensor)._set(
        t.empty(n_codes, dtype=t.u8, device=device), t.empty(n_scales, dtype=t.dtype[dt], device=device),
        t.empty(n_scales, dtype=t.u8, device=device) if zeros else None, rows, cols, group, dt, index)


def w4_quantize(w, group: int = 128, *, symmetric: bool = False, dtype: str | None = None, stream=None) -> W4Tensor:
    """A weight [N, K] (FP32, FP16 or BF16, any row stride) rounded to 4 bits with group scales (gemm_w4_quantize).

    dtype: of the scales, and of the activations that it is to be multiplied with ("bf16" or "f16"; default: w's,
    or "bf16").  symmetric: no zeros, w = (q - 8) * s.
    """
    what, t = "w4_quantize", _t()
    wdt, index = t.name.get(w.dtype), w.get_device()
    if wdt is None or w.dim() != 2 or index < 0:
        _refuse(what, "a 2-D CUDA tensor in f32, f16 or bf16 is wanted")
    dt = dtype or ("bf16" if wdt == "f32" else wdt)
    if dt not in ("f16", "bf16"):
        _refuse(what, "dtype: f16 or bf16 is wanted")
    if stream is not None or index != t.device_index():
        with t.on(stream, index) if stream is not None else t.torch.cuda.device(index):
            return w4_quantize(w, group, symmetric=symmetric, dtype=dtype)
    if not _rows_ok(w):
        w = w.contiguous()
    rows, cols = w.shape
    q = _new_w4(t, what, rows, cols, group, dt, not symmetric, w.device, index)
    rc = lib().gemm_w4_quantize(DTYPES[wdt], DTYPES[dt], rows, cols, group, w.data_ptr(), _ld(w), q._codes.data_ptr(),
                                q._scales.data_ptr(), _ptr(q._zeros), t.raw_stream(index))
    if rc != 0:
        raise GemmError(rc, what)
    return q


def w4_pack(codes, scales, zeros=None, group: int = 128, stream=None) -> W4Tensor:
    """A checkpoint's 4-bit weight in the library's layout (gemm_w4_pack).

    codes: uint8 [N, K], one code (0 to 15) a byte; scales: FP16 or BF16 [N, ceil(K / group)]; zeros: uint8 of the
    same shape (0 to 15), or None (8); rows contiguous.
    """
    what, t = "w4_pack", _t()
    index = codes.get_device()
    if index < 0 or codes.dtype is not t.u8 or codes.dim() != 2:
        _refuse(what, "codes: a 2-D uint8 CUDA tensor is wanted")
    rows, cols = codes.shape
    _w4_sizes(what, rows, cols, group)
    dt, shape = t.name.get(scales.dtype), (rows, -(-cols // group))
    if dt not in ("f16", "bf16") or any(
            a is not None and (tuple(a.shape) != shape or a.get_device() != index) for a in (scales, zeros)) \
            or (zeros is not None and zeros.dtype is not t.u8):
        _refuse(what, f"scales (f16 or bf16) and zeros (uint8) {list(shape)} on the codes' device are wanted")
    if stream is not None or index != t.device_index():
        with t.on(stream, index) if stream is not None else t.torch.cuda.device(index):
            return w4_pack(codes, scales, zeros, group)
    codes, scales, zeros = (a if a is None or _rows_ok(a) else a.contiguous() for a in (codes, scales, zeros))
    q = _new_w4(t, what, rows, cols, group, dt, zeros is not None, codes.device, index)
    rc = lib().gemm_w4_pack(rows, cols, group, codes.data_ptr(), _ld(codes), scales.data_ptr(), _ld(scales),
                            _ptr(zeros), 0 if zeros is None else _ld(zeros), q._codes.data_ptr(),
                            q._scales.data_ptr(), _ptr(q._zeros), t.raw_stream(index))
    if rc != 0:
        raise GemmError(rc, what)
    return q


def w4_dequantize(q: W4Tensor, dtype: str = "f32", out=None, stream=None):
    """The values (code - zero) * scale of a 4-bit weight as a tensor of `dtype` (gemm_w4_dequantize)."""
    what, t = "w4_dequantize", _t()
    code = DTYPES.get(dtype)
    if code is None:
        _refuse(what, f"unknown dtype {dtype!r}")
    if type(q) is not W4Tensor:
        _refuse(what, "a W4Tensor is wanted")
    index, shape = q._index, (q._rows, q._cols)
    if stream is not None or index != t.device_index():
        with t.on(stream, index) if stream is not None else t.torch.cuda.device(index):
            return w4_dequantize(q, dtype, out)
    if out is None:
        out = t.empty(shape, dtype=t.dtype[dtype], device=t.device(index))
    elif not _out_ok(t, out, shape, dtype, index):
        _refuse(what, "out: a row-major tensor of the weight's shape, dtype and device is wanted")
    rc = lib().gemm_w4_dequantize(code, DTYPES[q._dtype], *shape, q._group, q._codes.data_ptr(), q._scales.data_ptr(),
                                  _ptr(q._zeros), out.data_ptr(), _ld(out), t.raw_stream(index))
    if rc != 0:
        raise GemmError(rc, what)
    return out


def w4_matmul(x, w: W4Tensor, *, alpha=1.0, bias=None, act="none", residual=None, beta=1.0, out_dtype=None, out=None,
              stream=None):
    """y = cast(act(alpha * x @ W.T + bias) + beta * residual) for 1 to 64 tokens and a 4-bit weight (gemm_w4_run).

    x [M, K] in the dtype of W's scales, rows contiguous; bias: FP32 [N]; residual: FP32 [M, N]; out_dtype: "f32",
    "f16" or "bf16" (default: x's).  out overlaps no input.  A NaN stays one with any activation; should a wait inside the
    kernel run out, after 2 s, 128 columns of y are NaN.  With `stream`, the call runs, and allocates, as if that were the
    current stream.
    """
    what, t = "w4_matmul", _t()
    if type(w) is not W4Tensor:
        _refuse(what, "w: a W4Tensor is wanted")
    index = w._index
    if stream is not None or index != t.device_index():
        with t.on(stream, index) if stream is not None else t.torch.cuda.device(index):
            return w4_matmul(x, w, alpha=alpha, bias=bias, act=act, residual=residual, beta=beta,
                             out_dtype=out_dtype, out=out)
    if bias is not None or residual is not None:
        _check_epilogue(t, what, bias, residual, x.shape[0] if x.dim() == 2 else -1, w._rows, index)
    if out is not None and _overlaps(out, x, bias, residual, w._codes, w._scales, w._zeros):
        _refuse(what, "out overlaps an input")
    # what the checks look at: arguments that passed them once pass them again
    key = (x.shape, x.stride(), x.dtype, x.get_device(), out_dtype, act, bias is None, beta,
           None if residual is None else residual.stride(),
           None if out is None else (out.shape, out.stride(), out.dtype, out.get_device()))
    known = w._descs.get(key)
    if known is None:
        known = _check_w4(t, what, x, w, bias, act, residual, beta, out_dtype, out)
        if len(w._descs) > 256:
            w._descs.clear()
        w._descs[key] = known
    d, M, odt = known
    if out is None:
        out = t.empty((M, w._rows), dtype=odt, device=x.device)
    z = w._zeros
    rc = (_lib_of() or lib()).gemm_w4_run(d, x.data_ptr(), w._codes.data_ptr(), w._scales.data_ptr(),
                                          None if z is None else z.data_ptr(), out.data_ptr(),
                                          None if bias is None else bias.data_ptr(),
                                          None if residual is None else residual.data_ptr(), alpha,
                                          t.raw_stream(index))
    if rc != 0:
        raise GemmError(rc, what)
    return out


def _check_w4(t, what, x, w, bias, act, residual, beta, out_dtype, out):
    """(gemm_w4_desc_t, M, the output's torch dtype), or a refusal."""
    dt, index, N, K = w._dtype, w._index, w._rows, w._cols
    if x.dim() != 2 or t.name.get(x.dtype) != dt or x.get_device() != index or x.shape[1] != K:
        _refuse(what, f"x: [M, {K}] in {dt} on the weight's device is wanted")
    M = x.shape[0]
    if M > 64:
        _refuse(what, "at most 64 tokens (more: w4_dequantize, then matmul)")
    ldx, step = x.stride()
    if M <= 1:
        ldx = K
    if (K > 1 and step != 1) or ldx < K:
        _refuse(what, "x: rows contiguous and not overlapping are wanted")
    odt = dt if out_dtype is None else out_dtype
    if odt not in DTYPES or act not in ("none", "gelu", "relu"):
        _refuse(what, "out_dtype: f32, f16 or bf16; act: none, gelu or relu")
    if out is not None and not _out_ok(t, out, (M, N), odt, index):
        _refuse(what, f"out: a row-major {odt} [M, N] on the weight's device is wanted")
    ldy = N if out is None else _ld(out)
    ldr = 0 if residual is None else _ld(residual)
    d = _W4Desc(DTYPES[dt], DTYPES[odt], M, N, K, w._group, w._zeros is not None, bias is not None, ACTS[act],
                residual is not None, beta, ldx, ldy, ldr)
    return ctypes.byref(d), M, t.dtype[odt]


# ------------------------------------------------------------------ routing to experts
_route_descs: dict = {}


def route(logits, top_k: int, *, scores: str = "softmax", bias=None, groups: int = 1, top_groups: int | None = None,
          group_score: str = "max", normalize: bool = True, scale: float = 1.0, stream=None):
    """The experts of each token and their weights, from logits [T, E] (gemm_route).

    scores: "softmax" or "sigmoid"; bias: FP32 [E], enters the choice and not the weights; groups, top_groups: only
    the top_groups best of `groups` equal groups are chosen from (default: all), by their largest score
    (group_score "max") or the sum of their two largest ("top2").  Logits: FP32, FP16 or BF16, rows contiguous, any
    number of tokens.  Returns (expert ids int32 [T, top_k], weights FP32 [T, top_k]), largest first; moe_experts
    takes them.  With `stream`, the call runs, and allocates, as if that were the current stream.
    """
    what, t = "route", _t()
    index = logits.get_device()
    if stream is not None or (index != t.device_index() and index >= 0):
        with t.on(stream, index) if stream is not None else t.torch.cuda.device(index):
            return route(logits, top_k, scores=scores, bias=bias, groups=groups, top_groups=top_groups,
                         group_score=group_score, normalize=normalize, scale=scale)
    # what the checks look at: arguments that passed them once pass them again
    key = (logits.shape, logits.stride(), logits.dtype, index, top_k, scores, groups, top_groups, group_score, normalize,
           scale, None if bias is None else (bias.shape, bias.stride(), bias.dtype, bias.get_device()))
    known = _route_descs.get(key)
    if known is None:
        known = _check_route(t, what, logits, top_k, scores, bias, groups, top_groups, group_score, normalize, scale,
                             index)
        if len(_route_descs) > 4096:
            _route_descs.clear()
        _route_descs[key] = known
    d, T = known
    ids = t.empty((T, top_k), dtype=t.i32, device=logits.device)
    weights = t.empty((T, top_k), dtype=t.f32, device=logits.device)
    rc = (_lib_of() or lib()).gemm_route(d, logits.data_ptr(), None if bias is None else bias.data_ptr(),
                                         ids.data_ptr(), weights.data_ptr(), t.raw_stream(index))
    if rc != 0:
        raise GemmError(rc, what)
    return ids, weights


def _check_route(t, what, logits, top_k, scores, bias, groups, top_groups, group_score, normalize, scale, index):
    """(gemm_route_desc_t, T), or a refusal."""
    dt = t.name.get(logits.dtype)
    if dt is None or logits.dim() != 2 or index < 0:
        _refuse(what, "logits: a 2-D CUDA tensor in f32, f16 or bf16 is wanted")
    T, E = logits.shape
    ld, step = logits.stride()
    if T <= 1:
        ld = E
    if (E > 1 and step != 1) or ld < E:
        _refuse(what, "logits: rows contiguous and not overlapping are wanted")
    if scores not in ROUTE_SCORES or group_score not in ROUTE_GROUP_SCORES:
        _refuse(what, "scores: softmax or sigmoid; group_score: max or top2")
    if bias is not None and (bias.dtype is not t.f32 or bias.dim() != 1 or bias.shape[0] != E
                             or bias.get_device() != index or not bias.is_contiguous()):
        _refuse(what, "bias: contiguous FP32 [E] on the logits' device is wanted")
    if top_k < 1:
        _refuse(what, "top_k: at least 1 is wanted")
    d = _RouteDesc(DTYPES[dt], T, E, top_k, ROUTE_SCORES[scores], groups, groups if top_groups is None else top_groups,
                   ROUTE_GROUP_SCORES[group_score], bool(normalize), scale, ld)
    return ctypes.byref(d), T


def gemm_moe_run_routed(plan: MoePlan, X, expert_ids, expert_weights, W1, W2, Y, workspace, stream=None) -> int:
    """Enqueue one layer whose experts are chosen already on `stream` (default: torch's current stream)."""
    what, t = "gemm_moe_run_routed", _t()
    index = t.device_index()
    _on_device(what, index, X, expert_ids, expert_weights, W1, W2, Y, workspace)
    if hasattr(workspace, "numel") and workspace.numel() * workspace.element_size() < plan.workspace_bytes:
        _refuse(what, f"workspace: {plan.workspace_bytes} bytes are wanted")
    rc = lib().gemm_moe_run_routed(plan.handle, _ptr(X), _ptr(expert_ids), _ptr(expert_weights), _ptr(W1), _ptr(W2),
                                   _ptr(Y), _ptr(workspace), _stream(t, index, stream))
    if rc != 0:
        raise GemmError(rc, what)
    return rc


def moe_experts(x, w1, w2, expert_ids, expert_weights, *, act: str = "swiglu", out=None, stream=None):
    """The experts' part of a mixture-of-experts layer for 1 to 64 tokens (gemm_moe_run_routed).

    x [T, H], w1 and w2 as for moe_layer; expert_ids int32 [T, top_k] and expert_weights FP32 [T, top_k], contiguous, as
    route gives them (an id outside 0 .. E - 1 takes no part).  Returns y [T, H].  Plans, workspaces, `stream` and
    gemm_kept_status as for moe_layer.  out overlaps no input.
    """
    what, t = "moe_experts", _t()
    dt, dtype, index = t.name.get(x.dtype), x.dtype, x.get_device()
    if dt not in ("f16", "bf16") or act not in MOE_ACTS:
        _refuse(what, "FP16 or BF16 tensors and act gelu, relu or swiglu are wanted")
    if x.dim() != 2 or w1.dim() != 3 or w2.dim() != 3 or expert_ids.dim() != 2:
        _refuse(what, "x [T, H], w1 [E, I or 2I, H], w2 [E, H, I], expert_ids [T, top_k] are wanted")
    (T, H), (E, rows, H1), (E2, H2, I), (Tk, top_k) = x.shape, w1.shape, w2.shape, expert_ids.shape
    if not (H1 == H2 == H and E2 == E and Tk == T and rows == (2 * I if act == "swiglu" else I)) \
            or expert_weights.shape != expert_ids.shape or (out is not None and tuple(out.shape) != (T, H)):
        _refuse(what, "the shapes of x, w1, w2, expert_ids, expert_weights and out do not fit one another")
    if expert_ids.dtype is not t.i32 or expert_weights.dtype is not t.f32 or not expert_ids.is_contiguous() \
            or not expert_weights.is_contiguous():
        _refuse(what, "contiguous expert_ids (int32) and expert_weights (FP32) are wanted")
    if index < 0 or any(a.get_device() != index for a in (w1, w2, expert_ids, expert_weights)) \
            or w1.dtype is not dtype or w2.dtype is not dtype \
            or (out is not None and (out.get_device() != index or out.dtype is not dtype)):
        _refuse(what, "tensors of x's dtype on x's device, a GPU, are wanted")
    if out is not None and _overlaps(out, x, w1, w2, expert_ids, expert_weights):
        _refuse(what, "out overlaps an input")
    if stream is not None or index != t.device_index():
        with t.on(stream, index) if stream is not None else t.torch.cuda.device(index):
            return moe_experts(x, w1, w2, expert_ids, expert_weights, act=act, out=out)
    if out is None:
        out = t.empty((T, H), dtype=dtype, device=x.device)
    (ldx, cx), (ldy, cy), (st1, ld1, c1), (st2, ld2, c2) = x.stride(), out.stride(), w1.stride(), w2.stride()
    if (H > 1 and not cx == cy == c1 == 1) or (I > 1 and c2 != 1) or (T > 1 and (ldx < H or ldy < H)) \
            or (E > 1 and (st1 == 0 or st2 == 0)) or (rows > 1 and ld1 < H) or (H > 1 and ld2 < I):
        _refuse(what, "rows that are contiguous and not shared are wanted")
    # strides that no element uses may be anything
    if T <= 1:
        ldx = ldy = H
    if rows <= 1:
        ld1 = H
    if H <= 1:
        ld2 = I
    if E <= 1:
        st1, st2 = rows * ld1, H * ld2
    key = ("routed", dt, T, E, top_k, H, I, act, ldx, ld1, st1, ld2, st2, ldy, index)
    pl = _moe_plans.get(key)
    if pl is None:
        _no_capture(t, what)
        pl = _keep(_moe_plans, key, lambda: gemm_moe_plan(dt, T, E, top_k, H, I, act, ldx=ldx, ld_w1=ld1,
                                                          stride_w1=st1, ld_w2=ld2, stride_w2=st2, ldy=ldy))
    ws = t.empty(pl.workspace_bytes, dtype=t.u8, device=x.device)
    rc = lib().gemm_moe_run_routed(pl.handle, x.data_ptr(), expert_ids.data_ptr(), expert_weights.data_ptr(),
                                   w1.data_ptr(), w2.data_ptr(), out.data_ptr(), ws.data_ptr(), t.raw_stream(index))
    if rc != 0:
        raise GemmError(rc, what)
    return out
