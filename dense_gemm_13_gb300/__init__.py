"""Thin Python binding of libgemm13.so (the C ABI declared in include/gemm13.h).

Argument marshalling only: every step of the GEMM runs in the library's CUDA
kernels.  PyTorch is used for device memory and the current stream; tensors
are passed as raw device pointers.  If the shared object is missing or fails
to load, every call raises -- there is no fallback.

    import dense_gemm_13_gb300 as g13
    plan = g13.gemm_plan("bf16", M, N, K, lda, ldb, ldc, g13.Epilogue(b_layout="nk"))
    g13.gemm_run(plan, A, B, C, alpha=1.0)       # torch CUDA tensors
"""
from __future__ import annotations

import ctypes
import os
import threading

__all__ = ["Epilogue", "Config", "Plan", "GemmError", "gemm_plan", "gemm_run", "gemm_plan_status",
           "gemm_plan_info", "gemm_select_config", "gemm_cache_stats", "gemm_cache_clear",
           "gemm_strerror", "gemm_version", "gemm_run_noalloc", "lib", "load", "matmul", "DTYPES", "ACTS", "LAYOUTS",
           "KERNELS", "LIB_PATH", "FP4_FORMATS", "Fp4Tensor", "Fp4Plan", "fp4_quantize", "fp4_dequantize",
           "gemm_fp4_plan", "gemm_fp4_run", "gemm_fp4_status", "gemm_fp4_select_config", "fp4_matmul",
           "MOE_ACTS", "MoePlan", "gemm_moe_plan", "gemm_moe_run", "gemm_moe_status", "moe_layer", "gemm_kept_status"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgemm13.so")

DTYPES = {"f32": 0, "f16": 1, "bf16": 2}
ACTS = {"none": 0, "gelu": 1, "relu": 2, "softmax": 3}
LAYOUTS = {"kn": 0, "nk": 1}
KERNELS = {"auto": 0, "tc": 1, "ffma": 2, "skinny": 3, "tf32x3": 4}
KERNEL_NAMES = {v: k for k, v in KERNELS.items()}
FP4_FORMATS = {"mxfp4": 0, "nvfp4": 1}
MOE_ACTS = {"gelu": 0, "relu": 1, "swiglu": 2}
FLAG_FP32_TENSOR = 0x1         # FP32 inputs may run as 3xTF32 on the tensor cores
FLAG_TEST_STALL = 0x80000000
FLAG_TEST_STALL_PEER = 0x40000000   # test only: the second CTA withholds a tile

STATUS = {0: "GEMM_OK", -1: "GEMM_ERR_INVALID_ARG", -2: "GEMM_ERR_UNSUPPORTED",
          -3: "GEMM_ERR_MISALIGNED", -4: "GEMM_ERR_CUDA", -5: "GEMM_ERR_DEVICE_TIMEOUT",
          -6: "GEMM_ERR_BAD_PLAN", -7: "GEMM_ERR_NO_DEVICE", -8: "GEMM_ERR_OUT_OF_MEMORY",
          -9: "GEMM_ERR_SCRATCH_LIMIT"}


class GemmError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        name = STATUS.get(status, str(status))
        super().__init__(f"{what}: {name} ({_strerror(status)})" if what else name)


class _Epilogue(ctypes.Structure):
    _fields_ = [("b_layout", ctypes.c_int), ("out_dtype", ctypes.c_int), ("has_bias", ctypes.c_int),
                ("act", ctypes.c_int), ("has_residual", ctypes.c_int), ("beta", ctypes.c_float),
                ("ldr", ctypes.c_int64), ("batch", ctypes.c_int64), ("stride_a", ctypes.c_int64),
                ("stride_b", ctypes.c_int64), ("stride_c", ctypes.c_int64),
                ("stride_r", ctypes.c_int64), ("flags", ctypes.c_uint32),
                ("timeout_ms", ctypes.c_uint32)]


class _Config(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("bm", ctypes.c_int32), ("bn", ctypes.c_int32),
                ("bk", ctypes.c_int32), ("stages", ctypes.c_int32), ("split_k", ctypes.c_int32),
                ("raster_group", ctypes.c_int32), ("stage_a", ctypes.c_int32),
                ("stage_b", ctypes.c_int32), ("num_ctas", ctypes.c_int32),
                ("variant", ctypes.c_int32), ("stream_k", ctypes.c_int32)]


class _PlanInfo(ctypes.Structure):
    _fields_ = [("config", _Config), ("workspace_bytes", ctypes.c_int64),
                ("num_sms", ctypes.c_int32), ("device", ctypes.c_int32),
                ("cache_hit", ctypes.c_int32), ("kernels_per_run", ctypes.c_int32)]


class _MoeDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("T", ctypes.c_int64), ("E", ctypes.c_int64), ("top_k", ctypes.c_int64),
                ("H", ctypes.c_int64), ("I", ctypes.c_int64), ("act", ctypes.c_int), ("normalize", ctypes.c_int),
                ("ldx", ctypes.c_int64), ("ld_router", ctypes.c_int64), ("ld_w1", ctypes.c_int64),
                ("stride_w1", ctypes.c_int64), ("ld_w2", ctypes.c_int64), ("stride_w2", ctypes.c_int64),
                ("ldy", ctypes.c_int64), ("flags", ctypes.c_uint32), ("timeout_ms", ctypes.c_uint32)]


_lock = threading.Lock()
_lib = None


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libgemm13.so (built by __graft_entry__.build() / _build.build())."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is missing: build it with `python -m dense_gemm_13_gb300._build`"
                               " (no fallback path exists)")
        L = ctypes.CDLL(p)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        L.gemm_epilogue_init.argtypes = [ctypes.POINTER(_Epilogue)]
        L.gemm_epilogue_init.restype = None
        L.gemm_plan.argtypes = [i32, i64, i64, i64, i64, i64, i64, ctypes.POINTER(_Epilogue),
                                ctypes.POINTER(vp)]
        L.gemm_plan.restype = i32
        L.gemm_plan_with_config.argtypes = [i32, i64, i64, i64, i64, i64, i64,
                                            ctypes.POINTER(_Epilogue), ctypes.POINTER(_Config),
                                            ctypes.POINTER(vp)]
        L.gemm_plan_with_config.restype = i32
        L.gemm_run.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.c_float, vp]
        L.gemm_run.restype = i32
        L.gemm_plan_status.argtypes = [vp]
        L.gemm_plan_status.restype = i32
        L.gemm_plan_info.argtypes = [vp, ctypes.POINTER(_PlanInfo)]
        L.gemm_plan_info.restype = i32
        L.gemm_plan_destroy.argtypes = [vp]
        L.gemm_plan_destroy.restype = None
        L.gemm_select_config.argtypes = [i32, i64, i64, i64, i64, i64, i64,
                                         ctypes.POINTER(_Epilogue), ctypes.c_int32,
                                         ctypes.POINTER(_Config)]
        L.gemm_select_config.restype = i32
        L.gemm_cache_stats.argtypes = [ctypes.POINTER(i64)] * 3
        L.gemm_cache_stats.restype = None
        L.gemm_cache_clear.argtypes = []
        L.gemm_cache_clear.restype = None
        L.gemm_strerror.argtypes = [i32]
        L.gemm_strerror.restype = ctypes.c_char_p
        L.gemm_version.argtypes = []
        L.gemm_version.restype = ctypes.c_char_p
        L.gemm_run_noalloc.argtypes = [i32, i64, i64, i64, vp, i64, vp, i64, vp, i64,
                                       ctypes.POINTER(_Epilogue), vp, vp, ctypes.c_float, vp]
        L.gemm_run_noalloc.restype = i32
        L.gemm_fp4_row_bytes.argtypes = [i64]
        L.gemm_fp4_row_bytes.restype = i64
        L.gemm_fp4_scales_bytes.argtypes = [i32, i64, i64]
        L.gemm_fp4_scales_bytes.restype = i64
        L.gemm_fp4_quantize.argtypes = [i32, i32, i64, i64, vp, i64, vp, vp, vp, vp]
        L.gemm_fp4_quantize.restype = i32
        L.gemm_fp4_dequantize.argtypes = [i32, i32, i64, i64, vp, vp, vp, vp, i64, vp]
        L.gemm_fp4_dequantize.restype = i32
        L.gemm_fp4_plan.argtypes = [i32, i64, i64, i64, i64, ctypes.POINTER(_Epilogue), ctypes.POINTER(vp)]
        L.gemm_fp4_plan.restype = i32
        L.gemm_fp4_run.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, vp]
        L.gemm_fp4_run.restype = i32
        L.gemm_fp4_status.argtypes = [vp]
        L.gemm_fp4_status.restype = i32
        L.gemm_fp4_destroy.argtypes = [vp]
        L.gemm_fp4_destroy.restype = None
        L.gemm_fp4_select_config.argtypes = [i64, i64, i64, ctypes.c_int32, ctypes.POINTER(_Config)]
        L.gemm_fp4_select_config.restype = i32
        L.gemm_moe_desc_init.argtypes = [ctypes.POINTER(_MoeDesc)]
        L.gemm_moe_desc_init.restype = None
        L.gemm_moe_plan.argtypes = [ctypes.POINTER(_MoeDesc), ctypes.POINTER(vp)]
        L.gemm_moe_plan.restype = i32
        L.gemm_moe_workspace_bytes.argtypes = [vp]
        L.gemm_moe_workspace_bytes.restype = i64
        L.gemm_moe_run.argtypes = [vp] * 10
        L.gemm_moe_run.restype = i32
        L.gemm_moe_status.argtypes = [vp]
        L.gemm_moe_status.restype = i32
        L.gemm_moe_destroy.argtypes = [vp]
        L.gemm_moe_destroy.restype = None
        from . import blocks
        blocks.prototypes(L)
        if path is None:
            _lib = L
        return L


def lib() -> ctypes.CDLL:
    return _lib or load()


def _strerror(status: int) -> str:
    try:
        return lib().gemm_strerror(status).decode()
    except Exception:
        return "?"


def gemm_strerror(status: int) -> str:
    return lib().gemm_strerror(int(status)).decode()


def gemm_version() -> str:
    return lib().gemm_version().decode()


class Epilogue:
    """Python mirror of gemm_epilogue_t (defaults as in gemm_epilogue_init)."""

    def __init__(self, b_layout="kn", out_dtype="f32", bias=False, act="none", residual=False,
                 beta=1.0, ldr=0, batch=1, stride_a=0, stride_b=0, stride_c=0, stride_r=0,
                 flags=0, timeout_ms=0):
        self.b_layout, self.out_dtype, self.bias, self.act = b_layout, out_dtype, bias, act
        self.residual, self.beta, self.ldr, self.batch = residual, beta, ldr, batch
        self.stride_a, self.stride_b, self.stride_c, self.stride_r = stride_a, stride_b, stride_c, stride_r
        self.flags, self.timeout_ms = flags, timeout_ms

    def _c(self) -> _Epilogue:
        e = _Epilogue()
        lib().gemm_epilogue_init(ctypes.byref(e))
        e.b_layout = LAYOUTS[self.b_layout]
        e.out_dtype = DTYPES[self.out_dtype]
        e.has_bias = int(bool(self.bias))
        e.act = ACTS[self.act]
        e.has_residual = int(bool(self.residual))
        e.beta = float(self.beta)
        e.ldr, e.batch = int(self.ldr), int(self.batch)
        e.stride_a, e.stride_b = int(self.stride_a), int(self.stride_b)
        e.stride_c, e.stride_r = int(self.stride_c), int(self.stride_r)
        e.flags, e.timeout_ms = int(self.flags), int(self.timeout_ms)
        return e


class Config:
    """Python mirror of gemm_config_t."""

    def __init__(self, kernel="auto", bm=0, bn=0, bk=0, stages=0, split_k=1, raster_group=0,
                 stage_a=0, stage_b=0, num_ctas=0, variant=0, stream_k=0):
        self.kernel, self.bm, self.bn, self.bk, self.stages = kernel, bm, bn, bk, stages
        self.split_k, self.raster_group, self.stage_a, self.stage_b = split_k, raster_group, stage_a, stage_b
        self.num_ctas, self.variant, self.stream_k = num_ctas, variant, stream_k

    def _c(self) -> _Config:
        c = _Config()
        c.kernel = KERNELS[self.kernel]
        c.bm, c.bn, c.bk, c.stages = self.bm, self.bn, self.bk, self.stages
        c.split_k, c.raster_group = self.split_k, self.raster_group
        c.stage_a, c.stage_b, c.num_ctas = self.stage_a, self.stage_b, self.num_ctas
        c.variant, c.stream_k = self.variant, self.stream_k
        return c

    @staticmethod
    def _from(c: _Config) -> "Config":
        return Config(KERNEL_NAMES.get(c.kernel, str(c.kernel)), c.bm, c.bn, c.bk, c.stages,
                      c.split_k, c.raster_group, c.stage_a, c.stage_b, c.num_ctas, c.variant,
                      c.stream_k)

    def as_dict(self) -> dict:
        return dict(kernel=self.kernel, bm=self.bm, bn=self.bn, bk=self.bk, stages=self.stages,
                    split_k=self.split_k, raster_group=self.raster_group, stage_a=self.stage_a,
                    stage_b=self.stage_b, num_ctas=self.num_ctas, variant=self.variant,
                    stream_k=self.stream_k)

    def __repr__(self):
        return f"Config({self.as_dict()})"


class Plan:
    """Owns a gemm_plan_t; destroyed with the object (or explicitly)."""

    def __init__(self, handle: int, dtype: str, M: int, N: int, K: int, epilogue: Epilogue):
        self.handle = handle
        self.dtype, self.M, self.N, self.K, self.epilogue = dtype, M, N, K, epilogue

    def destroy(self):
        if self.handle:
            lib().gemm_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

    def run(self, A, B, C, bias=None, residual=None, alpha=1.0, stream=None):
        return gemm_run(self, A, B, C, bias, residual, alpha, stream)

    def info(self) -> dict:
        return gemm_plan_info(self)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def gemm_plan(dtype: str, M: int, N: int, K: int, lda: int, ldb: int, ldc: int,
              epilogue: Epilogue | None = None, config: Config | None = None) -> Plan:
    """gemm_plan / gemm_plan_with_config; raises GemmError on a non-OK status."""
    ep = epilogue or Epilogue()
    h = ctypes.c_void_p()
    ce = ep._c()
    if config is None:
        rc = lib().gemm_plan(DTYPES[dtype], M, N, K, lda, ldb, ldc, ctypes.byref(ce), ctypes.byref(h))
    else:
        cc = config._c()
        rc = lib().gemm_plan_with_config(DTYPES[dtype], M, N, K, lda, ldb, ldc, ctypes.byref(ce),
                                         ctypes.byref(cc), ctypes.byref(h))
    if rc != 0:
        raise GemmError(rc, "gemm_plan")
    return Plan(h.value, dtype, M, N, K, ep)


def gemm_run(plan: Plan, A, B, C, bias=None, residual=None, alpha: float = 1.0, stream=None) -> int:
    """Enqueue one GEMM on `stream` (default: torch's current stream); raises on error."""
    if stream is None:
        import torch
        stream = torch.cuda.current_stream().cuda_stream
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    rc = lib().gemm_run(plan.handle, _ptr(A), _ptr(B), _ptr(C), _ptr(bias), _ptr(residual),
                        float(alpha), stream)
    if rc != 0:
        raise GemmError(rc, "gemm_run")
    return rc


def gemm_plan_status(plan: Plan) -> int:
    """Synchronise and return the plan's sticky device status (0 or a negative code)."""
    return int(lib().gemm_plan_status(plan.handle))


def gemm_plan_info(plan: Plan) -> dict:
    info = _PlanInfo()
    rc = lib().gemm_plan_info(plan.handle, ctypes.byref(info))
    if rc != 0:
        raise GemmError(rc, "gemm_plan_info")
    return dict(config=Config._from(info.config), workspace_bytes=info.workspace_bytes,
                num_sms=info.num_sms, device=info.device, cache_hit=bool(info.cache_hit),
                kernels_per_run=info.kernels_per_run)


def gemm_select_config(dtype: str, M: int, N: int, K: int, lda: int, ldb: int, ldc: int,
                       epilogue: Epilogue | None = None, num_sms: int = 152) -> Config:
    """Host-only dispatcher query (no GPU needed)."""
    ep = (epilogue or Epilogue())._c()
    c = _Config()
    rc = lib().gemm_select_config(DTYPES[dtype], M, N, K, lda, ldb, ldc, ctypes.byref(ep), num_sms,
                                  ctypes.byref(c))
    if rc != 0:
        raise GemmError(rc, "gemm_select_config")
    return Config._from(c)


def gemm_cache_stats() -> tuple[int, int, int]:
    e, h, m = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    lib().gemm_cache_stats(ctypes.byref(e), ctypes.byref(h), ctypes.byref(m))
    return e.value, h.value, m.value


def gemm_cache_clear() -> None:
    lib().gemm_cache_clear()


def gemm_run_noalloc(dtype: str, M: int, N: int, K: int, A, lda: int, B, ldb: int, C, ldc: int,
                     epilogue: Epilogue | None = None, bias=None, residual=None,
                     alpha: float = 1.0, stream=None) -> int:
    """gemm_run_noalloc: one GEMM without any allocation (fixed in-library scratch).

    For callers that cannot allocate device memory where they run the GEMM;
    see include/gemm13.h for the scratch limit and the sharing rules.
    """
    if stream is None:
        import torch
        stream = torch.cuda.current_stream().cuda_stream
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    ce = (epilogue or Epilogue())._c()
    rc = lib().gemm_run_noalloc(DTYPES[dtype], M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc,
                                ctypes.byref(ce), _ptr(bias), _ptr(residual), float(alpha), stream)
    if rc != 0:
        raise GemmError(rc, "gemm_run_noalloc")
    return rc


_plans: dict = {}
_keep_lock = threading.Lock()


def _keep(plans: dict, key, make):
    """plans[key], made by the first call that wants it: two threads never make it twice, which would
    destroy one of the two while its kernel may still run."""
    with _keep_lock:
        pl = plans.get(key)
        if pl is None:
            pl = plans[key] = make()
    return pl


def matmul(A, B, *, b_layout="kn", alpha=1.0, bias=None, act="none", residual=None, beta=1.0,
           out_dtype="f32", out=None):
    """C = cast(act(alpha*A@B + bias) + beta*residual) for 2-D or 3-D (batched) CUDA tensors.

    Plans are created once per (shape, dtype, strides, epilogue) and kept; gemm_kept_status tells
    whether a kernel of one of them gave up on a wait.
    """
    import torch
    tdt = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
    dt = tdt[A.dtype]
    batched = A.dim() == 3
    M, K = A.shape[-2], A.shape[-1]
    N = B.shape[-1] if b_layout == "kn" else B.shape[-2]
    batch = A.shape[0] if batched else 1
    odt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[out_dtype]
    if out is None:
        out = torch.empty((batch, M, N) if batched else (M, N), dtype=odt, device=A.device)
    lda, ldb, ldc = A.stride(-2), B.stride(-2), out.stride(-2)
    ep = Epilogue(b_layout=b_layout, out_dtype=out_dtype, bias=bias is not None, act=act,
                  residual=residual is not None, beta=beta,
                  ldr=residual.stride(-2) if residual is not None else 0, batch=batch,
                  stride_a=A.stride(0) if batched else 0,
                  stride_b=B.stride(0) if (batched and B.dim() == 3) else 0,
                  stride_c=out.stride(0) if batched else 0,
                  stride_r=residual.stride(0) if (batched and residual is not None and residual.dim() == 3) else 0)
    key = (dt, M, N, K, lda, ldb, ldc, tuple(sorted(vars(ep).items())), A.device.index)
    pl = _plans.get(key)
    if pl is None:
        pl = _keep(_plans, key, lambda: gemm_plan(dt, M, N, K, lda, ldb, ldc, ep))
    gemm_run(pl, A, B, out, bias, residual, alpha)
    return out


# ------------------------------------------------------------------ 4-bit floats
class Fp4Tensor:
    """A matrix in microscaled 4-bit floats (layout: include/gemm13.h, "4-bit floats"); read-only.

    codes: uint8 [rows, row_bytes]; scales: uint8, flat; tensor_scale: None (1) or one FP32 value on
    the same device ("nvfp4" only).  Arrays that do not fit the sizes are refused here, once.
    """

    __slots__ = ("_codes", "_scales", "_rows", "_cols", "_format", "_g", "_index", "_both")

    def __init__(self, codes, scales, rows, cols, format, tensor_scale=None):
        self._index = _check_fp4(_t(), codes, scales, rows, cols, format, tensor_scale)
        self._codes, self._scales, self._rows, self._cols = codes, scales, rows, cols
        self._format, self._g, self._both = format, tensor_scale, None

    @property
    def codes(self):
        if self._codes is None:
            row = (self._cols + 31) // 32 * 16
            self._codes = self._both[: self._rows * row].view(self._rows, row)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            self._scales = self._both[self._rows * ((self._cols + 31) // 32 * 16):]
        return self._scales

    rows = property(lambda self: self._rows)
    cols = property(lambda self: self._cols)
    format = property(lambda self: self._format)
    tensor_scale = property(lambda self: self._g)

    def _ptrs(self):
        """Addresses of codes, scales and tensor scale."""
        g = self._g
        g = None if g is None else g.data_ptr()
        if self._both is not None:
            p = self._both.data_ptr()
            return p, p + self._rows * ((self._cols + 31) // 32 * 16), g
        return self._codes.data_ptr(), self._scales.data_ptr(), g


def _refuse(what: str, why: str):
    e = GemmError(-1, what)
    e.args = (f"{what}: {why}",)
    raise e


class _Torch:
    """torch, its dtypes by name and its current device and stream, looked up once (a call of a few
    microseconds on the GPU waits for every attribute lookup on the host)."""

    torch = None

    def __init__(self):
        import torch
        self.torch = torch
        self.name = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
        self.dtype = {v: k for k, v in self.name.items()}
        self.u8, self.f32, self.i32 = torch.uint8, torch.float32, torch.int32
        self.empty = torch.empty
        self._devices: dict = {}
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.raw_stream = raw or (lambda i: torch.cuda.current_stream(i).cuda_stream)
        self.device_index = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device

    def on(self, stream, index: int):
        """Context in which `stream` (a torch stream or a handle) is the current one: what a call allocates then
        belongs to the stream that uses it."""
        cuda = self.torch.cuda
        if isinstance(stream, int):
            # 0 and 1 (cudaStreamLegacy) are the default stream; ExternalStream(0) would be a new one of torch's pool
            stream = cuda.ExternalStream(stream, device=index) if stream > 1 else cuda.default_stream(index)
        elif stream.device.index != index:
            _refuse("stream", "it belongs to another device than the tensors")
        return cuda.stream(stream)

    def device(self, index: int):
        d = self._devices.get(index)
        if d is None:
            d = self._devices[index] = self.torch.device("cuda", index)
        return d


_torch_cache: list = []


def _t() -> _Torch:
    if not _torch_cache:
        _torch_cache.append(_Torch())
    return _torch_cache[0]


def _stream(t: _Torch, index: int, stream) -> int:
    if stream is None:
        return t.raw_stream(index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _no_capture(t: _Torch, what: str):
    """A plan allocates, which would break a graph capture."""
    if t.torch.cuda.is_current_stream_capturing():
        _refuse(what, "no plan for this shape yet: call it once before capturing a graph")


def _on_device(what: str, index: int, *tensors):
    """Refuses tensors that the kernels of the current device cannot read (None, addresses and objects that only
    have one pass)."""
    for x in tensors:
        device = getattr(x, "get_device", None)
        if device is not None and device() != index:
            _refuse(what, "tensors on the current device are wanted")


def _rows_ok(x) -> bool:
    """Row-major, rows not overlapping: what a C entry point takes as [rows][ld]."""
    rows, cols = x.shape
    return (cols <= 1 or x.stride(1) == 1) and (rows <= 1 or x.stride(0) >= cols)


def _ld(x) -> int:
    rows, cols = x.shape
    return x.stride(0) if rows > 1 else max(cols, 1)


def _check_scale(t: _Torch, what: str, g, format: str, index: int):
    if format != "nvfp4":
        _refuse(what, "only nvfp4 has a scale of the whole tensor")
    if g.dtype is not t.f32 or g.numel() != 1 or g.get_device() != index:
        _refuse(what, "tensor_scale: one FP32 value on the matrix's device is wanted")


def _check_fp4(t: _Torch, codes, scales, rows: int, cols: int, format: str, g) -> int:
    """Refuses arrays that are shorter than the kernels read; returns their device's index."""
    what = "Fp4Tensor"
    if format not in FP4_FORMATS:
        _refuse(what, f"unknown format {format!r}")
    per = 128 if format == "mxfp4" else 64  # elements of four blocks
    n_codes = rows * ((cols + 31) // 32 * 16)
    n_scales = (rows + 127) // 128 * ((cols + per - 1) // per) * 512
    index, u8 = codes.get_device(), t.u8
    if (index < 0 or scales.get_device() != index or codes.dtype is not u8 or scales.dtype is not u8 or rows < 0
            or cols < 0 or codes.numel() != n_codes or scales.numel() != n_scales or not codes.is_contiguous()
            or not scales.is_contiguous()):
        _refuse(what, f"{rows} x {cols} in {format}: codes ({n_codes} bytes) and scales ({n_scales} bytes), contiguous "
                      "uint8 on the GPU, are wanted")
    if g is not None:
        _check_scale(t, what, g, format, index)
    return index


def fp4_quantize(x, format: str = "nvfp4", tensor_scale=None, stream=None) -> Fp4Tensor:
    """A 2-D CUDA tensor (FP32, FP16 or BF16, any row stride) in 4-bit floats (gemm_fp4_quantize).

    tensor_scale ("nvfp4"): a positive FP32 CUDA tensor of one value; max|x| / (6 * 448) uses the
    whole range.  None means 1.
    """
    what, t = "fp4_quantize", _t()
    f = FP4_FORMATS.get(format)
    if f is None:
        _refuse(what, f"unknown format {format!r}")
    dt, index = t.name.get(x.dtype), x.get_device()
    if dt is None or x.dim() != 2 or index < 0:
        _refuse(what, "a 2-D CUDA tensor in f32, f16 or bf16 is wanted")
    if stream is not None:
        with t.on(stream, index):
            return fp4_quantize(x, format, tensor_scale)
    if index != t.device_index():
        with t.torch.cuda.device(index):
            return fp4_quantize(x, format, tensor_scale)
    if tensor_scale is not None:
        _check_scale(t, what, tensor_scale, format, index)
    rows, cols = x.shape
    ld, step = x.stride()
    if (cols > 1 and step != 1) or (rows > 1 and ld < cols):
        x = x.contiguous()
        ld = cols
    if rows <= 1 or ld < 1:
        ld = max(cols, 1)
    # codes and scales in one allocation (codes are a multiple of 16 bytes)
    per = 128 if f == 0 else 64  # elements of four blocks
    n_codes = rows * ((cols + 31) // 32 * 16)
    both = t.empty(n_codes + (rows + 127) // 128 * ((cols + per - 1) // per) * 512, dtype=t.u8, device=x.device)
    p = both.data_ptr()
    rc = (_lib or load()).gemm_fp4_quantize(f, DTYPES[dt], rows, cols, x.data_ptr(), ld, _ptr(tensor_scale), p,
                                            p + n_codes, t.raw_stream(index))
    if rc != 0:
        raise GemmError(rc, what)
    q = Fp4Tensor.__new__(Fp4Tensor)
    q._codes = q._scales = None
    q._rows, q._cols, q._format, q._g, q._index, q._both = rows, cols, format, tensor_scale, index, both
    return q


def fp4_dequantize(q: Fp4Tensor, dtype: str = "f32", out=None, stream=None):
    """The values of a 4-bit matrix as a tensor of `dtype` (gemm_fp4_dequantize)."""
    what, t = "fp4_dequantize", _t()
    code = DTYPES.get(dtype)
    if code is None:
        _refuse(what, f"unknown dtype {dtype!r}")
    index, rows, cols = q._index, q._rows, q._cols
    if q._format not in FP4_FORMATS:
        _refuse(what, "an Fp4Tensor is wanted")
    if stream is not None:
        with t.on(stream, index):
            return fp4_dequantize(q, dtype, out)
    if index != t.device_index():
        with t.torch.cuda.device(index):
            return fp4_dequantize(q, dtype, out)
    if out is None:
        out, ld = t.empty((rows, cols), dtype=t.dtype[dtype], device=t.device(index)), cols or 1
    else:
        if (tuple(out.shape) != (rows, cols) or t.name.get(out.dtype) != dtype or out.get_device() != index
                or not _rows_ok(out)):
            _refuse(what, "out: a row-major tensor of the matrix's shape, dtype and device is wanted")
        ld = _ld(out)
    codes, scales, g = q._ptrs()
    rc = (_lib or load()).gemm_fp4_dequantize(FP4_FORMATS[q._format], code, rows, cols, codes, scales, g,
                                              out.data_ptr(), ld, t.raw_stream(index))
    if rc != 0:
        raise GemmError(rc, what)
    return out


class Fp4Plan:
    """Owns a gemm_fp4_plan_t; destroyed with the object (or explicitly)."""

    def __init__(self, handle: int, format: str, M: int, N: int, K: int, epilogue: Epilogue):
        self.handle = handle
        self.format, self.M, self.N, self.K, self.epilogue = format, M, N, K, epilogue

    def destroy(self):
        if self.handle:
            lib().gemm_fp4_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def gemm_fp4_plan(format: str, M: int, N: int, K: int, ldc: int, epilogue: Epilogue | None = None) -> Fp4Plan:
    """gemm_fp4_plan; the epilogue's b_layout must be "nk".  Raises GemmError on a non-OK status."""
    ep = epilogue or Epilogue(b_layout="nk")
    h, ce = ctypes.c_void_p(), ep._c()
    rc = lib().gemm_fp4_plan(FP4_FORMATS[format], M, N, K, ldc, ctypes.byref(ce), ctypes.byref(h))
    if rc != 0:
        raise GemmError(rc, "gemm_fp4_plan")
    return Fp4Plan(h.value, format, M, N, K, ep)


def gemm_fp4_run(plan: Fp4Plan, A: Fp4Tensor, B: Fp4Tensor, C, bias=None, residual=None, alpha: float = 1.0,
                 stream=None) -> int:
    """Enqueue C = epilogue(A @ B.T) of a plan on `stream` (default: torch's current stream)."""
    if (A._rows, A._cols, B._rows, B._cols) != (plan.M, plan.K, plan.N, plan.K) or A._format != plan.format \
            or B._format != plan.format:
        _refuse("gemm_fp4_run", "the operands do not fit the plan")
    t = _t()
    index = t.device_index()
    if A._index != index or B._index != index:
        _refuse("gemm_fp4_run", "the operands are not on the current device")
    _on_device("gemm_fp4_run", index, C, bias, residual)
    rc = (_lib or load()).gemm_fp4_run(plan.handle, *A._ptrs(), *B._ptrs(), _ptr(C), _ptr(bias), _ptr(residual), alpha,
                                       _stream(t, index, stream))
    if rc != 0:
        raise GemmError(rc, "gemm_fp4_run")
    return rc


def gemm_fp4_status(plan: Fp4Plan) -> int:
    """Synchronise and return the plan's sticky device status (0 or a negative code)."""
    return int(lib().gemm_fp4_status(plan.handle))


def gemm_fp4_select_config(M: int, N: int, K: int, num_sms: int = 152) -> Config:
    """Host-only query of the 4-bit product's tile (no GPU needed)."""
    c = _Config()
    rc = lib().gemm_fp4_select_config(M, N, K, num_sms, ctypes.byref(c))
    if rc != 0:
        raise GemmError(rc, "gemm_fp4_select_config")
    return Config._from(c)


_fp4_plans: dict = {}


def fp4_matmul(A: Fp4Tensor, B: Fp4Tensor, *, alpha=1.0, bias=None, act="none", residual=None, beta=1.0,
               out_dtype="f32", out=None, stream=None):
    """C = cast(act(alpha * A @ B.T + bias) + beta * residual) of two 4-bit matrices.

    A [M, K] (activations), B [N, K] (a weight as it lies for x @ W.T), both in the same format.
    bias: FP32 [N]; residual: FP32 [M, N]; out overlaps none of the inputs.  Plans are created once per (shape, format, strides,
    epilogue, device) and kept; they hold no workspace, so calls may overlap on any streams.  (The
    first call of a shape makes its plan, and is refused while a graph is being captured.)  With
    `stream`, the call runs, and allocates, as if that were the current stream.  gemm_kept_status tells
    whether a kernel gave up on a wait: what it returned is then undefined.
    """
    what, t = "fp4_matmul", _t()
    index, format, M, K, N = A._index, A._format, A._rows, A._cols, B._rows
    if B._index != index or B._format != format or B._cols != K:
        _refuse(what, "A and B need the same format, K and device")
    if stream is not None or index != t.device_index():
        with t.on(stream, index) if stream is not None else t.torch.cuda.device(index):
            return fp4_matmul(A, B, alpha=alpha, bias=bias, act=act, residual=residual, beta=beta,
                              out_dtype=out_dtype, out=out)
    if out_dtype not in DTYPES or act not in ("none", "gelu", "relu"):
        _refuse(what, "out_dtype: f32, f16 or bf16; act: none, gelu or relu")
    if bias is not None and (bias.dtype is not t.f32 or tuple(bias.shape) != (N,) or bias.get_device() != index
                             or not bias.is_contiguous()):
        _refuse(what, "bias: contiguous FP32 [N] on the operands' device is wanted")
    if residual is not None and (tuple(residual.shape) != (M, N) or residual.dtype is not t.f32
                                 or residual.get_device() != index or not _rows_ok(residual)):
        _refuse(what, "residual: a row-major f32 [M, N] on the operands' device is wanted")
    if out is None:
        out, ldc = t.empty((M, N), dtype=t.dtype[out_dtype], device=t.device(index)), N or 1
    else:
        if tuple(out.shape) != (M, N) or t.name.get(out.dtype) != out_dtype or out.get_device() != index \
                or not _rows_ok(out):
            _refuse(what, f"out: a row-major {out_dtype} [M, N] on the operands' device is wanted")
        ldc = _ld(out)
    ldr = 0 if residual is None else _ld(residual)
    key = (format, M, N, K, ldc, ldr, out_dtype, bias is not None, act, beta, index)
    pl = _fp4_plans.get(key)
    if pl is None:
        if format not in FP4_FORMATS:
            _refuse(what, "Fp4Tensors are wanted")
        _no_capture(t, what)
        ep = Epilogue(b_layout="nk", out_dtype=out_dtype, bias=bias is not None, act=act,
                      residual=residual is not None, beta=beta, ldr=ldr)
        pl = _keep(_fp4_plans, key, lambda: gemm_fp4_plan(format, M, N, K, ldc, ep))
    rc = (_lib or load()).gemm_fp4_run(pl.handle, *A._ptrs(), *B._ptrs(), out.data_ptr(), _ptr(bias), _ptr(residual),
                                       alpha, t.raw_stream(index))
    if rc != 0:
        raise GemmError(rc, what)
    return out


# ------------------------------------------------------------------ mixture of experts
class MoePlan:
    """Owns a gemm_moe_plan_t; destroyed with the object (or explicitly)."""

    def __init__(self, handle: int, workspace_bytes: int):
        self.handle, self.workspace_bytes = handle, workspace_bytes

    def destroy(self):
        if self.handle:
            lib().gemm_moe_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def gemm_moe_plan(dtype: str, T: int, E: int, top_k: int, H: int, I: int, act: str = "swiglu",
                  normalize: bool = True, **fields) -> MoePlan:
    """gemm_moe_plan; `fields`: the other members of gemm_moe_desc_t.  Raises GemmError on a non-OK status."""
    d, h = _MoeDesc(), ctypes.c_void_p()
    lib().gemm_moe_desc_init(ctypes.byref(d))
    d.dtype, d.T, d.E, d.top_k, d.H, d.I = DTYPES[dtype], T, E, top_k, H, I
    d.act, d.normalize = MOE_ACTS[act], int(bool(normalize))
    for k, v in fields.items():
        setattr(d, k, int(v))
    rc = lib().gemm_moe_plan(ctypes.byref(d), ctypes.byref(h))
    if rc != 0:
        raise GemmError(rc, "gemm_moe_plan")
    return MoePlan(h.value, lib().gemm_moe_workspace_bytes(h))


def gemm_moe_run(plan: MoePlan, X, router, W1, W2, Y, workspace, expert_ids=None, expert_weights=None,
                 stream=None) -> int:
    """Enqueue one layer on `stream` (default: torch's current stream); raises on error."""
    t = _t()
    index = t.device_index()
    _on_device("gemm_moe_run", index, X, router, W1, W2, Y, workspace, expert_ids, expert_weights)
    if hasattr(workspace, "numel") and workspace.numel() * workspace.element_size() < plan.workspace_bytes:
        _refuse("gemm_moe_run", f"workspace: {plan.workspace_bytes} bytes are wanted")
    rc = lib().gemm_moe_run(plan.handle, _ptr(X), _ptr(router), _ptr(W1), _ptr(W2), _ptr(Y), _ptr(expert_ids),
                            _ptr(expert_weights), _ptr(workspace), _stream(t, index, stream))
    if rc != 0:
        raise GemmError(rc, "gemm_moe_run")
    return rc


def gemm_moe_status(plan: MoePlan) -> int:
    """Synchronise and return the plan's sticky device status (0 or a negative code)."""
    return int(lib().gemm_moe_status(plan.handle))


_moe_plans: dict = {}


def moe_layer(x, router, w1, w2, top_k: int, *, act: str = "swiglu", normalize: bool = True, out=None,
              return_routing: bool = False, stream=None):
    """A mixture-of-experts layer for 1 to 64 tokens (include/gemm13.h, gemm_moe_run).

    x [T, H], router [E, H], w1 [E, I, H] ("gelu", "relu") or [E, 2I, H] ("swiglu": gate rows, then up
    rows), w2 [E, H, I], all FP16 or all BF16, rows contiguous.  Returns y [T, H], or with
    return_routing (y, expert ids int32 [T, top_k], their weights FP32 [T, top_k]).  Plans are kept per
    shape, strides and device (the first call makes its plan, and is refused while a graph is being
    captured); every call has a workspace of its own from torch's allocator.  out overlaps no input.  With
    `stream`, the call runs, and allocates, as if that were the current stream.  gemm_kept_status tells
    whether a kernel gave up on a wait: what it returned is then undefined.
    """
    what, t = "moe_layer", _t()
    dt = t.name.get(x.dtype)
    if dt not in ("f16", "bf16") or act not in MOE_ACTS:
        _refuse(what, "FP16 or BF16 tensors and act gelu, relu or swiglu are wanted")
    if x.dim() != 2 or router.dim() != 2 or w1.dim() != 3 or w2.dim() != 3:
        _refuse(what, "x [T, H], router [E, H], w1 [E, I or 2I, H], w2 [E, H, I] are wanted")
    (T, H), (E, Hr), (E1, rows, H1), (E2, H2, I), dtype = x.shape, router.shape, w1.shape, w2.shape, x.dtype
    if not (Hr == H1 == H2 == H and E1 == E2 == E and rows == (2 * I if act == "swiglu" else I)):
        _refuse(what, "the shapes of x, router, w1 and w2 do not fit one another")
    if out is not None and tuple(out.shape) != (T, H):
        _refuse(what, "out: [T, H] is wanted")
    index = x.get_device()
    if index < 0 or router.get_device() != index or w1.get_device() != index or w2.get_device() != index \
            or router.dtype is not dtype or w1.dtype is not dtype or w2.dtype is not dtype \
            or (out is not None and (out.get_device() != index or out.dtype is not dtype)):
        _refuse(what, "tensors of x's dtype on x's device, a GPU, are wanted")
    if stream is not None or index != t.device_index():
        with t.on(stream, index) if stream is not None else t.torch.cuda.device(index):
            return moe_layer(x, router, w1, w2, top_k, act=act, normalize=normalize, out=out,
                             return_routing=return_routing)
    dev = x.device
    if out is None:
        out = t.empty((T, H), dtype=dtype, device=dev)
    (ldx, cx), (ldr, cr), (ldy, cy) = x.stride(), router.stride(), out.stride()
    (st1, ld1, c1), (st2, ld2, c2) = w1.stride(), w2.stride()
    if (H > 1 and not cx == cr == cy == c1 == 1) or (I > 1 and c2 != 1) or (T > 1 and (ldx < H or ldy < H)) \
            or (E > 1 and (ldr < H or st1 == 0 or st2 == 0)) or (rows > 1 and ld1 < H) or (H > 1 and ld2 < I):
        _refuse(what, "rows that are contiguous and not shared are wanted")
    # strides that no element uses may be anything
    if T <= 1:
        ldx = ldy = H
    if rows <= 1:
        ld1 = H
    if H <= 1:
        ld2 = I
    if E <= 1:
        ldr, st1, st2 = H, rows * ld1, H * ld2
    key = (dt, T, E, top_k, H, I, act, normalize, ldx, ldr, ld1, st1, ld2, st2, ldy, index)
    pl = _moe_plans.get(key)
    if pl is None:
        _no_capture(t, what)
        pl = _keep(_moe_plans, key, lambda: gemm_moe_plan(
            dt, T, E, top_k, H, I, act, normalize, ldx=ldx, ld_router=ldr, ld_w1=ld1, stride_w1=st1, ld_w2=ld2,
            stride_w2=st2, ldy=ldy))
    ids = wts = None
    if return_routing:
        ids = t.empty((T, top_k), dtype=t.i32, device=dev)
        wts = t.empty((T, top_k), dtype=t.f32, device=dev)
    ws = t.empty(pl.workspace_bytes, dtype=t.u8, device=dev)
    rc = (_lib or load()).gemm_moe_run(pl.handle, x.data_ptr(), router.data_ptr(), w1.data_ptr(), w2.data_ptr(), out.data_ptr(),
                            _ptr(ids), _ptr(wts), ws.data_ptr(), t.raw_stream(index))
    if rc != 0:
        raise GemmError(rc, what)
    return (out, ids, wts) if return_routing else out


def gemm_kept_status() -> int:
    """Synchronise and return the sticky device status of the plans that matmul, fp4_matmul, fp8_matmul and
    moe_layer keep.

    0, or the code of one whose kernel gave up on a wait (-5): what the calls of its shape have returned
    is not to be used.
    """
    for plans, status in ((_plans, gemm_plan_status), (_fp4_plans, gemm_fp4_status), (_moe_plans, gemm_moe_status),
                          (blocks._fp8_plans, gemm_fp8_status)):
        for key, plan in list(plans.items()):
            with _t().torch.cuda.device(key[-1]):
                rc = status(plan)
            if rc != 0:
                return rc
    return 0


from . import blocks  # noqa: E402  (it builds on what stands above)
from .blocks import *  # noqa: E402,F401,F403

__all__ += blocks.__all__
