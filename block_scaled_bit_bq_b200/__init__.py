"""Block-scaled tensor quantization on NVIDIA B200 (sm_100a).

A thin ctypes binding of libbq.so (C ABI in include/bq.h). The functions named
``bq_*`` marshal torch tensors (device memory) and the current CUDA stream into the
C entry points of the same names; every step of the computation runs in the CUDA
kernels. ``quantize`` / ``dequantize`` / ``qsnr`` add output allocation on top.

The library must be built (``python -m block_scaled_bit_bq_b200.build``); importing
this package without libbq.so raises, and there is no CPU fallback.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbq.so")

# enums of include/bq.h
DT = {"bf16": 0, "fp16": 1, "fp32": 2, "ue8m0": 3, "e4m3": 4}
FORMATS = {"int8_sym": 0, "int8_asym": 1, "int4_sym": 2, "uint4_asym": 3, "e4m3": 4, "e5m2": 5, "e2m1": 6,
           "e2m3": 7, "e3m2": 8}
GRANULARITIES = {"tensor": 0, "row": 1, "group": 2, "mx": 3, "nv": 4, "tile2d": 5}
ACTS = {"silu": 0, "gelu": 1}          # gated activations ("gelu": its tanh form)
LAYOUTS = {"rows": 0, "gemm": 1}       # MX / NV block scales: row-major, or a block-scaled GEMM's tiles
FOUR_BIT = {"int4_sym", "uint4_asym", "e2m1"}
ASYMMETRIC = {"int8_asym", "uint4_asym"}

STATUS = {0: "BQ_OK", 1: "BQ_ERR_INVALID_ARG", 2: "BQ_ERR_UNSUPPORTED", 3: "BQ_ERR_SHAPE",
          4: "BQ_ERR_ALIGNMENT", 5: "BQ_ERR_WORKSPACE", 6: "BQ_ERR_CUDA"}


class BqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_lib().bq_status_string(status).decode()}")


class BqScheme(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("granularity", ctypes.c_int32), ("block", ctypes.c_int32),
                ("scale_dtype", ctypes.c_int32), ("hadamard", ctypes.c_int32), ("scale_layout", ctypes.c_int32)]


class BqRowTransform(ctypes.Structure):
    _fields_ = [("col_scale", ctypes.c_void_p), ("sign_bits", ctypes.c_void_p), ("reserved", ctypes.c_int64)]


class BqStats(ctypes.Structure):
    _fields_ = [("err2", ctypes.c_double), ("x2", ctypes.c_double), ("kappa_sum", ctypes.c_double),
                ("kappa_max", ctypes.c_double), ("n_units", ctypes.c_double)]


_L = None


def _lib() -> ctypes.CDLL:
    global _L
    if _L is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m block_scaled_bit_bq_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        sp = ctypes.POINTER(BqScheme)
        L.bq_status_string.restype = ctypes.c_char_p
        L.bq_status_string.argtypes = [ctypes.c_int]
        L.bq_version.restype = ctypes.c_char_p
        L.bq_version.argtypes = []
        L.bq_buffer_sizes.restype = ctypes.c_int
        L.bq_buffer_sizes.argtypes = [sp, i64, i64, ctypes.POINTER(sz), ctypes.POINTER(sz),
                                      ctypes.POINTER(sz), ctypes.POINTER(sz)]
        L.bq_workspace_size.restype = ctypes.c_int
        L.bq_workspace_size.argtypes = [sp, i64, i64, ctypes.c_int, ctypes.POINTER(sz)]
        L.bq_quantize.restype = ctypes.c_int
        L.bq_quantize.argtypes = [vp, i32, i64, i64, sp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.bq_dequantize.restype = ctypes.c_int
        L.bq_dequantize.argtypes = [vp, vp, vp, vp, i64, i64, sp, vp, i32, vp]
        L.bq_qsnr.restype = ctypes.c_int
        L.bq_qsnr.argtypes = [vp, i32, vp, vp, vp, vp, i64, i64, sp, vp, vp, sz, vp]
        L.bq_quantize_noalloc.restype = ctypes.c_int
        L.bq_quantize_noalloc.argtypes = [vp, i32, i64, i64, sp, vp, vp, vp, vp, vp, vp]
        L.bq_stats_qsnr_db.restype = ctypes.c_double
        L.bq_stats_qsnr_db.argtypes = [ctypes.POINTER(BqStats)]
        L.bq_stats_to_db.restype = ctypes.c_double
        L.bq_stats_to_db.argtypes = [ctypes.POINTER(BqStats)]
        L.bq_tensor_range.restype = ctypes.c_int
        L.bq_tensor_range.argtypes = [vp, i32, i64, i64, sp, vp, vp, sz, vp]
        L.bq_quantize_with_range.restype = ctypes.c_int
        L.bq_quantize_with_range.argtypes = [vp, i32, i64, i64, sp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.bq_quantize_batch.restype = ctypes.c_int
        L.bq_quantize_batch.argtypes = [vp, i32, i64, i64, i64, sp, vp, vp, vp, vp, vp, sz, vp]
        L.bq_gemm.restype = ctypes.c_int
        L.bq_gemm.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, sp, vp, i32, vp]
        for f in (L.bq_linear, L.bq_linear_grad_input):
            f.restype = ctypes.c_int
            f.argtypes = [vp, i32, i64, vp, vp, vp, i64, i64, i64, sp, vp, i32, vp]
        L.bq_linear_grad_weight.restype = ctypes.c_int
        L.bq_linear_grad_weight.argtypes = [vp, i32, i64, vp, vp, i64, i64, i64, sp, vp, i32, vp]
        L.bq_glu.restype = ctypes.c_int
        L.bq_glu.argtypes = [vp, i64, vp, i64, i32, i64, i64, i32, vp, sp, vp, vp, vp, vp, vp]
        L.bq_glu_backward.restype = ctypes.c_int
        L.bq_glu_backward.argtypes = [vp, i64, i32, vp, vp, vp, vp, sp, i64, i64, i32, vp, i64, vp, i64, vp]
        L.bq_debug_skip_tile_copy.restype = ctypes.c_int
        L.bq_debug_skip_tile_copy.argtypes = [i32]
        L.bq_debug_skip_linear_copy.restype = ctypes.c_int
        L.bq_debug_skip_linear_copy.argtypes = [i32]
        L.bq_wait_timeouts.restype = ctypes.c_int
        L.bq_wait_timeouts.argtypes = [ctypes.POINTER(ctypes.c_uint32), i32]
        rtp = ctypes.POINTER(BqRowTransform)
        L.bq_quantize_rt.restype = ctypes.c_int
        L.bq_quantize_rt.argtypes = [vp, i32, i64, i64, sp, rtp, vp, vp, vp, vp, vp, sz, vp]
        L.bq_dequantize_rt.restype = ctypes.c_int
        L.bq_dequantize_rt.argtypes = [vp, vp, vp, i64, i64, sp, rtp, vp, i32, vp]
        _L = L
    return _L


def lib() -> ctypes.CDLL:
    """The loaded libbq.so (raises ImportError when it has not been built)."""
    return _lib()


@dataclass(frozen=True)
class Scheme:
    """A quantization scheme: element format, scaling granularity, group size, scale
    dtype, the Hadamard flag and the layout of MX / NV block scales ("rows", or "gemm":
    the tiles a block-scaled GEMM reads). block / scale_dtype default to the
    granularity's own (32 / ue8m0 for mx, 16 / e4m3 for nv, 128 / fp32 for tile2d
    (128 x 128 tiles), fp32 otherwise)."""
    fmt: str
    gran: str
    block: int = 0
    scale_dtype: str | None = None
    hadamard: bool = False
    layout: str = "rows"

    def resolved(self) -> "Scheme":
        sd = self.scale_dtype or {"mx": "ue8m0", "nv": "e4m3"}.get(self.gran, "fp32")
        blk = self.block or {"mx": 32, "nv": 16, "tile2d": 128}.get(self.gran, 0)
        return Scheme(self.fmt, self.gran, blk, sd, bool(self.hadamard), self.layout)

    def __getstate__(self):
        """The fields alone: what calls keep on the scheme (see _c_scheme) is not saved with it."""
        return {n: getattr(self, n) for n in self.__dataclass_fields__}

    def c(self) -> BqScheme:
        s = self.resolved()
        return BqScheme(FORMATS[s.fmt], GRANULARITIES[s.gran], s.block, DT[s.scale_dtype], int(s.hadamard),
                        LAYOUTS[s.layout])


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status: int, where: str):
    if status != 0:
        raise BqError(status, where)


# ---------------------------------------------------------------------------
# C entry points (same names), tensor marshalling only
# ---------------------------------------------------------------------------

def bq_version() -> str:
    return _lib().bq_version().decode()


def bq_status_string(status: int) -> str:
    return _lib().bq_status_string(status).decode()


def bq_buffer_sizes(scheme: Scheme, rows: int, cols: int):
    """(code_bytes, scale_bytes, zero_point_bytes, tensor_scale_bytes)."""
    out = [ctypes.c_size_t(0) for _ in range(4)]
    sc = scheme.c()
    _check(_lib().bq_buffer_sizes(ctypes.byref(sc), rows, cols, *[ctypes.byref(o) for o in out]),
           "bq_buffer_sizes")
    return tuple(int(o.value) for o in out)


def bq_workspace_size(scheme: Scheme, rows: int, cols: int, with_stats: bool) -> int:
    out = ctypes.c_size_t(0)
    sc = scheme.c()
    _check(_lib().bq_workspace_size(ctypes.byref(sc), rows, cols, int(with_stats), ctypes.byref(out)),
           "bq_workspace_size")
    return int(out.value)


def bq_quantize(x: torch.Tensor, scheme: Scheme, codes: torch.Tensor, scales: torch.Tensor,
                zero_points: torch.Tensor | None, tensor_scale: torch.Tensor | None,
                stats: torch.Tensor | None, workspace: torch.Tensor | None, stream=None,
                rows: int | None = None, cols: int | None = None) -> None:
    """x: bf16 [rows, cols] on the device; outputs are preallocated device tensors."""
    if rows is None:
        rows, cols = x.shape
    sc = scheme.c()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib().bq_quantize(_ptr(x), DT["bf16"], rows, cols, ctypes.byref(sc), _ptr(codes), _ptr(scales),
                              _ptr(zero_points), _ptr(tensor_scale), _ptr(stats), _ptr(workspace), ws_bytes,
                              _stream(stream)), "bq_quantize")


def bq_quantize_noalloc(x: torch.Tensor, scheme: Scheme, codes: torch.Tensor, scales: torch.Tensor,
                        zero_points: torch.Tensor | None, tensor_scale: torch.Tensor | None,
                        stats: torch.Tensor | None, stream=None) -> None:
    """bq_quantize with the library's own static device scratch instead of a workspace
    (for callers that cannot allocate device memory; calls must not overlap)."""
    rows, cols = x.shape
    sc = scheme.c()
    _check(_lib().bq_quantize_noalloc(_ptr(x), DT["bf16"], rows, cols, ctypes.byref(sc), _ptr(codes), _ptr(scales),
                                      _ptr(zero_points), _ptr(tensor_scale), _ptr(stats), _stream(stream)),
           "bq_quantize_noalloc")


def bq_tensor_range(x: torch.Tensor, scheme: Scheme, range_out: torch.Tensor, workspace: torch.Tensor,
                    stream=None) -> None:
    """The range pass of a per-tensor / NV scheme alone: range_out (fp32 [3] on the
    device) = {amax, min(min, 0), max(max, 0)} of the (rotated) tensor."""
    rows, cols = x.shape
    sc = scheme.c()
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(_lib().bq_tensor_range(_ptr(x), DT["bf16"], rows, cols, ctypes.byref(sc), _ptr(range_out),
                                  _ptr(workspace), ws_bytes, _stream(stream)), "bq_tensor_range")


def bq_quantize_with_range(x: torch.Tensor, scheme: Scheme, range_in: torch.Tensor, codes: torch.Tensor,
                           scales: torch.Tensor, zero_points: torch.Tensor | None,
                           tensor_scale: torch.Tensor | None, stats: torch.Tensor | None,
                           workspace: torch.Tensor | None, stream=None) -> None:
    """The quantize pass of a per-tensor / NV scheme against a given range (fp32 [3] on
    the device: amax, min, max)."""
    rows, cols = x.shape
    sc = scheme.c()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib().bq_quantize_with_range(_ptr(x), DT["bf16"], rows, cols, ctypes.byref(sc), _ptr(range_in),
                                         _ptr(codes), _ptr(scales), _ptr(zero_points), _ptr(tensor_scale),
                                         _ptr(stats), _ptr(workspace), ws_bytes, _stream(stream)),
           "bq_quantize_with_range")


def bq_quantize_batch(x: torch.Tensor, scheme: Scheme, codes: torch.Tensor, scales: torch.Tensor,
                      zero_points: torch.Tensor | None, stats: torch.Tensor | None,
                      workspace: torch.Tensor | None, stream=None) -> None:
    """x: bf16 [batch, rows, cols] on the device; outputs preallocated (see alloc_batch_outputs);
    stats: float64 [batch, 5] or None."""
    batch, rows, cols = x.shape
    sc = scheme.c()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib().bq_quantize_batch(_ptr(x), DT["bf16"], batch, rows, cols, ctypes.byref(sc), _ptr(codes),
                                    _ptr(scales), _ptr(zero_points), _ptr(stats), _ptr(workspace), ws_bytes,
                                    _stream(stream)), "bq_quantize_batch")


def bq_gemm(a: "Quantized", b: "Quantized", d: torch.Tensor, stream=None) -> None:
    """D[m, n] = A[m, k] B[n, k]^T on the tensor cores from two quantized operands (same
    MXFP8 or NVFP4 scheme, GEMM-layout scales); d: fp32 or bf16 [m, n] on the device."""
    if a.scheme != b.scheme or a.cols != b.cols:
        raise ValueError("operands need the same scheme and the same k")
    m, n, k = a.rows, b.rows, a.cols
    d_dt = {torch.bfloat16: DT["bf16"], torch.float32: DT["fp32"]}[d.dtype]
    sc = a.scheme.c()
    _check(_lib().bq_gemm(_ptr(a.codes), _ptr(a.scales), _ptr(a.tensor_scale), _ptr(b.codes), _ptr(b.scales),
                          _ptr(b.tensor_scale), m, n, k, ctypes.byref(sc), _ptr(d), d_dt, _stream(stream)), "bq_gemm")


def gemm(a: "Quantized", b: "Quantized", dtype=torch.float32, stream=None) -> torch.Tensor:
    """A B^T of two quantized operands (MXFP8 / NVFP4, GEMM-layout scales)."""
    for q in (a, b):
        _buffers(q, a.codes.device, q.rows, q.cols)
    d = torch.empty((a.rows, b.rows), dtype=dtype, device=a.codes.device)
    bq_gemm(a, b, d, stream)
    return d


def bq_debug_skip_tile_copy(warp: int) -> None:
    """Test hook: in the next flat quantize launch, warp `warp` issues no copy for its first
    staged tile, so its wait runs out (bounded) and bq_wait_timeouts counts it."""
    _check(_lib().bq_debug_skip_tile_copy(int(warp)), "bq_debug_skip_tile_copy")


def bq_debug_skip_linear_copy(cta: int) -> None:
    """Test hook: in the next product of the linear layer on the tensor cores, CTA `cta` issues no
    copies for its first stage, so that its waits run out (bounded) and bq_wait_timeouts counts
    them."""
    _check(_lib().bq_debug_skip_linear_copy(int(cta)), "bq_debug_skip_linear_copy")


def bq_dequantize(codes: torch.Tensor, scales: torch.Tensor, zero_points: torch.Tensor | None,
                  tensor_scale: torch.Tensor | None, rows: int, cols: int, scheme: Scheme,
                  out: torch.Tensor, stream=None) -> None:
    out_dt = {torch.bfloat16: DT["bf16"], torch.float32: DT["fp32"]}[out.dtype]
    sc = scheme.c()
    _check(_lib().bq_dequantize(_ptr(codes), _ptr(scales), _ptr(zero_points), _ptr(tensor_scale), rows, cols,
                                ctypes.byref(sc), _ptr(out), out_dt, _stream(stream)), "bq_dequantize")


def bq_qsnr(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, zero_points: torch.Tensor | None,
            tensor_scale: torch.Tensor | None, scheme: Scheme, stats: torch.Tensor,
            workspace: torch.Tensor, stream=None) -> None:
    rows, cols = x.shape
    sc = scheme.c()
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(_lib().bq_qsnr(_ptr(x), DT["bf16"], _ptr(codes), _ptr(scales), _ptr(zero_points), _ptr(tensor_scale),
                          rows, cols, ctypes.byref(sc), _ptr(stats), _ptr(workspace), ws_bytes, _stream(stream)),
           "bq_qsnr")


def _rt(col_scale: torch.Tensor | None, sign_bits: torch.Tensor | None) -> BqRowTransform:
    return BqRowTransform(_ptr(col_scale), _ptr(sign_bits), 0)


def bq_quantize_rt(x: torch.Tensor, scheme: Scheme, col_scale: torch.Tensor | None, sign_bits: torch.Tensor | None,
                   codes: torch.Tensor, scales: torch.Tensor, zero_points: torch.Tensor | None,
                   stats: torch.Tensor | None, workspace: torch.Tensor | None, stream=None) -> None:
    """x: bf16 [rows, cols]; col_scale: fp32 [cols] or None; sign_bits: int32 [cols / 32]
    (bit j % 32 of word j / 32 negates column j) or None (no rotation)."""
    rows, cols = x.shape
    sc = scheme.c()
    rt = _rt(col_scale, sign_bits)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib().bq_quantize_rt(_ptr(x), DT["bf16"], rows, cols, ctypes.byref(sc), ctypes.byref(rt), _ptr(codes),
                                 _ptr(scales), _ptr(zero_points), _ptr(stats), _ptr(workspace), ws_bytes,
                                 _stream(stream)), "bq_quantize_rt")


def bq_dequantize_rt(codes: torch.Tensor, scales: torch.Tensor, zero_points: torch.Tensor | None, rows: int,
                     cols: int, scheme: Scheme, col_scale: torch.Tensor | None, sign_bits: torch.Tensor | None,
                     out: torch.Tensor, stream=None) -> None:
    out_dt = {torch.bfloat16: DT["bf16"], torch.float32: DT["fp32"]}[out.dtype]
    sc = scheme.c()
    rt = _rt(col_scale, sign_bits)
    _check(_lib().bq_dequantize_rt(_ptr(codes), _ptr(scales), _ptr(zero_points), rows, cols, ctypes.byref(sc),
                                   ctypes.byref(rt), _ptr(out), out_dt, _stream(stream)), "bq_dequantize_rt")


def pack_sign_bits(signs, device=None) -> torch.Tensor:
    """Per-column 0/1 flags (1 = negate) -> int32 words, bit j % 32 of word j / 32."""
    f = torch.as_tensor(signs).to(torch.int64).reshape(-1, 32)
    w = (f << torch.arange(32, dtype=torch.int64)).sum(1)
    w = torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)
    return w.to(device) if device is not None else w


def bq_wait_timeouts(reset: bool = False) -> int:
    """Waits of the quantize, GEMM and linear kernels that gave up on the current device (each
    leaves its call's outputs incomplete); synchronizes with the device."""
    c = ctypes.c_uint32(0)
    _check(_lib().bq_wait_timeouts(ctypes.byref(c), 1 if reset else 0), "bq_wait_timeouts")
    return int(c.value)


def bq_stats_qsnr_db(stats_host) -> float:
    """QSNR in dB from a host copy of the five stats values (tensor or sequence)."""
    v = [float(a) for a in (stats_host.tolist() if hasattr(stats_host, "tolist") else stats_host)]
    s = BqStats(*v[:5])
    return float(_lib().bq_stats_qsnr_db(ctypes.byref(s)))


def bq_stats_to_db(stats_host) -> float:
    """The same as bq_stats_qsnr_db (the C ABI exports both names)."""
    v = [float(a) for a in (stats_host.tolist() if hasattr(stats_host, "tolist") else stats_host)]
    s = BqStats(*v[:5])
    return float(_lib().bq_stats_to_db(ctypes.byref(s)))


# ---------------------------------------------------------------------------
# Allocation helpers
# ---------------------------------------------------------------------------

def _scale_dtype_torch(scheme: Scheme):
    s = scheme.resolved()
    if s.gran in ("mx", "nv"):
        return torch.uint8
    return torch.float16 if s.scale_dtype == "fp16" else torch.float32


def new_workspace(device=None, nbytes: int | None = None) -> torch.Tensor:
    """A zero-filled workspace large enough for any call (bytes as uint8)."""
    if nbytes is None:
        nbytes = bq_workspace_size(Scheme("int8_sym", "tensor"), 1, 16, True)
    return torch.zeros(nbytes, dtype=torch.uint8, device=device or "cuda")


@dataclass
class Quantized:
    scheme: Scheme
    rows: int
    cols: int
    codes: torch.Tensor
    scales: torch.Tensor
    zero_points: torch.Tensor | None
    tensor_scale: torch.Tensor | None
    stats: torch.Tensor | None      # float64[5] on the device: err2, x2, kappa_sum, kappa_max, n_units

    def qsnr_db(self) -> float:
        return bq_stats_qsnr_db(self.stats.cpu())

    def mean_kappa(self) -> float:
        st = self.stats.cpu().tolist()
        return st[2] / st[4] if st[4] else math.nan


def alloc_outputs(scheme: Scheme, rows: int, cols: int, device, stats: bool = True) -> Quantized:
    s = scheme.resolved()
    cb, sb, zb, tb = bq_buffer_sizes(s, rows, cols)
    sdt = _scale_dtype_torch(s)
    esz = torch.tensor([], dtype=sdt).element_size()
    cols_b = cols // 2 if s.fmt in FOUR_BIT else cols
    codes = torch.empty((rows, cols_b), dtype=torch.uint8, device=device)
    scales = torch.empty(max(sb // esz, 1), dtype=sdt, device=device)
    zps = torch.empty(zb // esz, dtype=sdt, device=device) if zb else None
    ts = torch.empty(1, dtype=torch.float32, device=device) if tb else None
    st = torch.empty(5, dtype=torch.float64, device=device) if stats else None
    return Quantized(s, rows, cols, codes, scales, zps, ts, st)


# the bytes of a scheme's codes, scales, zero points and tensor scale for a shape (plain values)
_sizes = functools.lru_cache(maxsize=1024)(bq_buffer_sizes)


def _buffers(q, dev: torch.device, rows: int, cols: int, batch: int = 1) -> None:
    """Refuses a handle (Quantized, QuantizedBatch) whose buffers do not hold batch tensors of
    [rows, cols] under its scheme: another device, not contiguous, or too short."""
    if dev.type != "cuda":
        raise ValueError("the tensors must be on a CUDA device")
    cb, sb, zb, tb = _sizes(q.scheme, rows, cols)
    c, s = q.codes, q.scales
    if c.device != dev or not c.is_contiguous() or c.nbytes < cb * batch:
        raise ValueError(f"codes: expected {cb * batch} contiguous bytes on {dev}")
    if s.device != dev or not s.is_contiguous() or s.nbytes < sb * batch:
        raise ValueError(f"scales: expected {sb * batch} contiguous bytes on {dev}")
    if zb or tb:
        for name, need in (("zero_points", zb * batch), ("tensor_scale", tb)):
            t = getattr(q, name, None) if need else None
            if t is not None and (t.device != dev or not t.is_contiguous() or t.nbytes < need):
                raise ValueError(f"{name}: expected {need} contiguous bytes on {dev}")


@dataclass
class QuantizedBatch:
    scheme: Scheme
    batch: int
    rows: int
    cols: int
    codes: torch.Tensor             # uint8 [batch, rows, cols] (4-bit: [batch, rows, cols / 2])
    scales: torch.Tensor            # [batch, one tensor's scales]
    zero_points: torch.Tensor | None
    stats: torch.Tensor | None      # float64 [batch, 5]

    def tensor(self, b: int) -> Quantized:
        """Tensor b's outputs as a Quantized (views, no copy)."""
        return Quantized(self.scheme, self.rows, self.cols, self.codes[b], self.scales[b],
                         None if self.zero_points is None else self.zero_points[b], None,
                         None if self.stats is None else self.stats[b])


def alloc_batch_outputs(scheme: Scheme, batch: int, rows: int, cols: int, device, stats: bool = True) -> QuantizedBatch:
    s = scheme.resolved()
    cb, sb, zb, _ = bq_buffer_sizes(s, rows, cols)
    sdt = _scale_dtype_torch(s)
    esz = torch.tensor([], dtype=sdt).element_size()
    cols_b = cols // 2 if s.fmt in FOUR_BIT else cols
    codes = torch.empty((batch, rows, cols_b), dtype=torch.uint8, device=device)
    scales = torch.empty((batch, max(sb // esz, 1)), dtype=sdt, device=device)
    zps = torch.empty((batch, zb // esz), dtype=sdt, device=device) if zb else None
    st = torch.empty((batch, 5), dtype=torch.float64, device=device) if stats else None
    return QuantizedBatch(s, batch, rows, cols, codes, scales, zps, st)


def quantize_batch(x: torch.Tensor, scheme: Scheme, stats: bool = True, workspace: torch.Tensor | None = None,
                   out: QuantizedBatch | None = None, stream=None) -> QuantizedBatch:
    """Quantize a bf16 [batch, rows, cols] CUDA tensor (same-shape tensors, one launch);
    per-tensor QSNR / kappa sums in stats[b]."""
    if x.dtype != torch.bfloat16 or not x.is_cuda or x.dim() != 3:
        raise ValueError("x must be a 3-D bf16 CUDA tensor")
    x = x.contiguous()
    batch, rows, cols = x.shape
    q = out or alloc_batch_outputs(scheme, batch, rows, cols, x.device, stats)
    if out is not None:
        _buffers(q, x.device, rows, cols, batch)
    if stats and workspace is None:
        workspace = new_workspace(x.device)
    bq_quantize_batch(x, q.scheme, q.codes, q.scales, q.zero_points, q.stats if stats else None, workspace, stream)
    return q


def quantize(x: torch.Tensor, scheme: Scheme, stats: bool = True, workspace: torch.Tensor | None = None,
             out: Quantized | None = None, stream=None) -> Quantized:
    """Quantize a bf16 [rows, cols] CUDA tensor; returns codes, scales, zero points,
    tensor scale and (optionally) the QSNR / kappa sums, all on the device."""
    if x.dtype != torch.bfloat16 or not x.is_cuda or x.dim() != 2:
        raise ValueError("x must be a 2-D bf16 CUDA tensor")
    x = x.contiguous()
    rows, cols = x.shape
    q = out or alloc_outputs(scheme, rows, cols, x.device, stats)
    if out is not None:
        _buffers(q, x.device, rows, cols)
    if workspace is None and bq_workspace_size(q.scheme, rows, cols, stats) > 0:
        workspace = new_workspace(x.device)
    bq_quantize(x, q.scheme, q.codes, q.scales, q.zero_points, q.tensor_scale, q.stats if stats else None,
                workspace, stream)
    return q


def dequantize(q: Quantized, dtype=torch.bfloat16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    _buffers(q, q.codes.device, q.rows, q.cols)
    if out is None:
        out = torch.empty((q.rows, q.cols), dtype=dtype, device=q.codes.device)
    bq_dequantize(q.codes, q.scales, q.zero_points, q.tensor_scale, q.rows, q.cols, q.scheme, out, stream)
    return out


def quantize_rt(x: torch.Tensor, scheme: Scheme, col_scale: torch.Tensor | None = None,
                sign_bits: torch.Tensor | None = None, stats: bool = True, workspace: torch.Tensor | None = None,
                stream=None) -> Quantized:
    """Quantize a bf16 [rows, cols] CUDA tensor after the row transforms (per-column
    factor, randomized full-row Hadamard rotation); per-row, per-group and MX schemes."""
    if x.dtype != torch.bfloat16 or not x.is_cuda or x.dim() != 2:
        raise ValueError("x must be a 2-D bf16 CUDA tensor")
    x = x.contiguous()
    rows, cols = x.shape
    q = alloc_outputs(scheme, rows, cols, x.device, stats)
    if stats and workspace is None:
        workspace = new_workspace(x.device)
    bq_quantize_rt(x, q.scheme, col_scale, sign_bits, q.codes, q.scales, q.zero_points,
                   q.stats if stats else None, workspace, stream)
    return q


def dequantize_rt(q: Quantized, col_scale: torch.Tensor | None = None, sign_bits: torch.Tensor | None = None,
                  dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    _buffers(q, q.codes.device, q.rows, q.cols)
    out = torch.empty((q.rows, q.cols), dtype=dtype, device=q.codes.device)
    bq_dequantize_rt(q.codes, q.scales, q.zero_points, q.rows, q.cols, q.scheme, col_scale, sign_bits, out, stream)
    return out


def qsnr(x: torch.Tensor, q: Quantized, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Standalone QSNR sums (float64[5] on the device; kappa fields zero)."""
    _buffers(q, x.device, *x.shape)
    st = torch.empty(5, dtype=torch.float64, device=x.device)
    if workspace is None:
        workspace = new_workspace(x.device)
    bq_qsnr(x.contiguous(), q.codes, q.scales, q.zero_points, q.tensor_scale, q.scheme, st, workspace, stream)
    return st


# ---------------------------------------------------------------------------
# A linear layer over block-scaled data, and the gated activation between two of them
#
# Plain functions: results carry no autograd graph, whatever their inputs do. Rows of bf16 inputs
# may be apart; an input whose rows are not a multiple of 8 elements apart (16 in the gated
# activation), whose columns are not adjacent or whose start is not aligned to as many elements
# is copied first (2 bytes an element read and written once more). A contiguous [m, n] with n
# % 8 != 0 is one: a caller with an odd number of outputs who keeps dy in rows of a multiple of 8
# (a slice of a wider buffer) saves the copy on each call.
# ---------------------------------------------------------------------------

_OUT_DT = {torch.bfloat16: 0, torch.float32: 2}


def _c_scheme(scheme: Scheme):
    """A reference to scheme.c() as the C entry points take it, kept on the scheme (a frozen
    value), for the calls whose host time counts."""
    c = scheme.__dict__.get("_c")
    if c is None:
        c = ctypes.byref(scheme.c())
        object.__setattr__(scheme, "_c", c)
    return c


def _raw_stream(dev: torch.device) -> int:
    """The current stream of dev (torch.cuda.current_stream(dev).cuda_stream without the object)."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _elsewhere(dev: torch.device, stream) -> bool:
    if dev.type != "cuda":
        raise ValueError("the tensors must be on a CUDA device")
    return stream is not None or dev.index != torch._C._cuda_getDevice()     # (current_device() without its checks)


@contextlib.contextmanager
def _on(dev: torch.device, stream):
    """dev, and the given stream if any, current: whatever a call allocates, copies and launches
    goes there."""
    with torch.cuda.device(dev):
        if stream is None:
            yield
            return
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), dev) if int(stream) else torch.cuda.default_stream(dev)
        if stream.device != dev:
            raise ValueError(f"the stream is on {stream.device}, the codes on {dev}")
        with torch.cuda.stream(stream):
            yield


def _operand(t: torch.Tensor, name: str, rows: int | None, cols: int, dev: torch.device, step: int):
    """(t or a copy of it, elements between its rows): bf16 [rows, cols] on dev with unit column
    stride, rows a multiple of step elements apart and the first element 2 * step bytes
    aligned. (A tensor of at most one row, or of none to a row, has no such distance: any
    valid value.)"""
    if t.dtype is not torch.bfloat16 or t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a 2-D bf16 CUDA tensor")
    r, c = t.shape
    if c != cols or (rows is not None and r != rows):
        raise ValueError(f"{name} is [{r}, {c}], expected [{'any' if rows is None else rows}, {cols}]")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the codes on {dev}")
    ld, s1 = t.stride()
    if r <= 1 or c == 0:
        ld = -(-c // step) * step
    if (s1 == 1 or c == 1) and ld >= c and ld % step == 0 and t.data_ptr() % (2 * step) == 0:
        return t, ld
    ld = -(-c // step) * step
    buf = torch.empty((r, ld), dtype=t.dtype, device=dev)[:, :c]
    buf.copy_(t)
    return buf, ld


def _handle(q: Quantized, dev: torch.device) -> None:
    """Refuses a Quantized (a handle can be built by hand) whose buffers an MX or NV kernel would
    read or write past their end: on another device, not contiguous, or shorter than its scheme
    and shape ask. (Other schemes are refused by the calls that this serves.)"""
    s, rows, cols = q.scheme, q.rows, q.cols
    nv = s.gran == "nv"
    if not nv and s.gran != "mx":
        return
    codes, scales = q.codes, q.scales
    if (codes.device != dev or not codes.is_contiguous() or codes.element_size() != 1
            or codes.numel() < (rows * cols // 2 if s.fmt in FOUR_BIT else rows * cols)):
        raise ValueError(f"the codes are not contiguous bytes of a {s.fmt} [{rows}, {cols}] tensor on {dev}")
    if (scales.device != dev or not scales.is_contiguous() or scales.element_size() != 1
            or scales.numel() < ((rows + 127) // 128 * 128 if s.layout == "gemm" else rows) * (cols // (16 if nv else 32))):
        raise ValueError(f"the scales are not contiguous bytes of [{rows}, {cols // (16 if nv else 32)}] blocks on {dev}")
    if nv:
        ts = q.tensor_scale
        if ts is not None and (ts.device != dev or ts.dtype is not torch.float32 or ts.numel() < 1):
            raise ValueError(f"the tensor scale is not fp32 on {dev}")


def _out(out: torch.Tensor | None, rows: int, cols: int, dtype, dev: torch.device) -> torch.Tensor:
    if out is None:
        if dtype not in _OUT_DT:
            raise ValueError("dtype must be torch.bfloat16 or torch.float32")
        return torch.empty((rows, cols), dtype=dtype, device=dev)
    if out.shape != (rows, cols) or out.dtype not in _OUT_DT or not out.is_contiguous() or out.device != dev:
        raise ValueError(f"out must be a contiguous bf16 or fp32 [{rows}, {cols}] tensor on {dev}")
    return out


def linear(x: torch.Tensor, w: Quantized, dtype=torch.bfloat16, out: torch.Tensor | None = None,
           stream=None) -> torch.Tensor:
    """x W^T: bf16 x [m, k] (rows may be apart) and a 4-bit weight w (E2M1 under "mx" or "nv")
    of [n, k] -> [m, n] of dtype (or of out's). No autograd: linear_grad_input and
    linear_grad_weight are its gradients."""
    dev = w.codes.device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return linear(x, w, dtype, out)
    _handle(w, dev)
    x, ld = _operand(x, "x", None, w.cols, dev, 8)
    m, n = x.shape[0], w.rows
    y = _out(out, m, n, dtype, dev)
    _check(_lib().bq_linear(x.data_ptr(), 0, ld, w.codes.data_ptr(), w.scales.data_ptr(), _ptr(w.tensor_scale), m, n,
                            w.cols, _c_scheme(w.scheme), y.data_ptr(), _OUT_DT[y.dtype],
                            _raw_stream(dev)), "bq_linear")
    return y


def linear_grad_input(dy: torch.Tensor, w: Quantized, dtype=torch.bfloat16, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """dy W: the gradient of linear's x, from bf16 dy [m, n] and the weight [n, k] -> [m, k]. A
    dy whose rows are not a multiple of 8 elements apart is copied first."""
    dev = w.codes.device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return linear_grad_input(dy, w, dtype, out)
    _handle(w, dev)
    dy, ld = _operand(dy, "dy", None, w.rows, dev, 8)
    m, k = dy.shape[0], w.cols
    dx = _out(out, m, k, dtype, dev)
    _check(_lib().bq_linear_grad_input(dy.data_ptr(), 0, ld, w.codes.data_ptr(), w.scales.data_ptr(),
                                       _ptr(w.tensor_scale), m, w.rows, k, _c_scheme(w.scheme),
                                       dx.data_ptr(), _OUT_DT[dx.dtype], _raw_stream(dev)), "bq_linear_grad_input")
    return dx


def linear_grad_weight(dy: torch.Tensor, x: Quantized, dtype=torch.float32, out: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """dy^T X: the gradient of linear's weight, from bf16 dy [m, n] and the layer's input kept
    in 8 bits (E4M3, E5M2 or INT8 under "mx") x of [m, k] -> [n, k]. A dy whose rows are not a
    multiple of 8 elements apart is copied first."""
    dev = x.codes.device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return linear_grad_weight(dy, x, dtype, out)
    _handle(x, dev)
    dy, ld = _operand(dy, "dy", x.rows, dy.shape[-1], dev, 8)
    n, k = dy.shape[1], x.cols
    dw = _out(out, n, k, dtype, dev)
    _check(_lib().bq_linear_grad_weight(dy.data_ptr(), 0, ld, x.codes.data_ptr(), x.scales.data_ptr(), x.rows, n, k,
                                        _c_scheme(x.scheme), dw.data_ptr(), _OUT_DT[dw.dtype],
                                        _raw_stream(dev)), "bq_linear_grad_weight")
    return dw


def _resolved(scheme: Scheme) -> Scheme:
    """scheme.resolved(), kept on the scheme like its C form."""
    r = scheme.__dict__.get("_r")
    if r is None:
        r = scheme.resolved()
        object.__setattr__(scheme, "_r", r)
    return r


def _glu_copy(s: Scheme, rows: int, cols: int, dev: torch.device) -> Quantized:
    """Buffers of one 8-bit MX copy (alloc_outputs of the schemes that bq_glu takes; the others
    it refuses before they are written)."""
    return Quantized(s, rows, cols, torch.empty((rows, cols), dtype=torch.uint8, device=dev),
                     torch.empty(max(rows * cols // 32, 1), dtype=torch.uint8, device=dev), None, None, None)


@dataclass
class GluCheckpoint:
    """What glu keeps for glu_backward: the gate and the up projection in 8 bits."""
    gate: Quantized
    up: Quantized
    act: str


def glu(gate: torch.Tensor, up: torch.Tensor, scheme: Scheme | None = None, act: str = "silu",
        out: torch.Tensor | None = None, ckpt: GluCheckpoint | None = None, stream=None):
    """h = a(gate) up of bf16 [rows, cols] tensors (rows may be apart, e.g. the halves of one
    [rows, 2 cols] tensor) -> (h, GluCheckpoint), the copies quantized under scheme (E4M3,
    E5M2 or INT8 with "mx"; to ckpt's buffers when given); without a scheme (h, None)."""
    if gate.dim() != 2 or gate.shape != up.shape:
        raise ValueError("gate and up must be 2-D tensors of the same shape")
    rows, cols = gate.shape
    dev = gate.device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return glu(gate, up, scheme, act, out, ckpt)
    gate, ldg = _operand(gate, "gate", rows, cols, dev, 16)
    up, ldu = _operand(up, "up", rows, cols, dev, 16)
    h = _out(out, rows, cols, torch.bfloat16, dev)
    if h.dtype is not torch.bfloat16:
        raise ValueError("out must be bf16")
    if scheme is None:
        if ckpt is not None:
            raise ValueError("a checkpoint needs a scheme")
        _check(_lib().bq_glu(gate.data_ptr(), ldg, up.data_ptr(), ldu, 0, rows, cols, ACTS[act], h.data_ptr(), None, None,
                             None, None, None, _raw_stream(dev)), "bq_glu")
        return h, None
    a = ACTS[act]
    if ckpt is None:
        s = _resolved(scheme)
        g, u = _glu_copy(s, rows, cols, dev), _glu_copy(s, rows, cols, dev)
        ckpt = GluCheckpoint(g, u, act)
    else:
        s, g, u = _resolved(scheme), ckpt.gate, ckpt.up
        if g.scheme != s or u.scheme != s or (g.rows, g.cols) != (rows, cols) or (u.rows, u.cols) != (rows, cols):
            raise ValueError("the checkpoint's buffers are of another scheme or shape")
        _handle(g, dev)
        _handle(u, dev)
        ckpt.act = act
    _check(_lib().bq_glu(gate.data_ptr(), ldg, up.data_ptr(), ldu, 0, rows, cols, a, h.data_ptr(),
                         _c_scheme(s), g.codes.data_ptr(), g.scales.data_ptr(), u.codes.data_ptr(),
                         u.scales.data_ptr(), _raw_stream(dev)), "bq_glu")
    return h, ckpt


def glu_backward(dh: torch.Tensor, ckpt: GluCheckpoint, out=None, stream=None):
    """(dgate, dup) of glu from bf16 dh [rows, cols] and what glu kept; out: two bf16 tensors
    to write (unit column stride, rows a multiple of 16 elements apart, e.g. the halves of
    one [rows, 2 cols] tensor)."""
    g, u = ckpt.gate, ckpt.up
    dev, rows, cols = g.codes.device, g.rows, g.cols
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return glu_backward(dh, ckpt, out)
    if u.rows != rows or u.cols != cols or (u.scheme is not g.scheme and u.scheme != g.scheme):
        raise ValueError("the two copies must be of one shape and scheme")
    _handle(g, dev)
    _handle(u, dev)
    dh, ldh = _operand(dh, "dh", rows, cols, dev, 16)
    if out is None:
        dg = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev)
        du = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev)
        ldg = ldu = cols
    else:
        dg, du = out
        (tg, ldg), (tu, ldu) = _operand(dg, "out", rows, cols, dev, 16), _operand(du, "out", rows, cols, dev, 16)
        if tg is not dg or tu is not du:
            raise ValueError("out must have unit column stride, rows a multiple of 16 elements apart and be 32-byte aligned")
    _check(_lib().bq_glu_backward(dh.data_ptr(), ldh, 0, g.codes.data_ptr(), g.scales.data_ptr(), u.codes.data_ptr(),
                                  u.scales.data_ptr(), _c_scheme(g.scheme), rows, cols, ACTS[ckpt.act],
                                  dg.data_ptr(), ldg, du.data_ptr(), ldu, _raw_stream(dev)), "bq_glu_backward")
    return dg, du
