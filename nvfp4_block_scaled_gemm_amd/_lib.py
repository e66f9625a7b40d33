"""ctypes binding of libnvfp4.so (include/nvfp4.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels of the library.  torch supplies device memory (``data_ptr``) and the
current HIP stream.  If the library has not been built, loading raises;
there is no fallback implementation.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import functools
import os
import typing

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4.so")

NVFP4_OK = 0
NVFP4_ERR_INVALID_ARG = -1
NVFP4_ERR_UNSUPPORTED = -2
NVFP4_ERR_HIP = -3
NVFP4_F32 = 0
NVFP4_BF16 = 1
NVFP4_GLOBAL_SCALE_GIVEN = 1

EXPORTED = ("nvfp4_status_string", "nvfp4_version", "nvfp4_quantize_workspace_bytes",
            "nvfp4_quantize", "nvfp4_quantize_noalloc", "nvfp4_gemm", "nvfp4_gemm_nvfp4_out", "nvfp4_grouped_gemm",
            "nvfp4_grouped_gemm_gather", "nvfp4_grouped_gemm_multi", "nvfp4_mxfp4_quantize",
            "nvfp4_mxfp4_gemm", "nvfp4_fp8_quantize", "nvfp4_fp8_grouped_columns",
            "nvfp4_fp8_grouped_quantize", "nvfp4_fp8_gemm", "nvfp4_fp8_grouped_gemm",
            "nvfp4_fp8_grouped_wgrad", "nvfp4_moe_route_workspace_bytes", "nvfp4_moe_route",
            "nvfp4_moe_route_backward", "nvfp4_fp8_gated_gemm", "nvfp4_fp8_grouped_gated_gemm",
            "nvfp4_fp8_gated_backward", "nvfp4_fp8_grouped_gated_backward", "nvfp4_int8_quantize",
            "nvfp4_int8_gemm", "nvfp4_grad_workspace_bytes", "nvfp4_grad_norm_sq", "nvfp4_clip_grads")
NVFP4_ACCUMULATE = 1
NVFP4_ROUTE_RENORMALIZE = 1
NVFP4_SILU = 0
NVFP4_GELU = 1
NVFP4_GROUPED_MAX_PROBLEMS = 4

_lib = None


class GroupedProblem(ctypes.Structure):
    """nvfp4_grouped_problem of include/nvfp4.h (one grouped GEMM)."""
    _fields_ = [("G", ctypes.c_int32), ("m_offsets", ctypes.c_void_p),
                ("row_index", ctypes.c_void_p), ("total_m", ctypes.c_int64),
                ("a_rows", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("a_q", ctypes.c_void_p), ("a_s", ctypes.c_void_p), ("a_g", ctypes.c_void_p),
                ("b_q", ctypes.c_void_p), ("b_s", ctypes.c_void_p), ("b_g", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("y_dtype", ctypes.c_int), ("ld_y", ctypes.c_int64)]


class Grad(ctypes.Structure):
    """nvfp4_grad of include/nvfp4.h (one gradient of a list)."""
    _fields_ = [("g", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("g_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int)]


class Nvfp4Error(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed: {msg} ({status})")
        self.status = status


def load() -> ctypes.CDLL:
    """Load libnvfp4.so once; raises if it is missing (build it first)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing; run `python -m "
                          "nvfp4_block_scaled_gemm_amd.build` (hipcc, gfx950)")
    lib = ctypes.CDLL(LIB_PATH)
    p, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    lib.nvfp4_status_string.argtypes = [ctypes.c_int]
    lib.nvfp4_status_string.restype = ctypes.c_char_p
    lib.nvfp4_version.argtypes = []
    lib.nvfp4_version.restype = ctypes.c_char_p
    lib.nvfp4_quantize_workspace_bytes.argtypes = [i64, i64]
    lib.nvfp4_quantize_workspace_bytes.restype = sz
    lib.nvfp4_quantize.argtypes = [p, ctypes.c_int, i64, i64, i64, p, p, p, ctypes.c_uint,
                                   p, sz, p]
    lib.nvfp4_quantize.restype = ctypes.c_int
    lib.nvfp4_quantize_noalloc.argtypes = [p, ctypes.c_int, i64, i64, i64, p, p, p, ctypes.c_uint,
                                           p]
    lib.nvfp4_quantize_noalloc.restype = ctypes.c_int
    lib.nvfp4_gemm.argtypes = [i64, i64, i64, p, p, p, p, p, p, p, ctypes.c_int, i64, p]
    lib.nvfp4_gemm.restype = ctypes.c_int
    lib.nvfp4_gemm_nvfp4_out.argtypes = [i64, i64, i64, p, p, p, p, p, p, p, p, p, p]
    lib.nvfp4_gemm_nvfp4_out.restype = ctypes.c_int
    lib.nvfp4_grouped_gemm.argtypes = [i32, p, i64, i64, i64, p, p, p, p, p, p, p,
                                       ctypes.c_int, i64, p]
    lib.nvfp4_grouped_gemm.restype = ctypes.c_int
    lib.nvfp4_grouped_gemm_gather.argtypes = [i32, p, p, i64, i64, i64, i64, p, p, p, p, p, p,
                                              p, ctypes.c_int, i64, p]
    lib.nvfp4_grouped_gemm_gather.restype = ctypes.c_int
    lib.nvfp4_grouped_gemm_multi.argtypes = [i32, ctypes.POINTER(GroupedProblem), p]
    lib.nvfp4_grouped_gemm_multi.restype = ctypes.c_int
    lib.nvfp4_mxfp4_quantize.argtypes = [p, ctypes.c_int, i64, i64, i64, p, p, p]
    lib.nvfp4_mxfp4_quantize.restype = ctypes.c_int
    lib.nvfp4_mxfp4_gemm.argtypes = [i64, i64, i64, p, p, p, p, p, ctypes.c_int, i64, p]
    lib.nvfp4_mxfp4_gemm.restype = ctypes.c_int
    c_int, c_uint = ctypes.c_int, ctypes.c_uint
    lib.nvfp4_fp8_quantize.argtypes = [p, c_int, i64, i64, i64, i64, c_int, p, p, p, p, p]
    lib.nvfp4_fp8_quantize.restype = c_int
    lib.nvfp4_fp8_grouped_columns.argtypes = [i64, i32]
    lib.nvfp4_fp8_grouped_columns.restype = i64
    lib.nvfp4_fp8_grouped_quantize.argtypes = [p, c_int, i32, p, p, i64, i64, i64, i64, p, p, p, p,
                                               p]
    lib.nvfp4_fp8_grouped_quantize.restype = c_int
    lib.nvfp4_fp8_gemm.argtypes = [i64, i64, i64, p, p, p, p, c_int, p, c_int, i64, c_uint, p]
    lib.nvfp4_fp8_gemm.restype = c_int
    lib.nvfp4_fp8_grouped_gemm.argtypes = [i32, p, p, i64, i64, i64, i64, p, p, p, p, p, c_int, i64,
                                           p]
    lib.nvfp4_fp8_grouped_gemm.restype = c_int
    lib.nvfp4_fp8_grouped_wgrad.argtypes = [i32, p, i64, i64, i64, p, p, p, p, p, c_int, c_uint, p]
    lib.nvfp4_fp8_grouped_wgrad.restype = c_int
    lib.nvfp4_moe_route_workspace_bytes.argtypes = [i64, i64]
    lib.nvfp4_moe_route_workspace_bytes.restype = sz
    lib.nvfp4_moe_route.argtypes = [i64, i64, i32, p, c_int, i64, p, c_uint, p, p, p, p, p, p, p, p,
                                    p, sz, p]
    lib.nvfp4_moe_route.restype = c_int
    lib.nvfp4_moe_route_backward.argtypes = [i64, i64, i32, p, c_int, i64, p, c_uint, p, p, p, p, p,
                                             p, i64, p]
    lib.nvfp4_moe_route_backward.restype = c_int
    lib.nvfp4_fp8_gated_gemm.argtypes = [i64, i64, i64, p, p, p, p, c_int, c_int, p, c_int, i64, p, i64, p]
    lib.nvfp4_fp8_gated_gemm.restype = c_int
    lib.nvfp4_fp8_grouped_gated_gemm.argtypes = [i32, p, p, i64, i64, i64, i64, p, p, p, p, c_int, p, c_int,
                                                 i64, p, i64, p]
    lib.nvfp4_fp8_grouped_gated_gemm.restype = c_int
    lib.nvfp4_fp8_gated_backward.argtypes = [p, c_int, i64, p, c_int, i64, c_int, i64, i64, p, p, p, p, p]
    lib.nvfp4_fp8_gated_backward.restype = c_int
    lib.nvfp4_fp8_grouped_gated_backward.argtypes = [i32, p, p, c_int, i64, p, c_int, i64, c_int, i64, i64, p,
                                                     p, p, p, p]
    lib.nvfp4_fp8_grouped_gated_backward.restype = c_int
    lib.nvfp4_int8_quantize.argtypes = [p, c_int, i64, i64, i64, p, p, p]
    lib.nvfp4_int8_quantize.restype = c_int
    lib.nvfp4_int8_gemm.argtypes = [i64, i64, i64, p, p, p, p, p, c_int, i64, p]
    lib.nvfp4_int8_gemm.restype = c_int
    lib.nvfp4_grad_workspace_bytes.argtypes = [i64]
    lib.nvfp4_grad_workspace_bytes.restype = sz
    lib.nvfp4_grad_norm_sq.argtypes = [i64, p, p, p, sz, p]
    lib.nvfp4_grad_norm_sq.restype = c_int
    lib.nvfp4_clip_grads.argtypes = [i64, p, ctypes.c_double, p, p, p, sz, p]
    lib.nvfp4_clip_grads.restype = c_int
    _lib = lib
    return lib


def _check(fn: str, status: int):
    if status != NVFP4_OK:
        msg = load().nvfp4_status_string(status).decode()
        raise Nvfp4Error(fn, status, msg)


def _ptr(t):
    # the pointer arguments are declared c_void_p, so a plain int is passed
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None, dev: int | None = None):
    """HIP stream handle: ``stream`` (a torch stream or a raw handle), else the
    current stream of device ``dev`` (default: the current device)."""
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    if dev is None:
        dev = torch.cuda.current_device()
    if _raw_stream is not None:
        return _raw_stream(dev)
    return torch.cuda.current_stream(dev).cuda_stream


def _on_stream(stream, dev: int):
    """Context in which the wrapper's own torch work (output allocations, the
    static-scale copy, its internal workspace) is ordered on the same stream
    as the library call: ``stream`` when given (a torch stream or a raw
    handle), else nothing to change (the current stream is used by both)."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev)
    return torch.cuda.stream(stream)


_DT_IN = {torch.float32: NVFP4_F32, torch.bfloat16: NVFP4_BF16}
_DT_OUT = {"f32": (NVFP4_F32, torch.float32), "bf16": (NVFP4_BF16, torch.bfloat16)}


# The library reads packed operands as row-major [rows, K/2] and [rows, K/16]
# bytes and writes outputs of the dtype it is told; these checks keep a
# mismatched tensor from reaching it (they raise before any GPU work).  A
# packed operand is checked once, when it becomes a ``Packed``, so that the
# per-call cost stays small next to a few-microsecond decode GEMM.
def _need(cond: bool, msg: str):
    if not cond:
        raise ValueError(msg)


class Packed(tuple):
    """(q, s, g) of an NVFP4 tensor [rows, K], or of G expert weights
    [G, rows, K]: uint8 q [.., rows, K/2] and s [.., rows, K/16], both
    contiguous, and fp32 g (one value, or one per expert), all on one GPU.
    Checked when made; nvfp4_quantize returns one.  Changing the tensors'
    shapes in place afterwards is not supported."""

    def __new__(cls, ts, _trusted=None):
        q, s, g = ts
        self = super().__new__(cls, (q, s, g))
        if _trusted is not None:
            self.lead, self.rows, self.K, self.dev = _trusted
            return self
        _need(q.dim() >= 2, "q: at least 2-D")
        lead = tuple(q.shape[:-2])
        rows, K = q.shape[-2], q.shape[-1] * 2
        _need(q.dtype == torch.uint8 and s.dtype == torch.uint8, "q and s must be uint8")
        _need(tuple(s.shape) == (*lead, rows, K // 16) and K % 16 == 0,
              f"q {tuple(q.shape)} and s {tuple(s.shape)} do not pack [{rows}, {K}]")
        _need(q.is_contiguous() and s.is_contiguous(), "q and s must be contiguous")
        n_g = lead[0] if len(lead) == 1 else 1
        _need(len(lead) <= 1, "at most one leading (expert) dimension")
        _need(g.dtype == torch.float32 and g.numel() == n_g and g.is_contiguous(),
              f"g must be {n_g} contiguous fp32 value(s)")
        dev = q.get_device()
        _need(q.is_cuda and s.get_device() == dev and g.get_device() == dev,
              "q, s and g must be on one GPU")
        self.lead, self.rows, self.K, self.dev = lead, rows, K, dev
        return self


def _packed(t3) -> Packed:
    return t3 if type(t3) is Packed else Packed(t3)


def _out(y, rows: int, cols: int, dtype, dev: int, what: str = "y") -> int:
    """Checks an output [rows, cols] of ``dtype`` on GPU ``dev``; returns its
    row stride."""
    st = y.stride()
    if y.dtype == dtype and y.shape == (rows, cols) and (st[1] == 1 or cols <= 1) \
            and y.get_device() == dev:
        return st[0]
    _need(y.dtype == dtype, f"{what}: dtype {y.dtype}, expected {dtype}")
    _need(y.shape == (rows, cols), f"{what}: shape {tuple(y.shape)}, expected ({rows}, {cols})")
    _need(st[1] == 1 or cols <= 1, f"{what}: rows must have unit column stride")
    raise ValueError(f"{what}: must be on the operands' GPU")


def _on_dev(t, dev: int, what: str):
    _need(t.get_device() == dev, f"{what}: must be on the operands' GPU")


# --------------------------------------------------------------------------
# raw entry points (same names and arguments as the C ABI)
# --------------------------------------------------------------------------

def nvfp4_quantize_workspace_bytes(rows: int, cols: int) -> int:
    return int(load().nvfp4_quantize_workspace_bytes(rows, cols))


def nvfp4_quantize_raw(x, x_dtype, rows, cols, ld_x, q, s, global_scale, flags,
                       workspace, workspace_bytes, stream=None) -> int:
    return load().nvfp4_quantize(x, x_dtype, rows, cols, ld_x, q, s, global_scale, flags,
                                 workspace, workspace_bytes, _stream(stream))


def nvfp4_quantize_noalloc_raw(x, x_dtype, rows, cols, ld_x, q, s, global_scale, flags,
                               stream=None) -> int:
    return load().nvfp4_quantize_noalloc(x, x_dtype, rows, cols, ld_x, q, s, global_scale, flags,
                                         _stream(stream))


def nvfp4_gemm_raw(M, N, K, a_q, a_s, a_g, b_q, b_s, b_g, y, y_dtype, ld_y,
                   stream=None) -> int:
    return load().nvfp4_gemm(M, N, K, a_q, a_s, a_g, b_q, b_s, b_g, y, y_dtype, ld_y,
                             _stream(stream))


def nvfp4_gemm_nvfp4_out_raw(M, N, K, a_q, a_s, a_g, b_q, b_s, b_g, y_q, y_s, y_g,
                             stream=None) -> int:
    return load().nvfp4_gemm_nvfp4_out(M, N, K, a_q, a_s, a_g, b_q, b_s, b_g, y_q, y_s, y_g,
                                       _stream(stream))


def nvfp4_grouped_gemm_raw(G, m_offsets, total_m, N, K, a_q, a_s, a_g, b_q, b_s, b_g, y,
                           y_dtype, ld_y, stream=None) -> int:
    return load().nvfp4_grouped_gemm(G, m_offsets, total_m, N, K, a_q, a_s, a_g, b_q, b_s,
                                     b_g, y, y_dtype, ld_y, _stream(stream))


def nvfp4_grouped_gemm_gather_raw(G, m_offsets, row_index, total_m, a_rows, N, K, a_q, a_s,
                                  a_g, b_q, b_s, b_g, y, y_dtype, ld_y, stream=None) -> int:
    return load().nvfp4_grouped_gemm_gather(G, m_offsets, row_index, total_m, a_rows, N, K,
                                            a_q, a_s, a_g, b_q, b_s, b_g, y, y_dtype, ld_y,
                                            _stream(stream))


# --------------------------------------------------------------------------
# tensor-level wrappers (allocate outputs with torch, then call the C ABI)
# --------------------------------------------------------------------------

def nvfp4_quantize(x: torch.Tensor, global_scale: torch.Tensor | None = None,
                   out=None, workspace: torch.Tensor | None = None, stream=None):
    """x [rows, cols] fp32/bf16 on the GPU -> (q uint8 [rows, cols/2],
    s uint8 [rows, cols/16], g fp32 [1]).  ``global_scale`` (device fp32 [1])
    switches to the static-scale path; ``out`` = (q, s, g) reuses buffers."""
    _need(x.dim() == 2 and x.dtype in _DT_IN, "x: 2-D fp32 or bf16")
    _need(x.stride(1) == 1 or x.shape[1] <= 1, "x: rows must have unit column stride")
    rows, cols = x.shape
    _need(cols % 16 == 0, "x: columns must be a multiple of 16")
    _need(x.is_cuda, "x: must be on a GPU")
    with _on_stream(stream, x.get_device()):
        return _quantize(x, global_scale, out, workspace)


def _quantize(x, global_scale, out, workspace):
    rows, cols = x.shape
    dev = x.device
    di = x.get_device()
    if out is None:
        q = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
        s = torch.empty((rows, cols // 16), dtype=torch.uint8, device=dev)
        g = torch.empty(1, dtype=torch.float32, device=dev)
        res = Packed((q, s, g), _trusted=((), rows, cols, di))
    else:
        res = _packed(tuple(out))
        _need(not res.lead and res.rows == rows and res.K == cols and res.dev == di,
              f"out: does not pack x [{rows}, {cols}] on its GPU")
        q, s, g = res
    if global_scale is not None:
        _need(global_scale.dtype == torch.float32 and global_scale.numel() == 1,
              "global_scale: one fp32 value")
        _on_dev(global_scale, di, "global_scale")
    if workspace is not None:
        _on_dev(workspace, di, "workspace")
    flags = 0
    if global_scale is not None:
        g.copy_(global_scale.reshape(1))
        flags = NVFP4_GLOBAL_SCALE_GIVEN
    ws_bytes = nvfp4_quantize_workspace_bytes(rows, cols)
    if workspace is None and flags == 0:
        workspace = torch.empty(max(ws_bytes, 4), dtype=torch.uint8, device=dev)
    st = nvfp4_quantize_raw(_ptr(x), _DT_IN[x.dtype], rows, cols, x.stride(0), _ptr(q), _ptr(s),
                            _ptr(g), flags, _ptr(workspace),
                            0 if workspace is None else workspace.numel() * workspace.element_size(),
                            _stream(None, di))
    _check("nvfp4_quantize", st)
    return res


def nvfp4_gemm(a, b, out_dtype: str = "bf16", y: torch.Tensor | None = None, stream=None):
    """a = (q, s, g) of x [M, K]; b = (q, s, g) of W [N, K] -> y [M, N]."""
    if type(a) is not Packed:
        a = Packed(a)
    if type(b) is not Packed:
        b = Packed(b)
    if a.lead or b.lead or a.K != b.K or a.dev != b.dev:
        raise ValueError("a and b: 2-D packed operands with the same K on one GPU")
    a_q, a_s, a_g = a
    b_q, b_s, b_g = b
    M, N, K = a.rows, b.rows, a.K
    _need(out_dtype in _DT_OUT, f"out_dtype: one of {sorted(_DT_OUT)}")
    code, tdt = _DT_OUT[out_dtype]
    if y is None:
        with _on_stream(stream, a.dev):
            y = torch.empty((M, N), dtype=tdt, device=a_q.device)
    ld_y = _out(y, M, N, tdt, a.dev)
    st = nvfp4_gemm_raw(M, N, K, a_q.data_ptr(), a_s.data_ptr(), a_g.data_ptr(), b_q.data_ptr(),
                        b_s.data_ptr(), b_g.data_ptr(), y.data_ptr(), code, ld_y,
                        _stream(stream, a.dev))
    _check("nvfp4_gemm", st)
    return y


def nvfp4_gemm_nvfp4_out(a, b, y_g: torch.Tensor, out=None, stream=None):
    """a = (q, s, g) of x [M, K], b = (q, s, g) of W [N, K]; y_g = the output's
    static global scale (fp32 [1], GPU) -> (q [M, N/2], s [M, N/16], y_g): y
    quantised in the GEMM's epilogue.  ``out`` = (q, s) reuses buffers."""
    a, b = _packed(a), _packed(b)
    _need(not a.lead and not b.lead and a.K == b.K and a.dev == b.dev,
          "a and b: 2-D packed operands with the same K on one GPU")
    a_q, a_s, a_g = a
    b_q, b_s, b_g = b
    M, N, K = a.rows, b.rows, a.K
    _need(N % 16 == 0, "the output's columns (rows of b) must be a multiple of 16")
    if out is None:
        with _on_stream(stream, a.dev):
            q = torch.empty((M, N // 2), dtype=torch.uint8, device=a_q.device)
            s = torch.empty((M, N // 16), dtype=torch.uint8, device=a_q.device)
    else:
        q, s = out
    o = Packed((q, s, y_g))
    _need(not o.lead and o.rows == M and o.K == N and o.dev == a.dev,
          f"out: must pack the output [{M}, {N}] on the operands' GPU")
    st = nvfp4_gemm_nvfp4_out_raw(M, N, K, _ptr(a_q), _ptr(a_s), _ptr(a_g), _ptr(b_q),
                                  _ptr(b_s), _ptr(b_g), _ptr(q), _ptr(s), _ptr(y_g),
                                  _stream(stream, a.dev))
    _check("nvfp4_gemm_nvfp4_out", st)
    return q, s, y_g


def _grouped_problem(m_offsets, total_m, a, b, out_dtype, y, stream, row_index):
    """Checks one grouped call's tensors; returns (GroupedProblem, y, dev)."""
    a, b = _packed(a), _packed(b)
    _need(len(b.lead) == 1 and not a.lead and a.K == b.K and a.dev == b.dev,
          "b: [G, N, K/2] packed experts and a: packed rows with the same K, on one GPU")
    _need(row_index is not None or a.rows == total_m, "a: total_m rows (or give row_index)")
    a_q, a_s, a_g = a
    b_q, b_s, b_g = b
    G, N, K = b.lead[0], b.rows, b.K
    _need(m_offsets.dtype == torch.int32 and m_offsets.numel() == G + 1
          and m_offsets.is_contiguous(), "m_offsets: G + 1 contiguous int32")
    _on_dev(m_offsets, b.dev, "m_offsets")
    _need(out_dtype in _DT_OUT, f"out_dtype: one of {sorted(_DT_OUT)}")
    code, tdt = _DT_OUT[out_dtype]
    if y is None:
        with _on_stream(stream, b.dev):
            y = torch.empty((total_m, N), dtype=tdt, device=b_q.device)
    ld_y = _out(y, total_m, N, tdt, b.dev)
    a_rows = 0
    if row_index is not None:
        _need(row_index.dtype == torch.int32 and row_index.numel() == total_m
              and row_index.is_contiguous(), "row_index: total_m contiguous int32")
        _on_dev(row_index, b.dev, "row_index")
        a_rows = a_q.shape[0]
    prob = GroupedProblem(G, _ptr(m_offsets), _ptr(row_index) if row_index is not None else None,
                          total_m, a_rows, N, K, _ptr(a_q), _ptr(a_s), _ptr(a_g), _ptr(b_q),
                          _ptr(b_s), _ptr(b_g), _ptr(y), code, ld_y)
    return prob, y, b.dev


def nvfp4_grouped_gemm(m_offsets: torch.Tensor, total_m: int, a, b, out_dtype: str = "bf16",
                       y: torch.Tensor | None = None, stream=None,
                       row_index: torch.Tensor | None = None):
    """m_offsets int32 [G+1] (GPU); a = (q [total_m, K/2], s, g [1]);
    b = (q [G, N, K/2], s [G, N, K/16], g [G]) -> y [total_m, N].
    With row_index (int32 [total_m], GPU), grouped row r reads row
    row_index[r] of a = (q [a_rows, K/2], s, g) instead (no gathered copy)."""
    p, y, dev = _grouped_problem(m_offsets, total_m, a, b, out_dtype, y, stream, row_index)
    stream = _stream(stream, dev)
    if row_index is None:
        st = nvfp4_grouped_gemm_raw(p.G, p.m_offsets, total_m, p.N, p.K, p.a_q, p.a_s, p.a_g,
                                    p.b_q, p.b_s, p.b_g, p.y, p.y_dtype, p.ld_y, stream)
        _check("nvfp4_grouped_gemm", st)
        return y
    st = nvfp4_grouped_gemm_gather_raw(p.G, p.m_offsets, p.row_index, total_m, p.a_rows, p.N,
                                       p.K, p.a_q, p.a_s, p.a_g, p.b_q, p.b_s, p.b_g, p.y,
                                       p.y_dtype, p.ld_y, stream)
    _check("nvfp4_grouped_gemm_gather", st)
    return y


def nvfp4_grouped_gemm_multi_raw(problems, stream=None) -> int:
    """problems: a sequence of GroupedProblem (host structures)."""
    arr = (GroupedProblem * max(len(problems), 1))(*problems)
    return load().nvfp4_grouped_gemm_multi(len(problems), arr, _stream(stream))


def nvfp4_grouped_gemm_multi(calls, stream=None):
    """Several grouped GEMMs in one launch.  `calls` is a sequence (at most
    NVFP4_GROUPED_MAX_PROBLEMS) of dicts holding nvfp4_grouped_gemm's
    arguments (m_offsets, total_m, a, b and optionally out_dtype, y,
    row_index); returns their outputs, equal bit for bit to those of the
    separate calls."""
    _need(len(calls) <= NVFP4_GROUPED_MAX_PROBLEMS,
          f"at most {NVFP4_GROUPED_MAX_PROBLEMS} grouped problems per launch")
    probs, ys, devs = [], [], set()
    for c in calls:
        p, y, dev = _grouped_problem(c["m_offsets"], c["total_m"], c["a"], c["b"],
                                     c.get("out_dtype", "bf16"), c.get("y"), stream,
                                     c.get("row_index"))
        probs.append(p)
        ys.append(y)
        devs.add(dev)
    if not probs:
        return ys
    _need(len(devs) == 1, "all problems on one GPU")
    st = nvfp4_grouped_gemm_multi_raw(probs, _stream(stream, devs.pop()))
    _check("nvfp4_grouped_gemm_multi", st)
    return ys


# --------------------------------------------------------------------------
# MXFP4 variant (32-element blocks, E8M0 scales, no per-tensor scale)
# --------------------------------------------------------------------------

def nvfp4_mxfp4_quantize_raw(x, x_dtype, rows, cols, ld_x, q, s, stream=None) -> int:
    return load().nvfp4_mxfp4_quantize(x, x_dtype, rows, cols, ld_x, q, s, _stream(stream))


def nvfp4_mxfp4_gemm_raw(M, N, K, a_q, a_s, b_q, b_s, y, y_dtype, ld_y, stream=None) -> int:
    return load().nvfp4_mxfp4_gemm(M, N, K, a_q, a_s, b_q, b_s, y, y_dtype, ld_y,
                                   _stream(stream))


def _mx_operand(t2, what: str):
    """(q uint8 [rows, K/2], s uint8 [rows, K/32]) on one GPU -> (rows, K, dev)."""
    q, s = t2
    _need(q.dim() == 2 and q.dtype == torch.uint8 and s.dtype == torch.uint8,
          f"{what}: q and s must be 2-D uint8")
    rows, K = q.shape[0], q.shape[1] * 2
    _need(tuple(s.shape) == (rows, K // 32) and K % 32 == 0,
          f"{what}: q {tuple(q.shape)} and s {tuple(s.shape)} do not pack [{rows}, {K}] in blocks of 32")
    _need(q.is_contiguous() and s.is_contiguous(), f"{what}: q and s must be contiguous")
    _need(q.is_cuda and s.get_device() == q.get_device(), f"{what}: q and s must be on one GPU")
    return rows, K, q.get_device()


def nvfp4_mxfp4_quantize(x: torch.Tensor, out=None, stream=None):
    """x [rows, cols] fp32/bf16 on the GPU (cols % 32 == 0) -> (q uint8
    [rows, cols/2], s uint8 [rows, cols/32]) in MXFP4; ``out`` reuses
    buffers."""
    _need(x.dim() == 2 and x.dtype in _DT_IN, "x: 2-D fp32 or bf16")
    _need(x.stride(1) == 1 or x.shape[1] <= 1, "x: rows must have unit column stride")
    _need(x.is_cuda, "x: must be on a GPU")
    rows, cols = x.shape
    _need(cols % 32 == 0, "x: columns must be a multiple of 32")
    di = x.get_device()
    with _on_stream(stream, di):
        if out is None:
            q = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
            s = torch.empty((rows, cols // 32), dtype=torch.uint8, device=x.device)
        else:
            q, s = out
            r, K, dev = _mx_operand((q, s), "out")
            _need(r == rows and K == cols and dev == di, f"out: does not pack x [{rows}, {cols}] on its GPU")
        st = nvfp4_mxfp4_quantize_raw(_ptr(x), _DT_IN[x.dtype], rows, cols, x.stride(0), _ptr(q),
                                      _ptr(s), _stream(None, di))
    _check("nvfp4_mxfp4_quantize", st)
    return q, s


def nvfp4_mxfp4_gemm(a, b, out_dtype: str = "bf16", y: torch.Tensor | None = None, stream=None):
    """a = (q, s) of x [M, K]; b = (q, s) of W [N, K], both MXFP4 -> y [M, N]
    = x . W^T."""
    M, K, da = _mx_operand(a, "a")
    N, Kb, db = _mx_operand(b, "b")
    _need(K == Kb and da == db, "a and b: the same K, on one GPU")
    _need(out_dtype in _DT_OUT, f"out_dtype: one of {sorted(_DT_OUT)}")
    code, tdt = _DT_OUT[out_dtype]
    with _on_stream(stream, da):
        if y is None:
            y = torch.empty((M, N), dtype=tdt, device=a[0].device)
        ld_y = _out(y, M, N, tdt, da)
        st = nvfp4_mxfp4_gemm_raw(M, N, K, _ptr(a[0]), _ptr(a[1]), _ptr(b[0]), _ptr(b[1]), _ptr(y),
                                  code, ld_y, _stream(None, da))
    _check("nvfp4_mxfp4_gemm", st)
    return y


# --------------------------------------------------------------------------
# FP8 operands (E4M3 bytes, one fp32 scale per 128 elements of a row or per
# 128 x 128 block)
# --------------------------------------------------------------------------

_F8 = torch.float8_e4m3fn


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


@contextlib.contextmanager
def _there(stream, dev: int):
    """Context for a call on another stream than the current one, or on
    another GPU than the current one."""
    with torch.cuda.device(dev), _on_stream(stream, dev):
        yield


def _here(stream, dev: int) -> bool:
    """Whether a call runs on the current stream of the current GPU and needs
    no context (the usual case, kept cheap: a context costs about as much as
    a launch)."""
    return stream is None and _current_device() == dev


def _stride(t, cols: int, what: str) -> int:
    """Row stride of a 2-D tensor whose rows must be contiguous (a single
    row's stride says nothing, so its length stands in; neither do those of a
    tensor without elements, which passes whatever its order)."""
    _need(t.stride(-1) == 1 or cols <= 1 or t.numel() == 0, f"{what}: rows must have unit column stride")
    return t.stride(-2) if t.shape[-2] > 1 else cols


class Fp8Packed(tuple):
    """(q, s) of an FP8 operand [rows, K], or of G of them [G, rows, K]:
    float8_e4m3fn q and fp32 s [.., ceil(K/128), ceil(rows/block_rows)], both
    contiguous, on one GPU; block_rows is 1 or 128, told by s's shape.
    Checked when made; nvfp4_fp8_quantize returns one."""

    def __new__(cls, ts, _trusted=None):
        q, s = ts
        self = super().__new__(cls, (q, s))
        if _trusted is not None:
            self.lead, self.rows, self.K, self.block_rows, self.dev = _trusted
            return self
        shape, s_shape = tuple(q.shape), tuple(s.shape)
        _need(q.dtype == _F8 and s.dtype == torch.float32, "q must be float8_e4m3fn and s fp32")
        _need(2 <= len(shape) <= 3 and len(s_shape) == len(shape),
              "q and s: 2-D, or 3-D with one per matrix")
        rows, K = shape[-2:]
        n = s_shape[-1]
        if K % 16 != 0 or s_shape[:-1] != (*shape[:-2], -(-K // 128)) or n not in (rows, -(-rows // 128)):
            raise ValueError(f"q {shape} and s {s_shape} do not belong together (K % 16 == 0, "
                             "s [.., ceil(K/128), rows or ceil(rows/128)])")
        _need(q.is_contiguous() and s.is_contiguous(), "q and s must be contiguous")
        dev = q.get_device()
        _need(q.is_cuda and s.get_device() == dev, "q and s must be on one GPU")
        self.lead, self.rows, self.K, self.dev = shape[:-2], rows, K, dev
        self.block_rows = 1 if n == rows else 128
        return self


def _fp8(t2) -> Fp8Packed:
    return t2 if type(t2) is Fp8Packed else Fp8Packed(t2)


def nvfp4_fp8_quantize_raw(x, x_dtype, batch, rows, cols, ld_x, block_rows, q, s, qt, st,
                           stream=None) -> int:
    return load().nvfp4_fp8_quantize(x, x_dtype, batch, rows, cols, ld_x, block_rows, q, s, qt, st,
                                     _stream(stream))


def nvfp4_fp8_grouped_columns(total_m: int, G: int) -> int:
    return int(load().nvfp4_fp8_grouped_columns(total_m, G))


def nvfp4_fp8_grouped_quantize_raw(x, x_dtype, G, m_offsets, row_index, total_m, x_rows, cols, ld_x,
                                   q, s, qt, st, stream=None) -> int:
    return load().nvfp4_fp8_grouped_quantize(x, x_dtype, G, m_offsets, row_index, total_m, x_rows,
                                             cols, ld_x, q, s, qt, st, _stream(stream))


def nvfp4_fp8_gemm_raw(M, N, K, a_q, a_s, b_q, b_s, b_block_rows, y, y_dtype, ld_y, flags,
                       stream=None) -> int:
    return load().nvfp4_fp8_gemm(M, N, K, a_q, a_s, b_q, b_s, b_block_rows, y, y_dtype, ld_y, flags,
                                 _stream(stream))


def nvfp4_fp8_grouped_gemm_raw(G, m_offsets, row_index, total_m, a_rows, N, K, a_q, a_s, b_q, b_s,
                               y, y_dtype, ld_y, stream=None) -> int:
    return load().nvfp4_fp8_grouped_gemm(G, m_offsets, row_index, total_m, a_rows, N, K, a_q, a_s,
                                         b_q, b_s, y, y_dtype, ld_y, _stream(stream))


def nvfp4_fp8_grouped_wgrad_raw(G, m_offsets, total_m, N, K, a_q, a_s, b_q, b_s, dw, dw_dtype, flags,
                                stream=None) -> int:
    return load().nvfp4_fp8_grouped_wgrad(G, m_offsets, total_m, N, K, a_q, a_s, b_q, b_s, dw,
                                          dw_dtype, flags, _stream(stream))


def _fp8_buffer(out, q_shape, s_shape, block_rows: int, x, dev: int) -> Fp8Packed:
    """The operand a quantiser writes: new, or the caller's (checked)."""
    if out is None:
        return Fp8Packed((x.new_empty(q_shape, dtype=_F8), x.new_empty(s_shape, dtype=torch.float32)),
                         _trusted=(q_shape[:-2], q_shape[-2], q_shape[-1], block_rows, dev))
    o = _fp8(out)
    if tuple(o[0].shape) != q_shape or tuple(o[1].shape) != s_shape or o.dev != dev:
        raise ValueError(f"out: expected q {q_shape} and s {s_shape} on x's GPU")
    return o


def _fp8_outs(layout: str, out):
    """The caller's (rows, transposed) buffers for a layout, None where there
    are none."""
    if layout == "rows":
        return out, None
    if layout == "cols":
        return None, out
    _need(layout == "both", "layout: 'rows', 'cols' or 'both'")
    _need(out is None or len(out) == 2, "out: one operand per layout")
    return (None, None) if out is None else out


def _fp8_ptrs(rows, cols):
    return (None if rows is None else rows[0].data_ptr(), None if rows is None else rows[1].data_ptr(),
            None if cols is None else cols[0].data_ptr(), None if cols is None else cols[1].data_ptr())


def _fp8_result(rows, cols):
    return cols if rows is None else rows if cols is None else (rows, cols)


def nvfp4_fp8_quantize(x: torch.Tensor, block_rows: int = 1, layout: str = "rows", out=None,
                       stream=None):
    """x [rows, cols] or [G, rows, cols], fp32/bf16 on the GPU (cols % 16 == 0)
    -> Fp8Packed.  layout "rows": blocks along the rows, q [.., rows, cols];
    "cols": the transposed operand, blocks along the columns, q
    [.., cols, rows rounded up to 16]; "both": the two from one read, as a
    pair.  block_rows 1 scales 1 x 128 blocks, 128 scales 128 x 128 blocks
    (weights).  ``out`` reuses buffers."""
    dt = _DT_IN.get(x.dtype)
    _need(dt is not None and x.dim() in (2, 3), "x: 2-D or 3-D, fp32 or bf16")
    _need(x.is_cuda, "x: must be on a GPU")
    _need(block_rows in (1, 128), "block_rows: 1 or 128")
    _need(x.shape[-1] % 16 == 0, "x: columns must be a multiple of 16")
    dev = x.get_device()
    if _here(stream, dev):
        return _fp8_quantize(x, dt, block_rows, layout, out, dev)
    with _there(stream, dev):
        return _fp8_quantize(x, dt, block_rows, layout, out, dev)


def _fp8_quantize(x, dt: int, block_rows: int, layout: str, out, dev: int):
    *lead, rows, cols = x.shape
    batch = lead[0] if lead else 1
    ld = _stride(x, cols, "x")
    _need(batch <= 1 or x.stride(0) == rows * ld, "x: matrices must follow each other")
    kb = -(-cols // 128)
    out_r, out_c = _fp8_outs(layout, out)
    r = c = None
    if layout != "cols":
        r = _fp8_buffer(out_r, (*lead, rows, cols), (*lead, kb, -(-rows // block_rows)), block_rows, x, dev)
    if layout != "rows":
        rows_t = -(-rows // 16) * 16
        c = _fp8_buffer(out_c, (*lead, cols, rows_t),
                        (*lead, -(-rows_t // 128), cols if block_rows == 1 else kb), block_rows, x, dev)
    st = nvfp4_fp8_quantize_raw(x.data_ptr(), dt, batch, rows, cols, ld, block_rows,
                                *_fp8_ptrs(r, c), _stream(None, dev))
    if st != NVFP4_OK:
        _check("nvfp4_fp8_quantize", st)
    return _fp8_result(r, c)


def _groups(m_offsets, dev: int, G: int | None = None) -> int:
    _need(m_offsets.dtype == torch.int32 and m_offsets.dim() == 1 and m_offsets.numel() >= 1
          and m_offsets.is_contiguous(), "m_offsets: G + 1 contiguous int32")
    _need(G is None or m_offsets.numel() == G + 1, "m_offsets: G + 1 contiguous int32")
    _on_dev(m_offsets, dev, "m_offsets")
    return m_offsets.numel() - 1


def _row_index(row_index, total_m: int, dev: int):
    if row_index is not None:
        _need(row_index.dtype == torch.int32 and row_index.numel() == total_m
              and row_index.is_contiguous(), "row_index: total_m contiguous int32")
        _on_dev(row_index, dev, "row_index")


def nvfp4_fp8_grouped_quantize(x: torch.Tensor, m_offsets: torch.Tensor, layout: str = "cols",
                               row_index: torch.Tensor | None = None, out=None, stream=None):
    """Rows sorted by group (m_offsets int32 [G+1], GPU) -> Fp8Packed with 1 x
    128 blocks.  layout "cols": the transposed operand [cols, P] of
    nvfp4_fp8_grouped_wgrad, each group's tokens starting at a multiple of
    128 (P = nvfp4_fp8_grouped_columns(total_m, G)); "rows": q [total_m, cols]
    (rows of no group stay as they were); "both" as a pair.  With row_index
    (int32 [total_m], GPU), grouped row r is x[row_index[r]]."""
    _need(x.dim() == 2 and x.dtype in _DT_IN, "x: 2-D fp32 or bf16")
    _need(x.is_cuda, "x: must be on a GPU")
    x_rows, cols = x.shape
    _need(cols % 16 == 0, "x: columns must be a multiple of 16")
    ld, dev = _stride(x, cols, "x"), x.get_device()
    G = _groups(m_offsets, dev)
    total = x_rows if row_index is None else row_index.numel()
    _row_index(row_index, total, dev)
    _need(G > 0 or total == 0, "m_offsets: no groups for the rows")
    P = nvfp4_fp8_grouped_columns(total, G)
    with contextlib.nullcontext() if _here(stream, dev) else _there(stream, dev):
        out_r, out_c = _fp8_outs(layout, out)
        r = c = None
        if layout != "cols":
            r = _fp8_buffer(out_r, (total, cols), (-(-cols // 128), total), 1, x, dev)
        if layout != "rows":
            c = _fp8_buffer(out_c, (cols, P), (P // 128, cols), 1, x, dev)
        st = nvfp4_fp8_grouped_quantize_raw(_ptr(x), _DT_IN[x.dtype], G, _ptr(m_offsets),
                                            None if row_index is None else _ptr(row_index), total,
                                            x_rows, cols, ld, *_fp8_ptrs(r, c), _stream(None, dev))
    _check("nvfp4_fp8_grouped_quantize", st)
    return _fp8_result(r, c)


def _fp8_out(y, shape, out_dtype: str, accumulate: bool, like, dev: int):
    """The output (new, or the caller's, checked), its dtype code and row stride."""
    code_dt = _DT_OUT.get(out_dtype)
    _need(code_dt is not None, "out_dtype: 'f32' or 'bf16'")
    code, tdt = code_dt
    if y is None:
        _need(not accumulate, "accumulate: needs an fp32 output to add to")
        return like.new_empty(shape, dtype=tdt), code, shape[-1]
    _need(not accumulate or code == NVFP4_F32, "accumulate: needs an fp32 output to add to")
    if y.dtype != tdt or tuple(y.shape) != shape:
        raise ValueError(f"y: {tuple(y.shape)} {y.dtype}, expected {shape} {tdt}")
    _on_dev(y, dev, "y")
    return y, code, _stride(y, shape[-1], "y")


def nvfp4_fp8_gemm(a, b, out_dtype: str = "bf16", y: torch.Tensor | None = None,
                   accumulate: bool = False, stream=None):
    """a = Fp8Packed [M, K] with block_rows 1; b = Fp8Packed [N, K] with
    block_rows 1 or 128 -> y [M, N] = a . b^T.  With accumulate the product
    is added to the fp32 ``y``.  out_dtype "f32" keeps fp32 sums throughout;
    "bf16" may cut each product 2^-16 below the largest of its block
    (include/nvfp4.h has the bound).  A linear layer y = x W^T takes x (layout
    "rows") and W (block_rows 128, "rows"); its input gradient takes dy
    ("rows") and W ("cols"); its weight gradient dy ("cols") and x ("cols")."""
    a, b = _fp8(a), _fp8(b)
    _need(not a.lead and not b.lead and a.K == b.K and a.dev == b.dev,
          "a and b: 2-D operands with the same K on one GPU")
    _need(a.block_rows == 1, "a: must have block_rows 1")
    if _here(stream, a.dev):
        return _fp8_gemm(a, b, out_dtype, y, accumulate)
    with _there(stream, a.dev):
        return _fp8_gemm(a, b, out_dtype, y, accumulate)


def _fp8_gemm(a, b, out_dtype: str, y, accumulate: bool):
    a_q, a_s = a
    b_q, b_s = b
    y, code, ld = _fp8_out(y, (a.rows, b.rows), out_dtype, accumulate, a_q, a.dev)
    st = nvfp4_fp8_gemm_raw(a.rows, b.rows, a.K, a_q.data_ptr(), a_s.data_ptr(), b_q.data_ptr(),
                            b_s.data_ptr(), b.block_rows, y.data_ptr(), code, ld,
                            NVFP4_ACCUMULATE if accumulate else 0, _stream(None, a.dev))
    if st != NVFP4_OK:
        _check("nvfp4_fp8_gemm", st)
    return y


def nvfp4_fp8_grouped_gemm(m_offsets: torch.Tensor, total_m: int, a, b, out_dtype: str = "bf16",
                           y: torch.Tensor | None = None, stream=None,
                           row_index: torch.Tensor | None = None):
    """m_offsets int32 [G+1] (GPU); a = Fp8Packed [total_m, K] (block_rows 1);
    b = Fp8Packed [G, N, K] with block_rows 128 -> y [total_m, N].  With
    row_index (int32 [total_m], GPU), grouped row r reads row row_index[r] of
    a [a_rows, K].  Rows of y of no group stay as they were."""
    a, b = _fp8(a), _fp8(b)
    _need(len(b.lead) == 1 and not a.lead and a.K == b.K and a.dev == b.dev,
          "b: [G, N, K] experts and a: [rows, K] with the same K, on one GPU")
    _need(a.block_rows == 1, "a: must have block_rows 1")
    _need(b[1].shape[-1] == -(-b.rows // 128), "b: must have block_rows 128")
    _need(row_index is not None or a.rows == total_m, "a: total_m rows (or give row_index)")
    dev = b.dev
    G = _groups(m_offsets, dev, b.lead[0])
    _row_index(row_index, total_m, dev)
    with contextlib.nullcontext() if _here(stream, dev) else _there(stream, dev):
        y, code, ld = _fp8_out(y, (total_m, b.rows), out_dtype, False, b[0], dev)
        st = nvfp4_fp8_grouped_gemm_raw(G, _ptr(m_offsets),
                                        None if row_index is None else _ptr(row_index), total_m,
                                        a.rows, b.rows, b.K, _ptr(a[0]), _ptr(a[1]), _ptr(b[0]),
                                        _ptr(b[1]), _ptr(y), code, ld, _stream(None, dev))
    _check("nvfp4_fp8_grouped_gemm", st)
    return y


def nvfp4_fp8_grouped_wgrad(m_offsets: torch.Tensor, total_m: int, a, b, out_dtype: str = "f32",
                            dw: torch.Tensor | None = None, accumulate: bool = False, stream=None):
    """Experts' weight gradients dw [G, N, K] from the transposed operands of
    nvfp4_fp8_grouped_quantize: a = dy [N, P], b = x [K, P].  With accumulate
    they are added to the fp32 ``dw``."""
    a, b = _fp8(a), _fp8(b)
    _need(not a.lead and not b.lead and a.K == b.K and a.dev == b.dev,
          "a and b: 2-D transposed operands with the same columns on one GPU")
    _need(a.block_rows == 1 and b.block_rows == 1, "a and b: must have block_rows 1")
    dev = a.dev
    G = _groups(m_offsets, dev)
    if a.K != nvfp4_fp8_grouped_columns(total_m, G):
        raise ValueError(f"a and b: {a.K} columns, expected nvfp4_fp8_grouped_columns({total_m}, {G})")
    _need(G > 0 or total_m == 0, "m_offsets: no groups for the rows")
    with contextlib.nullcontext() if _here(stream, dev) else _there(stream, dev):
        dw, code, ld = _fp8_out(dw, (G, a.rows, b.rows), out_dtype, accumulate, a[0], dev)
        _need(dw.is_contiguous(), "dw: must be contiguous")
        st = nvfp4_fp8_grouped_wgrad_raw(G, _ptr(m_offsets), total_m, a.rows, b.rows, _ptr(a[0]),
                                         _ptr(a[1]), _ptr(b[0]), _ptr(b[1]), _ptr(dw), code,
                                         NVFP4_ACCUMULATE if accumulate else 0, _stream(None, dev))
    _check("nvfp4_fp8_grouped_wgrad", st)
    return dw


# --------------------------------------------------------------------------
# expert router: top-k, counts and order, balance loss, and their gradient
# --------------------------------------------------------------------------

class MoeRoute(typing.NamedTuple):
    """What nvfp4_moe_route writes (include/nvfp4.h has each one's meaning)."""
    expert_index: torch.Tensor   # int32 [T, topk]
    weights: torch.Tensor        # fp32 [T, topk]
    counts: torch.Tensor         # int32 [E]
    m_offsets: torch.Tensor      # int32 [E + 1]
    row_index: torch.Tensor      # int32 [T * topk]
    pair_row: torch.Tensor       # int32 [T, topk]
    routed: torch.Tensor         # int32 [1]
    loss: torch.Tensor           # fp32 [1]


@functools.lru_cache(maxsize=256)
def nvfp4_moe_route_workspace_bytes(T: int, E: int) -> int:
    return int(load().nvfp4_moe_route_workspace_bytes(T, E))


def nvfp4_moe_route_raw(T, E, topk, logits, logits_dtype, ld_logits, token_mask, flags,
                        expert_index, weights, counts, m_offsets, row_index, pair_row, routed, loss,
                        workspace, workspace_bytes, stream=None) -> int:
    return load().nvfp4_moe_route(T, E, topk, logits, logits_dtype, ld_logits, token_mask, flags,
                                  expert_index, weights, counts, m_offsets, row_index, pair_row,
                                  routed, loss, workspace, workspace_bytes, _stream(stream))


def nvfp4_moe_route_backward_raw(T, E, topk, logits, logits_dtype, ld_logits, token_mask, flags,
                                 expert_index, counts, routed, d_weights, d_loss, d_logits, ld_d,
                                 stream=None) -> int:
    return load().nvfp4_moe_route_backward(T, E, topk, logits, logits_dtype, ld_logits, token_mask,
                                           flags, expert_index, counts, routed, d_weights, d_loss,
                                           d_logits, ld_d, _stream(stream))


def _logits(logits, mask):
    _need(logits.dim() == 2 and logits.dtype in _DT_IN, "logits: 2-D fp32 or bf16")
    _need(logits.is_cuda, "logits: must be on a GPU")
    T, E = logits.shape
    _need(E >= 1, "logits: at least one expert")
    dev = logits.get_device()
    if mask is not None:
        _need(mask.dtype in (torch.bool, torch.uint8) and tuple(mask.shape) == (T,)
              and mask.is_contiguous(), "mask: T contiguous bool or uint8")
        _on_dev(mask, dev, "mask")
    return T, E, _stride(logits, E, "logits"), dev


def nvfp4_moe_route(logits: torch.Tensor, topk: int, mask: torch.Tensor | None = None,
                    renormalize: bool = False, workspace: torch.Tensor | None = None,
                    stream=None) -> MoeRoute:
    """logits [T, E] fp32/bf16 (GPU) -> MoeRoute: each token's topk experts and
    weights, the expert-sorted order the grouped GEMMs take (m_offsets,
    row_index, with pair_row the row of each choice), the per-expert counts
    and the balance loss.  ``mask`` [T]: tokens at 0 are not routed.
    ``renormalize``: weights are the softmax over the chosen experts."""
    T, E, ld, dev = _logits(logits, mask)
    _need(1 <= topk <= E, "topk: 1 to the number of experts")
    if workspace is not None:
        _on_dev(workspace, dev, "workspace")
        _need(workspace.is_contiguous(), "workspace: must be contiguous")
    if _here(stream, dev):
        return _moe_route(logits, topk, mask, renormalize, workspace, T, E, ld, dev)
    with _there(stream, dev):
        return _moe_route(logits, topk, mask, renormalize, workspace, T, E, ld, dev)


def _moe_route(logits, topk: int, mask, renormalize: bool, workspace, T: int, E: int, ld: int,
               dev: int) -> MoeRoute:
    # every output is an allocation of its own: writing one in place leaves the
    # others' versions alone (a backward may have saved them), and keeping one
    # keeps no other
    like = torch.empty_like
    ei = logits.new_empty((T, topk), dtype=torch.int32)
    new, routed = ei.new_empty, ei.new_empty(1)
    r = MoeRoute(ei, like(ei, dtype=torch.float32), new(E), new(E + 1), new(T * topk), like(ei), routed,
                 like(routed, dtype=torch.float32))
    if workspace is None:
        ws_bytes = nvfp4_moe_route_workspace_bytes(T, E)
        workspace = new(-(-ws_bytes // 4))
    else:
        ws_bytes = workspace.numel() * workspace.element_size()
    st = nvfp4_moe_route_raw(T, E, topk, logits.data_ptr(), _DT_IN[logits.dtype], ld,
                             None if mask is None else mask.data_ptr(),
                             NVFP4_ROUTE_RENORMALIZE if renormalize else 0, *[t.data_ptr() for t in r],
                             workspace.data_ptr(), ws_bytes, _stream(None, dev))
    if st != NVFP4_OK:
        _check("nvfp4_moe_route", st)
    return r


def nvfp4_moe_route_backward(logits: torch.Tensor, route: MoeRoute,
                             d_weights: torch.Tensor | None = None,
                             d_loss: torch.Tensor | None = None, mask: torch.Tensor | None = None,
                             renormalize: bool = False, out: torch.Tensor | None = None, stream=None):
    """Gradient of the logits from d_weights fp32 [T, topk] and d_loss (one
    fp32 value, GPU), given what nvfp4_moe_route returned for them and the
    same mask and renormalize; ``out`` reuses a buffer of the logits' shape."""
    T, E, ld, dev = _logits(logits, mask)
    e = route.expert_index
    _need(e.dim() == 2 and e.shape[0] == T and e.dtype == torch.int32 and e.is_contiguous()
          and route.counts.dtype == torch.int32 and route.counts.numel() == E
          and route.counts.is_contiguous() and route.routed.dtype == torch.int32
          and route.routed.numel() == 1, "route: not nvfp4_moe_route's answer for these logits")
    for t in (e, route.counts, route.routed):
        _on_dev(t, dev, "route")
    topk = e.shape[1]
    if d_weights is not None:
        _need(d_weights.dtype == torch.float32 and tuple(d_weights.shape) == (T, topk)
              and d_weights.is_contiguous(), "d_weights: contiguous fp32 [T, topk]")
        _on_dev(d_weights, dev, "d_weights")
    if d_loss is not None:
        _need(d_loss.dtype == torch.float32 and d_loss.numel() == 1, "d_loss: one fp32 value")
        _on_dev(d_loss, dev, "d_loss")
    with contextlib.nullcontext() if _here(stream, dev) else _there(stream, dev):
        if out is None:
            out = logits.new_empty((T, E))
        _need(out.dtype == logits.dtype and tuple(out.shape) == (T, E), "out: the logits' dtype and shape")
        _on_dev(out, dev, "out")
        st = nvfp4_moe_route_backward_raw(T, E, topk, _ptr(logits), _DT_IN[logits.dtype], ld,
                                          None if mask is None else _ptr(mask),
                                          NVFP4_ROUTE_RENORMALIZE if renormalize else 0, _ptr(e),
                                          _ptr(route.counts), _ptr(route.routed),
                                          None if d_weights is None else _ptr(d_weights),
                                          None if d_loss is None else _ptr(d_loss), _ptr(out),
                                          _stride(out, E, "out"), _stream(None, dev))
    _check("nvfp4_moe_route_backward", st)
    return out


# --------------------------------------------------------------------------
# gated feed-forward blocks on FP8 operands
# --------------------------------------------------------------------------

_ACT = {"silu": NVFP4_SILU, "gelu": NVFP4_GELU}


def nvfp4_fp8_gated_gemm_raw(M, F, K, a_q, a_s, w_q, w_s, w_block_rows, act, h, h_dtype, ld_h, gate_up,
                             ld_gate_up, stream=None) -> int:
    return load().nvfp4_fp8_gated_gemm(M, F, K, a_q, a_s, w_q, w_s, w_block_rows, act, h, h_dtype, ld_h,
                                       gate_up, ld_gate_up, _stream(stream))


def nvfp4_fp8_grouped_gated_gemm_raw(G, m_offsets, row_index, total_m, a_rows, F, K, a_q, a_s, w_q, w_s, act,
                                     h, h_dtype, ld_h, gate_up, ld_gate_up, stream=None) -> int:
    return load().nvfp4_fp8_grouped_gated_gemm(G, m_offsets, row_index, total_m, a_rows, F, K, a_q, a_s, w_q,
                                               w_s, act, h, h_dtype, ld_h, gate_up, ld_gate_up,
                                               _stream(stream))


def nvfp4_fp8_gated_backward_raw(dh, dh_dtype, ld_dh, gate_up, gate_up_dtype, ld_gate_up, act, rows, F, q, s,
                                 qt, st, stream=None) -> int:
    return load().nvfp4_fp8_gated_backward(dh, dh_dtype, ld_dh, gate_up, gate_up_dtype, ld_gate_up, act, rows,
                                           F, q, s, qt, st, _stream(stream))


def nvfp4_fp8_grouped_gated_backward_raw(G, m_offsets, dh, dh_dtype, ld_dh, gate_up, gate_up_dtype, ld_gate_up,
                                         act, total_m, F, q, s, qt, st, stream=None) -> int:
    return load().nvfp4_fp8_grouped_gated_backward(G, m_offsets, dh, dh_dtype, ld_dh, gate_up, gate_up_dtype,
                                                   ld_gate_up, act, total_m, F, q, s, qt, st, _stream(stream))


def _act(act: str) -> int:
    code = _ACT.get(act)
    _need(code is not None, "act: 'silu' or 'gelu'")
    return code


def _gate_up(gate_up, rows: int, F: int, like, dev: int):
    """The kept products' buffer and row stride (None, 0: not wanted)."""
    if gate_up is None or gate_up is False:
        return None, 0
    if gate_up is True:
        return like.new_empty((rows, 2 * F), dtype=torch.bfloat16), 2 * F
    _need(gate_up.dtype == torch.bfloat16 and tuple(gate_up.shape) == (rows, 2 * F),
          f"gate_up: expected bf16 ({rows}, {2 * F})")
    _on_dev(gate_up, dev, "gate_up")
    return gate_up, _stride(gate_up, 2 * F, "gate_up")


def nvfp4_fp8_gated_gemm(a, w, act: str = "silu", out_dtype: str = "bf16", h: torch.Tensor | None = None,
                         gate_up=None, stream=None):
    """a = Fp8Packed [M, K] with block_rows 1; w = Fp8Packed [2F, K] (gate rows,
    then up rows) with block_rows 1 or 128 -> h [M, F] = act(a . Wg^T) * (a .
    Wu^T), act "silu" or "gelu" (tanh form).  gate_up: True, or a bf16 [M, 2F]
    buffer, keeps the two products for nvfp4_fp8_gated_backward; the answer is
    then (h, gate_up).  ``h`` reuses a buffer of out_dtype, whose sums are as
    nvfp4_fp8_gemm's."""
    a, w = _fp8(a), _fp8(w)
    _need(not a.lead and not w.lead and a.K == w.K and a.dev == w.dev,
          "a and w: 2-D operands with the same K on one GPU")
    _need(a.block_rows == 1, "a: must have block_rows 1")
    _need(w.rows % 2 == 0, "w: an even number of rows, the gate's and the up projection's")
    if _here(stream, a.dev):
        return _fp8_gated_gemm(a, w, _act(act), out_dtype, h, gate_up)
    with _there(stream, a.dev):
        return _fp8_gated_gemm(a, w, _act(act), out_dtype, h, gate_up)


def _fp8_gated_gemm(a, w, act: int, out_dtype: str, h, gate_up):
    F = w.rows // 2
    h, code, ld = _fp8_out(h, (a.rows, F), out_dtype, False, a[0], a.dev)
    kept, ld2 = _gate_up(gate_up, a.rows, F, h, a.dev)
    st = nvfp4_fp8_gated_gemm_raw(a.rows, F, a.K, a[0].data_ptr(), a[1].data_ptr(), w[0].data_ptr(),
                                  w[1].data_ptr(), w.block_rows, act, h.data_ptr(), code, ld, _ptr(kept), ld2,
                                  _stream(None, a.dev))
    if st != NVFP4_OK:
        _check("nvfp4_fp8_gated_gemm", st)
    return h if kept is None else (h, kept)


def nvfp4_fp8_grouped_gated_gemm(m_offsets: torch.Tensor, total_m: int, a, w, act: str = "silu",
                                 out_dtype: str = "bf16", h: torch.Tensor | None = None, gate_up=None,
                                 stream=None, row_index: torch.Tensor | None = None):
    """nvfp4_fp8_gated_gemm of experts: m_offsets int32 [G+1] (GPU), a =
    Fp8Packed [total_m, K] (or with row_index [a_rows, K]), w = Fp8Packed
    [G, 2F, K] with block_rows 128 -> h [total_m, F], or (h, gate_up).  Rows of
    no group stay as they were."""
    a, w = _fp8(a), _fp8(w)
    _need(len(w.lead) == 1 and not a.lead and a.K == w.K and a.dev == w.dev,
          "w: [G, 2F, K] experts and a: [rows, K] with the same K, on one GPU")
    _need(a.block_rows == 1, "a: must have block_rows 1")
    _need(w.rows % 2 == 0, "w: an even number of rows, the gate's and the up projection's")
    _need(w[1].shape[-1] == -(-w.rows // 128), "w: must have block_rows 128")
    _need(row_index is not None or a.rows == total_m, "a: total_m rows (or give row_index)")
    dev, F, code_act = w.dev, w.rows // 2, _act(act)
    G = _groups(m_offsets, dev, w.lead[0])
    _row_index(row_index, total_m, dev)
    with contextlib.nullcontext() if _here(stream, dev) else _there(stream, dev):
        h, code, ld = _fp8_out(h, (total_m, F), out_dtype, False, w[0], dev)
        kept, ld2 = _gate_up(gate_up, total_m, F, h, dev)
        st = nvfp4_fp8_grouped_gated_gemm_raw(G, _ptr(m_offsets), _ptr(row_index), total_m, a.rows, F, w.K,
                                              _ptr(a[0]), _ptr(a[1]), _ptr(w[0]), _ptr(w[1]), code_act, _ptr(h),
                                              code, ld, _ptr(kept), ld2, _stream(None, dev))
    _check("nvfp4_fp8_grouped_gated_gemm", st)
    return h if kept is None else (h, kept)


def _gated_inputs(dh, gate_up):
    _need(dh.dim() == 2 and dh.dtype in _DT_IN and dh.is_cuda, "dh: 2-D fp32 or bf16 on a GPU")
    rows, F = dh.shape
    _need(F % 8 == 0, "dh: columns must be a multiple of 8")
    if gate_up.dtype not in _DT_IN or gate_up.shape != (rows, 2 * F):
        raise ValueError(f"gate_up: expected fp32 or bf16 ({rows}, {2 * F})")
    dev = dh.get_device()
    _on_dev(gate_up, dev, "gate_up")
    return rows, F, _stride(dh, F, "dh"), _stride(gate_up, 2 * F, "gate_up"), dev


def nvfp4_fp8_gated_backward(dh: torch.Tensor, gate_up: torch.Tensor, act: str = "silu", layout: str = "both",
                             out=None, stream=None):
    """Backward of h = act(g) * u: dh [M, F] and the kept products gate_up =
    [g, u] [M, 2F], fp32 or bf16 each -> [dg, du] as FP8 operands with 1 x 128
    blocks: layout "rows" (q [M, 2F], for dx = [dg, du] . W with W's "cols"
    layout), "cols" (q [2F, M rounded up to 16], for dW = [dg, du]^T . x) or
    "both" as a pair.  ``out`` reuses buffers."""
    sizes, code = _gated_inputs(dh, gate_up), _act(act)
    if _here(stream, sizes[-1]):
        return _fp8_gated_backward(dh, gate_up, code, layout, out, *sizes)
    with _there(stream, sizes[-1]):
        return _fp8_gated_backward(dh, gate_up, code, layout, out, *sizes)


def _fp8_gated_backward(dh, gate_up, act: int, layout: str, out, rows: int, F: int, ld_dh: int, ld_gu: int,
                        dev: int):
    out_r, out_c = _fp8_outs(layout, out)
    r = c = None
    if layout != "cols":
        r = _fp8_buffer(out_r, (rows, 2 * F), (-(-2 * F // 128), rows), 1, dh, dev)
    if layout != "rows":
        rows_t = -(-rows // 16) * 16
        c = _fp8_buffer(out_c, (2 * F, rows_t), (-(-rows_t // 128), 2 * F), 1, dh, dev)
    st = nvfp4_fp8_gated_backward_raw(dh.data_ptr(), _DT_IN[dh.dtype], ld_dh, gate_up.data_ptr(),
                                      _DT_IN[gate_up.dtype], ld_gu, act, rows, F, *_fp8_ptrs(r, c),
                                      _stream(None, dev))
    if st != NVFP4_OK:
        _check("nvfp4_fp8_gated_backward", st)
    return _fp8_result(r, c)


def nvfp4_fp8_grouped_gated_backward(dh: torch.Tensor, gate_up: torch.Tensor, m_offsets: torch.Tensor,
                                     act: str = "silu", layout: str = "both", out=None, stream=None):
    """nvfp4_fp8_gated_backward of rows sorted by group (m_offsets int32 [G+1],
    GPU): layouts as nvfp4_fp8_grouped_quantize's for 2F columns, "rows" for
    nvfp4_fp8_grouped_gemm and "cols" for nvfp4_fp8_grouped_wgrad."""
    total, F, ld_dh, ld_gu, dev = _gated_inputs(dh, gate_up)
    code, G = _act(act), _groups(m_offsets, dev)
    _need(G > 0 or total == 0, "m_offsets: no groups for the rows")
    P = nvfp4_fp8_grouped_columns(total, G)
    with contextlib.nullcontext() if _here(stream, dev) else _there(stream, dev):
        out_r, out_c = _fp8_outs(layout, out)
        r = c = None
        if layout != "cols":
            r = _fp8_buffer(out_r, (total, 2 * F), (-(-2 * F // 128), total), 1, dh, dev)
        if layout != "rows":
            c = _fp8_buffer(out_c, (2 * F, P), (P // 128, 2 * F), 1, dh, dev)
        st = nvfp4_fp8_grouped_gated_backward_raw(G, _ptr(m_offsets), _ptr(dh), _DT_IN[dh.dtype], ld_dh,
                                                  _ptr(gate_up), _DT_IN[gate_up.dtype], ld_gu, code, total, F,
                                                  *_fp8_ptrs(r, c), _stream(None, dev))
    _check("nvfp4_fp8_grouped_gated_backward", st)
    return _fp8_result(r, c)


# --------------------------------------------------------------------------
# INT8 operands (8-bit integers, one fp32 scale per row)
# --------------------------------------------------------------------------

class Int8Packed(tuple):
    """(q, s) of an INT8 operand [rows, K]: int8 q and fp32 s [rows], both
    contiguous, on one GPU.  Checked when made; nvfp4_int8_quantize returns
    one."""

    def __new__(cls, ts, _trusted=None):
        q, s = ts
        self = super().__new__(cls, (q, s))
        if _trusted is not None:
            self.rows, self.K, self.dev = _trusted
            return self
        _need(q.dtype == torch.int8 and s.dtype == torch.float32, "q must be int8 and s fp32")
        shape = tuple(q.shape)
        _need(len(shape) == 2 and shape[1] % 16 == 0 and tuple(s.shape) == shape[:1],
              f"q {shape} and s {tuple(s.shape)} do not belong together (q [rows, K] with K % 16 == 0, s [rows])")
        _need(q.is_contiguous() and s.is_contiguous(), "q and s must be contiguous")
        dev = q.get_device()
        _need(q.is_cuda and s.get_device() == dev, "q and s must be on one GPU")
        self.rows, self.K, self.dev = *shape, dev
        return self


def _int8(t2) -> Int8Packed:
    return t2 if type(t2) is Int8Packed else Int8Packed(t2)


def nvfp4_int8_quantize_raw(x, x_dtype, rows, cols, ld_x, q, s, stream=None) -> int:
    return load().nvfp4_int8_quantize(x, x_dtype, rows, cols, ld_x, q, s, _stream(stream))


def nvfp4_int8_gemm_raw(M, N, K, a_q, a_s, b_q, b_s, y, y_dtype, ld_y, stream=None) -> int:
    return load().nvfp4_int8_gemm(M, N, K, a_q, a_s, b_q, b_s, y, y_dtype, ld_y, _stream(stream))


def nvfp4_int8_quantize(x: torch.Tensor, out=None, stream=None) -> Int8Packed:
    """x [rows, cols], fp32/bf16 on the GPU (cols % 16 == 0) -> Int8Packed with a
    scale per row: of activations a scale per token, of a weight [N, K] one per
    output channel.  ``out`` reuses buffers."""
    dt = _DT_IN.get(x.dtype)
    _need(dt is not None and x.dim() == 2, "x: 2-D fp32 or bf16")
    _need(x.is_cuda, "x: must be on a GPU")
    _need(x.shape[1] % 16 == 0, "x: columns must be a multiple of 16")
    dev = x.get_device()
    if _here(stream, dev):
        return _int8_quantize(x, dt, out, dev)
    with _there(stream, dev):
        return _int8_quantize(x, dt, out, dev)


def _int8_quantize(x, dt: int, out, dev: int) -> Int8Packed:
    rows, cols = x.shape
    ld = _stride(x, cols, "x")
    if out is None:
        out = Int8Packed((x.new_empty((rows, cols), dtype=torch.int8), x.new_empty(rows, dtype=torch.float32)),
                         _trusted=(rows, cols, dev))
    else:
        out = _int8(out)
        if (out.rows, out.K, out.dev) != (rows, cols, dev):
            raise ValueError(f"out: expected q ({rows}, {cols}) and s ({rows},) on x's GPU")
    st = nvfp4_int8_quantize_raw(x.data_ptr(), dt, rows, cols, ld, out[0].data_ptr(), out[1].data_ptr(),
                                 _stream(None, dev))
    if st != NVFP4_OK:
        _check("nvfp4_int8_quantize", st)
    return out


def nvfp4_int8_gemm(a, b, out_dtype: str = "bf16", y: torch.Tensor | None = None, stream=None):
    """a = Int8Packed [M, K], b = Int8Packed [N, K] -> y [M, N] = a . b^T in fp32
    or bf16; the sums are exact integers.  ``y`` reuses a buffer."""
    a, b = _int8(a), _int8(b)
    _need(a.K == b.K and a.dev == b.dev, "a and b: operands with the same K on one GPU")
    if _here(stream, a.dev):
        return _int8_gemm(a, b, out_dtype, y)
    with _there(stream, a.dev):
        return _int8_gemm(a, b, out_dtype, y)


def _int8_gemm(a, b, out_dtype: str, y):
    y, code, ld = _fp8_out(y, (a.rows, b.rows), out_dtype, False, a[0], a.dev)
    st = nvfp4_int8_gemm_raw(a.rows, b.rows, a.K, a[0].data_ptr(), a[1].data_ptr(), b[0].data_ptr(),
                             b[1].data_ptr(), y.data_ptr(), code, ld, _stream(None, a.dev))
    if st != NVFP4_OK:
        _check("nvfp4_int8_gemm", st)
    return y


# --------------------------------------------------------------------------
# gradient norm and clipping over a list of tensors
# --------------------------------------------------------------------------

def nvfp4_grad_workspace_bytes(count: int) -> int:
    return int(load().nvfp4_grad_workspace_bytes(count))


def nvfp4_grad_norm_sq_raw(count, grads, norm_sq, workspace, workspace_bytes, stream=None) -> int:
    return load().nvfp4_grad_norm_sq(count, grads, norm_sq, workspace, workspace_bytes, _stream(stream))


def nvfp4_clip_grads_raw(count, grads, max_norm, norm_sq, norm, workspace, workspace_bytes, stream=None) -> int:
    return load().nvfp4_clip_grads(count, grads, max_norm, norm_sq, norm, workspace, workspace_bytes,
                                   _stream(stream))


def _grad_types(ts, dev: int, what: str):
    types = [_DT_IN.get(t.dtype) for t in ts]
    _need(None not in types and set(map(torch.Tensor.get_device, ts)) == {dev}
          and all(map(torch.Tensor.is_contiguous, ts)), f"{what}: contiguous fp32 or bf16 tensors on one GPU")
    return types


def _grad_list(grads, out):
    """The list as an array of nvfp4_grad (four 64-bit words each: g, out, n and
    the two types), its length and its GPU.  Whole passes over the list, since a
    model has hundreds of tensors and a Python step for each would cost more
    than the kernels."""
    dev = grads[0].get_device()
    _need(dev >= 0, "grads: must be on a GPU")
    types, sizes = _grad_types(grads, dev, "grads"), array.array("q", map(torch.Tensor.numel, grads))
    words = array.array("q", bytes(32 * len(sizes)))
    words[0::4] = array.array("q", map(torch.Tensor.data_ptr, grads))
    words[2::4] = sizes
    if out is not None:
        out_types = _grad_types(out, dev, "out")
        _need(array.array("q", map(torch.Tensor.numel, out)) == sizes, "out: must have the gradients' sizes")
        words[1::4] = array.array("q", map(torch.Tensor.data_ptr, out))
    else:
        out_types = types
    words[3::4] = array.array("q", [a | b << 32 for a, b in zip(types, out_types)])
    return words, len(sizes), dev


def _grad_workspace(workspace, count: int, like, dev: int):
    need = nvfp4_grad_workspace_bytes(count)
    if workspace is None:
        return like.new_empty(need // 8, dtype=torch.float64), need
    _on_dev(workspace, dev, "workspace")
    _need(workspace.is_contiguous(), "workspace: must be contiguous")
    return workspace, workspace.numel() * workspace.element_size()


def nvfp4_grad_norm_sq(grads, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Sum of the squares of all elements of a list of gradients (contiguous,
    fp32 or bf16, one GPU) -> fp64 [1].  Where gradients are spread over
    processes, all-reduce it and give the sum to nvfp4_clip_grads."""
    _need(len(grads) > 0, "grads: at least one tensor")
    words, count, dev = _grad_list(grads, None)
    with contextlib.nullcontext() if _here(stream, dev) else _there(stream, dev):
        ws, ws_bytes = _grad_workspace(workspace, count, grads[0], dev)
        n2 = grads[0].new_empty(1, dtype=torch.float64)
        st = nvfp4_grad_norm_sq_raw(count, words.buffer_info()[0], n2.data_ptr(), ws.data_ptr(), ws_bytes,
                                    _stream(None, dev))
    _check("nvfp4_grad_norm_sq", st)
    return n2


def nvfp4_clip_grads(grads, max_norm: float, norm_sq: torch.Tensor | None = None, out=None,
                     workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Scales a list of gradients (contiguous, fp32 or bf16, one GPU) so that
    their common norm is at most max_norm, in place or into the list ``out``
    (fp32 or bf16), and returns the norm before that, fp32 [1].  ``norm_sq``
    (fp64 [1], GPU): the squared norm, where it is known already.  A norm that
    is not finite leaves the values as they are."""
    _need(len(grads) > 0, "grads: at least one tensor")
    _need(out is None or len(out) == len(grads), "out: one tensor per gradient")
    _need(max_norm >= 0, "max_norm: must be at least 0")
    words, count, dev = _grad_list(grads, out)
    if norm_sq is not None:
        _need(norm_sq.dtype == torch.float64 and norm_sq.numel() == 1, "norm_sq: one fp64 value")
        _on_dev(norm_sq, dev, "norm_sq")
    with contextlib.nullcontext() if _here(stream, dev) else _there(stream, dev):
        ws, ws_bytes = (None, 0) if norm_sq is not None else _grad_workspace(workspace, count, grads[0], dev)
        norm = grads[0].new_empty(1, dtype=torch.float32)
        st = nvfp4_clip_grads_raw(count, words.buffer_info()[0], max_norm, _ptr(norm_sq), norm.data_ptr(),
                                  _ptr(ws), ws_bytes, _stream(None, dev))
    if st != NVFP4_OK:
        _check("nvfp4_clip_grads", st)
    return norm
