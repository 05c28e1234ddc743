"""Python binding of libwq.so, the GB300 W4A16 dequantise-GEMM library.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in include/wq.h.  There is no CPU path --
if the compiled library is missing, every call raises.

Low level (same names as the C ABI, integer pointers):
    wq_gemm, wq_gemm_ex, wq_dequant, wq_get_device_error, wq_selftest_timeout,
    wq_status_string, wq_version
Tensor level (torch CUDA tensors, raises WQError on a non-OK status):
    gemm(A, packed, scales, zeros, fmt, group=None, out_dtype="bf16", ...)
    dequant(packed, scales, zeros, fmt, group=None, out=None, ...)
    quantize(x, fmt, ...), fp4_operand(packed, scales, fmt, ...), gemm_fp4(A, B, ...),
    block_norm(x, weight, branch=..., ...): 4-bit activations
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libwq.so")

# constants of include/wq.h
WQ_NVFP4, WQ_MXFP4, WQ_INT4 = 0, 1, 2
WQ_OUT_F32 = 0x100
WQ_PATH_AUTO, WQ_PATH_GEMV, WQ_PATH_TC = 0, 1, 2
WQ_LAUNCH_OVERLAP = 0x100
WQ_LAUNCH_INPUTS_READY = 0x200
WQ_TYPE_BF16, WQ_TYPE_F32 = 0, 1
WQ_SCALES_ROWS, WQ_SCALES_TILED = 0, 1
WQ_NORM_RMS, WQ_NORM_LAYER = 0, 1
WQ_NORM_OUT_NONE, WQ_NORM_OUT_BF16, WQ_NORM_OUT_F32, WQ_NORM_OUT_NVFP4, WQ_NORM_OUT_MXFP4 = 0, 1, 2, 3, 4
WQ_OK = 0
WQ_ERR_INVALID_ARG = -1
WQ_ERR_UNSUPPORTED = -2
WQ_ERR_ALIGN = -3
WQ_ERR_CUDA = -4
WQ_ERR_DEVICE_TIMEOUT = -5

FORMATS = {"nvfp4": WQ_NVFP4, "mxfp4": WQ_MXFP4, "int4": WQ_INT4}
DEFAULT_GROUP = {"nvfp4": 16, "mxfp4": 32, "int4": 128}
LAYOUTS = {"rows": WQ_SCALES_ROWS, "tiled": WQ_SCALES_TILED}
NORM_KINDS = {"rms": WQ_NORM_RMS, "layer": WQ_NORM_LAYER}
PATHS = {"auto": WQ_PATH_AUTO, "gemv": WQ_PATH_GEMV, "tc": WQ_PATH_TC}

#: the C entry points include/wq.h declares: name -> (restype, argtypes)
_vp, _i = ctypes.c_void_p, ctypes.c_int
class wq_epilogue(ctypes.Structure):
    """The C struct of include/wq.h: bias, residual (device pointers or None), gated."""
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("gated", ctypes.c_int)]


class wq_fp4_quant(ctypes.Structure):
    """The C struct of include/wq.h: what wq_fp4_quantize reads and writes."""
    _fields_ = [("x", _vp), ("ldx", ctypes.c_longlong), ("x_type", _i), ("rows", _i), ("K", _i), ("format", _i),
                ("layout", _i), ("tensor_scale", _vp), ("packed", _vp), ("scales", _vp), ("values", _vp)]


class wq_fp4_gemm(ctypes.Structure):
    """The C struct of include/wq.h: what wq_gemm_fp4 reads and writes."""
    _fields_ = [("a_packed", _vp), ("a_scales", _vp), ("a_tensor_scale", _vp), ("b_packed", _vp), ("b_scales", _vp),
                ("b_tensor_scale", _vp), ("C", _vp), ("M", _i), ("N", _i), ("K", _i), ("format", _i),
                ("epilogue", wq_epilogue), ("path", _i)]


class wq_norm(ctypes.Structure):
    """The C struct of include/wq.h: what wq_block_norm reads and writes."""
    _fields_ = [("rows", _i), ("d", _i), ("kind", _i), ("post", _i), ("x", _vp), ("ldx", ctypes.c_longlong),
                ("x_type", _i), ("branch_type", _i), ("branch", _vp), ("ldb", ctypes.c_longlong), ("gate", _vp),
                ("gate_rows", _i), ("eps", ctypes.c_float), ("residual_scale", ctypes.c_float),
                ("branch_scale", ctypes.c_float), ("weight", _vp), ("bias", _vp), ("post_weight", _vp),
                ("post_bias", _vp), ("x_out", _vp), ("ldxo", ctypes.c_longlong), ("out", _vp),
                ("ldo", ctypes.c_longlong), ("out_type", _i), ("out_scale_layout", _i), ("out_scales", _vp),
                ("out_tensor_scale", _vp)]


SIGNATURES = {
    "wq_gemm": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i]),
    "wq_gemm_ex": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _i]),
    "wq_gemm_ws": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, ctypes.c_size_t, _vp, _i]),
    "wq_gemm_workspace_size": (ctypes.c_size_t, [_i, _i, _i, _i, _i]),
    "wq_workspace_bytes": (ctypes.c_size_t, [_i, _i, _i, _i, _i]),
    "wq_gemm_static": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _i]),
    "wq_gemm_fused": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, ctypes.POINTER(wq_epilogue), _vp,
                           ctypes.c_size_t, _vp, _i]),
    "wq_prepack_bytes": (ctypes.c_size_t, [_i, _i, _i, _i]),
    "wq_prepack": (_i, [_vp, _vp, _vp, _vp, ctypes.c_size_t, _i, _i, _i, _i, _vp]),
    "wq_gemm_prepacked": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, ctypes.POINTER(wq_epilogue), _vp,
                               ctypes.c_size_t, _vp, _i]),
    "wq_fp4_scale_bytes": (ctypes.c_size_t, [_i, _i, _i, _i]),
    "wq_fp4_quantize": (_i, [ctypes.POINTER(wq_fp4_quant), _vp]),
    "wq_fp4_tile_scales": (_i, [_vp, _vp, _i, _i, _i, _vp]),
    "wq_block_norm": (_i, [ctypes.POINTER(wq_norm), _vp]),
    "wq_gemm_fp4": (_i, [ctypes.POINTER(wq_fp4_gemm), _vp]),
    "wq_dequant": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp]),
    "wq_get_device_error": (_i, []),
    "wq_selftest_timeout": (_i, [_vp]),
    "wq_status_string": (ctypes.c_char_p, [_i]),
    "wq_version": (_i, []),
}


class WQError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})" if what else status_string(status))


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """Load libwq.so (built by __graft_entry__.build() / build.py); raise if absent."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`"
                    " (there is no CPU fallback)")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
            _lib = L
    return _lib


# -- the C ABI, same names ----------------------------------------------------
def wq_gemm(A, packed, scales, zeros, C, M, N, K, format, group) -> int:
    return lib().wq_gemm(A, packed, scales, zeros, C, M, N, K, format, group)


def wq_gemm_ex(A, packed, scales, zeros, C, M, N, K, format, group, stream, path) -> int:
    return lib().wq_gemm_ex(A, packed, scales, zeros, C, M, N, K, format, group, stream, path)


def wq_gemm_ws(A, packed, scales, zeros, C, M, N, K, format, group, workspace, workspace_bytes, stream,
               path) -> int:
    return lib().wq_gemm_ws(A, packed, scales, zeros, C, M, N, K, format, group, workspace, workspace_bytes,
                            stream, path)


def wq_gemm_static(A, packed, scales, zeros, C, M, N, K, format, group, stream, path) -> int:
    return lib().wq_gemm_static(A, packed, scales, zeros, C, M, N, K, format, group, stream, path)


def wq_gemm_fused(A, packed, scales, zeros, C, M, N, K, format, group, epilogue, workspace, workspace_bytes,
                  stream, path) -> int:
    return lib().wq_gemm_fused(A, packed, scales, zeros, C, M, N, K, format, group, epilogue, workspace,
                               workspace_bytes, stream, path)


def wq_gemm_workspace_size(M, N, K, format, group) -> int:
    return lib().wq_gemm_workspace_size(M, N, K, format, group)


def wq_workspace_bytes(M, N, K, format, group) -> int:
    return lib().wq_workspace_bytes(M, N, K, format, group)


def wq_prepack_bytes(N, K, format, group) -> int:
    return lib().wq_prepack_bytes(N, K, format, group)


def wq_prepack(packed, scales, zeros, prepacked, prepacked_bytes, N, K, format, group, stream) -> int:
    return lib().wq_prepack(packed, scales, zeros, prepacked, prepacked_bytes, N, K, format, group, stream)


def wq_gemm_prepacked(A, prepacked, C, M, N, K, format, group, epilogue, workspace, workspace_bytes, stream,
                      path) -> int:
    return lib().wq_gemm_prepacked(A, prepacked, C, M, N, K, format, group, epilogue, workspace, workspace_bytes,
                                   stream, path)


def wq_dequant(packed, scales, zeros, W, N, K, format, group, stream) -> int:
    return lib().wq_dequant(packed, scales, zeros, W, N, K, format, group, stream)


def wq_fp4_scale_bytes(rows, K, format, layout) -> int:
    return lib().wq_fp4_scale_bytes(rows, K, format, layout)


def wq_fp4_quantize(x, x_type, ldx, rows, K, format, tensor_scale, packed, scales, layout, values, stream) -> int:
    return lib().wq_fp4_quantize(wq_fp4_quant(x, ldx, x_type, rows, K, format, layout, tensor_scale, packed, scales,
                                              values), stream)


def wq_fp4_tile_scales(scales, tiled, rows, K, format, stream) -> int:
    return lib().wq_fp4_tile_scales(scales, tiled, rows, K, format, stream)


def wq_block_norm(args, stream) -> int:
    return lib().wq_block_norm(args, stream)


def wq_gemm_fp4(a_packed, a_scales, a_tensor_scale, b_packed, b_scales, b_tensor_scale, C, M, N, K, format, epilogue,
                stream, path) -> int:
    """epilogue: a wq_epilogue, byref() of one, or None."""
    epi = wq_epilogue() if epilogue is None else getattr(epilogue, "_obj", epilogue)
    return lib().wq_gemm_fp4(wq_fp4_gemm(a_packed, a_scales, a_tensor_scale, b_packed, b_scales, b_tensor_scale, C, M, N,
                                         K, format, epi, path), stream)


def wq_get_device_error() -> int:
    return lib().wq_get_device_error()


def wq_selftest_timeout(stream=None) -> int:
    return lib().wq_selftest_timeout(stream)


def wq_status_string(status: int) -> str:
    return lib().wq_status_string(int(status)).decode()


def wq_version() -> int:
    return lib().wq_version()


def status_string(status: int) -> str:
    try:
        return wq_status_string(status)
    except Exception:   # library not loadable: still give a message
        return f"wq status {status}"


# -- tensor-level helpers -------------------------------------------------------
def _fmt(fmt) -> int:
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def _fmt_name(fmt) -> str:
    if isinstance(fmt, str):
        return fmt
    return {v: k for k, v in FORMATS.items()}[int(fmt)]


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream, device):
    import torch
    s = torch.cuda.current_stream(device) if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


_workspaces = {}


def workspace(M, N, K, fmt, group=None, device=None):
    """A zeroed device workspace for wq_gemm_ws on this shape (None if the
    shape needs none), cached per device and grown as needed.  Completed calls
    leave its flag words zero, so it is reused across calls on one stream."""
    import torch
    group = group or DEFAULT_GROUP[_fmt_name(fmt)]
    nbytes = wq_gemm_workspace_size(M, N, K, _fmt(fmt), int(group))
    if nbytes == 0:
        return None
    dev = torch.device(device if device is not None else "cuda")
    key = dev.index if dev.index is not None else torch.cuda.current_device()
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=torch.device("cuda", key))
        _workspaces[key] = ws
    return ws


def _launch_bits(overlap, inputs_ready):
    return (WQ_LAUNCH_OVERLAP if overlap else 0) | (WQ_LAUNCH_INPUTS_READY if inputs_ready else 0)


def gemm(A, packed, scales, zeros, fmt, group=None, out_dtype="bf16", out=None, path="auto", stream=None,
         overlap=False, workspace=None, bias=None, residual=None, gated=False, inputs_ready=False):
    """C = A . deq(packed, scales, zeros)^T on A's device and current stream.

    overlap=True sets WQ_LAUNCH_OVERLAP (programmatic dependent launch): the
    caller guarantees the preceding kernel on the stream does not write the
    weights.  inputs_ready=True sets WQ_LAUNCH_INPUTS_READY: A, too, is
    written by no kernel that may still be running (include/wq.h).  workspace: a zeroed uint8 CUDA tensor (see workspace()) that
    lets the tensor-core path split tiles over the SMs; "auto" takes the
    cached one.  bias (N,) bf16, residual (M, outputs) bf16 and gated select
    the fused epilogue of wq_gemm_fused (gated: C has N / 2 columns).

    A: (M, K) bf16; packed: (N, K/2) uint8; scales: (N, K/group) uint8
    (nvfp4 e4m3 / mxfp4 e8m0 bytes) or bf16 (int4); zeros: (N, K/group)
    uint8 for int4, None otherwise.  Returns C (M, N) bf16 or fp32.
    """
    import torch
    f = _fmt(fmt)
    group = group or DEFAULT_GROUP[_fmt_name(fmt)]
    M, K = A.shape
    N = packed.shape[0]
    if packed.shape[1] * 2 != K:
        raise ValueError(f"packed {tuple(packed.shape)} does not match K={K}")
    for t in (A, packed, scales, zeros, out):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("all tensors must be contiguous CUDA tensors")
    if A.dtype != torch.bfloat16 or packed.dtype != torch.uint8:
        raise ValueError("A must be bf16 and packed uint8")
    odt = torch.float32 if out_dtype in ("fp32", torch.float32) else torch.bfloat16
    ncol = N // 2 if gated else N
    if out is None:
        out = torch.empty((M, ncol), dtype=odt, device=A.device)
    elif out.shape != (M, ncol) or out.dtype != odt:
        raise ValueError("out has the wrong shape or dtype")
    for t, shape in ((bias, (N,)), (residual, (M, ncol))):
        if t is not None and (t.dtype != torch.bfloat16 or tuple(t.shape) != shape or not t.is_cuda
                              or not t.is_contiguous()):
            raise ValueError(f"bias / residual must be contiguous bf16 CUDA tensors of shape {shape}")
    fmt_word = f | (WQ_OUT_F32 if odt == torch.float32 else 0)
    pcode = (PATHS[path] if isinstance(path, str) else int(path)) | _launch_bits(overlap, inputs_ready)
    if isinstance(workspace, str) and workspace == "auto":
        workspace = globals()["workspace"](M, N, K, fmt, group, A.device)
    if bias is not None or residual is not None or gated:
        epi = wq_epilogue(None if bias is None else bias.data_ptr(),
                          None if residual is None else residual.data_ptr(), 1 if gated else 0)
        if workspace is not None and (not workspace.is_cuda or workspace.dtype != torch.uint8):
            raise ValueError("workspace must be a uint8 CUDA tensor")
        st = wq_gemm_fused(_ptr(A), _ptr(packed), _ptr(scales), _ptr(zeros), _ptr(out), M, N, K, fmt_word,
                           int(group), ctypes.byref(epi), _ptr(workspace),
                           0 if workspace is None else workspace.numel(), _stream_handle(stream, A.device), pcode)
    elif workspace is None:
        st = wq_gemm_ex(_ptr(A), _ptr(packed), _ptr(scales), _ptr(zeros), _ptr(out), M, N, K, fmt_word,
                        int(group), _stream_handle(stream, A.device), pcode)
    else:
        if not workspace.is_cuda or workspace.dtype != torch.uint8:
            raise ValueError("workspace must be a uint8 CUDA tensor")
        st = wq_gemm_ws(_ptr(A), _ptr(packed), _ptr(scales), _ptr(zeros), _ptr(out), M, N, K, fmt_word,
                        int(group), _ptr(workspace), workspace.numel(), _stream_handle(stream, A.device), pcode)
    if st != WQ_OK:
        raise WQError(st, "wq_gemm")
    return out


class Prepacked:
    """A weight in the prepacked layout (wq_prepack): the uint8 device buffer
    and the description it was made from."""

    def __init__(self, buf, N, K, fmt, group):
        self.buf, self.N, self.K, self.fmt, self.group = buf, N, K, _fmt_name(fmt), group


def prepack(packed, scales, zeros, fmt, group=None, stream=None, out=None) -> Prepacked:
    """Repack one weight (wq_prepack) into a new uint8 CUDA tensor, or into
    `out` (a uint8 CUDA tensor of at least wq_prepack_bytes() elements)."""
    import torch
    f = _fmt(fmt)
    group = group or DEFAULT_GROUP[_fmt_name(fmt)]
    N, Kh = packed.shape
    K = 2 * Kh
    for t in (packed, scales, zeros):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("all tensors must be contiguous CUDA tensors")
    nbytes = wq_prepack_bytes(N, K, f, int(group))
    if nbytes == 0:
        raise WQError(WQ_ERR_UNSUPPORTED, "wq_prepack_bytes")
    if out is None:
        buf = torch.empty(nbytes, dtype=torch.uint8, device=packed.device)
    elif out.dtype != torch.uint8 or not out.is_cuda or not out.is_contiguous() or out.numel() < nbytes:
        raise ValueError(f"out must be a contiguous uint8 CUDA tensor of at least {nbytes} bytes")
    else:
        buf = out
    st = wq_prepack(_ptr(packed), _ptr(scales), _ptr(zeros), _ptr(buf), nbytes, N, K, f, int(group),
                    _stream_handle(stream, packed.device))
    if st != WQ_OK:
        raise WQError(st, "wq_prepack")
    return Prepacked(buf, N, K, fmt, int(group))


def gemm_prepacked(A, pre: Prepacked, out_dtype="bf16", out=None, stream=None, overlap=False, bias=None,
                   residual=None, gated=False, path="auto", workspace=None, inputs_ready=False):
    """C = A . deq(B)^T for a prepacked weight (wq_gemm_prepacked); the other
    arguments as for gemm()."""
    import torch
    M, K = A.shape
    N = pre.N
    if K != pre.K:
        raise ValueError(f"A has K={K}, the weight K={pre.K}")
    for t in (A, out):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("all tensors must be contiguous CUDA tensors")
    if A.dtype != torch.bfloat16:
        raise ValueError("A must be bf16")
    odt = torch.float32 if out_dtype in ("fp32", torch.float32) else torch.bfloat16
    ncol = N // 2 if gated else N
    if out is None:
        out = torch.empty((M, ncol), dtype=odt, device=A.device)
    elif out.shape != (M, ncol) or out.dtype != odt:
        raise ValueError("out has the wrong shape or dtype")
    for t, shape in ((bias, (N,)), (residual, (M, ncol))):
        if t is not None and (t.dtype != torch.bfloat16 or tuple(t.shape) != shape or not t.is_cuda
                              or not t.is_contiguous()):
            raise ValueError(f"bias / residual must be contiguous bf16 CUDA tensors of shape {shape}")
    epi = None
    if bias is not None or residual is not None or gated:
        epi = ctypes.byref(wq_epilogue(None if bias is None else bias.data_ptr(),
                                       None if residual is None else residual.data_ptr(), 1 if gated else 0))
    fmt_word = _fmt(pre.fmt) | (WQ_OUT_F32 if odt == torch.float32 else 0)
    pcode = (PATHS[path] if isinstance(path, str) else int(path)) | _launch_bits(overlap, inputs_ready)
    if isinstance(workspace, str) and workspace == "auto":
        workspace = globals()["workspace"](M, N, K, pre.fmt, pre.group, A.device)
    if workspace is not None and (not workspace.is_cuda or workspace.dtype != torch.uint8):
        raise ValueError("workspace must be a uint8 CUDA tensor")
    st = wq_gemm_prepacked(_ptr(A), _ptr(pre.buf), _ptr(out), M, N, K, fmt_word, pre.group, epi, _ptr(workspace),
                           0 if workspace is None else workspace.numel(), _stream_handle(stream, A.device), pcode)
    if st != WQ_OK:
        raise WQError(st, "wq_gemm_prepacked")
    return out


def dequant(packed, scales, zeros, fmt, group=None, out=None, stream=None):
    """W = deq(packed, scales, zeros) as an (N, K) bf16 tensor (bit-exact RNE)."""
    import torch
    f = _fmt(fmt)
    group = group or DEFAULT_GROUP[_fmt_name(fmt)]
    N, Kh = packed.shape
    K = 2 * Kh
    for t in (packed, scales, zeros, out):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("all tensors must be contiguous CUDA tensors")
    if out is None:
        out = torch.empty((N, K), dtype=torch.bfloat16, device=packed.device)
    st = wq_dequant(_ptr(packed), _ptr(scales), _ptr(zeros), _ptr(out), N, K, f, int(group),
                    _stream_handle(stream, packed.device))
    if st != WQ_OK:
        raise WQError(st, "wq_dequant")
    return out


# -- 4-bit activations ----------------------------------------------------------
# These calls are small on the GPU (a few microseconds), so their host side is
# kept short: each attribute of a tensor is read once, the C functions are
# looked up once, the current stream comes from torch's raw accessor (0.1 us
# against 2.3 us for the stream object), and their structs are packed by the
# struct module and passed as bytes (0.4 us against 1.1 for 12 arguments).
class Fp4:
    """A 4-bit tensor (rows, K): packed codes (rows, K / 2), its scale bytes in
    `layout` ("tiled", what gemm_fp4 takes, or "rows", what gemm, dequant and
    prepack take), its format and the tensor scale (a one-element fp32 CUDA
    tensor, NVFP4 only, or None)."""

    __slots__ = ("packed", "scales", "rows", "K", "fmt", "scale", "layout")

    def __init__(self, packed, scales, rows, K, fmt, scale=None, layout="tiled"):
        self.packed, self.scales, self.rows, self.K, self.fmt = packed, scales, rows, K, fmt
        self.scale, self.layout = scale, layout


_FP4 = {"nvfp4": (WQ_NVFP4, 16), "mxfp4": (WQ_MXFP4, 32)}
# struct wq_fp4_quant: x, ldx, x_type, rows, K, format, layout, tensor_scale, packed, scales, values
_QUANT_STRUCT = struct.Struct("@PqiiiiiPPPP")
# struct wq_fp4_gemm: a_packed, a_scales, a_tensor_scale, b_packed, b_scales, b_tensor_scale, C, M, N, K, format,
# bias, residual, gated, (the end of wq_epilogue,) path
_GEMM_STRUCT = struct.Struct("@PPPPPPPiiiiPPi4xi4x")
# struct wq_norm: rows, d, kind, post, x, ldx, x_type, branch_type, branch, ldb, gate, gate_rows, eps, residual_scale,
# branch_scale, weight, bias, post_weight, post_bias, x_out, ldxo, out, ldo, out_type, out_scale_layout,
# out_scales, out_tensor_scale
_NORM_STRUCT = struct.Struct("@iiiiPqiiPqPifffPPPPPqPqiiPP")
_fast = None


def _fast_calls():
    """The entry points the tensor helpers below call, and torch's raw stream accessor."""
    global _fast
    if _fast is None:
        import torch
        L = lib()
        proto = ctypes.CFUNCTYPE(_i, ctypes.c_char_p, _vp)
        quant, gemm4, norm = (proto(ctypes.cast(f, _vp).value) for f in (L.wq_fp4_quantize, L.wq_gemm_fp4,
                                                                         L.wq_block_norm))
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is None:
            def raw(index):
                return torch.cuda.current_stream(index).cuda_stream
        _fast = (quant, gemm4, norm, raw, torch.bfloat16, torch.float32, torch.uint8)
    return _fast


def _raise(st, what):
    raise WQError(st, what)


def _fp4_fmt(fmt):
    f = _FP4.get(fmt)
    if f is None:
        raise ValueError(f"format {fmt!r} is not one of 'nvfp4', 'mxfp4'")
    return f


def _fp4_scale_bytes(rows, K, fmt, layout):
    """wq_fp4_scale_bytes for a checked description (K a multiple of 32)."""
    G = K // _FP4[fmt][1]
    return (rows + 127) // 128 * ((G + 3) // 4) * 512 if layout == "tiled" else rows * G


def _bytes_ptr(t, n, u8):
    """The address of a contiguous uint8 CUDA tensor of at least n bytes."""
    if t.dtype is not u8 or not t.is_cuda or not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"codes and scales must be contiguous uint8 CUDA tensors; {n} bytes are needed here")
    return t.data_ptr()


def _fp4_out(out, rows, K, fmt, layout, device, u8):
    """(codes, scales, their addresses) a call writes: those of `out` (an Fp4 or
    a pair), checked, or new ones."""
    code = LAYOUTS.get(layout)
    if code is None:
        raise ValueError(f"layout {layout!r} is not one of 'tiled', 'rows'")
    if K % 32:
        raise WQError(WQ_ERR_UNSUPPORTED, f"4-bit rows of {K} elements (a multiple of 32 is needed)")
    nbytes = _fp4_scale_bytes(rows, K, fmt, layout)
    if out is None:
        import torch
        packed = torch.empty((rows, K // 2), dtype=u8, device=device)
        scales = torch.empty((rows, K // _FP4[fmt][1]) if layout == "rows" else nbytes, dtype=u8, device=device)
        return packed, scales, packed.data_ptr(), scales.data_ptr(), code
    packed, scales = (out.packed, out.scales) if isinstance(out, Fp4) else out
    return packed, scales, _bytes_ptr(packed, rows * K // 2, u8), _bytes_ptr(scales, nbytes, u8), code


def _rows_of(t, what, shape, bf16, f32):
    """(address, type code, row stride) of a 2-D bf16 / fp32 CUDA tensor of
    `shape` with contiguous rows."""
    dt = t.dtype
    code = WQ_TYPE_BF16 if dt is bf16 else WQ_TYPE_F32 if dt is f32 else -1
    if code < 0 or len(shape) != 2 or not t.is_cuda:
        raise ValueError(f"{what} must be a 2-D bf16 or fp32 CUDA tensor")
    if t.shape != shape:
        raise ValueError(f"{what} must have the shape {tuple(shape)}")
    if t.is_contiguous():
        return t.data_ptr(), code, shape[1]
    ld, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise ValueError(f"{what} must have contiguous rows")
    return t.data_ptr(), code, ld


def _bf16_ptr(t, what, shape, bf16):
    """The address of a contiguous bf16 CUDA tensor of `shape`, 0 for None."""
    if t is None:
        return 0
    if t.dtype is not bf16 or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous bf16 CUDA tensor of shape {tuple(shape)}")
    return t.data_ptr()


def _scale_ptr(scale, f32):
    if scale is None:
        return 0
    if scale.dtype is not f32 or not scale.is_cuda or scale.numel() != 1:
        raise ValueError("a tensor scale is one fp32 value on the GPU")
    return scale.data_ptr()


def quantize(x, fmt, scale=None, out=None, values=None, layout="tiled", stream=None) -> Fp4:
    """x (rows, K), bf16 or fp32 with contiguous rows (any row stride), as an
    Fp4 of "nvfp4" or "mxfp4" (wq_fp4_quantize).  scale: the NVFP4 tensor
    scale, e.g. max |x| / (6 * 448).  out: an Fp4, or a pair (codes, scales) of
    uint8 tensors, to write into.  values: a bf16 (rows, K) tensor that gets
    what the codes stand for.  layout "rows" makes weights for gemm, dequant
    and prepack, "tiled" operands for gemm_fp4."""
    call, _, _, raw, bf16, f32, u8 = _fast or _fast_calls()
    f = _fp4_fmt(fmt)[0]
    shape = x.shape
    xp, xt, ld = _rows_of(x, "x", shape, bf16, f32)
    rows, K = shape
    packed, scales, pp, sp, lay = _fp4_out(out, rows, K, fmt, layout, x.device, u8)
    st = call(_QUANT_STRUCT.pack(xp, ld, xt, rows, K, f, lay, 0 if scale is None else _scale_ptr(scale, f32), pp, sp,
                                 0 if values is None else _bf16_ptr(values, "values", shape, bf16)),
              raw(x.get_device()) if stream is None else stream.cuda_stream)
    if st:
        _raise(st, "wq_fp4_quantize")
    return Fp4(packed, scales, rows, K, fmt, scale, layout)


def fp4_operand(packed, scales, fmt, scale=None, stream=None) -> Fp4:
    """A weight held as gemm takes it -- packed (rows, K / 2), scales
    (rows, K / group) uint8 -- as an operand of gemm_fp4: the codes as they
    are, the scales re-ordered once (wq_fp4_tile_scales)."""
    import torch
    f, group = _fp4_fmt(fmt)
    rows, K = packed.shape[0], 2 * packed.shape[1]
    for t, n in ((packed, K // 2), (scales, K // group)):
        if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != (rows, n):
            raise ValueError("packed and scales must be contiguous uint8 CUDA tensors of (rows, K / 2) and "
                             "(rows, K / group)")
    _scale_ptr(scale, torch.float32)
    if K % 32:
        raise WQError(WQ_ERR_UNSUPPORTED, f"4-bit rows of {K} elements (a multiple of 32 is needed)")
    tiled = torch.empty(_fp4_scale_bytes(rows, K, fmt, "tiled"), dtype=torch.uint8, device=packed.device)
    st = wq_fp4_tile_scales(scales.data_ptr(), tiled.data_ptr(), rows, K, f, _stream_handle(stream, packed.device))
    if st != WQ_OK:
        raise WQError(st, "wq_fp4_tile_scales")
    return Fp4(packed, tiled, rows, K, fmt, scale)


def block_norm(x, weight, branch=None, bias=None, post_weight=None, post_bias=None, post=None, gate=None,
               residual_scale=1.0, branch_scale=1.0, kind="rms", eps=1e-5, x_out=None, out=None, out_dtype="bf16",
               fmt=None, layout="tiled", scale=None, stream=None):
    """(x', u) between two blocks (wq_block_norm): x' = residual_scale x +
    branch_scale gate N(branch), u = N(x').

    x (rows, d): the residual stream, bf16 or fp32; branch (rows, d): the
    block's output, normed first where post_weight is given or post=True; gate
    (gate_rows, d) bf16 with gate_rows dividing rows (1: per channel, rows: per
    element); weight, bias, post_weight, post_bias (d,) bf16 or None (1 and 0).
    x, branch, x_out and out may have any row stride.  x_out: where x' goes (x
    itself: in place); without a branch and without x_out, x' is not stored
    and None is returned for it.  u is bf16 or fp32 (out_dtype, or out's type),
    or with fmt "nvfp4" / "mxfp4" an Fp4 as quantize() would make of it
    (layout, scale, and out a pair of tensors, as there)."""
    _, _, call, raw, bf16, f32, u8 = _fast or _fast_calls()
    kcode = NORM_KINDS.get(kind)
    if kcode is None:
        raise ValueError(f"kind {kind!r} is not one of 'rms', 'layer'")
    shape = x.shape
    xp, xt, ldx = _rows_of(x, "x", shape, bf16, f32)
    rows, d = shape
    bp, bt, ldb = (0, WQ_TYPE_BF16, 0) if branch is None else _rows_of(branch, "branch", shape, bf16, f32)
    gp, gate_rows = 0, 0
    if gate is not None:
        gate_rows = gate.shape[0]
        gp = _bf16_ptr(gate, "gate", (gate_rows, d), bf16)
        if gate_rows == 0 or rows % gate_rows:
            raise ValueError("gate's rows must divide x's")
    vec = (d,)
    if branch is not None and x_out is None:
        import torch
        x_out = torch.empty(shape, dtype=x.dtype, device=x.device)
    xop, ldxo = 0, 0
    if x_out is not None:
        xop, xot, ldxo = _rows_of(x_out, "x_out", shape, bf16, f32)
        if xot != xt:
            raise ValueError("x_out must have x's type")
    if fmt is not None:
        otype = WQ_NORM_OUT_NVFP4 if _fp4_fmt(fmt)[0] == WQ_NVFP4 else WQ_NORM_OUT_MXFP4
        packed, scales, optr, osp, lay = _fp4_out(out, rows, d, fmt, layout, x.device, u8)
        tsp, ldo = 0 if scale is None else _scale_ptr(scale, f32), d
        u = Fp4(packed, scales, rows, d, fmt, scale, layout)
    else:
        if out is None:
            import torch
            out = torch.empty(shape, dtype=f32 if out_dtype in ("fp32", f32) else bf16, device=x.device)
        optr, ot, ldo = _rows_of(out, "out", shape, bf16, f32)
        otype = WQ_NORM_OUT_F32 if ot == WQ_TYPE_F32 else WQ_NORM_OUT_BF16
        osp, lay, tsp, u = 0, 0, 0, out
    if post is None:
        post = post_weight is not None
    args = _NORM_STRUCT.pack(rows, d, kcode, 1 if post else 0, xp, ldx, xt, bt, bp, ldb, gp, gate_rows, eps,
                             residual_scale, branch_scale,
                             0 if weight is None else _bf16_ptr(weight, "weight", vec, bf16),
                             0 if bias is None else _bf16_ptr(bias, "bias", vec, bf16),
                             0 if post_weight is None else _bf16_ptr(post_weight, "post_weight", vec, bf16),
                             0 if post_bias is None else _bf16_ptr(post_bias, "post_bias", vec, bf16), xop, ldxo, optr,
                             ldo, otype, lay, osp, tsp)
    st = call(args, raw(x.get_device()) if stream is None else stream.cuda_stream)
    if st:
        _raise(st, "wq_block_norm")
    return x_out, u


def gemm_fp4(A: Fp4, B: Fp4, out_dtype="bf16", out=None, bias=None, residual=None, gated=False, stream=None,
             overlap=False):
    """C = A . B^T for 4-bit operands with tiled scales (wq_gemm_fp4): A (M, K)
    the activations, B (N, K) the weights.  out (its type then is C's), bias,
    residual and gated as for gemm(); overlap=True as there, too: B is read
    ahead, and the caller guarantees that the preceding kernel on the stream
    does not write it."""
    _, call, _, raw, bf16, f32, u8 = _fast or _fast_calls()
    M, K, N, fmt, sa, sb = A.rows, A.K, B.rows, A.fmt, A.scale, B.scale
    f, group = _FP4.get(fmt) or _fp4_fmt(fmt)
    if B.K != K or B.fmt != fmt:
        raise ValueError(f"A is {fmt} with K={K}, B {B.fmt} with K={B.K}")
    if A.layout != "tiled" or B.layout != "tiled":
        raise ValueError("gemm_fp4 takes tiled scales (quantize(layout='tiled'), fp4_operand())")
    row_block = (K // group + 3) // 4 * 512   # scale bytes of 128 rows
    a = A.packed
    ap, asp = _bytes_ptr(a, M * K // 2, u8), _bytes_ptr(A.scales, (M + 127) // 128 * row_block, u8)
    wp, wsp = _bytes_ptr(B.packed, N * K // 2, u8), _bytes_ptr(B.scales, (N + 127) // 128 * row_block, u8)
    shape = (M, N // 2 if gated else N)
    if out is None:
        import torch
        out = torch.empty(shape, dtype=f32 if out_dtype in ("fp32", f32) else bf16, device=a.device)
    dt = out.dtype
    if dt is f32:
        f |= WQ_OUT_F32
    if out.shape != shape or not (dt is f32 or dt is bf16) or not out.is_cuda or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous bf16 or fp32 CUDA tensor of shape {shape}")
    st = call(_GEMM_STRUCT.pack(ap, asp, 0 if sa is None else _scale_ptr(sa, f32), wp, wsp,
                                0 if sb is None else _scale_ptr(sb, f32), out.data_ptr(), M, N, K, f,
                                0 if bias is None else _bf16_ptr(bias, "bias", (N,), bf16),
                                0 if residual is None else _bf16_ptr(residual, "residual", shape, bf16),
                                1 if gated else 0, WQ_LAUNCH_OVERLAP if overlap else 0),
              raw(a.get_device()) if stream is None else stream.cuda_stream)
    if st:
        _raise(st, "wq_gemm_fp4")
    return out
