"""Python binding of libnvfp4 (include/nvfp4.h): the NVFP4 W4A16 linear layer on B200.

Argument marshalling only: every entry point takes torch CUDA tensors, checks
dtypes and shapes, and passes raw device pointers, leading dimensions and the
current CUDA stream to the C ABI.  All arithmetic runs in the library's CUDA
kernels; there is no CPU path.  Importing fails loudly if the library has not
been built (``python gemm_decode_nvfp4_b200/build.py``).

Layouts follow the NVFP4 format of the pages (imp docs/quantization.md, format
table: packed nibbles, E4M3 micro-scales per 16, FP32 tensor scale):
q uint8 [N, K/2] (low nibble = even k), s uint8 [N, K/16], g float32 [1].
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

__all__ = [
    "Nvfp4Error", "LIB_PATH", "lib", "version", "amax", "quantize", "quantize_mse", "gemv", "gemm",
    "gemm_workspace_size", "quantize_new", "linear", "declared_symbols", "check_device_errors",
    "FLAG_STATIC_WEIGHTS", "gemm_noalloc", "GEMM_NOALLOC_SCRATCH_BYTES",
    "mx_quantize", "mx_quantize_new", "mx_gemv", "gemv_grouped", "mx_to_nvfp4",
    "GIVEN_AMAX", "w4a4_prepare_weights", "w4a4_quantize_x", "w4a4_gemm", "w4a4_linear",
    "w4a4_workspace_size", "AMAX_FLOATS",
    "fp8_rmsnorm", "fp8_quantize", "fp8_quantize_new", "fp8_quantize_weights", "fp8_quantize_weights_new",
    "fp8_gemm", "fp8_gemm_grouped", "fp8_linear",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnvfp4.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "nvfp4.h")
MX_HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "mxfp4.h")
W4A4_HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "nvfp4_w4a4.h")
FP8_HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "fp8.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python gemm_decode_nvfp4_b200/build.py`")

lib = ctypes.CDLL(LIB_PATH)

_p, _i64, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
lib.nvfp4_version.argtypes, lib.nvfp4_version.restype = [], ctypes.c_int
lib.nvfp4_last_error.argtypes, lib.nvfp4_last_error.restype = [], ctypes.c_char_p
lib.nvfp4_status_string.argtypes, lib.nvfp4_status_string.restype = [ctypes.c_int], ctypes.c_char_p
lib.nvfp4_amax.argtypes = [_p, _i64, _i64, _i64, _p, _p]
lib.nvfp4_quantize.argtypes = [_p, _i64, _i64, _i64, _p, _p, _p, _p, _p]
lib.nvfp4_quantize_mse.argtypes = [_p, _i64, _i64, _i64, _p, ctypes.c_int32, _p, _p, _p, _p]
lib.nvfp4_gemv.argtypes = [_p, _p, _p, _p, _p, _i64, _i64, _p]
lib.nvfp4_gemm.argtypes = [_p, _i64, _p, _p, _p, _p, _i64, _i64, _i64, _i64, _p, _sz, _p]
lib.nvfp4_gemv_ex.argtypes = [_p, _p, _p, _p, _p, _i64, _i64, ctypes.c_uint32, _p]
lib.nvfp4_gemm_ex.argtypes = [_p, _i64, _p, _p, _p, _p, _i64, _i64, _i64, _i64, _p, _sz, ctypes.c_uint32, _p]
lib.nvfp4_gemm_noalloc.argtypes = [_p, _i64, _p, _p, _p, _p, _i64, _i64, _i64, _i64, ctypes.c_uint32, _p]
lib.nvfp4_gemm_workspace_size.argtypes = [_i64, _i64, _i64]
lib.nvfp4_gemv_grouped.argtypes = [_p, _i64, _p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _i64, _i64, _i64,
                                   ctypes.c_uint32, _p]
lib.mxfp4_quantize.argtypes = [_p, _i64, _i64, _i64, _p, _p, _p]
lib.mxfp4_to_nvfp4_scales.argtypes = [_p, _p, _i64, _i64, _p, _p, _p]
lib.nvfp4_w4a4_weight_scales_bytes.argtypes, lib.nvfp4_w4a4_weight_scales_bytes.restype = [_i64, _i64], _sz
lib.nvfp4_w4a4_x_scales_bytes.argtypes, lib.nvfp4_w4a4_x_scales_bytes.restype = [_i64, _i64], _sz
lib.nvfp4_w4a4_workspace_size.argtypes, lib.nvfp4_w4a4_workspace_size.restype = [_i64, _i64], _sz
lib.nvfp4_w4a4_prepare_weights.argtypes = [_p, _i64, _i64, _p, _p]
lib.nvfp4_w4a4_quantize_x.argtypes = [_p, _i64, _i64, _i64, _p, _p, _p, ctypes.c_uint32, _p]
lib.nvfp4_w4a4_gemm.argtypes = [_p, _p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _i64, ctypes.c_uint32, _p]
lib.nvfp4_w4a4_linear.argtypes = [_p, _i64, _p, _p, _p, _p, _p, _i64, _i64, _i64, _i64, _p, _sz, ctypes.c_uint32, _p]
lib.mxfp4_gemv.argtypes = [_p, _p, _p, _p, _i64, _i64, _p]
lib.mxfp4_gemv_ex.argtypes = [_p, _p, _p, _p, _i64, _i64, ctypes.c_uint32, _p]
lib.fp8_rmsnorm.argtypes = [_p, _i64, _p, _p, _i64, _p, _i64, _p, _i64, _p, _p, _i64, _i64, ctypes.c_float, _p]
lib.fp8_quantize.argtypes = [_p, _i64, _i64, _i64, _p, _p, ctypes.c_uint32, _p]
lib.fp8_quantize_weights.argtypes = [_p, _i64, _i64, _i64, _p, _p, _p]
lib.fp8_gemm.argtypes = [_p, _p, _p, _p, _p, _i64, _i64, _i64, _i64, ctypes.c_uint32, _p]
lib.fp8_gemm_grouped.argtypes = [_p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _i64, _i64, ctypes.c_uint32, _p]
lib.nvfp4_gemm_workspace_size.restype = _sz
lib.nvfp4_check_device_errors.argtypes = []
for _f in (lib.nvfp4_amax, lib.nvfp4_quantize, lib.nvfp4_quantize_mse, lib.nvfp4_gemv, lib.nvfp4_gemm, lib.nvfp4_gemv_ex, lib.nvfp4_gemm_ex,
           lib.nvfp4_gemm_noalloc, lib.nvfp4_check_device_errors, lib.mxfp4_quantize, lib.mxfp4_gemv,
           lib.mxfp4_gemv_ex, lib.nvfp4_gemv_grouped, lib.mxfp4_to_nvfp4_scales,
           lib.nvfp4_w4a4_prepare_weights, lib.nvfp4_w4a4_quantize_x, lib.nvfp4_w4a4_gemm,
           lib.nvfp4_w4a4_linear, lib.fp8_rmsnorm, lib.fp8_quantize, lib.fp8_quantize_weights, lib.fp8_gemm,
           lib.fp8_gemm_grouped):
    _f.restype = ctypes.c_int


class Nvfp4Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        name = lib.nvfp4_status_string(status).decode()
        msg = lib.nvfp4_last_error().decode()
        super().__init__(f"{fn}: {name}: {msg}")


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise Nvfp4Error(fn, status)


def check_device_errors() -> None:
    """Raise if a CTA gave up on a bounded pipeline wait, or a grouped call had ids or
    offsets out of range (nvfp4_check_device_errors)."""
    _check("nvfp4_check_device_errors", lib.nvfp4_check_device_errors())


def version() -> int:
    return lib.nvfp4_version()


def declared_symbols() -> list[str]:
    """Names of the entry points include/nvfp4.h, mxfp4.h, nvfp4_w4a4.h and fp8.h declare."""
    names = []
    for path in (HEADER_PATH, MX_HEADER_PATH, W4A4_HEADER_PATH, FP8_HEADER_PATH):
        with open(path) as f:
            names += re.findall(r"NVFP4_API\s+[\w\s\*]+?\b((?:nvfp4|mxfp4|fp8)_\w+)\s*\(", f.read())
    return names


def _device(*tensors) -> torch.device:
    """The one CUDA device all the given tensors (None skipped) live on."""
    dev = None
    for t in tensors:
        if t is not None:
            if dev is None:
                dev = t.device
            elif t.device != dev:
                devs = sorted({str(u.device) for u in tensors if u is not None})
                raise ValueError(f"tensors must all be on one CUDA device, got {devs}")
    return dev


# the raw handle of a device's current stream, without making a Stream object of it
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream(stream, dev: torch.device) -> int:
    """The raw stream handle for a call on `dev`: the given stream (which must
    belong to `dev`) or that device's current stream."""
    if stream is None:
        return _current_raw_stream(dev.index)
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    return stream.cuda_stream


def _on_stream(stream, dev: torch.device, fn, *args, **kw):
    """fn(*args, **kw) with `stream` current, for the functions that allocate: what
    they allocate and copy then belongs to the stream that their kernels run on.
    (Memory of the current stream could still be in use by its earlier work, and
    a temporary of it would be handed on while `stream` reads it.)  The caller may
    use the returned tensors on the current stream, ordered after `stream`, and drop
    them there."""
    if dev.type == "cuda":
        _stream(stream, dev)
    with torch.cuda.stream(stream):
        out = fn(*args, **kw)
    if dev.type == "cuda" and out is not None:
        for t in out if isinstance(out, tuple) else (out,):
            t.record_stream(torch.cuda.current_stream(dev))
    return out


def _call(fn: str, dev: torch.device, *args) -> None:
    """Call lib.<fn>(*args) with `dev` current (the library launches on the
    current device) and raise on a non-zero status."""
    if torch.cuda.current_device() == dev.index:
        _check(fn, getattr(lib, fn)(*args))
        return
    with torch.cuda.device(dev):
        _check(fn, getattr(lib, fn)(*args))


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, dtype, what: str, ndim=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    dim = t.dim()
    if ndim is not None and dim != ndim:
        raise ValueError(f"{what} must be {ndim}-D, got shape {tuple(t.shape)}")
    if dim >= 1 and t.stride(-1) != 1 and t.numel() > 0:
        raise ValueError(f"{what} must be contiguous in its last dimension")


def _rows_ld(t: torch.Tensor):
    return (t.shape[0], t.stride(0)) if t.dim() == 2 else (1, t.shape[-1])


def amax(w: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """out = max(out, max|w|) for a BF16 matrix w (out: float32 [1] on the device)."""
    _need(w, torch.bfloat16, "w")
    _need(out, torch.float32, "out")
    dev = _device(w, out)
    if w.dim() != 2 and stream is not None:   # (reshape may copy)
        return _on_stream(stream, dev, amax, w, out)
    w2 = w if w.dim() == 2 else w.reshape(1, -1)
    _call("nvfp4_amax", dev, _ptr(w2), w2.shape[0], w2.shape[1], w2.stride(0), _ptr(out), _stream(stream, dev))


def quantize(w: torch.Tensor, q: torch.Tensor, s: torch.Tensor, g_out: torch.Tensor | None,
             amax: torch.Tensor | None = None, stream=None) -> None:
    """RTN NVFP4 of BF16 w [N, K] into q [N, K/2] u8 and s [N, K/16] u8; g_out gets
    g = amax / 2688.  With amax=None the tensor's own amax is used."""
    _need(w, torch.bfloat16, "w", 2)
    _need(q, torch.uint8, "q", 2)
    _need(s, torch.uint8, "s", 2)
    N, K = w.shape
    if q.shape != (N, K // 2) or s.shape != (N, K // 16) or not q.is_contiguous() or not s.is_contiguous():
        raise ValueError("q/s must be contiguous [N, K/2] / [N, K/16]")
    if g_out is not None:
        _need(g_out, torch.float32, "g_out")
    if amax is not None:
        _need(amax, torch.float32, "amax")
    dev = _device(w, q, s, g_out, amax)
    _call("nvfp4_quantize", dev, _ptr(w), N, K, w.stride(0), _ptr(amax), _ptr(q), _ptr(s), _ptr(g_out),
          _stream(stream, dev))


def quantize_mse(w: torch.Tensor, q: torch.Tensor, s: torch.Tensor, g_out: torch.Tensor | None,
                 amax: torch.Tensor | None = None, window: int = 8, stream=None) -> None:
    """NVFP4 of BF16 w [N, K] with each micro-scale chosen by the least fp64
    reconstruction error among the E4M3 codes within `window` of the
    round-to-nearest one (nvfp4_quantize_mse); otherwise as quantize()."""
    _need(w, torch.bfloat16, "w", 2)
    _need(q, torch.uint8, "q", 2)
    _need(s, torch.uint8, "s", 2)
    N, K = w.shape
    if q.shape != (N, K // 2) or s.shape != (N, K // 16) or not q.is_contiguous() or not s.is_contiguous():
        raise ValueError("q/s must be contiguous [N, K/2] / [N, K/16]")
    if g_out is not None:
        _need(g_out, torch.float32, "g_out")
    if amax is not None:
        _need(amax, torch.float32, "amax")
    dev = _device(w, q, s, g_out, amax)
    _call("nvfp4_quantize_mse", dev, _ptr(w), N, K, w.stride(0), _ptr(amax), int(window), _ptr(q), _ptr(s),
          _ptr(g_out), _stream(stream, dev))


FLAG_STATIC_WEIGHTS = 1
FLAG_W4A4_PAIR = 1 << 12


def _ksplit_flag(k_split: int) -> int:
    """NVFP4_FLAG_KSPLIT(k_split): 0 = the library's choice, else 1, 2, 4 or 8."""
    if k_split not in (0, 1, 2, 4, 8):
        raise ValueError(f"k_split must be 0, 1, 2, 4 or 8, got {k_split}")
    return k_split << 8


def gemv(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, g: torch.Tensor, y: torch.Tensor,
         stream=None, static_weights: bool = False, k_split: int = 0) -> None:
    """y[N] = bf16(g * W_deq . x) for BF16 x [K] (or [1, K]).  static_weights: q, s, g
    are not written by work still running on the stream (see NVFP4_FLAG_STATIC_WEIGHTS).
    k_split: CTAs of a cluster that split K (NVFP4_FLAG_KSPLIT); 0 = chosen per shape."""
    _need(x, torch.bfloat16, "x")
    _need(q, torch.uint8, "q", 2)
    _need(s, torch.uint8, "s", 2)
    _need(g, torch.float32, "g")
    _need(y, torch.bfloat16, "y")
    N, K = q.shape[0], q.shape[1] * 2
    if x.numel() != K or y.numel() != N or not x.is_contiguous() or not y.is_contiguous():
        raise ValueError("x must hold K and y N contiguous elements")
    if not q.is_contiguous() or not s.is_contiguous() or s.shape != (N, K // 16):
        raise ValueError("q/s must be contiguous [N, K/2] / [N, K/16]")
    flags = (FLAG_STATIC_WEIGHTS if static_weights else 0) | _ksplit_flag(k_split)
    dev = _device(x, q, s, g, y)
    _call("nvfp4_gemv_ex", dev, _ptr(x), _ptr(q), _ptr(s), _ptr(g), _ptr(y), N, K, flags, _stream(stream, dev))


def gemm_workspace_size(M: int, N: int, K: int) -> int:
    return lib.nvfp4_gemm_workspace_size(M, N, K)


def gemm(X: torch.Tensor, q: torch.Tensor, s: torch.Tensor, g: torch.Tensor, Y: torch.Tensor,
         workspace: torch.Tensor | None = None, stream=None, static_weights: bool = False) -> None:
    """Y [M, N] = bf16(g * X . W_deq^T) for BF16 X [M, K]."""
    _need(X, torch.bfloat16, "X", 2)
    _need(q, torch.uint8, "q", 2)
    _need(s, torch.uint8, "s", 2)
    _need(g, torch.float32, "g")
    _need(Y, torch.bfloat16, "Y", 2)
    M, K = X.shape
    N = q.shape[0]
    if q.shape[1] * 2 != K or Y.shape != (M, N):
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, q {tuple(q.shape)}, Y {tuple(Y.shape)}")
    if not q.is_contiguous() or not s.is_contiguous() or s.shape != (N, K // 16):
        raise ValueError("q/s must be contiguous [N, K/2] / [N, K/16]")
    ws_bytes = 0
    if workspace is not None:
        _need(workspace, torch.uint8, "workspace")
        ws_bytes = workspace.numel()
    flags = FLAG_STATIC_WEIGHTS if static_weights else 0
    dev = _device(X, q, s, g, Y, workspace)
    _call("nvfp4_gemm_ex", dev, _ptr(X), X.stride(0), _ptr(q), _ptr(s), _ptr(g), _ptr(Y), Y.stride(0), M, N, K,
          _ptr(workspace), ws_bytes, flags, _stream(stream, dev))


def _header_constant(name: str) -> int:
    with open(HEADER_PATH) as f:
        m = re.search(r"#define\s+" + name + r"\s+\(\(\(size_t\)(\d+) << (\d+)\) \+ (\d+)\)", f.read())
    if not m:
        raise ImportError(f"{name} not found in {HEADER_PATH}")
    return (int(m.group(1)) << int(m.group(2))) + int(m.group(3))


# Bytes of the scratch array built into the library for gemm_noalloc.
GEMM_NOALLOC_SCRATCH_BYTES = _header_constant("NVFP4_GEMM_NOALLOC_SCRATCH_BYTES")


def gemm_noalloc(X: torch.Tensor, q: torch.Tensor, s: torch.Tensor, g: torch.Tensor, Y: torch.Tensor,
                 stream=None, static_weights: bool = False) -> None:
    """gemm() with the library's built-in scratch instead of a workspace
    (nvfp4_gemm_noalloc): allocates nothing, for callers that cannot.  Calls on
    one device share the scratch and must be ordered (one stream)."""
    _need(X, torch.bfloat16, "X", 2)
    _need(q, torch.uint8, "q", 2)
    _need(s, torch.uint8, "s", 2)
    _need(g, torch.float32, "g")
    _need(Y, torch.bfloat16, "Y", 2)
    M, K = X.shape
    N = q.shape[0]
    if q.shape[1] * 2 != K or Y.shape != (M, N):
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, q {tuple(q.shape)}, Y {tuple(Y.shape)}")
    if not q.is_contiguous() or not s.is_contiguous() or s.shape != (N, K // 16):
        raise ValueError("q/s must be contiguous [N, K/2] / [N, K/16]")
    flags = FLAG_STATIC_WEIGHTS if static_weights else 0
    dev = _device(X, q, s, g, Y)  # the built-in scratch of this device is used
    _call("nvfp4_gemm_noalloc", dev, _ptr(X), X.stride(0), _ptr(q), _ptr(s), _ptr(g), _ptr(Y), Y.stride(0), M, N,
          K, flags, _stream(stream, dev))


# ------------------------------------------------------ allocating helpers

def quantize_new(w: torch.Tensor, amax: torch.Tensor | None = None, stream=None):
    """Allocate q, s, g on w's device and quantize into them."""
    if stream is not None:
        return _on_stream(stream, w.device, quantize_new, w, amax=amax)
    N, K = w.shape
    q = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    s = torch.empty((N, K // 16), dtype=torch.uint8, device=w.device)
    g = torch.empty((1,), dtype=torch.float32, device=w.device)
    quantize(w, q, s, g, amax=amax)
    return q, s, g


def linear(X: torch.Tensor, q: torch.Tensor, s: torch.Tensor, g: torch.Tensor, stream=None) -> torch.Tensor:
    """Allocate Y and run the GEMM (the GEMV when X has one row)."""
    if stream is not None:
        return _on_stream(stream, X.device, linear, X, q, s, g)
    X2 = X if X.dim() == 2 else X.reshape(1, -1)
    Y = torch.empty((X2.shape[0], q.shape[0]), dtype=torch.bfloat16, device=X.device)
    n_ws = gemm_workspace_size(X2.shape[0], q.shape[0], X2.shape[1])
    ws = torch.empty((n_ws,), dtype=torch.uint8, device=X.device) if n_ws else None
    gemm(X2, q, s, g, Y, workspace=ws)
    return Y if X.dim() == 2 else Y.reshape(-1)


# ---------------------------------------------------------------------- MXFP4
# imp docs/quantization.md, MXFP4 paragraph: NVFP4's nibble layout with one UE8M0
# micro-scale per 32 elements and no tensor scale (include/mxfp4.h).

def mx_quantize(w: torch.Tensor, q: torch.Tensor, s: torch.Tensor, stream=None) -> None:
    """Round-to-nearest MXFP4 of BF16 w [N, K] into q [N, K/2] and s [N, K/32]."""
    _need(w, torch.bfloat16, "w", 2)
    _need(q, torch.uint8, "q", 2)
    _need(s, torch.uint8, "s", 2)
    N, K = w.shape
    if w.stride(1) != 1 or not q.is_contiguous() or not s.is_contiguous():
        raise ValueError("w rows and q, s must be contiguous")
    if q.shape != (N, K // 2) or s.shape != (N, K // 32):
        raise ValueError("q/s must be [N, K/2] / [N, K/32]")
    dev = _device(w, q, s)
    _call("mxfp4_quantize", dev, _ptr(w), N, K, w.stride(0), _ptr(q), _ptr(s), _stream(stream, dev))


def mx_quantize_new(w: torch.Tensor, stream=None):
    """Allocate q, s on w's device and MXFP4-quantize into them."""
    if stream is not None:
        return _on_stream(stream, w.device, mx_quantize_new, w)
    N, K = w.shape
    q = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    s = torch.empty((N, K // 32), dtype=torch.uint8, device=w.device)
    mx_quantize(w, q, s)
    return q, s


def mx_gemv(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, y: torch.Tensor, stream=None,
            static_weights: bool = False, k_split: int = 0) -> None:
    """y[N] = bf16(W_deq . x) for MXFP4 weights and BF16 x [K]; k_split as for gemv()."""
    _need(x, torch.bfloat16, "x")
    _need(q, torch.uint8, "q", 2)
    _need(s, torch.uint8, "s", 2)
    _need(y, torch.bfloat16, "y")
    N, K = q.shape[0], q.shape[1] * 2
    if x.numel() != K or y.numel() != N or not x.is_contiguous() or not y.is_contiguous():
        raise ValueError("x must hold K and y N contiguous elements")
    if not q.is_contiguous() or not s.is_contiguous() or s.shape != (N, K // 32):
        raise ValueError("q/s must be contiguous [N, K/2] / [N, K/32]")
    flags = (FLAG_STATIC_WEIGHTS if static_weights else 0) | _ksplit_flag(k_split)
    dev = _device(x, q, s, y)
    _call("mxfp4_gemv_ex", dev, _ptr(x), _ptr(q), _ptr(s), _ptr(y), N, K, flags, _stream(stream, dev))


# ------------------------------------------------------------ grouped (MoE) GEMV

def gemv_grouped(X: torch.Tensor, q: torch.Tensor, s: torch.Tensor, g: torch.Tensor, expert_ids: torch.Tensor,
                 token_ids: torch.Tensor, Y: torch.Tensor, stream=None) -> None:
    """Y[p] = bf16(g[e] * W_deq[e] . X[t]) for e = expert_ids[p], t = token_ids[p]
    with stacked experts q [E, N, K/2], s [E, N, K/16], g [E] (imp docs/quantization.md,
    MoE layers: one contiguous [ne, N, K_packed] buffer per projection)."""
    _need(X, torch.bfloat16, "X", 2)
    _need(q, torch.uint8, "q", 3)
    _need(s, torch.uint8, "s", 3)
    _need(g, torch.float32, "g")
    _need(expert_ids, torch.int32, "expert_ids")
    _need(token_ids, torch.int32, "token_ids")
    _need(Y, torch.bfloat16, "Y", 2)
    E, N, K = q.shape[0], q.shape[1], q.shape[2] * 2
    T, P = X.shape[0], expert_ids.numel()
    if X.shape[1] != K or X.stride(1) != 1 or Y.stride(1) != 1 or Y.shape != (P, N):
        raise ValueError("X must be [T, K] and Y [P, N] with unit column stride")
    if not q.is_contiguous() or not s.is_contiguous() or s.shape != (E, N, K // 16) or g.numel() != E:
        raise ValueError("q/s/g must be contiguous [E, N, K/2] / [E, N, K/16] / [E]")
    if token_ids.numel() != P or not expert_ids.is_contiguous() or not token_ids.is_contiguous():
        raise ValueError("expert_ids and token_ids must be contiguous [P]")
    dev = _device(X, q, s, g, expert_ids, token_ids, Y)
    _call("nvfp4_gemv_grouped", dev,
          _ptr(X), X.stride(0), _ptr(q), _ptr(s), _ptr(g), _ptr(expert_ids), _ptr(token_ids), _ptr(Y), Y.stride(0),
          P, E, T, N, K, 0, _stream(stream, dev))


def mx_to_nvfp4(q: torch.Tensor, s_mx: torch.Tensor, stream=None):
    """MXFP4 scales s_mx [N, K/32] restated as NVFP4 scales [N, K/16] and a
    power-of-two tensor scale g [1] (exact within 17 binades; see
    include/mxfp4.h), so that (q, s_nv, g) runs on gemv/gemm."""
    _need(q, torch.uint8, "q", 2)
    _need(s_mx, torch.uint8, "s_mx", 2)
    N, K = q.shape[0], q.shape[1] * 2
    if not q.is_contiguous() or not s_mx.is_contiguous() or s_mx.shape != (N, K // 32):
        raise ValueError("q/s_mx must be contiguous [N, K/2] / [N, K/32]")
    dev = _device(q, s_mx)
    if stream is not None:
        return _on_stream(stream, dev, mx_to_nvfp4, q, s_mx)
    s_nv = torch.empty((N, K // 16), dtype=torch.uint8, device=q.device)
    g = torch.empty((1,), dtype=torch.float32, device=q.device)
    _call("mxfp4_to_nvfp4_scales", dev, _ptr(q), _ptr(s_mx), N, K, _ptr(s_nv), _ptr(g), _stream(stream, dev))
    return s_nv, g


# ----------------------------------------------------------------------- W4A4
# NVFP4 x NVFP4 prefill (include/nvfp4_w4a4.h): activations quantized by the
# weights' rule, block-scaled FP4 tensor-core GEMM.

GIVEN_AMAX = 2  # NVFP4_W4A4_GIVEN_AMAX
AMAX_FLOATS = 260  # NVFP4_W4A4_AMAX_FLOATS: the x_amax buffer of a dynamic quantize


def w4a4_prepare_weights(s: torch.Tensor, K: int, stream=None) -> torch.Tensor:
    """Row-major weight scales [N, K/16] -> the tensor-core scale layout (u8)."""
    _need(s, torch.uint8, "s", 2)
    N = s.shape[0]
    if not s.is_contiguous() or s.shape[1] * 16 != K:
        raise ValueError("s must be contiguous [N, K/16]")
    dev = _device(s)
    if stream is not None:
        return _on_stream(stream, dev, w4a4_prepare_weights, s, K)
    out = torch.empty((lib.nvfp4_w4a4_weight_scales_bytes(N, K),), dtype=torch.uint8, device=s.device)
    _call("nvfp4_w4a4_prepare_weights", dev, _ptr(s), N, K, _ptr(out), _stream(stream, dev))
    return out


def w4a4_quantize_x(X: torch.Tensor, x_amax: torch.Tensor, given_amax: bool = False, stream=None):
    """X [M, K] -> (qx [M, K/2], sx in the tensor-core scale layout).  x_amax:
    given_amax: [1] (or longer), read; else [AMAX_FLOATS], x_amax[0] receives
    max |X|."""
    _need(X, torch.bfloat16, "X", 2)
    _need(x_amax, torch.float32, "x_amax")
    if not given_amax and x_amax.numel() < AMAX_FLOATS:
        raise ValueError(f"x_amax needs {AMAX_FLOATS} floats for a dynamic amax")
    M, K = X.shape
    if X.stride(1) != 1:
        raise ValueError("X rows must be contiguous")
    ldx = X.stride(0)
    dev = _device(X, x_amax)
    if stream is not None:
        return _on_stream(stream, dev, w4a4_quantize_x, X, x_amax, given_amax=given_amax)
    qx = torch.empty((M, K // 2), dtype=torch.uint8, device=X.device)
    sx = torch.empty((lib.nvfp4_w4a4_x_scales_bytes(M, K),), dtype=torch.uint8, device=X.device)
    _call("nvfp4_w4a4_quantize_x", dev, _ptr(X), ldx, M, K, _ptr(qx), _ptr(sx), _ptr(x_amax),
          GIVEN_AMAX if given_amax else 0, _stream(stream, dev))
    return qx, sx


def _need_w4a4_weights(q: torch.Tensor, s_mma: torch.Tensor, g: torch.Tensor):
    """q [N, K/2] contiguous, s_mma holding the rearranged scales of [N, K/16]
    (w4a4_prepare_weights), g an fp32 tensor scale.  Returns (N, K)."""
    _need(q, torch.uint8, "q", 2)
    _need(s_mma, torch.uint8, "s_mma")
    _need(g, torch.float32, "g")
    if not q.is_contiguous() or not s_mma.is_contiguous():
        raise ValueError("q and s_mma must be contiguous")
    N, K = q.shape[0], q.shape[1] * 2
    if s_mma.numel() < lib.nvfp4_w4a4_weight_scales_bytes(N, K):
        raise ValueError(f"s_mma holds {s_mma.numel()} bytes, [{N}, {K}] needs "
                         f"{lib.nvfp4_w4a4_weight_scales_bytes(N, K)} (w4a4_prepare_weights)")
    return N, K


def w4a4_gemm(qx, sx, x_amax, q, s_mma, g, Y, stream=None, static_weights: bool = False, pair: bool = False) -> None:
    """Y [M, N] = bf16(g * (x_amax[0] / 2688) * Xq . Wq^T) from quantized
    activations (qx, sx, x_amax from w4a4_quantize_x) and weights (q, s_mma
    from w4a4_prepare_weights, g).  pair: tiles of 256 weight rows on pairs
    of SMs (NVFP4_FLAG_W4A4_PAIR)."""
    _need(Y, torch.bfloat16, "Y", 2)
    _need(qx, torch.uint8, "qx", 2)
    _need(sx, torch.uint8, "sx")
    _need(x_amax, torch.float32, "x_amax")
    N, K = _need_w4a4_weights(q, s_mma, g)
    M = Y.shape[0]
    if qx.shape != (M, K // 2) or Y.shape[1] != N or not qx.is_contiguous() or not sx.is_contiguous():
        raise ValueError(f"shape mismatch: qx {tuple(qx.shape)}, q {tuple(q.shape)}, Y {tuple(Y.shape)}")
    if sx.numel() < lib.nvfp4_w4a4_x_scales_bytes(M, K):
        raise ValueError(f"sx holds {sx.numel()} bytes, [{M}, {K}] needs {lib.nvfp4_w4a4_x_scales_bytes(M, K)}")
    flags = (FLAG_STATIC_WEIGHTS if static_weights else 0) | (FLAG_W4A4_PAIR if pair else 0)
    dev = _device(qx, sx, x_amax, q, s_mma, g, Y)
    _call("nvfp4_w4a4_gemm", dev, _ptr(qx), _ptr(sx), _ptr(x_amax), _ptr(q), _ptr(s_mma), _ptr(g), _ptr(Y),
          Y.stride(0), M, N, K, flags, _stream(stream, dev))


def w4a4_workspace_size(M: int, K: int) -> int:
    return lib.nvfp4_w4a4_workspace_size(M, K)


def w4a4_linear(X: torch.Tensor, q: torch.Tensor, s_mma: torch.Tensor, g: torch.Tensor, Y: torch.Tensor,
                workspace: torch.Tensor, x_amax: torch.Tensor | None = None, stream=None,
                static_weights: bool = False, pair: bool = False) -> None:
    """Y [M, N] = W4A4 product of BF16 X [M, K] (quantized on the fly into the
    workspace) and NVFP4 weights (q, s_mma from w4a4_prepare_weights, g)."""
    _need(X, torch.bfloat16, "X", 2)
    _need(Y, torch.bfloat16, "Y", 2)
    _need(workspace, torch.uint8, "workspace")
    if x_amax is not None:
        _need(x_amax, torch.float32, "x_amax")
    N, Kq = _need_w4a4_weights(q, s_mma, g)
    M, K = X.shape
    if Kq != K or Y.shape != (M, N):
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, q {tuple(q.shape)}, Y {tuple(Y.shape)}")
    flags = (FLAG_STATIC_WEIGHTS if static_weights else 0) | (FLAG_W4A4_PAIR if pair else 0)
    if X.stride(1) != 1:
        raise ValueError("X rows must be contiguous")
    dev = _device(X, x_amax, q, s_mma, g, Y, workspace)
    _call("nvfp4_w4a4_linear", dev, _ptr(X), X.stride(0), _ptr(x_amax), _ptr(q), _ptr(s_mma), _ptr(g), _ptr(Y),
          Y.stride(0), M, N, K, _ptr(workspace), workspace.numel(), flags, _stream(stream, dev))


# ------------------------------------------------------------------------ FP8
# 8-bit linear layer (include/fp8.h): E4M3 values with one fp32 scale per row
# and 128 columns (activations) or per 128 x 128 block (weights).

FLAG_FP8_GATED = 2
_F8 = torch.float8_e4m3fn


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _first(t: torch.Tensor, dtype, what: str, ndim: int):
    """Shape, device, address and leading dimension of the tensor that a call's
    other tensors are checked against."""
    _need(t, dtype, what, ndim)
    shape = t.shape
    # (the stride of a single row says nothing)
    return shape, t.device, t.data_ptr(), t.stride(0) if shape[0] > 1 else shape[-1]


def _rows(t: torch.Tensor, dtype, what: str, shape, dev: torch.device):
    """Address and leading dimension of 2-D `t` of the given shape."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev.index):
        _need(t, dtype, what, 2)
        raise ValueError(f"{what} is on {t.device}, not on {dev}")
    if t.shape != shape:
        raise ValueError(f"{what} must be {tuple(shape)}, got {tuple(t.shape)}")
    ld, step = t.stride()
    if step != 1:
        _need(t, dtype, what, 2)
    return t.data_ptr(), ld if shape[0] > 1 else shape[1]


def _dense(t: torch.Tensor, dtype, what: str, shape, dev: torch.device) -> int:
    """Address of contiguous `t` of the given shape."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev.index):
        _need(t, dtype, what)
        raise ValueError(f"{what} is on {t.device}, not on {dev}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


_BF16, _F32 = torch.bfloat16, torch.float32


def fp8_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
                residual_out: torch.Tensor | None = None, y: torch.Tensor | None = None,
                q: torch.Tensor | None = None, s: torch.Tensor | None = None, stream=None) -> None:
    """RMS norm of BF16 x [M, K] (+ residual) times weight [K].  With a residual,
    residual_out (default: residual itself, in place) receives bf16(x + residual),
    which is what is normed.  Outputs, at least one: y BF16 [M, K], and
    q float8_e4m3fn [M, K] with s float32 [M, ceil(K/128)]."""
    shape, dev, px, ldx = _first(x, _BF16, "x", 2)
    M, K = shape
    pw = _dense(weight, _BF16, "weight", (K,), dev)
    pr = po = py = pq = ps = None
    ldr = ldo = ldy = 0
    if residual is not None:
        pr, ldr = _rows(residual, _BF16, "residual", shape, dev)
        po, ldo = (pr, ldr) if residual_out is None else _rows(residual_out, _BF16, "residual_out", shape, dev)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if y is not None:
        py, ldy = _rows(y, _BF16, "y", shape, dev)
    if (q is None) != (s is None):
        raise ValueError("q and s go together")
    if q is not None:
        pq = _dense(q, _F8, "q", shape, dev)
        ps = _dense(s, _F32, "s", (M, (K + 127) // 128), dev)
    _call("fp8_rmsnorm", dev, px, ldx, pw, pr, ldr, po, ldo, py, ldy, pq, ps, M, K, eps, _stream(stream, dev))


def fp8_quantize(X: torch.Tensor, q: torch.Tensor, s: torch.Tensor, gated: bool = False, stream=None) -> None:
    """BF16 activations X [M, K] into q float8_e4m3fn [M, K] and s float32 [M, ceil(K/128)].
    gated: X is [M, 2K], gate then up columns, and silu(gate) * up is quantized."""
    (M, K), dev, px, ldx = _first(X, _BF16, "X", 2)
    if gated:
        if K % 2:
            raise ValueError(f"a gated X has an even number of columns, got {K}")
        K //= 2
    _call("fp8_quantize", dev, px, ldx, M, K, _dense(q, _F8, "q", (M, K), dev),
          _dense(s, _F32, "s", (M, (K + 127) // 128), dev), FLAG_FP8_GATED if gated else 0, _stream(stream, dev))


def fp8_quantize_weights(W: torch.Tensor, q: torch.Tensor, s: torch.Tensor, stream=None) -> None:
    """BF16 weights W [N, K] into q float8_e4m3fn [N, K] and s float32 [ceil(N/128), ceil(K/128)]."""
    (N, K), dev, pw, ldw = _first(W, _BF16, "W", 2)
    _call("fp8_quantize_weights", dev, pw, ldw, N, K, _dense(q, _F8, "q", (N, K), dev),
          _dense(s, _F32, "s", (_blocks(N), _blocks(K)), dev), _stream(stream, dev))


def fp8_gemm(x: torch.Tensor, sx: torch.Tensor, w: torch.Tensor, sw: torch.Tensor, Y: torch.Tensor, stream=None,
             static_weights: bool = False) -> None:
    """Y [M, N] = bf16((x * sx) . (w * sw)^T): activations x [M, K], sx [M, ceil(K/128)]
    (fp8_quantize, fp8_rmsnorm), weights w [N, K], sw [ceil(N/128), ceil(K/128)]
    (fp8_quantize_weights).  static_weights: w is not written by work still
    running on the stream (NVFP4_FLAG_STATIC_WEIGHTS)."""
    (M, K), dev, _, _ = _first(x, _F8, "x", 2)
    _need(w, _F8, "w", 2)
    N, kb = w.shape[0], (K + 127) // 128
    py, ldy = _rows(Y, _BF16, "Y", (M, N), dev)
    _call("fp8_gemm", dev, _dense(x, _F8, "x", (M, K), dev), _dense(sx, _F32, "sx", (M, kb), dev),
          _dense(w, _F8, "w", (N, K), dev), _dense(sw, _F32, "sw", ((N + 127) // 128, kb), dev), py, ldy, M, N, K,
          FLAG_STATIC_WEIGHTS if static_weights else 0, _stream(stream, dev))


def fp8_gemm_grouped(x: torch.Tensor, sx: torch.Tensor, w: torch.Tensor, sw: torch.Tensor, offsets: torch.Tensor,
                     Y: torch.Tensor, stream=None, static_weights: bool = False) -> None:
    """fp8_gemm by expert: rows offsets[e] .. offsets[e+1]-1 of x [T, K] and Y [T, N]
    belong to expert e of w [E, N, K], sw [E, ceil(N/128), ceil(K/128)].  offsets:
    int32 [E + 1] on the device, not decreasing.  Rows of Y outside
    offsets[0] .. offsets[E]-1 keep what they hold."""
    (E, N, K), dev, _, _ = _first(w, _F8, "w", 3)
    _need(x, _F8, "x", 2)
    T, kb = x.shape[0], (K + 127) // 128
    py, ldy = _rows(Y, _BF16, "Y", (T, N), dev)
    _call("fp8_gemm_grouped", dev, _dense(x, _F8, "x", (T, K), dev), _dense(sx, _F32, "sx", (T, kb), dev),
          _dense(w, _F8, "w", (E, N, K), dev), _dense(sw, _F32, "sw", (E, (N + 127) // 128, kb), dev),
          _dense(offsets, torch.int32, "offsets", (E + 1,), dev), py, ldy, T, E, N, K,
          FLAG_STATIC_WEIGHTS if static_weights else 0, _stream(stream, dev))


def fp8_quantize_new(X: torch.Tensor, gated: bool = False, stream=None):
    """Allocate q, s on X's device and quantize activations into them."""
    if stream is not None:
        return _on_stream(stream, X.device, fp8_quantize_new, X, gated=gated)
    M, K = X.shape[0], X.shape[1] // 2 if gated else X.shape[1]
    q = torch.empty((M, K), dtype=_F8, device=X.device)
    s = torch.empty((M, _blocks(K)), dtype=torch.float32, device=X.device)
    fp8_quantize(X, q, s, gated=gated)
    return q, s


def fp8_quantize_weights_new(W: torch.Tensor, stream=None):
    """Allocate q, s on W's device and quantize weights into them."""
    if stream is not None:
        return _on_stream(stream, W.device, fp8_quantize_weights_new, W)
    N, K = W.shape
    q = torch.empty((N, K), dtype=_F8, device=W.device)
    s = torch.empty((_blocks(N), _blocks(K)), dtype=torch.float32, device=W.device)
    fp8_quantize_weights(W, q, s)
    return q, s


def fp8_linear(X: torch.Tensor, w: torch.Tensor, sw: torch.Tensor, stream=None) -> torch.Tensor:
    """Quantize BF16 X [M, K] and multiply by 8-bit weights: allocates and returns Y [M, N]."""
    if stream is not None:
        return _on_stream(stream, X.device, fp8_linear, X, w, sw)
    X2 = X if X.dim() == 2 else X.reshape(1, -1)
    q, s = fp8_quantize_new(X2)
    Y = torch.empty((X2.shape[0], w.shape[0]), dtype=torch.bfloat16, device=X.device)
    fp8_gemm(q, s, w, sw, Y)
    return Y if X.dim() == 2 else Y.reshape(-1)
