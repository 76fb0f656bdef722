"""moe_ffn_gb300 — Python binding of libqmoe.so, the GB300 (sm_103a) GGUF
block-quantized GEMV and decode-time MoE FFN library.

This module only marshals arguments: every step of every call runs in the
library's CUDA kernels.  PyTorch supplies device memory (``tensor.data_ptr()``)
and streams (``torch.cuda.current_stream().cuda_stream``).  There is no CPU
fallback: if the compiled library is missing, loading it raises.

Function names follow the C ABI declared in ``include/qmoe.h``.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import subprocess
import sysconfig
import threading
import warnings

_HERE = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_HERE)
_CSRC = os.path.join(_HERE, "csrc")
LIB_PATH = os.path.join(_HERE, "libqmoe.so")
HEADER = os.path.join(_ROOT, "include", "qmoe.h")
# csrc/calls.c, the short way into the library, for this interpreter
CALLS_PATH = os.path.join(_HERE, "_calls" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

# qmoe_qtype
F32, Q8_0, Q4_0, Q4_K, Q5_K, Q6_K = 0, 1, 2, 3, 4, 5
QTYPES = {"F32": F32, "Q8_0": Q8_0, "Q4_0": Q4_0, "Q4_K": Q4_K, "Q5_K": Q5_K, "Q6_K": Q6_K}
BLOCK_ELEMS = {F32: 1, Q8_0: 32, Q4_0: 32, Q4_K: 256, Q5_K: 256, Q6_K: 256}
BLOCK_BYTES = {F32: 4, Q8_0: 34, Q4_0: 18, Q4_K: 144, Q5_K: 176, Q6_K: 210}

# element types beside F32
BF16, F16, E4M3 = 32, 33, 34

# qmoe_status
OK, ERR_INVALID_ARGUMENT, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT = 0, 1, 2, 3, 4
STATUS_NAMES = {0: "OK", 1: "INVALID_ARGUMENT", 2: "UNSUPPORTED", 3: "CUDA", 4: "TIMEOUT"}

NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-ftz=false",
              "-std=c++17", "-Xcompiler", "-fPIC"]
# Translation units of libqmoe.so, compiled in parallel and linked together.
UNITS = ("qmoe.cu", "batch.cu", "f8.cu", "moe_steps.cu", "w4.cu")


class QmoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")


def _sources(*endings):
    return sorted(os.path.join(_CSRC, f) for f in os.listdir(_CSRC) if f.endswith(endings))


def _stale(path: str, sources) -> bool:
    return not os.path.exists(path) or os.path.getmtime(path) < max(
        os.path.getmtime(s) for s in (*sources, HEADER))


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libqmoe.so in-tree for sm_103a with nvcc, and the binding's C module with
    the C compiler.  Where the module does not compile (no headers of the interpreter)
    the library is there all the same, and calls go through ctypes."""
    calls = None
    if force or _stale(CALLS_PATH, _sources(".c")):
        calls = _start_calls(verbose)
    try:
        if force or _stale(LIB_PATH, _sources(".cu", ".cuh")):
            _build_lib(verbose)
    finally:
        if calls is not None:
            _finish_calls(*calls)
    return LIB_PATH


def _build_lib(verbose: bool) -> None:
    nvcc = os.environ.get("NVCC", "nvcc")
    if not os.path.exists(nvcc) and os.path.exists("/usr/local/cuda/bin/nvcc"):
        nvcc = "/usr/local/cuda/bin/nvcc"
    objs = [os.path.join(_HERE, u.replace(".cu", f".{os.getpid()}.o")) for u in UNITS]
    procs = []
    for u, o in zip(UNITS, objs):
        cmd = [nvcc, *NVCC_FLAGS, "-c", "-o", o, os.path.join(_CSRC, u)]
        if verbose:
            print(" ".join(cmd))
        procs.append(subprocess.Popen(cmd))
    codes = [p.wait() for p in procs]
    try:
        for u, c in zip(UNITS, codes):
            if c:
                raise subprocess.CalledProcessError(c, f"nvcc {u}")
        tmp = LIB_PATH + f".{os.getpid()}.tmp"
        cmd = [nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-shared", "-o", tmp, *objs]
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB_PATH)
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)


def _start_calls(verbose: bool):
    """(the compiler's process or None, its output file)"""
    tmp = CALLS_PATH + f".{os.getpid()}.tmp"
    cmd = [os.environ.get("CC", "gcc"), "-O2", "-shared", "-fPIC",
           "-I" + sysconfig.get_paths()["include"], "-o", tmp, os.path.join(_CSRC, "calls.c")]
    if verbose:
        print(" ".join(cmd))
    try:
        return subprocess.Popen(cmd), tmp
    except OSError:
        return None, tmp


def _finish_calls(proc, tmp: str) -> None:
    global _calls
    if proc is not None and proc.wait() == 0:
        os.replace(tmp, CALLS_PATH)
        if _calls is _LONG_WAY:
            _calls = None
        return
    for f in (tmp, CALLS_PATH):  # (one of older sources would not fit the library)
        if os.path.exists(f):
            os.remove(f)
    warnings.warn("csrc/calls.c could not be compiled: calls go through ctypes, which costs the "
                  "host about 4 us more each", RuntimeWarning, stacklevel=3)


class _Shape(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("expert_dim", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("n_tokens", ctypes.c_int32), ("gate_qtype", ctypes.c_int32),
                ("up_qtype", ctypes.c_int32), ("down_qtype", ctypes.c_int32),
                ("route_flags", ctypes.c_int32)]


_lock = threading.Lock()
_libh = None

# Exported symbols and their ctypes signatures (mirrors include/qmoe.h).
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
SIGNATURES = {
    "qmv": (ctypes.c_int, [ctypes.c_int, _P, _I64, _I64, _P, _P, _P]),
    "ffn_swiglu_workspace_size": (ctypes.c_size_t, [_I64, _I64]),
    "ffn_swiglu": (ctypes.c_int, [_P, _P, _P, ctypes.c_int, ctypes.c_int, ctypes.c_int, _I64, _I64,
                                  _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_ffn_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(_Shape)]),
    "moe_ffn": (ctypes.c_int, [_P, _P, _P, _P, ctypes.POINTER(_Shape), _P, _P, _P, _P, _P,
                               ctypes.c_size_t, _P]),
    "moe_ffn_noalloc": (ctypes.c_int, [_P, _P, _P, _P, ctypes.POINTER(_Shape), _P, _P, _P, _P,
                                        _P]),
    "ffn_swiglu_rmsnorm_workspace_size": (ctypes.c_size_t, [_I64, _I64]),
    "ffn_swiglu_rmsnorm": (ctypes.c_int, [_P, _P, _P, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                          _I64, _I64, _P, ctypes.c_float, _P, _P, ctypes.c_size_t,
                                          _P]),
    "moe_ffn_rmsnorm_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(_Shape)]),
    "moe_ffn_rmsnorm": (ctypes.c_int, [_P, _P, _P, _P, ctypes.POINTER(_Shape), _P, ctypes.c_float,
                                       _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "f8_quantize": (ctypes.c_int, [ctypes.c_int, _P, _I64, _I64, _I64, _P, _P, _P]),
    "f8_mm": (ctypes.c_int, [_P, _P, _I64, _I64, _P, _P, _I64, _I64, ctypes.c_int, _P, _I64, _P]),
    "mm_grouped": (ctypes.c_int, [ctypes.c_int, _P, _P, ctypes.c_int32, _I64, _I64, _P, _P, _I64,
                                  _I64, _P, ctypes.c_int, _P, _I64, _P]),
    "moe_experts_f8_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(_Shape)]),
    "moe_experts_f8": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, ctypes.POINTER(_Shape),
                                      ctypes.c_int, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_route": (ctypes.c_int, [ctypes.c_int, _P, _I64, ctypes.c_int32, _I64, ctypes.c_int32,
                                 ctypes.c_int32, _P, _P, _P]),
    "moe_route_backward": (ctypes.c_int, [ctypes.c_int, _P, _I64, ctypes.c_int32, _I64,
                                          ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P, _I64,
                                          _P]),
    "moe_permute_workspace_size": (ctypes.c_size_t, [_I64, ctypes.c_int32, ctypes.c_int32]),
    "moe_permute": (ctypes.c_int, [ctypes.c_int, _P, _I64, _I64, _I64, _P, ctypes.c_int32,
                                   ctypes.c_int32, _P, _I64, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_combine": (ctypes.c_int, [ctypes.c_int, _P, _I64, _I64, _I64, _P, _P, _I64,
                                   ctypes.c_int32, ctypes.c_int, _P, _P, _I64, _P]),
    "moe_combine_backward": (ctypes.c_int, [ctypes.c_int, _P, _I64, _I64, _I64, _P, _P, _I64,
                                            ctypes.c_int32, ctypes.c_int, _P, _I64, _P, _I64, _P,
                                            _P]),
    "w4_mm": (ctypes.c_int, [_P, ctypes.c_int, _P, _P, ctypes.c_int32, _I64, _I64, ctypes.c_int,
                             _P, _I64, _I64, ctypes.c_int, _P, _I64, _P]),
    "w4_mm_grouped": (ctypes.c_int, [_P, ctypes.c_int, _P, _P, ctypes.c_int32, ctypes.c_int32,
                                     _I64, _I64, ctypes.c_int, _P, _I64, _I64, _P, ctypes.c_int,
                                     _P, _I64, _P]),
    "qmoe_device_status": (ctypes.c_int, [_P]),
    "qmoe_set_exec_mode": (ctypes.c_int, [ctypes.c_int]),
    "qmoe_set_fault_injection": (ctypes.c_int, [ctypes.c_uint64, ctypes.c_int]),
    "qmoe_last_error": (ctypes.c_char_p, []),
    "qmoe_row_bytes": (_I64, [ctypes.c_int, _I64]),
}


def lib():
    """The loaded library; raises if it has not been built."""
    global _libh
    with _lock:
        if _libh is None:
            if not os.path.exists(LIB_PATH):
                raise QmoeError(ERR_CUDA, f"{LIB_PATH} is missing: run moe_ffn_gb300.build()")
            h = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(h, name)
                fn.restype = res
                fn.argtypes = args
            _libh = h
    return _libh


def last_error() -> str:
    return lib().qmoe_last_error().decode()


def _check(status: int):
    if status != OK:
        raise QmoeError(status, last_error())


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def row_bytes(qtype: int, cols: int) -> int:
    return int(lib().qmoe_row_bytes(qtype, cols))


def qmv(qtype: int, W, rows: int, cols: int, x, y, stream=None) -> None:
    """y = W x (see include/qmoe.h)."""
    _check(lib().qmv(qtype, _ptr(W), rows, cols, _ptr(x), _ptr(y), _stream(stream)))


def ffn_swiglu_workspace_size(hidden: int, inter: int) -> int:
    return int(lib().ffn_swiglu_workspace_size(hidden, inter))


def ffn_swiglu(gate, up, down, gate_qtype, up_qtype, down_qtype, hidden, inter, x, residual,
               ws, ws_bytes=None, stream=None) -> None:
    """residual += down(silu(gate x) * (up x)) (see include/qmoe.h)."""
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    _check(lib().ffn_swiglu(_ptr(gate), _ptr(up), _ptr(down), gate_qtype, up_qtype, down_qtype,
                            hidden, inter, _ptr(x), _ptr(residual), _ptr(ws), ws_bytes,
                            _stream(stream)))


# shape.route_flags: routing weights are the softmax probabilities, not renormalised
ROUTE_NO_RENORM = 1


def moe_shape(hidden, expert_dim, num_experts, top_k, n_tokens, gate_qtype, up_qtype,
              down_qtype, renormalize: bool = True) -> _Shape:
    return _Shape(hidden, expert_dim, num_experts, top_k, n_tokens, gate_qtype, up_qtype,
                  down_qtype, 0 if renormalize else ROUTE_NO_RENORM)


def moe_ffn_workspace_size(shape: _Shape) -> int:
    return int(lib().moe_ffn_workspace_size(ctypes.byref(shape)))


def moe_ffn(router_W, gate_stack, up_stack, down_stack, shape: _Shape, x, residual,
            topk_idx=None, topk_w=None, ws=None, ws_bytes=None, stream=None) -> None:
    """One MoE FFN layer for shape.n_tokens tokens (see include/qmoe.h)."""
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    _check(lib().moe_ffn(_ptr(router_W), _ptr(gate_stack), _ptr(up_stack), _ptr(down_stack),
                         ctypes.byref(shape), _ptr(x), _ptr(residual), _ptr(topk_idx),
                         _ptr(topk_w), _ptr(ws), ws_bytes, _stream(stream)))


def ffn_swiglu_rmsnorm_workspace_size(hidden: int, inter: int) -> int:
    return int(lib().ffn_swiglu_rmsnorm_workspace_size(hidden, inter))


def ffn_swiglu_rmsnorm(gate, up, down, gate_qtype, up_qtype, down_qtype, hidden, inter, norm_w,
                       eps, residual, ws, ws_bytes=None, stream=None) -> None:
    """residual += FFN(rmsnorm(residual)) (see include/qmoe.h)."""
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    _check(lib().ffn_swiglu_rmsnorm(_ptr(gate), _ptr(up), _ptr(down), gate_qtype, up_qtype,
                                    down_qtype, hidden, inter, _ptr(norm_w), float(eps),
                                    _ptr(residual), _ptr(ws), ws_bytes, _stream(stream)))


def moe_ffn_rmsnorm_workspace_size(shape: _Shape) -> int:
    return int(lib().moe_ffn_rmsnorm_workspace_size(ctypes.byref(shape)))


def moe_ffn_rmsnorm(router_W, gate_stack, up_stack, down_stack, shape: _Shape, norm_w, eps,
                    residual, topk_idx=None, topk_w=None, ws=None, ws_bytes=None,
                    stream=None) -> None:
    """residual_t += MoE(rmsnorm(residual_t)) for every token (see include/qmoe.h)."""
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    _check(lib().moe_ffn_rmsnorm(_ptr(router_W), _ptr(gate_stack), _ptr(up_stack),
                                 _ptr(down_stack), ctypes.byref(shape), _ptr(norm_w), float(eps),
                                 _ptr(residual), _ptr(topk_idx), _ptr(topk_w), _ptr(ws), ws_bytes,
                                 _stream(stream)))


NOALLOC_SCRATCH_BYTES = 1 << 20


def moe_ffn_noalloc(router_W, gate_stack, up_stack, down_stack, shape: _Shape, x, residual,
                    topk_idx=None, topk_w=None, stream=None) -> None:
    """moe_ffn without a workspace argument: for callers that cannot allocate
    device memory.  Scratch is the library's built-in array
    (NOALLOC_SCRATCH_BYTES); calls share it, so calls that overlap on the
    GPU race (see include/qmoe.h)."""
    _check(lib().moe_ffn_noalloc(_ptr(router_W), _ptr(gate_stack), _ptr(up_stack),
                                 _ptr(down_stack), ctypes.byref(shape), _ptr(x), _ptr(residual),
                                 _ptr(topk_idx), _ptr(topk_w), _stream(stream)))


# ------------------------------- e4m3 / bf16 / f16 products (include/qmoe.h)
# One-token calls take a few microseconds on the GPU, so these functions keep
# their own cost low: cheap tensor checks, and the current device and stream
# asked of torch once per call.
_I32, _U8 = -1, -2
_DTYPES = {}


def _context(stream):
    """(current CUDA device or -1, stream address); an int stream is taken as is."""
    import torch
    if not _DTYPES:
        _DTYPES.update({F32: (torch.float32,), BF16: (torch.bfloat16,), F16: (torch.float16,),
                        E4M3: (torch.float8_e4m3fn, torch.uint8, torch.int8),
                        _I32: (torch.int32,), _U8: (torch.uint8,)})
    dev = torch.cuda.current_device() if torch.cuda.is_initialized() else -1
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev) if dev >= 0 else 0
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    return dev, stream


def _rows_apart(t, ld) -> bool:
    """Whether a tensor's rows are consecutive elements, `ld` apart."""
    if ld is None or t.dim() < 2 or (t.size(-1) > 1 and t.stride(-1) != 1):
        return False
    for i in range(t.dim() - 2, -1, -1):
        if t.size(i) > 1 and t.stride(i) != ld:
            return False
        ld *= t.size(i)
    return True


def _arg(fn: str, name: str, t, kind, need: int, dev: int, ld=None):
    """Address of a device array of at least `need` elements of type `kind`
    (None: any type).

    Integers (addresses) and None pass through unchecked; a tensor must live
    on the current CUDA device, have the element type the call names (one-byte
    types for E4M3) and reach `need` elements from its first one.  It must be
    contiguous; rows of a strided argument may lie `ld` apart."""
    if t is None or isinstance(t, int):
        return t
    if not t.is_cuda or t.get_device() != dev:
        raise QmoeError(ERR_INVALID_ARGUMENT,
                        f"{fn}: {name} is on {t.device}, not on the current CUDA device")
    # (an unknown type number is left to the library, which refuses it)
    if kind in _DTYPES and t.dtype not in _DTYPES[kind]:
        raise QmoeError(ERR_INVALID_ARGUMENT,
                        f"{fn}: {name} has dtype {t.dtype}, not {_DTYPES[kind][0]}")
    dense = t.is_contiguous()
    if not (dense or _rows_apart(t, ld)):
        raise QmoeError(ERR_INVALID_ARGUMENT,
                        f"{fn}: {name} has strides {tuple(t.stride())}, which are not those of "
                        + ("a contiguous array" if ld is None else f"rows {ld} apart"))
    if not (dense and t.numel() >= need):
        have = t.untyped_storage().nbytes() // t.element_size() - t.storage_offset()
        if have < need:
            raise QmoeError(ERR_INVALID_ARGUMENT,
                            f"{fn}: {name} holds {have} elements, {need} are needed")
    return t.data_ptr()


def _span(rows: int, cols: int, ld: int) -> int:
    return (rows - 1) * ld + cols if rows > 0 else 0


def _fit(fn: str, small, large=(), nbytes: int = 0) -> None:
    """Refuses integers that ctypes would cut to 32 (`small`) or 64 bits (`large`), or take
    for a huge number of bytes: the library would go by another type or size than the one
    the arrays were checked for.  (Callers first look at the OR of all of them, which is
    nearly always 0 to 2^31 - 1.)"""
    for bits, values in ((32, small), (64, large)):
        for v in values:
            if not -1 << bits - 1 <= v < 1 << bits - 1:
                raise QmoeError(ERR_INVALID_ARGUMENT, f"{fn}: {v} does not fit {bits} bits")
    if not 0 <= nbytes < 1 << 63:
        raise QmoeError(ERR_INVALID_ARGUMENT, f"{fn}: ws_bytes={nbytes} does not fit a size")


def f8_blocks(n: int) -> int:
    """Blocks of 128 that cover n elements (scales per row, or per column)."""
    return -(-n // 128)


def f8_quantize(xtype: int, x, rows: int, cols: int, q, scale, ldx=None, stream=None) -> None:
    """q, scale = e4m3 rows of x with one scale per 128 columns (see include/qmoe.h)."""
    fn, ldx = "f8_quantize", cols if ldx is None else ldx
    if (xtype | rows | cols | ldx) >> 31:
        _fit(fn, (xtype,), (rows, cols, ldx))
    dev, st = _context(stream)
    _check((_libh or lib()).f8_quantize(
        xtype, _arg(fn, "x", x, xtype, _span(rows, cols, ldx), dev, ldx), rows, cols, ldx,
        _arg(fn, "q", q, E4M3, rows * cols, dev),
        _arg(fn, "scale", scale, F32, rows * f8_blocks(cols), dev), st))


def f8_mm(W, w_scale, rows: int, cols: int, x, x_scale, n_tokens: int, ytype: int, y, ldx=None,
          ldy=None, stream=None) -> None:
    """y = x W^T with e4m3 operands and block scales (see include/qmoe.h)."""
    fn, kb = "f8_mm", f8_blocks(cols)
    ldx, ldy = cols if ldx is None else ldx, rows if ldy is None else ldy
    if (ytype | rows | cols | n_tokens | ldx | ldy) >> 31:
        _fit(fn, (ytype,), (rows, cols, n_tokens, ldx, ldy))
    dev, st = _context(stream)
    _check((_libh or lib()).f8_mm(
        _arg(fn, "W", W, E4M3, rows * cols, dev),
        _arg(fn, "w_scale", w_scale, F32, f8_blocks(rows) * kb, dev), rows, cols,
        _arg(fn, "x", x, E4M3, _span(n_tokens, cols, ldx), dev, ldx),
        _arg(fn, "x_scale", x_scale, F32, n_tokens * kb, dev), n_tokens, ldx, ytype,
        _arg(fn, "y", y, ytype, _span(n_tokens, rows, ldy), dev, ldy), ldy, st))


def mm_grouped(wtype: int, W, w_scale, num_groups: int, rows: int, cols: int, x, x_scale,
               n_rows: int, offsets, ytype: int, y, ldx=None, ldy=None, stream=None) -> None:
    """y[r] = W_g x[r] for the rows of every group (see include/qmoe.h)."""
    fn, kb = "mm_grouped", f8_blocks(cols)
    ldx, ldy = cols if ldx is None else ldx, rows if ldy is None else ldy
    if (wtype | num_groups | ytype | rows | cols | n_rows | ldx | ldy) >> 31:
        _fit(fn, (wtype, num_groups, ytype), (rows, cols, n_rows, ldx, ldy))
    dev, st = _context(stream)
    _check((_libh or lib()).mm_grouped(
        wtype, _arg(fn, "W", W, wtype, num_groups * rows * cols, dev),
        _arg(fn, "w_scale", w_scale, F32, num_groups * f8_blocks(rows) * kb, dev), num_groups,
        rows, cols, _arg(fn, "x", x, wtype, _span(n_rows, cols, ldx), dev, ldx),
        _arg(fn, "x_scale", x_scale, F32, n_rows * kb, dev), n_rows, ldx,
        _arg(fn, "offsets", offsets, _I32, num_groups + 1, dev), ytype,
        _arg(fn, "y", y, ytype, _span(n_rows, rows, ldy), dev, ldy), ldy, st))


def moe_experts_f8_workspace_size(shape: _Shape) -> int:
    n = int(lib().moe_experts_f8_workspace_size(ctypes.byref(shape)))
    if n == 0:
        raise QmoeError(ERR_INVALID_ARGUMENT, last_error())
    return n


def moe_experts_f8(gate_stack, gate_scale, up_stack, up_scale, down_stack, down_scale,
                   shape: _Shape, xtype: int, x, topk_idx, topk_w, residual, out, ws,
                   ws_bytes=None, stream=None) -> None:
    """out = residual + the routed experts' weighted outputs (see include/qmoe.h)."""
    fn = "moe_experts_f8"
    H, F, E, T = shape.hidden, shape.expert_dim, shape.num_experts, shape.n_tokens
    P, EFH, TH = T * shape.top_k, E * F * H, T * H
    blocks = E * f8_blocks(F) * f8_blocks(H)
    ws_need = 0
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    elif ws is not None and not isinstance(ws, int):
        ws_need = -(-ws_bytes // ws.element_size())
    if (xtype | ws_bytes) >> 31:
        _fit(fn, (xtype,), (), ws_bytes)
    dev, st = _context(stream)
    _check((_libh or lib()).moe_experts_f8(
        _arg(fn, "gate_stack", gate_stack, E4M3, EFH, dev),
        _arg(fn, "gate_scale", gate_scale, F32, blocks, dev),
        _arg(fn, "up_stack", up_stack, E4M3, EFH, dev),
        _arg(fn, "up_scale", up_scale, F32, blocks, dev),
        _arg(fn, "down_stack", down_stack, E4M3, EFH, dev),
        _arg(fn, "down_scale", down_scale, F32, blocks, dev), ctypes.byref(shape), xtype,
        _arg(fn, "x", x, xtype, TH, dev), _arg(fn, "topk_idx", topk_idx, _I32, P, dev),
        _arg(fn, "topk_w", topk_w, F32, P, dev), _arg(fn, "residual", residual, xtype, TH, dev),
        _arg(fn, "out", out, xtype, TH, dev), _arg(fn, "ws", ws, None, ws_need, dev), ws_bytes, st))


# ------------------- steps around the experts' products (include/qmoe.h)
# These calls first go the short way of csrc/calls.c, which answers None for whatever it
# leaves to the checks below.
class _LongWay:
    """In place of the module where it could not be built: leaves every call."""

    def __getattr__(self, name):
        return lambda *args: None


_LONG_WAY = _LongWay()
_calls = None


def _short_way():
    global _calls
    if os.path.exists(CALLS_PATH):
        return _bind_calls()
    warnings.warn(f"{CALLS_PATH} is missing (build() compiles it): calls go through ctypes",
                  RuntimeWarning, stacklevel=3)
    _calls = _LONG_WAY
    return _calls


def _bind_calls():
    """The module of csrc/calls.c, bound to the library; raises if it has not been built."""
    global _calls
    import torch
    h = lib()
    with _lock:
        if _calls is None or _calls is _LONG_WAY:
            if not os.path.exists(CALLS_PATH):
                raise QmoeError(ERR_CUDA, f"{CALLS_PATH} is missing: run moe_ffn_gb300.build()")
            spec = importlib.util.spec_from_file_location("moe_ffn_gb300._calls", CALLS_PATH)
            m = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(m)
            m.bind(tuple(ctypes.cast(getattr(h, f), _P).value for f in (
                "moe_route", "moe_route_backward", "moe_permute", "moe_combine",
                "moe_combine_backward", "w4_mm", "w4_mm_grouped")),
                (torch.float32, torch.bfloat16, torch.float16, torch.int32, torch.uint8),
                torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
            _calls = m
    return _calls


def _answered(status) -> bool:
    """Whether the short way took the call; raises for a status other than OK."""
    if status:
        raise QmoeError(status, last_error())
    return status is not None


def moe_route(ltype: int, logits, n_tokens: int, num_experts: int, top_k: int, topk_idx, topk_w,
              renormalize: bool = True, ldl=None, stream=None) -> None:
    """topk_idx, topk_w = the top-k experts of each token's logits and their softmax
    weights (see include/qmoe.h)."""
    if ldl is None and _answered((_calls or _short_way()).route(
            ltype, logits, n_tokens, num_experts, top_k, topk_idx, topk_w,
            0 if renormalize else ROUTE_NO_RENORM, stream)):
        return
    fn, ldl = "moe_route", num_experts if ldl is None else ldl
    if (ltype | num_experts | top_k | n_tokens | ldl) >> 31:
        _fit(fn, (ltype, num_experts, top_k), (n_tokens, ldl))
    dev, st = _context(stream)
    P = n_tokens * top_k
    _check((_libh or lib()).moe_route(
        ltype, _arg(fn, "logits", logits, ltype, _span(n_tokens, num_experts, ldl), dev, ldl),
        n_tokens, num_experts, ldl, top_k, 0 if renormalize else ROUTE_NO_RENORM,
        _arg(fn, "topk_idx", topk_idx, _I32, P, dev), _arg(fn, "topk_w", topk_w, F32, P, dev), st))


def moe_route_backward(ltype: int, logits, n_tokens: int, num_experts: int, top_k: int, topk_idx,
                       topk_w, grad_w, grad_logits, renormalize: bool = True, ldl=None, ldg=None,
                       stream=None) -> None:
    """grad_logits from the gradient of moe_route's weights (see include/qmoe.h)."""
    if ldl is None and ldg is None and _answered((_calls or _short_way()).route_backward(
            ltype, logits, n_tokens, num_experts, top_k, topk_idx, topk_w, grad_w, grad_logits,
            0 if renormalize else ROUTE_NO_RENORM, stream)):
        return
    fn = "moe_route_backward"
    ldl, ldg = num_experts if ldl is None else ldl, num_experts if ldg is None else ldg
    if (ltype | num_experts | top_k | n_tokens | ldl | ldg) >> 31:
        _fit(fn, (ltype, num_experts, top_k), (n_tokens, ldl, ldg))
    dev, st = _context(stream)
    P = n_tokens * top_k
    _check((_libh or lib()).moe_route_backward(
        ltype, _arg(fn, "logits", logits, ltype, _span(n_tokens, num_experts, ldl), dev, ldl),
        n_tokens, num_experts, ldl, top_k, 0 if renormalize else ROUTE_NO_RENORM,
        _arg(fn, "topk_idx", topk_idx, _I32, P, dev), _arg(fn, "topk_w", topk_w, F32, P, dev),
        _arg(fn, "grad_w", grad_w, F32, P, dev),
        _arg(fn, "grad_logits", grad_logits, ltype, _span(n_tokens, num_experts, ldg), dev, ldg),
        ldg, st))


def moe_permute_workspace_size(n_tokens: int, num_experts: int, top_k: int) -> int:
    _fit("moe_permute_workspace_size", (num_experts, top_k), (n_tokens,))
    n = int(lib().moe_permute_workspace_size(n_tokens, num_experts, top_k))
    if n == 0:
        raise QmoeError(ERR_INVALID_ARGUMENT, last_error())
    return n


def moe_permute(xtype: int, x, n_tokens: int, cols: int, topk_idx, num_experts: int, top_k: int,
                rows, offsets, pos, ws, ldx=None, ldr=None, ws_bytes=None, stream=None) -> None:
    """rows[pos[t][s]] = x[t], the rows sorted by expert (see include/qmoe.h)."""
    if ldx is None and ldr is None and ws_bytes is None and _answered((_calls or _short_way()).permute(
            xtype, x, n_tokens, cols, topk_idx, num_experts, top_k, rows, offsets, pos, ws, stream)):
        return
    fn = "moe_permute"
    ldx, ldr = cols if ldx is None else ldx, cols if ldr is None else ldr
    ws_need = 0
    if ws_bytes is None:
        ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    elif ws is not None and not isinstance(ws, int):
        ws_need = -(-ws_bytes // ws.element_size())
    if (xtype | num_experts | top_k | n_tokens | cols | ldx | ldr | ws_bytes) >> 31:
        _fit(fn, (xtype, num_experts, top_k), (n_tokens, cols, ldx, ldr), ws_bytes)
    dev, st = _context(stream)
    P = n_tokens * top_k
    _check((_libh or lib()).moe_permute(
        xtype, _arg(fn, "x", x, xtype, _span(n_tokens, cols, ldx), dev, ldx), n_tokens, cols, ldx,
        _arg(fn, "topk_idx", topk_idx, _I32, P, dev), num_experts, top_k,
        _arg(fn, "rows", rows, xtype, _span(P, cols, ldr), dev, ldr), ldr,
        _arg(fn, "offsets", offsets, _I32, num_experts + 1, dev),
        _arg(fn, "pos", pos, _I32, P, dev), _arg(fn, "ws", ws, None, ws_need, dev), ws_bytes, st))


def moe_combine(ytype: int, y, n_rows: int, cols: int, pos, topk_w, n_tokens: int, top_k: int,
                otype: int, residual, out, ldy=None, ldo=None, stream=None) -> None:
    """out[t] = residual[t] + sum_s topk_w[t][s] y[pos[t][s]] (see include/qmoe.h)."""
    if ldy is None and ldo is None and _answered((_calls or _short_way()).combine(
            ytype, y, n_rows, cols, pos, topk_w, n_tokens, top_k, otype, residual, out, stream)):
        return
    fn = "moe_combine"
    ldy, ldo = cols if ldy is None else ldy, cols if ldo is None else ldo
    if (ytype | otype | top_k | n_rows | cols | n_tokens | ldy | ldo) >> 31:
        _fit(fn, (ytype, otype, top_k), (n_rows, cols, n_tokens, ldy, ldo))
    dev, st = _context(stream)
    P, TH = n_tokens * top_k, _span(n_tokens, cols, ldo)
    _check((_libh or lib()).moe_combine(
        ytype, _arg(fn, "y", y, ytype, _span(n_rows, cols, ldy), dev, ldy), n_rows, cols, ldy,
        _arg(fn, "pos", pos, _I32, P, dev), _arg(fn, "topk_w", topk_w, F32, P, dev), n_tokens,
        top_k, otype, _arg(fn, "residual", residual, otype, TH, dev, ldo),
        _arg(fn, "out", out, otype, TH, dev, ldo), ldo, st))


def moe_combine_backward(ytype: int, y, n_rows: int, cols: int, pos, topk_w, n_tokens: int,
                         top_k: int, otype: int, grad_out, grad_y, grad_w, ldy=None, ldo=None,
                         ldg=None, stream=None) -> None:
    """grad_y and grad_w (either may be None) of moe_combine (see include/qmoe.h)."""
    if ldy is None and ldo is None and ldg is None and _answered((_calls or _short_way()).combine_backward(
            ytype, y, n_rows, cols, pos, topk_w, n_tokens, top_k, otype, grad_out, grad_y, grad_w,
            stream)):
        return
    fn = "moe_combine_backward"
    ldy, ldo = cols if ldy is None else ldy, cols if ldo is None else ldo
    ldg = cols if ldg is None else ldg
    if (ytype | otype | top_k | n_rows | cols | n_tokens | ldy | ldo | ldg) >> 31:
        _fit(fn, (ytype, otype, top_k), (n_rows, cols, n_tokens, ldy, ldo, ldg))
    dev, st = _context(stream)
    P = n_tokens * top_k
    _check((_libh or lib()).moe_combine_backward(
        ytype, _arg(fn, "y", y, ytype, _span(n_rows, cols, ldy), dev, ldy), n_rows, cols, ldy,
        _arg(fn, "pos", pos, _I32, P, dev), _arg(fn, "topk_w", topk_w, F32, P, dev), n_tokens,
        top_k, otype,
        _arg(fn, "grad_out", grad_out, otype, _span(n_tokens, cols, ldo), dev, ldo), ldo,
        _arg(fn, "grad_y", grad_y, ytype, _span(n_rows, cols, ldg), dev, ldg), ldg,
        _arg(fn, "grad_w", grad_w, F32, P, dev), st))


# --------------------------- products with 4-bit weights (include/qmoe.h)
def w4_mm(W, stype: int, scale, zero, scale_cols: int, rows: int, cols: int, xtype: int, x,
          n_tokens: int, ytype: int, y, ldx=None, ldy=None, stream=None) -> None:
    """y = x W^T with 4-bit weights, a scale and zero point per scale_cols columns (see
    include/qmoe.h)."""
    if ldx is None and ldy is None and _answered((_calls or _short_way()).w4(
            W, stype, scale, zero, scale_cols, -1, rows, cols, xtype, x, n_tokens, None, ytype, y,
            stream)):
        return
    fn = "w4_mm"
    ldx, ldy = cols if ldx is None else ldx, rows if ldy is None else ldy
    if (stype | scale_cols | xtype | ytype | rows | cols | n_tokens | ldx | ldy) >> 31:
        _fit(fn, (stype, scale_cols, xtype, ytype), (rows, cols, n_tokens, ldx, ldy))
    dev, st = _context(stream)
    blocks = rows * (cols // scale_cols) if scale_cols > 0 else 0
    _check((_libh or lib()).w4_mm(
        _arg(fn, "W", W, _U8, rows * cols // 2, dev), stype,
        _arg(fn, "scale", scale, stype, blocks, dev), _arg(fn, "zero", zero, _U8, blocks, dev),
        scale_cols, rows, cols, xtype,
        _arg(fn, "x", x, xtype, _span(n_tokens, cols, ldx), dev, ldx), n_tokens, ldx, ytype,
        _arg(fn, "y", y, ytype, _span(n_tokens, rows, ldy), dev, ldy), ldy, st))


def w4_mm_grouped(W, stype: int, scale, zero, scale_cols: int, num_groups: int, rows: int,
                  cols: int, xtype: int, x, n_rows: int, offsets, ytype: int, y, ldx=None,
                  ldy=None, stream=None) -> None:
    """y[r] = W_g x[r] for the rows of every group, with 4-bit weights (see
    include/qmoe.h)."""
    if ldx is None and ldy is None and _answered((_calls or _short_way()).w4(
            W, stype, scale, zero, scale_cols, num_groups, rows, cols, xtype, x, n_rows, offsets,
            ytype, y, stream)):
        return
    fn = "w4_mm_grouped"
    ldx, ldy = cols if ldx is None else ldx, rows if ldy is None else ldy
    if (stype | scale_cols | num_groups | xtype | ytype | rows | cols | n_rows | ldx | ldy) >> 31:
        _fit(fn, (stype, scale_cols, num_groups, xtype, ytype), (rows, cols, n_rows, ldx, ldy))
    dev, st = _context(stream)
    n = num_groups * rows
    blocks = n * (cols // scale_cols) if scale_cols > 0 else 0
    _check((_libh or lib()).w4_mm_grouped(
        _arg(fn, "W", W, _U8, n * cols // 2, dev), stype,
        _arg(fn, "scale", scale, stype, blocks, dev), _arg(fn, "zero", zero, _U8, blocks, dev),
        scale_cols, num_groups, rows, cols, xtype,
        _arg(fn, "x", x, xtype, _span(n_rows, cols, ldx), dev, ldx), n_rows, ldx,
        _arg(fn, "offsets", offsets, _I32, num_groups + 1, dev), ytype,
        _arg(fn, "y", y, ytype, _span(n_rows, rows, ldy), dev, ldy), ldy, st))


# qmoe_set_exec_mode
EXEC_DEFAULT, EXEC_SEPARATE, EXEC_UNBATCHED = 0, 1, 2


def set_exec_mode(mode: int) -> None:
    """Diagnostics and tests: which equivalent kernel forms later calls launch
    (EXEC_DEFAULT, EXEC_SEPARATE or EXEC_UNBATCHED; see include/qmoe.h)."""
    _check(lib().qmoe_set_exec_mode(mode))


def set_fault_injection(wait_limit_ns: int = 0, skip_arrive_cta: int = -1) -> None:
    """Failure-path tests only: shorten every bounded device wait and make one
    CTA of the cooperative kernels skip its grid-barrier arrivals, or one of the
    e4m3, bf16 and f16 products, or of the 4-bit products for many rows, load
    nothing; (0, -1) restores normal operation (see include/qmoe.h)."""
    _check(lib().qmoe_set_fault_injection(wait_limit_ns, skip_arrive_cta))


def device_status(stream=None) -> int:
    """Synchronise the stream and read/clear the device error word."""
    return int(lib().qmoe_device_status(_stream(stream)))
