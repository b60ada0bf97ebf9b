"""ctypes binding for libloftq: LoftQ initialisation on AMD Instinct MI355X (gfx950).

Argument marshalling only.  Every step of the computation runs in the HIP
kernels of ``libloftq.so`` (built in-tree by ``_build.build()``); torch is used
for device memory and the current stream.  Importing this package without the
built library raises ImportError: there is no CPU fallback.

The functions carry the C entry points' names (see include/loftq.h):
    loftq_nf4_quantize, loftq_double_quant, loftq_nf4_dequantize,
    loftq_nf4_merge, loftq_nf4_unmerge, loftq_lowrank_svd, loftq_init,
    loftq_qlora_forward, loftq_dropout, loftq_qlora_forward_dropout, loftq_qlora_backward,
    loftq_mxfp4_quantize, loftq_mxfp4_dequantize, loftq_mxfp4_forward, loftq_mxfp4_backward
and return freshly allocated torch tensors on the input's device (or fill the
caller's ``out`` / ``buffers`` where those are given).
With ``stream`` a call runs there instead of on the current stream, and what it returns
is allocated there: the caller has its inputs ready on that stream and keeps them until
the call is done (or records them on it), and a reader on another stream waits for it.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libloftq.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libloftq.so is not built ({LIB_PATH}); run __graft_entry__.build() first")

_lib = ctypes.CDLL(LIB_PATH)

LOFTQ_F32, LOFTQ_BF16 = 0, 1
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported configuration", 3: "workspace too small",
          4: "HIP runtime error"}

EXPORTS = ["loftq_init_batch", "loftq_batch_workspace_bytes", "loftq_nf4_quantize", "loftq_double_quant", "loftq_nf4_dequantize", "loftq_nf4_merge",
           "loftq_nf4_unmerge", "loftq_lowrank_svd",
           "loftq_lowrank_svd_workspace_bytes", "loftq_init", "loftq_workspace_bytes", "loftq_default_config",
           "loftq_status_string", "loftq_nf4_codebook", "loftq_nf_codebook", "loftq_qlora_forward",
           "loftq_qlora_forward_workspace_bytes", "loftq_qlora_forward_noalloc", "loftq_qlora_forward_noalloc_max_bytes",
           "loftq_profile_enable", "loftq_profile_collect", "loftq_profile_calibrate",
           "loftq_dropout", "loftq_qlora_forward_dropout", "loftq_qlora_forward_dropout_workspace_bytes",
           "loftq_qlora_backward", "loftq_qlora_backward_workspace_bytes", "loftq_mxfp4_packed_bytes",
           "loftq_mxfp4_scale_bytes", "loftq_mxfp4_quantize", "loftq_mxfp4_dequantize", "loftq_mxfp4_forward",
           "loftq_mxfp4_forward_workspace_bytes", "loftq_mxfp4_backward", "loftq_mxfp4_backward_workspace_bytes"]


class LoftqConfig(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("iterative_steps", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("blocksize", ctypes.c_int32), ("double_quant", ctypes.c_int32), ("dq_blocksize", ctypes.c_int32),
                ("oversample", ctypes.c_int32), ("power_iters", ctypes.c_int32), ("exact_svd", ctypes.c_int32),
                ("warm_start", ctypes.c_int32), ("seed", ctypes.c_uint64), ("init_from_BA", ctypes.c_int32),
                ("materialize_residual", ctypes.c_int32)]


_P, _I64, _I32, _U64, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint64, ctypes.c_size_t


class LoftqMatrix(ctypes.Structure):
    _fields_ = [("W", _P), ("rows", _I64), ("cols", _I64), ("packed", _P), ("absmax", _P), ("qabsmax", _P),
                ("dq_scale", _P), ("B", _P), ("A", _P), ("objective", _P), ("sigma", _P)]


class LoftqDropout(ctypes.Structure):
    _fields_ = [("p", ctypes.c_float), ("seed", _U64), ("offset", _U64), ("step", _P)]


def _sig(name, res, args):
    f = getattr(_lib, name, None)
    if f is None:
        return None
    f.restype, f.argtypes = res, args
    return f


_c_quant = _sig("loftq_nf4_quantize", ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _P, _P, _I32, _I32, _P, _P, _P])
_c_dq = _sig("loftq_double_quant", ctypes.c_int, [_P, _I64, _I32, _P, _P, _P])
_c_deq = _sig("loftq_nf4_dequantize", ctypes.c_int,
              [_P, _P, _P, _P, _I64, _I64, _I32, _I32, _P, ctypes.c_int, _P, _P, _P])
_MERGE_ARGS = [_P, _P, _P, _P, _I64, _I64, _I32, _I32, _P, _P, _I32, ctypes.c_float, _P, _P, _P, _P, _P]
_c_merge = _sig("loftq_nf4_merge", ctypes.c_int, _MERGE_ARGS)
_c_unmerge = _sig("loftq_nf4_unmerge", ctypes.c_int, _MERGE_ARGS)
_c_fwd = _sig("loftq_qlora_forward", ctypes.c_int,
              [_P, _I64, _I64, _I64, _P, _P, _P, _P, _I32, _P, _P, _I32, ctypes.c_float, _P, _P, _SZ, _P])
_c_fwd_ws = _sig("loftq_qlora_forward_workspace_bytes", _SZ, [_I64, _I32])
_c_fwd_na = _sig("loftq_qlora_forward_noalloc", ctypes.c_int,
                 [_P, _I64, _I64, _I64, _P, _P, _P, _P, _I32, _P, _P, _I32, ctypes.c_float, _P, _P])
_c_fwd_na_max = _sig("loftq_qlora_forward_noalloc_max_bytes", _SZ, [])
_DROP = ctypes.POINTER(LoftqDropout)
_NF_ARGS = [_P, _P, _P, _P, _I32]                       # packed, absmax, qabsmax, dq_scale, bits
_MX_ARGS = [_P, _P]                                     # packed, scales
_ADAPTER_ARGS = [_P, _P, _I32, ctypes.c_float, _DROP]   # B, A, r, alpha, drop
_FWD_OUT = [_P, ctypes.c_int, _P, _SZ, _P]
_BWD_OUT = [_P, ctypes.c_int, _P, _P, _P, _SZ, _P]
_c_dropout = _sig("loftq_dropout", ctypes.c_int, [_P, ctypes.c_int, _I64, _DROP, _P, _P])
_c_fwd_drop = _sig("loftq_qlora_forward_dropout", ctypes.c_int,
                   [_P, _I64, _I64, _I64] + _NF_ARGS + _ADAPTER_ARGS + _FWD_OUT)
_c_bwd = _sig("loftq_qlora_backward", ctypes.c_int, [_P, _P, _I64, _I64, _I64] + _NF_ARGS + _ADAPTER_ARGS + _BWD_OUT)
_c_mx_fwd = _sig("loftq_mxfp4_forward", ctypes.c_int, [_P, _I64, _I64, _I64] + _MX_ARGS + _ADAPTER_ARGS + _FWD_OUT)
_c_mx_bwd = _sig("loftq_mxfp4_backward", ctypes.c_int,
                 [_P, _P, _I64, _I64, _I64] + _MX_ARGS + _ADAPTER_ARGS + _BWD_OUT)
_LAYER_WS = [_I64, _I64, _I64, _I32]
_c_fwd_drop_ws = _sig("loftq_qlora_forward_dropout_workspace_bytes", _SZ, _LAYER_WS)
_c_bwd_ws = _sig("loftq_qlora_backward_workspace_bytes", _SZ, _LAYER_WS)
_c_mx_fwd_ws = _sig("loftq_mxfp4_forward_workspace_bytes", _SZ, _LAYER_WS)
_c_mx_bwd_ws = _sig("loftq_mxfp4_backward_workspace_bytes", _SZ, _LAYER_WS)
_c_mx_packed = _sig("loftq_mxfp4_packed_bytes", _SZ, [_I64, _I64])
_c_mx_scales = _sig("loftq_mxfp4_scale_bytes", _SZ, [_I64, _I64])
_c_mx_quant = _sig("loftq_mxfp4_quantize", ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _P, _P, _I32, _P, _P, _P])
_c_mx_deq = _sig("loftq_mxfp4_dequantize", ctypes.c_int,
                 [_P, _P, _I64, _I64, _P, ctypes.c_int, _P, ctypes.c_int, _P])
_c_svd = _sig("loftq_lowrank_svd", ctypes.c_int,
              [_P, _I64, _I64, _I32, _I32, _I32, _I32, _P, _U64, _I32, _P, _P, _P, _P, _SZ, _P])
_c_svd_ws = _sig("loftq_lowrank_svd_workspace_bytes", _SZ, [_I64, _I64, _I32, _I32, _I32])
_c_init = _sig("loftq_init", ctypes.c_int,
               [_P, ctypes.c_int, _I64, _I64, ctypes.POINTER(LoftqConfig), _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ,
                _P])
_c_init_ws = _sig("loftq_workspace_bytes", _SZ, [_I64, _I64, ctypes.POINTER(LoftqConfig)])
_c_batch = _sig("loftq_init_batch", ctypes.c_int,
                [ctypes.POINTER(LoftqMatrix), _I32, ctypes.c_int, ctypes.POINTER(LoftqConfig), _I32,
                 ctypes.POINTER(_P), ctypes.POINTER(_P), _SZ])
_c_batch_ws = _sig("loftq_batch_workspace_bytes", _SZ, [ctypes.POINTER(LoftqMatrix), _I32, ctypes.POINTER(LoftqConfig)])
_c_defaults = _sig("loftq_default_config", None, [ctypes.POINTER(LoftqConfig)])
_c_status = _sig("loftq_status_string", ctypes.c_char_p, [ctypes.c_int])
_c_codebook = _sig("loftq_nf4_codebook", None, [ctypes.POINTER(ctypes.c_float)])
_c_nf_codebook = _sig("loftq_nf_codebook", ctypes.c_int, [_I32, ctypes.POINTER(ctypes.c_float)])
_c_prof_on = _sig("loftq_profile_enable", None, [ctypes.c_int])
_c_prof_get = _sig("loftq_profile_collect", ctypes.c_int, [ctypes.c_int, ctypes.c_char_p, _P, _P])
_c_prof_cal = _sig("loftq_profile_calibrate", ctypes.c_int, [ctypes.c_int, _P])


class LoftqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {STATUS.get(status, status)} (status {status})")


def _check(fn: str, st: int) -> None:
    if st != 0:
        raise LoftqError(fn, st)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _on(stream):
    """Where a call on `stream` allocates: the memory comes from that stream's pool.  A block of the current stream's
    pool may still be in use there, and one dropped on return would go to the current stream's next tensor while the
    call's kernels use it."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """A new output of a call on `stream`.  The caller may read and drop it on the current stream, so its memory
    waits for that stream too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _scratch(nbytes, device, stream) -> torch.Tensor:
    """A new workspace of a call on `stream`, dropped when the call returns."""
    with _on(stream):
        return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def _wdtype(W: torch.Tensor) -> int:
    if W.dtype == torch.float32:
        return LOFTQ_F32
    if W.dtype == torch.bfloat16:
        return LOFTQ_BF16
    raise TypeError("W must be float32 or bfloat16")


def _contig(t: torch.Tensor, what: str) -> torch.Tensor:
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous device tensor")
    return t


def exported_symbols():
    """Names from include/loftq.h that the loaded library exports."""
    return [name for name in EXPORTS if hasattr(_lib, name)]


def nf4_codebook() -> list:
    buf = (ctypes.c_float * 16)()
    _c_codebook(buf)
    return list(buf)


def nf_codebook(bits: int) -> list:
    """The 2^bits k-bit NormalFloat levels (bits 2, 3 or 4)."""
    buf = (ctypes.c_float * 16)()
    _check("loftq_nf_codebook", _c_nf_codebook(int(bits), buf))
    return list(buf)[: 1 << int(bits)]


def default_config(**overrides) -> LoftqConfig:
    cfg = LoftqConfig()
    _c_defaults(ctypes.byref(cfg))
    for k, v in overrides.items():
        if not hasattr(cfg, k):
            raise KeyError(k)
        setattr(cfg, k, int(v))
    return cfg


def loftq_nf4_quantize(W: torch.Tensor, B: Optional[torch.Tensor] = None, A: Optional[torch.Tensor] = None,
                       packed: Optional[torch.Tensor] = None, absmax: Optional[torch.Tensor] = None, stream=None):
    """Quantize R = W - B A (or W) to packed NF4 codes and blockwise absmax."""
    _contig(W, "W")
    rows, cols = (W.shape[0], W.shape[1]) if W.dim() == 2 else (1, W.numel())
    n = rows * cols
    r = 0
    if B is not None:
        _contig(B, "B"), _contig(A, "A")
        r = B.shape[1]
    if packed is None:
        packed = _empty((n + 1) // 2, torch.uint8, W.device, stream)
    if absmax is None:
        absmax = _empty((n + 63) // 64, torch.float32, W.device, stream)
    _check("loftq_nf4_quantize", _c_quant(_ptr(W), _wdtype(W), rows, cols, _ptr(B), _ptr(A), r, 64, _ptr(packed),
                                          _ptr(absmax), _stream(stream)))
    return packed, absmax


def loftq_double_quant(absmax: torch.Tensor, stream=None):
    _contig(absmax, "absmax")
    nb = absmax.numel()
    q = _empty(nb, torch.int8, absmax.device, stream)
    s = _empty((nb + 255) // 256, torch.float32, absmax.device, stream)
    _check("loftq_double_quant", _c_dq(_ptr(absmax), nb, 256, _ptr(q), _ptr(s), _stream(stream)))
    return q, s


def loftq_nf4_dequantize(packed: torch.Tensor, shape, absmax: Optional[torch.Tensor] = None,
                         qabsmax: Optional[torch.Tensor] = None, dq_scale: Optional[torch.Tensor] = None,
                         W: Optional[torch.Tensor] = None, with_sumsq: bool = False, stream=None):
    """deq(Q), or W - deq(Q) when W is given; optionally also sum of squares (fp64)."""
    rows, cols = shape
    out = _empty((rows, cols), torch.float32, packed.device, stream)
    ss = _empty(1, torch.float64, packed.device, stream) if with_sumsq else None
    wdt = _wdtype(W) if W is not None else LOFTQ_F32
    _check("loftq_nf4_dequantize",
           _c_deq(_ptr(packed), _ptr(absmax), _ptr(qabsmax), _ptr(dq_scale), rows, cols, 64, 256, _ptr(W), wdt,
                  _ptr(out), _ptr(ss), _stream(stream)))
    return (out, ss) if with_sumsq else out


def _merge_call(fn, c_fn, packed, shape, absmax, qabsmax, dq_scale, B, A, alpha, double_quant, out, stream):
    rows, cols = shape
    n = rows * cols
    r = 0
    if B is not None:
        _contig(B, "B"), _contig(A, "A")
        r = B.shape[1]
    dev = packed.device
    if out is None:
        out = {"packed": _empty((n + 1) // 2, torch.uint8, dev, stream),
               "absmax": _empty((n + 63) // 64, torch.float32, dev, stream)}
        if double_quant:
            out["qabsmax"] = _empty((n + 63) // 64, torch.int8, dev, stream)
            out["dq_scale"] = _empty(((n + 63) // 64 + 255) // 256, torch.float32, dev, stream)
    _check(fn, c_fn(_ptr(packed), _ptr(absmax), _ptr(qabsmax), _ptr(dq_scale), rows, cols, 64, 256, _ptr(B), _ptr(A),
                    r, float(alpha), _ptr(out["packed"]), _ptr(out["absmax"]), _ptr(out.get("qabsmax")),
                    _ptr(out.get("dq_scale")), _stream(stream)))
    return out


def loftq_nf4_merge(packed: torch.Tensor, shape, B: Optional[torch.Tensor], A: Optional[torch.Tensor],
                    alpha: float = 1.0, absmax: Optional[torch.Tensor] = None, qabsmax: Optional[torch.Tensor] = None,
                    dq_scale: Optional[torch.Tensor] = None, double_quant: bool = False, out: Optional[dict] = None,
                    stream=None) -> dict:
    """Q' = NF4(deq(Q) + alpha B A): dict of packed, absmax (and qabsmax, dq_scale with double_quant).
    `out` may hold the input tensors themselves (in place)."""
    return _merge_call("loftq_nf4_merge", _c_merge, packed, shape, absmax, qabsmax, dq_scale, B, A, alpha,
                       double_quant, out, stream)


def loftq_nf4_unmerge(packed: torch.Tensor, shape, B: Optional[torch.Tensor], A: Optional[torch.Tensor],
                      alpha: float = 1.0, absmax: Optional[torch.Tensor] = None, qabsmax: Optional[torch.Tensor] = None,
                      dq_scale: Optional[torch.Tensor] = None, double_quant: bool = False, out: Optional[dict] = None,
                      stream=None) -> dict:
    """Q' = NF4(deq(Q) - alpha B A), the reverse of loftq_nf4_merge (not an exact inverse)."""
    return _merge_call("loftq_nf4_unmerge", _c_unmerge, packed, shape, absmax, qabsmax, dq_scale, B, A, alpha,
                       double_quant, out, stream)


def qlora_forward_workspace_bytes(n_tok: int, r: int) -> int:
    return int(_c_fwd_ws(n_tok, r))


def loftq_qlora_forward(X: torch.Tensor, packed: torch.Tensor, shape, absmax: Optional[torch.Tensor] = None,
                        qabsmax: Optional[torch.Tensor] = None, dq_scale: Optional[torch.Tensor] = None,
                        B: Optional[torch.Tensor] = None, A: Optional[torch.Tensor] = None, alpha: float = 1.0,
                        bits: int = 4, out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """Y = X bf16(deq(Q))^T + alpha (X bf16(A)^T) bf16(B)^T for bf16 X (n_tok x cols); Y fp32 n_tok x rows."""
    _contig(X, "X")
    if X.dtype != torch.bfloat16:
        raise TypeError("X must be bfloat16")
    rows, cols = shape
    n_tok = X.shape[0]
    r = 0
    if B is not None:
        _contig(B, "B"), _contig(A, "A")
        r = B.shape[1]
    if out is None:
        out = _empty((n_tok, rows), torch.float32, X.device, stream)
    ws_bytes = 0
    if B is not None:
        ws_bytes = qlora_forward_workspace_bytes(n_tok, r)
        if ws is None:
            ws = _scratch(ws_bytes, X.device, stream)
        else:
            ws_bytes = ws.numel() * ws.element_size()
    _check("loftq_qlora_forward",
           _c_fwd(_ptr(X), n_tok, rows, cols, _ptr(packed), _ptr(absmax), _ptr(qabsmax), _ptr(dq_scale), int(bits),
                  _ptr(B), _ptr(A), r, float(alpha), _ptr(out), _ptr(ws), ws_bytes, _stream(stream)))
    return out


def qlora_forward_noalloc_max_bytes() -> int:
    return int(_c_fwd_na_max())


def loftq_qlora_forward_noalloc(X: torch.Tensor, packed: torch.Tensor, shape, absmax: Optional[torch.Tensor] = None,
                                qabsmax: Optional[torch.Tensor] = None, dq_scale: Optional[torch.Tensor] = None,
                                B: Optional[torch.Tensor] = None, A: Optional[torch.Tensor] = None,
                                alpha: float = 1.0, bits: int = 4, out: Optional[torch.Tensor] = None,
                                stream=None) -> torch.Tensor:
    """loftq_qlora_forward without a workspace: the library's own device scratch holds the
    partial products (no allocation in the call; `out` is allocated here only if not given)."""
    _contig(X, "X")
    if X.dtype != torch.bfloat16:
        raise TypeError("X must be bfloat16")
    rows, cols = shape
    n_tok = X.shape[0]
    r = 0
    if B is not None:
        _contig(B, "B"), _contig(A, "A")
        r = B.shape[1]
    if out is None:
        out = _empty((n_tok, rows), torch.float32, X.device, stream)
    _check("loftq_qlora_forward_noalloc",
           _c_fwd_na(_ptr(X), n_tok, rows, cols, _ptr(packed), _ptr(absmax), _ptr(qabsmax), _ptr(dq_scale),
                     int(bits), _ptr(B), _ptr(A), r, float(alpha), _ptr(out), _stream(stream)))
    return out


# ---- training and serving an adapted layer ----

_M64 = 2 ** 64 - 1
_FLOATS = (torch.float32, torch.bfloat16)


def _first(t, what):
    """The tensor that says where a call runs: its device's number."""
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous device tensor")
    return t.get_device()


def _expect(t, what, dev, dtype, shape=None, least=0):
    """A contiguous tensor on device `dev` of the given type (None: fp32 or bf16) and of a shape or of at least so
    many elements; its address."""
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous device tensor")
    if t.get_device() != dev:
        raise ValueError(f"{what} must be on device {dev}")
    if t.dtype is not dtype and (dtype is not None or t.dtype not in _FLOATS):
        raise TypeError(f"{what} must be {dtype or 'float32 or bfloat16'}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what} must have the shape {tuple(shape)}")
    if t.numel() < least:
        raise ValueError(f"{what} must hold {least} elements")
    return t.data_ptr()


def _call(name, c_fn, dev, stream, *args):
    """c_fn on device `dev`, on `stream` or the device's current one."""
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(dev)
    else:
        s = stream.cuda_stream
    if torch.cuda.current_device() == dev:
        st = c_fn(*args, s)
    else:
        with torch.cuda.device(dev):
            st = c_fn(*args, s)
    if st != 0:
        raise LoftqError(name, st)


def _dropout(p, seed, offset, step, dev):
    at = None if step is None else _expect(step, "step", dev, torch.int64, (1,))
    if p == 0:
        return None
    return ctypes.byref(LoftqDropout(p, int(seed) & _M64, int(offset) & _M64, at))


def _out_dtype(t, dtype):
    dtype = t.dtype if t is not None else dtype
    if dtype not in _FLOATS:
        raise TypeError("outputs are float32 or bfloat16")
    return dtype


def _nf_args(dev, packed, rows, cols, absmax, qabsmax, dq_scale, bits):
    nb = (rows * cols + 63) // 64
    at = _expect(packed, "packed", dev, torch.uint8, least=(rows * cols + 1) // 2)
    if qabsmax is not None or dq_scale is not None:
        if qabsmax is None or dq_scale is None:
            raise ValueError("qabsmax and dq_scale are given together")
        return (at, None, _expect(qabsmax, "qabsmax", dev, torch.int8, least=nb),
                _expect(dq_scale, "dq_scale", dev, torch.float32, least=(nb + 255) // 256), bits)
    if absmax is None:
        raise ValueError("absmax, or qabsmax and dq_scale, must be given")
    return at, _expect(absmax, "absmax", dev, torch.float32, least=nb), None, None, bits


def _mx_args(dev, packed, scales, rows, cols):
    steps = (cols + 255) // 256
    return (_expect(packed, "packed", dev, torch.uint8, least=rows * steps * 128),
            _expect(scales, "scales", dev, torch.uint8, least=rows * steps * 8))


def _adapter_args(dev, B, A, rows, cols):
    """(B, A, r) of a call."""
    if B is None and A is None:
        return None, None, 0
    if B is None or A is None:
        raise ValueError("B and A are given together")
    r = B.shape[1] if B.dim() == 2 else -1
    return _expect(B, "B", dev, torch.float32, (rows, r)), _expect(A, "A", dev, torch.float32, (r, cols)), r


def _workspace(ws, query, sizes, like, stream):
    """(tensor, its address, its bytes); a new one of the size that `query` names where none is given."""
    if ws is None:
        ws = _scratch(query(*sizes), like.device, stream)
    elif not ws.is_cuda or not ws.is_contiguous() or ws.get_device() != like.get_device():
        raise ValueError(f"ws must be a contiguous tensor on {like.device}")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _layer_forward(name, c_fn, query, X, dev, base, rows, cols, B, A, alpha, drop, out, out_dtype, ws, stream):
    n = X.shape[0]
    out_dtype = _out_dtype(out, out_dtype)
    b, a, r = _adapter_args(dev, B, A, rows, cols)
    if out is None:
        out = _empty((n, rows), out_dtype, X.device, stream)
    y = _expect(out, "out", dev, out_dtype, (n, rows))
    ws, w, ws_bytes = _workspace(ws, query, (n, rows, cols, r), X, stream)
    _call(name, c_fn, dev, stream, X.data_ptr(), n, rows, cols, *base, b, a, r, alpha, drop, y,
          LOFTQ_BF16 if out_dtype is torch.bfloat16 else LOFTQ_F32, w, ws_bytes)
    return out


def _layer_backward(name, c_fn, query, dY, X, dev, base, rows, cols, B, A, alpha, drop, need_dx, out, dx_dtype, ws,
                    stream):
    n = dY.shape[0]
    b, a, r = _adapter_args(dev, B, A, rows, cols)
    if out is not None:
        dX, dB, dA = out
    else:
        dX = _empty((n, cols), _out_dtype(None, dx_dtype), dY.device, stream) if need_dx else None
        dB, dA = (_empty(t.shape, t.dtype, dY.device, stream) if r else None for t in (B, A))
    if X is None and dB is not None:
        raise ValueError("X must be given for dB and dA")
    x = None if X is None else _expect(X, "X", dev, torch.bfloat16, (n, cols))
    gx = None if dX is None else _expect(dX, "dX", dev, None, (n, cols))
    gb = None if dB is None else _expect(dB, "dB", dev, torch.float32, (rows, r))
    ga = None if dA is None else _expect(dA, "dA", dev, torch.float32, (r, cols))
    ws, w, ws_bytes = _workspace(ws, query, (n, rows, cols, r), dY, stream)
    _call(name, c_fn, dev, stream, dY.data_ptr(), x, n, rows, cols, *base, b, a, r, alpha, drop, gx,
          LOFTQ_F32 if dX is not None and dX.dtype is torch.float32 else LOFTQ_BF16, gb, ga, w, ws_bytes)
    return dX, dB, dA


def _tokens(X, what, width):
    dev = _first(X, what)
    if X.dtype is not torch.bfloat16:
        raise TypeError(f"{what} must be bfloat16")
    if X.dim() != 2 or X.shape[1] != width:
        raise ValueError(f"{what} must have {width} columns")
    return dev


def loftq_dropout(X: torch.Tensor, p: float, seed: int, offset: int = 0, step: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """X / (1 - p) where the mask of (p, seed, offset + step) keeps, else 0; the gradient is the same call
    on dY.  `step` is a one-element int64 device tensor that is read when the kernel runs.  `out` may be X."""
    dev = _first(X, "X")
    if X.dtype not in _FLOATS:
        raise TypeError("X must be float32 or bfloat16")
    dtype = LOFTQ_BF16 if X.dtype is torch.bfloat16 else LOFTQ_F32
    if out is None:
        out = _empty(X.shape, X.dtype, X.device, stream)
    y = _expect(out, "out", dev, X.dtype, X.shape)
    at = None if step is None else _expect(step, "step", dev, torch.int64, (1,))
    drop = LoftqDropout(p, int(seed) & _M64, int(offset) & _M64, at)
    _call("loftq_dropout", _c_dropout, dev, stream, X.data_ptr(), dtype, X.numel(), ctypes.byref(drop), y)
    return out


def qlora_forward_dropout_workspace_bytes(n_tok: int, rows: int, cols: int, r: int) -> int:
    return int(_c_fwd_drop_ws(n_tok, rows, cols, r))


def qlora_backward_workspace_bytes(n_tok: int, rows: int, cols: int, r: int) -> int:
    return int(_c_bwd_ws(n_tok, rows, cols, r))


def mxfp4_forward_workspace_bytes(n_tok: int, rows: int, cols: int, r: int) -> int:
    return int(_c_mx_fwd_ws(n_tok, rows, cols, r))


def mxfp4_backward_workspace_bytes(n_tok: int, rows: int, cols: int, r: int) -> int:
    return int(_c_mx_bwd_ws(n_tok, rows, cols, r))


def loftq_qlora_forward_dropout(X: torch.Tensor, packed: torch.Tensor, shape, absmax: Optional[torch.Tensor] = None,
                                qabsmax: Optional[torch.Tensor] = None, dq_scale: Optional[torch.Tensor] = None,
                                B: Optional[torch.Tensor] = None, A: Optional[torch.Tensor] = None,
                                alpha: float = 1.0, p: float = 0.0, seed: int = 0, offset: int = 0,
                                step: Optional[torch.Tensor] = None, bits: int = 4,
                                out: Optional[torch.Tensor] = None, out_dtype=torch.float32,
                                ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y = X bf16(deq(Q))^T + alpha / (1 - p) (keep(X) bf16(A)^T) bf16(B)^T for bf16 X (n_tok x cols)."""
    rows, cols = shape
    dev = _tokens(X, "X", cols)
    return _layer_forward("loftq_qlora_forward_dropout", _c_fwd_drop, _c_fwd_drop_ws, X, dev,
                          _nf_args(dev, packed, rows, cols, absmax, qabsmax, dq_scale, bits), rows, cols, B, A, alpha,
                          _dropout(p, seed, offset, step, dev), out, out_dtype, ws, stream)


def loftq_qlora_backward(dY: torch.Tensor, X: Optional[torch.Tensor], packed: torch.Tensor, shape,
                         absmax: Optional[torch.Tensor] = None, qabsmax: Optional[torch.Tensor] = None,
                         dq_scale: Optional[torch.Tensor] = None, B: Optional[torch.Tensor] = None,
                         A: Optional[torch.Tensor] = None, alpha: float = 1.0, p: float = 0.0, seed: int = 0,
                         offset: int = 0, step: Optional[torch.Tensor] = None, bits: int = 4, need_dx: bool = True,
                         out=None, dx_dtype=torch.bfloat16, ws: Optional[torch.Tensor] = None, stream=None):
    """(dX, dB, dA) of loftq_qlora_forward_dropout for bf16 dY (n_tok x rows) and the forward's X and mask.
    `out`: the three tensors to fill, None for one that is not wanted (dB and dA both or neither)."""
    rows, cols = shape
    dev = _tokens(dY, "dY", rows)
    return _layer_backward("loftq_qlora_backward", _c_bwd, _c_bwd_ws, dY, X, dev,
                           _nf_args(dev, packed, rows, cols, absmax, qabsmax, dq_scale, bits), rows, cols, B, A, alpha,
                           _dropout(p, seed, offset, step, dev), need_dx, out, dx_dtype, ws, stream)


def loftq_mxfp4_quantize(W: torch.Tensor, B: Optional[torch.Tensor] = None, A: Optional[torch.Tensor] = None,
                         packed: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None, stream=None):
    """W - B A (or W) in MXFP4: codes (rows x 128-byte steps of 256 columns) and scales (steps x rows x 8)."""
    dev, dtype = _first(W, "W"), _wdtype(W)
    if W.dim() != 2:
        raise ValueError("W must be a matrix")
    rows, cols = W.shape
    steps = (cols + 255) // 256
    b, a, r = _adapter_args(dev, B, A, rows, cols)
    if packed is None:
        packed = _empty((rows, steps * 128), torch.uint8, W.device, stream)
    if scales is None:
        scales = _empty((steps, rows, 8), torch.uint8, W.device, stream)
    _call("loftq_mxfp4_quantize", _c_mx_quant, dev, stream, W.data_ptr(), dtype, rows, cols, b, a, r,
          *_mx_args(dev, packed, scales, rows, cols))
    return packed, scales


def loftq_mxfp4_dequantize(packed: torch.Tensor, scales: torch.Tensor, shape, W: Optional[torch.Tensor] = None,
                           out: Optional[torch.Tensor] = None, out_dtype=torch.float32, stream=None) -> torch.Tensor:
    """deq(Q), or W - deq(Q) when W is given; formed in fp32 and rounded to out_dtype."""
    rows, cols = shape
    dev = _first(packed, "packed")
    base = _mx_args(dev, packed, scales, rows, cols)
    w = None if W is None else _expect(W, "W", dev, None, (rows, cols))
    out_dtype = _out_dtype(out, out_dtype)
    if out is None:
        out = _empty((rows, cols), out_dtype, packed.device, stream)
    _call("loftq_mxfp4_dequantize", _c_mx_deq, dev, stream, *base, rows, cols, w,
          LOFTQ_BF16 if W is not None and W.dtype is torch.bfloat16 else LOFTQ_F32,
          _expect(out, "out", dev, out_dtype, (rows, cols)),
          LOFTQ_BF16 if out_dtype is torch.bfloat16 else LOFTQ_F32)
    return out


def loftq_mxfp4_forward(X: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, shape,
                        B: Optional[torch.Tensor] = None, A: Optional[torch.Tensor] = None, alpha: float = 1.0,
                        p: float = 0.0, seed: int = 0, offset: int = 0, step: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, out_dtype=torch.float32,
                        ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y = MX(X) deq(Q)^T + alpha / (1 - p) (keep(X) bf16(A)^T) bf16(B)^T for bf16 X (n_tok x cols)."""
    rows, cols = shape
    dev = _tokens(X, "X", cols)
    return _layer_forward("loftq_mxfp4_forward", _c_mx_fwd, _c_mx_fwd_ws, X, dev,
                          _mx_args(dev, packed, scales, rows, cols), rows, cols, B, A, alpha,
                          _dropout(p, seed, offset, step, dev), out, out_dtype, ws, stream)


def loftq_mxfp4_backward(dY: torch.Tensor, X: Optional[torch.Tensor], packed: torch.Tensor, scales: torch.Tensor,
                         shape, B: Optional[torch.Tensor] = None, A: Optional[torch.Tensor] = None,
                         alpha: float = 1.0, p: float = 0.0, seed: int = 0, offset: int = 0,
                         step: Optional[torch.Tensor] = None, need_dx: bool = True, out=None,
                         dx_dtype=torch.bfloat16, ws: Optional[torch.Tensor] = None, stream=None):
    """(dX, dB, dA) of loftq_mxfp4_forward, the rounding of X passing the gradient as it is; `out` as in
    loftq_qlora_backward."""
    rows, cols = shape
    dev = _tokens(dY, "dY", rows)
    return _layer_backward("loftq_mxfp4_backward", _c_mx_bwd, _c_mx_bwd_ws, dY, X, dev,
                           _mx_args(dev, packed, scales, rows, cols), rows, cols, B, A, alpha,
                           _dropout(p, seed, offset, step, dev), need_dx, out, dx_dtype, ws, stream)


def lowrank_workspace_bytes(rows: int, cols: int, r: int, oversample: int, exact: bool) -> int:
    return int(_c_svd_ws(rows, cols, r, oversample, int(bool(exact))))


def loftq_lowrank_svd(E: torch.Tensor, r: int, oversample: int = 8, power_iters: int = 2, exact: bool = False,
                      omega: Optional[torch.Tensor] = None, seed: int = 42, t: int = 1, stream=None):
    """Rank-r factors (B, A, sigma) of E by exact or randomized SVD."""
    _contig(E, "E")
    rows, cols = E.shape
    ws_bytes = lowrank_workspace_bytes(rows, cols, r, oversample, exact)
    ws = _scratch(ws_bytes, E.device, stream)
    B = _empty((rows, r), torch.float32, E.device, stream)
    A = _empty((r, cols), torch.float32, E.device, stream)
    sigma = _empty(r, torch.float32, E.device, stream)
    _check("loftq_lowrank_svd",
           _c_svd(_ptr(E), rows, cols, r, oversample, power_iters, int(bool(exact)), _ptr(omega), seed, t, _ptr(B),
                  _ptr(A), _ptr(sigma), _ptr(ws), ws_bytes, _stream(stream)))
    return B, A, sigma


def workspace_bytes(rows: int, cols: int, cfg: LoftqConfig) -> int:
    return int(_c_init_ws(rows, cols, ctypes.byref(cfg)))


class InitBuffers:
    """Caller-owned outputs and workspace for repeated loftq_init calls on one shape, on `stream` where the calls
    run on another than the current one."""

    def __init__(self, rows: int, cols: int, cfg: LoftqConfig, device="cuda", workspace: bool = True, stream=None):
        n = rows * cols
        nb = (n + 63) // 64
        self.cfg = cfg
        self.packed = _empty((n + 1) // 2, torch.uint8, device, stream)
        self.absmax = _empty(nb, torch.float32, device, stream)
        self.qabsmax = _empty(max(nb, 1), torch.int8, device, stream)
        self.dq_scale = _empty(max((nb + 255) // 256, 1), torch.float32, device, stream)
        self.B = _empty((rows, cfg.rank), torch.float32, device, stream)
        self.A = _empty((cfg.rank, cols), torch.float32, device, stream)
        self.sigma = _empty(cfg.rank, torch.float32, device, stream)
        self.objective = _empty(cfg.iterative_steps + 1, torch.float64, device, stream)
        self.ws_bytes = workspace_bytes(rows, cols, cfg) if workspace else 0
        self.ws = _scratch(self.ws_bytes, device, stream) if workspace else None

    def matrix(self, W: torch.Tensor) -> LoftqMatrix:
        """This buffer set as one loftq_matrix_t of a batch, for weight W."""
        rows, cols = W.shape
        dq = bool(self.cfg.double_quant)
        return LoftqMatrix(W.data_ptr(), rows, cols, self.packed.data_ptr(), self.absmax.data_ptr(),
                           self.qabsmax.data_ptr() if dq else None, self.dq_scale.data_ptr() if dq else None,
                           self.B.data_ptr(), self.A.data_ptr(), self.objective.data_ptr(), self.sigma.data_ptr())


def loftq_init(W: torch.Tensor, cfg: Optional[LoftqConfig] = None, buffers: Optional[InitBuffers] = None,
               stream=None, **overrides):
    """LoftQ initialisation of one matrix; returns a dict of device tensors."""
    _contig(W, "W")
    if cfg is None:
        cfg = default_config(**overrides)
    rows, cols = W.shape
    bufs = buffers if buffers is not None else InitBuffers(rows, cols, cfg, W.device, stream=stream)
    _check("loftq_init",
           _c_init(_ptr(W), _wdtype(W), rows, cols, ctypes.byref(cfg), _ptr(bufs.packed), _ptr(bufs.absmax),
                   _ptr(bufs.qabsmax), _ptr(bufs.dq_scale), _ptr(bufs.B), _ptr(bufs.A), _ptr(bufs.objective),
                   _ptr(bufs.sigma), _ptr(bufs.ws), bufs.ws_bytes, _stream(stream)))
    out = dict(packed=bufs.packed, absmax=bufs.absmax, B=bufs.B, A=bufs.A, sigma=bufs.sigma,
               objective=bufs.objective)
    if cfg.double_quant:
        out.update(qabsmax=bufs.qabsmax, dq_scale=bufs.dq_scale)
    return out


class BatchRunner:
    """Caller-owned outputs, per-stream workspaces and streams for repeated loftq_init_batch
    calls over one list of weights (all of one storage dtype)."""

    def __init__(self, Ws, cfg: LoftqConfig, nstreams: int = 4, device="cuda"):
        self.Ws = list(Ws)
        for W in self.Ws:
            _contig(W, "W")
        self.wdt = _wdtype(self.Ws[0])
        if any(_wdtype(W) != self.wdt for W in self.Ws):
            raise TypeError("every W of a batch must have the same dtype")
        self.cfg = cfg
        self.buffers = [InitBuffers(W.shape[0], W.shape[1], cfg, device, workspace=False) for W in self.Ws]
        n = len(self.Ws)
        self.mats = (LoftqMatrix * n)(*[b.matrix(W) for b, W in zip(self.buffers, self.Ws)])
        self.ws_bytes = int(_c_batch_ws(self.mats, n, ctypes.byref(cfg)))
        if self.ws_bytes == 0:
            raise LoftqError("loftq_batch_workspace_bytes", 1)
        self.nstreams = int(nstreams)
        # streams at the default priority
        self.streams = [torch.cuda.Stream(device=device) for _ in range(self.nstreams)]
        self.ws = [torch.empty(self.ws_bytes, dtype=torch.uint8, device=device) for _ in range(self.nstreams)]
        self._c_streams = (_P * self.nstreams)(*[s.cuda_stream for s in self.streams])
        self._c_ws = (_P * self.nstreams)(*[w.data_ptr() for w in self.ws])

    def run(self):
        """Enqueue the batch; the current stream then waits for every batch stream."""
        cur = torch.cuda.current_stream()
        for s in self.streams:
            s.wait_stream(cur)
        _check("loftq_init_batch", _c_batch(self.mats, len(self.Ws), self.wdt, ctypes.byref(self.cfg),
                                            self.nstreams, self._c_streams, self._c_ws, self.ws_bytes))
        for s in self.streams:
            cur.wait_stream(s)
        return self.buffers


def loftq_init_batch(Ws, cfg: Optional[LoftqConfig] = None, nstreams: int = 4, **overrides):
    """LoftQ initialisation of a list of weights in one batched call; returns one InitBuffers per weight."""
    if cfg is None:
        cfg = default_config(**overrides)
    return BatchRunner(Ws, cfg, nstreams).run()


def profile_enable(on: bool = True) -> None:
    """Bracket every library kernel launch with HIP events on its stream (measurement only)."""
    _c_prof_on(1 if on else 0)


def profile_calibrate(n: int = 256, stream=None) -> None:
    """n bracketed launches of an empty kernel (recorded as "event_overhead" while timing is enabled)."""
    _check("loftq_profile_calibrate", _c_prof_cal(n, _stream(stream)))


def profile_collect(max_entries: int = 64) -> dict:
    """{kernel name: (launches, total milliseconds)} for the launches recorded since the last collect."""
    names = ctypes.create_string_buffer(64 * max_entries)
    launches = (ctypes.c_int64 * max_entries)()
    total = (ctypes.c_double * max_entries)()
    n = _c_prof_get(max_entries, names, ctypes.cast(launches, ctypes.c_void_p), ctypes.cast(total, ctypes.c_void_p))
    out = {}
    for i in range(n):
        nm = names.raw[64 * i:64 * i + 64].split(b"\0", 1)[0].decode()
        out[nm] = (int(launches[i]), float(total[i]))
    return out
