"""ctypes binding of libwc.so (include/wc.h): argument marshalling only.
(`calls` has the calls of the training-step operators, which reach the library
without ctypes; here are two of them for buffers that the caller lays out,
`embedding_grad` and `fp8_quant`.)

Every function takes torch CUDA tensors, checks dtype, device, contiguity and
sizes, and calls the entry point of the same name on the tensors' current
stream.  All arithmetic happens in the CUDA kernels; there is no CPU or
PyTorch fallback -- if the library is missing or a call fails, an exception
is raised.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
from pathlib import Path

import torch

from . import build as _build

WC_OK, WC_EINVAL, WC_EALIGN, WC_ERANGE, WC_ECUDA = 0, -1, -2, -3, -4
WC_F32, WC_BF16 = 0, 1
WC_I32, WC_I64 = 0, 1

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int
_F = ctypes.c_float
_U32 = ctypes.c_uint32
_D = ctypes.c_double


class WcSpan(ctypes.Structure):
    """wc_span: one tensor of a list."""
    _fields_ = [("data", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("pad", ctypes.c_int32)]


_SPANS = ctypes.POINTER(WcSpan)

# name -> argtypes (all return int except those in RESTYPES)
SIGNATURES = {
    "wc_ef_quant_int4": [_P, _P, _P, _P, _I64, _I, _I, _I, _F, _F, _P],
    "wc_dequant_reduce": [_P, _P, _I64, _I, _I, _I, _F, _P, _I, _P],
    "wc_dequant_reduce_requant": [_P, _P, _I64, _I, _I, _I, _P, _P, _P],
    "wc_dequant_reduce_requant_ef": [_P, _P, _I64, _I, _I, _I, _P, _P, _P, _F, _F, _P],
    "wc_qgz_step_fused": [_P, _P, _P, _P, _I64, _I, _I, _F, _F, _F, _P, _I, _P],
    "wc_qgz_step_fused_bf16ef": [_P, _P, _P, _P, _I64, _I, _I, _F, _F, _F, _P, _I, _P],
    "wc_qgz_step_fused_int8ef": [_P, _P, _P, _P, _P, _I64, _I, _I, _F, _F, _F, _P, _I, _P],
    "wc_qgz_first_hop_fused": [_P, _P, _P, _P, _I64, _I, _I, _I, _F, _F, _P, _P, _P, _P],
    "wc_qgz_first_hop_fused_bf16ef": [_P, _P, _P, _P, _I64, _I, _I, _I, _F, _F, _P, _P, _P, _P],
    "wc_qgz_first_hop_fused_int8ef": [_P, _P, _P, _P, _P, _I64, _I, _I, _I, _F, _F, _P, _P, _P,
                                      _P],
    "wc_ef_quant_int4_bf16ef": [_P, _P, _P, _P, _I64, _I, _I, _I, _F, _F, _P],
    "wc_ef_quant_int4_int8ef": [_P, _P, _P, _P, _P, _I64, _I, _I, _I, _F, _F, _P],
    "wc_qwz_quant_int8": [_P, _P, _P, _I64, _I, _P],
    "wc_qwz_quant_replica_int8": [_P, _P, _P, _P, _I64, _I, _P],
    "wc_qwz_dequant_int8": [_P, _P, _P, _I64, _I, _P],
    "wc_sr_accumulate_bf16": [_P, _P, _I64, _U32, _U32, _P],
    "wc_grad_norm_workspace": [_I],
    "wc_grad_norm": [_SPANS, _I, _P, _P, _I64, _P],
    "wc_grad_clip": [_SPANS, _SPANS, _I, _D, _D, _P, _P, _I64, _P],
    "wc_embedding": [_P, _I, _I64, _P, _I, _I64, _I64, _I64, _I64, _F, _P, _I64, _P],
    "wc_embedding_grad_workspace": [_I64, _I64, _I64],
    "wc_embedding_grad": [_P, _I, _I64, _P, _I, _I64, _I64, _I64, _I64, _F, _I, _P, _I, _I64, _P,
                          _I64, _P],
    "wc_fp8_quant": [_P, _I, _I64, _I64, _I64, _I, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P],
    "wc_fp8_matmul": [_P, _I64, _P, _I64, _I, _P, _I64, _P, _I64, _I, _I64, _I64, _I64, _P, _I,
                      _I64, _I, _P],
    "wc_wait_timeouts": [_I],
    "wc_checked_violations": [_I],
    "wc_last_error": [],
    "wc_version": [],
}
RESTYPES = {"wc_last_error": ctypes.c_char_p, "wc_grad_norm_workspace": _I64,
            "wc_embedding_grad_workspace": _I64}


class WcError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed with status {code}: {msg}")
        self.code = code


_lib: ctypes.CDLL | None = None


def library_path() -> Path:
    """The in-tree libwc.so, or the file named by the WC_LIBRARY environment
    variable (for instance the bounds-checked build)."""
    env = os.environ.get("WC_LIBRARY")
    return Path(env) if env else _build.LIB


def load(path: str | Path | None = None) -> ctypes.CDLL:
    """Load libwc.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = Path(path) if path is not None else library_path()
    if not p.exists():
        raise RuntimeError(f"CUDA library {p} is missing: build it with "
                           "`python -m weight_communication_gb300.build`")
    lib = ctypes.CDLL(str(p))
    for name, args in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = RESTYPES.get(name, ctypes.c_int)
    if path is None:
        _lib = lib
    return lib


_calls = None


def calls():
    """The extension module with the Python calls of the training-step
    operators, set up to call the loaded library.  Raises if it has not been
    built."""
    global _calls
    if _calls is not None:
        return _calls
    lib = load()
    if not _build.CALLS.exists():
        why = _build.CALLS_LOG.read_text().strip() if _build.CALLS_LOG.exists() else ""
        raise RuntimeError(f"extension module {_build.CALLS} is missing: build it with "
                           "`python -m weight_communication_gb300.build`"
                           + (f" (the last build stopped at: {why})" if why else ""))
    loader = importlib.machinery.ExtensionFileLoader("wc_calls", str(_build.CALLS))
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("wc_calls", loader))
    loader.exec_module(module)
    module.setup({name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in SIGNATURES},
                 WcError)
    _calls = module
    return module


def on_stream(stream, device: torch.device, call, *args):
    """call(*args), which allocates and launches on the current stream, with
    `stream` as the current one if it is given."""
    if stream is None:
        return call(*args)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.stream(stream):
        return call(*args)


def last_error() -> str:
    return load().wc_last_error().decode()


def version() -> int:
    return load().wc_version()


WC_CHECK_RESET, WC_CHECK_PROBE = 1, 2


def checked_violations(reset: bool = False, probe: bool = False) -> int:
    """wc_checked_violations: accesses a checked build skipped (synchronize
    first); probe adds one deliberate violation per kernel file first.
    Raises WcError on an ordinary build."""
    lib = load()
    rc = lib.wc_checked_violations((WC_CHECK_RESET if reset else 0) |
                                   (WC_CHECK_PROBE if probe else 0))
    if rc < 0:
        raise WcError("wc_checked_violations", rc, lib.wc_last_error().decode())
    return rc


def wait_timeouts(reset: bool = False) -> int:
    """wc_wait_timeouts: waits of the product's kernels that were given up
    (synchronize first); 0 unless a launch went wrong."""
    lib = load()
    rc = lib.wc_wait_timeouts(1 if reset else 0)
    if rc < 0:
        raise WcError("wc_wait_timeouts", rc, lib.wc_last_error().decode())
    return rc


def _call(device: torch.device, name: str, *args) -> None:
    """Calls the entry point with the tensors' GPU as the current device (the
    kernels launch on the current device)."""
    lib = _lib or load()
    if device.type != "cuda" or torch._C._cuda_getDevice() == device.index:
        rc = getattr(lib, name)(*args)
    else:
        with torch.cuda.device(device):
            rc = getattr(lib, name)(*args)
    if rc != WC_OK:
        raise WcError(name, rc, lib.wc_last_error().decode())


def _stream(t: torch.Tensor, stream: torch.cuda.Stream | None):
    """The launch stream: `stream`, which must belong to the tensors' GPU, or
    that GPU's current stream."""
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)
    if stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {t.device}")
    return ctypes.c_void_p(stream.cuda_stream)


def _dev(t: torch.Tensor | None, name: str, dtype: torch.dtype, numel: int, device=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
    return ctypes.c_void_p(t.data_ptr())


def ef_quant_int4(g: torch.Tensor, ef: torch.Tensor | None, codes: torch.Tensor,
                  scales: torch.Tensor, N: int, R: int, G: int, B: int,
                  err_scale: float = 1.0, err_beta: float = 0.0, stream=None) -> None:
    """wc_ef_quant_int4: g bf16 [R*N], ef fp32 [R*N] (in place) or None,
    codes uint8 [R*N/2], scales fp32 [R*N/B] -- all written in send order."""
    d = g.device
    _call(d, "wc_ef_quant_int4", _dev(g, "g", torch.bfloat16, R * N, d),
          _dev(ef, "ef", torch.float32, R * N, d), _dev(codes, "codes", torch.uint8, R * N // 2, d),
          _dev(scales, "scales", torch.float32, R * N // B, d), N, R, G, B, err_scale, err_beta,
          _stream(g, stream))


def dequant_reduce(codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor, N: int,
                   R: int, G: int, B: int, out_scale: float = 1.0, stream=None) -> None:
    """wc_dequant_reduce: out fp32 or bf16 [R*S] = [N] in destination order.
    G == 1: codes/scales are the ranks' send buffers ([R*N/2], [R*N/B]);
    G > 1: they are the first hop's outputs ([G*N/2], [G*N/B])."""
    d = codes.device
    span = N * (G if G > 1 else R)
    if out.dtype == torch.float32:
        od = WC_F32
    elif out.dtype == torch.bfloat16:
        od = WC_BF16
    else:
        raise TypeError("out must be float32 or bfloat16")
    _call(d, "wc_dequant_reduce", _dev(codes, "codes", torch.uint8, span // 2, d),
          _dev(scales, "scales", torch.float32, span // B, d), N, R, G, B, out_scale,
          _dev(out, "out", out.dtype, N, d), od, _stream(codes, stream))


def dequant_reduce_requant(codes: torch.Tensor, scales: torch.Tensor, out_codes: torch.Tensor,
                           out_scales: torch.Tensor, N: int, R: int, G: int, B: int,
                           stream=None) -> None:
    """wc_dequant_reduce_requant: first hop; out_codes uint8 [G*N/2],
    out_scales fp32 [G*N/B] (unit u = g*L + l holds G*S values)."""
    d = codes.device
    _call(d, "wc_dequant_reduce_requant", _dev(codes, "codes", torch.uint8, R * N // 2, d),
          _dev(scales, "scales", torch.float32, R * N // B, d), N, R, G, B,
          _dev(out_codes, "out_codes", torch.uint8, G * N // 2, d),
          _dev(out_scales, "out_scales", torch.float32, G * N // B, d), _stream(codes, stream))


def dequant_reduce_requant_ef(codes: torch.Tensor, scales: torch.Tensor, out_codes: torch.Tensor,
                              out_scales: torch.Tensor, ef1: torch.Tensor, N: int, R: int, G: int,
                              B: int, err_scale: float = 1.0, err_beta: float = 0.0,
                              stream=None) -> None:
    """wc_dequant_reduce_requant_ef: first hop with error feedback on the
    requantization; ef1 fp32 [G*N] updated in place."""
    d = codes.device
    _call(d, "wc_dequant_reduce_requant_ef", _dev(codes, "codes", torch.uint8, R * N // 2, d),
          _dev(scales, "scales", torch.float32, R * N // B, d), N, R, G, B,
          _dev(out_codes, "out_codes", torch.uint8, G * N // 2, d),
          _dev(out_scales, "out_scales", torch.float32, G * N // B, d),
          _dev(ef1, "ef1", torch.float32, G * N, d), err_scale, err_beta, _stream(codes, stream))


def _fused_error(ef: torch.Tensor | None, ef_scales: torch.Tensor | None, n: int, B: int, d):
    """The fused entry point's suffix and error-buffer pointers for ef's
    dtype: fp32 (or None), bf16, or int8 with its block scales."""
    if ef is None or ef.dtype == torch.float32:
        if ef_scales is not None:
            raise ValueError("ef_scales goes with an int8 error buffer only")
        return "", [_dev(ef, "ef", torch.float32, n, d)]
    if ef.dtype == torch.bfloat16:
        if ef_scales is not None:
            raise ValueError("ef_scales goes with an int8 error buffer only")
        return "_bf16ef", [_dev(ef, "ef", torch.bfloat16, n, d)]
    if ef.dtype == torch.int8:
        if ef_scales is None:
            raise ValueError("an int8 error buffer needs ef_scales")
        return "_int8ef", [_dev(ef, "ef", torch.int8, n, d),
                           _dev(ef_scales, "ef_scales", torch.float32, n // B, d)]
    raise TypeError(f"ef must be float32, bfloat16 or int8, got {ef.dtype}")


def qgz_step_fused(g: torch.Tensor, ef: torch.Tensor | None, codes: torch.Tensor | None,
                   scales: torch.Tensor | None, out: torch.Tensor, N: int, R: int, B: int,
                   err_scale: float = 1.0, err_beta: float = 0.0, out_scale: float = 1.0,
                   stream=None, ef_scales: torch.Tensor | None = None) -> None:
    """wc_qgz_step_fused (fp32 or no error buffer), _bf16ef (bf16 ef) or
    _int8ef (int8 ef with fp32 ef_scales [R*N/B]): flat EF-quant +
    dequant-reduce in one kernel.  codes/scales (the send buffers) may both be
    None to skip writing them."""
    d = g.device
    if out.dtype == torch.float32:
        od = WC_F32
    elif out.dtype == torch.bfloat16:
        od = WC_BF16
    else:
        raise TypeError("out must be float32 or bfloat16")
    suffix, err = _fused_error(ef, ef_scales, R * N, B, d)
    _call(d, "wc_qgz_step_fused" + suffix, _dev(g, "g", torch.bfloat16, R * N, d), *err,
          _dev(codes, "codes", torch.uint8, R * N // 2, d),
          _dev(scales, "scales", torch.float32, R * N // B, d), N, R, B, err_scale, err_beta,
          out_scale, _dev(out, "out", out.dtype, N, d), od, _stream(g, stream))


def qgz_first_hop_fused(g: torch.Tensor, ef: torch.Tensor | None, codes: torch.Tensor | None,
                        scales: torch.Tensor | None, out_codes: torch.Tensor,
                        out_scales: torch.Tensor, N: int, R: int, G: int, B: int,
                        err_scale: float = 1.0, err_beta: float = 0.0, stream=None,
                        ef1: torch.Tensor | None = None,
                        ef_scales: torch.Tensor | None = None) -> None:
    """wc_qgz_first_hop_fused (fp32 or no error buffer), _bf16ef or _int8ef
    (by ef's dtype, as qgz_step_fused): every rank's EF-quant and the first
    hop in one kernel.  codes/scales (the send buffers) may both be None to
    skip writing them; out_codes/out_scales receive the first hop's output;
    ef1 (fp32 [G*N], or None) is the first hop's own error buffer."""
    d = g.device
    suffix, err = _fused_error(ef, ef_scales, R * N, B, d)
    _call(d, "wc_qgz_first_hop_fused" + suffix, _dev(g, "g", torch.bfloat16, R * N, d), *err,
          _dev(codes, "codes", torch.uint8, R * N // 2, d),
          _dev(scales, "scales", torch.float32, R * N // B, d), N, R, G, B, err_scale, err_beta,
          _dev(out_codes, "out_codes", torch.uint8, G * N // 2, d),
          _dev(out_scales, "out_scales", torch.float32, G * N // B, d),
          _dev(ef1, "ef1", torch.float32, G * N, d), _stream(g, stream))


def qwz_quant_int8(w: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, B: int,
                   stream=None) -> None:
    n = w.numel()
    d = w.device
    _call(d, "wc_qwz_quant_int8", _dev(w, "w", torch.bfloat16, n, d),
          _dev(codes, "codes", torch.int8, n, d), _dev(scales, "scales", torch.float32, n // B, d),
          n, B, _stream(w, stream))


def ef_quant_int4_bf16ef(g: torch.Tensor, ef16: torch.Tensor, codes: torch.Tensor,
                         scales: torch.Tensor, N: int, R: int, G: int, B: int,
                         err_scale: float = 1.0, err_beta: float = 0.0, stream=None) -> None:
    """wc_ef_quant_int4_bf16ef: as ef_quant_int4 with a bf16 error buffer."""
    d = g.device
    _call(d, "wc_ef_quant_int4_bf16ef", _dev(g, "g", torch.bfloat16, R * N, d),
          _dev(ef16, "ef16", torch.bfloat16, R * N, d),
          _dev(codes, "codes", torch.uint8, R * N // 2, d),
          _dev(scales, "scales", torch.float32, R * N // B, d), N, R, G, B, err_scale, err_beta,
          _stream(g, stream))


def ef_quant_int4_int8ef(g: torch.Tensor, ef8: torch.Tensor, ef8_scales: torch.Tensor,
                         codes: torch.Tensor, scales: torch.Tensor, N: int, R: int, G: int, B: int,
                         err_scale: float = 1.0, err_beta: float = 0.0, stream=None) -> None:
    """wc_ef_quant_int4_int8ef: as ef_quant_int4 with an int8 error buffer
    (ef8 int8 [R*N] codes, ef8_scales fp32 [R*N/B], both in place)."""
    d = g.device
    _call(d, "wc_ef_quant_int4_int8ef", _dev(g, "g", torch.bfloat16, R * N, d),
          _dev(ef8, "ef8", torch.int8, R * N, d),
          _dev(ef8_scales, "ef8_scales", torch.float32, R * N // B, d),
          _dev(codes, "codes", torch.uint8, R * N // 2, d),
          _dev(scales, "scales", torch.float32, R * N // B, d), N, R, G, B, err_scale, err_beta,
          _stream(g, stream))


def qwz_quant_replica_int8(w: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                           replica: torch.Tensor, B: int, stream=None) -> None:
    """wc_qwz_quant_replica_int8: codes, scales and the bf16 replica in one pass."""
    n = w.numel()
    d = w.device
    _call(d, "wc_qwz_quant_replica_int8", _dev(w, "w", torch.bfloat16, n, d),
          _dev(codes, "codes", torch.int8, n, d), _dev(scales, "scales", torch.float32, n // B, d),
          _dev(replica, "replica", torch.bfloat16, n, d), n, B, _stream(w, stream))


def qwz_dequant_int8(codes: torch.Tensor, scales: torch.Tensor, w_out: torch.Tensor, B: int,
                     stream=None) -> None:
    n = codes.numel()
    d = codes.device
    _call(d, "wc_qwz_dequant_int8", _dev(codes, "codes", torch.int8, n, d),
          _dev(scales, "scales", torch.float32, n // B, d),
          _dev(w_out, "w_out", torch.bfloat16, n, d), n, B, _stream(codes, stream))


def sr_accumulate_bf16(dst: torch.Tensor, src: torch.Tensor, seed: int, step: int,
                       stream=None) -> None:
    """dst <- SR_bf16(dst + src) in place; src <- 0."""
    n = dst.numel()
    d = dst.device
    _call(d, "wc_sr_accumulate_bf16", _dev(dst, "dst", torch.bfloat16, n, d),
          _dev(src, "src", torch.bfloat16, n, d), n, seed & 0xFFFFFFFF, step & 0xFFFFFFFF,
          _stream(dst, stream))


def _float_type(t: torch.Tensor, name: str) -> int:
    if t.dtype == torch.float32:
        return WC_F32
    if t.dtype == torch.bfloat16:
        return WC_BF16
    raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")


def _matrix(t: torch.Tensor, name: str, rows: int, cols: int, device):
    """Pointer and row stride of a CUDA matrix [rows, >= cols] whose rows are
    consecutive values."""
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] < cols:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected ({rows}, {cols})")
    ld, step = t.stride()
    if shape[1] > 1 and step != 1:
        raise ValueError(f"{name} must have consecutive values in a row")
    if rows <= 1:
        ld = shape[1]
    elif ld < shape[1]:
        raise ValueError(f"{name} must not have overlapping rows")
    return t.data_ptr(), ld


def _ids(ids: torch.Tensor, device) -> tuple:
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids must be int32 or int64, got {ids.dtype}")
    if ids.device != device:
        raise ValueError(f"ids is on {ids.device}, expected {device}")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    return ids.data_ptr(), WC_I64 if ids.dtype == torch.int64 else WC_I32


def _workspace(t: torch.Tensor, device) -> tuple:
    if t.dtype != torch.uint8:
        raise TypeError(f"workspace must be uint8, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"workspace is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t.data_ptr(), t.numel()


def embedding_grad(dy: torch.Tensor, ids: torch.Tensor, dtable: torch.Tensor,
                   workspace: torch.Tensor, scale: float = 1.0, first_row: int = 0,
                   accumulate: bool = False, stream=None) -> None:
    """wc_embedding_grad: dtable [V, D] <- (or +=) scale * the sum of dy's rows
    over the tokens of each row; workspace uint8."""
    d = dy.device
    if dtable.dim() != 2:
        raise ValueError(f"dtable must be a matrix, got shape {tuple(dtable.shape)}")
    V, D = dtable.shape
    n = ids.numel()
    yp, ld_dy = _matrix(dy, "dy", n, D, d)
    if dy.shape[1] != D:
        raise ValueError(f"dy has {dy.shape[1]} columns, dtable {D}")
    ip, it = _ids(ids, d)
    op, ld_out = _matrix(dtable, "dtable", V, D, d)
    _call(d, "wc_embedding_grad", yp, _float_type(dy, "dy"), ld_dy, ip, it, n, first_row, V, D,
          scale, 1 if accumulate else 0, op, _float_type(dtable, "dtable"), ld_out,
          *_workspace(workspace, d), _stream(dy, stream))


def _fp8_part(codes, scales, name: str, rows: int, cols: int, square: bool, device):
    """Pointers and strides of codes [rows, >= cols], with room for their rows'
    padding to 16 bytes, and scales [ceil(cols/128), >= rows or ceil(rows/128)],
    or NULLs."""
    if (codes is None) != (scales is None):
        raise ValueError(f"{name}: codes and scales must both be given or both be None")
    if codes is None:
        return None, 0, None, 0
    if codes.dtype != torch.float8_e4m3fn:
        raise TypeError(f"{name} codes must be float8_e4m3fn, got {codes.dtype}")
    if scales.dtype != torch.float32:
        raise TypeError(f"{name} scales must be float32, got {scales.dtype}")
    per = -(-rows // 128) if square else rows
    padded = -(-cols // 16) * 16
    cp, ld = _matrix(codes, f"{name} codes", rows, padded, device)
    if rows <= 1 or codes.shape[1] == 0:
        ld = padded  # there is no second row to be apart from
    sp, lds = _matrix(scales, f"{name} scales", -(-cols // 128), per, device)
    return cp, ld, sp, lds


def fp8_quant(x: torch.Tensor, codes: torch.Tensor | None, scales: torch.Tensor | None,
              codes_t: torch.Tensor | None = None, scales_t: torch.Tensor | None = None,
              square: bool = False, stream=None) -> None:
    """wc_fp8_quant: x [rows, cols] to e4m3 codes and scales by blocks of 128
    along the columns (codes, scales), along the rows of the transposed matrix
    (codes_t, scales_t), or both; square: one scale per 128 x 128."""
    if x.dim() != 2:
        raise ValueError(f"x must be a matrix, got shape {tuple(x.shape)}")
    d = x.device
    rows, cols = x.shape
    xp, ld = _matrix(x, "x", rows, cols, d)
    q, ldq, s, lds = _fp8_part(codes, scales, "row", rows, cols, square, d)
    qt, ldqt, st, ldst = _fp8_part(codes_t, scales_t, "transposed", cols, rows, square, d)
    _call(d, "wc_fp8_quant", xp, _float_type(x, "x"), rows, cols, ld, 1 if square else 0,
          q, ldq, s, lds, qt, ldqt, st, ldst, _stream(x, stream))
