"""ctypes binding of the second part of libfp8bw.so's C ABI (``include/fp8bw_moe.h``):
the operators around the experts' products, under the same names.

Like ``binding``: argument marshalling only, with checks of each tensor's
dtype, device, layout and shape, and ``Fp8bwError`` on a nonzero status.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as B

SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
MAX_EXPERTS, MAX_TOP_K, MAX_GROUPS = 1024, 32, 32

_P, _I64, _INT, _F32C, _SIZE = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t

_SIGNATURES = {
    "fp8bw_moe_route": [_P, _INT, _P, _I64, _I64, _I64, _I64, _I64, _I64, _INT, _INT, _F32C, _P, _P, _P],
    "fp8bw_moe_route_bwd": [_P, _P, _INT, _P, _I64, _I64, _I64, _INT, _INT, _F32C, _P, _P],
    "fp8bw_moe_plan_rows": [_I64, _I64, _I64],
    "fp8bw_moe_plan_workspace_bytes": [_I64, _I64, _I64],
    "fp8bw_moe_plan": [_P, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _SIZE, _P],
    "mxfp8_moe_gather_quant": [_P, _P, _P, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _INT, _P],
    "fp8bw_moe_combine": [_P, _P, _P, _P, _I64, _I64, _I64, _I64, _P, _P],
    "fp8bw_moe_combine_dweights": [_P, _P, _P, _I64, _I64, _I64, _I64, _P, _P],
    "mxfp8_swiglu": [_P, _I64, _I64, _P, _P, _P, _P, _P, _P, _INT, _P],
    "mxfp8_swiglu_bwd": [_P, _P, _P, _I64, _I64, _P, _P, _P, _P, _INT, _P],
}

_LIB = None


def lib() -> ctypes.CDLL:
    """libfp8bw.so with the calls of this part declared; raises if it has not been built."""
    global _LIB
    if _LIB is None:
        handle = B.lib()
        for name, args in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = {"fp8bw_moe_plan_rows": _I64, "fp8bw_moe_plan_workspace_bytes": _SIZE}.get(name, _INT)
        _LIB = handle
    return _LIB


_BF16, _U8, _F32, _I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32


def _arg(t: torch.Tensor | None, dtype: torch.dtype, name: str, *shape: int):
    """The tensor's address, once its dtype, device, layout and shape are what the call reads or writes."""
    if t is None:
        return None
    if (t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous()
            and (B._one_device or not B._elsewhere(t))):
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
    return B._ptr(t, dtype, name)  # raises with what is wrong


def _stream(stream, t: torch.Tensor):
    """The stream's handle; None is the current stream of the tensor's device, the current one (``_arg`` checks)."""
    # torch.cuda.current_stream() builds a Stream object: 2.9 us a call on a Grace core, the raw handle 0.1 us
    return torch._C._cuda_getCurrentRawStream(t.get_device()) if stream is None else B._stream(stream)


def _logits(t: torch.Tensor, name: str, *shape: int):
    if t.dtype not in (_F32, _BF16):
        raise TypeError(f"{name}: expected {_F32} or {_BF16}, got {t.dtype}")
    return _arg(t, t.dtype, name, *shape), int(t.dtype == _BF16)


def fp8bw_moe_route(logits, bias, top_k, experts, weights, groups=1, groups_kept=1, group_top=1, score=SCORE_SOFTMAX,
                    renorm=True, scale=1.0, stream=None) -> None:
    M, E = logits.shape
    p, kind = _logits(logits, "logits", M, E)
    B._check(lib().fp8bw_moe_route(p, kind, _arg(bias, _F32, "bias", E), M, E, top_k, groups, groups_kept, group_top,
                                   score, int(renorm), scale, _arg(experts, _I32, "experts", M, top_k),
                                   _arg(weights, _F32, "weights", M, top_k), _stream(stream, logits)))


def fp8bw_moe_route_bwd(dweights, logits, experts, dlogits, score=SCORE_SOFTMAX, renorm=True, scale=1.0,
                        stream=None) -> None:
    M, E = logits.shape
    top_k = experts.shape[1]
    p, kind = _logits(logits, "logits", M, E)
    B._check(lib().fp8bw_moe_route_bwd(_arg(dweights, _F32, "dweights", M, top_k), p, kind,
                                       _arg(experts, _I32, "experts", M, top_k), M, E, top_k, score, int(renorm),
                                       scale, _arg(dlogits, logits.dtype, "dlogits", M, E), _stream(stream, logits)))


def fp8bw_moe_plan_rows(M: int, E: int, top_k: int) -> int:
    return int(lib().fp8bw_moe_plan_rows(M, E, top_k))


def fp8bw_moe_plan_workspace_bytes(M: int, E: int, top_k: int) -> int:
    return int(lib().fp8bw_moe_plan_workspace_bytes(M, E, top_k))


def fp8bw_moe_plan(experts, E, group_end, counts, row_of, src_of, workspace=None, stream=None) -> None:
    M, top_k = experts.shape
    P = src_of.shape[0]
    n = 0 if workspace is None else workspace.numel()
    B._check(lib().fp8bw_moe_plan(_arg(experts, _I32, "experts", M, top_k), M, E, top_k, P,
                                  _arg(group_end, _I32, "group_end", E), _arg(counts, _I32, "counts", E),
                                  _arg(row_of, _I32, "row_of", M, top_k), _arg(src_of, _I32, "src_of", P),
                                  _arg(workspace, _U8, "workspace", n), n,
                                  _stream(stream, experts)))


def mxfp8_moe_gather_quant(x, weights, src_of, top_k, q, e8, qT=None, e8T=None, mode=B.MX_RCEIL, stream=None) -> None:
    M, C = x.shape
    P = src_of.shape[0]
    B._check(lib().mxfp8_moe_gather_quant(_arg(x, _BF16, "x", M, C), _arg(weights, _F32, "weights", M, top_k),
                                          _arg(src_of, _I32, "src_of", P), M, top_k, P, C, _arg(q, _U8, "q", P, C),
                                          _arg(e8, _U8, "e8", P, C // 32), _arg(qT, _U8, "qT", C, P),
                                          _arg(e8T, _U8, "e8T", C, P // 32), mode, _stream(stream, x)))


def fp8bw_moe_combine(y, weights, row_of, base, out, stream=None) -> None:
    M, top_k = row_of.shape
    P, C = y.shape
    B._check(lib().fp8bw_moe_combine(_arg(y, _BF16, "y", P, C), _arg(weights, _F32, "weights", M, top_k),
                                     _arg(row_of, _I32, "row_of", M, top_k), _arg(base, _BF16, "base", M, C), M, top_k,
                                     P, C, _arg(out, _BF16, "out", M, C), _stream(stream, y)))


def fp8bw_moe_combine_dweights(dout, y, row_of, dweights, stream=None) -> None:
    M, top_k = row_of.shape
    P, C = y.shape
    B._check(lib().fp8bw_moe_combine_dweights(_arg(dout, _BF16, "dout", M, C), _arg(y, _BF16, "y", P, C),
                                              _arg(row_of, _I32, "row_of", M, top_k), M, top_k, P, C,
                                              _arg(dweights, _F32, "dweights", M, top_k), _stream(stream, y)))


def mxfp8_swiglu(h, aq, ae, aqT=None, aeT=None, hq=None, he=None, mode=B.MX_RCEIL, stream=None) -> None:
    R, F = h.shape[0], h.shape[1] // 2
    B._check(lib().mxfp8_swiglu(_arg(h, _BF16, "h", R, 2 * F), R, F, _arg(aq, _U8, "aq", R, F),
                                _arg(ae, _U8, "ae", R, F // 32), _arg(aqT, _U8, "aqT", F, R),
                                _arg(aeT, _U8, "aeT", F, R // 32), _arg(hq, _U8, "hq", R, 2 * F),
                                _arg(he, _U8, "he", R, F // 16), mode, _stream(stream, h)))


def mxfp8_swiglu_bwd(da, hq, he, dq, de, dqT, deT, mode=B.MX_RCEIL, stream=None) -> None:
    R, F = da.shape
    B._check(lib().mxfp8_swiglu_bwd(_arg(da, _BF16, "da", R, F), _arg(hq, _U8, "hq", R, 2 * F),
                                    _arg(he, _U8, "he", R, F // 16), R, F, _arg(dq, _U8, "dq", R, 2 * F),
                                    _arg(de, _U8, "de", R, F // 16), _arg(dqT, _U8, "dqT", 2 * F, R),
                                    _arg(deT, _U8, "deT", 2 * F, R // 32), mode, _stream(stream, da)))
