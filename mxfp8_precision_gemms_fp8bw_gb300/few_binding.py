"""ctypes binding of the third part of libfp8bw.so's C ABI (``include/fp8bw_few.h``):
MX weights in 4 bits, and products of a few tokens with MX weights, under the same names.

Like ``binding``: argument marshalling only, with checks of each tensor's
dtype, device, layout and shape, and ``Fp8bwError`` on a nonzero status.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

from . import binding as B
from .moe_binding import _BF16, _F32, _F32C, _I64, _INT, _P, _SIZE, _U8, SCORE_SOFTMAX, _arg, _stream

FEW_TOKENS = 32
_U32 = ctypes.c_uint32

_SIGNATURES = {
    "mxfp4_quant_1x32_row": [_P, _I64, _I64, _P, _P, _INT, _P],
    "mxfp4_to_mxfp8": [_P, _I64, _I64, _P, _P],
    "mx_few_linear_workspace_bytes": [_I64, _I64, _I64],
    "mx_few_linear": [_P, _P, _P, _INT, _I64, _I64, _I64, _P, _P, _SIZE, _P],
    "mx_few_moe_workspace_bytes": [_I64, _I64, _I64, _I64, _I64],
    "mx_few_moe": [_P, _P, _P, _P, _P, _P, _P, _INT, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _INT, _INT, _F32C, _P,
                   _P, _SIZE, _P],
    "mx_few_linear_shape": [_I64, _I64, _I64, _INT, _P],
    "mx_few_moe_shape": [_I64, _I64, _I64, _I64, _I64, _INT, _P, _P, _P],
    "fp8bw_selftest_few_linear": [_P, _P, _P, _INT, _I64, _I64, _I64, _P, _P, _SIZE, _U32, _P],
    "fp8bw_selftest_few_moe": [_P, _P, _P, _P, _P, _P, _P, _INT, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _INT, _INT, _F32C,
                               _P, _P, _SIZE, _U32, _P],
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
            fn.restype = _SIZE if name.endswith("_workspace_bytes") else _INT
        _LIB = handle
    return _LIB


def mxfp4_quant_1x32_row(w, q, e8, mode=B.MX_RCEIL, stream=None) -> None:
    *lead, C = w.shape
    R = math.prod(lead)
    B._check(lib().mxfp4_quant_1x32_row(_arg(w, _BF16, "w", *lead, C), R, C, _arg(q, _U8, "q", *lead, C // 2),
                                        _arg(e8, _U8, "e8", R, C // 32), mode, _stream(stream, w)))


def mxfp4_to_mxfp8(q4, q8, stream=None) -> None:
    *lead, C = q8.shape
    B._check(lib().mxfp4_to_mxfp8(_arg(q4, _U8, "q4", *lead, C // 2), math.prod(lead), C, _arg(q8, _U8, "q8", *lead, C),
                                  _stream(stream, q4)))


def mx_few_linear_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().mx_few_linear_workspace_bytes(M, N, K))


def _linear_args(x, w, e8, bits, y, workspace):
    M, K = x.shape
    N, n = w.shape[0], 0 if workspace is None else workspace.shape[0]
    return (_arg(x, _BF16, "x", M, K), _arg(w, _U8, "w", N, K * bits // 8), _arg(e8, _U8, "e8", N, K // 32), bits, M, N, K,
            _arg(y, _BF16, "y", M, N), _arg(workspace, _U8, "workspace", n), n)


def mx_few_linear(x, w, e8, bits, y, workspace=None, stream=None) -> None:
    B._check(lib().mx_few_linear(*_linear_args(x, w, e8, bits, y, workspace), _stream(stream, x)))


def fp8bw_selftest_few_linear(x, w, e8, bits, y, workspace=None, wait_ns=0, stream=None) -> None:
    B._check(lib().fp8bw_selftest_few_linear(*_linear_args(x, w, e8, bits, y, workspace), wait_ns, _stream(stream, x)))


def mx_few_moe_workspace_bytes(M: int, E: int, top_k: int, C: int, F: int) -> int:
    return int(lib().mx_few_moe_workspace_bytes(M, E, top_k, C, F))


def _moe_args(x, router, bias, w13, e13, w2, e2, bits, top_k, y, workspace, groups, groups_kept, group_top, score, renorm, scale):
    M, C = x.shape
    E, F2 = w13.shape[:2]
    F, n = F2 // 2, workspace.shape[0]
    return (_arg(x, _BF16, "x", M, C), _arg(router, _F32, "router", E, C), _arg(bias, _F32, "bias", E),
            _arg(w13, _U8, "w13", E, 2 * F, C * bits // 8), _arg(e13, _U8, "e13", E * 2 * F, C // 32),
            _arg(w2, _U8, "w2", E, C, F * bits // 8), _arg(e2, _U8, "e2", E * C, F // 32), bits, M, E, top_k, C, F, groups,
            groups_kept, group_top, score, int(renorm), scale, _arg(y, _BF16, "y", M, C), _arg(workspace, _U8, "workspace", n), n)


def mx_few_moe(x, router, bias, w13, e13, w2, e2, bits, top_k, y, workspace, groups=1, groups_kept=1, group_top=1,
               score=SCORE_SOFTMAX, renorm=True, scale=1.0, stream=None) -> None:
    B._check(lib().mx_few_moe(*_moe_args(x, router, bias, w13, e13, w2, e2, bits, top_k, y, workspace, groups, groups_kept,
                                         group_top, score, renorm, scale), _stream(stream, x)))


def fp8bw_selftest_few_moe(x, router, bias, w13, e13, w2, e2, bits, top_k, y, workspace, groups=1, groups_kept=1, group_top=1,
                           score=SCORE_SOFTMAX, renorm=True, scale=1.0, wait_ns=0, stream=None) -> None:
    B._check(lib().fp8bw_selftest_few_moe(*_moe_args(x, router, bias, w13, e13, w2, e2, bits, top_k, y, workspace, groups,
                                                     groups_kept, group_top, score, renorm, scale), wait_ns, _stream(stream, x)))


class ProductShape(NamedTuple):
    """How a product is divided."""
    cluster: int
    stages: int
    chunks: int
    in_turn: int
    held: int
    spread: int


def mx_few_linear_shape(M: int, N: int, K: int, bits: int) -> ProductShape:
    product = (ctypes.c_int32 * 6)()
    B._check(lib().mx_few_linear_shape(M, N, K, bits, product))
    return ProductShape(*product)


def mx_few_moe_shape(M: int, E: int, top_k: int, C: int, F: int, bits: int) -> tuple[ProductShape, ProductShape, int]:
    """Of the two products, and the slices of the logits."""
    up, down, slices = (ctypes.c_int32 * 6)(), (ctypes.c_int32 * 6)(), (ctypes.c_int32 * 1)()
    B._check(lib().mx_few_moe_shape(M, E, top_k, C, F, bits, up, down, slices))
    return ProductShape(*up), ProductShape(*down), slices[0]
