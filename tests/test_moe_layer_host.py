"""The mixture-of-experts layer's host side (no GPU needed: what it refuses before a launch, and its autograd functions with
the kernels replaced by torch)."""
import dataclasses

import pytest
import torch

from mxfp8_precision_gemms_fp8bw_gb300 import linear as L
from mxfp8_precision_gemms_fp8bw_gb300 import moe


def codes_like(layer):
    u8 = lambda *shape: torch.zeros(shape, dtype=torch.uint8)  # noqa: E731
    return tuple(L.MxExpertWeights(u8(E, N, K), u8(E * N, K // 32), u8(E, K, N), u8(E, K, N // 32))
                 for E, N, K in (layer.w13.shape, layer.w2.shape))


@pytest.mark.parametrize("which,name", [(i, f.name) for i in (0, 1) for f in dataclasses.fields(L.MxExpertWeights)])
def test_codes_of_other_weights_are_refused(which, name):
    layer = moe.MxMoEFFN(256, 512, 4, 2)
    fewer = moe.MxMoEFFN(256, 512, 2, 2)
    x = torch.zeros(5, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="codes"):
        layer(x, codes_like(fewer))
    with pytest.raises(ValueError, match="codes"):
        layer(x, codes_like(layer)[::-1])
    codes = codes_like(layer)
    setattr(codes[which], name, getattr(codes[which], name)[1:])
    with pytest.raises(ValueError, match=name):
        layer(x, codes)
