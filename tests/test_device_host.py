"""Tensors of another device than the current one are refused on the host, by both bindings (no GPU needed: the tensors are
stand-ins, and nothing is launched)."""
import pytest
import torch

from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import build
from mxfp8_precision_gemms_fp8bw_gb300 import moe_binding as MB

U8, F32, I32, BF = torch.uint8, torch.float32, torch.int32, torch.bfloat16


class On:
    """What the bindings ask of a CUDA tensor, on a device of its own."""
    is_cuda = True

    def __init__(self, device, dtype, *shape):
        self.device_index, self.dtype, self.shape = device, dtype, torch.Size(shape)

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.device_index

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 1 << 20


def calls(d):
    """Calls of both bindings, d(i) the device of the i-th tensor."""
    return {
        "route": lambda: MB.fp8bw_moe_route(On(d(0), F32, 4, 8), On(d(1), F32, 8), 2, On(d(2), I32, 4, 2),
                                            On(d(3), F32, 4, 2), stream=0),
        "plan": lambda: MB.fp8bw_moe_plan(On(d(0), I32, 4, 2), 8, On(d(1), I32, 8), On(d(2), I32, 8), On(d(3), I32, 4, 2),
                                          On(d(4), I32, 256), stream=0),
        "gather": lambda: MB.mxfp8_moe_gather_quant(On(d(0), BF, 4, 32), None, On(d(1), I32, 32), 2, On(d(2), U8, 32, 32),
                                                    On(d(3), U8, 32, 1), stream=0),
        "combine": lambda: MB.fp8bw_moe_combine(On(d(0), BF, 32, 32), None, On(d(1), I32, 4, 2), None, On(d(2), BF, 4, 32),
                                                stream=0),
        "swiglu": lambda: MB.mxfp8_swiglu(On(d(0), BF, 32, 64), On(d(1), U8, 32, 32), On(d(2), U8, 32, 1), stream=0),
        "row quantizer": lambda: B.mxfp8_quant_1x32_row(On(d(0), BF, 32, 32), On(d(1), U8, 32, 32), On(d(2), U8, 32, 1),
                                                        stream=0),
        "expert quantizer": lambda: B.mxfp8_quant_1x32_rowcol(On(d(0), BF, 2, 32, 32), On(d(1), U8, 64, 32),
                                                              On(d(2), U8, 64, 1), On(d(3), U8, 2, 32, 32),
                                                              On(d(4), U8, 2, 32, 1), stream=0),
        "grouped gemm": lambda: B.mxfp8_grouped_gemm(0, On(d(0), U8, 32, 256), On(d(1), U8, 32, 8),
                                                     On(d(2), U8, 1, 256, 256), On(d(3), U8, 256, 8), On(d(4), I32, 1), 1, 32,
                                                     256, 256, On(d(5), BF, 32, 256), On(d(6), U8, 4096), stream=0),
    }


TENSORS = {"route": 4, "plan": 5, "gather": 4, "combine": 3, "swiglu": 3, "row quantizer": 3, "expert quantizer": 5,
           "grouped gemm": 7}


@pytest.fixture(autouse=True)
def _no_launch(monkeypatch):
    """Device 0 of several is current, and a call that reaches the library ends there."""
    build.build()
    monkeypatch.setattr(B, "_one_device", False, raising=False)
    monkeypatch.setattr(B, "_current_device", lambda: 0, raising=False)

    class Library:
        def __getattr__(self, name):
            return lambda *a: (_ for _ in ()).throw(AssertionError(f"{name} was called"))

    monkeypatch.setattr(B, "lib", Library)
    monkeypatch.setattr(MB, "lib", Library)


@pytest.mark.parametrize("name", sorted(TENSORS))
def test_refused(name):
    with pytest.raises(ValueError, match="cuda:1"):
        calls(lambda i: 1)[name]()
    for n in range(TENSORS[name]):
        with pytest.raises(ValueError, match="cuda:1"):
            calls(lambda i: int(i == n))[name]()


@pytest.mark.parametrize("name", sorted(TENSORS))
def test_let_through_on_the_current_device(name):
    with pytest.raises(AssertionError, match="was called"):
        calls(lambda i: 0)[name]()


def test_one_device_is_never_asked(monkeypatch):
    monkeypatch.setattr(B, "_one_device", None)
    monkeypatch.setattr(torch._C, "_cuda_getDeviceCount", lambda: 1, raising=False)
    monkeypatch.setattr(B, "_current_device", lambda: pytest.fail("asked"))
    for name in TENSORS:
        with pytest.raises(AssertionError, match="was called"):
            calls(lambda i: 0)[name]()
    assert B._one_device is True


def test_several_devices_are_counted_once(monkeypatch):
    counted = []
    monkeypatch.setattr(B, "_one_device", None)
    monkeypatch.setattr(torch._C, "_cuda_getDeviceCount", lambda: counted.append(1) or 2, raising=False)
    with pytest.raises(ValueError, match="cuda:1"):
        calls(lambda i: 1)["route"]()
    with pytest.raises(AssertionError, match="was called"):
        calls(lambda i: 0)["route"]()
    assert counted == [1] and B._one_device is False
