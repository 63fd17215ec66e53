"""The MXFP8 mixture-of-experts layer end to end: its output and gradients against the same layer in fp32 with the same
choices, and the example that trains it."""
import importlib.util
import os

import pytest
import torch

from gpu_util import lib
from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import moe

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib()


def sqnr(ref, got):
    ref, got = ref.detach().double(), got.detach().double()
    return float(10 * torch.log10(ref.square().sum() / (ref - got).square().sum()))


def reference(layer, x, experts):
    """The layer in fp32 torch on the given choices."""
    top_k, score, renormalize, scale = layer.how[:4]
    logits = x @ layer.router.t()
    s = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    w = s.gather(1, experts.long())
    w = scale * (w / w.sum(1, keepdim=True) if renormalize else w)
    out = torch.zeros_like(x)
    for e in range(layer.w13.shape[0]):
        gate, up = (x @ layer.w13[e].t()).chunk(2, dim=1)
        y = (torch.nn.functional.silu(gate) * up) @ layer.w2[e].t()
        out = out + y * (w * (experts == e)).sum(1, keepdim=True)
    return out


@pytest.mark.parametrize("tokens,experts,top_k,score", [(1000, 4, 2, "softmax"), (37, 8, 3, "sigmoid"), (1, 8, 2, "softmax")])
def test_layer_against_fp32(tokens, experts, top_k, score):
    torch.manual_seed(tokens)
    dim, hidden = 256, 512
    layer = moe.MxMoEFFN(dim, hidden, experts, top_k, score=score, scale=1.5, device="cuda")
    x = torch.randn(tokens, dim, device="cuda").bfloat16().requires_grad_(True)
    dout = torch.randn(tokens, dim, device="cuda").bfloat16()
    out = layer(x)
    out.backward(dout)
    B.fp8bw_sync_status()
    assert int(layer.counts.sum()) == tokens * top_k

    ref = moe.MxMoEFFN(dim, hidden, experts, top_k, score=score, scale=1.5, device="cuda").float()
    ref.load_state_dict({n: v.float() for n, v in layer.state_dict().items()})
    xf = x.detach().float().requires_grad_(True)
    chosen = moe.route(torch.nn.functional.linear(xf.detach(), ref.router), top_k, score=score)[0]
    want = reference(ref, xf, chosen)
    want.backward(dout.float())
    # e4m3 in blocks of 32 is off by 2.6 % rms (31.7 dB) per operand.  Six of them reach the output (the two operands of
    # each product and the activation's two factors): 31.7 - 10 log10(6) = 23.9 dB.  Ten to twelve reach a gradient with
    # the kept activation among them: about 21 dB.  3 dB of margin, and 6 for the router, whose gradient is a difference.
    assert sqnr(want, out) >= 20.9
    for got, ref_grad in ((x.grad, xf.grad), (layer.w13.grad, ref.w13.grad), (layer.w2.grad, ref.w2.grad)):
        assert sqnr(ref_grad, got) >= 18.0
    assert sqnr(ref.router.grad, layer.router.grad) >= 15.0


def test_inference_keeps_nothing_and_agrees():
    torch.manual_seed(1)
    layer = moe.MxMoEFFN(256, 256, 8, 2, device="cuda")
    x = torch.randn(50, 256, device="cuda").bfloat16()
    out = layer(x)
    assert out.requires_grad
    with torch.no_grad():
        assert torch.equal(layer(x), out)


@pytest.mark.parametrize("how", ["no_grad", "frozen"])
def test_inference_makes_nothing_for_backward(how, monkeypatch):
    layer = moe.MxMoEFFN(256, 256, 8, 2, device="cuda").requires_grad_(how != "frozen")
    x = torch.randn(50, 256, device="cuda").bfloat16()
    made = []
    quantized, activation = moe.MB.mxfp8_moe_gather_quant, moe.MB.mxfp8_swiglu
    monkeypatch.setattr(moe.MB, "mxfp8_moe_gather_quant", lambda *a: (made.append(a[6:8]), quantized(*a)))
    monkeypatch.setattr(moe.MB, "mxfp8_swiglu", lambda *a, **k: (made.append(a[3:7]), activation(*a, **k)))
    with torch.set_grad_enabled(how == "frozen"):
        layer(x)
    assert made == [(None, None), (None,) * 4]


def test_kept_weight_codes_change_nothing():
    torch.manual_seed(2)
    layer = moe.MxMoEFFN(256, 512, 4, 2, device="cuda")
    codes = layer.weight_codes()
    grads = []
    for kept in (None, codes):
        x = torch.randn(70, 256, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).bfloat16().requires_grad_(True)
        layer.zero_grad()
        out = layer(x) if kept is None else layer(x, kept)
        out.backward(torch.ones_like(out))
        grads.append((out, x.grad, layer.w13.grad, layer.w2.grad, layer.router.grad))
    assert all(torch.equal(a, b) for a, b in zip(*grads))
    with torch.no_grad():
        assert torch.equal(layer(x, codes), grads[0][0])


def test_a_batch_without_tokens():
    """Outputs of no rows, empty groups, and gradients of zero."""
    logits = torch.empty(0, 8, device="cuda")
    experts, weights = moe.route(logits, 2)
    assert experts.shape == weights.shape == (0, 2)
    assert moe.route_backward(weights, logits, experts).shape == (0, 8)
    p = moe.plan(experts, 8)
    assert p.group_end.tolist() == [0] * 7 + [p.rows] and p.rows % 32 == 0
    assert not p.counts.any() and bool((p.src_of == -1).all()) and p.row_of.shape == (0, 2)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    rows = moe.dispatch(x, p)
    assert rows.qT.shape == (64, p.rows) and not any(t.any() for t in (rows.q, rows.e8, rows.qT, rows.e8T))
    y = torch.ones(p.rows, 64, dtype=torch.bfloat16, device="cuda")
    assert moe.combine(y, weights, p).shape == (0, 64)
    dy, dw = moe.combine_backward(x, y, weights, p)
    assert not dy.qT.any() and dw.shape == (0, 2)

    layer = moe.MxMoEFFN(256, 256, 4, 2, device="cuda")
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    out = layer(x)
    out.backward(torch.empty_like(out))
    B.fp8bw_sync_status()
    assert out.shape == x.grad.shape == (0, 256)
    assert not layer.w13.grad.any() and not layer.w2.grad.any() and not layer.router.grad.any()


def test_update_balance_moves_against_the_load():
    layer = moe.MxMoEFFN(256, 256, 4, 1, device="cuda")
    with pytest.raises(RuntimeError):
        layer.update_balance()
    layer.counts = torch.tensor([10, 0, 5, 5], dtype=torch.int32, device="cuda")
    layer.update_balance(0.5)
    assert layer.balance.tolist() == [-0.5, 0.5, 0.0, 0.0]


def test_example_learns():
    spec = importlib.util.spec_from_file_location("moe_ffn_example", os.path.join(ROOT, "examples", "moe_ffn.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, together, alone = example.main()
    assert losses[-1] < 0.9 * losses[0]
    assert torch.equal(together, alone)
