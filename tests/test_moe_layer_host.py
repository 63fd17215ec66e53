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


def test_rowwise_codes_are_refused_where_a_gradient_reads_the_others(monkeypatch):
    layer = moe.MxMoEFFN(256, 512, 4, 2)
    codes = tuple(dataclasses.replace(c, qT_col=None, e8_col=None) for c in codes_like(layer))
    x = torch.zeros(5, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="colwise"):
        layer(x, codes)

    class Reached(Exception):
        pass

    def route(*a, **k):
        raise Reached

    monkeypatch.setattr(moe, "route", route)
    with torch.no_grad(), pytest.raises(Reached):
        layer(x, codes)
    with pytest.raises(Reached):
        layer.requires_grad_(False)(x, codes)


# ------------------------------------------------------------------ second derivatives

def plain_route(logits, top_k, *, bias=None, score="softmax", renormalize=True, scale=1.0, groups=1, groups_kept=1,
                group_top=1):
    s = torch.softmax(logits.detach(), 1)
    w, experts = s.topk(top_k, dim=1)
    return experts.to(torch.int32), scale * (w / w.sum(1, keepdim=True) if renormalize else w)


def plain_route_backward(dweights, logits, experts, *, score="softmax", renormalize=True, scale=1.0):
    with torch.enable_grad():
        leaf = logits.detach().requires_grad_(True)
        w = torch.softmax(leaf, 1).gather(1, experts.long())
        w = scale * (w / w.sum(1, keepdim=True) if renormalize else w)
        return torch.autograd.grad(w, leaf, dweights.detach())[0]


def routed(monkeypatch):
    """Weights of tokens through the router product and _Route, whose kernels are these formulas in torch."""
    monkeypatch.setattr(moe, "route", plain_route)
    monkeypatch.setattr(moe, "route_backward", plain_route_backward)
    torch.manual_seed(0)
    x = torch.randn(6, 16, requires_grad=True)
    router = torch.randn(8, 16, requires_grad=True)
    logits = torch.nn.functional.linear(x, router)
    _, weights = moe._Route.apply(logits, None, 2, "softmax", True, 1.0, 1, 1, 1)
    return x, router, logits, weights


def test_the_first_derivative_is_autograds(monkeypatch):
    x, router, logits, weights = routed(monkeypatch)
    dw = torch.randn(6, 2)
    s = torch.softmax(logits, 1).topk(2, dim=1)[0]
    want = torch.autograd.grad(s / s.sum(1, keepdim=True), (x, router), dw, retain_graph=True)
    for a, b in zip(torch.autograd.grad(weights, (x, router), dw), want):
        assert torch.allclose(a, b, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("linear", [True, False])
def test_a_second_derivative_is_an_error(monkeypatch, linear):
    """The kernels' gradients have no graph: what autograd would make of the products around them is part of an answer.
    Whether the loss is linear in the weights or not, so that the incoming gradient does or does not have one."""
    x, router, _, weights = routed(monkeypatch)
    dw = torch.randn(6, 2)
    loss = (weights * dw).sum() if linear else weights.square().sum()
    with pytest.raises(RuntimeError, match="no second derivative"):
        (dx,) = torch.autograd.grad(loss, x, create_graph=True)
        torch.autograd.grad(dx.square().sum(), router)


# ------------------------------------------------------------------ the router product

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_router_product_stays_fp32_under_autocast(dtype):
    torch.manual_seed(1)
    x = torch.randn(9, 32).bfloat16().requires_grad_(True)
    router = torch.randn(8, 32, requires_grad=True)
    d = torch.randn(9, 8)
    want = torch.nn.functional.linear(x.float(), router)
    wants = torch.autograd.grad(want, (x, router), d)
    with torch.autocast("cpu", dtype=dtype):
        got = moe._RouterLogits.apply(x.float(), router)
        gots = torch.autograd.grad(got, (x, router), d)
    assert got.dtype == torch.float32 and torch.equal(got, want)
    for a, b in zip(gots, wants):
        assert a.dtype == b.dtype and torch.allclose(a, b, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("frozen", ["x", "router"])
def test_router_product_keeps_what_its_gradients_read(frozen):
    torch.manual_seed(2)
    x = torch.randn(9, 32, requires_grad=frozen != "x")
    router = torch.randn(8, 32, requires_grad=frozen != "router")
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: (kept.append(t), t)[1], lambda t: t):
        out = moe._RouterLogits.apply(x, router)
    assert [t.data_ptr() for t in kept] == [(x if frozen == "x" else router).data_ptr()]
    out.sum().backward()
    want = torch.ones(9, 8)
    if frozen == "x":
        assert x.grad is None and torch.allclose(router.grad, want.t() @ x, rtol=1e-5, atol=1e-6)
    else:
        assert router.grad is None and torch.allclose(x.grad, want @ router, rtol=1e-5, atol=1e-6)


# ------------------------------------------------------------------ casts

@pytest.mark.parametrize("cast", [lambda m: m.bfloat16(), lambda m: m.to(torch.bfloat16), lambda m: m.half().bfloat16(),
                                  lambda m: torch.nn.Sequential(m).to("cpu", torch.bfloat16)[0]])
def test_a_cast_module_keeps_its_router_in_fp32(cast):
    layer = moe.MxMoEFFN(256, 512, 4, 2)
    layer.balance += 0.501
    layer.router.grad = torch.randn_like(layer.router)
    router, grad, balance = layer.router.detach().clone(), layer.router.grad.clone(), layer.balance.clone()
    layer = cast(layer)
    assert torch.equal(layer.router.detach(), router) and torch.equal(layer.router.grad, grad)
    assert torch.equal(layer.balance, balance)
    assert layer.w13.dtype == layer.w2.dtype == torch.bfloat16
    x = torch.randn(3, 256).bfloat16()
    assert moe._RouterLogits.apply(x.float(), layer.router).dtype == torch.float32


def test_a_module_still_moves():
    layer = moe.MxMoEFFN(256, 512, 4, 2).to("meta", torch.bfloat16)
    assert layer.router.is_meta and layer.balance.is_meta and layer.w2.is_meta
    assert layer.router.dtype == torch.float32 and isinstance(layer.router, torch.nn.Parameter)
