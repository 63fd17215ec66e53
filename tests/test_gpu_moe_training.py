"""The mixture-of-experts layer in a training program: what it refuses, what it keeps and what it computes for partly frozen
or cast modules."""
import pytest
import torch

from gpu_util import lib
from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import linear as L
from mxfp8_precision_gemms_fp8bw_gb300 import moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib()


def layer_and_tokens(tokens=70, dim=256, hidden=512, experts=4, top_k=2, **how):
    torch.manual_seed(5)
    layer = moe.MxMoEFFN(dim, hidden, experts, top_k, device="cuda", **how)
    return layer, torch.randn(tokens, dim, device="cuda").bfloat16().requires_grad_(True)


@pytest.mark.parametrize("linear", [True, False])
def test_a_second_derivative_is_an_error(linear):
    layer, x = layer_and_tokens()
    out = layer(x)
    loss = out.float().sum() if linear else out.float().square().sum()
    with pytest.raises(RuntimeError, match="no second derivative"):
        dx, dw = torch.autograd.grad(loss, (x, layer.w13), create_graph=True)
        torch.autograd.grad(dx.float().square().sum() + dw.float().square().sum(), layer.router)
    loss.backward()
    assert x.grad is not None and layer.router.grad is not None


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_autocast_changes_nothing(dtype, score):
    """Neither in the forward pass nor in a backward pass under it."""
    layer, x = layer_and_tokens(tokens=300, experts=8, score=score)
    made = []
    for on in (False, True):
        layer.zero_grad()
        x.grad = None
        with torch.autocast("cuda", dtype=dtype, enabled=on):
            out = layer(x)
            out.backward(torch.ones_like(out))
            with torch.no_grad():
                again = layer(x)
        made.append((layer.counts, out, x.grad, layer.router.grad, layer.w13.grad, layer.w2.grad, again))
    B.fp8bw_sync_status()
    assert all(torch.equal(a, b) for a, b in zip(*made))


def test_what_is_kept_for_backward():
    """Beside codes and tables: the tokens in fp32 for the router, and in bf16 the experts' output alone."""
    layer, x = layer_and_tokens(tokens=96)
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: (kept.append(t), t)[1], lambda t: t):
        layer(x)
    big = sorted((str(t.dtype), tuple(t.shape)) for t in kept
                 if t.dtype in (torch.float32, torch.bfloat16) and t.numel() >= x.numel())
    rows = moe.MB.fp8bw_moe_plan_rows(96, 4, 2)
    assert big == [("torch.bfloat16", (rows, 256)), ("torch.float32", (96, 256))]


def test_the_tokens_may_change_in_place_before_the_backward_pass():
    layer, x = layer_and_tokens()
    layer(x).backward(torch.ones_like(x))
    want = layer.router.grad.clone(), layer.w13.grad.clone(), x.grad.clone()
    layer.zero_grad()
    y = x.detach().clone().requires_grad_(True)
    out = layer(y)
    with torch.no_grad():
        y.zero_()
    out.backward(torch.ones_like(out))
    assert all(torch.equal(a, b) for a, b in zip((layer.router.grad, layer.w13.grad, y.grad), want))


def test_a_layer_cast_to_bf16_runs_as_before():
    layer, x = layer_and_tokens(score="sigmoid")
    layer.balance.copy_(torch.randn(4, device="cuda") * 1e-2)
    want = layer(x)
    got = layer.bfloat16()(x)
    assert torch.equal(got, want)
    got.backward(torch.ones_like(got))
    layer.update_balance()
    B.fp8bw_sync_status()
    assert layer.router.grad.dtype == layer.balance.dtype == torch.float32


@pytest.mark.parametrize("how", ["no_grad", "frozen"])
def test_without_gradients_no_column_codes_of_the_weights(how, monkeypatch):
    layer, x = layer_and_tokens()
    want = layer(x).detach()
    x = x.detach()
    layer.requires_grad_(how != "frozen")
    monkeypatch.setattr(L.B, "alloc_mx_3d_col", lambda w: pytest.fail("column codes of the weights"))
    monkeypatch.setattr(L.B, "mxfp8_quant_1x32_rowcol", lambda *a: pytest.fail("column codes of the weights"))
    with torch.set_grad_enabled(how == "frozen"):
        assert torch.equal(layer(x), want)
        codes = layer.weight_codes(colwise=False)
        assert all(c.qT_col is None and c.e8_col is None for c in codes)
        assert torch.equal(layer(x, codes), want)
    B.fp8bw_sync_status()


@pytest.mark.parametrize("mode", [B.MX_RCEIL, B.MX_FLOOR])
@pytest.mark.parametrize("rows", [65535 * 32, 256, 160])
def test_rowwise_expert_codes_are_those_of_both_layouts(rows, mode, monkeypatch):
    monkeypatch.setattr(L, "MX_ROWS_PER_CALL", rows)
    w = torch.randn(5, 96, 128, device="cuda").bfloat16()
    a, b = L.mx_quantize_experts(w, mode), L.mx_quantize_experts(w, mode, colwise=False)
    B.fp8bw_sync_status()
    assert torch.equal(a.q_row, b.q_row) and torch.equal(a.e8_row, b.e8_row)


def test_more_expert_rows_than_one_call_takes():
    w = torch.randn(66, 32768, 32, device="cuda").bfloat16()
    assert w.shape[0] * w.shape[1] > 65535 * 32
    a, b = L.mx_quantize_experts(w), L.mx_quantize_experts(w, colwise=False)
    B.fp8bw_sync_status()
    assert torch.equal(a.q_row, b.q_row) and torch.equal(a.e8_row, b.e8_row)


NAMES = ("x", "router", "w13", "w2")


@pytest.mark.parametrize("wanted", [[n for i, n in enumerate(NAMES) if bits >> i & 1] for bits in range(1, 16)],
                         ids="+".join)
def test_what_no_gradient_asks_for_is_not_computed(wanted, monkeypatch):
    """Partly frozen layers: the same gradients to the bit, from no more products than they need."""
    layer, x = layer_and_tokens()
    leaves = {"x": x, "router": layer.router, "w13": layer.w13, "w2": layer.w2}
    dout = torch.randn(x.shape, device="cuda").bfloat16()
    layer(x).backward(dout)
    full = {n: t.grad.clone() for n, t in leaves.items()}
    for n, t in leaves.items():
        t.grad = None
        t.requires_grad_(n in wanted)
    kinds, grouped = [], moe._grouped
    monkeypatch.setattr(moe, "_grouped", lambda kind, *a: (kinds.append(kind), grouped(kind, *a))[1])
    layer(x).backward(dout)
    B.fp8bw_sync_status()
    for n, t in leaves.items():
        assert t.grad is None if n not in wanted else torch.equal(t.grad, full[n])
    through = "x" in wanted or "w13" in wanted
    assert kinds.count(B.GROUPED_FWD) == 2
    assert kinds.count(B.GROUPED_DGRAD) == through + ("x" in wanted)
    assert kinds.count(B.GROUPED_WGRAD) == ("w13" in wanted) + ("w2" in wanted)


def test_rowwise_codes_serve_where_only_the_router_or_w2_trains():
    layer, x = layer_and_tokens()
    x = x.detach()
    layer.w13.requires_grad_(False)
    layer(x).backward(torch.ones_like(x))
    want = layer.router.grad.clone(), layer.w2.grad.clone()
    layer.zero_grad()
    layer(x, layer.weight_codes(colwise=False)).backward(torch.ones_like(x))
    assert torch.equal(layer.router.grad, want[0]) and torch.equal(layer.w2.grad, want[1])


def test_an_evaluation_does_not_move_the_balance():
    layer, x = layer_and_tokens(tokens=400, experts=8, score="sigmoid")
    layer.eval()
    with torch.no_grad():
        layer(x)
    with pytest.raises(RuntimeError):
        layer.update_balance()
    layer.train()
    layer(x)
    counts = layer.counts
    layer.eval()
    with torch.no_grad():
        layer(x[:7])
    assert layer.counts is counts and int(counts.sum()) == 800
    layer.update_balance(0.5)
    assert torch.equal(layer.balance, 0.5 * torch.sign(100 - counts.float()))


@pytest.mark.parametrize("reentrant", [False, True])
def test_under_activation_checkpointing(reentrant):
    """The forward pass run again in the backward pass: the same gradients, and no refusal of it as a second derivative."""
    from torch.utils.checkpoint import checkpoint

    layer, x = layer_and_tokens()
    made = []
    for run in (layer, lambda t: checkpoint(layer, t, use_reentrant=reentrant)):
        layer.zero_grad()
        x.grad = None
        out = run(x)
        out.backward(torch.ones_like(out))
        made.append((out, x.grad, layer.router.grad, layer.w13.grad, layer.w2.grad))
    B.fp8bw_sync_status()
    assert all(torch.equal(a, b) for a, b in zip(*made))


def test_kept_tensors_may_wait_on_the_host():
    layer, x = layer_and_tokens()
    layer(x).backward(torch.ones_like(x))
    want = [t.grad.clone() for t in (x, layer.router, layer.w13, layer.w2)]
    layer.zero_grad()
    x.grad = None
    with torch.autograd.graph.save_on_cpu():
        out = layer(x)
    out.backward(torch.ones_like(x))
    B.fp8bw_sync_status()
    assert all(torch.equal(t.grad, w) for t, w in zip((x, layer.router, layer.w13, layer.w2), want))


def test_rowwise_codes_are_refused_by_the_grouped_backward():
    w = torch.randn(2, 256, 256, device="cuda").bfloat16()
    x, dy = (torch.randn(64, 256, device="cuda").bfloat16() for _ in range(2))
    end = torch.tensor([32, 64], dtype=torch.int32, device="cuda")
    with pytest.raises(B.Fp8bwError) as e:
        L.mx_moe_backward(dy, x, L.mx_quantize_experts(w, colwise=False), end)
    assert e.value.code == B.ERR_NULL
    B.fp8bw_sync_status()
