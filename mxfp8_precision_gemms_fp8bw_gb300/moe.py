"""A mixture-of-experts layer in MXFP8: the operators around the experts' products and the layer they make.

Each function allocates its outputs, runs on the current stream and returns
without waiting; a batch may have no tokens.  The work is in libfp8bw's
kernels (``include/fp8bw_moe.h`` has the formulas).  For ``linear``'s grouped GEMMs, ``Plan.group_end`` is the group
table and ``MxRows`` holds their operands.

    experts, weights = route(logits, top_k)          x -> experts of each token
    p = plan(experts, num_experts)                   rows of the experts
    rows = dispatch(x, p)                            MX codes of the gathered tokens
    a, kept = swiglu(h)                              h = [gate | up] of the first product
    out = combine(y, weights, p)                     y the second product

and each has its ``..._backward``.  ``MxMoEFFN`` is the layer.
"""
from __future__ import annotations

import functools
from dataclasses import dataclass

import torch

from . import binding as B
from . import linear as L
from . import moe_binding as MB

_U8, _F32, _I32, _BF16 = torch.uint8, torch.float32, torch.int32, torch.bfloat16
_SCORES = {"softmax": MB.SCORE_SOFTMAX, "sigmoid": MB.SCORE_SIGMOID}


def _score(name: str) -> int:
    if name not in _SCORES:
        raise ValueError(f"score: expected one of {sorted(_SCORES)}, got {name!r}")
    return _SCORES[name]


# ------------------------------------------------------------------ routing

def route(logits: torch.Tensor, top_k: int, *, bias: torch.Tensor | None = None, score: str = "softmax",
          renormalize: bool = True, scale: float = 1.0, groups: int = 1, groups_kept: int = 1, group_top: int = 1):
    """The ``top_k`` experts of each token (int32 [M, top_k], best first) and
    their fp32 weights, from router logits [M, E] in fp32 or bf16.  ``bias``
    (fp32 [E]) shifts the choice and not the weights; -inf logits or biases
    mask experts, and a token left with fewer than ``top_k`` gets expert -1
    with weight 0 in the rest."""
    M = logits.shape[0]
    experts = torch.empty((M, top_k), dtype=_I32, device=logits.device)
    weights = torch.empty((M, top_k), dtype=_F32, device=logits.device)
    if M == 0:
        return experts, weights
    MB.fp8bw_moe_route(logits, bias, top_k, experts, weights, groups, groups_kept, group_top, _score(score),
                       renormalize, scale)
    return experts, weights


def route_backward(dweights: torch.Tensor, logits: torch.Tensor, experts: torch.Tensor, *, score: str = "softmax",
                   renormalize: bool = True, scale: float = 1.0) -> torch.Tensor:
    """Gradient of the logits (their dtype) from that of ``route``'s weights."""
    dlogits = torch.empty_like(logits, memory_format=torch.contiguous_format)
    if logits.shape[0] == 0:
        return dlogits
    MB.fp8bw_moe_route_bwd(dweights, logits, experts, dlogits, _score(score), renormalize, scale)
    return dlogits


# ------------------------------------------------------------------ rows of the experts

@dataclass
class Plan:
    """Where the entries (token, choice) of a batch go among the experts' rows."""
    group_end: torch.Tensor   # int32 [E]: end of each expert's rows, multiples of 32; the last is the row count P
    counts: torch.Tensor      # int32 [E]: entries of each expert
    row_of: torch.Tensor      # int32 [M, top_k]: an entry's row, -1 without one
    src_of: torch.Tensor      # int32 [P]: a row's entry (token * top_k + choice), -1 for an empty row

    @property
    def rows(self) -> int:
        return self.src_of.shape[0]


@dataclass
class MxRows:
    """MX codes of a matrix [R, C] in the layouts the grouped GEMMs read."""
    q: torch.Tensor                     # e4m3 [R, C]
    e8: torch.Tensor                    # E8M0 [R, C/32]
    qT: torch.Tensor | None = None      # e4m3 [C, R]
    e8T: torch.Tensor | None = None     # E8M0 [C, R/32]


def _mx_rows(R: int, C: int, device, colwise: bool = True) -> MxRows:
    e = lambda *shape: torch.empty(shape, dtype=_U8, device=device)  # noqa: E731
    return MxRows(e(R, C), e(R, C // 32), *((e(C, R), e(C, R // 32)) if colwise else ()))


def plan(experts: torch.Tensor, num_experts: int) -> Plan:
    """Sorts the entries of ``experts`` (int32 [M, top_k]; -1: no expert) into
    groups of whole 32-row blocks, without the host learning the counts."""
    M, top_k = experts.shape
    dev = experts.device
    P, ws_bytes = _plan_sizes(max(M, 1), num_experts, top_k)
    e = lambda *shape: torch.empty(shape, dtype=_I32, device=dev)  # noqa: E731
    if M == 0:  # no entries: every row is empty
        p = Plan(e(num_experts).zero_(), e(num_experts).zero_(), e(0, top_k), e(P).fill_(-1))
        p.group_end[-1:] = P
        return p
    p = Plan(e(num_experts), e(num_experts), e(M, top_k), e(P))
    ws = torch.empty(ws_bytes, dtype=_U8, device=dev) if ws_bytes else None
    MB.fp8bw_moe_plan(experts, num_experts, p.group_end, p.counts, p.row_of, p.src_of, ws)
    return p


@functools.lru_cache(maxsize=256)
def _plan_sizes(M: int, num_experts: int, top_k: int) -> tuple[int, int]:
    """Rows and workspace bytes of a plan: functions of the dims alone."""
    P = MB.fp8bw_moe_plan_rows(M, num_experts, top_k)
    if P == 0:
        raise B.Fp8bwError(B.ERR_SHAPE, f"invalid plan dims: {M} tokens, {num_experts} experts, top_k {top_k}")
    return P, MB.fp8bw_moe_plan_workspace_bytes(M, num_experts, top_k)


def _tokens(t: torch.Tensor, p: Plan, name: str) -> None:
    if t.shape[0] != p.row_of.shape[0]:
        raise ValueError(f"{name}: the plan has {p.row_of.shape[0]} tokens, got {t.shape[0]}")


def _gathered(x: torch.Tensor, weights: torch.Tensor | None, p: Plan, colwise: bool, mode: int) -> MxRows:
    _tokens(x, p, "x" if weights is None else "dout")
    out = _mx_rows(p.rows, x.shape[1], x.device, colwise)
    if x.shape[0] == 0:  # rows of zeros are codes and scales of 0
        for t in (out.q, out.e8, *((out.qT, out.e8T) if colwise else ())):
            t.zero_()
        return out
    MB.mxfp8_moe_gather_quant(x, weights, p.src_of, p.row_of.shape[1], out.q, out.e8, out.qT, out.e8T, mode)
    return out


def dispatch(x: torch.Tensor, p: Plan, colwise: bool = True, mode: int = B.MX_RCEIL) -> MxRows:
    """MX codes of the experts' rows of x (bf16 [M, C]); ``colwise`` adds the
    layout the weight gradient reads."""
    return _gathered(x, None, p, colwise, mode)


def dispatch_backward(drows: torch.Tensor, p: Plan) -> torch.Tensor:
    """Gradient of ``dispatch``'s x from that of its rows (bf16 [P, C])."""
    return combine(drows, None, p)


def combine(y: torch.Tensor, weights: torch.Tensor | None, p: Plan, base: torch.Tensor | None = None) -> torch.Tensor:
    """out[t] = base[t] + the sum of token t's rows of y (bf16 [P, C]) times
    their weights (fp32 [M, top_k]; None: one each)."""
    out = torch.empty((p.row_of.shape[0], y.shape[1]), dtype=_BF16, device=y.device)
    if out.shape[0] == 0:
        return out
    MB.fp8bw_moe_combine(y, weights, p.row_of, base, out)
    return out


def combine_backward(dout: torch.Tensor, y: torch.Tensor, weights: torch.Tensor, p: Plan, mode: int = B.MX_RCEIL):
    """Gradients of ``combine``: that of y as MX codes in both layouts, and
    that of the weights."""
    _tokens(weights, p, "weights")
    return _gathered(dout, weights, p, True, mode), _dweights(dout, y, p)


def _dweights(dout: torch.Tensor, y: torch.Tensor, p: Plan) -> torch.Tensor:
    dweights = torch.empty(p.row_of.shape, dtype=_F32, device=dout.device)
    if dout.shape[0] > 0:
        MB.fp8bw_moe_combine_dweights(dout, y, p.row_of, dweights)
    return dweights


# ------------------------------------------------------------------ gated activation

def swiglu(h: torch.Tensor, keep: bool = True, colwise: bool = True, mode: int = B.MX_RCEIL):
    """a = silu(gate) * up of h = [gate | up] (bf16 [R, 2F]) as MX codes, and,
    with ``keep``, h's own rowwise codes: the 8-bit activation checkpoint that
    ``swiglu_backward`` works from (None without)."""
    R, F = h.shape[0], h.shape[1] // 2
    a = _mx_rows(R, F, h.device, colwise)
    kept = _mx_rows(R, 2 * F, h.device, colwise=False) if keep else None
    MB.mxfp8_swiglu(h, a.q, a.e8, a.qT, a.e8T, *((kept.q, kept.e8) if keep else (None, None)), mode=mode)
    return a, kept


def swiglu_backward(da: torch.Tensor, kept: MxRows, mode: int = B.MX_RCEIL) -> MxRows:
    """Gradient of ``swiglu``'s h as MX codes in both layouts, from da
    (bf16 [R, F]) and the kept codes."""
    R, F = da.shape
    dh = _mx_rows(R, 2 * F, da.device)
    MB.mxfp8_swiglu_bwd(da, kept.q, kept.e8, dh.q, dh.e8, dh.qT, dh.e8T, mode)
    return dh


# ------------------------------------------------------------------ the layer

def _grouped(kind: int, a, a_e8, b, b_e8, p: Plan, N: int, K: int, out: torch.Tensor) -> torch.Tensor:
    G, P = p.group_end.shape[0], p.rows
    ws = B.alloc_grouped_workspace(kind, G, P, N, K, out.device)
    B.mxfp8_grouped_gemm(kind, a, a_e8, b, b_e8, p.group_end, G, P, N, K, out, ws)
    return out


def _differentiable_once(backward):
    """For a backward made of kernel calls, whose results have no graph: a second derivative would leave out their part and
    say nothing, so ``create_graph`` is refused.  (torch's ``once_differentiable`` marks what depends on the incoming
    gradient; these results depend on the forward's inputs too.)"""
    @functools.wraps(backward)
    def wrapper(ctx, *douts):
        if torch.is_grad_enabled():  # in a backward: create_graph
            raise RuntimeError("the mixture-of-experts operators have no second derivative (create_graph=True)")
        return backward(ctx, *douts)
    return wrapper


def _without_autocast(product, a: torch.Tensor, b: torch.Tensor) -> torch.Tensor:
    if not torch.is_autocast_enabled(a.device.type):
        return product(a, b)
    with torch.autocast(a.device.type, enabled=False):
        return product(a, b)


class _RouterLogits(torch.autograd.Function):
    """x router^T of fp32 x, in fp32 whatever autocast says, forward and backward: logits rounded to bf16 choose other
    experts."""

    @staticmethod
    def forward(ctx, x, router):
        need_dx, need_drouter = ctx.needs_input_grad
        ctx.save_for_backward(x if need_drouter else None, router if need_dx else None)
        return _without_autocast(torch.nn.functional.linear, x, router)

    @staticmethod
    @_differentiable_once
    def backward(ctx, dlogits):
        x, router = ctx.saved_tensors
        return (None if router is None else _without_autocast(torch.matmul, dlogits, router),
                None if x is None else _without_autocast(torch.matmul, dlogits.t(), x))


def _check_codes(codes: L.MxExpertWeights, w: torch.Tensor, colwise: bool) -> None:
    """The grouped GEMMs take sizes from the layer and read the codes by address; a gradient reads the colwise ones."""
    E, N, K = w.shape
    for name, shape in (("q_row", (E, N, K)), ("e8_row", (E * N, K // 32)), ("qT_col", (E, K, N)),
                        ("e8_col", (E, K, N // 32))):
        t = getattr(codes, name)
        if t is None and name.endswith("col"):
            if colwise:
                raise ValueError(f"codes: gradients read {name}, which weight_codes(colwise=False) leaves out")
        elif tuple(t.shape) != shape:
            raise ValueError(f"codes: {name} of weights {tuple(w.shape)} is {shape}, got {tuple(t.shape)}")


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, bias, top_k, score, renormalize, scale, groups, groups_kept, group_top):
        experts, weights = route(logits, top_k, bias=bias, score=score, renormalize=renormalize, scale=scale,
                                 groups=groups, groups_kept=groups_kept, group_top=group_top)
        ctx.how = dict(score=score, renormalize=renormalize, scale=scale)
        ctx.save_for_backward(logits, experts)
        ctx.mark_non_differentiable(experts)
        return experts, weights

    @staticmethod
    @_differentiable_once
    def backward(ctx, _, dweights):
        logits, experts = ctx.saved_tensors
        return (route_backward(dweights.contiguous(), logits, experts, **ctx.how),) + (None,) * 8


class _Experts(torch.autograd.Function):
    """sum over a token's experts of weight * W2 (silu(Wg x) * Wu x), with [Wg; Wu] = w13.

    Kept for backward, each only where a gradient that is asked for reads it:
    the colwise MX codes of the gathered tokens (dw13) and of the activation
    (dw2), h as rowwise codes and the weights' column codes (what goes on to
    dw13 and dx), and y, the only bf16 one (the gradient of the choices'
    weights)."""

    @staticmethod
    def forward(ctx, x, weights, experts, w13, w2, codes, mode, train, counts):
        E, F2, C = w13.shape
        F = F2 // 2
        need_x, need_weights, _, need_13, need_2 = (train and n for n in ctx.needs_input_grad[:5])
        through = need_x or need_13  # the gradient goes on through the activation
        p = plan(experts, E)
        counts.append(p.counts)
        rows = dispatch(x, p, colwise=need_13, mode=mode)
        q13, q2 = codes
        bf = lambda *shape: torch.empty(shape, dtype=_BF16, device=x.device)  # noqa: E731
        h = _grouped(B.GROUPED_FWD, rows.q, rows.e8, q13.q_row, q13.e8_row, p, F2, C, bf(p.rows, F2))
        a, kept = swiglu(h, keep=through, colwise=need_2, mode=mode)
        y = _grouped(B.GROUPED_FWD, a.q, a.e8, q2.q_row, q2.e8_row, p, C, F, bf(p.rows, C))
        if train:
            ctx.mode, ctx.dims, ctx.need = mode, (E, C, F), (need_x, need_weights, need_13, need_2)
            kept = kept or MxRows(None, None)
            ctx.save_for_backward(weights if through or need_2 else None, y if need_weights else None, kept.q, kept.e8,
                                  *((q2.qT_col, q2.e8_col) if through else (None, None)),
                                  *((q13.qT_col, q13.e8_col) if need_x else (None, None)),
                                  rows.qT, rows.e8T, a.qT, a.e8T, p.group_end, p.counts, p.row_of, p.src_of)
        return combine(y, weights, p)

    @staticmethod
    @_differentiable_once
    def backward(ctx, dout):
        weights, y, hq, he, w2T, w2e, w13T, w13e, xT, xeT, aT, aeT, *tables = ctx.saved_tensors
        p, mode, (E, C, F) = Plan(*tables), ctx.mode, ctx.dims
        need_x, need_weights, need_13, need_2 = ctx.need
        dout = dout.contiguous()
        bf = lambda *shape: torch.empty(shape, dtype=_BF16, device=dout.device)  # noqa: E731
        dx = dweights = dw13 = dw2 = None
        if need_weights:
            dweights = _dweights(dout, y, p)
        if need_x or need_13 or need_2:
            dy = _gathered(dout, weights, p, need_2, mode)
        if need_2:
            dw2 = _grouped(B.GROUPED_WGRAD, dy.qT, dy.e8T, aT, aeT, p, C, F, bf(E, C, F))
        if need_x or need_13:
            da = _grouped(B.GROUPED_DGRAD, dy.q, dy.e8, w2T, w2e, p, C, F, bf(p.rows, F))
            dh = swiglu_backward(da, MxRows(hq, he), mode=mode)
        if need_x:
            dx = dispatch_backward(_grouped(B.GROUPED_DGRAD, dh.q, dh.e8, w13T, w13e, p, 2 * F, C, bf(p.rows, C)), p)
        if need_13:
            dw13 = _grouped(B.GROUPED_WGRAD, dh.qT, dh.e8T, xT, xeT, p, 2 * F, C, bf(E, 2 * F, C))
        return dx, dweights, None, dw13, dw2, None, None, None, None


class MxMoEFFN(torch.nn.Module):
    """Mixture of gated feed-forward experts whose products run in MXFP8.

    Inputs are 2D bf16 CUDA tensors [tokens, dim]; dim and hidden must be
    multiples of 256, the token count is free.  The router's logits are a
    plain fp32 product, under autocast too (and in TF32 only where the program
    has turned that on for fp32 products); its gradient keeps x in fp32.
    ``balance`` (a buffer, not a parameter) is the bias that shifts the choice
    of experts; ``update_balance`` moves it against ``counts``, the loads of
    the last forward in training mode.  ``route``'s keyword arguments are taken
    too.
    Casting the module (``bfloat16()``, ``to(dtype)``) leaves the router and
    ``balance`` in fp32: a bias in bf16 would lose its steps.
    """

    def __init__(self, dim: int, hidden: int, num_experts: int, top_k: int, *, score: str = "softmax",
                 renormalize: bool = True, scale: float = 1.0, groups: int = 1, groups_kept: int = 1,
                 group_top: int = 1, mode: int = B.MX_RCEIL, device=None):
        super().__init__()
        new = lambda *shape, dtype=_BF16: torch.nn.Parameter(  # noqa: E731
            torch.nn.init.normal_(torch.empty(shape, dtype=dtype, device=device), std=0.02))
        self.router = new(num_experts, dim, dtype=_F32)
        self.w13 = new(num_experts, 2 * hidden, dim)
        self.w2 = new(num_experts, dim, hidden)
        self.register_buffer("balance", torch.zeros(num_experts, dtype=_F32, device=device))
        self.how = (top_k, score, renormalize, scale, groups, groups_kept, group_top)
        self.mode = mode
        self.counts = None

    def _apply(self, fn, recurse=True):
        fp32 = [t for t in (self.router, self.router.grad, self.balance) if t is not None]

        def but_keep_fp32(t):
            new = fn(t)
            return t.to(new.device) if new.dtype != t.dtype and any(t is k for k in fp32) else new

        return super()._apply(but_keep_fp32, recurse)

    def weight_codes(self, colwise: bool = True) -> tuple[L.MxExpertWeights, L.MxExpertWeights]:
        """MX codes of w13 and w2 as they are now, for calls between two changes of the weights.  Without ``colwise`` those
        that a forward pass reads, half of the bytes: for calls without gradients."""
        return tuple(L.mx_quantize_experts(w.detach(), self.mode, colwise=colwise) for w in (self.w13, self.w2))

    def forward(self, x: torch.Tensor, codes: tuple[L.MxExpertWeights, L.MxExpertWeights] | None = None) -> torch.Tensor:
        """``codes``: ``weight_codes()`` kept by the caller (a decoder, or the micro-batches of a step); by default
        the weights are quantized in every call."""
        # needs_input_grad does not know of no_grad, where the layouts and codes for backward would be for nothing
        grad = torch.is_grad_enabled()
        train = grad and any(t.requires_grad for t in (x, self.router, self.w13, self.w2))
        need_x = grad and x.requires_grad
        weights13, weights2 = (self.w13, need_x), (self.w2, need_x or grad and self.w13.requires_grad)
        if codes is None:
            codes = tuple(L.mx_quantize_experts(w.detach(), self.mode, colwise=c) for w, c in (weights13, weights2))
        else:
            for got, (w, colwise) in zip(codes, (weights13, weights2)):
                _check_codes(got, w, colwise)
        if train:
            logits = _RouterLogits.apply(x.float(), self.router)
        else:
            logits = _without_autocast(torch.nn.functional.linear, x.float(), self.router)
        experts, weights = _Route.apply(logits, self.balance, *self.how)
        counts = []
        out = _Experts.apply(x, weights, experts, self.w13, self.w2, codes, self.mode, train, counts)
        if self.training:
            self.counts = counts[0]
        return out

    @torch.no_grad()
    def update_balance(self, rate: float = 1e-3) -> None:
        """Moves each expert's bias one step up where its last load was below the mean, down where above."""
        if self.counts is None:
            raise RuntimeError("update_balance needs a forward pass in training mode first")
        load = self.counts.float()
        self.balance += rate * torch.sign(load.mean() - load)
