"""The operators that answer a few tokens with weights held in MX codes, as work to be measured.

    linear  y = x W^T for 1 to 32 tokens, W in 4 or 8 bits
    layer   a whole mixture-of-experts layer for 1 to 32 tokens: router, choice, gated experts, weighted sum
    weights bf16 weights brought to 4-bit codes, and those widened to the 8-bit codes that a prompt's products read

MX: blocks of 32 along the contraction share 2^E; elements are e2m1 (4 bits, two to a byte, the lower nibble first) or
e4m3 (8 bits).  2^E is the smallest power of two with 6 * 2^E (448 * 2^E) >= the block's largest magnitude, E >= -127.
Activations stay as they are: sums run in 32 bits and the result is rounded once.

``run`` computes the plain form (32-bit torch operations) unless ``own`` is set; then it calls the framework.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
MOST_WEIGHTS = 8 * 3 * 5120 * 4096  # of a layer: the largest listed one's


# ------------------------------------------------------------------ cases

def _linear(name, tokens, outs, ins, bits):
    return {"name": name, "op": "linear", "tokens": tokens, "outs": outs, "ins": ins, "bits": bits}


def _layer(name, tokens, experts, top_k, dim, hidden, bits, score="softmax", bias=False, groups=1, groups_kept=1,
           group_top=1, renormalize=True, scale=1.0, off=0.0):
    return {"name": name, "op": "layer", "tokens": tokens, "experts": experts, "top_k": top_k, "dim": dim, "hidden": hidden,
            "bits": bits, "score": score, "bias": bias, "groups": groups, "groups_kept": groups_kept,
            "group_top": group_top, "renormalize": renormalize, "scale": scale, "off": off}


def _weights(name, matrices, outs, ins):
    return {"name": name, "op": "weights", "matrices": matrices, "outs": outs, "ins": ins}


def listed():
    return [
        # one token through a small projection: latency is all there is
        _linear("linear one token, small", 1, 2048, 2048, 4),
        # one token through the large projection
        _linear("linear one token", 1, 8192, 5120, 4),
        # a few drafted or batched tokens, sizes that fill no whole tile
        _linear("linear odd", 5, 6001, 7136, 4),
        # the largest decode batch
        _linear("linear batch", 32, 8192, 5120, 4),
        # weights kept in the 8-bit codes that prompts use
        _linear("linear eight bits", 8, 8192, 5120, 8),
        # one token through many small experts
        _layer("layer one token, many experts", 1, 64, 4, 2048, 1024, 8),
        # one token through few large experts
        _layer("layer one token", 1, 8, 2, 5120, 4096, 4),
        # a decode batch over many experts with sigmoid scores, a balance bias and group-limited choice, some experts off
        _layer("layer batch, many experts", 17, 64, 4, 2048, 1024, 4, score="sigmoid", bias=True, groups=8, groups_kept=4,
               group_top=2, scale=2.5, off=0.05),
        # the largest decode batch over few large experts: every weight is read
        _layer("layer batch", 32, 8, 2, 5120, 4096, 8),
        # one small matrix, a width that fills no whole tile
        _weights("weights small", 1, 288, 2080),
        # the large projection
        _weights("weights projection", 1, 8192, 5120),
        # the first products of all experts
        _weights("weights experts", 8, 8192, 5120),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("linear", "layer", "layer", "weights"))
    if op == "linear":
        ins = 32 * _spread(rng, 2, 512)
        outs = _spread(rng, 16, min(16384, 2 * 8192 * 5120 // ins))
        case = _linear("", _spread(rng, 1, 32), outs, ins, rng.choice((4, 4, 8)))
    elif op == "weights":
        ins = 32 * _spread(rng, 1, 512)
        outs = _spread(rng, 1, 8 * 8192 * 5120 // ins // 4)
        case = _weights("", rng.choice((1, 1, 2, 4)), min(outs, 65536), ins)
    else:
        score = rng.choice(("softmax", "sigmoid"))
        groups = rng.choice((1, 1, 2, 4))
        size = _spread(rng, 2, 128 // groups)
        kept = rng.randint(1, groups)
        experts = groups * size
        dim, hidden = 32 * _spread(rng, 8, 224), 32 * _spread(rng, 4, 160)
        while experts * 3 * dim * hidden > MOST_WEIGHTS:
            dim, hidden = dim // 64 * 32, hidden // 64 * 32
        case = _layer("", _spread(rng, 1, 32), experts, rng.randint(1, min(8, kept * size)), max(dim, 64), max(hidden, 64),
                      rng.choice((4, 8)), score=score, bias=rng.random() < 0.5, groups=groups, groups_kept=kept,
                      group_top=rng.choice((1, 2)), renormalize=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)),
                      off=rng.choice((0.0, 0.1)))
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def _generator(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1013 + sum(ord(c) for c in case["op"]))
    return g


def _normal(g, shape, std=1.0, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _tokens(g, M, C):
    """Activations: a few features are much larger than the others, as in trained models."""
    x = _normal(g, (M, C))
    return (x * torch.where(torch.rand(C, generator=g, device="cuda") < 0.01, 8.0, 1.0)).to(torch.bfloat16)


def _codes(g, shape, bits):
    """MX codes [..., K] (two to a byte for 4 bits) and scales [..., K / 32] of normal weights, a matrix at a time."""
    parts = [_mx(_normal(g, shape[1:], 0.02, torch.bfloat16), bits) for _ in range(shape[0])]
    return torch.stack([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def prepare(case, seed):
    g = _generator(case, seed)
    state = {"case": case}
    if case["op"] == "weights":
        shape = (case["matrices"], case["outs"], case["ins"])
        state["w"] = _normal(g, shape, 0.02, torch.bfloat16)
    elif case["op"] == "linear":
        state["x"] = _tokens(g, case["tokens"], case["ins"])
        q, e8 = _codes(g, (1, case["outs"], case["ins"]), case["bits"])
        state["w"] = (q[0], e8)
    else:
        E, C, F = case["experts"], case["dim"], case["hidden"]
        state["x"] = _tokens(g, case["tokens"], C)
        state["router"] = _normal(g, (E, C), 1.5 / math.sqrt(C))
        bias = torch.round(_normal(g, (E,), 20.0)) * 1e-3  # a balance bias moves by a fixed small step
        bias = torch.where(torch.rand(E, generator=g, device="cuda") < case["off"], float("-inf"), bias if case["bias"] else 0.0)
        state["bias"] = bias if case["bias"] or case["off"] else None
        state["w13"] = _codes(g, (E, 2 * F, C), case["bits"])
        state["w2"] = _codes(g, (E, C, F), case["bits"])
    return state


# ------------------------------------------------------------------ plain forms

def _mx(w, bits):
    """MX codes of w in blocks of 32 along its last dimension, and the bytes of their scales."""
    blocks = w.float().view(*w.shape[:-1], -1, 32)
    top = blocks.abs().amax(dim=-1).view(torch.int32)
    if bits == 8:  # one more where the mantissa is over 1.75 = 448 / 256
        t = (((top + 0x1FFFFF) >> 23) - 8).clamp(min=0)
    else:          # over 1.5 = 6 / 4
        t = (((top + 0x3FFFFF) >> 23) - 2).clamp(min=0)
    v = blocks * ((254 - t) << 23).view(torch.float32)[..., None]
    e8 = t.to(torch.uint8).view(-1, w.shape[-1] // 32)
    if bits == 8:
        return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(w.shape), e8
    v = v.view(w.shape)
    size = v.abs().clamp(max=6.0)
    step = torch.where(size < 2, 0.5, torch.where(size < 4, 1.0, 2.0))
    size = torch.round(size / step) * step  # ties to even; 0 .5 1 1.5 2 3 4 6 are codes 0 to 7
    code = torch.where(size < 2, size * 2, torch.where(size < 4, size + 2, size / 2 + 4)).to(torch.uint8)
    code = code | (torch.signbit(v).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4), e8


def _values(q, e8, bits, dtype=torch.float32):
    """The weights that codes and scales stand for."""
    if bits == 8:
        v = q.view(torch.float8_e4m3fn).to(dtype)
    else:
        pair = torch.tensor([[E2M1[b & 15], E2M1[b >> 4]] for b in range(256)], dtype=dtype, device=q.device)
        v = pair[q.int()].view(*q.shape[:-1], -1)
    scale = e8.view(torch.float8_e8m0fnu).to(dtype).view(*v.shape[:-1], -1)
    return (v.view(*scale.shape, 32) * scale[..., None]).view(v.shape)


def _choice(x, router, bias, case):
    """Experts (-1: none) and weights of each token.  Scores next to a border need 64 bits."""
    M, n = x.shape[0], case["groups"]
    logits = x.double() @ router.double().t()
    s = 1 / (1 + torch.exp(-logits)) if case["score"] == "sigmoid" else torch.exp(logits - logits.amax(dim=1, keepdim=True))
    if case["score"] != "sigmoid":
        s = s / s.sum(dim=1, keepdim=True)
    key = s if bias is None else s + bias
    if n > 1:
        parts = key.view(M, n, -1)
        best = torch.sort(parts, dim=2, descending=True, stable=True).values[:, :, :case["group_top"]]
        total = torch.where(best[:, :, 0] == float("-inf"), float("-inf"), torch.where(best == float("-inf"), 0, best).sum(dim=2))
        first = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :case["groups_kept"]]
        kept = torch.zeros_like(total, dtype=torch.bool).scatter_(1, first, True)
        key = torch.where(kept[:, :, None], parts, float("-inf")).view(M, -1)
    value, index = torch.sort(key, dim=1, descending=True, stable=True)
    value, index = value[:, :case["top_k"]], index[:, :case["top_k"]]
    none = value == float("-inf")
    w = torch.where(none, 0, s.gather(1, index))
    if case["renormalize"]:
        w = w / (w.sum(dim=1, keepdim=True) + 1e-20)
    return torch.where(none, -1, index), w * case["scale"]


def _layer_plain(state):
    case, x = state["case"], state["x"].float()
    M, E, F, k, bits = case["tokens"], case["experts"], case["hidden"], case["top_k"], case["bits"]
    experts, w = _choice(state["x"], state["router"], state["bias"], case)
    w, to = w.float(), experts.clamp(min=0)
    codes = [(q, e8.view(E, -1, e8.shape[1])) for q, e8 in (state["w13"], state["w2"])]
    if M * k < E:  # fewer entries than experts: the chosen ones' weights, entry by entry
        (q13, e13), (q2, e2) = ((q[to.view(-1)], e8[to.view(-1)]) for q, e8 in codes)
        rows = x.repeat_interleave(k, dim=0)[:, :, None]
        w = w.view(-1, 1)
    else:          # every expert on every token, most of them under a weight of 0
        (q13, e13), (q2, e2) = codes
        rows = x.t()[None]
        w = torch.zeros(M, E, device=x.device).scatter_add_(1, to, torch.where(experts < 0, 0, w)).t()
    h = _values(q13, e13, bits) @ rows                      # [entries or experts, 2F, 1 or M]
    gate, up = h[:, :F], h[:, F:]
    y = _values(q2, e2, bits) @ (gate / (1 + torch.exp(-gate)) * up)
    y = y * w[:, None, :]
    y = y.view(M, k, -1).sum(dim=1) if M * k < E else y.sum(dim=0).t()
    return y.to(torch.bfloat16)


def _run_plain(state):
    case = state["case"]
    if case["op"] == "linear":
        return (state["x"].float() @ _values(*state["w"], case["bits"]).t()).to(torch.bfloat16)
    if case["op"] == "layer":
        return _layer_plain(state)
    q, e8 = _mx(state["w"], 4)
    code = torch.stack((q & 15, q >> 4), dim=-1).view(state["w"].shape)
    size = code & 7  # e4m3 of 0 .5 1 1.5 2 3 4 6: 0, and from 1 (0x30) on a step of the last of the three codes' bits
    wide = torch.where(size == 0, 0, torch.where(size == 1, 0x30, 0x30 + size * 4)) | ((code & 8) << 4)
    return {"q": wide.view(torch.float8_e4m3fn), "e8": e8.view(torch.float8_e8m0fnu)}


# ------------------------------------------------------------------ the framework's calls

def _held(w, bits):
    from mxfp8_precision_gemms_fp8bw_gb300 import linear as L

    return L.Mx4Weights(*w) if bits == 4 else L.MxExpertWeights(*w, None, None)


def _run_own(state):
    from mxfp8_precision_gemms_fp8bw_gb300 import linear as L
    from mxfp8_precision_gemms_fp8bw_gb300 import moe

    case = state["case"]
    if case["op"] == "linear":
        return L.mx_linear_few(state["x"], _held(state["w"], case["bits"]))
    if case["op"] == "layer":
        w13, w2 = (_held(state[n], case["bits"]) for n in ("w13", "w2"))
        how = {n: case[n] for n in ("score", "renormalize", "scale", "groups", "groups_kept", "group_top")}
        return moe.ffn_few(state["x"], state["router"], w13, w2, case["top_k"], bias=state["bias"], **how)
    w4 = L.mx4_quantize(state["w"])
    wide = L.mx4_widen(w4)
    return {"q": wide.q_row.view(torch.float8_e4m3fn), "e8": w4.e8.view(torch.float8_e8m0fnu)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    if case["op"] == "weights":
        n = case["matrices"] * case["outs"] * case["ins"]
        return {"bytes": n * (2 + 0.5 + 1 / 32 + 1), "flops": 4 * n}
    held = case["bits"] / 8 + 1 / 32
    if case["op"] == "linear":
        M, N, K = case["tokens"], case["outs"], case["ins"]
        return {"bytes": N * K * held + 2 * M * (N + K), "flops": 2 * M * N * K}
    M, E, k, C, F = (case[n] for n in ("tokens", "experts", "top_k", "dim", "hidden"))
    met = E * (1 - (1 - k / E) ** M)  # experts that some token chose, with even loads
    return {"bytes": met * 3 * C * F * held + 4 * E * C + 4 * M * C, "flops": 6 * M * k * C * F + 2 * M * E * C}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_weight(q, e8, bits):
    if bits == 8:
        v = q.view(torch.float8_e4m3fn).double()
    else:
        code = torch.stack((q % 16, q // 16), dim=-1).flatten(-2).long()
        size = code % 8
        fraction, power = (size % 2).double(), size // 2
        v = torch.where(power == 0, fraction / 2, (1 + fraction / 2) * torch.exp2(power.double() - 1))
        v = torch.where(code >= 8, -v, v)
    return v * torch.exp2(e8.double() - 127).repeat_interleave(32, dim=-1)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "weights":
        q, scales = [], []
        for m in state["w"]:
            blocks = m.double().unflatten(1, (-1, 32))
            top = blocks.abs().amax(dim=2)
            f, ex = torch.frexp(top / 6)  # f 2^ex, 1/2 <= f < 1: a power of two itself has f = 1/2
            E = torch.where(top > 0, ex - (f == 0.5).to(ex.dtype), -127).clamp(min=-127).double()
            v = (blocks / torch.exp2(E)[..., None]).flatten(1)
            code = torch.zeros_like(v)
            for i, border in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):  # on it the even one of codes i and i + 1
                code += v.abs() >= border if i % 2 else v.abs() > border
            size = torch.where(code < 4, code / 2, torch.where(code < 6, code - 2, 2 * code - 8))
            q.append(torch.copysign(size, v))
            scales.append(torch.exp2(E))
        return {"q": torch.stack(q), "e8": torch.cat(scales)}
    x = state["x"].double()
    if case["op"] == "linear":
        return x @ _exact_weight(*state["w"], case["bits"]).t()
    E, F, k, n = case["experts"], case["hidden"], case["top_k"], case["groups"]
    logits = x @ state["router"].double().t()
    s = torch.sigmoid(logits) if case["score"] == "sigmoid" else torch.softmax(logits, dim=1)
    key = s if state["bias"] is None else s + state["bias"].double()
    if n > 1:
        parts = key.unflatten(1, (n, -1))
        best = parts.topk(case["group_top"], dim=2).values
        total = best[..., 0]
        if case["group_top"] == 2:
            total = total + torch.where(best[..., 1] == float("-inf"), 0.0, best[..., 1])
        place = total.argsort(dim=1, descending=True, stable=True).argsort(dim=1)
        key = torch.where(place[:, :, None] < case["groups_kept"], parts, float("-inf")).flatten(1)
    value, index = key.sort(dim=1, descending=True, stable=True)
    value, index = value[:, :k], index[:, :k]
    w = s.gather(1, index) * (value > float("-inf"))
    if case["renormalize"]:
        w = w / (w.sum(dim=1, keepdim=True) + 1e-20)
    w = w * case["scale"]
    y = torch.zeros_like(x)
    scales13, scales2 = state["w13"][1].view(E, 2 * F, -1), state["w2"][1].view(E, case["dim"], -1)
    for e in range(E):
        token, choice = torch.nonzero((index == e) & (value > float("-inf")), as_tuple=True)
        if token.numel() == 0:
            continue
        h = x[token] @ _exact_weight(state["w13"][0][e], scales13[e], case["bits"]).t()
        a = h[:, :F] * torch.sigmoid(h[:, :F]) * h[:, F:]
        y.index_add_(0, token, (a @ _exact_weight(state["w2"][0][e], scales2[e], case["bits"]).t()) * w[token, choice][:, None])
    return y
