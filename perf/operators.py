"""The operators around the experts' products of a mixture-of-experts layer, as work to be measured.

    route     scores from router logits, a bias for balance, groups, top-k, weights; and its gradient
    dispatch  tokens sorted into expert groups of whole 32-row blocks, gathered and held as MXFP8 codes; and its gradient
    combine   the experts' output rows summed back into their tokens; and its gradient, held as MXFP8 codes
    swiglu    the gated activation held as MXFP8 codes, with its input kept in 8 bits; and its gradient from those 8 bits

MXFP8: blocks of 32 share 2^E, the smallest power of two with 448 * 2^E >= the block's largest magnitude (E >= -127),
and each element is e4m3 of x / 2^E.  Codes come back as the float8 values they are, scales as the powers of two they are.

``run`` computes the plain form (32-bit torch operations) unless ``own`` is set; then it calls the framework.
"""
import math

import torch

own = False

LOWEST = -3.4028234663852886e38


# ------------------------------------------------------------------ cases

def _route(name, tokens, experts, top_k, score="softmax", dtype="bf16", bias=False, groups=1, groups_kept=1, group_top=1,
           renormalize=True, scale=1.0, padding=0.0, train=False):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "top_k": top_k, "score": score,
            "dtype": dtype, "bias": bias, "groups": groups, "groups_kept": groups_kept, "group_top": group_top,
            "renormalize": renormalize, "scale": scale, "padding": padding, "train": train}


def _rows(name, op, tokens, experts, top_k, width, padding=0.0, train=False):
    return {"name": name, "op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "width": width,
            "padding": padding, "train": train}


def _swiglu(name, rows, width, train=False):
    return {"name": name, "op": "swiglu", "rows": rows, "width": width, "train": train}


def listed():
    return [
        # one token being generated: latency is all there is
        _route("route one token", 1, 64, 4),
        # a training step of a layer with few experts, a ragged token count
        _route("route few experts", 4097, 8, 2, train=True),
        # a training step with sigmoid scores, a balance bias and group-limited choice, 32-bit logits
        _route("route groups and bias", 16384, 128, 6, score="sigmoid", dtype="fp32", bias=True, groups=8, groups_kept=3,
               group_top=2, scale=1.5, train=True),
        # the longest batch, an expert count that is no power of two, weights left unnormalised, padding tokens
        _route("route long batch", 127999, 160, 4, dtype="fp32", renormalize=False, padding=0.01, train=True),
        # a decode batch: a handful of tokens over many experts, no backward
        _rows("dispatch decode", "dispatch", 17, 64, 4, 2048),
        # the 16384-row MoE step: 8192 tokens, two experts each, over 8 experts
        _rows("dispatch step", "dispatch", 8192, 8, 2, 5120, train=True),
        # many rows of a narrower layer, many experts, ragged, some padding tokens that no expert gets
        _rows("dispatch long", "dispatch", 15999, 64, 8, 2048, padding=0.02, train=True),
        # the way back of the decode batch
        _rows("combine decode", "combine", 17, 64, 4, 2048),
        # the way back of the MoE step and its backward
        _rows("combine step", "combine", 8192, 8, 2, 5120, train=True),
        # the activation of a few decoded rows: no backward, so nothing is kept; a width that fills no whole 64
        _swiglu("swiglu decode", 96, 2080),
        # the activation of the 16384-row MoE step (8192 = gate and up of 4096 each), forward and backward
        _swiglu("swiglu step", 16640, 4096, train=True),
        # the 128000-token layer with 2048 = gate and up of 1024 each
        _swiglu("swiglu long", 130048, 1024, train=True),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _wide(rng, low, high):
    """A multiple of 32, even over its logarithm; neither it nor its double is 3072."""
    n = 32 * _spread(rng, low // 32, high // 32)
    return n + 32 if n in (1536, 3072) else n


def draw(rng):
    op = rng.choice(("route", "dispatch", "combine", "swiglu"))
    train = rng.random() < 0.6
    if op == "swiglu":
        width = _wide(rng, 256, 8192)
        rows = 32 * _spread(rng, 1, max(1, 130048 * 1024 // (32 * width)))
        case = _swiglu("", rows + 32 if rows == 3072 else rows, width, train)
    elif op == "route":
        score = rng.choice(("softmax", "sigmoid"))
        groups = rng.choice((1, 1, 2, 4, 8))
        size = rng.randint(4, 256 // groups) if groups > 1 else rng.randint(4, 256)
        kept = rng.randint(1, groups)
        tokens = min(_spread(rng, 1, 127999), 127999 * 160 // (groups * size))
        case = _route("", tokens + 1 if tokens == 3072 else tokens, groups * size, rng.randint(1, min(10, kept * size)), score=score, dtype=rng.choice(("bf16", "fp32")),
                      bias=rng.random() < 0.5, groups=groups, groups_kept=kept, group_top=rng.choice((1, 2)),
                      renormalize=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)), padding=rng.choice((0.0, 0.03)), train=train)
    else:
        experts, width = _spread(rng, 2, 128), _wide(rng, 256, 8192)
        top_k = rng.randint(1, min(8, experts))
        most = 250_000_000 // (top_k * width)  # rows * width, padding rows included, stays under the largest listed case's
        tokens = _spread(rng, 1, min(65536, most))
        case = _rows("", op, tokens + 1 if tokens == 3072 else tokens, experts, top_k, width, rng.choice((0.0, 0.05)), train)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def _capacity(tokens, top_k, experts):
    """Rows that hold any choice of experts with every group padded to whole 32-row blocks."""
    n = tokens * top_k
    return max(32, (n + 31 * min(experts, n)) // 32 * 32)


def _generator(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1009 + sum(ord(c) for c in case["op"]))
    return g


def _normal(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda") * std


def _choices(g, case):
    """Experts of each token as a router gives them: unequal loads, distinct per token, -1 for padding tokens."""
    M, E, k = case["tokens"], case["experts"], case["top_k"]
    liked = _normal(g, (E,), 0.7)
    experts = (_normal(g, (M, E)) + liked).argsort(dim=1, descending=True)[:, :k].to(torch.int32)
    if case["padding"]:
        experts[torch.rand(M, generator=g, device="cuda") < case["padding"]] = -1
    return experts.contiguous()


def _gate_weights(g, shape):
    w = torch.rand(shape, generator=g, device="cuda") + 0.1
    return w / w.sum(dim=1, keepdim=True)


def _plan_plain(experts, E):
    """Rows of the grouped products: entry (t, j) of expert e goes behind the earlier entries of e."""
    M, k = experts.shape
    flat = experts.reshape(-1).long()
    mine = flat[:, None] == torch.arange(E, device=flat.device)
    before = torch.cumsum(mine, dim=0, dtype=torch.int32)
    counts = before[-1]
    padded = (counts + 31) // 32 * 32
    end = torch.cumsum(padded, dim=0, dtype=torch.int32)
    start = end - padded
    P = _capacity(M, k, E)
    here = flat >= 0
    to = flat.clamp(min=0)
    rank = before.gather(1, to[:, None])[:, 0] - 1
    row_of = torch.where(here, start[to] + rank, -1)
    src_of = torch.full((P + 1,), -1, dtype=torch.int32, device=flat.device)
    src_of[torch.where(here, row_of, P).long()] = torch.arange(M * k, dtype=torch.int32, device=flat.device)
    group_end = end.clone()
    group_end[-1:] = P
    return {"group_end": group_end, "counts": counts.clone(), "row_of": row_of.to(torch.int32).view(M, k),
            "src_of": src_of[:P]}


def prepare(case, seed):
    g = _generator(case, seed)
    bf = torch.bfloat16
    state = {"case": case}
    if case["op"] == "route":
        M, E = case["tokens"], case["experts"]
        logits = _normal(g, (M, E), 1.5) + _normal(g, (E,), 0.5)
        if case["padding"]:
            logits[torch.rand(M, generator=g, device="cuda") < case["padding"]] = float("-inf")
        state["logits"] = logits.to(bf if case["dtype"] == "bf16" else torch.float32)
        # a balance bias moves by a fixed small step, so it is a multiple of one
        state["bias"] = torch.round(_normal(g, (E,), 20.0)) * 1e-3 if case["bias"] else None
        state["dweights"] = _normal(g, (M, case["top_k"]), 1e-2)
    elif case["op"] == "swiglu":
        R, F = case["rows"], case["width"]
        state["h"] = _normal(g, (R, 2 * F)).to(bf)
        state["da"] = _normal(g, (R, F), 1e-3).to(bf)
    else:
        M, C, k = case["tokens"], case["width"], case["top_k"]
        experts = _choices(g, case)
        P = _capacity(M, k, case["experts"])
        if case["op"] == "dispatch":
            state["experts"] = experts
            state["x"] = _normal(g, (M, C)).to(bf)
            state["drows"] = _normal(g, (P, C), 1e-3).to(bf) if case["train"] else None
        else:
            state["plan"] = _plan_plain(experts, case["experts"])
            state["weights"] = _gate_weights(g, (M, k))
            state["y"] = _normal(g, (P, C)).to(bf)
            state["dout"] = _normal(g, (M, C), 1e-3).to(bf) if case["train"] else None
    return state


# ------------------------------------------------------------------ plain forms

def _halved(x):
    """The row sums by halves: x[i] + x[i + n/2], again until one is left, so that they do not depend on who adds them."""
    n = x.shape[1]
    if n == 1:
        return x
    if n & (n - 1):
        return _halved(torch.nn.functional.pad(x, (0, (1 << n.bit_length()) - n)))
    return _halved(x[:, :n // 2] + x[:, n // 2:])


def _scores(logits, score):
    x = logits.float()
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    top = x.max(dim=1, keepdim=True).values
    empty = top == float("-inf")
    e = torch.exp(x - torch.where(empty, 0, top))
    return torch.where(empty, 0, e / _halved(e))


def _best_first(x):
    """Descending along the last dimension, the lowest index first among equals."""
    return torch.sort(x, dim=-1, descending=True, stable=True)


def _route_plain(logits, bias, case):
    M, E = logits.shape
    k, n = case["top_k"], case["groups"]
    s = _scores(logits, case["score"])
    key = s if bias is None else s + bias
    masked = logits.float() == float("-inf")
    masked = masked if bias is None else masked | (bias == float("-inf"))
    key = torch.where(masked, float("-inf"), key)
    if n > 1:
        best = _best_first(key.view(M, n, E // n)).values[:, :, :case["group_top"]]
        total = torch.where(best == float("-inf"), 0, best).sum(dim=2).clamp(min=LOWEST)
        total = torch.where(best[:, :, 0] == float("-inf"), float("-inf"), total)
        kept = torch.zeros(M, n, dtype=torch.bool, device=key.device)
        kept.scatter_(1, _best_first(total).indices[:, :case["groups_kept"]], True)
        key = torch.where(kept.repeat_interleave(E // n, dim=1), key, float("-inf"))
    value, index = _best_first(key)
    value, index = value[:, :k], index[:, :k]
    none = value == float("-inf")
    chosen = torch.where(none, 0, s.gather(1, index))
    w = chosen / (chosen.sum(dim=1, keepdim=True) + 1e-20) if case["renormalize"] else chosen
    return torch.where(none, -1, index).to(torch.int32), w * case["scale"]


def _route_back_plain(dw, logits, experts, case):
    s = _scores(logits, case["score"])
    to, none = experts.long().clamp(min=0), experts < 0
    chosen = torch.where(none, 0, s.gather(1, to))
    ds = torch.where(none, 0, dw * case["scale"])
    if case["renormalize"]:
        total = chosen.sum(dim=1, keepdim=True) + 1e-20
        ds = torch.where(none, 0, ds - (ds * chosen).sum(dim=1, keepdim=True) / total) / total
    full = torch.zeros_like(s).scatter_add_(1, to, ds)
    if case["score"] == "sigmoid":
        d = full * s * (1 - s)
    else:
        d = s * (full - (ds * chosen).sum(dim=1, keepdim=True))
    return d.to(logits.dtype)


def _mx(v):
    """MXFP8 of 32-bit v in blocks of 32 along its last dimension: e4m3 values and powers of two."""
    blocks = v.view(*v.shape[:-1], -1, 32)
    top = blocks.abs().amax(dim=-1).view(torch.int32)
    t = ((top + 0x1FFFFF) >> 23).clamp(min=8)  # the exponent, one more where the mantissa is over 1.75 = 448 / 256
    scaled = blocks * ((262 - t) << 23).view(torch.float32)[..., None]
    return (scaled.clamp(-448, 448).to(torch.float8_e4m3fn).view(v.shape),
            (t - 8).to(torch.uint8).view(torch.float8_e8m0fnu))


def _mx_both(v, colwise=True):
    q, e8 = _mx(v)
    if not colwise:
        return {"q": q, "e8": e8}
    qT, e8T = _mx(v.t().contiguous())
    return {"q": q, "e8": e8, "qT": qT, "e8T": e8T}


def _undo(q, e8):
    return (q.float().view(*e8.shape, 32) * e8.float()[..., None]).view(q.shape)


def _gathered(x, src_of, top_k):
    rows = x.float()[(src_of.clamp(min=0) // top_k).long()]
    return torch.where((src_of >= 0)[:, None], rows, 0)


def _summed(rows, row_of, weights=None):
    """The rows of each token, times their weights, added up in 32 bits."""
    v = torch.where((row_of >= 0)[..., None], rows[row_of.clamp(min=0).long()].float(), 0)
    return (v if weights is None else v * weights[..., None]).sum(dim=1).to(rows.dtype)


def _run_plain(state):
    case = state["case"]
    if case["op"] == "route":
        experts, weights = _route_plain(state["logits"], state["bias"], case)
        out = {"experts": experts, "weights": weights}
        if case["train"]:
            out["dlogits"] = _route_back_plain(state["dweights"], state["logits"], experts, case)
        return out
    if case["op"] == "dispatch":
        plan = _plan_plain(state["experts"], case["experts"])
        out = {"plan": plan, "rows": _mx_both(_gathered(state["x"], plan["src_of"], case["top_k"]), case["train"])}
        if case["train"]:
            out["dx"] = _summed(state["drows"], plan["row_of"])
        return out
    if case["op"] == "combine":
        plan, w, y = state["plan"], state["weights"], state["y"]
        out = {"out": _summed(y, plan["row_of"], w)}
        if case["train"]:
            src, dout = plan["src_of"], state["dout"]
            mine = w.reshape(-1)[src.clamp(min=0).long()]
            out["drows"] = _mx_both(_gathered(dout, src, case["top_k"]) * mine[:, None])
            row, here = plan["row_of"].clamp(min=0).long(), plan["row_of"] >= 0
            out["dweights"] = torch.where(here, (y[row].float() * dout.float()[:, None]).sum(dim=2), 0)
        return out
    F = case["width"]
    h = state["h"].float()
    gate, up = h[:, :F], h[:, F:]
    out = {"a": _mx_both(gate / (1 + torch.exp(-gate)) * up, case["train"])}
    if case["train"]:
        out["kept"] = dict(zip(("q", "e8"), _mx(h)))
        h, da = _undo(*out["kept"].values()), state["da"].float()
        gate, up = h[:, :F], h[:, F:]
        sig = 1 / (1 + torch.exp(-gate))
        out["dh"] = _mx_both(torch.cat((da * up * sig * (1 + gate * (1 - sig)), da * gate * sig), dim=1))
    return out


# ------------------------------------------------------------------ the framework's calls

def _pair(p):
    return {n: v.view(torch.float8_e4m3fn if n[0] == "q" else torch.float8_e8m0fnu)
            for n, v in (("q", p.q), ("e8", p.e8), ("qT", p.qT), ("e8T", p.e8T)) if v is not None}


def _run_own(state):
    from mxfp8_precision_gemms_fp8bw_gb300 import moe

    case = state["case"]
    if case["op"] == "route":
        how = {n: case[n] for n in ("score", "renormalize", "scale")}
        experts, weights = moe.route(state["logits"], case["top_k"], bias=state["bias"], groups=case["groups"],
                                     groups_kept=case["groups_kept"], group_top=case["group_top"], **how)
        out = {"experts": experts, "weights": weights}
        if case["train"]:
            out["dlogits"] = moe.route_backward(state["dweights"], state["logits"], experts, **how)
        return out
    if case["op"] == "dispatch":
        plan = moe.plan(state["experts"], case["experts"])
        out = {"plan": {n: getattr(plan, n) for n in ("group_end", "counts", "row_of", "src_of")},
               "rows": _pair(moe.dispatch(state["x"], plan, colwise=case["train"]))}
        if case["train"]:
            out["dx"] = moe.dispatch_backward(state["drows"], plan)
        return out
    if case["op"] == "combine":
        plan = moe.Plan(**state["plan"])
        out = {"out": moe.combine(state["y"], state["weights"], plan)}
        if case["train"]:
            drows, out["dweights"] = moe.combine_backward(state["dout"], state["y"], state["weights"], plan)
            out["drows"] = _pair(drows)
        return out
    a, kept = moe.swiglu(state["h"], keep=case["train"], colwise=case["train"])
    out = {"a": _pair(a)}
    if case["train"]:
        out["kept"] = _pair(kept)
        out["dh"] = _pair(moe.swiglu_backward(state["da"], kept))
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    if case["op"] == "route":
        size = 2 if case["dtype"] == "bf16" else 4
        n, chosen = case["tokens"] * case["experts"], case["tokens"] * case["top_k"]
        return {"bytes": n * size * (2 if case["train"] else 1) + chosen * (12 if case["train"] else 8),
                "flops": n * (8 if case["train"] else 4)}
    if case["op"] == "swiglu":
        n = case["rows"] * case["width"]
        if not case["train"]:
            return {"bytes": n * (4 + 33 / 32), "flops": 8 * n}
        return {"bytes": n * (4 + 33 / 16 + 33 / 16 + 2 + 33 / 8), "flops": 30 * n}
    entries = int(case["tokens"] * (1 - case["padding"])) * case["top_k"]
    P = _capacity(case["tokens"], case["top_k"], case["experts"])
    token, moved, held = 2 * case["tokens"] * case["width"], 2 * entries * case["width"], P * case["width"] * 33 / 32
    if case["op"] == "dispatch":
        ints = 4 * (2 * case["tokens"] * case["top_k"] + P + 2 * case["experts"])
        return {"bytes": ints + token + (2 * held + moved + token if case["train"] else held),
                "flops": case["width"] * (4 * P + (entries if case["train"] else 0))}
    ints = 4 * (2 * case["tokens"] * case["top_k"])
    return {"bytes": ints + moved + token + (token + 2 * held + ints + 4 * P if case["train"] else 0),
            "flops": case["width"] * (2 * entries + (4 * P + 2 * entries if case["train"] else 0))}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_scores(x, score):
    if score == "sigmoid":
        return torch.sigmoid(x)
    return torch.nan_to_num(torch.softmax(x, dim=1), nan=0.0)  # a row with nothing in it has no scores


def _exact_pair(v, colwise=True):
    """What the codes and scales stand for before the elements are rounded to 8 bits."""
    out = {}
    for q, e8, w in (("q", "e8", v), ("qT", "e8T", v.t()))[:2 if colwise else 1]:
        blocks = w.reshape(w.shape[0], -1, 32)
        top = blocks.abs().amax(dim=2, keepdim=True)
        m, ex = torch.frexp(top / 448)  # top / 448 = m 2^ex, 1/2 <= m < 1: the power of two itself has m = 1/2
        E = torch.where(top > 0, ex - (m == 0.5).to(ex.dtype), -127).clamp(-127, 127).double()
        out[q], out[e8] = (blocks / torch.exp2(E)).reshape(w.shape), torch.exp2(E)[..., 0]
    return out


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "route":
        x = state["logits"].double()
        s = _exact_scores(x, case["score"])
        b = 0.0 if state["bias"] is None else state["bias"].double()
        key = torch.where(x == float("-inf"), float("-inf"), s + b)
        if case["groups"] > 1:
            parts = key.unflatten(1, (case["groups"], -1))
            total = parts.topk(case["group_top"], dim=2).values.clamp(min=LOWEST).sum(dim=2)
            order = total.argsort(dim=1, descending=True, stable=True)
            place = order.argsort(dim=1)[:, :, None]
            key = torch.where(place < case["groups_kept"], parts, float("-inf")).flatten(1)
        value, index = key.sort(dim=1, descending=True, stable=True)
        value, index = value[:, :case["top_k"]], index[:, :case["top_k"]]
        leaf = s.clone().requires_grad_(True)
        live = (value > float("-inf")).double()
        w = leaf.gather(1, index) * live
        if case["renormalize"]:
            w = w / (w.sum(dim=1, keepdim=True) + 1e-20)
        w = w * case["scale"]
        out = {"experts": None, "weights": w.detach()}
        if case["train"]:
            (ds,) = torch.autograd.grad(w, leaf, state["dweights"].double())
            out["dlogits"] = s * (1 - s) * ds if case["score"] == "sigmoid" else s * (ds - (s * ds).sum(dim=1, keepdim=True))
        return out
    if case["op"] == "swiglu":
        h, F = state["h"].double(), case["width"]
        act = lambda t: t[:, :F] * torch.sigmoid(t[:, :F]) * t[:, F:]  # noqa: E731
        out = {"a": _exact_pair(act(h), case["train"])}
        if case["train"]:
            out["kept"] = _exact_pair(h, colwise=False)
            # the gradient is that of the input as it is kept, in 8 bits
            codes = out["kept"]["q"].float().to(torch.float8_e4m3fn).double().view(h.shape[0], -1, 32)
            kept = (codes * out["kept"]["e8"][..., None]).view(h.shape)
            del codes, h
            gate, up = kept[:, :F], kept[:, F:]
            da, sig = state["da"].double(), torch.sigmoid(gate)
            dh = torch.cat((da * up * (sig + gate * sig * (1 - sig)), da * gate * sig), dim=1)
            del kept, gate, up, da, sig
            out["dh"] = _exact_pair(dh)
        return out
    k = case["top_k"]
    if case["op"] == "dispatch":
        experts, x = state["experts"].long().reshape(-1), state["x"].double()
        order = torch.sort(torch.where(experts < 0, case["experts"], experts), stable=True).indices
        counts = torch.bincount(experts[experts >= 0], minlength=case["experts"])
        blocks = (counts + 31) // 32 * 32
        shift = torch.cumsum(blocks - counts, 0) - (blocks - counts)
        order = order[:int(counts.sum())]
        place = torch.arange(order.numel(), device="cuda") + shift[experts[order]]
        rows = torch.zeros(_capacity(case["tokens"], k, case["experts"]), case["width"], dtype=torch.float64, device="cuda")
        rows[place] = x[order // k]
        out = {"plan": {n: None for n in ("group_end", "counts", "row_of", "src_of")}, "rows": _exact_pair(rows, case["train"])}
        if case["train"]:
            out["dx"] = torch.zeros_like(x).index_add_(0, order // k, state["drows"].double()[place])
        return out
    plan, w = state["plan"], state["weights"].double().reshape(-1)
    here = torch.nonzero(plan["src_of"] >= 0)[:, 0]
    entry = plan["src_of"][here].long()
    y = state["y"][here].double()
    total = torch.zeros(case["tokens"], case["width"], dtype=torch.float64, device="cuda")
    out = {"out": total.index_add_(0, entry // k, y * w[entry][:, None])}
    if case["train"]:
        dout = state["dout"].double()[entry // k]
        rows = torch.zeros(state["y"].shape, dtype=torch.float64, device="cuda")
        rows[here] = dout * w[entry][:, None]
        out["drows"] = _exact_pair(rows)
        out["dweights"] = torch.zeros_like(w).index_add_(0, entry, (dout * y).sum(dim=1)).view(case["tokens"], k)
    return out
