"""What the operators of a block of experts on packed weights are measured on.

Four operators: routing (the k experts of every token, their weights, and the tokens' places where
they are sorted by expert; for training the gradient of the weights), spreading (tokens into
the sorted rows; its gradient), combining (sorted rows back into tokens, weighted; its gradients), and
the product with packed low-bit weights whose epilogue adds a bias, applies an activation, gated or
not, and adds a residual: of one projection for all rows, or of each expert for its own.  The plain
forms below are their definitions in elementary torch operations.

Pair t k + j is token t's j-th expert.  Sorted by expert, an expert's pairs in their own order:
`order` [T k] names the pair of each sorted row, `place` [T, k] the row of each pair, `offsets` [E + 1]
where each expert's rows begin.  Pairs of an expert outside [0, E), one that another GPU holds, come
last, past offsets[E]: their rows are zero and add nothing.

Packed weights: codes_t [K/32, rows, bits] words, 32 codes of `bits` bits each in a row's words, lowest
bits first; meta_t [K/group, rows, 2] the group's step and zero point; weight = (code - zero) step.
The rows of all experts stand one after another; gated, an expert's first half are the gates.
"""

import math
import random

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}


def _lib():
    import post_weight_quantization_act_amd as awq
    return awq


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one token of a decode step: latency
        dict(name="route-step", op="route", tokens=1, experts=128, of=128, k=8, score="softmax", normalise=True,
             bias=False, type="bf16", train=False),
        # a long prompt, many experts, selection by a balancing bias
        dict(name="route-prompt", op="route", tokens=16381, experts=256, of=256, k=8, score="sigmoid",
             normalise=True, bias=True, type="f32", train=False),
        # a training step's router, weights as they come out of the softmax, and its gradient
        dict(name="route-train", op="route", tokens=8191, experts=64, of=64, k=6, score="softmax", normalise=False,
             bias=False, type="bf16", train=True),
        # a prompt's tokens into their experts' rows
        dict(name="spread-prompt", op="spread", tokens=8191, experts=128, of=128, k=8, columns=2048, type="bf16",
             weighted=False, train=False),
        # a small decode batch's rows back, onto the residual stream: latency
        dict(name="combine-step", op="combine", tokens=5, experts=128, of=128, k=8, columns=2048, type="bf16",
             weighted=True, residual=True, train=False),
        # a training step: rows back, and the gradients of rows and weights
        dict(name="combine-train", op="combine", tokens=4095, experts=64, of=64, k=6, columns=4096, type="f16",
             weighted=True, residual=False, train=True),
        # one token through a large up projection, 3 bits, bias and activation
        dict(name="linear-step", op="linear", rows=1, n=28672, kk=8192, bits=3, group=128, act="gelu_tanh",
             gated=False, bias=True, residual=False, type="bf16", out="bf16"),
        # a prompt through a down projection, onto the residual stream
        dict(name="linear-prompt", op="linear", rows=2047, n=4096, kk=11008, bits=4, group=128, act="none",
             gated=False, bias=False, residual=True, type="f16", out="f16"),
        # one token through its eight experts' gate and up projections: latency
        dict(name="experts-step", op="experts", tokens=1, experts=128, of=128, k=8, n=1536, kk=2048, bits=4,
             group=128, act="silu", gated=True, bias=False, sorted=False, type="bf16", out="bf16"),
        # a decode batch through them: a few rows for each expert
        dict(name="experts-batch", op="experts", tokens=61, experts=128, of=128, k=8, n=1536, kk=2048, bits=4,
             group=128, act="silu", gated=True, bias=False, sorted=False, type="bf16", out="bf16"),
        # a prompt through the experts' gate and up projections, rows taken from the tokens
        dict(name="experts-prompt", op="experts", tokens=4095, experts=64, of=64, k=6, n=2816, kk=2048, bits=4,
             group=128, act="silu", gated=True, bias=False, sorted=False, type="bf16", out="bf16"),
        # the same prompt's sorted rows through their down projections
        dict(name="experts-down", op="experts", tokens=4095, experts=64, of=64, k=6, n=2048, kk=1408, bits=4,
             group=128, act="none", gated=False, bias=False, sorted=True, type="bf16", out="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "spread", "combine", "linear", "linear", "experts", "experts"])
    kind = rng.choice(["f16", "bf16"])
    experts = rng.choice([8, 16, 60, 64, 128, 160, 256])
    # all experts here, or this GPU's share of them
    of = experts if rng.random() < 0.75 else 2 * experts
    k = rng.choice([1, 2, 4, 6, 8])
    if op == "route":
        return dict(op=op, tokens=_log(rng, 1, 16381 * 256 // max(of, 64)), experts=experts, of=of, k=k,
                    score=rng.choice(["softmax", "sigmoid"]), normalise=rng.random() < 0.6,
                    bias=rng.random() < 0.4, type=rng.choice(["f32", kind]), train=rng.random() < 0.4)
    if op in ("spread", "combine"):
        columns = _log(rng, 64, 8192)
        columns = columns // 8 * 8 if rng.random() < 0.8 else columns
        case = dict(op=op, tokens=_log(rng, 1, min(16384, 8191 * 8 * 2048 // (2 * k * columns))), experts=experts, of=of,
                    k=k, columns=columns, type=rng.choice(["f32", kind, kind]), weighted=rng.random() < 0.6,
                    train=rng.random() < 0.4)
        return case if op == "spread" else dict(case, residual=rng.random() < 0.5)
    bits, group = rng.choice([2, 3, 3, 4, 4, 4, 5, 6, 8]), rng.choice([32, 64, 128, 128, 128, 256])
    act, gated = rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh"]), rng.random() < 0.4
    bias, out = rng.random() < 0.3, rng.choice(["f32", kind, kind])
    if op == "linear":
        kk = group * _log(rng, 1, 11008 // group)
        n = _log(rng, 16, min(28672, 110000000 // kk))
        n = n // 2 * 2 if gated else n
        rows = _log(rng, 1, max(1, min(4096, 2047 * 4096 * 11008 // (n * kk))))
        return dict(op=op, rows=rows, n=n, kk=kk, bits=bits, group=group, act=act, gated=gated, bias=bias,
                    residual=rng.random() < 0.4, type=kind, out=out)
    experts, of, k = min(experts, 128), min(of, 256), min(k, 6)
    of = experts if of < 2 * experts else of
    kk = group * _log(rng, max(1, 256 // group), 2048 // group)
    n = _log(rng, 64, min(8192, 200000000 // (experts * kk)))
    n = n // 2 * 2 if gated else n
    tokens = _log(rng, 1, max(1, min(4095, 4095 * 6 * 2816 * 2048 // (2 * k * n * kk))))
    return dict(op=op, tokens=tokens, experts=experts, of=of, k=k, n=n, kk=kk, bits=bits, group=group, act=act,
                gated=gated, bias=bias, sorted=rng.random() < 0.4, type=kind, out=out)


def work(case):
    op, of = case["op"], case.get("of")
    if op == "route":
        t, k, size = case["tokens"], case["k"], _BYTES[case["type"]]
        # logits in; weights, experts, order and place out; for training weights' gradient in, logits' out
        return {"bytes": t * of * size * (2 if case["train"] else 1) + t * k * (20 if case["train"] else 16)
                + 4 * case["experts"] + (4 * of if case["bias"] else 0),
                "flops": t * of * (12 if case["train"] else 8)}
    if op in ("spread", "combine"):
        t, k, c, size = case["tokens"], case["k"], case["columns"], _BYTES[case["type"]]
        kept = t * k * case["experts"] // of
        # tokens on one side, sorted rows on the other; the gradients the other way, and for weights
        # what they are the products of
        token, rows = t * c * size, t * k * c * size if op == "spread" else kept * c * size
        total, flops = token + rows + t * k * 8, kept * c * 2
        if op == "combine" and case["residual"]:
            total += token
        if case["train"]:
            total += token + t * k * c * size + t * k * 4
            flops += kept * c * (4 if case["weighted"] else 1)
        return {"bytes": total, "flops": flops}
    n, kk, size, wide = case["n"], case["kk"], _BYTES[case["type"]], _BYTES[case["out"]]
    outs = n // 2 if case["gated"] else n
    if op == "linear":
        rows = kept = sources = case["rows"]
        held = 1
    else:
        rows = case["tokens"] * case["k"]
        kept = rows * case["experts"] / of
        sources = kept if case["sorted"] else case["tokens"]
        # experts that some token takes, were all taken alike
        held = case["experts"] * (1 - (1 - case["k"] / of) ** case["tokens"])
    return {"bytes": int(held * n * (kk * case["bits"] / 8 + kk / case["group"] * 8 + (4 if case["bias"] else 0))
                         + sources * kk * size + rows * outs * wide * (2 if case.get("residual") else 1)),
            "flops": int(2.0 * kept * n * kk)}


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------
def _pack(gen, rows, kk, bits, group):
    """Codes and (step, zero) of weights whose groups are normal: most codes lie near the zero point."""
    top = 2 ** bits - 1
    words = torch.empty((kk // 32, rows, bits), dtype=torch.int32, device="cuda")
    for part in words.split(max(1, (1 << 24) // (rows * 32))):
        c = torch.randn((*part.shape[:2], 32), generator=gen, device="cuda").mul_((top + 1) / 5.3).add_(top / 2)
        c = c.round_().clamp_(0, top).long()
        for w in range(bits):
            word = torch.zeros(part.shape[:2], dtype=torch.int64, device="cuda")
            for i in range(32):
                at = i * bits - 32 * w
                if -bits < at < 32:
                    word |= c[..., i] << at if at >= 0 else c[..., i] >> -at
            word &= 0xFFFFFFFF
            part[..., w] = torch.where(word >= 2 ** 31, word - 2 ** 32, word).int()
    meta = torch.empty((kk // group, rows, 2), dtype=torch.float32, device="cuda")
    meta[..., 0] = (torch.randn(meta.shape[:2], generator=gen, device="cuda") * 0.15).exp_() * (5.3 / (top + 1) * kk ** -0.5)
    meta[..., 1] = (torch.randn(meta.shape[:2], generator=gen, device="cuda") * 0.5 + top / 2).round_().clamp_(0, top)
    return words, meta


def _sorted(experts, count):
    """offsets, order and place of the experts [T, k]; those outside [0, count) last."""
    e = torch.where((experts >= 0) & (experts < count), experts, count).flatten().long()
    order = torch.sort(e, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device="cuda")
    offsets = torch.zeros(count + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = (e[:, None] == torch.arange(count, device="cuda")).sum(0).cumsum(0)
    return offsets.int(), order.int(), place.view(experts.shape).int()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 6151 + 29)

    def normal(*shape, dtype):
        # a few channels are large, as in the activations of real layers
        x = torch.randn(shape, generator=gen, device="cuda")
        x.mul_(torch.where(torch.rand(shape[-1], generator=gen, device="cuda") < 0.03, 6.0, 1.0))
        return x.to(_TYPES[dtype])

    s = {"case": case}
    if case["op"] != "linear":
        t, of, k = case["tokens"], case["of"], case["k"]
        # some experts are liked more than others
        logits = torch.randn((t, of), generator=gen, device="cuda") * 1.5 + torch.randn(of, generator=gen, device="cuda") * 0.3
        if case["op"] == "route":
            s["logits"] = logits.to(_TYPES[case["type"]])
            s["bias"] = torch.randn(of, generator=gen, device="cuda") * 0.1 if case["bias"] else None
            s["dweights"] = torch.randn((t, k), generator=gen, device="cuda")
            return s
        s["experts"] = logits.topk(k, dim=-1).indices.int()
        s["weights"] = logits.topk(k, dim=-1).values.softmax(-1)
        s["offsets"], s["order"], s["place"] = _sorted(s["experts"], case["experts"])
    if case["op"] in ("spread", "combine"):
        c, n = case["columns"], t * k
        if case["op"] == "spread":
            s["x"] = normal(t, c, dtype=case["type"])
            s["dout"] = normal(n, c, dtype=case["type"]) if case["train"] else None
            return s
        s["rows"] = normal(n, c, dtype=case["type"])
        s["residual"] = normal(t, c, dtype=case["type"]) if case["residual"] else None
        s["dout"] = normal(t, c, dtype=case["type"]) if case["train"] else None
        return s
    n, kk = case["n"], case["kk"]
    count = case.get("experts", 1)
    s["codes"], s["meta"] = _pack(gen, count * n, kk, case["bits"], case["group"])
    s["bias"] = torch.randn((count, n), generator=gen, device="cuda") * 0.2 if case["bias"] else None
    if case["op"] == "linear":
        s["x"] = normal(case["rows"], kk, dtype=case["type"])
        outs = n // 2 if case["gated"] else n
        s["residual"] = normal(case["rows"], outs, dtype=case["out"]) if case["residual"] else None
    else:
        s["x"] = normal(t * k if case["sorted"] else t, kk, dtype=case["type"])
        # rows of the expert that has most: what the plain form's batch is padded to
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    return s


# ---------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------
def _plain_route(s):
    c = s["case"]
    l64 = s["logits"].double()
    # the choice lies next to a border: 64 bits
    key = torch.sigmoid(l64) if c["score"] == "sigmoid" else l64
    if s["bias"] is not None:
        key = key + s["bias"].double()
    experts = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, : c["k"]]
    l = s["logits"].float()
    if c["score"] == "softmax":
        p = (l - l.amax(-1, keepdim=True)).exp()
        p = p / p.sum(-1, keepdim=True)
    else:
        p = 1 / (1 + (-l).exp())
    chosen = torch.gather(p, 1, experts)
    total = chosen.sum(-1, keepdim=True)
    w = chosen / total if c["normalise"] else chosen
    w = w * _scale(c)
    offsets, order, place = _sorted(experts, c["experts"])
    out = {"experts": experts.int(), "weights": w, "offsets": offsets, "order": order, "place": place}
    if c["train"]:
        g = s["dweights"] * _scale(c)
        if c["normalise"]:  # through the division by the sum
            g = (g - (g * chosen).sum(-1, keepdim=True) / total) / total
        dp = torch.zeros_like(p).scatter_(1, experts, g)
        if c["score"] == "softmax":
            dl = p * (dp - (dp * p).sum(-1, keepdim=True))
        else:
            dl = dp * p * (1 - p)
        out["dlogits"] = dl.to(s["logits"].dtype)
    return out


def _scale(case):
    return 2.5 if case["score"] == "sigmoid" else 1.0


def _kept(s):
    """Which pairs an expert here has, [T, k]."""
    return s["place"] < s["offsets"][-1]


def _plain_spread(s):
    c = s["case"]
    t, k = s["experts"].shape
    w = torch.where(_kept(s), s["weights"] if c["weighted"] else 1.0, 0.0)
    order = s["order"].long()
    rows = (s["x"].float()[order // k] * w.flatten()[order, None]).to(s["x"].dtype)
    if not c["train"]:
        return {"rows": rows}
    d = s["dout"].float()[s["place"].long()]                                   # [T, k, C]
    out = {"rows": rows, "dx": (d * w[..., None]).sum(1).to(s["x"].dtype)}
    if c["weighted"]:
        out["dweights"] = torch.where(_kept(s), (d * s["x"].float()[:, None]).sum(-1), 0.0)
    return out


def _plain_combine(s):
    c = s["case"]
    t, k = s["experts"].shape
    kept = _kept(s)
    w = torch.where(kept, s["weights"] if c["weighted"] else 1.0, 0.0)
    r = s["rows"].float()[s["place"].long()]                                   # [T, k, C]
    y = (r * w[..., None]).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"y": y.to(s["rows"].dtype)}
    if c["train"]:
        order, d = s["order"].long(), s["dout"].float()
        out["drows"] = (d[order // k] * w.flatten()[order, None]).to(s["rows"].dtype)
        if c["weighted"]:
            out["dweights"] = torch.where(kept, (r * d[:, None]).sum(-1), 0.0)
    return out


def _weights(codes, meta, bits, group):
    """Packed rows [..., K/32, n, bits] and [..., K/group, n, 2] as values [..., K, n] in 32 bits."""
    i = torch.arange(32, device="cuda") * bits
    low = codes.long() & 0xFFFFFFFF
    both = low | (torch.cat((low[..., 1:], low[..., :1]), -1) << 32)            # a code may end in the next word
    c = (both[..., i // 32] >> (i % 32)) & (2 ** bits - 1)                       # [..., K/32, n, 32]
    c = c.float().transpose(-1, -2).flatten(-3, -2)                              # [..., K, n]
    step, zero = meta.repeat_interleave(group, -3).unbind(-1)
    return (c - zero) * step


def _act(y, act):
    if act == "relu":
        return y.clamp(min=0)
    if act == "silu":
        return y / (1 + (-y).exp())
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh((2 / math.pi) ** 0.5 * (y + 0.044715 * y * y * y)))
    return y


def _finish(case, y):
    if not case["gated"]:
        return _act(y, case["act"])
    gate, up = y.chunk(2, -1)
    return _act(gate, case["act"]) * up


def _plain_linear(s):
    c = s["case"]
    y = s["x"].float() @ _weights(s["codes"], s["meta"], c["bits"], c["group"])
    if s["bias"] is not None:
        y = y + s["bias"]
    y = _finish(c, y)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(_TYPES[c["out"]])}


def _plain_experts(s):
    c = s["case"]
    n, e = c["n"], c["experts"]
    rows = s["order"].numel()
    codes = s["codes"].view(-1, e, n, c["bits"]).transpose(0, 1)                # [E, K/32, n, bits]
    meta = s["meta"].view(-1, e, n, 2).transpose(0, 1)
    bias = s["bias"]
    source = torch.arange(rows, device="cuda") if c["sorted"] else s["order"].long() // c["k"]
    out = torch.zeros((rows, n // 2 if c["gated"] else n), dtype=_TYPES[c["out"]], device="cuda")
    if rows <= e:                                                               # fewer rows than experts: each row's own
        mine = s["experts"].flatten()[s["order"].long()].long()
        there = (mine < e)[:, None]
        mine = mine.clamp(max=e - 1)
        y = torch.bmm(s["x"].float()[source][:, None], _weights(codes[mine], meta[mine], c["bits"], c["group"]))[:, 0]
        y = y + bias[mine] if bias is not None else y
        return {"y": torch.where(there, _finish(c, y).to(out.dtype), out)}
    # every expert's rows, padded to those of the one that has most
    at = s["offsets"][:-1, None].long() + torch.arange(s["most"], device="cuda")
    there = at < s["offsets"][1:, None]
    x = s["x"].float()[source[at.clamp(max=rows - 1)]]
    y = torch.bmm(x, _weights(codes, meta, c["bits"], c["group"]))
    y = y + bias[:, None] if bias is not None else y
    out[at[there]] = _finish(c, y).to(out.dtype)[there]
    return {"y": out}


# ---------------------------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------------------------
def _own(s):
    awq, c = _lib(), s["case"]
    if c["op"] == "route":
        logits = s["logits"].detach().requires_grad_() if c["train"] else s["logits"]
        r = awq.awq_moe_route(logits, c["k"], score=c["score"], bias=s["bias"], normalise=c["normalise"],
                              scale=_scale(c), num_experts=c["experts"])
        out = {"experts": r.experts, "weights": r.weights.detach(), "offsets": r.offsets, "order": r.order,
               "place": r.place}
        if c["train"]:
            out["dlogits"], = torch.autograd.grad(r.weights, logits, s["dweights"])
        return out
    if c["op"] == "linear":
        return {"y": awq.awq_lowbit_linear(s["x"], s["codes"], s["meta"], c["bits"], c["group"], bias=s["bias"],
                                           activation=c["act"], gated=c["gated"], residual=s["residual"],
                                           out_dtype=_TYPES[c["out"]])}
    routing = awq.Routing(s["experts"], s["weights"], s["offsets"], s["order"], s["place"])
    if c["op"] == "experts":
        return {"y": awq.awq_lowbit_linear(s["x"], s["codes"], s["meta"], c["bits"], c["group"], bias=s["bias"],
                                           activation=c["act"], gated=c["gated"], routing=routing,
                                           gather=not c["sorted"], out_dtype=_TYPES[c["out"]])}
    weights = s["weights"] if c["weighted"] else None
    if not c["train"]:
        if c["op"] == "spread":
            return {"rows": awq.awq_moe_gather(s["x"], routing, weights)}
        return {"y": awq.awq_moe_combine(s["rows"], routing, weights, residual=s["residual"])}
    leaf = (s["x"] if c["op"] == "spread" else s["rows"]).detach().requires_grad_()
    leaves = [leaf]
    if weights is not None:
        weights = weights.detach().requires_grad_()
        leaves.append(weights)
    if c["op"] == "spread":
        y = awq.awq_moe_gather(leaf, routing, weights)
    else:
        y = awq.awq_moe_combine(leaf, routing, weights, residual=s["residual"])
    grads = torch.autograd.grad(y, leaves, s["dout"])
    out = dict(zip(("dx", "dweights") if c["op"] == "spread" else ("drows", "dweights"), grads))
    out["rows" if c["op"] == "spread" else "y"] = y.detach()
    return out


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "spread": _plain_spread, "combine": _plain_combine, "linear": _plain_linear,
            "experts": _plain_experts}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------
# 64 bits, token by token or expert by expert
# ---------------------------------------------------------------------------------------------
def _exact_route(s):
    c = s["case"]
    l = s["logits"].double().requires_grad_()
    key = (torch.sigmoid(l) if c["score"] == "sigmoid" else l).detach().clone()
    if s["bias"] is not None:
        key += s["bias"].double()
    picks = []
    for _ in range(c["k"]):                                   # the largest, the lowest of equals, k times
        best = key.amax(-1, keepdim=True)
        index = torch.where(key == best, torch.arange(key.shape[1], device="cuda"), key.shape[1]).amin(-1, keepdim=True)
        picks.append(index)
        key.scatter_(1, index, -math.inf)
    at = torch.cat(picks, 1)
    p = torch.softmax(l, -1) if c["score"] == "softmax" else torch.sigmoid(l)
    w = p.gather(1, at)
    w = _scale(c) * (w / w.sum(-1, keepdim=True) if c["normalise"] else w)
    out = {"experts": None, "weights": w.detach(), "offsets": None, "order": None, "place": None}
    if c["train"]:
        out["dlogits"], = torch.autograd.grad(w, l, s["dweights"].double())
    return out


def _exact_rows(s):
    """Spread and combine, one choice of every token after another."""
    c, (t, k) = s["case"], s["experts"].shape
    here = s["experts"] < c["experts"]
    tokens = s["x"] if c["op"] == "spread" else s["dout"]     # what goes to the rows
    rows = s["dout"] if c["op"] == "spread" else s["rows"]    # what comes back from them
    there = back = None
    if tokens is not None:
        there = torch.zeros((t * k, c["columns"]), dtype=torch.float64, device="cuda")
    if rows is not None:
        back = torch.zeros((t, c["columns"]), dtype=torch.float64, device="cuda")
    dots = torch.zeros((t, k), dtype=torch.float64, device="cuda")
    for j in range(k):
        w = (s["weights"][:, j].double() if c["weighted"] else torch.ones(t, dtype=torch.float64, device="cuda")) * here[:, j]
        at = s["place"][:, j].long()
        if there is not None:
            there[at] = tokens.double() * w[:, None]
        if back is not None:
            back += rows[at].double() * w[:, None]
        if there is not None and back is not None:
            dots[:, j] = torch.linalg.vecdot(tokens.double(), rows[at].double()) * here[:, j]
    more = {"dweights": dots} if c["train"] and c["weighted"] else {}
    if c["op"] == "spread":
        return {"rows": there, **({"dx": back} if c["train"] else {}), **more}
    if s["residual"] is not None:
        back += s["residual"].double()
    return {"y": back, **({"drows": there} if c["train"] else {}), **more}


def _exact_weights(case, codes, meta):
    """[n, K] from the bits of the words' bytes, lowest first."""
    b = case["bits"]
    at = torch.arange(8, device="cuda", dtype=torch.uint8)
    stream = ((codes.contiguous().view(torch.uint8)[..., None] >> at) & 1).flatten(-2).unflatten(-1, (32, b))
    value = (stream.double() * (2.0 ** torch.arange(b, device="cuda", dtype=torch.float64))).sum(-1)      # [K/32, n, 32]
    value = value.permute(1, 0, 2).reshape(codes.shape[1], -1, case["group"])
    m = meta.double().permute(1, 0, 2)
    return ((value - m[..., 1:]) * m[..., :1]).flatten(1)


def _exact_finish(case, y):
    if case["gated"]:
        half = y.shape[1] // 2
        y, up = y[:, :half], y[:, half:]
    act = {"none": lambda v: v, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
           "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[case["act"]]
    return act(y) * up if case["gated"] else act(y)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    if case["op"] in ("spread", "combine"):
        return _exact_rows(s)
    n, x = case["n"], s["x"].double()
    if case["op"] == "linear":
        y = torch.empty((case["rows"], n), dtype=torch.float64, device="cuda")
        for r in range(0, n, 2048):
            part = slice(r, r + 2048)
            y[:, part] = x @ _exact_weights(case, s["codes"][:, part], s["meta"][:, part]).T
        y = y if s["bias"] is None else y + s["bias"].double()
        y = _exact_finish(case, y)
        return {"y": y if s["residual"] is None else y + s["residual"].double()}
    out = torch.zeros((case["tokens"] * case["k"], n // 2 if case["gated"] else n), dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        pairs = (s["experts"] == e).flatten().nonzero()[:, 0]
        if not pairs.numel():
            continue
        to = s["place"].flatten()[pairs].long()
        own_rows = slice(e * n, (e + 1) * n)
        w = _exact_weights(case, s["codes"][:, own_rows], s["meta"][:, own_rows])
        y = (x[to] if case["sorted"] else x[pairs // case["k"]]) @ w.T
        out[to] = _exact_finish(case, y if s["bias"] is None else y + s["bias"][e].double())
    return {"y": out}
