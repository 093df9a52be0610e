"""The router and its gradient at the ends of their ranges on the GPU, against the 64-bit oracle."""

import numpy as np
import pytest
import torch

import post_weight_quantization_act_amd as awq
from oracle import moe_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    awq.library()
    yield
    torch.cuda.synchronize()


def wide(t):
    """Exact fp64 NumPy copy."""
    return t.detach().double().cpu().numpy()


def ints(t):
    return t.cpu().numpy().astype(np.int64)


# ---------------------------------------------------------------------------------------------
# sigmoids of logits far below 0
# ---------------------------------------------------------------------------------------------
LEVELS = [0, -70, -79, -81, -87, -88.5, -90, -97, -103, -110, -200, -400, -690]


def low_logits(rng, E, kind):
    """Rows about each level, rows of which some are ordinary and the rest low, rows all but two masked."""
    rows = [level + rng.normal(size=E) * 2 for level in LEVELS for _ in range(3)]
    for level in LEVELS:
        row = level + rng.normal(size=E)
        row[rng.permutation(E)[:2]] += 45
        rows.append(row)
        row = np.full(E, -np.inf)
        row[rng.permutation(E)[:2]] = level + rng.normal(size=2)
        rows.append(row)
    x = np.stack(rows)[rng.permutation(len(rows))].astype(np.float32)
    return torch.from_numpy(x).to(TYPES[kind]).cuda()


@pytest.mark.parametrize("E,k", [(8, 2), (40, 6), (70, 17)])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("normalise", [True, False])
def test_low_sigmoids(E, k, kind, normalise):
    rng = np.random.default_rng(E + k)
    logits = low_logits(rng, E, kind)
    x = wide(logits)
    r = awq.awq_moe_route(logits, k, score="sigmoid", normalise=normalise, scale=1.5)
    e = ref.choose(x, k, "sigmoid")
    assert (ints(r.experts) == e).all()
    w = ref.route_weights(x, e, "sigmoid", normalise, 1.5)
    # an exponential (2 ulp), a sum, a quotient, their sum, a quotient and a product; below 2^-126 half a step
    # of the subnormals
    assert (np.abs(wide(r.weights) - w) <= (8 + E / 16) * 2.0 ** -24 * w + TINY["f32"]).all()
    if normalise:
        assert (np.abs(wide(r.weights).sum(1) - 1.5) < 1e-5).all()       # every row has some that are not -inf


@pytest.mark.parametrize("E,k", [(8, 2), (40, 6), (70, 17)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("normalise", [True, False])
def test_gradient_of_low_sigmoids(E, k, kind, normalise):
    rng = np.random.default_rng(E * 3 + k)
    logits = low_logits(rng, E, kind).requires_grad_()
    g = torch.from_numpy(rng.normal(size=(logits.shape[0], k)).astype(np.float32)).cuda()
    r = awq.awq_moe_route(logits, k, score="sigmoid", normalise=normalise, scale=0.7)
    d, = torch.autograd.grad(r.weights, logits, g)
    x, e, gn = wide(logits), ints(r.experts), wide(g)
    want = ref.route_grad(x, e, gn, "sigmoid", normalise, 0.7)
    # share (g - sum g share) (1 - p): each factor as the weights above, the sum k additions more
    q = ref.route_weights(x, e, "sigmoid", normalise)
    size = np.zeros_like(x)
    np.put_along_axis(size, e, 0.7 * q * (np.abs(gn) + (q * np.abs(gn)).sum(1, keepdims=True)), 1)
    bound = (3 * (8 + E / 16) + k + 8) * 2.0 ** -24 * size + 4 * TINY["f32"]
    assert (np.abs(wide(d) - want) <= bound + HALF_ULP[kind] * np.abs(want) + TINY[kind]).all()


def test_low_rows_do_not_change_their_neighbours():
    rng = np.random.default_rng(2)
    logits = torch.from_numpy(rng.normal(size=(64, 16)).astype(np.float32)).cuda()
    alone = awq.awq_moe_route(logits, 4, score="sigmoid").weights
    mixed = logits.clone()
    mixed[1::2] -= 95
    got = awq.awq_moe_route(mixed, 4, score="sigmoid").weights
    assert torch.equal(got[::2], alone[::2]) and not torch.equal(got[1::2], alone[1::2])


# ---------------------------------------------------------------------------------------------
# more tokens than one launch has threads for
# ---------------------------------------------------------------------------------------------
def test_gradient_of_more_than_two_to_the_28_tokens():
    """Sixteen threads a token: 2^32 and more. The last token, those around the first launch's end, and all."""
    T = 2 ** 28 + 2 ** 20 + 7
    gen = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.empty((T, 2), dtype=torch.float16, device="cuda").normal_(generator=gen).requires_grad_()
    g = torch.empty((T, 1), device="cuda").normal_(generator=gen)
    r = awq.awq_moe_route(logits, 1, score="sigmoid", normalise=False)
    d, = torch.autograd.grad(r.weights, logits, g)
    for lo in range(0, T, 2 ** 24):
        part = slice(lo, lo + 2 ** 24)
        x, e = logits.detach()[part].double(), r.experts[part].long()
        assert torch.equal(e, (x[:, 1:] > x[:, :1]).long())
        p = torch.sigmoid(x)
        want = torch.zeros_like(x).scatter_(1, e, g[part].double()) * p * (1 - p)
        # five roundings in fp32 and the exponentials' two ulp, one to fp16
        bound = (16 * 2.0 ** -24 + HALF_ULP["f16"]) * want.abs() + TINY["f16"]
        assert bool(((d[part].double() - want).abs() <= bound).all()), lo


# ---------------------------------------------------------------------------------------------
# derivatives that are not recorded, and what a backward pass has kept
# ---------------------------------------------------------------------------------------------
def test_tangents_are_refused():
    from torch.autograd import forward_ad

    logits, x, rows = (torch.randn(s, device="cuda") for s in ((5, 8), (5, 16), (10, 16)))
    w, bias = torch.randn(5, 2, device="cuda"), torch.zeros(8, device="cuda")
    with forward_ad.dual_level():
        def d(t):
            return forward_ad.make_dual(t, torch.ones_like(t))

        r = awq.awq_moe_route(logits, 2, bias=bias)
        awq.awq_moe_combine(awq.awq_moe_gather(x, r, w), r, w, residual=x)
        for call in (lambda: awq.awq_moe_route(d(logits), 2), lambda: awq.awq_moe_route(logits, 2, bias=d(bias)),
                     lambda: awq.awq_moe_route_grad(logits, r.experts, d(w)), lambda: awq.awq_moe_gather(d(x), r),
                     lambda: awq.awq_moe_gather(x, r, d(w)), lambda: awq.awq_moe_gather(d(x), r, out=torch.empty_like(rows)),
                     lambda: awq.awq_moe_combine(d(rows), r), lambda: awq.awq_moe_combine(rows, r, d(w)),
                     lambda: awq.awq_moe_combine(rows, r, residual=d(x)), lambda: awq.awq_moe_combine_grad(d(x), r, rows=rows),
                     lambda: awq.awq_moe_combine_grad(x, r, rows=d(rows))):
            with pytest.raises(RuntimeError, match="forward-mode"):
                call()


@pytest.mark.parametrize("which", ["place", "offsets"])
def test_lists_that_are_written_before_the_backward_pass_are_found_out(which):
    x, rows = torch.randn(5, 16, device="cuda", requires_grad=True), torch.randn(10, 16, device="cuda", requires_grad=True)
    logits = torch.randn(5, 8, device="cuda")
    for call in (lambda r: awq.awq_moe_gather(x, r), lambda r: awq.awq_moe_combine(rows, r),
                 lambda r: awq.awq_moe_gather(x, r, r.weights), lambda r: awq.awq_moe_combine(rows, r, r.weights)):
        r = awq.awq_moe_route(logits, 2)
        y = call(r)
        want = torch.autograd.grad(y, [x, rows], torch.ones_like(y), retain_graph=True, allow_unused=True)
        getattr(r, which).zero_()
        with pytest.raises(RuntimeError, match="inplace"):
            y.sum().backward()
        # another list in the routing's place changes nothing
        r = awq.awq_moe_route(logits, 2)
        y = call(r)
        setattr(r, which, torch.zeros_like(getattr(r, which)))
        got = torch.autograd.grad(y, [x, rows], torch.ones_like(y), allow_unused=True)
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, want))


# ---------------------------------------------------------------------------------------------
# scores that 32 bits cannot tell apart
# ---------------------------------------------------------------------------------------------
def near_scores(rng, T, E, k, score, every):
    """fp32 logits and biases: on every `every`-th token experts of one cluster, whose scores lie within some
    2^-26 of each other in random order, stand around the k-th place; the rest are well apart."""
    bias = rng.uniform(2.0 ** -4, 2.0 ** -3, size=E).astype(np.float32)
    b = bias.astype(np.float64)
    middle = 1.5 if score == "softmax" else 0.625
    x = np.empty((T, E), np.float32)
    close = np.arange(T) % every == 1 % every
    for t in range(T):
        order = rng.permutation(E)
        # well apart: their scores 2^-12 and more from each other and from the cluster's
        want = middle + (np.arange(E) - rng.integers(0, E)) * (0.2 / E) + 0.05 / E
        s = np.empty(E)
        s[order] = want
        if close[t]:
            few = min(E, rng.integers(2, 9))
            first = min(max(0, E - k - rng.integers(0, few)), E - few)      # in rising order, around the k-th largest
            s[order[first:first + few]] = middle + 0.2 * (first - E / 2) / E + rng.integers(-8, 9, size=few) * 2.0 ** -28
            low = order[:first]
            s[low] = np.minimum(s[low], middle + 0.2 * (first - E / 2) / E - 2.0 ** -14 * (1 + np.arange(first)[::-1]))
            high = order[first + few:]
            s[high] = np.maximum(s[high], middle + 0.2 * (first - E / 2) / E + 2.0 ** -14 * (1 + np.arange(len(high))))
        v = s - b
        x[t] = v if score == "softmax" else np.log(v / (1 - v))
    return x, bias, close


def fp32_scores(x, bias, score):
    x = x.astype(np.float32)
    return (x if score == "softmax" else np.float32(1) / (np.float32(1) + np.exp(-x))) + bias


@pytest.mark.parametrize("T,E,k,every", [(3, 8, 3, 1), (300, 12, 12, 1), (400, 60, 4, 4), (90, 100, 8, 1), (700, 256, 8, 4),
                                         (130, 300, 32, 2), (100, 1000, 6, 1), (2500, 40, 17, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_near_scores_are_told_apart_in_64_bits(T, E, k, every, score):
    rng = np.random.default_rng(E * 7 + k)
    x, bias, close = near_scores(rng, T, E, k, score, every)
    want = ref.choose(x, k, score, bias)
    # in 32 bits others are chosen, or in another order, on the tokens that are close, and on no more
    off = (ref.choose(fp32_scores(x, bias, score), k) != want).any(1)
    assert off[close].mean() > 0.3 and not off[~close].any()
    r = awq.awq_moe_route(torch.from_numpy(x).cuda(), k, score=score, bias=torch.from_numpy(bias).cuda())
    assert (ints(r.experts) == want).all()
    offsets, order, place = ref.sort_pairs(want, 0, E)
    assert (ints(r.offsets) == offsets).all() and (ints(r.order) == order).all() and (ints(r.place) == place).all()


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalise", [True, False])
def test_gradient_of_a_choice_by_bias(kind, score, normalise):
    """The bias moves the choice; weights and their gradient are those of the logits of what is chosen."""
    rng = np.random.default_rng(17)
    T, E, k = 70, 40, 5
    logits = torch.from_numpy(rng.normal(size=(T, E)).astype(np.float32)).to(TYPES[kind]).cuda().requires_grad_()
    bias = torch.from_numpy((rng.normal(size=E) * 2).astype(np.float32)).cuda()
    g = torch.from_numpy(rng.normal(size=(T, k)).astype(np.float32)).cuda()
    r = awq.awq_moe_route(logits, k, score=score, bias=bias, normalise=normalise, scale=0.7)
    d, = torch.autograd.grad(r.weights, logits, g)
    x, e, gn = wide(logits), ints(r.experts), wide(g)
    assert (e == ref.choose(x, k, score, wide(bias))).all() and (np.sort(e) != np.sort(ref.choose(x, k, score))).any()
    w = ref.route_weights(x, e, score, normalise, 0.7)
    # differences of logits below 12, an exponential, a sum, a quotient, a product
    steps = 2 * (4 + 12) + E / 16 + 8
    assert (np.abs(wide(r.weights) - w) <= steps * 2.0 ** -24 * w).all()
    want = ref.route_grad(x, e, gn, score, normalise, 0.7)
    if score == "softmax" and not normalise:       # p g - p sum p g, over all experts
        p = np.exp(x) / np.exp(x).sum(1, keepdims=True)
        size = 0.7 * p * (np.take_along_axis(p, e, 1) * np.abs(gn)).sum(1, keepdims=True)
    else:
        q = w / 0.7
        p, size = np.ones_like(x), np.zeros_like(x)
        np.put_along_axis(size, e, 0.7 * q * (q * np.abs(gn)).sum(1, keepdims=True), 1)
    here = np.zeros_like(x)
    np.put_along_axis(here, e, 0.7 * np.abs(gn) * w / 0.7, 1)
    bound = (3 * steps + k + 8) * 2.0 ** -24 * (size + here)
    assert (np.abs(wide(d) - want) <= bound + HALF_ULP[kind] * np.abs(want) + TINY[kind]).all()
