"""The router, tokens sorted by expert and back, and their gradients on the GPU against the 64-bit oracle."""

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


def normal(rng, shape, kind):
    return torch.from_numpy(rng.normal(size=shape).astype(np.float32)).to(TYPES[kind]).cuda()


def check_lists(r, experts, first, count):
    offsets, order, place = ref.sort_pairs(experts, first, count)
    assert (ints(r.offsets) == offsets).all() and (ints(r.order) == order).all() and (ints(r.place) == place).all()


# ---------------------------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------------------------
ROUTES = [   # T, E, k, kind, score, normalise, bias, stride
    (1, 128, 8, "bf16", "softmax", True, False, 0), (1, 1, 1, "f32", "softmax", False, False, 0),
    (3, 8, 8, "f16", "sigmoid", True, True, 0), (17, 16, 2, "f32", "sigmoid", False, True, 5),
    (33, 60, 4, "bf16", "softmax", False, True, 0), (64, 64, 16, "f16", "softmax", True, False, 3),
    (65, 65, 17, "f32", "softmax", True, True, 0), (130, 256, 32, "f32", "softmax", False, False, 0),
    (257, 257, 6, "bf16", "sigmoid", True, True, 0), (129, 512, 8, "f16", "sigmoid", True, False, 1),
    (40, 1000, 10, "bf16", "softmax", True, True, 0), (31, 1024, 32, "f32", "sigmoid", False, True, 0),
    (2050, 40, 3, "bf16", "softmax", True, False, 0), (1025, 15, 1, "f32", "softmax", True, False, 0),
]


@pytest.mark.parametrize("T,E,k,kind,score,normalise,biased,pad", ROUTES)
def test_route(T, E, k, kind, score, normalise, biased, pad):
    rng = np.random.default_rng(T * 1000 + E)
    logits = normal(rng, (T, E + pad), kind)[:, :E]            # with pad: rows apart
    bias = normal(rng, (E,), "f32") * 0.3 if biased else None
    r = awq.awq_moe_route(logits, k, score=score, bias=bias, normalise=normalise, scale=1.5)
    x = wide(logits)
    want = ref.choose(x, k, score, None if bias is None else wide(bias))
    assert (ints(r.experts) == want).all()
    w = ref.route_weights(x, want, score, normalise, 1.5)
    # a difference of logits, its exponential (2 ulp and the argument's rounding: |l - max| below 12), the sum
    # over up to E (each term's error, and E additions by 16 lanes: E / 16 + 4), quotient and product
    assert (np.abs(wide(r.weights) - w) <= (2 * (4 + 12) + E / 16 + 8) * 2.0 ** -24 * w).all()
    check_lists(r, want, 0, E)


def test_route_ties_take_the_lowest_number():
    logits = torch.zeros(70, 33, device="cuda")
    logits[:, 7] = logits[:, 20] = 1.0
    logits[::2, 3] = -0.0
    r = awq.awq_moe_route(logits, 5)
    assert (ints(r.experts) == [7, 20, 0, 1, 2]).all()
    r = awq.awq_moe_route(logits, 5, score="sigmoid", bias=torch.zeros(33, device="cuda"))
    assert (ints(r.experts) == [7, 20, 0, 1, 2]).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_masked_and_invalid_logits(score, biased):
    inf, nan = float("inf"), float("nan")
    logits = torch.tensor([[1.0, -inf, -inf, -inf], [-inf] * 4, [nan, 2.0, 1.0, nan], [nan] * 4,
                           [torch.finfo(torch.float32).min] * 4, [200.0, -200.0, 100.0, 0.0]], device="cuda")
    bias = torch.zeros(4, device="cuda") if biased else None
    r = awq.awq_moe_route(logits, 2, score=score, bias=bias)
    want = ref.choose(wide(logits), 2, score, [0.0] * 4 if biased else None)
    if score == "sigmoid" and biased:
        want[5] = [0, 2]       # both sigmoids are 1 in 64 bits: equals, as the definition has it
    assert (ints(r.experts) == want).all()
    w = wide(r.weights)
    assert w[0].tolist() == [1, 0]                  # one expert is left: it has all the weight
    assert w[1].tolist() == [0, 0]                  # none is
    if score == "softmax":
        assert w[4].tolist() == [0.5, 0.5]
        assert w[5, 0] == 1 and 0 <= w[5, 1] < 2.0 ** -143      # exp(-100) = 2^-144.3
    else:
        assert w[4].tolist() == [0, 0]
        assert w[5].tolist() == [0.5, 0.5]
    assert np.isnan(w[3]).all() and (ints(r.experts)[3] == [0, 1]).all()
    check_lists(r, want, 0, 4)


@pytest.mark.parametrize("T", [0, 7, 700])
def test_route_of_a_share_of_the_experts(T):
    rng = np.random.default_rng(T)
    logits = normal(rng, (T, 24), "f32")
    r = awq.awq_moe_route(logits, 4, num_experts=9, first_expert=8)
    want = ref.choose(wide(logits), 4)
    assert (ints(r.experts) == want).all() and r.count == 9
    check_lists(r, want, 8, 9)


@pytest.mark.parametrize("T,E,k,kind,score,normalise,biased,pad", ROUTES)
def test_route_gradient(T, E, k, kind, score, normalise, biased, pad):
    rng = np.random.default_rng(T * 77 + E)
    logits = normal(rng, (T, E + pad), kind)[:, :E].requires_grad_()
    g = normal(rng, (T, k), "f32")
    r = awq.awq_moe_route(logits, k, score=score, normalise=normalise, scale=0.7)
    assert r.weights.requires_grad and not r.place.requires_grad
    d, = torch.autograd.grad(r.weights, logits, g)
    assert d.dtype is TYPES[kind] and d.shape == logits.shape
    x, e = wide(logits), ints(r.experts)
    want = ref.route_grad(x, e, wide(g), score, normalise, 0.7)
    # each term p g and p sum g p: as the weights' bound above, k + E / 16 more additions in the sum
    most = 0.7 * np.abs(wide(g)).max(1, keepdims=True)
    w = np.maximum(ref.route_weights(x, e, score, normalise).max(1, keepdims=True), 2.0 ** -30)
    bound = 3 * (2 * (4 + 12) + E / 16 + k + 16) * 2.0 ** -24 * most * w * np.maximum(1, k * w)
    assert (np.abs(wide(d) - want) <= bound + HALF_ULP[kind] * np.abs(want) + TINY[kind]).all()


def test_route_gradient_of_masked_rows_is_finite():
    inf = float("inf")
    logits = torch.tensor([[1.0, -inf, 0.5, -inf], [-inf] * 4], device="cuda").requires_grad_()
    for score in ("softmax", "sigmoid"):
        for normalise in (True, False):
            r = awq.awq_moe_route(logits, 3, score=score, normalise=normalise)
            d, = torch.autograd.grad(r.weights, logits, torch.ones_like(r.weights) * torch.arange(3, device="cuda"))
            assert torch.isfinite(d).all() and (d[1] == 0).all() and (d[0, 1] == 0).all() and (d[0, 3] == 0).all()


# ---------------------------------------------------------------------------------------------
# sorting
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("T,k,E", [(0, 2, 8), (1, 1, 1), (5, 3, 4), (64, 16, 7), (1024, 1, 1024), (1025, 1, 1024),
                                   (513, 2, 3), (5000, 3, 130), (40001, 8, 255), (300, 32, 64)])
@pytest.mark.parametrize("kind", ["spread", "one", "outside", "share"])
def test_sort(T, k, E, kind):
    rng = np.random.default_rng(T + E)
    first = 0
    if kind == "spread":
        e = rng.integers(0, E, size=(T, k))
    elif kind == "one":
        e = np.full((T, k), E - 1)
    elif kind == "outside":       # any number may stand there
        e = rng.choice([-1, E, E + 1, 2 ** 31 - 1, -2 ** 31, 0], size=(T, k))
    else:
        first = 3
        e = rng.integers(0, 2 * E + 3, size=(T, k))
    r = awq.awq_moe_sort(torch.from_numpy(e.astype(np.int32)).cuda(), E, first_expert=first)
    # the oracle's loop, vectorised: a stable sort by bucket
    b = np.where((e >= first) & (e < first + E), e - first, E).ravel()
    order = np.argsort(b, kind="stable")
    place = np.empty_like(order)
    place[order] = np.arange(order.size)
    assert (ints(r.order) == order).all() and (ints(r.place).ravel() == place).all()
    assert (ints(r.offsets) == np.searchsorted(b[order], np.arange(E + 1))).all()
    if T * k < 600:
        check_lists(r, e, first, E)


# ---------------------------------------------------------------------------------------------
# rows there and back
# ---------------------------------------------------------------------------------------------
def routed(rng, T, k, of, count, first=0):
    e = np.stack([rng.permutation(of)[:k] for _ in range(T)]) if T else np.zeros((0, k))
    r = awq.awq_moe_sort(torch.from_numpy(e.astype(np.int32)).cuda(), count, first_expert=first,
                         weights=torch.from_numpy(rng.normal(size=(T, k)).astype(np.float32)).cuda())
    return r, ref.sort_pairs(e, first, count)


SHAPES = [   # T, k, of, count, C, kind, pad
    (1, 1, 1, 1, 1, "f32", 0), (1, 8, 16, 16, 64, "bf16", 0), (5, 2, 8, 3, 7, "f16", 0), (33, 3, 9, 9, 129, "bf16", 3),
    (7, 9, 12, 6, 2048, "f16", 0), (3, 17, 40, 20, 2056, "f32", 8), (2, 4, 4, 2, 5001, "bf16", 1), (130, 6, 64, 64, 40, "f32", 0),
    (257, 2, 5, 1, 24, "bf16", 0), (9, 32, 33, 30, 255, "f16", 1), (0, 2, 4, 4, 16, "f32", 0), (4, 3, 8, 8, 513, "f32", 0),
]


@pytest.mark.parametrize("T,k,of,count,C,kind,pad", SHAPES)
@pytest.mark.parametrize("weighted", [False, True])
def test_gather(T, k, of, count, C, kind, pad, weighted):
    rng = np.random.default_rng(C + T)
    r, (offsets, _, place) = routed(rng, T, k, of, count)
    x = normal(rng, (T, C + pad), kind)[:, :C]
    out = awq.awq_moe_gather(x, r, r.weights if weighted else None)
    want = ref.gather(wide(x), offsets, place, wide(r.weights) if weighted else None)
    # one product in fp32, rounded once more to 16 bits
    slack = (2.0 ** -24 + HALF_ULP[kind]) * np.abs(want) + TINY[kind] if weighted else 0
    assert out.shape == (T * k, C) and (np.abs(wide(out) - want) <= slack).all()


@pytest.mark.parametrize("T,k,of,count,C,kind,pad", SHAPES)
@pytest.mark.parametrize("weighted,residual,out", [(False, False, None), (True, True, None), (True, True, "f32"), (True, False, "bf16")])
def test_combine(T, k, of, count, C, kind, pad, weighted, residual, out):
    rng = np.random.default_rng(C + T)
    r, (offsets, _, place) = routed(rng, T, k, of, count)
    rows = normal(rng, (T * k, C), kind)
    rows[offsets[-1]:] = float("nan")                # rows that nobody has are not read
    out = out or kind
    res = normal(rng, (T, C + pad), out)[:, :C] if residual else None
    w = r.weights if weighted else None
    y = awq.awq_moe_combine(rows, r, w, residual=res, out_dtype=TYPES[out])
    x, w = wide(rows), np.ones((T, k)) if w is None else wide(w)
    want = ref.combine(x, offsets, place, w, None if res is None else wide(res))
    size = ref.combine(np.abs(x), offsets, place, np.abs(w), None if res is None else np.abs(wide(res)))
    # k multiply-adds in fp32, one rounding
    assert (np.abs(wide(y) - want) <= (k + 1) * 2.0 ** -24 * size + HALF_ULP[out] * np.abs(want) + TINY[out]).all()


@pytest.mark.parametrize("T,k,of,count,C,kind,pad", [s for s in SHAPES if s[0]])
@pytest.mark.parametrize("weighted", [False, True])
def test_gradients(T, k, of, count, C, kind, pad, weighted):
    rng = np.random.default_rng(C * 3 + T)
    r, (offsets, _, place) = routed(rng, T, k, of, count)
    w = r.weights.requires_grad_() if weighted else None
    wn = wide(r.weights) if weighted else np.ones((T, k))
    here = place < offsets[-1]

    x = normal(rng, (T, C + pad), kind)[:, :C].requires_grad_()
    g = normal(rng, (T * k, C), kind)
    got = torch.autograd.grad(awq.awq_moe_gather(x, r, w), [x, w] if weighted else [x], g)
    gn, xn = wide(g), wide(x)
    want, size = ref.combine(gn, offsets, place, wn), ref.combine(np.abs(gn), offsets, place, np.abs(wn))
    assert got[0].dtype is x.dtype
    assert (np.abs(wide(got[0]) - want) <= (k + 1) * 2.0 ** -24 * size + HALF_ULP[kind] * np.abs(want) + TINY[kind]).all()
    # C products: a thread adds up to C / 256 + 8 of them, 64 lanes and four waves ten more
    adds = C / 256 + 20
    if weighted:
        want, size = ref.dots(xn, gn, offsets, place), ref.dots(np.abs(xn), np.abs(gn), offsets, place)
        assert (np.abs(wide(got[1]) - want) <= adds * 2.0 ** -24 * size).all()
        assert (wide(got[1])[~here] == 0).all()

    rows = normal(rng, (T * k, C), kind)
    rows[offsets[-1]:] = float("nan")
    rows.requires_grad_()
    res = normal(rng, (T, C), kind).requires_grad_()
    dy = normal(rng, (T, C), kind)
    leaves = [rows, res, w] if weighted else [rows, res]
    got = torch.autograd.grad(awq.awq_moe_combine(rows, r, w, residual=res), leaves, dy)
    dn = wide(dy)
    want = ref.gather(dn, offsets, place, wn)
    assert (np.abs(wide(got[0]) - want) <= (2.0 ** -24 + HALF_ULP[kind]) * np.abs(want) + TINY[kind]).all()
    assert torch.equal(got[1], dy)
    if weighted:
        rn = np.nan_to_num(wide(rows))
        want, size = ref.dots(dn, rn, offsets, place), ref.dots(np.abs(dn), np.abs(rn), offsets, place)
        assert (np.abs(wide(got[2]) - want) <= adds * 2.0 ** -24 * size).all()
        assert (wide(got[2])[~here] == 0).all()


def test_gradient_of_a_wider_output_and_of_a_sum():
    """bf16 rows into an fp32 result: its gradient is taken as it is; a sum's, whose strides are 0."""
    rng = np.random.default_rng(8)
    r, (offsets, _, place) = routed(rng, 6, 2, 4, 4)
    rows = normal(rng, (12, 48), "bf16").requires_grad_()
    w = r.weights.requires_grad_()
    g = normal(rng, (6, 48), "f32")
    d, dw = torch.autograd.grad(awq.awq_moe_combine(rows, r, w, out_dtype=torch.float32), [rows, w], g)
    want = ref.gather(wide(g), offsets, place, wide(w))
    assert d.dtype is torch.bfloat16
    assert (np.abs(wide(d) - want) <= (2.0 ** -24 + HALF_ULP["bf16"]) * np.abs(want) + TINY["bf16"]).all()
    size = ref.dots(np.abs(wide(g)), np.abs(wide(rows)), offsets, place)
    assert (np.abs(wide(dw) - ref.dots(wide(g), wide(rows), offsets, place)) <= 21 * 2.0 ** -24 * size).all()
    x = normal(rng, (6, 48), "f32").requires_grad_()
    awq.awq_moe_gather(x, r).sum().backward()
    assert (wide(x.grad) == 2).all()
    rows.grad = None
    awq.awq_moe_combine(rows, r).sum().backward()
    assert (wide(rows.grad) == 1).all()


def test_more_than_two_to_the_31_elements():
    """There and back: eight times each row, exactly, and the same for the gradients."""
    T, k, C = 131081, 8, 2056
    gen = torch.Generator(device="cuda").manual_seed(1)
    e = torch.rand((T, 16), generator=gen, device="cuda").topk(k).indices.int()
    x = torch.randn((T, C), generator=gen, device="cuda").bfloat16()
    r = awq.awq_moe_sort(e, 16)
    rows = awq.awq_moe_gather(x, r)
    y = awq.awq_moe_combine(rows, r)
    assert torch.equal(y, x * 8)
    drows, dweights = awq.awq_moe_combine_grad(y, r, rows=rows)
    at = torch.tensor([0, 70000, T - 1], device="cuda")
    assert torch.equal(drows[r.place[at].long()], y[at][:, None].expand(3, k, C))
    want = (y[at].double() * x[at].double()).sum(-1)
    # C products, exact in 48 bits, rounded to fp32 and added: C additions at most
    assert ((dweights[at].double() - want[:, None]).abs() <= 1.01 * (C + 1) * 2.0 ** -24 * want[:, None]).all()


def test_shared_residual_row_and_out():
    rng = np.random.default_rng(1)
    r, (offsets, _, place) = routed(rng, 5, 2, 6, 6)
    rows, one = normal(rng, (10, 32), "f32"), normal(rng, (1, 32), "f32").requires_grad_()
    y = awq.awq_moe_combine(rows, r, residual=one.expand(5, 32))
    want = ref.combine(wide(rows), offsets, place, None, np.repeat(wide(one), 5, 0))
    assert np.abs(wide(y) - want).max() <= 3 * 2.0 ** -24 * (np.abs(wide(rows)).max() * 2 + np.abs(wide(one)).max())
    y.sum().backward()
    assert (wide(one.grad) == 5).all()
    out = torch.empty_like(y)
    assert awq.awq_moe_combine(rows, r, residual=one.expand(5, 32), out=out) is out and torch.equal(out, y.detach())
    g = torch.empty(10, 32, device="cuda")
    x = normal(rng, (5, 32), "f32")
    assert awq.awq_moe_gather(x, r, out=g) is g and torch.equal(g, awq.awq_moe_gather(x, r))


def test_second_gradients_are_refused():
    rng = np.random.default_rng(2)
    r, _ = routed(rng, 3, 2, 4, 4)
    x = normal(rng, (3, 8), "f32").requires_grad_()
    d, = torch.autograd.grad(awq.awq_moe_gather(x, r).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        d.sum().backward()


def test_lists_that_lie_outside_write_and_read_nothing():
    """place past the rows or below 0 is passed over; the offsets' end past them counts as the rows' end."""
    place = torch.tensor([[0, 99], [-5, 1]], dtype=torch.int32, device="cuda")
    order = torch.zeros(4, dtype=torch.int32, device="cuda")
    r = awq.Routing(None, None, torch.tensor([0, 77], dtype=torch.int32, device="cuda"), order, place)
    x = torch.arange(6.0, device="cuda").view(2, 3)
    out = awq.awq_moe_gather(x, r, out=torch.full((4, 3), -1.0, device="cuda"))
    assert out.tolist() == [[0, 1, 2], [3, 4, 5], [-1] * 3, [-1] * 3]
    y = awq.awq_moe_combine(torch.ones(4, 3, device="cuda"), r)
    assert y.tolist() == [[1] * 3, [1] * 3]
    _, dw = awq.awq_moe_combine_grad(x, r, rows=torch.ones(4, 3, device="cuda"), need_rows=False)
    assert dw.tolist() == [[3, 0], [0, 12]]


def test_binding_refuses():
    rng = np.random.default_rng(3)
    r, _ = routed(rng, 4, 2, 4, 4)
    x = normal(rng, (4, 16), "f32")
    for call in (lambda: awq.awq_moe_route(x, 17), lambda: awq.awq_moe_route(x, 0), lambda: awq.awq_moe_route(x, -1),
                 lambda: awq.awq_moe_route(x, 2, score="tanh"), lambda: awq.awq_moe_route(x.T, 2),
                 lambda: awq.awq_moe_route(x, 2, bias=x[0].half()), lambda: awq.awq_moe_route(x, 2, num_experts=0),
                 lambda: awq.awq_moe_gather(x[:3], r), lambda: awq.awq_moe_gather(x.T, r),
                 lambda: awq.awq_moe_gather(x, r, r.weights[:2]), lambda: awq.awq_moe_combine(x, r),
                 lambda: awq.awq_moe_combine(normal(rng, (8, 16), "f32"), r, residual=x.half()),
                 lambda: awq.awq_moe_combine_grad(x, r), lambda: awq.awq_moe_sort(x, 4),
                 lambda: awq.Routing(None, None, r.offsets, r.order[:3], r.place),
                 lambda: awq.awq_moe_route_grad(x, r.experts, r.weights[:2])):
        with pytest.raises((ValueError, awq.AwqError)):
            call()
    with pytest.raises(TypeError):
        awq.awq_moe_route(x.double(), 2)


# ---------------------------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------------------------
def test_on_another_stream():
    rng = np.random.default_rng(5)
    logits, x = normal(rng, (900, 32), "f32"), normal(rng, (900, 128), "bf16")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        r = awq.awq_moe_route(logits, 4)
        y = awq.awq_moe_combine(awq.awq_moe_gather(x, r), r, r.weights)
    side.synchronize()
    check_lists(r, ref.choose(wide(logits), 4), 0, 32)
    # the weights of a token add up to 1: four products and sums, and the roundings
    assert (np.abs(wide(y) - wide(x)) <= (HALF_ULP["bf16"] + 16 * 2.0 ** -24) * np.abs(wide(x)) + TINY["bf16"]).all()


@pytest.mark.parametrize("T", [4, 700])
def test_captured_and_replayed(T):
    rng = np.random.default_rng(6)
    logits, x = normal(rng, (T, 24), "f32"), normal(rng, (T, 96), "f16")

    def step():
        r = awq.awq_moe_route(logits, 3, num_experts=20)
        rows = awq.awq_moe_gather(x, r)
        return r.offsets, r.order, r.place, r.weights, awq.awq_moe_combine(rows, r, r.weights, residual=x)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        logits.copy_(normal(rng, (T, 24), "f32"))
        x.copy_(normal(rng, (T, 96), "f16"))
        graph.replay()
        kept = [g.clone() for g in got]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want)), i


def test_backward_captured_and_replayed():
    """Gradients through the router's weights and the rows, in a graph of their own leaves."""
    rng = np.random.default_rng(7)
    logits, x, dy = normal(rng, (300, 16), "f32"), normal(rng, (300, 64), "f32"), normal(rng, (300, 64), "f32")

    def step():
        a, b = logits.detach().requires_grad_(), x.detach().requires_grad_()
        r = awq.awq_moe_route(a, 2)
        y = awq.awq_moe_combine(awq.awq_moe_gather(b, r) * 2, r, r.weights)
        return torch.autograd.grad(y, [a, b], dy)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        for t in (logits, x, dy):
            t.copy_(normal(rng, t.shape, "f32"))
        graph.replay()
        kept = [g.clone() for g in got]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want)), i


def test_same_results_every_time():
    rng = np.random.default_rng(11)
    logits, x = normal(rng, (3001, 64), "bf16"), normal(rng, (3001, 72), "f32")
    first = None
    for _ in range(3):
        r = awq.awq_moe_route(logits, 6)
        got = (r.order, r.place, r.weights, awq.awq_moe_combine(awq.awq_moe_gather(x, r), r, r.weights),
               awq.awq_moe_combine_grad(x, r, r.weights, awq.awq_moe_gather(x, r))[1])
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
