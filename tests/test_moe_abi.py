"""What the entry points of a block of experts refuse, before anything is enqueued (CPU): the C calls
get pointers that are never followed; the binding gets CPU tensors."""

import pytest
import torch

import post_weight_quantization_act_amd as awq

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
P = 1 << 20     # an aligned address nothing reads
BIG = 1 << 40


def status(fn, args):
    got = getattr(awq.library(), fn)(*args.values())
    if got != 0:
        assert awq.library().awq_last_error()
    return got


def sort_args(**over):
    a = dict(experts=P, n=4096, first=0, count=8, offsets=P, order=P, place=P, ws=P, size=BIG, stream=None)
    a.update(over)
    return a


LISTS = [
    (dict(offsets=P + 2), UNSUPPORTED), (dict(order=P + 2), UNSUPPORTED), (dict(place=P + 1), UNSUPPORTED),
    (dict(order=None), INVALID), (dict(place=None), INVALID), (dict(first=1 << 31), INVALID),
    (dict(first=-(1 << 31) - 1), INVALID), (dict(count=0), INVALID), (dict(count=-3), INVALID),
    (dict(count=1025), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(size=8), WORKSPACE),
    (dict(ws=P + 2), WORKSPACE),
]


@pytest.mark.parametrize("over,want", LISTS + [
    (dict(n=-1), INVALID), (dict(n=1 << 31), UNSUPPORTED), (dict(experts=None), INVALID),
    (dict(experts=P + 2), UNSUPPORTED), (dict(offsets=None), INVALID),
])
def test_sort_refuses(over, want):
    assert status("awq_moe_sort", sort_args(**over)) == want


def test_sort_workspace():
    size = awq.awq_moe_sort_workspace_size
    assert size(0, 8) == size(1024, 8) == 0
    assert 0 < size(1025, 8) <= size(4096, 8) <= size(1 << 30, 8) <= size(1 << 30, 1024)
    assert size(-1, 8) == size(1 << 31, 8) == size(4096, 0) == size(4096, 1025) == 0


def route_args(**over):
    a = dict(logits=P, dtype=0, T=512, E=16, stride=16, k=8, bias=P, score=0, flags=1, scale=1.0, experts=P,
             weights=P, first=0, count=8, offsets=P, order=P, place=P, ws=P, size=BIG, stream=None)
    a.update(over)
    return a


SCORES = [
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(T=-1), INVALID), (dict(E=0), INVALID),
    (dict(E=1025), UNSUPPORTED), (dict(k=0), INVALID), (dict(k=-2), INVALID), (dict(k=17), INVALID),
    (dict(k=33, E=64), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED), (dict(T=1 << 62), UNSUPPORTED),
    (dict(stride=-1), INVALID), (dict(score=2), INVALID), (dict(score=-1), INVALID), (dict(flags=2), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=1e39), INVALID),
    (dict(logits=None), INVALID), (dict(logits=P + 2), UNSUPPORTED), (dict(logits=P + 1, dtype=1), UNSUPPORTED),
    (dict(experts=None), INVALID), (dict(experts=P + 2), UNSUPPORTED),
]


@pytest.mark.parametrize("over,want", LISTS + SCORES + [
    (dict(weights=None), INVALID), (dict(weights=P + 2), UNSUPPORTED), (dict(bias=P + 2), UNSUPPORTED),
    (dict(T=0, offsets=None), 0),
])
def test_route_refuses(over, want):
    assert status("awq_moe_route", route_args(**over)) == want


def route_grad_args(**over):
    a = dict(logits=P, dtype=0, T=512, E=16, stride=16, k=8, score=0, flags=1, scale=1.0, experts=P, dw=P, dl=P,
             stream=None)
    a.update(over)
    return a


@pytest.mark.parametrize("over,want", SCORES + [
    (dict(dw=None), INVALID), (dict(dl=None), INVALID), (dict(dw=P + 2), UNSUPPORTED), (dict(dl=P + 2), UNSUPPORTED),
    (dict(T=0), 0),
])
def test_route_grad_refuses(over, want):
    assert status("awq_moe_route_grad", route_grad_args(**over)) == want


def gather_args(**over):
    a = dict(x=P, dtype=1, T=5, C=64, stride=64, k=2, count=4, offsets=P, place=P, weights=P, out=P, stream=None)
    a.update(over)
    return a


def combine_args(**over):
    a = dict(rows=P, dtype=1, T=5, C=64, k=2, count=4, offsets=P, place=P, weights=P, residual=P, stride=64, out=P,
             out_dtype=2, stream=None)
    a.update(over)
    return a


def combine_grad_args(**over):
    a = dict(dy=P, dy_dtype=0, T=5, C=64, stride=64, k=2, count=4, offsets=P, place=P, weights=P, rows=P, dtype=1,
             drows=P, dw=P, stream=None)
    a.update(over)
    return a


ROWS = [
    (dict(dtype=5), INVALID), (dict(T=-1), INVALID), (dict(C=0), INVALID), (dict(C=-8), INVALID),
    (dict(C=(1 << 31) - 1), UNSUPPORTED), (dict(k=0), INVALID), (dict(k=33), UNSUPPORTED), (dict(count=0), INVALID),
    (dict(count=1025), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED), (dict(stride=-1), INVALID),
    (dict(offsets=None), INVALID), (dict(place=None), INVALID), (dict(offsets=P + 2), UNSUPPORTED),
    (dict(place=P + 2), UNSUPPORTED), (dict(weights=P + 2), UNSUPPORTED), (dict(T=0), 0),
]


@pytest.mark.parametrize("over,want", ROWS + [
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(x=P + 1), UNSUPPORTED), (dict(out=P + 1), UNSUPPORTED),
])
def test_gather_refuses(over, want):
    assert status("awq_moe_gather", gather_args(**over)) == want


@pytest.mark.parametrize("over,want", ROWS + [
    (dict(rows=None), INVALID), (dict(out=None), INVALID), (dict(rows=P + 1), UNSUPPORTED), (dict(out=P + 1), UNSUPPORTED),
    (dict(residual=P + 1), UNSUPPORTED), (dict(out_dtype=-7), INVALID), (dict(out=P + 2, out_dtype=0), UNSUPPORTED),
])
def test_combine_refuses(over, want):
    assert status("awq_moe_combine", combine_args(**over)) == want


@pytest.mark.parametrize("over,want", ROWS + [
    (dict(dy=None), INVALID), (dict(rows=None), INVALID), (dict(dy=P + 2), UNSUPPORTED), (dict(rows=P + 1), UNSUPPORTED),
    (dict(drows=P + 1), UNSUPPORTED), (dict(dw=P + 2), UNSUPPORTED), (dict(dy_dtype=3), INVALID),
    (dict(drows=None, dw=None), 0),
])
def test_combine_grad_refuses(over, want):
    assert status("awq_moe_combine_grad", combine_grad_args(**over)) == want


def linear_args(**over):
    a = dict(x=P, dtype=1, x_rows=6, K=256, stride=256, codes=P, meta=P, N=64, experts=4, bits=4, group=64, bias=P, act=2,
             flags=1, offsets=P, order=P, per_token=2, rows=12, residual=P, rstride=32, out=P, out_dtype=2, ws=P,
             size=BIG, stream=None)
    a.update(over)
    return a


@pytest.mark.parametrize("over,want", [
    (dict(dtype=9), INVALID), (dict(out_dtype=-1), INVALID), (dict(dtype=0), UNSUPPORTED), (dict(N=0), INVALID),
    (dict(K=0), INVALID), (dict(experts=0), INVALID), (dict(x_rows=-1), INVALID), (dict(rows=-1), INVALID),
    (dict(bits=1), UNSUPPORTED), (dict(bits=9), UNSUPPORTED), (dict(group=16), UNSUPPORTED), (dict(group=96), UNSUPPORTED),
    (dict(group=1024), UNSUPPORTED), (dict(K=288), INVALID), (dict(act=-1), INVALID), (dict(act=5), INVALID),
    (dict(flags=2), INVALID), (dict(N=63), INVALID), (dict(stride=-8), UNSUPPORTED), (dict(stride=257), UNSUPPORTED),
    (dict(rstride=-1), INVALID), (dict(offsets=None), INVALID), (dict(offsets=None, order=None, experts=1), INVALID),
    (dict(offsets=None, experts=1, x_rows=12), INVALID), (dict(per_token=0), INVALID), (dict(order=None), INVALID),
    (dict(experts=1025), UNSUPPORTED), (dict(N=1 << 30), UNSUPPORTED), (dict(rows=1 << 30), UNSUPPORTED),
    (dict(x_rows=1 << 31), UNSUPPORTED), (dict(K=1 << 30), UNSUPPORTED), (dict(rows=0), 0), (dict(x_rows=0), INVALID),
    (dict(N=1 << 20, K=8192), UNSUPPORTED), (dict(N=1 << 23, bits=8), UNSUPPORTED),
    (dict(x_rows=1 << 24, stride=256), UNSUPPORTED), (dict(stride=1 << 31), UNSUPPORTED), (dict(stride=1 << 60), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(meta=None), INVALID), (dict(out=None), INVALID),
    (dict(x=P + 8), UNSUPPORTED), (dict(codes=P + 2), UNSUPPORTED), (dict(meta=P + 4), UNSUPPORTED),
    (dict(bias=P + 2), UNSUPPORTED), (dict(offsets=P + 2), UNSUPPORTED), (dict(order=P + 2), UNSUPPORTED),
    (dict(out=P + 1), UNSUPPORTED), (dict(out=P + 2, out_dtype=0), UNSUPPORTED), (dict(residual=P + 1), UNSUPPORTED),
    # a grid of more than 2^32 threads
    (dict(offsets=None, order=None, experts=1, x_rows=1 << 25, rows=1 << 25, K=32, stride=32, group=32, N=1 << 20),
     UNSUPPORTED),
])
def test_linear_refuses(over, want):
    assert status("awq_lowbit_linear", linear_args(**over)) == want


def test_linear_workspace_of_what_is_refused():
    size = awq.library().awq_lowbit_linear_workspace_size
    good = dict(dtype=2, rows=4096, x_rows=4096, N=4096, K=4096, experts=1, flags=0)
    for over in (dict(dtype=7), dict(rows=0), dict(rows=-1), dict(x_rows=0), dict(N=0), dict(K=0), dict(experts=0),
                 dict(rows=1 << 31), dict(x_rows=1 << 31), dict(N=1 << 31), dict(experts=1025)):
        assert size(*{**good, **over}.values()) == 0


def test_binding_refuses_cpu_tensors_and_wrong_names():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        awq.awq_moe_route(x, 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        awq.awq_moe_sort(torch.zeros(4, 2, dtype=torch.int32), 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        awq.Routing(None, None, torch.zeros(9, dtype=torch.int32), torch.zeros(8, dtype=torch.int32),
                    torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(TypeError, match="Routing"):
        awq.awq_moe_gather(x, None)
    with pytest.raises(TypeError, match="Routing"):
        awq.awq_moe_combine(x, (1, 2))
    with pytest.raises(ValueError, match="GPU tensor"):
        awq.awq_lowbit_linear(x, x, x, 4, 32)
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        awq.awq_moe_route([[1.0]], 1)
