"""The packed product at the ends of its range on the GPU, against the 64-bit oracle."""

import numpy as np
import pytest
import torch

import post_weight_quantization_act_amd as awq
from oracle import moe_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    awq.library()
    yield
    torch.cuda.synchronize()


def wide(t):
    return t.detach().double().cpu().numpy()


def packed(codes, steps, zeros, bits):
    words, meta = ref.repack(codes, steps, zeros, bits)
    return torch.from_numpy(words.view(np.int32)).cuda(), torch.from_numpy(meta).cuda()


def summed(x, W, group):
    """What sums in fp32 may be off: K exact products, K additions at most, two roundings a group, eight waves'."""
    K = x.shape[1]
    return 1.02 * (K + 2 * K / group + 14) * 2.0 ** -24 * (np.abs(x) @ np.abs(W).T)


# ---------------------------------------------------------------------------------------------
# rows with elements far apart
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("routed", [False, True])
@pytest.mark.parametrize("far", [12, 20, 28])
def test_an_outlier_leaves_the_others_their_bits(routed, far):
    """bf16 rows of a large call whose largest element lies 2^far above the rest and meets weights of 0: what is
    left are the others' products, each of which has all its bits down to 2^-32 of the largest, and is
    within 2^-40 of it below."""
    rng = np.random.default_rng(far)
    rows, n, K, bits, group = 1100, 8100, 128, 4, 64
    x = rng.normal(size=(rows, K))
    x[:, 37] = 2.0 ** far * (1 + rng.random(rows))
    x = torch.from_numpy(x.astype(np.float32)).bfloat16().cuda()
    codes = rng.integers(0, 16, size=(n, K)).astype(np.uint8)
    zeros = rng.integers(0, 16, size=(n, K // group))
    codes[:, 37] = zeros[:, 0]
    steps = (0.02 * np.exp(0.2 * rng.normal(size=zeros.shape))).astype(np.float32)
    ct, mt = packed(codes, steps, zeros, bits)
    more = {}
    if routed:       # one expert of all rows, each taken from its token
        more = dict(routing=awq.awq_moe_sort(torch.zeros((rows, 1), dtype=torch.int32, device="cuda"), 1), gather=True)
    assert awq.awq_lowbit_linear_workspace_size(torch.bfloat16, rows, rows, n, K) >= rows * K * 2
    y = awq.awq_lowbit_linear(x, ct, mt, bits, group, out_dtype=torch.float32, **more)
    xn, W = wide(x), ref.weights_of(codes, steps, zeros, group)
    off = summed(xn, W, group) + 1.02 * 2.0 ** -40 * np.abs(xn).max(1)[:, None] * np.abs(W).sum(1)[None]
    assert (np.abs(wide(y) - xn @ W.T) <= off).all()


def test_rows_at_the_ends_of_bfloat16():
    """Largest elements from 2^-133 to just below 2^128, exactly where a row has one element alone."""
    rng = np.random.default_rng(1)
    rows, n, K, bits, group = 1024, 8192, 64, 4, 64
    x = np.zeros((rows, K))
    e = np.arange(rows) % 261 - 133
    at = rng.integers(0, K, size=rows)
    x[np.arange(rows), at] = np.ldexp(np.where(e >= -126, 255 / 128, 1.0), np.maximum(e, -133)) * rng.choice([-1, 1], size=rows)
    x = torch.from_numpy(x.astype(np.float32)).bfloat16().cuda()
    xn = wide(x)
    assert np.isfinite(xn).all() and (xn != 0).any(1).all()
    codes = rng.integers(0, 16, size=(n, K)).astype(np.uint8)
    zeros = rng.integers(0, 16, size=(n, 1))
    steps = np.full((n, 1), 2.0 ** -5, np.float32)
    ct, mt = packed(codes, steps, zeros, bits)
    y = wide(awq.awq_lowbit_linear(x, ct, mt, bits, group, out_dtype=torch.float32))
    want = xn @ ref.weights_of(codes, steps, zeros, group).T
    # one product of 8 and 4 bits and a power of two: exact but for fp32's subnormals
    assert (np.abs(y - want) <= np.where(np.abs(want) < 2.0 ** -126, 2.0 ** -149, 0)).all()


# ---------------------------------------------------------------------------------------------
# steps far apart
# ---------------------------------------------------------------------------------------------
FAR = [   # rows, n, K, bits, group, kind, gated, experts
    (8, 60, 512, 4, 32, "bf16", False, 0), (20, 1300, 256, 4, 128, "bf16", False, 0), (40, 300, 4096, 4, 128, "bf16", False, 0),
    (33, 258, 2080, 3, 32, "f16", True, 0), (150, 130, 640, 5, 64, "bf16", True, 0), (500, 70, 1152, 8, 128, "f16", False, 0),
    (1000, 8100, 160, 4, 32, "bf16", False, 0), (1030, 7300, 256, 4, 128, "f16", False, 0), (2500, 800, 128, 2, 32, "bf16", False, 0),
    (130, 130, 384, 4, 128, "bf16", False, 4), (700, 300, 160, 7, 32, "f16", True, 6), (61, 96, 288, 6, 32, "bf16", True, 8),
]


@pytest.mark.parametrize("case", FAR, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("spread,size", [(0, 70), (15, 60), (30, 20), (40, 0), (50, -10)])
def test_steps_far_apart(case, spread, size):
    """Steps up to 2^(2 spread) apart, rows of about 2^size (fp16: 1), up to the limit that the header states: the
    largest step over the smallest, times the sums of |x (c - z)|, within fp32.  One row is not finite and
    stays alone."""
    rows, n, K, bits, group, kind, gated, experts = case
    rng = np.random.default_rng(rows + spread)
    if kind == "f16":
        size = 0
    codes = rng.integers(0, 2 ** bits, size=(max(1, experts) * n, K)).astype(np.uint8)
    zeros = rng.integers(0, 2 ** bits, size=(len(codes), K // group))
    # gated results are squares: about 1
    steps = np.exp2(rng.uniform(-spread, spread, size=zeros.shape) - (size + spread if gated else size / 2)).astype(np.float32)
    steps[rng.random(steps.shape) < 0.05] = 0
    ct, mt = packed(codes, steps, zeros, bits)
    W = ref.weights_of(codes, steps, zeros, group).reshape(max(1, experts), n, K)
    x = torch.from_numpy((rng.normal(size=(rows, K)) * 2.0 ** size).astype(np.float32)).to(TYPES[kind]).cuda()
    bad = min(3, rows - 1)
    x[bad, K // 2] = float("nan")
    more, own = {}, np.zeros(rows, dtype=np.int64)
    if experts:
        r = awq.awq_moe_sort(torch.from_numpy(rng.integers(0, experts, size=(rows, 1)).astype(np.int32)).cuda(), experts)
        more, order = dict(routing=r, gather=True), r.order.cpu().numpy()
        own = np.searchsorted(r.offsets.cpu().numpy(), np.arange(rows), side="right") - 1
    else:
        order = np.arange(rows)
    y = wide(awq.awq_lowbit_linear(x, ct, mt, bits, group, gated=gated, out_dtype=torch.float32, **more))
    xn = np.nan_to_num(wide(x))[order]
    v, dv = np.empty((rows, n)), np.empty((rows, n))
    for e in range(max(1, experts)):
        v[own == e], dv[own == e] = xn[own == e] @ W[e].T, summed(xn[own == e], W[e], group)
    if gated:
        g, u, dg, du = v[:, :n // 2], v[:, n // 2:], dv[:, :n // 2], dv[:, n // 2:]
        want, off = g * u, np.abs(g) * du + np.abs(u) * dg + dg * du
    else:
        want, off = v, dv
    off = off + 2.0 ** -23 * (np.abs(want) + off) + 2.0 ** -149
    assert np.abs(want).max() < 2.0 ** 126
    ratio = max((row[row > 0].max() / row[row > 0].min() for row in steps.astype(np.float64) if row.any()), default=1)
    assert ratio * K * 2 ** bits * np.abs(xn).max() < 2.0 ** 127
    keep = order != bad
    assert not np.isfinite(y[~keep]).any() and np.isfinite(y[keep]).all()
    assert (np.abs(y - want)[keep] <= off[keep]).all()


# ---------------------------------------------------------------------------------------------
# one workspace for all batches
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_the_largest_batchs_workspace_serves_smaller_ones(kind):
    rng = np.random.default_rng(12)
    n, K, bits, group, most = 4200, 2048, 4, 128, 2300
    codes, zeros = rng.integers(0, 16, size=(n, K)).astype(np.uint8), rng.integers(0, 16, size=(n, K // group))
    ct, mt = packed(codes, (0.01 * np.exp(0.2 * rng.normal(size=zeros.shape))).astype(np.float32), zeros, bits)
    bytes_ = awq.awq_lowbit_linear_workspace_size(TYPES[kind], most, most, n, K)
    space = torch.full((bytes_ + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    x = torch.from_numpy(rng.normal(size=(most, K)).astype(np.float32)).to(TYPES[kind]).cuda()
    for rows in (most, 900, 512, 300, 256, 130, 64, 33, 17, 1):
        y = awq.awq_lowbit_linear(x[:rows], ct, mt, bits, group, workspace=space[:bytes_])
        assert torch.equal(y, awq.awq_lowbit_linear(x[:rows], ct, mt, bits, group)), rows
    assert (space[bytes_:] == 0xA5).all()


def small_call():
    rng = np.random.default_rng(3)
    codes, zeros = rng.integers(0, 16, size=(24, 64)).astype(np.uint8), rng.integers(0, 16, size=(24, 2))
    ct, mt = packed(codes, np.full((24, 2), 0.1, np.float32), zeros, 4)
    x = torch.from_numpy(rng.normal(size=(5, 64)).astype(np.float32)).half().cuda()
    return x, ct, mt, dict(bias=torch.zeros(1, 24, device="cuda"), residual=torch.zeros(5, 24, device="cuda").half())


def test_any_input_that_requires_a_gradient_is_refused():
    x, ct, mt, more = small_call()
    awq.awq_lowbit_linear(x, ct, mt, 4, 32, **more)
    for t in (x, mt, more["bias"], more["residual"]):
        t.requires_grad_()
        with pytest.raises(RuntimeError, match="no gradient"):
            awq.awq_lowbit_linear(x, ct, mt, 4, 32, **more)
        with torch.no_grad():
            awq.awq_lowbit_linear(x, ct, mt, 4, 32, **more)
        t.requires_grad_(False)


def test_tangents_are_refused():
    from torch.autograd import forward_ad

    x, ct, mt, more = small_call()
    with forward_ad.dual_level():
        awq.awq_lowbit_linear(x, ct, mt, 4, 32, **more)
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        with pytest.raises(RuntimeError, match="forward-mode"):
            awq.awq_lowbit_linear(dual, ct, mt, 4, 32, **more)
        with pytest.raises(RuntimeError, match="forward-mode"):
            awq.awq_lowbit_linear(x, ct, forward_ad.make_dual(mt, torch.ones_like(mt)), 4, 32, **more)
        for name in more:
            with pytest.raises(RuntimeError, match="forward-mode"):
                awq.awq_lowbit_linear(x, ct, mt, 4, 32, **{**more, name: forward_ad.make_dual(more[name], more[name] + 1)})
