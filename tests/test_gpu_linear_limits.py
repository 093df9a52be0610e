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
