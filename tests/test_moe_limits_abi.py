"""Sizes of workspaces of the entry points of a block of experts (CPU)."""

import random

import pytest
import torch

import post_weight_quantization_act_amd as awq

size, needed = awq.awq_lowbit_linear_workspace_size, awq.awq_lowbit_linear_workspace_needed
TYPES = (torch.float16, torch.bfloat16)


@pytest.mark.parametrize("N,K", [(4096, 4096), (4096, 11008), (28672, 4096), (300, 4096), (8100, 64), (130, 32768), (64, 2048)])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_workspace_covers_fewer_rows(N, K, gated):
    """The most that any smaller number of rows needs, no less and no more; it never falls."""
    for dtype in TYPES:
        most = 0
        for rows in list(range(1, 1400)) + [1536, 2047, 2048, 4095, 4096, 8192, 16383, 16384, 16385, 20000, 70000]:
            own = needed(dtype, rows, rows, N, K, 1, gated)
            most = max(most, own)
            got = size(dtype, rows, rows, N, K, 1, gated)
            assert got >= own and got >= most, rows
            if rows < 1400:
                assert got == most, rows
    assert size(torch.float16, 4096, 4096, 4096, 4096) >= needed(torch.float16, 512, 512, 4096, 4096) > 0


def test_linear_workspace_of_drawn_sizes():
    rng = random.Random(5)
    for _ in range(4000):
        dtype, N, K = rng.choice(TYPES), rng.randint(1, 9000), 32 * rng.randint(1, 300)
        experts, gated = rng.choice([1, 1, 1, 2, 8, 60, 1024]), rng.random() < 0.4
        rows, x_rows = int(2 ** rng.uniform(0, 17)), int(2 ** rng.uniform(0, 17))
        less, x_less = rng.randint(1, rows), rng.randint(1, x_rows)
        assert size(dtype, rows, x_rows, N, K, experts, gated) >= max(needed(dtype, rows, x_rows, N, K, experts, gated),
                                                                     needed(dtype, less, x_less, N, K, experts, gated))


def test_linear_workspace_needed_of_what_is_refused():
    f = awq.library().awq_lowbit_linear_workspace_needed
    good = dict(dtype=2, rows=4096, x_rows=4096, N=4096, K=4096, experts=1, flags=0)
    for over in (dict(dtype=7), dict(rows=0), dict(rows=-1), dict(x_rows=0), dict(N=0), dict(K=0), dict(experts=0),
                 dict(rows=1 << 31), dict(x_rows=1 << 31), dict(N=1 << 31), dict(experts=1025)):
        assert f(*{**good, **over}.values()) == 0


def test_the_scaling_pass_stays_in_one_launch():
    """A wave a row: rows of 32 columns are scaled up to where their waves would be 2^32 threads."""
    assert needed(torch.bfloat16, 2 ** 26 - 5, 2 ** 26 - 5, 4096, 32) >= (2 ** 26 - 5) * 68
    for rows in range(2 ** 26 - 4, 2 ** 26 + 4):
        assert needed(torch.bfloat16, rows, rows, 4096, 32) == 0
