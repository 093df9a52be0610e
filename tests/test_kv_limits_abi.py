"""What the rotary and cache entry points decide on the host, at the edges of their sizes (CPU): the
C calls get pointers that are never followed, and return before anything is enqueued."""

import ctypes
import random
import re

import pytest

import post_weight_quantization_act_amd as awq
from test_kv_abi import (INVALID, UNSUPPORTED, WORKSPACE, append_args, attention_args, cache, read_args, rope_args,
                         status, strides, table_args)


def test_append_of_no_rows_takes_an_empty_q():
    """Torch's empty tensors have null pointers."""
    nothing = dict(T=0, k=None, v=None, q=None, q_out=None)
    assert status("awq_kv_append", append_args(**nothing)) == 0
    assert status("awq_kv_append", append_args(**nothing, B=0, starts=None, lens=None, pages=None)) == 0
    assert status("awq_kv_append", append_args(q=None)) == INVALID


size, needed = awq.awq_kv_attention_workspace_size, awq.awq_kv_attention_workspace_needed


def asked(B, hq, heads, dim, max_len, max_pages, page, new=1, **over):
    """What the call says that it needs, given nothing; only for calls that need something."""
    got = status("awq_kv_attention", attention_args(
        cache=cache(kv_heads=heads, head_dim=dim, page=page), T=B * new, B=B, Hq=hq, qs=strides(hq * dim, dim),
        starts=None if new == 1 else 1 << 20, max_pages=max_pages, max_new=new, max_len=max_len, ws=None, ws_bytes=0,
        **over))
    assert got == WORKSPACE
    return int(re.search(rb"needs (\d+) workspace", awq.library().awq_last_error()).group(1))


@pytest.mark.parametrize("B,hq,heads,dim,max_len,max_pages,page", [
    (8, 64, 8, 128, 33024, 513, 64), (64, 64, 8, 128, 8193, 128, 64), (1, 64, 8, 128, 2 ** 31 - 1, 4096, 16),
    (1, 8, 8, 64, 1 << 30, 1 << 20, 64), (300, 8, 1, 256, 1 << 20, 2048, 32),
])
def test_the_documented_workspace_is_enough_whatever_the_table_holds(B, hq, heads, dim, max_len, max_pages, page):
    reach = min(max_len, max_pages * page)
    assert needed(B, B, hq, heads, dim, 1, reach) > 0
    want = asked(B, hq, heads, dim, max_len, max_pages, page)
    assert want == needed(B, B, hq, heads, dim, 1, reach) <= size(B, B, hq, heads, dim, 1, max_len)


def test_a_workspace_for_the_largest_call_is_enough_for_the_smaller_ones():
    rng = random.Random(1)
    around = [1, 2, 3, 7, 8, 31, 64, 255, 256, 257, 300, 511, 512, 513, 5000]
    lens = [1, 64, 511, 512, 513, 4096, 8192, 8193, 32768, 33024, 131071, 1 << 20, 1 << 25, 1 << 30, 1 << 31]
    some = 0
    for heads, group, dim in ((1, 1, 8), (8, 8, 128), (2, 7, 80), (32, 1, 128), (1, 64, 64), (1, 100, 96), (4, 16, 256),
                              (8, 4, 200), (2, 8, 192)):
        hq = heads * group
        for _ in range(3000):
            B, new, long = rng.choice(around), rng.choice([1, 1, 2, 4, 5, 9, 33, 64, 65, 700, 4096]), rng.choice(lens)
            T = min(B * new, rng.choice([B, B * new, B * new // 2 + 1]))
            b, n = rng.choice([x for x in around if x <= B]), rng.randint(1, new)
            t = rng.randint(1, min(T, b * n))
            short = rng.choice([x for x in lens if x <= long] + [rng.randint(1, long)])
            have, want = size(T, B, hq, heads, dim, new, long), needed(t, b, hq, heads, dim, n, short)
            assert want <= have, (T, B, hq, heads, dim, new, long, t, b, n, short)
            some += want > 0
            # one call alone, rows that no sequence has among them, its table of any length
            T += rng.choice([0, 0, 10, 100000])
            assert needed(T, B, hq, heads, dim, new, short) <= size(T, B, hq, heads, dim, new, long)
    assert some > 5000


def test_the_workspace_stays_in_bounds():
    # a decode step of 64 long sequences, a prompt's piece, one long sequence
    assert size(64, 64, 64, 8, 128, 1, 131072) < 1 << 28
    assert size(16384, 8, 64, 8, 128, 4096, 131072) < 1 << 28
    assert size(1, 1, 64, 8, 128, 1, 1 << 20) < 1 << 28
    assert size(64, 64, 64, 8, 128, 1, 512) == 0 and needed(64, 64, 64, 8, 128, 1, 512) == 0
    assert status("awq_kv_attention", attention_args(T=(1 << 31) - 1, Hq=64, cache=cache(kv_heads=64))) == UNSUPPORTED
    assert size((1 << 31) - 1, 2, 64, 64, 64, 1, 4096) == 0


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 9, 2 ** 31 - 1])
def test_enumerations_of_any_value_are_refused(bad):
    for name in ("x_dtype", "out_dtype"):
        assert status("awq_rope", rope_args(**{name: bad})) == INVALID
    for name in ("dtype", "q_dtype"):
        assert status("awq_kv_append", append_args(**{name: bad})) == INVALID
    assert status("awq_kv_attention", attention_args(dtype=bad)) == INVALID
    assert status("awq_kv_read", read_args(dtype=bad)) == INVALID
    scaling = ctypes.byref(awq.RopeScaling(bad, 1, 1, 1, 2, 1))
    assert status("awq_rope_table", table_args(scaling=scaling)) == INVALID
