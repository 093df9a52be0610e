"""Calls at the edges of their own limits: fewer rows allowed than a sequence has, lengths cut short,
windows and bounds as large as they may be, and grids of more workgroups than one launch holds."""

import numpy as np
import pytest
import torch

import post_weight_quantization_act_amd as awq
from oracle import kv_ref
from test_gpu_kv import (TYPES, assert_same_cache, attention_bound, check_attention, f32, ints, new_cache,
                         page_table, wide)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    awq.library()
    yield
    torch.cuda.synchronize()


def starts_of(rows):
    return np.concatenate(([0], np.cumsum(rows))).tolist()


# ---------------------------------------------------------------------------------------------
# fewer rows allowed than a sequence has
# ---------------------------------------------------------------------------------------------
LIMITED = [   # rows of each sequence, max_new, lengths, q heads, kv heads, D, page
    ([10], 4, [10], 2, 1, 32, 16), ([10, 3, 1], 4, [40, 3, 7], 8, 2, 64, 16), ([9, 20], 5, [300, 200], 16, 1, 64, 32),
    ([6, 2, 9], 3, [1500, 700, 90], 8, 2, 64, 64), ([12], 2, [3001], 4, 1, 128, 64), ([40], 17, [900], 8, 2, 96, 32),
    ([5], 1, [4], 4, 4, 256, 64),
]


def first_rows(rows, most):
    """Which rows of a call are among the first `most` of their sequence."""
    return np.concatenate([np.arange(n) < most for n in rows])


@pytest.mark.parametrize("window,causal", [(0, True), (7, True), (0, False), (9, False)])
@pytest.mark.parametrize("shape", LIMITED)
def test_attention_of_the_first_rows(shape, window, causal):
    """Rows beyond max_new are left out; those before it keep their tokens."""
    rows, most, lens, hq, heads, dim, page = shape
    rng = np.random.default_rng(sum(lens) + dim)
    per_seq = -(-max(lens) // page)
    dev, ref = new_cache(rng, len(rows) * per_seq, heads, page, dim)
    table = page_table(rng, len(rows), dev.n_pages, per_seq)
    starts, T = starts_of(rows), sum(rows)
    q = torch.from_numpy(rng.standard_normal((T, hq, dim)).astype(f32)).half().cuda()
    out = torch.full_like(q, 7.0)
    awq.awq_kv_attention(dev, q, ints(lens), ints(table.tolist()), starts=ints(starts), max_new=most,
                         max_len=max(lens), window=window, causal=causal, out=out)
    scale = dim ** -0.5
    want, _, spread, top = ref.attention(wide(q), lens, table, starts, scale, window, causal)
    _, bound = attention_bound(ref, wide(q), scale, spread, top, want, "f16", dim)
    taken = first_rows(rows, most)
    assert (np.abs(wide(out) - want) <= bound)[taken].all()
    assert (wide(out)[~taken] == 7).all()


APPEND_LIMITED = [   # rows of each sequence, max_new, tokens before, kv heads, q heads, D, rot, page
    ([20], 1, [0], 1, 2, 128, 128, 64), ([20, 3], 2, [5, 30], 2, 4, 128, 64, 64), ([90, 7], 33, [10, 60], 2, 2, 64, 24, 32),
    ([50], 40, [15], 1, 1, 80, 20, 16), ([300], 5, [250], 2, 2, 96, 72, 256), ([9], 4, [-6], 1, 2, 64, 0, 16),
]


@pytest.mark.parametrize("kind", ["f32", "f16"])
@pytest.mark.parametrize("shape", APPEND_LIMITED)
def test_append_of_the_first_rows(shape, kind):
    rows, most, before, heads, hq, dim, rot, page = shape
    rng = np.random.default_rng(sum(rows) + dim)
    B, T = len(rows), sum(rows)
    lens = [n + m for n, m in zip(rows, before)]
    per_seq = -(-max(lens) // page)
    dev, ref = new_cache(rng, B * per_seq, heads, page, dim)
    table = page_table(rng, B, dev.n_pages, per_seq)
    qkv = torch.from_numpy(rng.standard_normal((T, hq + 2 * heads, dim)).astype(f32)).to(TYPES[kind]).cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq: hq + heads], qkv[:, hq + heads:]
    rope = awq.awq_rope_table(max(lens), rot) if rot else None
    at = np.concatenate([np.arange(m, n) for m, n in zip(before, lens)])
    turn = (lambda x: kv_ref.rope(wide(x), wide(rope), at)) if rot else wide
    q_out = torch.full_like(q, 7.0, dtype=torch.float32, memory_format=torch.contiguous_format)
    awq.awq_kv_append(dev, k, v, ints(lens), ints(table.tolist()), starts=ints(starts_of(rows)), max_new=most,
                      table=rope, q=q, q_out=q_out)
    taken = np.concatenate([np.arange(n) < most for n in rows])
    kept = [min(n, most) for n in rows]
    ref.append(turn(k)[taken], wide(v)[taken], [m + n for m, n in zip(before, kept)], table, starts_of(kept))
    # places past the tokens that were appended are nobody's
    for b, n in enumerate(kept):
        p, t = (before[b] + n) // page, (before[b] + n) % page
        if t > 0:
            ref.k_codes[table[b, p], :, t:] = dev.k_codes[table[b, p], :, t:].cpu().numpy()
            ref.v_codes[table[b, p], :, :, t:] = dev.v_codes[table[b, p], :, :, t:].cpu().numpy()
    assert_same_cache(dev, ref)
    turned = taken & (at >= 0)       # tokens before a sequence's start are dropped, their queries with them
    np.testing.assert_array_equal(wide(q_out)[turned], turn(q)[turned])
    assert (wide(q_out)[~turned] == 7).all()


@pytest.mark.parametrize("most", [1, 3, 16, 19])
def test_read_of_the_first_tokens(most):
    rng = np.random.default_rng(most)
    dev, ref = new_cache(rng, 8, 2, 16, 24)
    table = page_table(rng, 2, 8, 4)
    first, count = [5, 30], [40, 20]
    k = torch.full((60, 2, 24), 7.0, device="cuda")
    v = k.clone()
    lib, struct = awq.library(), dev._ref
    starts, at, pages = ints(starts_of(count)), ints(first), ints(table.tolist())
    assert lib.awq_kv_read(struct, 60, starts.data_ptr(), at.data_ptr(), 2, pages.data_ptr(), 4, most,
                           k.data_ptr(), v.data_ptr(), awq.AWQ_F32,
                           torch.cuda.current_stream().cuda_stream) == 0
    taken = np.concatenate([np.arange(n) < most for n in count])
    want = [ref.tokens(b, first[b], first[b] + count[b], table) for b in range(2)]
    for got, i in ((k, 0), (v, 1)):
        np.testing.assert_array_equal(wide(got)[taken], np.concatenate([w[i] for w in want])[taken])
        assert (wide(got)[~taken] == 7).all()


# ---------------------------------------------------------------------------------------------
# windows and lengths
# ---------------------------------------------------------------------------------------------
class Cut(kv_ref.Cache):
    """The oracle's cache of which only the first max_len tokens of a sequence are attended to."""

    def __init__(self, ref, max_len):
        self.__dict__.update(ref.__dict__)
        self.max_len = max_len

    def tokens(self, b, lo, hi, pages):
        k, v, there = super().tokens(b, lo, hi, pages)
        return k, v, there & (np.arange(lo, hi) < self.max_len)


CUT = [   # rows of each sequence, lengths, max_len, window, q heads, kv heads, D, page
    ([4], [21], 18, 1, 2, 1, 32, 16), ([4, 6], [21, 30], 18, 3, 4, 2, 64, 32), ([70], [100], 50, 5, 2, 1, 64, 32),
    ([60, 8], [700, 40], 661, 20, 4, 1, 128, 64), ([5, 5, 5], [1300, 1299, 1297], 1297, 2, 2, 2, 96, 64),
    ([6], [21], 18, 0, 2, 1, 32, 16), ([3], [40], 17, 4, 2, 2, 256, 16),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", CUT)
def test_attention_windows_that_begin_past_max_len(shape, causal):
    """Such a row sees nothing, and nothing of what lies past max_len, numbers or not."""
    rows, lens, max_len, window, hq, heads, dim, page = shape
    rng = np.random.default_rng(sum(lens) + dim)
    per_seq = -(-max(lens) // page)
    dev, ref = new_cache(rng, len(rows) * per_seq, heads, page, dim)
    table = page_table(rng, len(rows), dev.n_pages, per_seq)
    past = table[:, -(-max_len // page):].reshape(-1).tolist()
    dev.k_steps[past], dev.v_steps[past] = float("nan"), float("nan")
    q = torch.from_numpy(rng.standard_normal((sum(rows), hq, dim)).astype(f32)).half().cuda()
    check_attention(dev, Cut(ref, max_len), q, lens, table, starts_of(rows), "f16", window, causal,
                    max_new=max(rows), max_len=max_len)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 40])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_windows_longer_than_any_sequence(window, causal):
    """More rows than tokens, so that the first rows' windows begin before the sequence."""
    rng = np.random.default_rng(21)
    dev, ref = new_cache(rng, 8, 1, 16, 32)
    table = page_table(rng, 2, 8, 4)
    q = torch.from_numpy(rng.standard_normal((11, 2, 32)).astype(f32)).half().cuda()
    check_attention(dev, ref, q, [2, 60], table, [0, 5, 11], "f16", window, causal, max_new=6, max_len=64)


def test_attention_over_more_tiles_than_half_a_32_bit_sum():
    """256 sequences of 2^28 tokens, all of them the same page of equal values: every sequence's sum has to
    come whole from its splits.  A wave adds 2^19 or 2^20 equal addends, each sum rounded to 2^-24 of itself:
    up to 2^-4 of an addend, so of the result, in the sum of the probabilities; twice (two products a tile)
    in the values'."""
    cache = awq.KvCache(torch.full((1, 1, 256, 8), 128, dtype=torch.uint8, device="cuda"),
                        torch.full((1, 1, 8, 256), 129, dtype=torch.uint8, device="cuda"),
                        torch.ones(1, 1, device="cuda"), torch.ones(1, 1, device="cuda"))
    B, tokens = 256, 1 << 28
    pages = torch.zeros((B, tokens // 256), dtype=torch.int32, device="cuda")
    q = torch.ones((B, 1, 8), dtype=torch.float16, device="cuda")
    ws = torch.zeros(awq.awq_kv_attention_workspace_size(B, B, 1, 1, 8, 1, tokens), dtype=torch.uint8, device="cuda")
    out, lse = awq.awq_kv_attention(cache, q, ints([tokens] * B), pages, max_len=tokens, return_lse=True, workspace=ws)
    assert (np.abs(wide(out) - 1) <= 3 * 2.0 ** -4).all()
    assert (np.abs(wide(lse) - 28 * np.log(2)) <= 2 * 2.0 ** -4).all()
