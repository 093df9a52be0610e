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


def test_append_of_no_rows():
    cache = awq.KvCache.empty(2, 2, 16, 16)
    k = torch.zeros((3, 6, 16), device="cuda")
    q = awq.awq_kv_append(cache, k[:0, :2], k[:0, 2:4], ints([5]), ints([[0, 1]]), starts=ints([0, 0]), q=k[:0],
                          q_dtype=torch.float16)
    assert q.shape == (0, 6, 16) and q.dtype == torch.float16


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


# ---------------------------------------------------------------------------------------------
# more workgroups than one launch holds (2^32 threads): bounds far above what a call has
# ---------------------------------------------------------------------------------------------
FAR = 1 << 28    # rows of a sequence: 2^24 pages of 16 tokens


def test_append_and_read_with_a_far_bound():
    rng = np.random.default_rng(22)
    dev, ref = new_cache(rng, 6, 1, 16, 8)
    table = page_table(rng, 2, 6, 3)
    k = torch.from_numpy(rng.standard_normal((40, 1, 8)).astype(f32)).cuda()
    starts, lens = [0, 30, 40], [40, 10]
    for rope in (None, awq.awq_rope_table(64, 6)):       # vectors, pair by pair
        turned = wide(k) if rope is None else kv_ref.rope(wide(k), wide(rope), list(range(10, 40)) + list(range(10)))
        q = awq.awq_kv_append(dev, k, k, ints(lens), ints(table.tolist()), starts=ints(starts), max_new=FAR,
                              table=rope, q=k)
        np.testing.assert_array_equal(wide(q), turned)
        ref.append(turned, wide(k), lens, table, starts)
        for b, n in enumerate(lens):
            p, t = table[b, n // 16], n % 16
            ref.k_codes[p, :, t:] = dev.k_codes[p, :, t:].cpu().numpy()
            ref.v_codes[p, :, :, t:] = dev.v_codes[p, :, :, t:].cpu().numpy()
        assert_same_cache(dev, ref)
    got = awq.awq_kv_read(dev, ints([10, 0]), ints(table.tolist()), starts=ints(starts), total=40, max_count=FAR)
    want = [ref.tokens(0, 10, 40, table), ref.tokens(1, 0, 10, table)]
    for i in (0, 1):
        np.testing.assert_array_equal(wide(got[i]), np.concatenate([w[i] for w in want]))


def test_attention_with_a_far_bound():
    rng = np.random.default_rng(23)
    dev, ref = new_cache(rng, 8, 1, 16, 32)
    table = page_table(rng, 1, 8, 8)
    q = torch.from_numpy(rng.standard_normal((90, 2, 32)).astype(f32)).half().cuda()
    check_attention(dev, ref, q, [120], table, [0, 90], "f16", max_new=2 ** 30 - 1, max_len=128)


@pytest.mark.parametrize("rot", [0, 6])
def test_append_and_read_of_many_sequences_with_the_default_bounds(rot):
    """2^12 sequences of 64 of 2^18 rows, any of which might have them all: 2^26 pages, one by one."""
    B, n = 1 << 12, 64
    gen = torch.Generator(device="cuda").manual_seed(26)
    k = torch.randn((B * n, 1, 8), generator=gen, device="cuda")
    pages = torch.randperm(4 * B, generator=gen, device="cuda").int().view(B, 4)
    lens, starts = ints([n] * B), torch.arange(0, B * n + 1, n, device="cuda", dtype=torch.int32)
    table = awq.awq_rope_table(n, rot) if rot else None
    got = []
    for bound in (None, n):
        cache = awq.KvCache.empty(4 * B, 1, 16, 8)
        q = awq.awq_kv_append(cache, k, -k, lens, pages, starts=starts, max_new=bound, table=table, q=k)
        back = awq.awq_kv_read(cache, lens - n, pages, starts=starts, total=B * n, max_count=bound)
        got.append((q, cache.k_codes, cache.v_codes, cache.k_steps, cache.v_steps, *back))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert torch.equal(got[0][0], k) if not rot else torch.equal(got[0][0][..., 6:], k[..., 6:])
    assert (got[0][6] + k).abs().max() <= k.abs().max() / 254 * 1.001       # half a step


def test_attention_of_many_sequences_with_the_default_bounds():
    B, n = 1 << 12, 64
    gen = torch.Generator(device="cuda").manual_seed(27)
    cache = awq.KvCache.empty(4 * B, 1, 16, 8)
    q = torch.randn((B * n, 8, 8), generator=gen, device="cuda").half()
    pages = torch.randperm(4 * B, generator=gen, device="cuda").int().view(B, 4)
    lens, starts = ints([n] * B), torch.arange(0, B * n + 1, n, device="cuda", dtype=torch.int32)
    awq.awq_kv_append(cache, q[:, :1], q[:, 1:2], lens, pages, starts=starts, max_new=n)
    want = awq.awq_kv_attention(cache, q, lens, pages, starts=starts, max_new=n)
    assert torch.equal(awq.awq_kv_attention(cache, q, lens, pages, starts=starts), want)


def test_attention_of_more_sequences_than_a_launch_has_workgroups():
    """2^24 sequences of one token, which might have 4112: two splits each, and their join."""
    B = 1 << 24
    cache = awq.KvCache(*(torch.full(s, 130, dtype=torch.uint8, device="cuda") for s in ((1, 1, 16, 8), (1, 1, 8, 16))),
                        torch.ones(1, 1, device="cuda"), torch.ones(1, 1, device="cuda"))
    q = torch.randn((B, 1, 8), device="cuda").half()
    out, lse = awq.awq_kv_attention(cache, q, torch.ones(B, dtype=torch.int32, device="cuda"),
                                    torch.zeros((B, 257), dtype=torch.int32, device="cuda"), scale=0.5, return_lse=True)
    assert (out == 2).all()
    # one score of eight products, a few roundings of 2^-24 of at most 8 x 2 x 6
    assert (lse.double() - q.double().sum(-1)).abs().max() <= 16 * 2.0 ** -24 * 96


def test_rope_table_of_more_pairs_than_a_launch_has_threads():
    n = 1 << 32
    table = awq.awq_rope_table(n, 2)
    at = [0, 1, 12345, (1 << 32) - 257, (1 << 32) - 256, (1 << 32) - 1]
    got = table[at, 0].cpu().numpy()
    want = np.stack([np.cos(np.array(at, float)), np.sin(np.array(at, float))], -1)
    assert (np.abs(got - want) <= 2.0 ** -24).all()


@pytest.mark.parametrize("dim,rot", [(2, 2), (8, 8)])
def test_rope_of_more_items_than_a_launch_has_threads(dim, rot):
    """2^32 pairs one by one; and 2^24 rows of 129 vectors, a workgroup each."""
    S, H = (1 << 22, (1 << 10) + 1) if dim == 2 else (1 << 24, 129)
    x = torch.randn((1, H, dim), device="cuda").bfloat16().expand(S, H, dim)
    table = awq.awq_rope_table(2, rot)
    at = torch.zeros(S, dtype=torch.int32, device="cuda")
    at[-1] = 1
    out = awq.awq_rope(x, table, at)
    want = awq.awq_rope(x[:1], table, at[:1])
    for part, x0 in ((out[:-1].split(1 << 20), want), (out[-1:].split(1), awq.awq_rope(x[-1:], table, at[-1:]))):
        for p in part:
            assert torch.equal(p, x0.expand_as(p))


def test_rope_of_a_row_of_more_units_than_32_bits_count():
    """One row of 1.4e9 heads of three units."""
    H = (1 << 32) // 3 + 100
    x = torch.randn((1, 1, 24), device="cuda").bfloat16().expand(1, H, 24)
    table = awq.awq_rope_table(2, 8)
    out = torch.full((1, H, 24), 7.0, device="cuda", dtype=torch.bfloat16)
    awq.awq_rope(x, table, ints([1]), out=out)
    want = awq.awq_rope(x[:, :1], table, ints([1]))[0]
    for p in out[0].split(1 << 24):
        assert torch.equal(p, want.expand_as(p))


# ---------------------------------------------------------------------------------------------
# the rotation's gradient is recorded
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("into,out", [("f32", "f32"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "f32")])
def test_rope_records_its_gradient(into, out, interleaved):
    gen = torch.Generator(device="cuda").manual_seed(24)
    table = awq.awq_rope_table(50, 24)
    base = torch.randn((2, 7, 5, 32), generator=gen, device="cuda").to(TYPES[into])
    leaf = base.clone().requires_grad_()
    at = torch.randint(0, 50, (2, 7), generator=gen, device="cuda", dtype=torch.int32)
    x = leaf[:, :, 1:4].transpose(1, 2).transpose(1, 2)          # a view with strides of its own
    y = awq.awq_rope(x, table, at, interleaved=interleaved, out_dtype=TYPES[out])
    assert torch.equal(y, awq.awq_rope(base[:, :, 1:4], table, at, interleaved=interleaved, out_dtype=TYPES[out]))
    g = torch.randn(y.shape, generator=gen, device="cuda").to(y.dtype)
    y.backward(g)
    want = torch.zeros_like(base)
    want[:, :, 1:4] = awq.awq_rope(g, table, at, interleaved=interleaved, transpose=True, out_dtype=TYPES[into])
    assert leaf.grad.dtype == leaf.dtype and torch.equal(leaf.grad, want)


def test_rope_gradients_of_a_broadcast_sum_and_of_the_gradient():
    table = awq.awq_rope_table(9, 8)
    x = torch.randn(1, 2, 8, device="cuda", requires_grad=True)
    y = awq.awq_rope(x.expand(9, 2, 8), table)
    (gx,) = torch.autograd.grad(y.sum(), x)                      # the sum's gradient has no strides
    rows = awq.awq_rope(torch.ones(9, 2, 8, device="cuda"), table, transpose=True)
    assert torch.equal(gx, rows.sum(0, keepdim=True))
    g = torch.randn(9, 2, 8, device="cuda", requires_grad=True)
    (gx,) = torch.autograd.grad(awq.awq_rope(x.expand(9, 2, 8), table), x, g, create_graph=True)
    h = torch.randn_like(gx)
    (gg,) = torch.autograd.grad(gx, g, h)
    assert torch.equal(gg, awq.awq_rope(h.expand(9, 2, 8), table))
    with torch.no_grad():
        assert not awq.awq_rope(x, table).requires_grad


# ---------------------------------------------------------------------------------------------
# instances that the other shapes do not reach
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("size", [2.0 ** -110, 2.0 ** -70, 2.0 ** -61 * 127, 2.0 ** 60 * 127, 2.0 ** 64, 2.0 ** 110])
def test_append_of_values_whose_steps_are_scaled(size, kind):
    """Steps below 2^-60 and above 2^60, where codes come from scaled quotients, and next to them."""
    rng = np.random.default_rng(25)
    dev, ref = new_cache(rng, 4, 2, 16, 32, steps=(0.0, 0.0))
    table = page_table(rng, 1, 4, 3)
    at = 0
    for n, factor in ((5, 0.5), (20, 1.0), (1, 4.0), (9, 2.0 ** -8)):
        k, v = (torch.from_numpy((rng.standard_normal((n, 2, 32)) * size * factor).astype(f32)).to(TYPES[kind]).cuda()
                for _ in range(2))
        at += n
        awq.awq_kv_append(dev, k, v, ints([at]), ints(table.tolist()), starts=ints([0, n]), max_new=n)
        ref.append(wide(k), wide(v), [at], table, [0, n])
    k, v = awq.awq_kv_read(dev, ints([0]), ints(table.tolist()), starts=ints([0, at]), total=at)
    want = ref.tokens(0, 0, at, table)
    np.testing.assert_array_equal(wide(k), want[0])
    np.testing.assert_array_equal(wide(v), want[1])


FULL_PAGES = [   # new tokens, tokens before, D, rot, page: four units of four pairs a thread
    (600, 3, 72, 72, 256), (259, 250, 120, 8, 256), (300, 0, 128, 120, 256), (500, 9, 104, 24, 256), (257, 127, 256, 248, 128),
    (130, 100, 200, 104, 128),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", FULL_PAGES)
def test_append_of_full_pages_by_runs_of_four(shape, kind, interleaved):
    new, before, dim, rot, page = shape
    rng = np.random.default_rng(new + dim)
    length = new + before
    per_seq = -(-length // page)
    dev, ref = new_cache(rng, per_seq + 1, 2, page, dim)
    table = page_table(rng, 1, dev.n_pages, per_seq)
    qkv = torch.from_numpy(rng.standard_normal((new, 6, dim)).astype(f32)
                           * rng.choice([0.3, 30.0], (new, 1, 1)).astype(f32)).to(TYPES[kind]).cuda()
    rope = awq.awq_rope_table(length, rot)
    at = np.arange(before, length)
    q = awq.awq_kv_append(dev, qkv[:, 2:4], qkv[:, 4:], ints([length]), ints(table.tolist()), starts=ints([0, new]),
                          max_new=new, table=rope, interleaved=interleaved, q=qkv[:, :2], q_dtype=torch.float32)
    turn = lambda x: kv_ref.rope(wide(x), wide(rope), at, interleaved)       # noqa: E731
    np.testing.assert_array_equal(wide(q), turn(qkv[:, :2]))
    ref.append(turn(qkv[:, 2:4]), wide(qkv[:, 4:]), [length], table, [0, new])
    if length % page:
        p, t = table[0, length // page], length % page
        ref.k_codes[p, :, t:] = dev.k_codes[p, :, t:].cpu().numpy()
        ref.v_codes[p, :, :, t:] = dev.v_codes[p, :, :, t:].cpu().numpy()
    assert_same_cache(dev, ref)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("rows", ["one short", "one long", "uneven", "two tiles", "two tiles long",
                                  "two tiles uneven", "many"])
@pytest.mark.parametrize("dim", [104, 120, 128, 136, 160, 168, 192, 200, 224, 256])
def test_attention_of_every_width(dim, rows, kind):
    """The kernels' instances above 96 columns, by each of their forms: eight waves, splits that are joined, splits that
    the lengths choose, 17 to 64 rows of a head, and more."""
    new, lens, hq, heads, page = {
        "one short": ([1, 1], [300, 77], 8, 2, 16), "one long": ([1], [2600], 16, 1, 64),
        "uneven": ([1, 1, 1], [1500, 4, 700], 8, 2, 32), "two tiles": ([9, 4], [333, 90], 8, 2, 64),
        "two tiles long": ([13], [2600], 6, 2, 64), "two tiles uneven": ([9, 2, 5], [700, 1500, 30], 8, 2, 16),
        "many": ([50, 21], [200, 90], 4, 2, 32)}[rows]
    rng = np.random.default_rng(dim + len(rows))
    per_seq = -(-max(lens) // page)
    dev, ref = new_cache(rng, len(new) * per_seq, heads, page, dim)
    table = page_table(rng, len(new), dev.n_pages, per_seq)
    q = torch.from_numpy(rng.standard_normal((sum(new), hq, dim)).astype(f32)).to(TYPES[kind]).cuda()
    starts = None if max(new) == 1 else starts_of(new)
    for window in (0, 40):
        check_attention(dev, ref, q, lens, table, starts, kind, window, max_new=max(new), max_len=max(lens))
