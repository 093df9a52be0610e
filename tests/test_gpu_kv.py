"""Rotary positions, the paged 8-bit cache and its attention on the GPU against the 64-bit
oracle (turned keys, steps and codes: bit for bit against its fp32 emulation)."""

import numpy as np
import pytest
import torch

import post_weight_quantization_act_amd as awq
from oracle import kv_ref

pytestmark = pytest.mark.gpu

f32 = np.float32
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


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def wide(t):
    """Exact fp32 NumPy copy."""
    return t.detach().float().cpu().numpy()


def rounded(x, kind):
    return wide(torch.from_numpy(np.ascontiguousarray(x, dtype=f32)).to(TYPES[kind]))


# ---------------------------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("kw", [
    dict(), dict(scaling="linear", factor=4.0), dict(base=500000.0, magnitude=1.25),
    dict(scaling="turns", factor=8.0, original=64.0, low=1.0, high=4.0),
    dict(scaling="log_turns", factor=8.0, original=64.0, low=0.5, high=8.0, magnitude=0.9),
])
def test_table(kw):
    got = wide(awq.awq_rope_table(1000, 48, **kw))
    magnitude = kw.pop("magnitude", 1.0)
    want = kv_ref.rope_table(1000, 48, magnitude=magnitude, **kw)
    # one rounding to fp32; the angle p f carries a few fp64 roundings of up to 1000 radians
    assert (np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + 1000 * 2.0 ** -49 * magnitude).all()


ROPE_SHAPES = [   # B, S, H, D, rot, order of the memory, offset of the first element
    (1, 1, 1, 8, 8, "bshd", 0), (1, 1, 40, 128, 128, "bshd", 0), (2, 33, 3, 96, 64, "bhsd", 0),
    (1, 257, 5, 80, 80, "bshd", 0), (3, 7, 2, 256, 32, "sbhd", 0), (1, 65, 4, 64, 62, "bshd", 0),
    (2, 19, 3, 33, 6, "bshd", 0), (1, 100, 2, 128, 128, "bshd", 1), (1, 70, 2, 128, 64, "bhsd", 8),
    (2, 37, 5, 80, 40, "bhsd", 0), (1, 41, 3, 256, 8, "bshd", 1), (3, 9, 33, 72, 56, "sbhd", 0),
    (2, 300, 64, 96, 72, "bshd", 0),
]


def placed(shape, order, offset, dtype, gen, extra=1):
    """A [B, S, H, D] view whose memory is in another order, from a buffer that holds more."""
    at = {"b": 0, "s": 1, "h": 2}
    mem = [shape[at[c]] for c in order[:3]] + [shape[3]]
    mem[1] += extra
    buf = torch.randn(int(np.prod(mem)) + offset, generator=gen, device="cuda").to(dtype)
    t = buf[offset:].view(mem)[:, extra:]
    return t.permute(*[order.index(c) for c in "bsh"], 3)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("into,out", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f32", "bf16"),
                                      ("bf16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("shape", ROPE_SHAPES)
def test_rope(shape, into, out, interleaved):
    B, S, H, D, rot, order, offset = shape
    gen = torch.Generator(device="cuda").manual_seed(S * D + H)
    x = placed((B, S, H, D), order, offset, TYPES[into], gen)
    table = awq.awq_rope_table(4 * S + 3, rot)
    positions = torch.randint(0, 4 * S + 3, (B, S), generator=gen, device="cuda", dtype=torch.int32)
    for transpose in (False, True):
        got = awq.awq_rope(x, table, positions, interleaved=interleaved, transpose=transpose,
                           out_dtype=TYPES[out])
        assert got.dtype == TYPES[out] and got.is_contiguous()
        want = np.stack([kv_ref.rope(wide(x)[b], wide(table), positions[b].cpu().numpy(), interleaved,
                                     transpose) for b in range(B)])
        np.testing.assert_array_equal(wide(got), rounded(want, out))
    shared = awq.awq_rope(x, table, positions[0].contiguous(), interleaved=interleaved)
    want = kv_ref.rope(wide(x), wide(table), positions[0].cpu().numpy(), interleaved)
    np.testing.assert_array_equal(wide(shared), rounded(want, into))


def test_rope_in_place_strided_out_and_no_positions():
    gen = torch.Generator(device="cuda").manual_seed(5)
    table = awq.awq_rope_table(64, 32)
    x = placed((2, 50, 4, 64), "bhsd", 0, torch.bfloat16, gen)
    want = rounded(kv_ref.rope(wide(x), wide(table), np.arange(50)), "bf16")
    out = placed((2, 50, 4, 64), "sbhd", 0, torch.bfloat16, gen)
    before = wide(x)
    assert awq.awq_rope(x, table, out=out) is out
    np.testing.assert_array_equal(wide(out), want)
    np.testing.assert_array_equal(wide(x), before)
    assert awq.awq_rope(x, table, out=x) is x
    np.testing.assert_array_equal(wide(x), want)
    y = torch.randn(50, 4, 64, generator=gen, device="cuda")        # [T, H, D]
    np.testing.assert_array_equal(wide(awq.awq_rope(y, table)),
                                  kv_ref.rope(wide(y), wide(table), np.arange(50)))
    assert awq.awq_rope(y[:0], table).shape == (0, 4, 64)


def test_rope_position_outside_the_table_is_nan():
    x = torch.ones(4, 2, 16, device="cuda")
    table = awq.awq_rope_table(8, 8)
    got = wide(awq.awq_rope(x, table, ints([7, 8, -1, 2 ** 31 - 1])))
    assert np.isfinite(got[0]).all() and np.isnan(got[1:, :, :8]).all() and (got[..., 8:] == 1).all()


def test_rope_transpose_is_the_gradient_by_differences():
    gen = torch.Generator(device="cuda").manual_seed(9)
    table = awq.awq_rope_table(100, 12, magnitude=1.5)
    x, g = torch.randn(2, 3, 2, 16, generator=gen, device="cuda")
    at = ints([3, 50, 99])
    dx = wide(awq.awq_rope(g, table, at, transpose=True)).astype(np.float64)
    for i in range(x.numel()):
        e = torch.zeros(x.numel(), device="cuda")
        e[i] = 1.0
        e = e.view_as(x)
        d = (awq.awq_rope(x + e, table, at).double() - awq.awq_rope(x - e, table, at).double()) / 2
        # linear: only fp32 roundings of values below 8 * 1.5 * sqrt(2), two terms an output
        assert abs(float((d * g.double()).sum()) - dx.reshape(-1)[i]) < 2 ** -24 * 17 * 8 * 3


@pytest.mark.parametrize("call", [
    lambda x, t, p: awq.awq_rope(x.permute(0, 2, 1), t),
    lambda x, t, p: awq.awq_rope(x, t.double()),
    lambda x, t, p: awq.awq_rope(x, t, p.long()),
    lambda x, t, p: awq.awq_rope(x, t, p[:-1]),
    lambda x, t, p: awq.awq_rope(x, t, out=x.half(), out_dtype=torch.float32),
    lambda x, t, p: awq.awq_rope(x[0], t),
])
def test_rope_binding_refuses(call):
    x = torch.zeros(4, 3, 16, device="cuda")
    with pytest.raises(ValueError):
        call(x, awq.awq_rope_table(8, 8), ints([0, 1, 2, 3]))
    with pytest.raises(TypeError):
        awq.awq_rope(x.double(), awq.awq_rope_table(8, 8))
    with pytest.raises(awq.AwqError):
        awq.awq_rope(x, awq.awq_rope_table(8, 18))


# ---------------------------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------------------------
def new_cache(rng, n_pages, heads, page, dim, steps=(0.01, 0.05)):
    """A GPU cache of random codes with its oracle copy."""
    ref = kv_ref.Cache(rng.integers(1, 256, (n_pages, heads, page, dim), dtype=np.uint8),
                       rng.integers(1, 256, (n_pages, heads, dim, page), dtype=np.uint8),
                       rng.uniform(*steps, (n_pages, heads)), rng.uniform(*steps, (n_pages, heads)))
    dev = awq.KvCache(*(torch.from_numpy(t.copy()).cuda() for t in
                        (ref.k_codes, ref.v_codes, ref.k_steps, ref.v_steps)))
    return dev, ref


def page_table(rng, B, n_pages, per_seq):
    return rng.permutation(n_pages)[: B * per_seq].reshape(B, per_seq).astype(np.int32)


def assert_same_cache(dev, ref):
    np.testing.assert_array_equal(wide(dev.k_steps), ref.k_steps)
    np.testing.assert_array_equal(wide(dev.v_steps), ref.v_steps)
    np.testing.assert_array_equal(dev.k_codes.cpu().numpy(), ref.k_codes)
    np.testing.assert_array_equal(dev.v_codes.cpu().numpy(), ref.v_codes)


APPENDS = [   # new tokens of each sequence, tokens before, kv heads, q heads, D, rot, page
    ([1], [0], 1, 1, 8, 8, 16), ([1], [15], 2, 8, 64, 64, 16), ([1, 1, 1], [16, 0, 37], 8, 8, 128, 128, 32),
    ([5, 0, 70], [3, 9, 60], 2, 4, 96, 48, 32), ([200], [0], 3, 0, 80, 80, 64), ([33, 1], [100, 255], 1, 7, 256, 64, 256),
    ([17, 16, 15], [15, 16, 17], 4, 4, 40, 24, 16), ([129], [127], 2, 2, 128, 128, 128),
    ([64, 300], [64, 20], 1, 2, 72, 72, 64), ([300, 256], [10, 0], 1, 1, 256, 256, 256),
    ([250, 3], [255, 6], 1, 2, 256, 16, 256), ([3], [29], 2, 6, 24, 0, 32),
    ([1, 1], [64, 3], 5, 10, 80, 40, 64), ([90, 2], [6, 31], 2, 6, 80, 40, 64), ([300, 7], [250, 9], 2, 2, 96, 72, 256),
    ([290], [3], 1, 2, 256, 8, 256), ([1], [5], 2, 2, 256, 248, 16), ([1], [5], 2, 2, 64, 6, 16),
]


def steps_alone(new, before):
    """Whether every sequence has one row (then starts may be left out)."""
    return all(n == 1 for n in new)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", APPENDS)
def test_append(shape, kind, interleaved):
    new, before, heads, hq, dim, rot, page = shape
    rng = np.random.default_rng(sum(new) + dim)
    B, T = len(new), sum(new)
    lens = [n + m for n, m in zip(new, before)]
    per_seq = -(-max(lens) // page)
    dev, ref = new_cache(rng, B * per_seq + 2, heads, page, dim)
    table = page_table(rng, B, dev.n_pages, per_seq)
    starts = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    # one projection's output, queries first; a block in two has values that raise the step
    qkv = torch.from_numpy(rng.standard_normal((T, hq + 2 * heads + 1, dim)).astype(f32)
                           * rng.choice([0.3, 30.0], (T, 1, 1)).astype(f32)).to(TYPES[kind]).cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq: hq + heads], qkv[:, hq + heads: -1]
    rope = awq.awq_rope_table(max(lens), rot) if rot else None
    at = np.concatenate([np.arange(m, n) for m, n in zip(before, lens)]).astype(np.int32)
    turn = (lambda x: kv_ref.rope(wide(x), wide(rope), at, interleaved)) if rot else wide
    out = awq.awq_kv_append(dev, k, v, ints(lens), ints(table.tolist()),
                            starts=None if steps_alone(new, before) else ints(starts.tolist()),
                            max_new=max(new), table=rope, interleaved=interleaved,
                            q=q if hq else None, q_dtype=torch.bfloat16 if hq else None)
    if hq:
        np.testing.assert_array_equal(wide(out), rounded(turn(q), "bf16"))
    else:
        assert out is None
    ref.append(turn(k), wide(v), lens, table, starts)
    # places past a sequence's end in a page that it holds are nobody's
    for b, n in enumerate(lens):
        if n % page and new[b]:
            p, t = table[b, n // page], n % page
            ref.k_codes[p, :, t:] = dev.k_codes[p, :, t:].cpu().numpy()
            ref.v_codes[p, :, :, t:] = dev.v_codes[p, :, :, t:].cpu().numpy()
    assert_same_cache(dev, ref)


def test_append_step_by_step_equals_the_oracle_and_reads_back():
    rng = np.random.default_rng(3)
    dev, ref = new_cache(rng, 9, 2, 16, 32, steps=(50.0, 60.0))     # what the pages held before does not count
    table = page_table(rng, 2, 9, 3)
    for n in range(1, 41):
        lens = [n, min(n, 7)] if n > 7 else [n, n]
        B = 1 if n > 7 else 2
        k, v = (torch.from_numpy((rng.standard_normal((B, 2, 32)) * rng.choice([0.1, 1, 5])).astype(f32)).cuda()
                for _ in range(2))
        awq.awq_kv_append(dev, k, v, ints(lens[:B]), ints(table[:B].tolist()))
        ref.append(wide(k), wide(v), lens[:B], table[:B], list(range(B + 1)))
    for dtype in ("f32", "f16", "bf16"):
        k, v = awq.awq_kv_read(dev, ints([1, 0]), ints(table.tolist()), starts=ints([0, 39, 46]), total=46,
                               max_count=39, dtype=TYPES[dtype])
        want = [ref.tokens(0, 1, 40, table), ref.tokens(1, 0, 7, table)]
        np.testing.assert_array_equal(wide(k), rounded(np.concatenate([w[0] for w in want]), dtype))
        np.testing.assert_array_equal(wide(v), rounded(np.concatenate([w[1] for w in want]), dtype))
    k, v = awq.awq_kv_read(dev, ints([39, 6]), ints(table.tolist()))           # one token each
    np.testing.assert_array_equal(wide(k)[1], ref.tokens(1, 6, 7, table)[0][0])
    np.testing.assert_array_equal(wide(v)[0], ref.tokens(0, 39, 40, table)[1][0])


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim,page", [(128, 64), (80, 16), (24, 256), (256, 32)])
def test_read_rounds_the_fp32_product(dim, page, kind):
    """Enough values that one rounding in place of two shows in fp16."""
    rng = np.random.default_rng(dim)
    dev, ref = new_cache(rng, 40, 3, page, dim)
    table = page_table(rng, 2, 40, 20)
    first, count = [5, page], [17 * page, 3 * page + 1]
    k, v = awq.awq_kv_read(dev, ints(first), ints(table.tolist()), starts=ints([0, count[0], sum(count)]),
                           total=sum(count), max_count=max(count), dtype=TYPES[kind])
    want = [ref.tokens(b, first[b], first[b] + count[b], table) for b in range(2)]
    np.testing.assert_array_equal(wide(k), rounded(np.concatenate([w[0] for w in want]), kind))
    np.testing.assert_array_equal(wide(v), rounded(np.concatenate([w[1] for w in want]), kind))


def test_append_with_positions_of_its_own():
    rng = np.random.default_rng(4)
    dev, ref = new_cache(rng, 2, 1, 16, 16)
    rope = awq.awq_rope_table(500, 16)
    k = torch.from_numpy(rng.standard_normal((2, 1, 16)).astype(f32)).cuda()
    at = np.array([499, 0], np.int32)
    q = awq.awq_kv_append(dev, k, k, ints([3, 2]), ints([[0], [1]]), table=rope, positions=ints(at.tolist()), q=k)
    turned = kv_ref.rope(wide(k), wide(rope), at)
    np.testing.assert_array_equal(wide(q), turned)
    ref.append(turned, wide(k), [3, 2], np.array([[0], [1]]), [0, 1, 2])
    np.testing.assert_array_equal(wide(dev.k_steps), ref.k_steps)
    np.testing.assert_array_equal(dev.k_codes[0, 0, :3].cpu().numpy(), ref.k_codes[0, 0, :3])


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_what_is_not_finite_poisons_its_block_alone(bad):
    rng = np.random.default_rng(6)
    dev, ref = new_cache(rng, 4, 2, 16, 16)
    k = torch.from_numpy(rng.standard_normal((20, 2, 16)).astype(f32)).cuda()
    v = k.clone()
    k[17, 1, 3] = bad
    v[2, 0, 15] = bad
    table = np.array([[2, 1]], np.int32)
    awq.awq_kv_append(dev, k, v, ints([20]), ints(table.tolist()), starts=ints([0, 20]), max_new=20)
    ref.append(wide(k), wide(v), [20], table, [0, 20])
    np.testing.assert_array_equal(wide(dev.k_steps), ref.k_steps)
    np.testing.assert_array_equal(wide(dev.v_steps), ref.v_steps)
    q = torch.ones(20, 2, 16, device="cuda", dtype=torch.float16)
    out = wide(awq.awq_kv_attention(dev, q, ints([20]), ints(table.tolist()), starts=ints([0, 20]), max_new=20))
    assert np.isnan(out[:, 0]).all()                     # head 0 sees the bad values' block from its first row on
    assert np.isfinite(out[:16, 1]).all() and np.isnan(out[16:, 1]).all()


def test_append_drops_what_has_no_page_and_keeps_to_its_own():
    rng = np.random.default_rng(8)
    dev, ref = new_cache(rng, 5, 1, 16, 8)
    k = torch.from_numpy(rng.standard_normal((30, 1, 8)).astype(f32)).cuda()
    table = np.array([[-1, 3], [7, 5], [2 ** 30, -2 ** 31]], np.int32)
    starts, lens = [0, 24, 27, 30], [24, 4, 40]          # the last is longer than its table
    awq.awq_kv_append(dev, k, k, ints(lens), ints(table.tolist()), starts=ints(starts), max_new=24)
    ref.append(wide(k), wide(k), lens, table, starts)
    ref.k_codes[3, :, 8:], ref.v_codes[3, :, :, 8:] = dev.k_codes[3, :, 8:].cpu().numpy(), dev.v_codes[3, :, :, 8:].cpu().numpy()
    assert_same_cache(dev, ref)
    kk, vv = awq.awq_kv_read(dev, ints([0, 0, 10]), ints(table.tolist()), starts=ints([0, 24, 28, 68]), total=68,
                             max_count=40)
    assert (wide(kk)[:16] == 0).all() and (wide(vv)[24:] == 0).all()
    np.testing.assert_array_equal(wide(kk)[16:24], ref.tokens(0, 16, 24, table)[0])


# ---------------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------------
ATTENTION = [   # new rows, lengths, q heads, kv heads, D, page
    ([1], [1], 1, 1, 8, 16), ([1], [513], 32, 32, 128, 16), ([1, 1, 1, 1], [0, 1, 64, 777], 8, 1, 128, 64),
    ([1, 1], [1000, 65], 14, 2, 80, 32), ([1, 1, 1], [300, 40, 129], 32, 2, 64, 16), ([1], [515], 48, 2, 128, 128),
    ([1, 1], [700, 31], 4, 4, 256, 256), ([3, 0, 4], [130, 90, 4], 8, 2, 96, 32), ([70, 1, 33], [70, 200, 97], 6, 3, 128, 64),
    ([129], [300], 2, 1, 40, 16), ([5, 2], [333, 90], 16, 2, 256, 64), ([40], [150], 8, 2, 248, 16), ([80], [200], 1, 1, 192, 32), ([20, 5], [10, 5], 4, 2, 64, 16), ([65], [1100], 16, 2, 24, 32),
]


def attention_bound(ref, q, scale, spread, top, out, kind, dim):
    """What the roundings of the kernel can make: the output's own, fp16 probabilities (half an ulp each,
    numerator alone), and scores whose products sum_d q_d c_d (|c| <= 127, exact) carry fp32 roundings:
    (dim / 8 + 4) of the partial sums' size, an absolute error that a probability takes relatively
    (twice: numerator and denominator)."""
    step = top / 127
    score = (dim / 8 + 4) * 2.0 ** -24 * 127 * np.abs(q).sum(-1) * scale * step
    score = score + 8 * 2.0 ** -24 * (np.abs(q).sum(-1) * scale * top + 1)
    rel = 2.0 ** -11 + 2 * np.expm1(2 * score) + 2.0 ** -18
    return score, HALF_ULP[kind] * np.abs(out) + rel[..., None] * spread + TINY[kind]


def check_attention(dev, ref, q, lens, table, starts, kind, window=0, causal=True, scale=None, **kw):
    dim, T = ref.dim, q.shape[0]
    s = dim ** -0.5 if scale is None else scale
    out, lse = awq.awq_kv_attention(dev, q, ints(lens), ints(table.tolist()),
                                    starts=None if starts is None else ints(starts), window=window,
                                    causal=causal, scale=scale, return_lse=True, **kw)
    assert out.dtype == q.dtype and out.shape == q.shape
    st = list(range(len(lens) + 1)) if starts is None else starts
    want, wl, spread, top = ref.attention(wide(q), lens, table, st, s, window, causal)
    score, bound = attention_bound(ref, wide(q), s, spread, top, want, kind, dim)
    most = torch.finfo(q.dtype).max     # an output past the type's range is infinite
    err = np.abs(wide(out).astype(np.float64).clip(-most, most) - want.clip(-most, most))
    assert (err <= bound).all(), (err - bound).max()
    got = wide(lse)
    np.testing.assert_array_equal(np.isneginf(got), np.isneginf(wl))
    fin = np.isfinite(wl)
    assert (np.abs(got[fin] - wl[fin]) <= 2 * score[fin] + 2.0 ** -18 + 2.0 ** -21 * np.abs(wl[fin])).all()
    assert (wide(out)[~fin] == 0).all()
    return out, lse


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("window,causal", [(0, True), (1, True), (37, True), (0, False), (50, False)])
@pytest.mark.parametrize("shape", ATTENTION)
def test_attention(shape, window, causal, kind):
    new, lens, hq, heads, dim, page = shape
    rng = np.random.default_rng(sum(lens) + dim + window)
    B, T = len(new), sum(new)
    per_seq = max(1, -(-max(lens) // page)) + 1
    dev, ref = new_cache(rng, B * per_seq + 1, heads, page, dim)
    table = page_table(rng, B, dev.n_pages, per_seq)
    starts = np.concatenate(([0], np.cumsum(new))).tolist()
    q = torch.from_numpy(rng.standard_normal((T, hq, dim)).astype(f32) * 1.5).to(TYPES[kind]).cuda()
    # nothing past a sequence's end may matter: not codes, not steps that are not numbers
    used = np.zeros(dev.n_pages, bool)
    for b, n in enumerate(lens):
        used[table[b, : -(-n // page)]] = True
    for t in (dev.k_steps, dev.v_steps):
        t[torch.from_numpy(~used).cuda()] = float("nan")
    check_attention(dev, ref, q, lens, table, None if all(n == 1 for n in new) else starts, kind,
                    window, causal, max_new=max(new), max_len=max(max(lens), 1))


@pytest.mark.parametrize("extra", [0, 1, 40])
def test_attention_with_pages_gone_and_loose_limits(extra):
    rng = np.random.default_rng(11)
    dev, ref = new_cache(rng, 40, 2, 32, 64)
    table = page_table(rng, 3, 40, 10)
    table[0, :4] = -1                   # left behind
    table[1, 1::2] = 2 ** 31 - 1
    table[2, :] = -7                    # a sequence without pages sees nothing
    q = torch.from_numpy(rng.standard_normal((3, 8, 64)).astype(f32)).half().cuda()
    check_attention(dev, ref, q, [320, 200, 100], table, None, "f16")
    check_attention(dev, ref, q, [320, 200, 100], table, None, "f16", max_new=1 + extra, max_len=320 + 1000 * extra)
    check_attention(dev, ref, q, [320, 200, 100], table, None, "f16", window=60)


def test_attention_lengths_past_the_table():
    rng = np.random.default_rng(12)
    dev, ref = new_cache(rng, 8, 1, 16, 32)
    table = page_table(rng, 2, 8, 3)
    q = torch.from_numpy(rng.standard_normal((4, 2, 32)).astype(f32)).half().cuda()
    check_attention(dev, ref, q, [60, -3], table, [0, 2, 4], "f16", max_new=2)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_attention_over_steps_far_apart(kind):
    """Blocks whose steps differ by up to 2^60 and blocks of zeros: what counts is what they add."""
    rng = np.random.default_rng(13)
    dev, ref = new_cache(rng, 12, 2, 16, 64)
    table = page_table(rng, 1, 12, 12)
    # keys of zero in some blocks, values of zero, tiny and large in others
    ks, vs = rng.uniform(0.005, 0.02, (12, 2)).astype(f32), (2.0 ** rng.integers(-30, 12, (12, 2))).astype(f32)
    ks[::5] = 0
    vs[::4] = 0
    vs[3] = 2.0 ** -60
    for t, x in ((dev.k_steps, ks), (dev.v_steps, vs)):
        t.copy_(torch.from_numpy(x))
    ref.k_steps[:], ref.v_steps[:] = ks, vs
    q = torch.from_numpy(rng.standard_normal((5, 8, 64)).astype(f32) * 4).to(TYPES[kind]).cuda()
    check_attention(dev, ref, q, [190], table, [0, 5], kind, max_new=5)
    vs[:] = 0
    dev.v_steps.zero_()
    ref.v_steps[:] = 0
    check_attention(dev, ref, q, [190], table, [0, 5], kind, max_new=5)


def test_attention_of_small_and_large_queries():
    rng = np.random.default_rng(14)
    dev, ref = new_cache(rng, 8, 1, 32, 64)
    table = page_table(rng, 1, 8, 8)
    q = torch.from_numpy(rng.standard_normal((6, 4, 64)).astype(f32)
                         * np.array([1e-30, 1e-6, 1, 30, 1e4, 0])[:, None, None].astype(f32)).bfloat16().cuda()
    # large ones all but pick a token: the scale keeps the scores' rounding in bounds
    check_attention(dev, ref, q, [250], table, [0, 6], "bf16", max_new=6, scale=1e-3)
    check_attention(dev, ref, q, [250], table, [0, 6], "bf16", max_new=6, scale=0.0)


def test_attention_of_a_query_that_is_not_finite_stays_in_its_row():
    rng = np.random.default_rng(15)
    dev, ref = new_cache(rng, 8, 2, 32, 64)
    table = page_table(rng, 2, 8, 3)
    q = torch.from_numpy(rng.standard_normal((6, 4, 64)).astype(f32)).half().cuda()
    clean = awq.awq_kv_attention(dev, q, ints([70, 90]), ints(table.tolist()), starts=ints([0, 3, 6]), max_new=3)
    q2 = q.clone()
    q2[1, 2, 7] = float("nan")
    q2[4, 0, 0] = float("inf")
    out = awq.awq_kv_attention(dev, q2, ints([70, 90]), ints(table.tolist()), starts=ints([0, 3, 6]), max_new=3)
    assert torch.isnan(out[1, 2]).all()
    out[1, 2], out[4, 0] = clean[1, 2], clean[4, 0]
    assert torch.equal(out, clean)


def test_attention_strides_stream_and_repeat():
    rng = np.random.default_rng(16)
    dev, ref = new_cache(rng, 20, 2, 32, 128)
    table = page_table(rng, 2, 20, 10)
    big = torch.from_numpy(rng.standard_normal((2, 13, 128)).astype(f32)).bfloat16().cuda()
    q = big[:, 2:10]
    out, lse = check_attention(dev, ref, q, [300, 211], table, None, "bf16")
    odd = torch.from_numpy(rng.standard_normal(2 * 8 * 128 + 1).astype(f32)).bfloat16().cuda()
    check_attention(dev, ref, odd[1:].view(8, 2, 128).transpose(0, 1), [300, 211], table, None, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = awq.awq_kv_attention(dev, q, ints([300, 211]), ints(table.tolist()))
    side.synchronize()
    assert torch.equal(again, out)
    for _ in range(3):
        o, l = awq.awq_kv_attention(dev, q, ints([300, 211]), ints(table.tolist()), return_lse=True)
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_attention_long_and_split():
    rng = np.random.default_rng(17)
    dev, ref = new_cache(rng, 160, 1, 64, 64)
    table = page_table(rng, 1, 160, 157)
    q = torch.from_numpy(rng.standard_normal((1, 8, 64)).astype(f32)).half().cuda()
    check_attention(dev, ref, q, [10000], table, None, "f16")
    check_attention(dev, ref, q, [10000], table, None, "f16", window=4097)


UNEVEN = [   # sequences, rows of each, shortest, longest, q heads, kv heads, D, page, window
    (3, 1, 1, 2300, 8, 2, 64, 64, 0), (300, 1, 0, 1100, 4, 1, 32, 16, 0), (40, 1, 700, 1500, 6, 6, 64, 128, 0),
    (7, 3, 2, 1300, 16, 2, 40, 32, 0), (5, 2, 600, 1800, 24, 1, 128, 64, 900), (2, 45, 700, 1400, 4, 2, 64, 16, 0), (256, 1, 1, 800, 2, 2, 16, 32, 0), (257, 2, 0, 5000, 2, 1, 8, 256, 4700),
    (1, 40, 2500, 2500, 4, 1, 64, 64, 0), (1, 33, 1100, 1100, 3, 1, 96, 64, 300), (600, 1, 0, 700, 1, 1, 16, 64, 0),
]


@pytest.mark.parametrize("shape", UNEVEN)
def test_attention_of_uneven_sequences(shape):
    """Splits that the device chooses by the lengths, sequences of every length among them."""
    B, n, lo, hi, hq, heads, dim, page, window = shape
    rng = np.random.default_rng(B + hi)
    lens = rng.permutation(np.linspace(max(lo, n if lo else 0), hi, B).astype(int)).tolist()
    per_seq = -(-hi // page)
    dev, ref = new_cache(rng, min(B * per_seq, 3000) + 1, heads, page, dim)
    table = np.full((B, per_seq), -1, np.int32)
    free = rng.permutation(dev.n_pages)
    at = 0
    for b, length in enumerate(lens):      # only the pages that a sequence holds; read pages may be shared
        held = -(-length // page)
        table[b, :held] = free[(at + np.arange(held)) % dev.n_pages]
        at += held
    q = torch.from_numpy(rng.standard_normal((B * n, hq, dim)).astype(f32)).half().cuda()
    starts = None if n == 1 else (np.arange(B + 1) * n).tolist()
    check_attention(dev, ref, q, lens, table, starts, "f16", window, max_new=n, max_len=hi)


@pytest.mark.parametrize("longest", [515, 1030, 2051])
def test_attention_whose_last_rows_alone_reach_another_split(longest):
    """64 rows of a head in two row tiles: the tokens that only the second one sees begin a split."""
    rng = np.random.default_rng(longest)
    lens = [longest, 513, 600, 1025, 8]
    dev, ref = new_cache(rng, 5 * 33, 1, 64, 32)
    table = page_table(rng, 5, 165, 33)
    q = torch.from_numpy(rng.standard_normal((40, 8, 32)).astype(f32)).half().cuda()
    check_attention(dev, ref, q, lens, table, list(range(0, 41, 8)), "f16", max_new=8, max_len=max(lens))


def test_cache_past_four_gibibytes():
    """Pages whose codes lie beyond a 32-bit offset."""
    n, heads, page, dim = 5 * (1 << 30) // (2 * 128 * 128), 2, 128, 128
    dev = awq.KvCache.empty(n, heads, page, dim)
    rng = np.random.default_rng(18)
    table = np.array([[n - 1, 3, n - 2]], np.int32)
    k, v = (torch.from_numpy(rng.standard_normal((300, heads, dim)).astype(f32)).bfloat16().cuda() for _ in range(2))
    awq.awq_kv_append(dev, k, v, ints([300]), ints(table.tolist()), starts=ints([0, 300]), max_new=300)
    small = kv_ref.Cache(np.zeros((3, heads, page, dim), np.uint8), np.zeros((3, heads, dim, page), np.uint8),
                         np.zeros((3, heads)), np.zeros((3, heads)))
    t3 = np.array([[0, 1, 2]])
    small.append(wide(k), wide(v), [300], t3, [0, 300])
    kk, vv = awq.awq_kv_read(dev, ints([0]), ints(table.tolist()), starts=ints([0, 300]), total=300)
    want = small.tokens(0, 0, 300, t3)
    np.testing.assert_array_equal(wide(kk), want[0])
    np.testing.assert_array_equal(wide(vv), want[1])
    q = torch.from_numpy(rng.standard_normal((1, 4, dim)).astype(f32)).bfloat16().cuda()
    got = awq.awq_kv_attention(dev, q, ints([300]), ints(table.tolist()))
    out, _, spread, top = small.attention(wide(q), [300], t3, [0, 1], dim ** -0.5)
    _, bound = attention_bound(small, wide(q), dim ** -0.5, spread, top, out, "bf16", dim)
    assert (np.abs(wide(got) - out) <= bound).all()


def test_decode_step_in_a_graph():
    """Append, attention and read captured once and replayed as the sequences grow on the device."""
    rng = np.random.default_rng(19)
    dev, ref = new_cache(rng, 12, 2, 16, 64)
    table = page_table(rng, 2, 12, 5)
    rope = awq.awq_rope_table(128, 64)
    qkv = torch.zeros(2, 8, 64, device="cuda", dtype=torch.float16)
    lens, pages = ints([30, 47]), ints(table.tolist())
    q_out, out = torch.empty(2, 4, 64, device="cuda", dtype=torch.float16), None
    ws = torch.empty(max(1, awq.awq_kv_attention_workspace_size(2, 2, 4, 2, 64, 1, 80)), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q_out)

    def step():
        awq.awq_kv_append(dev, qkv[:, 4:6], qkv[:, 6:], lens, pages, table=rope, q=qkv[:, :4], q_out=q_out)
        awq.awq_kv_attention(dev, q_out, lens, pages, max_len=80, out=out, workspace=ws)

    twin = awq.KvCache(*(t.clone() for t in (dev.k_codes, dev.v_codes, dev.k_steps, dev.v_steps)))
    step()
    for a, b in ((dev.k_codes, twin.k_codes), (dev.v_codes, twin.v_codes), (dev.k_steps, twin.k_steps),
                 (dev.v_steps, twin.v_steps)):
        a.copy_(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for a, b in ((dev.k_codes, twin.k_codes), (dev.v_codes, twin.v_codes), (dev.k_steps, twin.k_steps),
                 (dev.v_steps, twin.v_steps)):
        a.copy_(b)
    for i in range(6):
        qkv.copy_(torch.from_numpy(rng.standard_normal((2, 8, 64)).astype(f32) * (i + 1)).half())
        lens += 1
        graph.replay()
        torch.cuda.synchronize()
        q = awq.awq_kv_append(twin, qkv[:, 4:6], qkv[:, 6:], lens, pages, table=rope, q=qkv[:, :4])
        want = awq.awq_kv_attention(twin, q, lens, pages, max_len=80)
        torch.cuda.synchronize()
        assert torch.equal(q, q_out) and torch.equal(want, out)
    assert torch.equal(dev.k_codes, twin.k_codes) and torch.equal(dev.v_codes, twin.v_codes)


@pytest.mark.parametrize("call", [
    lambda c, q, l, p: awq.awq_kv_attention(c, q.float(), l, p),
    lambda c, q, l, p: awq.awq_kv_attention(c, q[..., :8], l, p),
    lambda c, q, l, p: awq.awq_kv_attention(c, q[:, :3], l, p),
    lambda c, q, l, p: awq.awq_kv_attention(c, q, l.long(), p),
    lambda c, q, l, p: awq.awq_kv_attention(c, q, l, p[0]),
    lambda c, q, l, p: awq.awq_kv_attention(c, q, l[:1], p),
    lambda c, q, l, p: awq.awq_kv_attention(c, q, l, p, scale=-1.0),
    lambda c, q, l, p: awq.awq_kv_attention(c, q, l, p, window=-1),
    lambda c, q, l, p: awq.awq_kv_attention(c, q, l, p, out=q.float()),
    lambda c, q, l, p: awq.awq_kv_append(c, q[:, :1], q[:, :1], l, p),
    lambda c, q, l, p: awq.awq_kv_append(c, q[:, :2], q[:, :2].float(), l, p),
    lambda c, q, l, p: awq.awq_kv_append(c, q[:, :2], q[:, :2], l, p, starts=p[0]),
    lambda c, q, l, p: awq.awq_kv_append(c, q[:, :2], q[:, :2], l, p, q_out=q),
    lambda c, q, l, p: awq.awq_kv_read(c, l, p, starts=l),
])
def test_cache_binding_refuses(call):
    cache = awq.KvCache.empty(4, 2, 16, 16)
    q = torch.zeros(2, 4, 16, device="cuda", dtype=torch.float16)
    with pytest.raises((ValueError, awq.AwqError)):
        call(cache, q, ints([1, 1]), ints([[0], [1]]))
