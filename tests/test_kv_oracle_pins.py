"""The oracle of the rotary positions, the 8-bit cache and its attention, on cases whose answers
are known by hand or by another route (CPU)."""

import numpy as np
import pytest

from oracle import kv_ref

f32 = np.float32


def test_frequencies_by_hand():
    np.testing.assert_allclose(kv_ref.rope_frequencies(4, base=100.0), [1.0, 0.1])
    np.testing.assert_allclose(kv_ref.rope_frequencies(4, base=100.0, scaling="linear", factor=4),
                               [0.25, 0.025])
    # 2 pi 100 positions: the pairs make 100 and 10 turns; between 1 and 19 the second keeps a half
    kw = dict(base=100.0, factor=4, original=2 * np.pi * 100, low=1.0, high=19.0)
    np.testing.assert_allclose(kv_ref.rope_frequencies(4, scaling="turns", **kw),
                               [1.0, 0.5 * 0.1 + 0.5 * 0.025])
    # between 1 and 100 turns, ten lie half way on the logarithm
    kw["high"] = 100.0
    np.testing.assert_allclose(kv_ref.rope_frequencies(4, scaling="log_turns", **kw),
                               [1.0, 0.5 * 0.1 + 0.5 * 0.025])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_depends_on_distance(interleaved):
    rng = np.random.default_rng(1)
    table = kv_ref.rope_table(50, 12)
    q, k = rng.standard_normal((2, 1, 3, 16))
    turned = {p: kv_ref.rope(k, table, [p], interleaved) for p in (3, 20)}
    np.testing.assert_allclose(np.linalg.norm(turned[3], axis=-1), np.linalg.norm(k, axis=-1))
    a = (kv_ref.rope(q, table, [7], interleaved) * turned[3]).sum(-1)
    b = (kv_ref.rope(q, table, [24], interleaved) * turned[20]).sum(-1)
    np.testing.assert_allclose(a, b)
    np.testing.assert_array_equal(kv_ref.rope(k, table, [0], interleaved), k)
    np.testing.assert_array_equal(turned[3][..., 12:], k[..., 12:])


def test_quarter_turn_by_hand():
    table = np.array([[[0.0, 1.0], [1.0, 0.0]]])
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    np.testing.assert_array_equal(kv_ref.rope(x, table, [0]), [[[-3.0, 2.0, 1.0, 4.0, 5.0]]])
    np.testing.assert_array_equal(kv_ref.rope(x, table, [0], interleaved=True),
                                  [[[-2.0, 1.0, 3.0, 4.0, 5.0]]])


@pytest.mark.parametrize("interleaved", [False, True])
def test_transpose_is_the_gradient_by_differences(interleaved):
    rng = np.random.default_rng(2)
    table = kv_ref.rope_table(9, 6, magnitude=1.3)
    x, g = rng.standard_normal((2, 2, 1, 8))
    got = kv_ref.rope(g, table, [4, 8], interleaved, transpose=True)
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = 0.5     # the map is linear: the difference is exact but for rounding
        d = ((kv_ref.rope(x + e, table, [4, 8], interleaved)
              - kv_ref.rope(x - e, table, [4, 8], interleaved)) * g).sum()
        assert abs(d - got[at]) < 1e-12


def cache(pages=3, heads=1, page=16, dim=8):
    return kv_ref.Cache(np.full((pages, heads, page, dim), 255, np.uint8),
                        np.full((pages, heads, dim, page), 255, np.uint8),
                        np.full((pages, heads), np.nan), np.full((pages, heads), np.nan))


def test_append_moves_older_codes_to_a_larger_step():
    c, table = cache(), np.array([[2, 0]])
    one = np.zeros((1, 1, 8), f32)
    one[0, 0, :2] = [127, -64]
    c.append(one, one / 2, [1], table, [0, 1])
    assert c.k_steps[2, 0] == 1 and c.v_steps[2, 0] == 0.5
    assert c.k_codes[2, 0, 0, :3].tolist() == [255, 64, 128]
    two = np.zeros((1, 1, 8), f32)
    two[0, 0, 3] = 254                                     # the step doubles
    c.append(two, one * 0, [2], table, [0, 1])
    assert c.k_steps[2, 0] == 2 and c.v_steps[2, 0] == 0.5
    # rint(63.5) = 64 and rint(-32) = -32
    assert c.k_codes[2, 0, 0, :3].tolist() == [192, 96, 128]
    assert c.k_codes[2, 0, 1, 3] == 255 and c.v_codes[2, 0, 0, 1] == 128
    assert c.v_codes[2, 0, :3, 0].tolist() == [255, 64, 128]


def test_append_of_zeros_and_of_what_is_not_finite():
    c, table = cache(), np.array([[1]])
    c.append(np.zeros((1, 1, 8), f32), np.zeros((1, 1, 8), f32), [1], table, [0, 1])
    assert c.k_steps[1, 0] == 0 and (c.k_codes[1, 0, 0] == 128).all()
    x = np.ones((1, 1, 8), f32)
    x[0, 0, 5] = np.nan
    c.append(x, np.full((1, 1, 8), np.inf, f32), [2], table, [0, 1])
    assert np.isnan(c.k_steps[1, 0]) and np.isinf(c.v_steps[1, 0])
    k, v, there = c.tokens(0, 0, 2, table)
    assert np.isnan(k).all() and np.isnan(v).all() and there.all()


def test_attention_by_hand():
    c, table = cache(dim=8), np.array([[0, 1]])
    v = np.zeros((20, 1, 8), f32)
    v[:, 0, 0] = 127 - 2 * np.arange(20)     # representable: page steps divide them
    v[16, 0, 0], v[0, 0, 0] = 127, 127
    c.append(np.ones((20, 1, 8), f32), v, [20], table, [0, 20])
    q = np.zeros((2, 2, 8))
    out, lse, _, _ = c.attention(q, [20], table, [0, 2], 1.0)       # equal weights
    np.testing.assert_allclose(out[0, :, 0], v[:19, 0, 0].mean())
    np.testing.assert_allclose(out[1, :, 0], v[:, 0, 0].mean())
    np.testing.assert_allclose(lse, np.log([[19, 19], [20, 20]]))
    out, lse, _, _ = c.attention(q, [20], table, [0, 2], 1.0, window=1)
    np.testing.assert_allclose(out[:, 0, 0], v[18:, 0, 0])
    out, lse, _, _ = c.attention(q, [0], table, [0, 2], 1.0)        # nothing to see
    assert (out == 0).all() and np.isneginf(lse).all()
    out, lse, _, _ = c.attention(q, [20], np.array([[-1, 1]]), [0, 2], 1.0)   # first page gone
    np.testing.assert_allclose(out[1, 0, 0], v[16:, 0, 0].mean())
