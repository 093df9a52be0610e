"""Pins of the oracle of a block of experts (CPU): hand-worked examples, identities, gradients
against differences."""

import numpy as np
import pytest

from oracle import awq_ref, moe_ref as ref


def test_choice_by_hand():
    logits = np.array([[1.0, 3.0, 2.0, 3.0], [-0.0, 0.0, -np.inf, np.nan]])
    assert ref.choose(logits, 3).tolist() == [[1, 3, 2], [0, 1, 2]]
    # sigmoid: 0.5, 0.731; the bias turns them round
    assert ref.choose(np.array([[0.0, 1.0]]), 1, "sigmoid", bias=[0.25, 0.0]).tolist() == [[0]]
    assert ref.choose(np.array([[0.0, 1.0]]), 1, "softmax", bias=[0.25, 0.0]).tolist() == [[1]]


def test_weights_by_hand():
    logits = np.log(np.array([[1.0, 2.0, 5.0]]))
    e = np.array([[2, 1]])
    np.testing.assert_allclose(ref.route_weights(logits, e, normalise=False), [[5 / 8, 2 / 8]])
    np.testing.assert_allclose(ref.route_weights(logits, e, scale=2.0), [[10 / 7, 4 / 7]])
    # sigmoid(log v) = v / (1 + v)
    np.testing.assert_allclose(ref.route_weights(logits, e, "sigmoid", False), [[5 / 6, 2 / 3]])
    np.testing.assert_allclose(ref.route_weights(logits, e, "sigmoid"), [[5 / 9, 4 / 9]])
    assert ref.route_weights(np.full((1, 3), -np.inf), e).tolist() == [[0, 0]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalise", [True, False])
def test_route_gradient_is_the_differences(score, normalise):
    rng = np.random.default_rng(3)
    logits, g = rng.normal(size=(4, 9)), rng.normal(size=(4, 3))
    e = ref.choose(logits, 3, score)
    got = ref.route_grad(logits, e, g, score, normalise, 1.7)
    for t in range(4):
        for c in range(9):
            ends = []
            for h in (1e-6, -1e-6):
                moved = logits.copy()
                moved[t, c] += h
                ends.append((ref.route_weights(moved, e, score, normalise, 1.7) * g).sum())
            # central differences: h^2 / 6 times a third derivative of order 1, and 2^-53 / h
            assert abs((ends[0] - ends[1]) / 2e-6 - got[t, c]) < 1e-8


def test_sort_by_hand():
    experts = np.array([[2, 0], [0, 7], [2, 1], [-1, 0]])
    offsets, order, place = ref.sort_pairs(experts, 0, 3)
    assert offsets.tolist() == [0, 3, 4, 6]
    assert order.tolist() == [1, 2, 7, 5, 0, 4, 3, 6]
    assert place.tolist() == [[4, 0], [1, 6], [5, 3], [7, 2]]
    offsets, order, _ = ref.sort_pairs(experts, 1, 2)
    assert offsets.tolist() == [0, 1, 3] and order.tolist()[:3] == [5, 0, 4]


def test_rows_there_and_back():
    rng = np.random.default_rng(4)
    experts = np.stack([rng.permutation(6)[:3] for _ in range(7)])
    offsets, order, place = ref.sort_pairs(experts, 1, 4)
    x, r, w = rng.normal(size=(7, 5)), rng.normal(size=(21, 5)), rng.normal(size=(7, 3))
    out = ref.gather(x, offsets, place, w)
    for row in range(21):
        t, j = divmod(order[row], 3)
        want = x[t] * w[t, j] if 1 <= experts[t, j] < 5 else 0 * x[t]
        np.testing.assert_array_equal(out[row], want)
    # each is the other's transpose, and weights' gradient the products of the pairs
    a, b = (out * r).sum(), (x * ref.combine(r, offsets, place, w)).sum()
    c = (ref.dots(x, r, offsets, place) * w).sum()
    assert abs(a - b) < 1e-12 and abs(a - c) < 1e-12
    np.testing.assert_allclose(ref.combine(r, offsets, place, w, x), x + ref.combine(r, offsets, place, w))


def test_activations():
    v = np.array([-3.0, -1.0, 0.0, 0.5, 2.0])
    assert ref.activate(v, "relu").tolist() == [0, 0, 0, 0.5, 2.0]
    np.testing.assert_allclose(ref.activate(v, "silu"), v * (1 + np.tanh(v / 2)) / 2)
    # gelu: v times the normal distribution's integral; 0.84134474 at 1
    assert abs(ref.activate(np.array([1.0]), "gelu")[0] - 0.8413447460685429) < 1e-15
    assert np.abs(ref.activate(v, "gelu_tanh") - ref.activate(v, "gelu")).max() < 1e-3
    y = ref.finish(np.array([[1.0, -2.0, 3.0, 4.0]]), "relu", gated=True, residual=np.array([[10.0, 20.0]]))
    assert y.tolist() == [[13.0, 20.0]]


@pytest.mark.parametrize("bits", range(2, 9))
def test_packed_weights_read_back(bits):
    rng = np.random.default_rng(bits)
    codes = rng.integers(0, 2 ** bits, size=(5, 96)).astype(np.uint8)
    steps, zeros = rng.random((5, 3)).astype(np.float32), rng.integers(0, 2 ** bits, size=(5, 3))
    words, meta = ref.repack(codes, steps, zeros, bits)
    assert words.shape == (3, 5, bits) and meta.shape == (3, 5, 2)
    W = ref.weights_of(codes, steps, zeros, 32)
    for n in range(5):
        for k in range(96):
            stream = sum(int(w) << (32 * i) for i, w in enumerate(words[k // 32, n]))
            c = (stream >> (bits * (k % 32))) & (2 ** bits - 1)
            assert c == codes[n, k]
            assert W[n, k] == (c - float(meta[k // 32, n, 1])) * float(meta[k // 32, n, 0])
    np.testing.assert_array_equal(awq_ref.unpack_codes(awq_ref.pack_codes(codes, bits), bits, 96), codes)


def test_experts_product():
    rng = np.random.default_rng(9)
    W, x = rng.normal(size=(3, 4, 8)), rng.normal(size=(5, 8))
    v = ref.experts_product(x, W, np.array([0, 2, 2, 4]), source=[0, 0, 4, 1, 2])
    np.testing.assert_allclose(v, np.stack([W[0] @ x[0], W[0] @ x[0], W[2] @ x[4], W[2] @ x[1], np.zeros(4)]))
