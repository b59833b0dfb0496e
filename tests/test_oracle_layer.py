"""Pins of the oracle of the convolution, the rotation and the attention of packed rows (CPU)."""
import math

import numpy as np
import pytest

from oracle import layer as Y
from oracle import sequence as S


def test_conv_by_hand():
    w = np.array([[1.0, 10.0, 100.0]])  # the newest input's tap last
    y, _, _, state = Y.conv(np.array([[1.0], [2.0]]), np.array([[3.0], [4.0]]), w, np.array([0.5]), False)
    assert y.tolist() == [[3 + 40 + 100 + 0.5], [4 + 10 + 200 + 0.5]]
    assert state.tolist() == [[1.0], [2.0]]


@pytest.mark.parametrize("L", [0, 1, 2, 3, 9])
def test_conv_is_a_convolution(L):
    rng = np.random.default_rng(L)
    u, s, w, b = rng.normal(size=(L, 5)), rng.normal(size=(3, 5)), rng.normal(size=(5, 4)), rng.normal(size=5)
    y, _, raw, state = Y.conv(u, s, w, b, True)
    both = np.concatenate([s, u])
    for c in range(5):
        want = np.convolve(both[:, c], w[c, ::-1], "valid") + b[c]
        assert np.allclose(raw[:, c], want[len(want) - L:], atol=1e-13)
    assert np.allclose(y, raw * 0.5 * (1 + np.tanh(raw / 2)), atol=1e-13)
    assert np.array_equal(state, both[-3:])


def test_rope_turns_pairs():
    x = np.array([[3.0, 0.0, 0.0, 2.0, 7.0]])
    out, _ = Y.rope(x, 1, [math.pi / 2, math.pi], None, 0.0, False)  # pairs (0, 2) by a quarter, (1, 3) by a half
    assert np.allclose(out, [[0, 0, 3, -2, 7]], atol=1e-15)
    out, _ = Y.rope(x, 1, [math.pi / 2, math.pi], None, 0.0, True)  # pairs (0, 1) and (2, 3)
    assert np.allclose(out, [[0, 3, 0, -2, 7]], atol=1e-15)


def test_rope_depends_on_distance_alone():
    rng = np.random.default_rng(1)
    q, k, f = rng.normal(size=(1, 8)), rng.normal(size=(1, 8)), 10.0 ** -np.arange(4.0)
    dots = [(Y.rope(q, p + 5, f, None, 0, il)[0] * Y.rope(k, p, f, None, 0, il)[0]).sum() for p in (0, 3, 40) for il in (False, True)]
    assert np.allclose(dots[::2], dots[0]) and np.allclose(dots[1::2], dots[1])


def test_norm_has_unit_mean_square():
    x = np.random.default_rng(2).normal(size=(3, 16))
    out, _ = Y.rope(x, 9, [0.3], np.ones(16), 0.0, False)
    assert np.allclose((out ** 2).mean(-1), 1)
    twice, _ = Y.rope(5 * x, 9, [0.3], 2 * np.ones(16), 0.0, False)
    assert np.allclose(twice, 2 * out)


def test_sees():
    assert [j for j in range(12) if Y.sees(9, j, 3, 2)] == [0, 1, 7, 8, 9]
    assert [j for j in range(12) if Y.sees(9, j, 0, 0)] == list(range(10))
    assert [j for j in range(12) if Y.sees(1, j, 3, 4)] == [0, 1]


def test_attend_is_the_tree_attention_of_a_chain():
    rng = np.random.default_rng(3)
    q, kc, vc = rng.normal(size=(6, 4, 8)), rng.normal(size=(15, 2, 8)), rng.normal(size=(15, 2, 8))
    want = S.attend(q, kc[9:], vc[9:], np.arange(-1, 5), kc[:9], vc[:9], 0.3)
    got = Y.attend(q, 9, kc, vc, 0.3)
    for a, b in zip(got, want):
        assert np.allclose(a, b, atol=1e-13)
    # a window as long as all positions changes nothing; one of a single position leaves a row its own value
    assert np.allclose(Y.attend(q, 9, kc, vc, 0.3, window=15)[0], got[0], atol=1e-13)
    assert np.allclose(Y.attend(q, 9, kc, vc, 0.3, window=1)[0], np.repeat(vc[9:], 2, 1))
