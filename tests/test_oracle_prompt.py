"""Pins of the prompt path's oracle: closed forms, published values and independent formulations."""
import math

import numpy as np
import pytest
from scipy.special import logsumexp, softmax

from oracle import prompt as O


def test_frequencies_plain_and_linear():
    f, a = O.frequencies(8, 10000.0)
    assert a == 1.0 and np.allclose(f, [1.0, 0.1, 0.01, 0.001], rtol=1e-12)
    g, a = O.frequencies(8, 10000.0, "linear", 4.0)
    assert a == 1.0 and np.allclose(g, f / 4, rtol=1e-12)


def test_frequencies_of_long_contexts():
    """YaRN: pairs that turn more than beta_fast times over the original length keep their frequency, those that turn
    less than beta_slow times are slowed by the whole factor, and in between the share falls along a line."""
    dim, base, factor, orig = 64, 10000.0, 8.0, 4096.0
    f, _ = O.frequencies(dim, base)
    g, a = O.frequencies(dim, base, "yarn", factor, orig)
    assert a == pytest.approx(0.1 * math.log(8) + 1)
    turns = orig * f / (2 * math.pi)
    assert np.allclose(g[turns > 40], f[turns > 40], rtol=1e-12) and (turns > 40).any()
    assert np.allclose(g[turns < 0.7], f[turns < 0.7] / factor, rtol=1e-12) and (turns < 0.7).any()
    share = (g / f - 1) / (1 / factor - 1)
    step = np.diff(share)
    inside = (share[:-1] > 0) & (share[1:] < 1)
    assert np.all(step >= -1e-12) and np.ptp(step[inside]) < 1e-9


@pytest.mark.parametrize("half", [False, True])
def test_rotation_by_hand(half):
    f = np.array([math.pi / 2, math.pi / 6])
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    pairs = [(0, 2), (1, 3)] if half else [(0, 1), (2, 3)]
    y = O.rotate(x, [1], f, 1.0, half)[0, 0]
    a, b = pairs[0]
    assert y[a] == pytest.approx(-x[0, 0, b]) and y[b] == pytest.approx(x[0, 0, a])           # a quarter turn
    a, b = pairs[1]
    c, s = math.sqrt(3) / 2, 0.5
    assert y[a] == pytest.approx(c * x[0, 0, a] - s * x[0, 0, b]) and y[b] == pytest.approx(c * x[0, 0, b] + s * x[0, 0, a])
    assert np.array_equal(O.rotate(x, [0], f, 1.0, half), x)
    assert np.allclose(O.rotate(x, [0], f, 1.5, half), 1.5 * x)


@pytest.mark.parametrize("half", [False, True])
def test_rotation_keeps_lengths_and_depends_on_distances(half):
    g = np.random.default_rng(1)
    f, _ = O.frequencies(64, 10000.0)
    q, k = g.normal(size=(1, 3, 64)), g.normal(size=(1, 3, 64))
    assert np.allclose(np.linalg.norm(O.rotate(q, [777], f, 1, half)), np.linalg.norm(q))
    near = (O.rotate(q, [40], f, 1, half) * O.rotate(k, [7], f, 1, half)).sum(-1)
    far = (O.rotate(q, [100040], f, 1, half) * O.rotate(k, [100007], f, 1, half)).sum(-1)
    assert np.allclose(near, far, atol=1e-9)


def test_complex_form():
    """The interleaved pairs as complex numbers times exp(i angle)."""
    g = np.random.default_rng(2)
    f, _ = O.frequencies(32, 500.0)
    x = g.normal(size=(4, 2, 32))
    pos = [0, 3, 1000, 65535]
    z = x[..., 0::2] + 1j * x[..., 1::2]
    z = z * np.exp(1j * np.array(pos)[:, None, None] * f)
    y = O.rotate(x, pos, f, 1.0, False)
    assert np.allclose(y[..., 0::2], z.real, atol=1e-9) and np.allclose(y[..., 1::2], z.imag, atol=1e-9)


def test_rms_norm():
    x = np.array([[3.0, -4.0], [0.0, 0.0]])
    y = O.rms_norm(x, np.array([1.0, 2.0]), 0.0 + 1e-30)
    assert np.allclose(y[0], [3 / math.sqrt(12.5), -8 / math.sqrt(12.5)]) and np.array_equal(y[1], [0, 0])
    assert np.allclose(O.rms_norm(x, np.ones(2), 12.5)[0], x[0] / 5)


@pytest.mark.parametrize("causal", [False, True])
def test_attention_against_scipy(causal):
    g = np.random.default_rng(3)
    q, k, v = g.normal(size=(5, 4, 16)), g.normal(size=(9, 2, 16)), g.normal(size=(9, 2, 8))
    out, lse = O.attend(q, k, v, 0.25, causal)
    for h in range(4):
        s = 0.25 * q[:, h] @ k[:, h // 2].T
        if causal:
            s = np.where(np.tri(5, 9, 4, dtype=bool), s, -np.inf)
        assert np.allclose(lse[:, h], logsumexp(s, axis=1), atol=1e-12)
        assert np.allclose(out[:, h], softmax(s, axis=1) @ v[:, h // 2], atol=1e-12)


def test_attention_closed_forms():
    one = np.ones((1, 1, 4))
    out, lse = O.attend(one, 2 * one, np.arange(4.0).reshape(1, 1, 4), 0.5, True)
    assert np.array_equal(out[0, 0], np.arange(4.0)) and lse[0, 0] == 4.0          # one key: its value, its score
    v = np.random.default_rng(4).normal(size=(6, 1, 4))
    out, lse = O.attend(np.zeros((3, 1, 4)), np.ones((6, 1, 4)), v, 1.0, True)
    for i in range(3):                                                             # equal scores: the mean of those seen
        assert np.allclose(out[i, 0], v[:4 + i, 0].mean(0)) and lse[i, 0] == pytest.approx(math.log(4 + i))
    out, lse = O.attend(np.ones((3, 1, 4)), np.ones((1, 1, 4)), v[:1], 1.0, True)  # two rows see nothing
    assert not out[:2].any() and np.all(np.isneginf(lse[:2])) and np.array_equal(out[2, 0], v[0, 0])
    out, lse = O.attend(np.ones((2, 1, 4)), np.ones((0, 1, 4)), v[:0], 1.0, False)
    assert not out.any() and np.all(np.isneginf(lse))
