"""Pins for the block oracle: hand-computed means and scores, and attention over lists against the
contiguous fp64 definition."""
import numpy as np
import pytest

from oracle import attend as OA
from oracle import blocks as K


def _bits(x):
    return (np.ascontiguousarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def _values(b):
    return (b.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def test_block_keys_by_hand():
    lat, rope = np.zeros((130, 512)), np.zeros((130, 64))
    lat[:, 0] = np.arange(130)
    rope[128:, 63] = [3.0, 5.0]
    k = K.block_keys(lat, rope)
    assert k.shape == (3, 576)
    assert k[:, 0].tolist() == [31.5, 95.5, 128.5] and k[2, 575] == 4.0 and k[0, 575] == 0.0


def test_block_scores_by_hand():
    keys = np.zeros((4, 576))
    keys[:, 0] = [1.0, -1.0, 2.0, 4.0]
    q = np.zeros((2, 2, 576))
    q[:, 0, 0], q[:, 1, 0] = 1.0, -3.0      # head 0 likes positive keys, head 1 negative ones
    # rows at positions 191 and 192: own blocks 2 and 3
    x = K.block_scores(q, keys, 193, None, 0.5, 0, 1)
    assert x[0].tolist() == [0.5, 1.5, np.inf, -np.inf]
    assert x[1].tolist() == [0.5, 1.5, 1.0, np.inf]
    w = np.array([[2.0, -1.0], [0.0, 1.0]])
    x = K.block_scores(q, keys, 193, w, 0.5, 1, 1)
    assert x[0].tolist() == [np.inf, -1.5, np.inf, -np.inf]
    assert x[1].tolist() == [np.inf, 1.5, 0.0, np.inf]


def test_rows_of_a_list():
    assert K.rows_of_list([1, -1, 0], 66).tolist() == [64, 65, 66] + list(range(64))
    assert K.rows_of_list([3, -1], 66).tolist() == []


@pytest.mark.parametrize("seed", range(3))
def test_attend_rows_is_the_contiguous_definition(seed):
    g = np.random.default_rng(seed)
    lat, rope, q = (_bits(g.standard_normal(s)) for s in ((200, 512), (200, 64), (3, 576)))
    rows = g.permutation(200)[:150]
    o, l = K.attend_rows(_values(q), _values(lat), _values(rope), rows, 0.04)
    o2, l2 = OA.attend_sparse(q, lat, rope, rows, 0.04)
    assert np.allclose(o, o2, rtol=0, atol=1e-12) and np.allclose(l, l2, rtol=0, atol=1e-12)
    o, l = K.attend_rows(_values(q), _values(lat), _values(rope), [], 0.04)
    assert not o.any() and np.all(np.isneginf(l))
