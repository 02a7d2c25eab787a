"""Pins of the rotary oracle against things other than itself: single rotations by hand, the
defining invariants (norms kept, scores depend on position differences only), and a float64 matrix
form."""
import math

import numpy as np
import pytest

from oracle import rope
from oracle.paged_attention import OracleError


@pytest.mark.parametrize("interleaved", [False, True])
def test_quarter_turn_by_hand(interleaved):
    # one pair turned by 90 degrees: (1, 2) -> (-2, 1); the other pair stays
    cs = np.array([[0.0, 1.0, 1.0, 0.0]], dtype=np.float32)   # cos (0, 1), sin (1, 0)
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    y = rope.rotate(x, [0], cs, interleaved)[0, 0]
    if interleaved:   # pairs (0, 1), (2, 3)
        assert y.tolist() == [-2.0, 1.0, 3.0, 4.0, 5.0]
    else:             # pairs (0, 2), (1, 3)
        assert y.tolist() == [-3.0, 2.0, 1.0, 4.0, 5.0]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 32])
def test_norms_kept_and_scores_depend_on_distance(interleaved, rot):
    rng = np.random.default_rng(3)
    D = 32
    freq = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    ang = np.arange(400)[:, None] * freq
    cs = np.concatenate((np.cos(ang), np.sin(ang)), axis=1)   # float64: exact to rounding
    q, k = rng.standard_normal((1, 1, D)), rng.standard_normal((1, 1, D))
    r = lambda x, p: rope.rotate(x, [p], cs, interleaved)[0, 0]
    assert abs(np.linalg.norm(r(q, 371)) - np.linalg.norm(q)) < 1e-12
    scores = [r(q, 40 + p) @ r(k, p) for p in (0, 1, 99, 359)]
    assert max(scores) - min(scores) < 1e-11
    assert abs(scores[0] - q[0, 0] @ k[0, 0]) > 1e-3        # and do depend on it
    assert (r(q, 371)[rot:] == q[0, 0, rot:]).all()


def test_rotation_matrix_form():
    # the same as one block-diagonal rotation matrix per position
    rng = np.random.default_rng(4)
    cs = rope.table(50, 16)
    x = rng.standard_normal((3, 2, 24))
    pos = [0, 17, 49]
    y = rope.rotate(x, pos, cs, False)
    for t, p in enumerate(pos):
        m = np.eye(24)
        for j, (a, b) in enumerate(rope.pairs(16, False)):
            c, s = float(cs[p, j]), float(cs[p, 8 + j])
            m[a, a], m[a, b], m[b, a], m[b, b] = c, -s, s, c
        assert np.abs(y[t] - x[t] @ m.T).max() < 1e-14


def test_table_and_positions():
    cs = rope.table(8, 16, base=100.0)
    assert cs.dtype == np.float32 and cs.shape == (8, 16)
    assert cs[3, 2] == np.float32(math.cos(3 * 100.0 ** (-4 / 16)))
    assert cs[3, 8 + 2] == np.float32(math.sin(3 * 100.0 ** (-4 / 16)))
    pos = rope.positions_of(np.array([0, 1, 1, 4]), np.array([10, 5, 7]))
    assert pos.tolist() == [9, 4, 5, 6]
    with pytest.raises(OracleError):
        rope.pairs(5, False)
