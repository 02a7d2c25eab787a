"""The oracle of the quantised cache and of changed scores, pinned to the format's definition, torch's own
conversion, the plain attention oracle and closed forms."""
import math

import numpy as np
import pytest
import torch

from oracle import paged_attention as opa
from oracle import quant as oq


def test_the_256_values():
    t = oq.e4m3_table()
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(ref))
    assert np.array_equal(t[~np.isnan(t)], ref[~np.isnan(ref)])
    assert np.nanmax(t) == 448.0 and t[1] == 2.0 ** -9


def test_rounding_matches_torch():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(5000) * s for s in (1e-3, 0.02, 1, 30, 200)])
    t = oq.e4m3_table()[:127]
    ties = (t[:-1] + t[1:]) / 2
    x = np.clip(np.concatenate([x, ties, -ties, t, -t, [0.0, -0.0]]), -448, 448).astype(np.float32)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oq.to_code(x.astype(np.float64)), ref)


def test_rows():
    x = np.zeros((6, 64))
    x[1, 3] = 448.0
    x[2, 3] = 448.0000001
    x[3, 0], x[3, 5], x[3, 6], x[3, 7] = 1.0, math.nan, math.inf, -math.inf
    x[4, 0] = 1e30
    x[5, :] = -3e-20
    codes, sc = oq.quantise(x)
    assert sc.tolist() == [95, 127, 128, 255, 158, 95]
    v = oq.values(codes, sc)
    assert v[1, 3] == 448 and v[2, 3] == 448 and np.isnan(v[3]).all() and (codes[3] == 0x7F).all()
    assert v[4, 0] == 448 * 2.0 ** 31 and (v[5] == 0).all() and (v[0] == 0).all()


def test_error_of_a_row():
    x = np.random.default_rng(2).standard_normal((200, 128)) * np.exp(np.random.default_rng(3).standard_normal((200, 1)) * 4)
    codes, sc = oq.quantise(x)
    err = np.abs(oq.values(codes, sc) - x)
    e = sc.astype(int) - 127
    assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** (e - 10.0)[:, None]))
    assert np.all(np.abs(x).max(1) <= 448 * 2.0 ** e) and np.all(np.abs(x).max(1) > 224 * 2.0 ** e)


def test_attention_without_changes_is_the_plain_one():
    rng = np.random.default_rng(4)
    q, K, V = rng.standard_normal((5, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    for window in (0, 3):
        out, lse, _ = oq.scored_attention(q, K, V, 4, 0.3, window=window)
        ref, ref_lse = opa.attention_one_sequence(q, K, V, 4, 0.3, window)
        assert np.allclose(out, ref, atol=1e-13) and np.allclose(lse, ref_lse, atol=1e-13)
    assert np.allclose(oq.scored_attention(q, K, V, 4, 0.3, softcap=1e9)[0],
                       oq.scored_attention(q, K, V, 4, 0.3)[0], atol=1e-9)


def test_changes_in_closed_form():
    q, K = np.zeros((1, 1, 2)), np.zeros((3, 1, 2))
    V = np.array([[[1.0, 0]], [[0, 1.0]], [[2.0, 2.0]]])
    out, lse, _ = oq.scored_attention(q, K, V, 2, 1.0, slopes=[math.log(2)])
    w = np.array([0.25, 0.5, 1.0])          # 2^(key - position)
    assert np.allclose(out[0, 0], w @ V[:, 0] / w.sum()) and np.allclose(lse, math.log(w.sum()))
    q1, K1 = np.full((1, 1, 1), 10.0), np.array([[[1.0]], [[-1.0]]])
    _, lse, _ = oq.scored_attention(q1, K1, np.zeros((2, 1, 1)), 1, 1.0, softcap=2.0)
    t = 2 * math.tanh(5.0)
    assert lse[0, 0] == pytest.approx(math.log(math.exp(t) + math.exp(-t)), abs=1e-12)
    # a prefix read both ways: the first of two queries sees the second's key
    out, _, _ = oq.scored_attention(np.zeros((2, 1, 2)), K[:2], V[:2], 0, 1.0, visible=2)
    assert np.allclose(out[0, 0], [0.5, 0.5]) and np.allclose(out[1, 0], [0.5, 0.5])
