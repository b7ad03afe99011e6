"""Pins of the oracle's layer operators that do not call its formulas again: hand-worked rows, torch's
own routines, and what the definitions imply (no GPU needed)."""
import numpy as np
import pytest
import torch

import oracle


def test_rms_norm_hand_row_and_library():
    out, v = oracle.rms_norm(np.array([[3.0, 4.0]]), np.array([[0.0, 0.0]]), np.array([1.0, 2.0]), eps=0.0)
    # mean square 12.5
    assert np.allclose(out, [[3 / 12.5 ** 0.5, 8 / 12.5 ** 0.5]], rtol=1e-15)
    g = np.random.default_rng(0)
    x, r, w = g.normal(size=(5, 33)), g.normal(size=(5, 33)), g.normal(size=33)
    out, v = oracle.rms_norm(x, r, w, eps=1e-5)
    ref = torch.nn.functional.rms_norm(torch.from_numpy(x + r), (33,), torch.from_numpy(w), 1e-5).numpy()
    assert np.allclose(out, ref, rtol=1e-13) and np.array_equal(v, x + r)


def test_row_codes_borders_and_odd_rows():
    # 127 t / 254 = t / 2: odd t are ties, which go to the even code
    q, m = oracle.row_codes(np.array([[254.0, 1.0, 3.0, -1.0, -3.0, 5.0, 2.0]]))
    assert q.tolist() == [[127, 0, 2, 0, -2, 2, 1]] and m[0] == 254
    q, m = oracle.row_codes(np.array([[0.0, 0.0], [np.inf, 1.0], [np.nan, 1.0], [-2.0, 1.0]]))
    assert q.tolist() == [[0, 0], [0, 0], [0, 0], [-127, 64]]
    assert m[0] == 0 and np.isnan(m[1]) and np.isnan(m[2]) and m[3] == 2


def test_codes_of_the_norm_stand_for_its_output_to_half_a_step():
    g = np.random.default_rng(1)
    x, r, w = g.normal(size=(7, 64)) * 5, g.normal(size=(7, 64)), 1 + 0.2 * g.normal(size=64)
    q, scale, _ = oracle.rms_norm_i8(x, r, w)
    out, _ = oracle.rms_norm(x, r, w)
    assert (np.abs(q * scale[:, None] - out) <= scale[:, None] * (0.5 + 1e-9)).all() and np.abs(q).max() == 127


def test_linear_i8_whole_numbers():
    x, w = np.full((1, 70000), -128, dtype=np.int8), np.full((2, 70000), 127, dtype=np.int8)
    w[1, 0] = -128
    out, p = oracle.linear_i8(x, [1.0], w, [1.0, 0.5], [0.0, 3.0])
    assert out[0, 0] == -128 * 127 * 70000 and p[0, 1] == 0.5 * (-128 * 127 * 69999 + 128 * 128) and out[0, 1] == p[0, 1] + 3


@pytest.mark.parametrize("halves", [False, True])
def test_rope_is_complex_multiplication_and_keeps_relative_positions(halves):
    g = np.random.default_rng(2)
    axes, d = (4, 6, 6), 16
    q, k = g.normal(size=(1, d)), g.normal(size=(1, d))
    one = oracle.rope(q, oracle.rope_angles([[0, 0, 0]], axes, 100.0), halves)
    assert np.array_equal(one, q)                                     # position zero turns nothing
    assert np.array_equal(oracle.rope(q, np.full((1, 8), np.nan), halves), q)

    def score(pq, pk):
        a = oracle.rope(q, oracle.rope_angles([pq], axes, 100.0), halves)
        b = oracle.rope(k, oracle.rope_angles([pk], axes, 100.0), halves)
        assert np.isclose((a * a).sum(), (q * q).sum())
        return float((a * b).sum())
    assert np.isclose(score((3, 5, 7), (1, 2, 9)), score((13, 4, 8), (11, 1, 10)))   # same difference on every axis
    assert not np.isclose(score((3, 5, 7), (1, 2, 9)), score((3, 5, 7), (1, 3, 9)))
    # second pair of the height axis by hand: pair 2 + 1, frequency 100^(-2/6)
    ang = oracle.rope_angles([[0, 2, 0]], axes, 100.0)
    assert np.isclose(ang[0, 3], 2 * 100.0 ** (-1 / 3)) and ang[0, 0] == 0 and ang[0, 5] == 0
    ia, ib = (3, 11) if halves else (6, 7)
    z = (q[0, ia] + 1j * q[0, ib]) * np.exp(1j * ang[0, 3])
    got = oracle.rope(q, ang, halves)[0]
    assert np.isclose(got[ia], z.real) and np.isclose(got[ib], z.imag)
