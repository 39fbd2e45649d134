"""Pins of the 4-bit cache's oracle: its tables against the formats' listed
values, its rounding against hand-worked ties and a brute-force check, its
attention against the dense oracle, its eviction against hand-worked cases."""
import numpy as np
import pytest

from oracle import attention as A
from oracle import kv4 as K


def test_tables():
    assert list(K.E2M1[:8]) == [0, 0.5, 1, 1.5, 2, 3, 4, 6] and list(K.E2M1[8:]) == [-x for x in K.E2M1[:8]]
    assert K.E4M3[0x7E] == 448 and K.E4M3[1] == 2.0 ** -9 and K.E4M3[0x38] == 1 and np.isnan(K.E4M3[0x7F])
    assert all(a < b for a, b in zip(K.E4M3[:126], K.E4M3[1:127]))


@pytest.mark.parametrize("x,code", [(0.25, 0), (0.26, 1), (0.75, 2), (0.74, 1), (1.25, 2), (1.75, 4), (2.5, 4),
                                    (3.5, 6), (5.0, 6), (5.01, 7), (6.0, 7), (100.0, 7)])
def test_code_ties_go_to_the_even_code(x, code):
    assert K.nearest_even(x, 1.0, K.E2M1[:8]) == code
    assert K.nearest_even(x * 0.3125, 0.3125, K.E2M1[:8]) == code


def test_block():
    # max 6.375 = 6 * 1.0625, halfway between the scales 1 and 1.125: the even one (1)
    c, s = K.quantise_block([6.375, -0.25, 0.75, -6.0], 1.0)
    assert (c, K.E4M3[s]) == ([7, 8, 2, 15], 1.0)
    assert K.quantise_block([0.0, -0.0], 1.0) == ([0, 8], 0)
    assert K.quantise_block([1.0, np.inf], 1.0)[1] == 0x7F
    assert K.quantise_block([1e30, -1e30], 1.0) == ([7, 15], 0x7E)
    # below half the smallest scale: everything is zero
    assert K.quantise_block([0.005, -0.001], 1.0) == ([0, 8], 0)


def test_row_values_round_trip():
    rng = np.random.default_rng(5)
    for D in (8, 40, 128):
        x = rng.normal(size=D)
        c, s = K.quantise_row(x, 0.25)
        y = K.values(c, s, 0.25)
        assert y.shape == (D,) and len(s) == -(-D // 16)
        d = np.repeat(K.E4M3[s] * 0.25, 16)[:D]
        # half the widest step (between 4 and 6), or the cut at 6 of a scale rounded down by at most 1/16
        assert (np.abs(x - y) <= d * 1.0 + 1e-12).all()


def test_attend_is_the_dense_oracle():
    rng = np.random.default_rng(6)
    n, D = 37, 16
    q, k, v = (rng.normal(size=(n, D)) for _ in range(3))
    o, lse = A.forward(q, k, v, 0.25)[:2]
    for T in (1, 5, n):
        got, gl, w = K.attend(q[None, n - T:], k, v, n, 0.25)
        assert np.allclose(got[0], o[n - T:]) and np.allclose(gl[0], lse[n - T:]) and np.allclose(w.sum(-1), 1)
    got, gl, _ = K.attend(q[None, :5], k, v, 2, 0.25)       # more queries than slots: the first see nothing
    assert (got[0, :3] == 0).all() and np.isinf(gl[0, :3]).all() and np.isfinite(gl[0, 3:]).all()


def test_key_mass_sums_the_rows():
    rng = np.random.default_rng(7)
    n, D = 50, 8
    q, k = rng.normal(size=(2, n, D)), rng.normal(size=(n, D))
    lse = np.stack([A.forward(x, k, k, 0.3)[1] for x in q])
    m = K.key_mass(q, k, lse, [(0, 20, 0, 0), (20, n, 0, 0)], 0.3)
    assert np.isclose(m.sum(), 2 * n) and np.allclose(m, K.key_mass(q, k, lse, [(0, n, 0, 0)], 0.3))
    last = K.key_mass(q, k, lse, [(n - 1, n, 0, 0)], 0.3)
    assert np.allclose(last, sum(K.attend(x[None, -1:], k, k, n, 0.3)[2][0, 0] for x in q))


def test_evict_hand_worked():
    m = np.array([3.0, 1.0, 3.0, 2.0, 9.0, 0.0])
    assert K.evict(m, 6, 3, 1) == [0, 4, 5]                 # the tie of 0 and 2: the lower
    assert K.evict(m, 6, 4, 0) == [0, 2, 3, 4]
    assert K.evict(m, 6, 4, 9) == [2, 3, 4, 5]
    assert K.evict(m, 2, 4, 1) == [0, 1] and K.evict(m, 0, 4, 1) == []
    assert K.evict(np.array([5.0, np.nan, -np.inf, np.inf]), 4, 2, 0) == [1, 3]
    assert K.evict(np.array([-0.0, 0.0, -1.0]), 3, 1, 0) == [0]
