"""Pins of the attention oracle: cases small enough to work out by hand, and the
same quantities by another route (complex rotation, one token at a time)."""

import numpy as np

from oracle import attention as at


def test_rotation_by_a_quarter_turn():
    table = np.array([[1.0, 1.0, 0.0, 0.0], [0.0, 0.0, 1.0, 1.0]])    # positions 0 and 1
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)                          # 4 of 6 elements turn
    assert np.array_equal(at.rotate(x, [0], table, False), x)
    assert at.rotate(x, [1], table, False).tolist() == [[[-3, -4, 1, 2, 5, 6]]]
    assert at.rotate(x, [1], table, True).tolist() == [[[-2, 1, -4, 3, 5, 6]]]
    # positions past the table are its ends
    assert np.array_equal(at.rotate(x, [7], table, True), at.rotate(x, [1], table, True))
    assert np.array_equal(at.rotate(x, [-3], table, True), x)


def test_rotation_is_a_complex_product():
    r = np.random.default_rng(0)
    ang = r.uniform(0, 6, (5, 8))
    table = np.concatenate((np.cos(ang), np.sin(ang)), 1)
    x, pos = r.standard_normal((3, 2, 16)), [4, 0, 2]
    y = at.rotate(x, pos, table, False)
    z = (x[..., :8] + 1j * x[..., 8:]) * np.exp(1j * ang[pos])[:, None]
    assert np.allclose(y, np.concatenate((z.real, z.imag), -1), rtol=1e-14, atol=1e-14)


def test_slots():
    rows, page, place = at.slots_of([5, -1, 12, 11, 0], 3, 4)
    assert rows.tolist() == [0, 3, 4] and page.tolist() == [1, 2, 0] and place.tolist() == [1, 3, 0]


def test_tokens_follow_the_table():
    cache = np.arange(3 * 2 * 4 * 1.0).reshape(3, 2, 4, 1)
    t = at.tokens(cache, [2, 0, 9], 10)
    assert t[:, 0, 0].tolist() == [16, 17, 18, 19, 0, 1, 2, 3, 16, 17]
    assert t[:, 1, 0].tolist() == [20, 21, 22, 23, 4, 5, 6, 7, 20, 21]


def test_what_a_row_sees():
    assert at.visible(4, 7, 0, 0).tolist() == [1, 1, 1, 1, 1, 0, 0]
    assert at.visible(4, 7, 2, 0).tolist() == [0, 0, 0, 1, 1, 0, 0]
    assert at.visible(4, 7, 2, 1).tolist() == [1, 0, 0, 1, 1, 0, 0]
    assert at.visible(4, 7, 1, 9).tolist() == [1, 1, 1, 1, 1, 0, 0]
    assert not at.visible(-1, 7, 0, 3).any()


def test_two_tokens():
    q, k = np.array([[1.0, 0.0], [0.0, 2.0]]), np.array([[[0.0, 0.0]], [[np.log(3.0), 5.0]]])
    v = np.array([[[4.0, 0.0]], [[8.0, 4.0]]])
    y, lse, w, _ = at.attend(q, k, v, 1, 1.0)
    assert np.allclose(w[0], [0.25, 0.75]) and np.allclose(y[0], [7.0, 3.0])
    assert np.allclose(lse, [np.log(4.0), np.log(1 + np.exp(10.0))])
    y, lse, _, _ = at.attend(q, k, v, 0, 1.0)
    assert np.allclose(y, [[4, 0], [4, 0]]) and np.allclose(lse, 0.0)
    y, lse, _, _ = at.attend(q, k, v, -1, 1.0)
    assert not y.any() and np.all(lse == -np.inf)


def test_one_token_at_a_time():
    """The running form of the softmax sum gives the same."""
    r = np.random.default_rng(1)
    q, k, v = r.standard_normal((4, 8)), r.standard_normal((9, 2, 8)), r.standard_normal((9, 2, 8))
    y, lse, _, _ = at.attend(q, k, v, 7, 0.5, window=4, sinks=2)
    for h in range(4):
        m, l, o = -np.inf, 0.0, np.zeros(8)
        for j in (0, 1, 4, 5, 6, 7):
            z = 0.5 * q[h] @ k[j, h // 2]
            n = max(m, z)
            l, o = l * np.exp(m - n) + np.exp(z - n), o * np.exp(m - n) + np.exp(z - n) * v[j, h // 2]
            m = n
        assert np.allclose(y[h], o / l) and np.isclose(lse[h], m + np.log(l))
