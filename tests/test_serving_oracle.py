"""Pins of the serving step's float64 oracle (CPU)."""

import numpy as np
import pytest

from oracle import attention_forward
from oracle import serving_oracle as so

MODES = [(0, 1), (1, 1), (2, 3), (2, 15), (3, 3), (4, 15)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("scaling", ["none", "linear", "base", "bands"])
def test_rope_is_a_rotation_by_position(interleaved, scaling):
    rng = np.random.default_rng(0)
    f = so.frequencies(32, scaling=scaling, factor=4.0, original_length=64, low=1.0, high=4.0)
    x, y = rng.standard_normal((2, 40, 64))
    m = np.arange(40) * 1000
    turn = lambda v, at, back=False: so.rope(v, at, f, interleaved, back)[0]     # noqa: E731
    assert np.allclose(np.linalg.norm(turn(x, m), axis=1), np.linalg.norm(x, axis=1))
    assert np.allclose(turn(turn(x, m), m, back=True), x)                       # back is the inverse ...
    assert np.allclose((turn(x, m) * y).sum(1), (x * turn(y, m, back=True)).sum(1))   # ... and the transpose: the gradient
    assert np.array_equal(turn(x, m)[:, 32:], x[:, 32:])
    assert np.array_equal(turn(x, 0 * m), x)
    # q.k depends on the positions' difference alone
    assert np.allclose((turn(x, m + 7) * turn(y, m)).sum(1), (turn(x, 0 * m + 7) * y).sum(1))


def test_rope_by_hand():
    x = np.zeros((1, 16))
    x[0, 1], x[0, 8] = 1.0, 2.0
    f = so.frequencies(16, base=100.0)
    assert np.isclose(f[1], 100.0 ** -0.125) and f[0] == 1.0
    y = so.rope(x, [3], f)[0][0]                # pairs (0, 8) and (1, 9)
    assert np.allclose([y[0], y[8], y[1], y[9]], [-2 * np.sin(3), 2 * np.cos(3), np.cos(3 * f[1]), np.sin(3 * f[1])])
    y = so.rope(x, [3], f, interleaved=True)[0][0]      # pairs (0, 1) and (8, 9), the fourth
    assert np.allclose(y[[0, 1, 8, 9]], [-np.sin(3), np.cos(3), 2 * np.cos(3 * f[4]), 2 * np.sin(3 * f[4])])


def test_rope_far_positions():
    # 2^31 - 1 turns of a frequency that is a fraction of a turn: the angle by whole numbers
    f = np.array([2 * np.pi * 3 / 2 ** 20])
    m = 2 ** 31 - 1
    y = so.rope(np.array([[1.0, 0.0]]), [m], f)[0][0]
    angle = 2 * np.pi * (3 * m % 2 ** 20) / 2 ** 20
    assert np.allclose(y, [np.cos(angle), np.sin(angle)], atol=2.0 ** 31 * 2.0 ** -52)


@pytest.mark.parametrize("mode,p", MODES)
def test_attend_rows_are_the_last_rows_of_the_forward(mode, p):
    rng = np.random.default_rng(1)
    hkv, G, d, page, lens, counts = 2, 2, 64, 8, [20, 5, 0, 33], [20, 1, 0, 7]
    table = rng.permutation(20).reshape(4, 5)
    kp, vp = rng.standard_normal((2, 20, hkv, page, d))
    q = rng.standard_normal((4, hkv * G, 20, d))
    got = so.paged_attend(q, kp, vp, table, lens, counts, mode, p, 0.0)
    assert len(got) == hkv * (20 + 1 + 7)
    for b, (n, c) in enumerate(zip(lens, counts)):
        k = np.concatenate([kp[g] for g in table[b]], axis=1)[:, :n]
        v = np.concatenate([vp[g] for g in table[b]], axis=1)[:, :n]
        for h in range(hkv * G):
            if c:
                qs = np.zeros((n, d))
                qs[n - c:] = q[b, h, :c]
                ref = attention_forward(qs, k[h // G], v[h // G], mode, p)[n - c:]
                out = np.stack([got[b, h // G, t][0][h % G] for t in range(c)])
                assert np.allclose(out, ref, rtol=1e-11, atol=1e-13)


@pytest.mark.parametrize("mode,p", MODES)
def test_attend_bound_holds_for_inputs_off_by_one_rounding(mode, p):
    from oracle import paged_oracle as po
    rng = np.random.default_rng(5)
    q, k = rng.standard_normal((4, 64)), rng.standard_normal((300, 64))
    w, e = po.row_weights(q, k, mode, p), so.attend_bound(q, k, mode, p)
    off = np.abs(po.row_weights(q * (1 + 2.0 ** -24 * rng.uniform(-1, 1, q.shape)), k, mode, p) - w)
    assert (off <= e).all() and e.max() < 1e-2


def test_pages_by_hand():
    table = np.full((3, 4), -1)
    free = np.array([10, 11, 12, 13, 14, 15])
    t, counts, left = so.reserve(table, [8, 3, 0], [9, 5, 1], 8, free, 5)
    # 8 + 9 tokens: two pages more; 3 + 5: none more than the one held; 0 + 1: one
    assert t.tolist() == [[-1, 14, 13, -1], [-1] * 4, [12, -1, -1, -1]] and counts == [9, 5, 1] and left == 2
    t, counts, left = so.reserve(table, [8, 3, 0], [9, 5, 1], 8, free, 1)
    assert counts == [0, 5, 0] and left == 1 and (t == -1).all()
    table = np.array([[1, 2, 3, -1], [4, -1, -1, -1], [5, 6, -1, -1]])
    free, count = so.release(table, [24, 3, 9], [8, 3, 0], 8, np.arange(100, 107), 2)
    assert free.tolist() == [100, 101, 2, 3, 5, 6, 106] and count == 6
