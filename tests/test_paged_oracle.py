"""Pins of the paged cache's float64 oracle (CPU)."""

import numpy as np
import pytest

from oracle import attention_forward
from oracle import paged_oracle as po

MODES = [(0, 1), (1, 1), (2, 3), (2, 15), (3, 3), (4, 15)]


@pytest.mark.parametrize("mode,p", MODES)
@pytest.mark.parametrize("page", [8, 24])
def test_decode_is_the_last_row_of_the_forward(mode, p, page):
    rng = np.random.default_rng(page)
    B, hkv, G, d, lens = 3, 2, 3, 64, [1, 29, 50]
    width = -(-max(lens) // page)
    table = rng.permutation(B * width).reshape(B, width)
    kp, vp = rng.standard_normal((2, B * width, hkv, page, d))
    q = rng.standard_normal((B, hkv * G, d))
    scores = rng.random((B, hkv, width * page))
    out, new, _, _ = po.paged_decode(q, kp, vp, table, lens, mode, p, scores)
    for b, n in enumerate(lens):
        k = np.concatenate([kp[g] for g in table[b]], axis=1)[:, :n]
        v = np.concatenate([vp[g] for g in table[b]], axis=1)[:, :n]
        for h in range(hkv * G):
            qs = np.zeros((n, d))
            qs[-1] = q[b, h]
            ref = attention_forward(qs, k[h // G], v[h // G], mode, p, rows=np.array([n]))[0]
            assert np.allclose(out[b, h], ref, rtol=1e-12, atol=1e-14)
        # every query head hands out a weight of one
        assert np.allclose((new - scores)[b].sum(axis=1), G)
        assert np.array_equal(new[b, :, n:], scores[b, :, n:])


@pytest.mark.parametrize("mode,p", MODES)
def test_weight_bound_holds_for_float32_inputs_off_by_one_rounding(mode, p):
    # scores moved by what the bound allows for them move the weights by less than it says
    rng = np.random.default_rng(5)
    q, k = rng.standard_normal((4, 64)), rng.standard_normal((300, 64))
    w, e = po.row_weights(q, k, mode, p), po.weight_bound(q, k, mode, p)
    off = np.abs(po.row_weights(q * (1 + 2.0 ** -24 * rng.uniform(-1, 1, q.shape)), k, mode, p) - w)
    assert (off <= e).all() and e.max() < 1e-2
    assert np.allclose(w.sum(axis=1), 1)


def test_evict_by_hand():
    #            slot 0  1  2  3  4  5  6
    scores = np.array([5., 0., 2., 2., 9., 2., 0.])
    pos = np.arange(7)
    # keep 4: slots 4, 0, then 2, 3 of the three equal ones (5 goes)
    assert po.evict_moves(scores, pos, 7, 4, 0, 0) == [(4, 1)]
    # the newest two stay: 5, 6, then 4, 0
    assert po.evict_moves(scores, pos, 7, 4, 2, 0) == [(4, 1), (5, 2), (6, 3)]
    # the first two positions stay: 0, 1, then 4, 2
    assert po.evict_moves(scores, pos, 7, 4, 0, 2) == [(4, 3)]
    assert po.evict_moves(scores, pos, 7, 7, 0, 0) == []
    assert po.evict_moves(np.array([np.nan, -1., 0., -0.]), pos, 4, 2, 0, 0) == [(2, 0), (3, 1)]


def test_append_by_hand():
    kp, vp = np.zeros((3, 1, 8, 64)), np.zeros((3, 1, 8, 64))
    new = np.arange(1, 4)[None, None, :, None] * np.ones((2, 1, 3, 64))
    sc, pos = np.ones((2, 1, 16)), np.full((2, 1, 16), -1)
    k, v, sc, pos, lens = po.paged_append(new, 10 * new, kp, vp, [[2, 0], [1, 1]], [6, 0], [3, 1], [100, 7], sc, pos)
    assert lens.tolist() == [9, 1]
    assert k[2, 0, 6:, 0].tolist() == [1, 2] and k[0, 0, 0, 0] == 3 and k[1, 0, 0, 0] == 1 and k.sum() == 64 * 7
    assert v.sum() == 640 * 7
    assert pos[0, 0, 6:9].tolist() == [100, 101, 102] and pos[1, 0, 0] == 7 and sc.sum() == 32 - 4
