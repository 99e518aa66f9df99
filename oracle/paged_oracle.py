"""Float64 NumPy oracle of the paged key-value cache: append, decode, evict.

TEST INFRASTRUCTURE ONLY, written to be checked by eye.  The cache is a list
of pages; a slot s of sequence b is row ``s % page_size`` of page
``table[b][s // page_size]``.  The decode step is row i = length of the pinned
forward oracle (:mod:`oracle.lssar_oracle`); nothing here is fused or blocked.
"""

import math

import numpy as np

from .lssar_oracle import (MODE_LSSA, MODE_LSSAR, MODE_SIGMOID_RW, MODE_SOFTMAX, MODE_SOFTMAX_RW, l2_normalize_rows,
                           length_scale, lssa_rows, reweight_rows, sigmoid, softmax_rows)

REWEIGHTED = (MODE_LSSAR, MODE_SOFTMAX_RW, MODE_SIGMOID_RW)


def gather(pages, table_row, n):
    """Slots 0..n-1 of one sequence, [n, Hkv, d], from pages [n_pages, Hkv, page_size, d]."""
    ps = pages.shape[2]
    return np.stack([pages[table_row[s // ps], :, s % ps] for s in range(n)]) if n else pages[:0, :, 0]


def row_weights(q, k, mode, p=3):
    """The normalised weights, [G, n], of the queries q [G, d] on all the keys
    k [n, d]: row i = n of the attention."""
    n, d = k.shape
    rows = np.full(len(q), n)
    if mode in (MODE_SOFTMAX, MODE_SOFTMAX_RW):
        a = softmax_rows(q, k, rows, d)
    else:
        a = lssa_rows(q, k, rows, d, phi=sigmoid if mode == MODE_SIGMOID_RW else None)
    return reweight_rows(a, rows, p) if mode in REWEIGHTED else a


def weight_bound(q, k, mode, p=3):
    """How far float32 evaluation may move each weight of :func:`row_weights`,
    [G, n], from the rounding of each step (u = 2^-24, worst case throughout).

    The score product sums d exact products, each partial sum off by at most
    2u of sum |q_c k_c| (a tensor unit may truncate) and its scale by a few u:
    |dx| <= (2d + 16) u c sum_c |q_c k_c|, c the row's factor, plus 4u|x|.
    The normaliser phi then moves by phi'(x) dx and by its own evaluation, at
    most 2^-20 phi, the exponential's argument rounded to 4u|x|; for softplus
    min(2^-20 (1 + phi), 2^-18 phi): a polynomial's 2^-19 and the exponential's 2^-22.
    Row sums add (n / 16 + 64) u.  A weight max(n phi / S1 - O, 0)^p is increasing
    in phi: it lies between its values at both ends.
    """
    u = 2.0 ** -24
    n, d = k.shape
    if mode in (MODE_SOFTMAX, MODE_SOFTMAX_RW):
        qq, kk, c = q, k, 1 / math.sqrt(d)
    else:
        qq, kk, c = l2_normalize_rows(q), l2_normalize_rows(k), float(length_scale(n, d))
    x = c * (qq @ kk.T)
    dx = (2 * d + 16) * u * c * (np.abs(qq) @ np.abs(kk).T) + 4 * u * np.abs(x)
    if mode in (MODE_SOFTMAX, MODE_SOFTMAX_RW):
        top = x.max(axis=1, keepdims=True)
        phi = np.exp(x - top)
        dphi = phi * (np.expm1(dx + dx.max(axis=1, keepdims=True) + 4 * u * np.abs(x - top)) + 2.0 ** -20)
    elif mode == MODE_SIGMOID_RW:
        phi = sigmoid(x)
        dphi = phi * (1 - phi) * dx + 2.0 ** -20 * phi
    else:
        phi = np.logaddexp(0.0, x)
        dphi = sigmoid(x) * dx + np.minimum(2.0 ** -20 * (1 + phi), 2.0 ** -18 * phi)
    s1 = phi.sum(axis=1, keepdims=True)
    ds1 = dphi.sum(axis=1, keepdims=True) / s1 + (n / 16 + 64) * u
    if mode in REWEIGHTED:
        y = n * phi / s1 - (0.0 if n <= 3 else 1.0)
        dy = n * dphi / s1 + n * phi / s1 * ds1 + 8 * u * (1 + np.abs(y))
        lo, hi = np.maximum(y - dy, 0.0), np.maximum(y + dy, 0.0)
        best = np.maximum(y.max(axis=1, keepdims=True), 1e-300)
        w, lo, hi = ((np.maximum(t, 0.0) / best) ** p for t in (y, lo, hi))
        spread = hi - lo + 4 * p * u * w
    else:
        w, spread = phi, dphi
    total = np.maximum(w.sum(axis=1, keepdims=True), 1e-300)
    r, e = w / total, spread / total
    if mode in REWEIGHTED:
        same = y.max(axis=1) <= 1e-10                # uniform rows: exactly 1/n
        e[same], r[same] = 0.0, 1.0 / n
    return e + r * (e.sum(axis=1, keepdims=True) + (n / 16 + 64) * u)


def paged_decode(q, k_pages, v_pages, table, lens, mode, p=3, scores=None):
    """out [B, H, d], the new scores (or None), and bounds on the float32
    errors of both, before any rounding of the output."""
    B, H, d = q.shape
    hkv = k_pages.shape[1]
    G = H // hkv
    out, out_err = np.zeros((B, H, d)), np.zeros((B, H, d))
    new = None if scores is None else np.array(scores, dtype=np.float64)
    new_err = None if scores is None else np.zeros(scores.shape)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        kb, vb = gather(k_pages, table[b], n), gather(v_pages, table[b], n)
        for h in range(hkv):
            qs = q[b, h * G:(h + 1) * G]
            w, e = row_weights(qs, kb[:, h], mode, p), weight_bound(qs, kb[:, h], mode, p)
            out[b, h * G:(h + 1) * G] = w @ vb[:, h]
            # weights split into two 16-bit parts, and the value sum in float32
            e_pv = 2.0 ** -15 + (n / 4 + 64) * 2.0 ** -24
            out_err[b, h * G:(h + 1) * G] = (e + e_pv * w) @ np.abs(vb[:, h])
            if scores is not None:
                new[b, h, :n] += w.sum(axis=0)
                new_err[b, h, :n] = e.sum(axis=0) + (G + 2) * 2.0 ** -24 * np.abs(new[b, h, :n])
    return out, new, out_err, new_err


def paged_append(k_new, v_new, k_pages, v_pages, table, lens, counts, first=None, scores=None, positions=None):
    """The same arrays after the append (copies), and the new lengths."""
    k_pages, v_pages = k_pages.copy(), v_pages.copy()
    scores = None if scores is None else scores.copy()
    positions = None if positions is None else positions.copy()
    ps = k_pages.shape[2]
    for b, n in enumerate(lens):
        for t in range(counts[b]):
            s = n + t
            page, row = table[b][s // ps], s % ps
            k_pages[page, :, row], v_pages[page, :, row] = k_new[b, :, t], v_new[b, :, t]
            if scores is not None:
                scores[b, :, s] = 0
            if positions is not None:
                positions[b, :, s] = (n if first is None else first[b]) + t
    return k_pages, v_pages, scores, positions, np.asarray(lens) + np.asarray(counts)


def evict_moves(scores, positions, n, keep, recent, sinks):
    """(mover, hole) slots of one row of n cached tokens, in order."""
    if n <= keep:
        return []
    newest = max(int(x) for x in positions[:n])

    def rank(s):
        safe = positions[s] < sinks or int(positions[s]) > newest - recent
        x = float(scores[s])
        return (0 if safe else 1, 0.0 if safe else (math.inf if math.isnan(x) else -x), not safe and math.isnan(x), s)

    kept = set(sorted(range(n), key=rank)[:keep])
    holes = [s for s in range(keep) if s not in kept]
    movers = [s for s in range(keep, n) if s in kept]
    assert len(holes) == len(movers)
    return list(zip(movers, holes))


def paged_evict(k_pages, v_pages, table, lens, scores, positions, keep, recent=0, sinks=0):
    """The same arrays after an in-place eviction (copies), and the new lengths."""
    k_pages, v_pages, scores, positions = (x.copy() for x in (k_pages, v_pages, scores, positions))
    ps = k_pages.shape[2]
    for b, n in enumerate(lens):
        for h in range(k_pages.shape[1]):
            for s, t in evict_moves(scores[b, h], positions[b, h], n, keep, recent, sinks):
                of, to = (table[b][s // ps], h, s % ps), (table[b][t // ps], h, t % ps)
                k_pages[to], v_pages[to] = k_pages[of], v_pages[of]
                scores[b, h, t], positions[b, h, t] = scores[b, h, s], positions[b, h, s]
    return k_pages, v_pages, scores, positions, np.minimum(lens, keep)
