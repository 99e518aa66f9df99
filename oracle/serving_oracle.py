"""Float64 NumPy oracle of a serving step around the paged cache: rotary
positions, the attention of a chunk, pages taken from and given back to a list.

TEST INFRASTRUCTURE ONLY, written to be checked by eye: rows one at a time,
pages one at a time.
"""

import math

import numpy as np

from .lssar_oracle import MODE_LSSAR, MODE_SIGMOID_RW, MODE_SOFTMAX, MODE_SOFTMAX_RW, l2_normalize_rows, length_scale, sigmoid
from .paged_oracle import REWEIGHTED, gather, row_weights


# ---------------------------------------------------------------- rotary positions

def frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, original_length=1, low=1.0, high=32.0):
    """Radians per position of each pair."""
    f = []
    for c in range(rot_dim // 2):
        b = base * factor ** (rot_dim / (rot_dim - 2)) if scaling == "base" else base
        x = b ** (-2.0 * c / rot_dim)
        if scaling == "linear":
            x /= factor
        if scaling == "bands":
            turns = original_length * x / (2 * math.pi)
            g = min(1.0, max(0.0, (turns - low) / (high - low)))
            x *= g + (1 - g) / factor
        f.append(x)
    return np.array(f)


def rope(x, positions, freq, interleaved=False, back=False):
    """x [..., n, d] turned by positions [..., n] (broadcast), and a bound on the
    float32 errors before the output's rounding.

    Angles: modulo a turn in extended precision here; the kernel's are off by
    |m| f 2^-47 (its frequencies), 2^-32 turns (phase) and 2^-25 half turns
    (its conversion), together 2^-23 and the first; sines and cosines by 2^-23 more;
    three roundings of each product.
    """
    rot = 2 * len(freq)
    m = np.asarray(positions, dtype=np.longdouble)[..., None]
    turn = 8 * np.arctan(np.longdouble(1))
    angle = np.fmod(m * freq.astype(np.longdouble), turn).astype(np.float64)
    c, s = np.cos(angle), np.sin(-angle if back else angle)
    y, err = x.astype(np.float64).copy(), np.zeros(x.shape)
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    u, v = x[..., one], x[..., two]
    y[..., one], y[..., two] = u * c - v * s, u * s + v * c
    off = (np.abs(m).astype(np.float64) * freq * 2.0 ** -47 + 2.0 ** -22 + 3 * 2.0 ** -24) * (np.abs(u) + np.abs(v))
    err[..., one] = err[..., two] = off
    return y, err


# ---------------------------------------------------------------- attention of a chunk

def attend_bound(q, k, mode, p=3):
    """How far float32 evaluation may move each weight of
    :func:`paged_oracle.row_weights` in a kernel that evaluates the softplus of
    a row in one of several forms (u = 2^-24, worst case throughout).

    Scores as in paged_oracle.weight_bound.  Normalisers: exponentials and
    sigmoids 2^-20 of their value; softplus 2^-19 (1 + its value), or, where all
    scores of the row are negative, at most 2^-18 of its value.  The row sum of
    softplus is taken as logarithms of products of 64 factors, each rounded:
    64 u / ln 2 in log2 units for every 64 keys whose largest score is not negative, and
    whose sum is at least 1; 2^-17 of the sum, and (n / 16 + 64) u for the sums.
    """
    u = 2.0 ** -24
    n, d = k.shape
    raw = mode in (MODE_SOFTMAX, MODE_SOFTMAX_RW)
    qq, kk, c = (q, k, 1 / math.sqrt(d)) if raw else (l2_normalize_rows(q), l2_normalize_rows(k), float(length_scale(n, d)))
    x = c * (qq @ kk.T)
    dx = (2 * d + 16) * u * c * (np.abs(qq) @ np.abs(kk).T) + 6 * u * np.abs(x)
    if raw:
        top = x.max(axis=1, keepdims=True)
        phi = np.exp(x - top)
        dphi = phi * (np.expm1(dx + dx.max(axis=1, keepdims=True) + 4 * u * np.abs(x - top)) + 2.0 ** -20)
    elif mode == MODE_SIGMOID_RW:
        phi = sigmoid(x)
        dphi = phi * (1 - phi) * dx + 2.0 ** -20 * phi
    else:
        phi = np.logaddexp(0.0, x)
        away = x.max(axis=1, keepdims=True) < 0
        dphi = sigmoid(x) * dx + np.where(away, 2.0 ** -18 * phi, 2.0 ** -19 * (1 + phi))
    s1 = phi.sum(axis=1, keepdims=True)
    ds1 = dphi.sum(axis=1, keepdims=True) / s1 + (n / 16 + 64) * u + (2.0 ** -17 if mode == MODE_LSSAR else 0.0)
    if mode in REWEIGHTED:
        y = n * phi / s1 - (0.0 if n <= 3 else 1.0)
        dy = n * dphi / s1 + n * phi / s1 * ds1 + 8 * u * (1 + np.abs(y))
        best = np.maximum(y.max(axis=1, keepdims=True), 1e-300)
        w, lo, hi = (np.minimum(np.maximum(t, 0.0) / best, 2.0) ** p for t in (y, y - dy, y + dy))
        spread = hi - lo + 4 * p * u * w
    else:
        w, spread = phi, dphi
    total = np.maximum(w.sum(axis=1, keepdims=True), 1e-300)
    r, e = w / total, spread / total
    if mode in REWEIGHTED:
        same = y.max(axis=1) <= 1e-10                # uniform rows: exactly 1/n
        e[same], r[same] = 0.0, 1.0 / n
    e_total = e.sum(axis=1, keepdims=True)
    return e + r * (e_total + (n / 16 + 64) * u)


def attend_row(q, k, v, mode, p, half_step):
    """One row's outputs [G, d] over all of k, v [n, d], and the bound on their
    error before the output's rounding: the weights', their rounding to 16 bits
    (half_step; of fp16 also half its least step, 2^-25, against a largest weight
    of 0.69 2^8 or more), and the value sum in float32.  LSSAR from p = 4 on may use the
    one-exponential softplus, which moves the weights in sum by at most 2e-4 of
    their total, and the output by twice that of the largest value."""
    n = len(k)
    w, e = row_weights(q, k, mode, p), attend_bound(q, k, mode, p)
    least = 2.0 ** -32 * w.max(axis=1, keepdims=True) if half_step == 2.0 ** -11 else 0.0
    err = (e + (half_step + 2.0 ** -20 + (n / 4 + 64) * 2.0 ** -24) * w + least) @ np.abs(v)
    return w @ v, err + (4e-4 * np.abs(v).max(axis=0) if mode == MODE_LSSAR and p >= 4 else 0.0)


def paged_attend(q, k_pages, v_pages, table, lens, counts, mode, p, half_step, rows=None):
    """{(b, h, t): (out [G, d], bound)} of the rows t < counts[b], or of those of
    them that are in rows[b]; G query heads of key head h."""
    hkv, G = k_pages.shape[1], q.shape[1] // k_pages.shape[1]
    got = {}
    for b, (n, count) in enumerate(zip(lens, counts)):
        if count == 0:
            continue
        kb, vb = gather(k_pages, table[b], n), gather(v_pages, table[b], n)
        for h in range(hkv):
            for t in range(count) if rows is None else [t for t in rows[b] if t < count]:
                i = n - count + t + 1
                got[b, h, t] = attend_row(q[b, h * G:(h + 1) * G, t], kb[:i, h], vb[:i, h], mode, p, half_step)
    return got


# ---------------------------------------------------------------- pages

def pages_of(n, page_size):
    return -(-n // page_size)


def reserve(table, lens, counts, page_size, free_pages, free_count):
    """The table after the call (a copy), counts_out and the free pages left."""
    table, out, taken, full = table.copy(), [], 0, False
    for b, (n, count) in enumerate(zip(lens, counts)):
        if n < 0 or count < 0 or n + count > table.shape[1] * page_size:
            out.append(0)
            continue
        have, want = pages_of(n, page_size), pages_of(n + count, page_size)
        if want > have and (full or taken + want - have > free_count):
            full = True
            out.append(0)
            continue
        for c in range(have, want):
            table[b, c] = free_pages[free_count - 1 - taken]
            taken += 1
        out.append(count)
    return table, out, free_count - taken


def release(table, lens, lens_new, page_size, free_pages, free_count):
    """The list after the call (a copy) and the number of free pages."""
    free_pages = free_pages.copy()
    for b, (n, m) in enumerate(zip(lens, lens_new)):
        if n < 0 or n > table.shape[1] * page_size or m < 0 or m > n:
            continue
        for c in range(pages_of(m, page_size), pages_of(n, page_size)):
            free_pages[free_count] = table[b, c]
            free_count += 1
    return free_pages, free_count
