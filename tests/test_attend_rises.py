"""Chunks over the paged cache whose rows' largest score rises from tile to tile
(one-pass modes: sums so far are rescaled, in the middle of a segment), against
the float64 oracle.  The values of a key undo its weight, so that every key, of
the first tile or the last, has an equal part in the output."""

import numpy as np
import pytest

from lssar_attn_fwd_gb300.inputs import MODE_LSSA, MODE_SOFTMAX
from oracle import paged_oracle as po
from oracle import serving_oracle as so
from test_paged import Cache, host, torch_mod  # noqa: F401

HEADS, LEN, ROWS = 24, 2000, 300
LOG2E = 1 / np.log(2)
TILE, HALF, ITEM_COST = 128, 64, 6

# mode, half precision, largest step that a reference lags behind, levels' first and step, the values' largest exponent
CASES = {
    "softmax-bf16": (MODE_SOFTMAX, False, 8.0, 0.0, 9.5, 60.0),
    "softmax-fp16": (MODE_SOFTMAX, True, 3.875, 0.0, 4.5, 60.0),
    "lssa-bf16-below": (MODE_LSSA, False, 8.0, -44.0, 9.5, 60.0),
    "lssa-bf16-through": (MODE_LSSA, False, 8.0, -30.0, 9.5, 10.0),
    "lssa-fp16-below": (MODE_LSSA, True, 6.0, -27.0, 6.5, 60.0),
    "lssa-fp16-through": (MODE_LSSA, True, 6.0, -20.0, 6.5, 10.0),
}


def inputs(case, d, seed):
    """q [HEADS, ROWS, d], k and v [HEADS, LEN, d] in float64, before their rounding."""
    mode, half, _, first, step, cap = CASES[case]
    g = np.random.default_rng(seed)
    # a head's level steps up at some of its 64-key halves, at a key somewhere within
    n_halves = -(-LEN // HALF)
    up = (g.random((HEADS, n_halves)) < 0.3) & (np.cumsum(np.ones(n_halves)) > 1)
    at = np.arange(n_halves) * HALF + g.integers(0, HALF, (HEADS, n_halves))
    j = np.arange(LEN)
    level = np.zeros((HEADS, LEN))
    for h in range(HEADS):
        for i in range(n_halves):
            if up[h, i]:
                level[h, j >= at[h, i]] += 1
    level = first + step * np.minimum(level, 4)
    z = level - 3 * g.random((HEADS, LEN)) * (np.diff(level, axis=1, prepend=-1e9) == 0)
    # rows that lean towards the keys by different amounts, one of them away
    lean = np.array([1.0, 0.97, 0.7, 0.45, -0.2])[np.arange(ROWS) % 5]
    q, k = np.zeros((HEADS, ROWS, d)), 0.5 * g.standard_normal((HEADS, LEN, d))
    if mode == MODE_SOFTMAX:
        q[:, :, 0], q[:, :, 1:] = 16 * lean, 0.02 * g.standard_normal((HEADS, ROWS, d - 1))
        k[:, :, 0] = z / LOG2E * np.sqrt(d) / 16
    else:
        q[:, :, 0], q[:, :, 1] = lean, np.sqrt(1 - lean ** 2)
        cos = np.maximum(z / (LOG2E * float(po.length_scale(LEN, d))), -0.98)
        k[:, :, 0] = k[:, :, 1] = 0
        k /= np.linalg.norm(k, axis=2, keepdims=True)
        k = np.sqrt(1 - cos ** 2)[..., None] * k
        k[:, :, 0] = cos
        k *= np.sqrt(d)
    top = 14.0 - (0 if mode == MODE_SOFTMAX else -first) if half else 0.0
    v = 2.0 ** np.minimum(top - level, cap)[..., None] * (1 + 0.5 * g.standard_normal((HEADS, LEN, d)))
    return q, k, v


def segments(sms):
    """(head, first token, rows, tiles of each row slot): the plan's equal runs of the numbered work."""
    items = []
    for t0 in range(0, ROWS, 256):
        rows = min(256, ROWS - t0)
        each = 2 if rows > TILE else 1
        items += [(h, t0, rows, each, ITEM_COST + each * -(-(LEN - ROWS + t0 + rows) // TILE)) for h in range(HEADS)]
    starts = np.cumsum([0] + [x[-1] for x in items])
    run = max(2, -(-int(starts[-1]) // sms))
    got = []
    for cta in range(-(-int(starts[-1]) // run)):
        for (h, t0, rows, each, cost), start in zip(items, starts):
            a, b = max(cta * run, start) - start, min((cta + 1) * run, start + cost) - start
            kt0, kt1 = max(a - ITEM_COST, 0) // each, max(b - ITEM_COST, 0) // each
            if a < b and kt0 < kt1:
                step = 1 if rows > TILE else 2
                got.append((h, t0, rows, [range(kt0 + (w if step == 2 else 0), kt1, step) for w in range(2)]))
    return got


def rises(case, d, z, sms):
    """How often a row's reference rises behind a segment's first tile, by place."""
    mode, _, lag, *_ = CASES[case]
    halves = -(-LEN // TILE) * 2
    turns = mode == MODE_SOFTMAX and d == 128
    got = dict(first=0, second=0, last_second=0, consecutive=0, some=0, to_zero=0, longest=0)
    limit = LEN - ROWS + np.arange(ROWS)
    for h, t0, rows, slots in segments(sms):
        zz = np.full((rows, halves * HALF), -np.inf)
        zz[:, :LEN] = np.where(np.arange(LEN) <= limit[t0:t0 + rows, None], z[h, t0:t0 + rows], -np.inf)
        tops = zz.reshape(rows, halves, HALF).max(axis=2)
        for w, tiles in enumerate(slots):
            mine = slice(w * TILE, (w + 1) * TILE) if rows > TILE else slice(0, rows)
            x = tops[mine]
            if len(tiles) == 0 or len(x) == 0:
                continue
            got["longest"] = max(got["longest"], len(tiles))
            ref = x[:, 2 * tiles[0]:2 * tiles[0] + 2].max(axis=1)
            if mode == MODE_LSSA:
                ref = np.minimum(ref, 0)
            before = np.zeros(len(x), bool)
            for kt in tiles[1:]:
                for half in range(2):
                    if turns:
                        top = x[:, 2 * kt + half]
                    elif half == 1:
                        before = np.zeros(len(x), bool)
                        continue
                    else:
                        top = x[:, 2 * kt:2 * kt + 2].max(axis=1)
                    if mode == MODE_LSSA:
                        top = np.minimum(top, 0)
                    zero = (mode == MODE_LSSA) & (top >= 0) & (ref < 0)
                    with np.errstate(invalid="ignore"):           # (-inf - -inf: nothing seen yet, no rise)
                        up = (top - ref > lag + 0.25) | zero      # (by a margin: not a matter of rounding)
                    got["second" if half else "first"] += up.sum()
                    got["last_second"] += up.sum() if half and kt == tiles[-1] else 0
                    got["consecutive"] += (up & before).sum()
                    got["to_zero"] += zero.sum()
                    for warp in range(0, len(x), 32):
                        part = up[warp:warp + 32]
                        got["some"] += bool(part.any() and not part.all())
                    ref, before = np.where(up, top, ref), up
    return got


def scores(case, d, q, k):
    """log2 units, [HEADS, ROWS, LEN]."""
    if CASES[case][0] == MODE_SOFTMAX:
        return q @ k.transpose(0, 2, 1) * (LOG2E / np.sqrt(d))
    unit = lambda x: x / np.linalg.norm(x, axis=2, keepdims=True)   # noqa: E731
    i = LEN - ROWS + 1 + np.arange(ROWS)
    return unit(q) @ unit(k).transpose(0, 2, 1) * (LOG2E * np.log(d) * np.log(i))[:, None]


def check_rises(case, d, q, k, sms):
    """What the test is for does happen: more than one tile to a slot, rises in every place."""
    got = rises(case, d, scores(case, d, q, k), sms)
    assert got["longest"] >= 4, got
    needed = ["first", "some"]
    if CASES[case][0] == MODE_SOFTMAX and d == 128:
        needed += ["second", "last_second", "consecutive"]
    if "through" in case:
        needed.append("to_zero")
    assert all(got[x] > 10 for x in needed), got


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", CASES)
def test_the_inputs_rise_in_every_place(case, d):
    q, k, _ = inputs(case, d, d)
    check_rises(case, d, q, k, 152)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", CASES)
def test_references_that_rise(torch_mod, case, d):
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    mode, half, *_ = CASES[case]
    c = Cache(torch, [LEN], HEADS, d, 16, half=half, seed=1)
    q, k, v = (torch.from_numpy(x).to(c.dt).cuda() for x in inputs(case, d, d))
    slot = torch.arange(LEN).cuda()
    pages, rows = c.table[0].long()[slot // 16], slot % 16
    c.k[pages, :, rows], c.v[pages, :, rows] = k.transpose(0, 1), v.transpose(0, 1)
    check_rises(case, d, host(q), host(k), torch.cuda.get_device_properties(0).multi_processor_count)
    outs = [api.lssar_paged_attend(q[None], *c.args(), mode=mode) for _ in range(2)]
    assert api.device_error_word() == 0
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))
    got, qh, kh, vh = host(outs[0])[0], host(q), host(k), host(v)
    half_step = torch.finfo(c.dt).eps / 2
    tiny = 2.0 ** -25 if half else 0.0
    for h in range(HEADS):
        for t in [*range(0, 10), 31, 32, 63, 64, 95, 96, 127, 128, *range(129, 134), 200, 254, 255, 256, *range(257, 262), 298, 299]:
            i = LEN - ROWS + t + 1
            ref, err = so.attend_row(qh[h, t:t + 1], kh[h, :i], vh[h, :i], mode, 1, half_step)
            # rises: ten at most, with those of the parts' sum; each an exponential (2^-22) and a product
            err = err + 10 * 2.0 ** -21 * po.row_weights(qh[h, t:t + 1], kh[h, :i], mode, 1) @ np.abs(vh[h, :i])
            bad = np.abs(got[h, t] - ref) - (err + half_step * (np.abs(ref) + err) + tiny)
            assert bad.max() <= 0, (h, t, bad.max(), err.max(), np.abs(ref).max())
