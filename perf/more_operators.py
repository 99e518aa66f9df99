"""Measured cases of a serving step around the paged cache, and of rotary positions.

A serving program that takes prompts in chunks reserves pages for the new
tokens, turns queries and keys by their positions while the keys and values go
to their pages, and computes the attention of the chunk's rows over all cached
tokens (in one of the modes of this repository); pages of finished or cut
sequences go back to the pool.  A training program turns queries and keys
before the attention, and their gradients back after it.

``run`` computes these in plain torch operations, or, with ``own`` set, by the
package's kernels.  ``exact`` is the same from the definitions in float64.
"""

import math

import numpy as np
import torch

own = False

SOFTMAX, LSSA, LSSAR, SOFTMAX_RW, SIGMOID_RW = range(5)   # the package's modes


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a short follow-up question of one user: all latency (12 heads of 64, as the GPT-2-small shape)
        {"name": "attend 64 on 200", "op": "attend", "B": 1, "H": 12, "Hkv": 12, "d": 64, "page": 16, "past_lo": 200,
         "past_hi": 200, "n": 64, "least": 64, "mode": LSSAR, "p": 3, "half": False},
        # the last chunk of a 16K prompt, the dense decode workload's length
        {"name": "attend 2K on 14K", "op": "attend", "B": 1, "H": 12, "Hkv": 12, "d": 64, "page": 64, "past_lo": 14336,
         "past_hi": 14336, "n": 2048, "least": 2048, "mode": LSSAR, "p": 15, "half": False},
        # a mixed batch in service: single tokens beside chunks, grouped heads, plain softmax, fp16
        {"name": "attend ragged grouped", "op": "attend", "B": 16, "H": 32, "Hkv": 8, "d": 128, "page": 32,
         "past_lo": 16, "past_hi": 7900, "n": 256, "least": 1, "mode": SOFTMAX, "p": 1, "half": True},
        # odd page size, lengths and counts, three query heads to a key head, the ablation on softmax
        {"name": "attend odd pages", "op": "attend", "B": 6, "H": 12, "Hkv": 4, "d": 64, "page": 24, "past_lo": 1,
         "past_hi": 4301, "n": 777, "least": 99, "mode": SOFTMAX_RW, "p": 3, "half": False},
        # whole prompts in one chunk, heads of the wide workload
        {"name": "attend whole prompts", "op": "attend", "B": 4, "H": 16, "Hkv": 16, "d": 128, "page": 16, "past_lo": 0,
         "past_hi": 0, "n": 4096, "least": 4096, "mode": LSSA, "p": 1, "half": False},
        # a chunk at the end of a very long context, eight query heads to a key head
        {"name": "attend 512 on 128K", "op": "attend", "B": 1, "H": 16, "Hkv": 2, "d": 128, "page": 128,
         "past_lo": 130000, "past_hi": 130000, "n": 512, "least": 512, "mode": LSSAR, "p": 15, "half": False},
        # a training step's queries and keys at the GPT-2-small shape, as slices of one projection
        {"name": "rope GPT-2", "op": "rope", "B": 8, "H": 12, "Hkv": 12, "L": 1024, "d": 64, "rot": 64,
         "interleaved": False, "scaling": "none", "back": False, "far": 0, "half": False},
        # gradients of the wide workload, half of each head turned, long-context frequencies
        {"name": "rope wide, back", "op": "rope", "B": 4, "H": 16, "Hkv": 16, "L": 4096, "d": 128, "rot": 64,
         "interleaved": True, "scaling": "bands", "back": True, "far": 0, "half": False},
        # the positions and the append of every decode step
        {"name": "append turned 1 token", "op": "append", "B": 8, "H": 12, "Hkv": 12, "d": 64, "page": 16,
         "past_lo": 100, "past_hi": 16000, "n": 1, "least": 1, "rot": 64, "interleaved": False, "scaling": "none",
         "far": 0, "track": True, "half": False},
        # a batch of prompts, padded to the longest, grouped heads, far positions
        {"name": "append turned prompts", "op": "append", "B": 6, "H": 32, "Hkv": 8, "d": 128, "page": 16,
         "past_lo": 1, "past_hi": 900, "n": 4096, "least": 700, "rot": 128, "interleaved": False, "scaling": "bands",
         "far": 1000000, "track": True, "half": False},
        # the pages of a decode step of many users, one new token each
        {"name": "reserve 256 users", "op": "reserve", "B": 256, "page": 16, "past_lo": 1, "past_hi": 16000, "n": 1,
         "least": 1, "enough": True},
        # sequences that have ended, that an eviction has cut, and that go on
        {"name": "release 96 of 32K", "op": "release", "B": 96, "page": 16, "past_lo": 3, "past_hi": 32000, "n": 0,
         "least": 0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "rope", "append", "reserve", "release"])
    d = rng.choice([64, 128])
    page = rng.choice([8, 16, 24, 32, 64, 96, 128, 256])
    half = rng.random() < 0.3
    hkv = rng.choice([1, 2, 3, 4, 8, 12, 16])
    group = rng.choice([1, 1, 2, 3, 4, 7, 8])
    turn = {"rot": rng.choice([d, d, d // 2, 48, 16]), "interleaved": rng.random() < 0.4,
            "scaling": rng.choice(["none", "none", "linear", "base", "bands"])}
    if op == "attend":
        mode = rng.choice([SOFTMAX, LSSA, LSSAR, LSSAR, SOFTMAX_RW, SIGMOID_RW])
        p = rng.choice([1, 2, 3, 15]) if mode >= LSSAR else 1
        B = _log_int(rng, 1, 32)
        most = 500_000_000 // (B * hkv * group)               # scores of the padded batch
        n = _log_int(rng, 1, min(4096, max(2, int(math.sqrt(most)))))
        past = _log_int(rng, 1, max(2, min(131072, most // n, 200_000_000 // (B * hkv * d)))) - 1
        return {"op": op, "B": B, "H": hkv * group, "Hkv": hkv, "d": d, "page": page,
                "past_lo": rng.randrange(past + 1), "past_hi": past, "n": n, "least": rng.randrange(1, n + 1),
                "mode": mode, "p": p, "half": half}
    if op == "rope":
        B = _log_int(rng, 1, 16)
        L = _log_int(rng, 1, min(32768, 33_000_000 // (B * hkv * (group + 1) * d)))
        return {"op": op, "B": B, "H": hkv * group, "Hkv": hkv, "L": L, "d": d, **turn, "back": rng.random() < 0.5,
                "far": rng.choice([0, 0, 5000, 1000000]), "half": half}
    if op == "append":
        B = _log_int(rng, 1, 32)
        n = _log_int(rng, 1, min(8192, 100_000_000 // (B * hkv * (group + 2) * d)))
        past = _log_int(rng, 1, 4000)
        return {"op": op, "B": B, "H": hkv * group, "Hkv": hkv, "d": d, "page": page,
                "past_lo": rng.randrange(past + 1), "past_hi": past, "n": n, "least": rng.randrange(n + 1), **turn,
                "far": rng.choice([0, 0, 5000, 1000000]), "track": rng.random() < 0.7, "half": half}
    B = _log_int(rng, 1, 2000)
    past = _log_int(rng, 1, min(131072, 40_000_000 // B))
    if op == "release":
        return {"op": op, "B": B, "page": page, "past_lo": rng.randrange(past + 1), "past_hi": past, "n": 0, "least": 0}
    n = _log_int(rng, 1, min(32768, 20_000_000 // B))
    return {"op": op, "B": B, "page": page, "past_lo": rng.randrange(past + 1), "past_hi": past, "n": n,
            "least": rng.randrange(n + 1), "enough": rng.random() < 0.7}


def _spread(lo, hi, count, step):
    """`count` whole numbers from lo to hi, evenly over their logarithm, in a fixed mixed order."""
    if count == 1:
        return np.array([hi], dtype=np.int64)
    while math.gcd(step, count) > 1:
        step += 1
    f = np.arange(count, dtype=np.int64) * step % count / (count - 1)
    return np.rint((hi + 1.0) ** f * (lo + 1.0) ** (1 - f)).astype(np.int64) - 1


def _past(case):
    return _spread(case["past_lo"], case["past_hi"], case["B"], 7)


def _counts(case):
    return _spread(case["least"], case["n"], case["B"], 5)


def work(case):
    if case["op"] == "rope":
        rows = float(case["B"]) * case["L"] * (case["H"] + case["Hkv"])
        return {"bytes": rows * case["d"] * 4 + 4 * case["B"], "flops": 3 * rows * case["rot"]}
    B, past, new = case["B"], _past(case).astype(np.float64), _counts(case).astype(np.float64)
    pages = lambda n: np.ceil(n / case["page"])            # noqa: E731
    if case["op"] == "reserve":
        return {"bytes": 12.0 * B + 8 * float((pages(past + new) - pages(past)).sum()), "flops": 0}
    if case["op"] == "release":
        return {"bytes": 8.0 * B + 4 * float(pages(past).sum()), "flops": 0}
    H, hkv, d = case["H"], case["Hkv"], case["d"]
    table = 4 * float(pages(past + new).sum()) + 8 * B
    if case["op"] == "append":
        rows = float(new.sum())
        return {"bytes": rows * (4 * d * (H + 2 * hkv) + (8 * hkv if case["track"] else 0)) + table + 4 * B,
                "flops": 3 * rows * (H + hkv) * case["rot"]}
    pairs = float((new * past + new * (new + 1) / 2).sum())
    return {"bytes": 4 * d * hkv * float(((past + new) * (new > 0)).sum()) + 4 * d * H * float(new.sum()) + table,
            "flops": 4 * pairs * H * d}


# ---------------------------------------------------------------- inputs

ORIGINAL, FACTOR, LOW, HIGH, BASE = 4096, 8.0, 1.0, 32.0, 10000.0   # of the long-context frequencies


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, B = case["op"], case["B"]
    s = dict(case)
    ints = lambda x: torch.from_numpy(np.asarray(x).astype(np.int32)).cuda()     # noqa: E731
    if op in ("reserve", "release"):
        return _prepare_pages(case, s, g, ints)
    d, H, hkv = case["d"], case["H"], case["Hkv"]
    dt = torch.float16 if case["half"] else torch.bfloat16
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda", dtype=dt)    # noqa: E731
    if op != "attend":
        from_far = torch.randint(0, 1000, (B,), generator=g, device="cuda", dtype=torch.int32) + case["far"]
        s["rotary"] = _rotary(case)
    if op == "rope":
        # queries and keys (or their gradients) as slices of one projection's output [B, L, H + Hkv, d]
        both = normal(B, case["L"], H + hkv, d)
        s["q"], s["k"], s["first"] = both[:, :, :H].transpose(1, 2), both[:, :, H:].transpose(1, 2), from_far
        return s
    ps, n = case["page"], case["n"]
    past, new = _past(case), _counts(case)
    pages_each = -(-max(1, int((past + new).max())) // ps)
    n_pages = B * pages_each + 3
    # pages in no order, as a pool that has been in use hands them out
    order = torch.randperm(n_pages, generator=g, device="cuda")
    s["table"] = order[:B * pages_each].reshape(B, pages_each).to(torch.int32)
    s["k_pages"], s["v_pages"] = normal(n_pages, hkv, ps, d), normal(n_pages, hkv, ps, d)
    s["counts"] = ints(new)
    if op == "append":
        s["lens"], cap = ints(past), pages_each * ps
        # queries, keys and values as slices of one projection's output
        both = normal(B, n, H + 2 * hkv, d).transpose(1, 2)
        s["q"], s["k_new"], s["v_new"] = both[:, :H], both[:, H:H + hkv], both[:, H + hkv:]
        s["first"] = s["lens"] + from_far
        s["q_out"] = torch.zeros(B, H, n, d, device="cuda", dtype=dt)
        track = case["track"]
        s["scores"] = torch.rand(B, hkv, cap, generator=g, device="cuda") if track else None
        s["positions"] = torch.arange(cap, device="cuda", dtype=torch.int32).repeat(B, hkv, 1) if track else None
        return s
    s["lens"] = ints(past + new)
    # queries that lean towards one cached key each, as trained heads do
    i = (s["lens"] - s["counts"])[:, None, None] + torch.arange(1, n + 1, device="cuda")
    j = (torch.rand(B, hkv, n, generator=g, device="cuda") * i).long().clamp(max=int((past + new).max()) - 1)
    b, h = torch.arange(B, device="cuda")[:, None, None], torch.arange(hkv, device="cuda")[None, :, None]
    k = s["k_pages"][s["table"][b, j // ps].long(), h, j % ps].float()
    k = 0.5 * k / k.norm(dim=-1, keepdim=True).clamp(min=1e-6)
    noise = torch.randn(B, hkv, H // hkv, n, d, generator=g, device="cuda") / math.sqrt(d)
    q = (math.sqrt(d) * (k[:, :, None] + noise)).to(dt).reshape(B, H, n, d)
    s["q"] = q.transpose(1, 2).contiguous().transpose(1, 2)        # as a projection's output [B, n, H, d]
    s["out"] = torch.zeros(B, H, n, d, device="cuda", dtype=dt)
    return s


def _prepare_pages(case, s, g, ints):
    B, ps = case["B"], case["page"]
    past, new = _past(case), _counts(case)
    have, want = -(-past // ps), -(-(past + new) // ps)
    width = max(1, int(want.max()))
    n_pages = max(1, int(want.sum())) + 5
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    # the pages that the sequences hold, and the rest of the pool in a list of free pages
    held = torch.arange(width, device="cuda") < ints(have)[:, None]
    s["table"] = torch.full((B, width), -1, device="cuda", dtype=torch.int32)
    used = int(have.sum())
    s["table"][held] = order[:used]
    s["free_pages"] = torch.cat([order[used:], order[:used]])
    s["lens"], s["counts"] = ints(past), ints(new)
    if case["op"] == "reserve":
        left = n_pages - used
        s["free_count"] = ints([left if case["enough"] else left * 2 // 3])
    else:
        s["free_count"] = ints([n_pages - used])
        # a third has ended, a third was cut, a third stays as it is
        fate = torch.randint(0, 3, (B,), generator=g, device="cuda")
        cut = (torch.rand(B, generator=g, device="cuda") * s["lens"]).to(torch.int32)
        s["lens_new"] = torch.where(fate == 0, 0, torch.where(fate == 1, torch.minimum(cut, s["lens"]), s["lens"])).to(torch.int32)
    return s


def _rotary(case):
    """The description that a program keeps beside its model's configuration."""
    return {"d": case["d"], "rot_dim": case["rot"], "base": BASE, "interleaved": case["interleaved"],
            "scaling": case["scaling"], "factor": FACTOR, "original_length": ORIGINAL, "low": LOW, "high": HIGH}


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _own(s)
    return {"attend": _attend, "rope": _rope, "append": _append, "reserve": _reserve, "release": _release}[s["op"]](s)


def _own(s):
    from lssar_attn_fwd_gb300 import api
    op = s["op"]
    if op == "attend":
        return [api.lssar_paged_attend(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], counts=s["counts"],
                                       p=s["p"], mode=s["mode"], out=s["out"])]
    if op == "reserve":
        counts, left = api.lssar_paged_reserve(s["table"], s["lens"], s["counts"], s["page"], s["free_pages"],
                                               s["free_count"])
        return [counts, left, s["table"]]
    if op == "release":
        left = api.lssar_paged_release(s["table"], s["lens"], s["lens_new"], s["page"], s["free_pages"], s["free_count"])
        return [left, s["free_pages"]]
    rotary = api.Rotary(**s["rotary"])
    if op == "rope":
        turn = api.lssar_rope_bwd if s["back"] else api.lssar_rope
        return list(turn(s["q"], s["k"], rotary, positions=s["first"]))
    q, lens = api.lssar_paged_append_rope(s["q"], s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], s["table"],
                                          s["lens"], rotary, counts=s["counts"], first_positions=s["first"],
                                          scores=s["scores"], positions=s["positions"], q_out=s["q_out"])
    kept = [] if s["scores"] is None else [s["scores"], s["positions"]]
    return [q, lens, s["k_pages"], s["v_pages"]] + kept


def _rows(pages, table):
    """The cached rows of every sequence, [B, Hkv, slots, d]."""
    x = pages[table.long()].permute(0, 2, 1, 3, 4)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[4])


def _attend(s):
    mode, p, n = s["mode"], s["p"], s["n"]
    k, v = _rows(s["k_pages"], s["table"]).float(), _rows(s["v_pages"], s["table"]).float()
    B, hkv, cap, d = k.shape
    q = s["q"].float().reshape(B, hkv, -1, n, d)
    t = torch.arange(n, device=q.device)
    i = ((s["lens"] - s["counts"])[:, None] + t + 1).view(B, 1, 1, n, 1)     # tokens that row t attends to
    there = torch.arange(cap, device=q.device) < i                          # [B, 1, 1, n, cap]
    f = i.clamp(min=1).float()
    k, v = k[:, :, None], v[:, :, None]
    if mode in (SOFTMAX, SOFTMAX_RW):
        x = (q @ k.transpose(-1, -2) / math.sqrt(d)).masked_fill(~there, -math.inf)
        a = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-3e38))
    else:
        q = q / q.square().sum(-1, keepdim=True).sqrt().clamp(min=1e-12)
        k = k / k.square().sum(-1, keepdim=True).sqrt().clamp(min=1e-12)
        x = q @ k.transpose(-1, -2) * (math.log(d) * torch.log(f))
        e = torch.exp(-x.abs())
        a = torch.where(x >= 0, 1 / (1 + e), e / (1 + e)) if mode == SIGMOID_RW else x.clamp(min=0) + torch.log1p(e)
        a = a * there
    w = a / a.sum(-1, keepdim=True).clamp(min=1e-30)
    if mode >= LSSAR:
        y = (f * w - (f > 3).float()).clamp(min=0) * there
        top = y.amax(-1, keepdim=True)
        r = torch.where(top > 0, (y / top.clamp(min=1e-30)) ** p, there.float())
        w = r / r.sum(-1, keepdim=True).clamp(min=1e-30)
    out = (w @ v).reshape(B, -1, n, d).to(s["q"].dtype)
    live = (t < s["counts"][:, None]).view(B, 1, n, 1)                       # rows behind a sequence's count stay
    return [torch.where(live, out, s["out"])]


def _frequencies(r, device):
    """Radians per position of each pair, in float64."""
    at = torch.arange(0, r["rot_dim"], 2, device=device, dtype=torch.float64) / r["rot_dim"]
    if r["scaling"] == "base":
        return (r["base"] * r["factor"] ** (r["rot_dim"] / (r["rot_dim"] - 2))) ** -at
    f = r["base"] ** -at
    if r["scaling"] == "linear":
        f = f / r["factor"]
    elif r["scaling"] == "bands":
        turns = r["original_length"] * f / (2 * math.pi)
        keep = ((turns - r["low"]) / (r["high"] - r["low"])).clamp(0, 1)
        f = f * (keep + (1 - keep) / r["factor"])
    return f


def _turn(x, first, r, sign):
    """x [B, H, n, d] turned by the angles of positions first[b] + t."""
    n, rot = x.shape[2], r["rot_dim"]
    at = (first[:, None] + torch.arange(n, device=x.device)).double()
    angle = at[:, None, :, None] * _frequencies(r, x.device)               # [B, 1, n, rot / 2]
    c, s = torch.cos(angle).float(), sign * torch.sin(angle).float()
    y = x.float()
    if r["interleaved"]:
        u, v = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([u * c - v * s, u * s + v * c], dim=-1).flatten(-2)
    else:
        u, v = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([u * c - v * s, u * s + v * c], dim=-1)
    return torch.cat([turned, y[..., rot:]], dim=-1).to(x.dtype)


def _rope(s):
    sign = -1.0 if s["back"] else 1.0
    return [_turn(x, s["first"], s["rotary"], sign) for x in (s["q"], s["k"])]


def _append(s):
    lens, ps, n = s["lens"].long(), s["page"], s["n"]
    q, k = _turn(s["q"], s["first"], s["rotary"], 1.0), _turn(s["k_new"], s["first"], s["rotary"], 1.0)
    live = torch.arange(n, device=lens.device) < s["counts"][:, None]
    b, t = live.nonzero(as_tuple=True)
    slot = lens[b] + t
    page = s["table"][b, slot // ps].long()
    s["k_pages"][page, :, slot % ps] = k[b, :, t]
    s["v_pages"][page, :, slot % ps] = s["v_new"][b, :, t]
    q = torch.where(live[:, None, :, None], q, s["q_out"])
    out = [q, (lens + s["counts"]).to(torch.int32), s["k_pages"], s["v_pages"]]
    if s["scores"] is None:
        return out
    s["scores"][b, :, slot] = 0.0
    s["positions"][b, :, slot] = (s["first"][b] + t).to(torch.int32)[:, None]
    return out + [s["scores"], s["positions"]]


def _reserve(s):
    ps, lens, counts, free = s["page"], s["lens"].long(), s["counts"].long(), s["free_count"].long()
    have, want = (lens + ps - 1) // ps, (lens + counts + ps - 1) // ps
    need = want - have
    end = need.cumsum(0)
    served = (need == 0) | (end <= free)
    column = torch.arange(s["table"].shape[1], device=lens.device)
    new = (column >= have[:, None]) & (column < want[:, None]) & served[:, None]
    from_top = (end - need - have)[:, None] + column                       # pages taken before this one
    page = s["free_pages"][(free - 1 - from_top).clamp(0, s["free_pages"].numel() - 1)]
    s["table"].copy_(torch.where(new, page, s["table"]))
    left = free - torch.where(end <= free, end, 0).amax()
    return [torch.where(served, counts, 0).to(torch.int32), left.to(torch.int32), s["table"]]


def _release(s):
    ps, free = s["page"], s["free_count"].long()
    have, keep = (s["lens"].long() + ps - 1) // ps, (s["lens_new"].long() + ps - 1) // ps
    gone = have - keep
    end = gone.cumsum(0)
    column = torch.arange(s["table"].shape[1], device=free.device)
    b, c = ((column >= keep[:, None]) & (column < have[:, None])).nonzero(as_tuple=True)
    s["free_pages"][free + (end - gone - keep)[b] + c] = s["table"][b, c]
    return [(free + end[-1]).to(torch.int32), s["free_pages"]]


# ---------------------------------------------------------------- float64

def exact(case, seed):
    """From the definitions in float64: the attention one sequence and one query
    head at a time, the turned rows by complex numbers; moved page numbers and
    copied rows are not computed."""
    if case["op"] in ("reserve", "release"):
        return None
    s = prepare(case, seed)
    if case["op"] == "attend":
        return [_exact_attend(case, s)]
    if case["op"] == "rope":
        return [_exact_turn(x, s["first"], s["rotary"], case["back"]).cpu() for x in (s["q"], s["k"])]
    q = _exact_turn(s["q"], s["first"], s["rotary"], False)
    key = _exact_turn(s["k_new"], s["first"], s["rotary"], False)
    q_out, pages, ps = s["q_out"].double(), s["k_pages"].double(), case["page"]
    for b, (n, count) in enumerate(zip(s["lens"].tolist(), s["counts"].tolist())):
        slot = torch.arange(n, n + count, device="cuda")
        q_out[b, :, :count] = q[b, :, :count]
        pages[s["table"][b, slot // ps].long(), :, slot % ps] = key[b, :, :count].transpose(0, 1)
    return [q_out.cpu(), None, pages.cpu(), None] + ([None, None] if case["track"] else [])


def _exact_attend(case, s):
    d, ps, group = case["d"], case["page"], case["H"] // case["Hkv"]
    out = s["out"].double()
    for b, (n, count) in enumerate(zip(s["lens"].tolist(), s["counts"].tolist())):
        pages = s["table"][b, :-(-n // ps)].long()
        for h in range(case["Hkv"]) if count else ():
            key = s["k_pages"][pages, h].reshape(-1, d)[:n].double()
            val = s["v_pages"][pages, h].reshape(-1, d)[:n].double()
            for g in range(group):
                rows = s["q"][b, h * group + g, :count].double()
                out[b, h * group + g, :count] = _exact_rows(rows, key, val, case["mode"], case["p"])
    return out.cpu()


def _exact_rows(q, key, val, mode, p):
    """The last len(q) rows of the attention over the keys."""
    count, n, d = len(q), len(key), q.shape[1]
    i = torch.arange(n - count + 1, n + 1, device="cuda", dtype=torch.float64)[:, None]
    ahead = torch.arange(n, device="cuda") >= i
    if mode in (SOFTMAX, SOFTMAX_RW):
        a = torch.softmax((torch.einsum("rd,jd->rj", q, key) / d ** 0.5).masked_fill_(ahead, -math.inf), dim=1)
    else:
        x = torch.einsum("rd,jd->rj", q, key)
        x /= torch.linalg.norm(q, dim=1).clamp(min=1e-12)[:, None]
        x /= torch.linalg.norm(key, dim=1).clamp(min=1e-12)
        x *= math.log(d) * torch.log(i)
        a = torch.sigmoid(x) if mode == SIGMOID_RW else torch.logaddexp(x, torch.zeros((), device="cuda", dtype=torch.float64))
        a.masked_fill_(ahead, 0.0)
        a /= a.sum(dim=1, keepdim=True)
    if mode >= LSSAR:
        y = torch.relu(i * a - (i >= 4).double())
        y = torch.where(y > 1e-10, y, torch.zeros_like(y)).masked_fill_(ahead, 0.0)     # a uniform row's residues of 0
        top = y.max(dim=1, keepdim=True).values
        r = torch.where(top > 0, (y / top.clamp(min=1e-300)).pow(p), (~ahead).double())
        a = r / r.sum(dim=1, keepdim=True)
    return torch.einsum("rj,jd->rd", a, val)


def _exact_turn(x, first, r, back):
    rot, half = r["rot_dim"], r["rot_dim"] // 2
    freq = []
    for c in range(half):
        f = math.pow(r["base"], -2.0 * c / rot)
        if r["scaling"] == "linear":
            f /= r["factor"]
        elif r["scaling"] == "base":
            f = math.pow(r["base"] * math.pow(r["factor"], rot / (rot - 2.0)), -2.0 * c / rot)
        elif r["scaling"] == "bands":
            keep = min(1.0, max(0.0, (r["original_length"] * f / math.tau - r["low"]) / (r["high"] - r["low"])))
            f *= keep + (1 - keep) / r["factor"]
        freq.append(f)
    at = first.double()[:, None] + torch.arange(x.shape[2], device="cuda", dtype=torch.float64)
    angle = torch.einsum("bt,c->btc", at, torch.tensor(freq, device="cuda", dtype=torch.float64))
    z = torch.polar(torch.ones_like(angle), -angle if back else angle)[:, None]
    y = x.double().clone()
    re, im = (slice(0, rot, 2), slice(1, rot, 2)) if r["interleaved"] else (slice(0, half), slice(half, rot))
    w = torch.complex(y[..., re], y[..., im]) * z
    y[..., re], y[..., im] = w.real, w.imag
    return y
