"""Measured cases of the paged-cache operators: append, decode and evict.

A serving program keeps the keys and values of its sequences in pages
(``k_pages, v_pages [n_pages, Hkv, page_size, d]``), a table of page numbers
per sequence and its length.  Each step it appends the new tokens' rows,
computes one query row per sequence (the attention of this repository, in one
of its modes) while it adds up the attention weight that every cached token
receives, and, when the cache is full, evicts the tokens of least weight.

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
        # a chat's first tokens, one user: all latency (12 heads of 64, as the GPT-2-small shape)
        {"name": "decode 1 user", "op": "decode", "B": 1, "H": 12, "Hkv": 12, "d": 64, "page": 16, "shortest": 200,
         "longest": 200, "mode": LSSAR, "p": 3, "scores": False, "half": False},
        # the 16K decode workload of the dense cache, with the weights added up for a later eviction
        {"name": "decode 8 x 16K", "op": "decode", "B": 8, "H": 12, "Hkv": 12, "d": 64, "page": 64, "shortest": 16384,
         "longest": 16384, "mode": LSSAR, "p": 15, "scores": True, "half": False},
        # a mixed batch in service: lengths over three decades, grouped heads, plain softmax, fp16
        {"name": "decode ragged grouped", "op": "decode", "B": 32, "H": 32, "Hkv": 8, "d": 128, "page": 32,
         "shortest": 17, "longest": 24576, "mode": SOFTMAX, "p": 1, "scores": False, "half": True},
        # many short sequences, heads of the wide workload
        {"name": "decode 64 short", "op": "decode", "B": 64, "H": 16, "Hkv": 16, "d": 128, "page": 16, "shortest": 1,
         "longest": 1500, "mode": LSSA, "p": 1, "scores": False, "half": False},
        # odd page size and lengths, three query heads to a key head, the ablation on softmax
        {"name": "decode odd pages", "op": "decode", "B": 48, "H": 12, "Hkv": 4, "d": 64, "page": 24, "shortest": 333,
         "longest": 5001, "mode": SOFTMAX_RW, "p": 3, "scores": True, "half": False},
        # two very long contexts, eight query heads to a key head
        {"name": "decode 2 x 128K", "op": "decode", "B": 2, "H": 16, "Hkv": 2, "d": 128, "page": 128,
         "shortest": 100001, "longest": 131071, "mode": LSSAR, "p": 15, "scores": True, "half": False},
        # the append of every decode step
        {"name": "append 1 token", "op": "append", "B": 8, "Hkv": 12, "d": 64, "page": 16, "shortest": 100,
         "longest": 16000, "n": 1, "least": 1, "track": True, "half": False},
        # a batch of prompts, padded to the longest, as slices of one fused projection
        {"name": "append prompts", "op": "append", "B": 6, "Hkv": 16, "d": 128, "page": 16, "shortest": 1,
         "longest": 900, "n": 4096, "least": 700, "track": True, "half": False},
        # long documents into a half-precision cache
        {"name": "append 8 x 32K", "op": "append", "B": 8, "Hkv": 8, "d": 128, "page": 64, "shortest": 0, "longest": 0,
         "n": 32768, "least": 32768, "track": False, "half": True},
        # the steady state: the cache at its bound, a few tokens over
        {"name": "evict a few", "op": "evict", "B": 8, "Hkv": 12, "d": 64, "page": 16, "shortest": 2049,
         "longest": 2056, "keep": 2048, "recent": 256, "sinks": 4, "fresh": False, "half": False},
        # a prompt cut to half after its decode has shown what is used
        {"name": "evict half", "op": "evict", "B": 8, "Hkv": 12, "d": 64, "page": 64, "shortest": 12001,
         "longest": 16384, "keep": 8192, "recent": 512, "sinks": 4, "fresh": True, "half": False},
        # long contexts cut to a quarter
        {"name": "evict 128K", "op": "evict", "B": 4, "Hkv": 8, "d": 128, "page": 128, "shortest": 90001,
         "longest": 131072, "keep": 32768, "recent": 1024, "sinks": 16, "fresh": True, "half": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "evict"])
    d = rng.choice([64, 128])
    page = rng.choice([8, 16, 24, 32, 64, 96, 128, 256])
    half = rng.random() < 0.3
    if op == "decode":
        hkv = rng.choice([1, 2, 3, 4, 8, 12, 16])
        group = rng.choice([1, 2, 3, 4, 7, 8])
        mode = rng.choice([SOFTMAX, LSSA, LSSAR, LSSAR, SOFTMAX_RW, SIGMOID_RW])
        p = rng.choice([1, 2, 3, 15]) if mode >= LSSAR else 1
        B = _log_int(rng, 1, 64)
        most = 400_000_000 // (B * hkv * d)      # cached elements as in the larger listed cases
        longest = _log_int(rng, 30, min(131072, most))
        shortest = max(1, min(longest, int(longest * rng.random())))
        return {"op": op, "B": B, "H": hkv * group, "Hkv": hkv, "d": d, "page": page, "shortest": shortest,
                "longest": longest, "mode": mode, "p": p, "scores": rng.random() < 0.5, "half": half}
    hkv = rng.choice([1, 2, 4, 8, 12, 16])
    if op == "append":
        B = _log_int(rng, 1, 48)
        n = _log_int(rng, 1, min(32768, 260_000_000 // (B * hkv * d)))
        longest = _log_int(rng, 1, 4000)
        return {"op": op, "B": B, "Hkv": hkv, "d": d, "page": page, "shortest": rng.randrange(longest + 1),
                "longest": longest, "n": n, "least": rng.randrange(n + 1), "track": rng.random() < 0.7, "half": half}
    B = _log_int(rng, 1, 16)
    longest = _log_int(rng, 64, min(131072, 520_000_000 // (B * hkv * d)))
    keep = max(24, int(longest * rng.uniform(0.2, 0.99)))
    return {"op": op, "B": B, "Hkv": hkv, "d": d, "page": page, "shortest": max(1, int(longest * rng.uniform(0.5, 1))),
            "longest": longest, "keep": keep, "recent": keep // rng.choice([2, 4, 16]), "sinks": rng.choice([0, 4]),
            "fresh": rng.random() < 0.5, "half": half}


def _spread(lo, hi, count):
    """`count` whole numbers from lo to hi, evenly over their logarithm, in a fixed mixed order."""
    at = np.arange(count, dtype=np.int64) * (7 if count % 7 else 5) % count if count > 7 else np.arange(count)[::-1]
    f = at / max(1, count - 1)
    return np.rint((hi + 1.0) ** f * (lo + 1.0) ** (1 - f)).astype(np.int64) - 1


def _lengths(case):
    return _spread(case["shortest"], case["longest"], case["B"])


def _counts(case):
    return _spread(case["least"], case["n"], case["B"])


def work(case):
    B, hkv, d = case["B"], case["Hkv"], case["d"]
    n = _lengths(case).astype(np.float64)
    table = 4 * float(np.ceil(n / case["page"]).sum()) + 4 * B
    if case["op"] == "decode":
        rows = float(n.sum()) * hkv
        return {"bytes": rows * d * 4 + 4 * B * case["H"] * d + table + (8 * rows if case["scores"] else 0),
                "flops": 4 * rows * (case["H"] // hkv) * d}
    if case["op"] == "append":
        rows = float(_counts(case).sum()) * hkv
        return {"bytes": rows * (8 * d + (8 if case["track"] else 0)) + table + 8 * B, "flops": 0}
    # a slot below `keep` is a hole as often as any unprotected slot is evicted
    keep, safe = case["keep"], case["recent"] + case["sinks"]
    over = np.maximum(n - keep, 0)
    holes = over * (keep - (safe if not case["fresh"] else case["sinks"])) / np.maximum(n - safe, 1)
    return {"bytes": float((8 * n + 8 * np.minimum(n, keep)).sum()) * hkv + 8.0 * d * hkv * float(holes.sum()) + table,
            "flops": 0}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, hkv, d, ps = case["B"], case["Hkv"], case["d"], case["page"]
    dt = torch.float16 if case["half"] else torch.bfloat16
    rand = lambda *shape: torch.rand(*shape, generator=g, device="cuda")       # noqa: E731
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda", dtype=dt)   # noqa: E731
    lens = torch.from_numpy(_lengths(case).astype(np.int32)).cuda()
    most = int(_lengths(case).max() if case["op"] != "append" else (_lengths(case) + _counts(case)).max())
    pages_each = -(-max(1, most) // ps)
    n_pages = B * pages_each + 3
    s = {"op": case["op"], "lens": lens, "p": case.get("p", 1), "mode": case.get("mode", LSSAR)}
    # pages in no order, as a pool that has been in use hands them out
    order = torch.randperm(n_pages, generator=g, device="cuda")
    s["table"] = order[:B * pages_each].reshape(B, pages_each).to(torch.int32)
    s["k_pages"], s["v_pages"] = normal(n_pages, hkv, ps, d), normal(n_pages, hkv, ps, d)
    cap = pages_each * ps
    if case["op"] == "decode":
        # queries that lean towards one cached key each, as trained heads do
        j = (rand(B, hkv) * lens[:, None].clamp(min=1)).long().clamp(max=most - 1)
        b, h = torch.arange(B, device="cuda")[:, None], torch.arange(hkv, device="cuda")[None]
        k = s["k_pages"][s["table"][b, j // ps].long(), h, j % ps].float()
        k = 0.5 * k / k.norm(dim=-1, keepdim=True).clamp(min=1e-6)
        noise = torch.randn(B, hkv, case["H"] // hkv, d, generator=g, device="cuda") / math.sqrt(d)
        s["q"] = (math.sqrt(d) * (k[:, :, None] + noise)).to(dt).reshape(B, case["H"], d)
        # weight that a few steps before have added up: about 1 / length each
        steps = 4 * case["H"] // hkv / lens.clamp(min=1).view(B, 1, 1)
        s["scores"] = rand(B, hkv, cap) * steps if case["scores"] else None
        s["scores_out"] = torch.zeros_like(s["scores"]) if case["scores"] else None
    elif case["op"] == "append":
        # keys and values as slices of one projection's output [B, n, 2, Hkv, d]
        both = normal(B, case["n"], 2, hkv, d)
        s["k_new"], s["v_new"] = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
        s["counts"] = torch.from_numpy(_counts(case).astype(np.int32)).cuda()
        s["first"] = lens + torch.randint(0, 1000, (B,), generator=g, device="cuda", dtype=torch.int32)
        track = case["track"]
        s["scores"] = rand(B, hkv, cap) if track else None
        s["positions"] = torch.arange(cap, device="cuda", dtype=torch.int32).repeat(B, hkv, 1) if track else None
    else:
        s["keep"], s["recent"], s["sinks"] = case["keep"], case["recent"], case["sinks"]
        # added-up weights: heavy tails, and many tokens that the re-weighting has never let through
        w = torch.exp(2 * torch.randn(B, hkv, cap, generator=g, device="cuda"))
        s["scores"] = torch.where(rand(B, hkv, cap) < 0.3, torch.zeros_like(w), w)
        at = torch.arange(cap, device="cuda", dtype=torch.int32).repeat(B, hkv, 1)
        s["positions"] = at if case["fresh"] else rand(B, hkv, cap).argsort(-1).to(torch.int32)
        s["scores_out"], s["positions_out"] = torch.zeros_like(s["scores"]), torch.zeros_like(s["positions"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _own(s)
    if s["op"] == "decode":
        return _decode(s)
    return _append(s) if s["op"] == "append" else _evict(s)


def _own(s):
    from lssar_attn_fwd_gb300 import api
    cache = s["k_pages"], s["v_pages"], s["table"], s["lens"]
    if s["op"] == "decode":
        out = api.lssar_paged_decode(s["q"], *cache, p=s["p"], mode=s["mode"], scores=s["scores"],
                                     scores_out=s["scores_out"])
        return [out] if s["scores"] is None else [out, s["scores_out"]]
    if s["op"] == "append":
        lens = api.lssar_paged_append(s["k_new"], s["v_new"], *cache, counts=s["counts"], first_positions=s["first"],
                                      scores=s["scores"], positions=s["positions"])
        kept = [] if s["scores"] is None else [s["scores"], s["positions"]]
        return [lens, s["k_pages"], s["v_pages"]] + kept
    lens, scores, positions = api.lssar_paged_evict(*cache, s["scores"], s["positions"], s["keep"], recent=s["recent"],
                                                    sinks=s["sinks"], scores_out=s["scores_out"],
                                                    positions_out=s["positions_out"])
    return [lens, scores, positions, s["k_pages"], s["v_pages"]]


def _rows(pages, table):
    """The cached rows of every sequence, [B, Hkv, slots, d]."""
    x = pages[table.long()].permute(0, 2, 1, 3, 4)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[4])


def _decode(s):
    q, mode, p = s["q"].float(), s["mode"], s["p"]
    k, v = _rows(s["k_pages"], s["table"]).float(), _rows(s["v_pages"], s["table"]).float()
    B, hkv, cap, d = k.shape
    q = q.reshape(B, hkv, -1, d)
    n = s["lens"].view(B, 1, 1, 1)
    there = torch.arange(cap, device=q.device) < n                     # [B, 1, 1, cap]
    nf = n.clamp(min=1).float()
    if mode in (SOFTMAX, SOFTMAX_RW):
        x = (q @ k.transpose(-1, -2) / math.sqrt(d)).masked_fill(~there, -math.inf)
        a = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-3e38))
    else:
        q = q / q.square().sum(-1, keepdim=True).sqrt().clamp(min=1e-12)
        k = k / k.square().sum(-1, keepdim=True).sqrt().clamp(min=1e-12)
        x = q @ k.transpose(-1, -2) * (math.log(d) * torch.log(nf))
        e = torch.exp(-x.abs())
        a = torch.where(x >= 0, 1 / (1 + e), e / (1 + e)) if mode == SIGMOID_RW else x.clamp(min=0) + torch.log1p(e)
        a = a * there
    w = a / a.sum(-1, keepdim=True).clamp(min=1e-30)
    if mode >= LSSAR:
        y = (nf * w - (nf > 3).float()).clamp(min=0) * there
        top = y.amax(-1, keepdim=True)
        r = torch.where(top > 0, (y / top.clamp(min=1e-30)) ** p, there.float())
        w = r / r.sum(-1, keepdim=True).clamp(min=1e-30)
    out = (w @ torch.where(there.transpose(-1, -2), v, 0.0)).reshape(s["q"].shape).to(s["q"].dtype)
    if s["scores"] is None:
        return [out]
    there = there[:, :, 0].expand_as(s["scores"])
    return [out, torch.where(there, s["scores"] + w.sum(2), s["scores_out"])]


def _append(s):
    lens, ps = s["lens"].long(), s["k_pages"].shape[2]
    n = s["k_new"].shape[2]
    b, t = (torch.arange(n, device=lens.device) < s["counts"][:, None]).nonzero(as_tuple=True)
    slot = lens[b] + t
    page = s["table"][b, slot // ps].long()
    s["k_pages"][page, :, slot % ps] = s["k_new"][b, :, t]
    s["v_pages"][page, :, slot % ps] = s["v_new"][b, :, t]
    out = [(lens + s["counts"]).to(torch.int32), s["k_pages"], s["v_pages"]]
    if s["scores"] is None:
        return out
    s["scores"][b, :, slot] = 0.0
    s["positions"][b, :, slot] = (s["first"][b] + t).to(torch.int32)[:, None]
    return out + [s["scores"], s["positions"]]


def _evict(s):
    scores, positions, ps = s["scores"], s["positions"], s["k_pages"].shape[2]
    cap = scores.shape[2]
    n = s["lens"].long().view(-1, 1, 1)
    new = n.clamp(max=s["keep"])
    slot = torch.arange(cap, device=scores.device)
    there = slot < n
    newest = positions.masked_fill(~there, -1).amax(-1, keepdim=True)
    safe = (positions < s["sinks"]) | (positions > newest - s["recent"])
    rank = torch.where(safe, math.inf, scores).masked_fill(~there, -math.inf)
    order = rank.sort(dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(there.expand_as(scores)).scatter(-1, order, (slot < new).expand_as(scores))
    b, h, dst = ((slot < new) & ~kept).nonzero(as_tuple=True)
    _, _, src = (kept & (slot >= new)).nonzero(as_tuple=True)
    to, of = s["table"][b, dst // ps].long(), s["table"][b, src // ps].long()
    s["k_pages"][to, h, dst % ps] = s["k_pages"][of, h, src % ps]
    s["v_pages"][to, h, dst % ps] = s["v_pages"][of, h, src % ps]
    out = []
    live = (slot < new).expand_as(scores)
    moved = scores.clone(), positions.clone()
    moved[0][b, h, dst], moved[1][b, h, dst] = scores[b, h, src], positions[b, h, src]
    out = [torch.where(live, moved[0], s["scores_out"]), torch.where(live, moved[1], s["positions_out"])]
    return [new.view(-1).to(torch.int32)] + out + [s["k_pages"], s["v_pages"]]


# ---------------------------------------------------------------- float64

def exact(case, seed):
    """The decode step from its definition, one sequence and one key head at a
    time, in float64; appended and evicted rows are copies, not computed."""
    if case["op"] != "decode":
        return None
    s = prepare(case, seed)
    d, ps, group = case["d"], case["page"], case["H"] // case["Hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64)
    tracked = s["scores"] is not None
    added = s["scores_out"].double().cpu() if tracked else None
    for b, i in enumerate(s["lens"].tolist()):
        if i == 0:
            continue
        pages = s["table"][b, :-(-i // ps)].long()
        for h in range(case["Hkv"]):
            key = s["k_pages"][pages, h].reshape(-1, d)[:i].double()
            val = s["v_pages"][pages, h].reshape(-1, d)[:i].double()
            qs = s["q"][b, h * group:(h + 1) * group].double()
            if case["mode"] in (SOFTMAX, SOFTMAX_RW):
                a = torch.softmax(torch.einsum("gd,jd->gj", qs, key) / d ** 0.5, dim=1)
            else:
                cos = torch.einsum("gd,jd->gj", qs, key)
                cos = cos / torch.linalg.norm(qs, dim=1).clamp(min=1e-12)[:, None]
                cos = cos / torch.linalg.norm(key, dim=1).clamp(min=1e-12)
                x = math.log(d) * math.log(i) * cos
                a = torch.sigmoid(x) if case["mode"] == SIGMOID_RW else torch.logaddexp(x, torch.zeros_like(x))
                a = a / a.sum(dim=1, keepdim=True)
            if case["mode"] >= LSSAR:
                y = torch.relu(i * a - (1.0 if i >= 4 else 0.0))
                y = torch.where(y > 1e-10, y, torch.zeros_like(y))     # a uniform row's residues of 0
                top = y.max(dim=1, keepdim=True).values
                r = torch.where(top > 0, (y / top.clamp(min=1e-300)).pow(case["p"]), torch.ones_like(y))
                a = r / r.sum(dim=1, keepdim=True)
            out[b, h * group:(h + 1) * group] = torch.einsum("gj,jd->gd", a, val).cpu()
            if tracked:
                added[b, h, :i] = (s["scores"][b, h, :i].double() + a.sum(dim=0)).cpu()
    return [out, added] if tracked else [out]
