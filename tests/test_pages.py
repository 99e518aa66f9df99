"""Pages reserved and released on the GPU, against a loop over sequences and
pages; argument checks on the CPU."""

import random

import numpy as np
import pytest

from oracle import serving_oracle as so
from test_paged import LENGTH, PAGE, Cache, host, lib, torch_mod  # noqa: F401

TAB, LENS, CNT, FREE, FC, CO, FO = (i << 40 for i in range(1, 8))


def reserve(lib, tab=TAB, max_pages=4, ps=16, lens=LENS, cnt=CNT, B=3, free=FREE, n=10, fc=FC, co=CO, fo=FO):
    return lib.lssar_paged_reserve(tab, max_pages, ps, lens, cnt, B, free, n, fc, co, fo, None)


def release(lib, tab=TAB, max_pages=4, ps=16, lens=LENS, cnt=CNT, B=3, free=FREE, n=10, fc=FC, fo=FO):
    return lib.lssar_paged_release(tab, max_pages, ps, lens, cnt, B, free, n, fc, fo, None)


@pytest.mark.parametrize("call", [reserve, release])
def test_bad_calls_are_refused(lib, call):
    for name in ("tab", "lens", "free", "fc", "fo"):
        assert call(lib, **{name: None}) == -1, name
    for bad in (dict(B=0), dict(B=1 << 25), dict(max_pages=0), dict(max_pages=1 << 21)):
        assert call(lib, **bad) == -2, bad
    for bad in (dict(ps=0), dict(ps=12), dict(ps=264), dict(n=0)):
        assert call(lib, **bad) == -10, bad
    for name in ("tab", "lens", "cnt", "free", "fc", "fo"):
        assert call(lib, **{name: (9 << 40) + 2}) == -6, name
    for bad in (dict(fo=FC), dict(fo=LENS), dict(fo=CNT + 8), dict(fo=TAB), dict(fo=FREE + 36), dict(tab=FREE)):
        assert call(lib, **bad) == -8, bad


def test_more_that_is_refused(lib):
    assert reserve(lib, co=None) == -1
    assert release(lib, cnt=None) == -1
    assert reserve(lib, co=(9 << 40) + 2) == -6
    for bad in (dict(co=CNT), dict(co=LENS + 8), dict(co=FO - 4), dict(co=TAB + 40), dict(tab=LENS), dict(tab=CNT), dict(tab=FC)):
        assert reserve(lib, **bad) == -8, bad
    for bad in (dict(free=LENS), dict(free=CNT), dict(free=FC)):
        assert release(lib, **bad) == -8, bad


def test_binding_refuses(lib):
    import torch
    from lssar_attn_fwd_gb300 import api
    t = torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.lssar_paged_reserve(t, t[0], None, 16, t[0], t[0, :1])
    with pytest.raises(ValueError):
        api.lssar_paged_release(t, t[0], None, 16, t[0], t[0, :1])


def ints(torch, *x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 2, 31, 257, 700, 3001])
@pytest.mark.parametrize("page,longest", [(8, 3), (16, 200), (24, 1000), (256, 5000)])
def test_reserve_and_release(torch_mod, B, page, longest):
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    rng = random.Random(B + page)
    lens = [rng.choice([0, 1, page, page - 1, rng.randrange(longest + 1)]) for _ in range(B)]
    counts = [rng.choice([0, 1, page, rng.randrange(longest + 1)]) for _ in range(B)]
    width = max(-(-(a + b) // page) for a, b in zip(lens, counts)) or 1
    need = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(lens, counts))
    n_pages = need + 7
    order = rng.sample(range(n_pages), n_pages)
    for free_count in (n_pages, need, need * 2 // 3, 0):
        table = np.full((B, width), -1, dtype=np.int32)
        want_t, want_c, left = so.reserve(table, lens, counts, page, np.array(order), free_count)
        t, l, f = torch.from_numpy(table).cuda(), ints(torch, *lens), ints(torch, *order)
        c, fo = api.lssar_paged_reserve(t, l, ints(torch, *counts), page, f, ints(torch, free_count))
        assert api.device_error_word() == 0
        assert np.array_equal(host(t), want_t) and c.tolist() == want_c and fo.item() == left
        assert f.tolist() == order
        # some end, some are cut, some stay
        now = [a + b for a, b in zip(lens, want_c)]
        after = [rng.choice([0, n, rng.randrange(n + 1)]) for n in now]
        held = [-(-a // page) for a in lens]
        for b in range(B):
            want_t[b, :held[b]] = np.arange(held[b]) % n_pages      # what it held before, any pages
        more = sum(-(-a // page) - -(-z // page) for a, z in zip(now, after))
        pool = np.array(order + [0] * (left + more), dtype=np.int32)
        want_f, want_n = so.release(want_t, now, after, page, pool, left)
        t, f = torch.from_numpy(want_t).cuda(), torch.from_numpy(pool).cuda()
        fo2 = api.lssar_paged_release(t, ints(torch, *now), ints(torch, *after), page, f, fo)
        assert api.device_error_word() == 0
        assert fo2.item() == want_n and np.array_equal(host(f), want_f) and np.array_equal(host(t), want_t)


@pytest.mark.gpu
def test_reserve_one_token_each_by_default(torch_mod):
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    t = torch.full((4, 3), -1, dtype=torch.int32).cuda()
    free = ints(torch, 5, 6, 7, 0, 1, 2, 3, 4)             # page numbers are below the list's length
    c, fo = api.lssar_paged_reserve(t, ints(torch, 0, 16, 17, 47), None, 16, free, ints(torch, 3))
    assert c.tolist() == [1, 1, 1, 1] and fo.item() == 1
    assert t.tolist() == [[7, -1, -1], [-1, 6, -1], [-1] * 3, [-1] * 3]


@pytest.mark.gpu
def test_bad_lengths_counts_and_pages(torch_mod):
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    free = ints(torch, 0, 1, 2, 3, 4, 5)
    for lens, counts in (((-1, 3, 8), (4, 20, 8)), ((2 ** 31 - 1, 3, 8), (4, 20, 8)), ((5, 3, 8), (-1, 20, 8)), ((5, 3, 8), (28, 20, 8)),
                         ((5, 3, 8), (2 ** 31 - 1, 20, 8))):
        t = torch.full((3, 4), -1, dtype=torch.int32).cuda()
        c, fo = api.lssar_paged_reserve(t, ints(torch, *lens), ints(torch, *counts), 8, free, ints(torch, 6))
        assert api.device_error_word() == LENGTH
        assert c.tolist() == [0, 20, 8] and fo.item() == 3 and t.tolist() == [[-1] * 4, [-1, 5, 4, -1], [-1, 3, -1, -1]]
    for bad in (-1, 7, 2 ** 31 - 1):
        t = torch.full((3, 4), -1, dtype=torch.int32).cuda()
        c, fo = api.lssar_paged_reserve(t, ints(torch, 0, 0, 0), ints(torch, 1, 0, 1), 8, free, ints(torch, bad))
        assert api.device_error_word() == LENGTH and c.tolist() == [0, 0, 0] and fo.item() == bad and (t == -1).all()
        f = free.clone()
        fo = api.lssar_paged_release(t, ints(torch, 8, 8, 8), ints(torch, 0, 0, 8), 8, f, ints(torch, bad))
        assert api.device_error_word() == LENGTH and fo.item() == bad and torch.equal(f, free)
    # entries that are no pages
    t = torch.full((1, 4), -1, dtype=torch.int32).cuda()
    c, fo = api.lssar_paged_reserve(t, ints(torch, 0), ints(torch, 24), 8, ints(torch, 9, 1, -5, 6, 2), ints(torch, 4))
    assert api.device_error_word() == PAGE and t.tolist() == [[-1, -1, 1, -1]] and c.tolist() == [24] and fo.item() == 1
    f = ints(torch, 9, 1, 0, 0, 0)
    fo = api.lssar_paged_release(ints(torch, 3, 77, 1, 0).view(1, 4), ints(torch, 24), ints(torch, 3), 8, f, ints(torch, 2))
    assert api.device_error_word() == PAGE and f.tolist() == [9, 1, 77, 1, 0] and fo.item() == 4
    # lengths that grow, and more pages than the list holds
    f = ints(torch, 9, 1, 0, 0, 0)
    t = torch.arange(8, dtype=torch.int32).cuda().view(2, 4)
    fo = api.lssar_paged_release(t, ints(torch, 8, 9), ints(torch, 9, 8), 8, f, ints(torch, 2))
    assert api.device_error_word() == LENGTH and fo.item() == 3 and f.tolist() == [9, 1, 5, 0, 0]
    fo = api.lssar_paged_release(t, ints(torch, 32, 9), ints(torch, 0, 8), 8, f, ints(torch, 2))
    assert api.device_error_word() == LENGTH and fo.item() == 2 and f.tolist() == [9, 1, 5, 0, 0]


@pytest.mark.gpu
def test_wide_sequences(torch_mod):
    # two sequences that take a whole pool of 2^19 pages, and give it back
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    n = 1 << 19
    f = torch.randperm(n, generator=torch.Generator().manual_seed(0)).to(torch.int32).cuda()
    t = torch.full((2, 1 << 18), -1, dtype=torch.int32).cuda()
    lens, counts = ints(torch, 0, 0), ints(torch, 1 << 21, (1 << 21) - 7)
    c, fo = api.lssar_paged_reserve(t, lens, counts, 8, f, ints(torch, n))
    assert torch.equal(c, counts) and fo.item() == 0 and torch.equal(t.flatten(), f.flip(0))
    g = torch.full_like(f, -1)
    fo = api.lssar_paged_release(t, counts, lens, 8, g, fo)
    assert api.device_error_word() == 0 and fo.item() == n and torch.equal(g, f.flip(0))


@pytest.mark.gpu
def test_in_a_graph(torch_mod):
    # captured once, replayed for steps whose lengths are on the device
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    B, page = 40, 8
    t = torch.full((B, 6), -1, dtype=torch.int32).cuda()
    lens, f = torch.arange(B, dtype=torch.int32).cuda() * 0, torch.arange(200, dtype=torch.int32).cuda()
    free, c, fo = ints(torch, 200), torch.empty_like(lens), ints(torch, 0)
    api.lssar_paged_reserve(t.clone(), lens, None, page, f, free, counts_out=c, free_out=fo)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.lssar_paged_reserve(t, lens, None, page, f, free, counts_out=c, free_out=fo)
        lens.add_(c)
        free.copy_(fo)
    for step in range(41):
        g.replay()
    # 200 pages hold 40 tokens each: the 41st of every sequence finds none
    assert lens.tolist() == [40] * B and free.item() == 0 and c.tolist() == [0] * B
    assert sorted(t[:, :5].flatten().tolist()) == list(range(200)) and (t[:, 5] == -1).all()
