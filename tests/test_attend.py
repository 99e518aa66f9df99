"""Attention of a chunk over the paged cache, and a serving run of all the paged
calls together, through the package's entry points, against the float64 oracle;
argument checks on the CPU."""

import ctypes

import numpy as np
import pytest

from lssar_attn_fwd_gb300.inputs import MODE_LSSA, MODE_LSSAR, MODE_SIGMOID_RW, MODE_SOFTMAX, MODE_SOFTMAX_RW
from oracle import paged_oracle as po
from oracle import serving_oracle as so
from test_paged import LENGTH, MODES, OUT, PAGE, Q, TAB, VP, Cache, desc, host, keys_below, lib, longs, torch_mod  # noqa: F401

CNT = 30 << 40


# ---------------------------------------------------------------- argument checks (no GPU)

def attend(lib, c, q=Q, qs=(1 << 16, 4096, 64), out=OUT, H=4, n=8, counts=None, p=3, mode=2):
    return lib.lssar_paged_attend(ctypes.byref(c) if c else None, q, longs(*qs), out, H, n, counts, p, mode, None)


def test_bad_calls_are_refused(lib):
    call = lambda **kw: attend(lib, desc(), **kw)   # noqa: E731
    assert attend(lib, None) == -1
    assert attend(lib, desc(table=None)) == -1
    assert attend(lib, desc(d=96)) == -3
    assert attend(lib, desc(page_size=12)) == -10
    assert attend(lib, desc(dtype=2)) == -11
    assert attend(lib, desc(v_pages=VP + 8)) == -6
    for bad in (dict(q=None), dict(out=None)):
        assert call(**bad) == -1, bad
    for bad in (dict(H=3), dict(H=0), dict(H=2 * 129), dict(n=0), dict(n=-1), dict(n=(1 << 24) + 1), dict(n=1 << 24, H=256),
                dict(qs=(1 << 16, -64, 64))):
        assert call(**bad) == -2, bad
    for bad in (dict(mode=5), dict(mode=-1)):
        assert call(**bad) == -5, bad
    for bad in (dict(p=0), dict(p=1025)):
        assert call(**bad) == -4, bad
        assert call(mode=4, **bad) == -4
    for bad in (dict(qs=(1 << 16, 4096, 60)), dict(q=Q + 8), dict(out=OUT + 2), dict(counts=CNT + 2)):
        assert call(**bad) == -6, bad
    for bad in (dict(out=Q), dict(out=VP + 2048), dict(out=TAB), dict(counts=OUT + 64)):
        assert call(**bad) == -8, bad


def test_binding_refuses(lib):
    import torch
    from lssar_attn_fwd_gb300 import api
    k = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.lssar_paged_attend(k[:1], k, k.clone(), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


# ---------------------------------------------------------------- GPU

def ints(torch, *x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def chunk_q(c, H, n):
    """Queries as a slice of a projection's output [B, n, H + 1, d]."""
    return c.torch.randn(c.B, n, H + 1, c.d, generator=c.g).to(c.dt).cuda().transpose(1, 2)[:, :H]


def check_attend(torch, c, q, counts, mode, p, rows=None, got=None):
    """The chunk's rows against the oracle at its own bounds, plus the output's rounding."""
    from lssar_attn_fwd_gb300 import api
    B, H, n, d = q.shape
    if got is None:
        got = torch.full((B, H, n, d), 7.0, dtype=c.dt).cuda()
        api.lssar_paged_attend(q, *c.args(), counts=None if counts is None else ints(torch, *counts), p=p, mode=mode, out=got)
        assert api.device_error_word() == 0
    lens, counts = c.lens.tolist(), counts or [n] * B
    half_step = torch.finfo(c.dt).eps / 2
    tiny = 2.0 ** -25 if c.dt == torch.float16 else 0.0       # half a step below fp16's normal range
    out, G = host(got), H // c.hkv
    want = so.paged_attend(host(q), host(c.k), host(c.v), host(c.table), lens, counts, mode, p, half_step, rows)
    for (b, h, t), (ref, err) in want.items():
        bad = np.abs(out[b, h * G:(h + 1) * G, t] - ref) - (err + half_step * (np.abs(ref) + err) + tiny)
        assert bad.max() <= 0, (mode, p, b, h, t, bad.max(), err.max())
    for b in range(B):
        assert (got[b, :, counts[b]:] == 7.0).all()
    return got


LENS = [0, 1, 2, 3, 5, 17, 64, 129, 200, 257, 300, 700]
COUNTS = [0, 1, 2, 1, 5, 17, 3, 129, 1, 200, 77, 260]


@pytest.mark.gpu
@pytest.mark.parametrize("mode,p", MODES)
@pytest.mark.parametrize("d,page,hkv,G,half", [(64, 16, 2, 1, False), (128, 24, 1, 8, False), (64, 8, 1, 3, True),
                                                (128, 256, 2, 2, True), (64, 64, 1, 7, False)])
def test_lengths_and_layouts(torch_mod, mode, p, d, page, hkv, G, half):
    c = Cache(torch_mod, LENS, hkv, d, page, half=half, seed=d + page, interleaved=page == 24)
    q = chunk_q(c, hkv * G, 260)
    for b, count in enumerate(COUNTS):
        q[b, :, count:] = float("nan")                # not read
    # every row of the short sequences, those at the tiles' ends of the long ones
    rows = [range(260)] * 8 + [[0, 1, 2, 31, 32, 41, 42, 63, 64, 76, 85, 127, 128, 129, 169, 199, 255, 256, 259]] * 4
    check_attend(torch_mod, c, q, COUNTS, mode, p, rows)


@pytest.mark.gpu
@pytest.mark.parametrize("G", [9, 20, 33, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_large_groups(torch_mod, G, d):
    c = Cache(torch_mod, [300, 1, 0, 77], 2 if G < 100 else 1, d, 32, seed=G)
    for mode, p in ((MODE_LSSAR, 3), (MODE_SOFTMAX, 1), (MODE_LSSA, 1)):
        check_attend(torch_mod, c, chunk_q(c, c.hkv * G, 20), [20, 1, 0, 13], mode, p, [[0, 1, 2, 7, 15, 19]] * 4)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,counts,hkv,G,d,page", [
    ([30000], [300], 1, 4, 64, 16), ([9000, 30, 5000], [700, 30, 1], 2, 1, 128, 128), ([150] * 40, [1] * 20 + [60] * 20, 12, 1, 64, 16),
    ([1500] * 3 + [3] * 30, [1500, 600, 1] + [3] * 30, 4, 2, 64, 48), ([3000], [3000], 1, 1, 128, 64), ([20000], [1], 1, 1, 64, 64)])
def test_long_and_many(torch_mod, lens, counts, hkv, G, d, page):
    c = Cache(torch_mod, lens, hkv, d, page, seed=1)
    q = chunk_q(c, hkv * G, max(counts))
    some = sorted({0, 1, 2, 3, 127, 128, 255, 256, 511, 512, 1023, *(x - 1 for x in counts), *(x // 2 for x in counts)})
    for mode, p in ((MODE_LSSAR, 15), (MODE_SOFTMAX, 1), (MODE_SOFTMAX_RW, 3), (MODE_SIGMOID_RW, 3), (MODE_LSSA, 1)):
        check_attend(torch_mod, c, q, counts, mode, p, [some] * len(lens))


@pytest.mark.gpu
@pytest.mark.parametrize("mode,p", [(MODE_LSSAR, 3), (MODE_SOFTMAX, 1)])
def test_many_sequences(torch_mod, mode, p):
    lens = [(7 * b) % 23 if b % 3 else 0 for b in range(700)]
    lens[0], lens[255], lens[256], lens[699] = 400, 129, 1, 300
    counts = [min(n, (5 * b) % 9) for b, n in enumerate(lens)]
    c = Cache(torch_mod, lens, 2, 64, 16, seed=2)
    check_attend(torch_mod, c, chunk_q(c, 4, 8), counts, mode, p)


@pytest.mark.gpu
@pytest.mark.parametrize("mode,p", [(MODE_LSSAR, 15), (MODE_SOFTMAX_RW, 3), (MODE_SIGMOID_RW, 2), (MODE_LSSA, 1), (MODE_SOFTMAX, 1)])
def test_equal_keys_and_zero_rows(torch_mod, mode, p):
    # equal keys: the uniform row; zero queries and keys: the norm's floor
    c = Cache(torch_mod, [1, 4, 9, 64, 300], 2, 64, 16, seed=3, equal_keys=True)
    q, counts = chunk_q(c, 4, 64), [1, 4, 8, 64, 50]
    check_attend(torch_mod, c, q, counts, mode, p)
    q[:, 1] = 0
    check_attend(torch_mod, c, q, counts, mode, p)
    c = Cache(torch_mod, [5, 70], 2, 64, 16, seed=3)
    for b, n in enumerate((5, 70)):
        c.k[c.table[b, (n - 1) // 16].long(), :, (n - 1) % 16] = 0
    check_attend(torch_mod, c, q[:2], [3, 64], mode, p)


@pytest.mark.gpu
@pytest.mark.parametrize("mode,p", [(MODE_LSSAR, 1), (MODE_LSSAR, 15), (MODE_SIGMOID_RW, 1), (MODE_SIGMOID_RW, 15), (MODE_LSSA, 1)])
@pytest.mark.parametrize("n,d,top,half", [(300, 64, -8, False), (300, 64, -14, True), (5000, 128, -14, False), (16000, 64, -30, False),
                                          (20000, 128, -36, True)])
def test_rows_of_keys_away_from_the_query(torch_mod, mode, p, n, d, top, half):
    # every score is far below 0, and they differ: the weights do too
    c = Cache(torch_mod, [n, n // 3], 1, d, 16, half=half, seed=n)
    one = torch_mod.randn(2, 1, 1, d, generator=c.g)
    q = (one * torch_mod.tensor([1.0, 2.5, 0.1]).view(1, 3, 1, 1) + 0.01).repeat(1, 1, 4, 1).to(c.dt)
    for b, count in enumerate((n, n // 3)):
        keys_below(torch_mod, c, q[b, 0, 0], b, count, top)
    q = q.cuda()
    for b, count in enumerate((n, n // 3)):
        kb = po.gather(host(c.k), c.table[b].tolist(), count)[:, 0]
        w, e = po.row_weights(host(q[b, :, 3]), kb, mode, p), so.attend_bound(host(q[b, :, 3]), kb, mode, p)
        # not uniform by far, and resolved: the comparison can fail
        assert np.abs(w - 1 / count).sum(axis=1).min() > 0.5 and e.sum(axis=1).max() < 0.1
    check_attend(torch_mod, c, q, [4, 3], mode, p)


@pytest.mark.gpu
@pytest.mark.parametrize("mode,p,log2_weight", [(MODE_SOFTMAX, 1, -25.5), (MODE_SOFTMAX, 1, -20.5), (MODE_SOFTMAX_RW, 3, -8.0), (MODE_LSSA, 1, -29.0)])
@pytest.mark.parametrize("n,d", [(131071, 64), (9000, 128)])
def test_fp16_of_many_small_weights(torch_mod, mode, p, log2_weight, n, d):
    # one key of a large weight whose value is 0, and many of small ones that make the output
    torch = torch_mod
    c = Cache(torch, [n], 1, d, 128, half=True, seed=1)
    x = torch.zeros(c.cap, d)
    big = n // 3
    q = torch.zeros(1, 1, 2, d)
    if mode == MODE_LSSA:
        q[0, 0, :, 0] = 4.0
        cos = torch.full((c.cap,), log2_weight * np.log(2) / float(po.length_scale(n, d)))
        cos[big] = 0.3
        x[:, 0], x[:, 1] = 16 * cos, 16 * (1 - cos ** 2).sqrt()
    else:
        q[0, 0, :, 0] = 16.0
        if mode == MODE_SOFTMAX_RW:
            x[1::2, 0] = -40.0                     # half of the keys: no weight at all
        x[big, 0] = -log2_weight * np.log(2) * d ** 0.5 / 16
    pages = c.table[0].long()
    c.k[pages, 0] = x.view(-1, 128, d).to(c.dt).cuda()
    c.v[pages, 0] = (1 + 0.5 * torch.randn(c.cap, d, generator=c.g)).view(-1, 128, d).to(c.dt).cuda()
    c.v[pages[big // 128], 0, big % 128] = 0
    out = check_attend(torch, c, q.to(c.dt).cuda(), None, mode, p)
    assert (out != 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("mode,p", [(MODE_SOFTMAX, 1), (MODE_SOFTMAX_RW, 3)])
@pytest.mark.parametrize("size", [300, 4000, 30000])
@pytest.mark.parametrize("grows", [False, True])
def test_fp16_of_huge_scores(torch_mod, mode, p, size, grows):
    # scores from 2^20 to 2^33, whose steps pass the weights' range: the best key takes all
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    c = Cache(torch, [390], 1, 64, 16, half=True, seed=size)
    a = 1 - torch.arange(390) / 400
    slot = torch.arange(390)
    pages = c.table[0].long().cpu()[slot // 16].cuda()
    c.k[pages, 0, (slot % 16).cuda()] = (size * (a.flip(0) if grows else a)).view(-1, 1).repeat(1, 64).to(c.dt).cuda()
    q = torch.full((1, 2, 3, 64), float(size)).to(c.dt).cuda()
    out = api.lssar_paged_attend(q, *c.args(), p=p, mode=mode)
    assert api.device_error_word() == 0
    for t in range(3):
        best = 387 + t if grows else 0
        v = c.v[c.table[0, best // 16].long(), 0, best % 16].float()
        # the weight is exact (one key); the output's half step
        assert ((out[0, :, t].float() - v).abs() <= (2.0 ** -15 + 2.0 ** -11) * v.abs() + 2.0 ** -25).all()


@pytest.mark.gpu
def test_wide_table_and_far_pages(torch_mod):
    # a table much wider than its sequences; pages 2^28 + 8 elements apart: the same bits as close together
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    c = Cache(torch, [33, 0, 500], 3, 64, 16, width=700, seed=8)
    check_attend(torch, c, chunk_q(c, 6, 33), [33, 0, 20], MODE_LSSAR, 3, [[0, 5, 19, 32]] * 3)
    n_pages, hkv, page, d, far = 10, 2, 16, 64, 2 ** 28 + 8
    k, v = (torch.randn(n_pages, hkv, page, d, generator=c.g).bfloat16().cuda() for _ in range(2))
    pool = torch.empty(n_pages * far, dtype=torch.bfloat16, device="cuda")
    shape, strides = (n_pages, hkv, page, d), (far, page * d, d, 1)
    kf, vf = pool.as_strided(shape, strides), pool.as_strided(shape, strides, 2 ** 27)
    kf.copy_(k)
    vf.copy_(v)
    table, lens = ints(torch, 9, 0, 8, 2, 7, 1, 6, 3).view(2, 4), ints(torch, 20, 61)
    q = torch.randn(2, 6, 20, d, generator=c.g).bfloat16().cuda()
    r = api.Rotary(d)

    def serve(k, v):
        got = [api.lssar_paged_attend(q, k, v, table, lens, mode=m) for m in (MODE_LSSAR, MODE_SOFTMAX)]
        new = torch.ones(2, hkv, 3, d, dtype=torch.bfloat16, device="cuda")
        got += api.lssar_paged_append_rope(q[:, :, :3], new, new, k, v, table, lens, r)
        return got + [k, v]

    for x, y in zip(serve(k, v), serve(kf, vf)):
        assert torch.equal(x, y) and x.isfinite().all()
    assert api.device_error_word() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("mode,p", [(MODE_LSSAR, 3), (MODE_SOFTMAX, 1), (MODE_LSSA, 1)])
def test_rows_of_chunks_are_rows_of_the_whole(torch_mod, mode, p):
    # a prompt in chunks of any sizes, in one, and token by token through the decode step; and the dense forward
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    B, H, L, d = 2, 3, 333, 64
    c = Cache(torch, [L] * B, H, d, 16, seed=2)
    q = chunk_q(c, H, L)
    whole = api.lssar_paged_attend(q, *c.args(), p=p, mode=mode)
    dense = api.lssar_attn_fwd(q.contiguous(), *(x[c.table.long()].permute(0, 2, 1, 3, 4).reshape(B, H, -1, d)[:, :, :L].contiguous()
                                                 for x in (c.k, c.v)), p=p, mode=mode)
    assert (whole.float() - dense.float()).abs().max() <= 4e-2        # each is within 2e-2 of exact
    at = 0
    for n in (1, 100, 31, 128, 73):
        c.lens.fill_(at + n)
        part = api.lssar_paged_attend(q[:, :, at:at + n], *c.args(), p=p, mode=mode)
        # both are within half a step and the weights' rounding of exact: 2^-8 of the sum of w |v|, at most of the largest value
        assert (part.float() - whole[:, :, at:at + n].float()).abs().max() <= 2 ** -6 * 5
        at += n
        step = api.lssar_paged_decode(q[:, :, at - 1].contiguous(), *c.args(), p=p, mode=mode)
        assert (step.float() - whole[:, :, at - 1].float()).abs().max() <= 2 ** -6 * 5
    assert at == L and api.device_error_word() == 0


@pytest.mark.gpu
def test_bad_lengths_counts_and_pages(torch_mod):
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    c = Cache(torch, [300, 300, 300, 300], 2, 64, 16, seed=4)
    q = chunk_q(c, 4, 150)
    for mode in (MODE_LSSAR, MODE_SOFTMAX, MODE_LSSA):
        run = lambda table=c.table, counts=(150, 140, 130, 1): api.lssar_paged_attend(   # noqa: E731
            q, c.k, c.v, table, c.lens, counts=ints(torch, *counts), mode=mode)
        good = run()
        assert api.device_error_word() == 0
        same = lambda out, rows: torch.equal(out[rows], good[rows])   # noqa: E731
        for value in (-1, c.cap + 1, 2 ** 31 - 1, 139):
            c.lens[1] = value
            out = run()
            assert api.device_error_word() == LENGTH and out[1].isnan().all() and same(out, [0, 2, 3])
        c.lens[1] = 300
        for value in (-1, 151, 2 ** 31 - 1):
            out = run(counts=(150, value, 130, 1))
            assert api.device_error_word() == LENGTH and out[1].isnan().all() and same(out, [0, 2, 3])
        for value in (-1, c.k.shape[0], 2 ** 31 - 1):
            for column in (3, 18):
                table = c.table.clone()
                table[2, column] = value
                out = run(table)
                assert api.device_error_word() == PAGE and same(out, [0, 1, 3])
                # rows i = 171 .. 300 of the sequence; those that attend to the page's slots, from 16 column on
                first = max(0, 16 * column + 1 - 171)
                assert out[2, :, first:130].isnan().all() and (out[2, :, 130:] == 0).all()
                assert torch.equal(out[2, :, :first], good[2, :, :first])
        assert torch.equal(run(), good) and api.device_error_word() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d,page,half", [(64, 16, False), (128, 24, True)])
def test_same_bits_again_and_in_the_debug_build(torch_mod, monkeypatch, d, page, half):
    # the debug-check build (bounds checks that record a code) gives the same bits and records nothing
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api, build
    build.build(debug=True)
    results = []
    for lib in (api.load_library(), api.load_library(), api.load_debug_library()):
        monkeypatch.setattr(api, "_LIB", lib)
        c = Cache(torch, LENS, 2, d, page, half=half, seed=5)
        q, counts = chunk_q(c, 6, 260), ints(torch, *COUNTS)
        got = [api.lssar_paged_attend(q, *c.args(), counts=counts, p=p, mode=mode) for mode, p in MODES]
        r = api.Rotary(d, rot_dim=48)
        got += api.lssar_rope(q, q[:, :2], r)
        lens = torch.tensor([max(0, n - 9) for n in LENS], dtype=torch.int32).cuda()
        got += api.lssar_paged_append_rope(q[:, :, :2], q[:, :2, :2], q[:, :2, :2], c.k, c.v, c.table, lens, r, counts=lens.clamp(max=2))
        torch.cuda.synchronize()
        assert api.device_error_word() == 0
        results.append(got + [c.k, c.v])
    for other in results[1:]:
        for a, b in zip(results[0], other):
            view = torch.int16 if a.element_size() == 2 else torch.int32
            assert torch.equal(a.view(view), b.view(view))


class Serving:
    """A small service: sequences that begin, take prompts in chunks, decode, are evicted and end."""

    def __init__(self, torch, seed, hkv=2, G=2, d=64, page=16, B=3, width=8, n_pages=26):
        from lssar_attn_fwd_gb300 import api
        self.torch, self.api, self.B, self.page, self.d = torch, api, B, page, d
        self.g = torch.Generator().manual_seed(seed)
        self.k, self.v = (torch.full((n_pages, hkv, page, d), float("nan"), dtype=torch.bfloat16).cuda() for _ in range(2))
        self.table = torch.full((B, width), -1, dtype=torch.int32).cuda()
        self.lens, self.seen = (torch.zeros(B, dtype=torch.int32).cuda() for _ in range(2))
        self.free, self.free_count = torch.randperm(n_pages, generator=self.g).to(torch.int32).cuda(), ints(torch, n_pages)
        self.scores = torch.zeros(B, hkv, width * page).cuda()
        self.positions = torch.zeros(B, hkv, width * page, dtype=torch.int32).cuda()
        self.rotary = api.Rotary(d, scaling="bands", factor=4.0, original_length=64)
        self.counts, self.left, self.after = (torch.empty_like(self.lens) for _ in range(3))
        self.fo, self.H, self.hkv = torch.empty_like(self.free_count), hkv * G, hkv

    def inputs(self, n):
        x = self.torch.randn(self.B, n, self.H + 2 * self.hkv, self.d, generator=self.g).bfloat16().cuda().transpose(1, 2)
        return x[:, :self.H], x[:, self.H:self.H + self.hkv], x[:, self.H + self.hkv:]

    def chunk(self, q, k, v, want, stream=None, **kw):
        """reserve, append with positions, attend: the rows' outputs."""
        api, kv = self.api, (self.k, self.v, self.table)
        api.lssar_paged_reserve(self.table, self.lens, want, self.page, self.free, self.free_count, counts_out=self.counts,
                                free_out=self.fo, stream=stream)
        qr, _ = api.lssar_paged_append_rope(q, k, v, *kv, self.lens, self.rotary, counts=self.counts, first_positions=self.seen,
                                            scores=self.scores, positions=self.positions, lens_out=self.after, stream=stream, **kw)
        return qr, api.lssar_paged_attend(qr, *kv, self.after, counts=self.counts, p=15, stream=stream)


@pytest.mark.gpu
def test_serving_run(torch_mod):
    torch = torch_mod
    s = Serving(torch, 1)
    api, page, want_page = s.api, s.page, lambda n: -(-n // s.page)
    tokens = [[] for _ in range(s.B)]                  # (key, value, position) of each cached token, from the inputs

    def advance(want):
        n = max(want)
        q, k, v = s.inputs(n)
        before, free = s.lens.tolist(), s.free_count.item()
        qr, out = s.chunk(q, k, v, ints(torch, *want))
        counts = s.counts.tolist()
        taken = sum(want_page(a + x) - want_page(a) for a, x in zip(before, counts))
        assert s.fo.item() == free - taken and s.after.tolist() == [a + x for a, x in zip(before, counts)]
        kr, _ = api.lssar_rope(k, None, s.rotary, positions=s.seen)
        freq = so.frequencies(s.d, scaling="bands", factor=4.0, original_length=64)
        for b in range(s.B):
            at = s.seen[b].item()
            kw, err = so.rope(host(k[b]), at + np.arange(n), freq)
            assert (np.abs(host(kr[b]) - kw) <= err + 2.0 ** -8 * (np.abs(kw) + err)).all()
            tokens[b] += [(host(kr[b, :, t]), host(v[b, :, t]), at + t) for t in range(counts[b])]
        s.lens.copy_(s.after), s.free_count.copy_(s.fo), s.seen.add_(s.counts)
        for b in range(s.B):
            assert len(tokens[b]) == s.lens[b]
            for h in range(s.hkv):
                for t in range(counts[b]):
                    i = len(tokens[b]) - counts[b] + t + 1
                    key, val = (np.stack([x[j][h] for x in tokens[b][:i]]) for j in (0, 1))
                    ref, err = so.attend_row(host(qr[b, 2 * h:2 * h + 2, t]), key, val, MODE_LSSAR, 15, 2.0 ** -8)
                    got = host(out[b, 2 * h:2 * h + 2, t])
                    assert (np.abs(got - ref) <= err + 2.0 ** -8 * (np.abs(ref) + err)).all()
            assert (out[b, :, counts[b]:] == 0).all()
        return counts

    assert advance([40, 1, 17]) == [40, 1, 17]
    assert advance([30, 50, 1]) == [30, 50, 1]
    assert advance([58, 70, 60]) == [58, 70, 60]       # all of the pool: 8 + 8 + 5 pages of 26
    held = set()
    for b in range(s.B):
        held |= set(s.table[b, :want_page(s.lens[b].item())].tolist())
    assert len(held) == 21 and held.isdisjoint(s.free[:s.free_count.item()].tolist())
    # decode steps through the eviction's scores; the pages past the cut go back
    qs, _, _ = s.inputs(1)
    api.lssar_paged_decode(qs[:, :, 0], s.k, s.v, s.table, s.lens, p=3, scores=s.scores)
    keep = 60
    moves = [[po.evict_moves(host(s.scores)[b, h], host(s.positions)[b, h], len(tokens[b]), keep, 8, 2) for h in range(s.hkv)] for b in range(s.B)]
    before = s.lens.clone()
    lens, _, _ = api.lssar_paged_evict(s.k, s.v, s.table, s.lens, s.scores, s.positions, keep, recent=8, sinks=2)
    s.free_count.copy_(api.lssar_paged_release(s.table, before, lens, page, s.free, s.free_count))
    s.lens.copy_(lens)
    assert s.lens.tolist() == [60, 60, 60] and s.free_count.item() == 26 - 12
    for b in range(s.B):
        rows = [[(tokens[b][t][0][h], tokens[b][t][1][h]) for t in range(len(tokens[b]))] for h in range(s.hkv)]
        for h in range(s.hkv):
            for src, dst in moves[b][h]:
                rows[h][dst] = rows[h][src]
        tokens[b] = [(np.stack([rows[h][t][0] for h in range(s.hkv)]), np.stack([rows[h][t][1] for h in range(s.hkv)]), 0) for t in range(keep)]
    advance([4, 20, 33])
    # one ends: its pages serve another
    gone = s.lens.clone()
    s.lens[1] = 0
    s.free_count.copy_(api.lssar_paged_release(s.table, gone, s.lens, page, s.free, s.free_count))
    s.seen[1], tokens[1] = 0, []
    assert advance([64, 128, 35]) == [64, 128, 35]
    assert api.device_error_word() == 0
    assert s.lens.tolist() == [128, 128, 128] and s.free_count.item() == 2


@pytest.mark.gpu
def test_streams_and_graphs(torch_mod):
    # one chunk of serving captured twice (two graphs share the library's pool), both replayed at once on two streams
    torch = torch_mod
    sizes, want = 20, []
    for seed in (1, 2):
        s = Serving(torch, seed, n_pages=40)
        q, k, v = s.inputs(sizes)
        outs = []
        for _ in range(4):
            qr, out = s.chunk(q, k, v, ints(torch, 20, 7, 13))
            s.lens.copy_(s.after), s.free_count.copy_(s.fo), s.seen.add_(s.counts)
            outs.append((qr.clone(), out.clone()))
        want.append((s, outs))
    graphs, got, held = [], [], []              # (held: what the graphs read stays alive)
    for seed in (1, 2):
        s = Serving(torch, seed, n_pages=40)
        q, k, v = s.inputs(sizes)
        counts = ints(torch, 20, 7, 13)
        q_out = torch.zeros(s.B, s.H, sizes, s.d, dtype=torch.bfloat16).cuda()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qr, out = s.chunk(q, k, v, counts, q_out=q_out)
            s.lens.copy_(s.after), s.free_count.copy_(s.fo), s.seen.add_(s.counts)
        graphs.append(g)
        got.append((s, qr, out))
        held.append((q, k, v, counts))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(4):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for (s, outs), (_, qr, out) in zip(want, got):
            assert torch.equal(qr, outs[i][0]) and torch.equal(out, outs[i][1])
    for (a, _), (b, _, _) in zip(want, got):
        for name in ("lens", "free_count", "table", "scores", "positions", "seen"):
            assert torch.equal(getattr(a, name), getattr(b, name)), name
        assert torch.equal(a.k.view(torch.int16), b.k.view(torch.int16)) and torch.equal(a.v.view(torch.int16), b.v.view(torch.int16))
    assert s.api.device_error_word() == 0


@pytest.mark.gpu
def test_calls_on_two_streams_at_once(torch_mod):
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    caches = [Cache(torch, [3000, 17, 900], 4, 64, 16, seed=s) for s in (1, 2)]
    counts = ints(torch, 300, 17, 1)
    qs = [chunk_q(c, 8, 300) for c in caches]
    want = [api.lssar_paged_attend(q, *c.args(), counts=counts, p=15) for q, c in zip(qs, caches)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for j in range(10):
        for i in (0, 1):
            got[i].append(api.lssar_paged_attend(qs[i], *caches[i].args(), counts=counts, p=15,
                                                 stream=streams[i] if j % 2 else streams[i].cuda_stream))
    torch.cuda.synchronize()
    assert api.device_error_word() == 0
    for i in (0, 1):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_chunks_of_too_many_tiles_are_refused(lib):
    # 65535 sequences x 32 pairs of tiles x 2055 units, 8192 key heads x 64 x 4103: more than an int numbers
    c = desc(B=65535, Hkv=1, max_pages=8192, page_stride=1024)
    assert attend(lib, c, qs=(1 << 20, 64, 8192), H=128, n=64, mode=0) == -2
    c = desc(B=4096, Hkv=2, max_pages=16384, page_stride=2048)
    assert attend(lib, c, qs=(1 << 22, 64, 128), H=2, n=16384, mode=0) == -2


@pytest.mark.gpu
@pytest.mark.parametrize("p", [2, 4, 5, 6, 7, 9, 16, 27, 45, 127, 243, 1000, 1024])
@pytest.mark.parametrize("mode", [MODE_LSSAR, MODE_SOFTMAX_RW])
def test_exponents(torch_mod, mode, p):
    c = Cache(torch_mod, [200, 3, 41], 2, 64, 16, seed=p)
    check_attend(torch_mod, c, chunk_q(c, 4, 41), [30, 3, 41], mode, p)


@pytest.mark.gpu
@pytest.mark.parametrize("d,half", [(64, False), (128, False), (64, True), (128, True)])
def test_chunks_of_one_tile_of_rows_beside_larger_ones(torch_mod, d, half):
    # items of at most 128 rows (both row slots share their keys) of 1, 2, 3, .. tiles, between items of more rows:
    # several of either kind for each SM, in any order
    lens = [40, 128, 129, 256, 257, 384, 385, 700, 130, 1, 300, 900] * 4
    counts = [3, 100, 1, 40, 257, 64, 2, 300, 130, 1, 129, 128] * 4
    c = Cache(torch_mod, lens, 9, d, 16, half=half, seed=d)
    some = [sorted({0, n // 2, n - 1, min(127, n - 1), min(128, n - 1)}) for n in counts]
    q = chunk_q(c, 18, 300)
    for b, n in enumerate(counts):
        q[b, :, n:] = float("nan")
    for mode, p in MODES:
        check_attend(torch_mod, c, q, counts, mode, p, some)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_bad_pages_under_one_tile_of_rows(torch_mod, d):
    # 40 rows on 1 to 4 tiles, whose slots take turns: NaN where a row attends to the page, the oracle's values elsewhere;
    # the same bits whatever ran between, since nothing of what the tile held before is read
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    c, other = Cache(torch, [60, 200, 330, 500], 2, d, 16, seed=6), Cache(torch, [900], 2, d, 16, seed=7)
    other.k *= 100
    q, q_other = chunk_q(c, 2, 40), chunk_q(other, 2, 300)
    for mode, p in ((MODE_LSSAR, 3), (MODE_SOFTMAX, 1), (MODE_LSSA, 1), (MODE_SIGMOID_RW, 3), (MODE_SOFTMAX_RW, 3)):
        good = check_attend(torch, c, q, None, mode, p)
        for b, n in enumerate(c.lens.tolist()):
            for column in sorted({0, 9, 17, 19, 26, (n - 20) // 16}):
                if 16 * column >= n:
                    continue
                table = c.table.clone()
                table[b, column] = -1
                outs = []
                for _ in range(3):
                    outs.append(api.lssar_paged_attend(q, c.k, c.v, table, c.lens, p=p, mode=mode))
                    assert api.device_error_word() == PAGE
                    api.lssar_paged_attend(q_other, *other.args(), p=p, mode=mode)
                first = max(0, 16 * column - (n - 40))           # row t attends to slots up to n - 40 + t
                want = torch.zeros_like(good, dtype=torch.bool)
                want[b, :, first:] = True
                assert torch.equal(outs[0].isnan(), want), (mode, b, column)
                assert all(torch.equal(x.nan_to_num(), outs[0].nan_to_num()) for x in outs[1:]), (mode, b, column)
                check_attend(torch, c, q, None, mode, p, [range(first) if x == b else [0, 39] for x in range(4)], got=outs[0])


@pytest.mark.gpu
def test_results_on_another_stream_take_no_block_in_use(torch_mod):
    # blocks of the results' sizes, just freed on the current stream, are still written by what is queued there
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    c = Cache(torch, [40, 30], 2, 64, 16, seed=3)
    lens, counts = ints(torch, 20, 2), ints(torch, 1, 3)
    q, new, r = chunk_q(c, 4, 8), chunk_q(c, 2, 8), api.Rotary(64)
    free, count = torch.arange(40, dtype=torch.int32).cuda(), ints(torch, 30)
    calls = [lambda s: [api.lssar_paged_attend(q, *c.args(), stream=s)],
             lambda s: list(api.lssar_rope(q, new, r, stream=s)),
             lambda s: list(api.lssar_rope_bwd(q, new, r, stream=s)),
             lambda s: list(api.lssar_paged_append_rope(q, new, new, c.k, c.v, c.table, lens, r, stream=s)),
             lambda s: list(api.lssar_paged_reserve(c.table.clone(), lens, counts, 16, free, count, stream=s)),
             lambda s: [api.lssar_paged_release(c.table, ints(torch, 40, 30), lens, 16, free.clone(), count, stream=s)]]
    side = torch.cuda.Stream()
    for i, call in enumerate(calls):
        want = call(None)
        torch.cuda.synchronize()
        for stream in (side, side.cuda_stream):
            blocks = [torch.empty_like(w) for w in want for _ in range(4)]
            torch.cuda._sleep(100_000_000)     # about 50 ms
            for b in blocks:
                b.fill_(77)
            del blocks, b
            got = call(stream)
            torch.cuda.synchronize()
            for a, w in zip(got, want):
                view = torch.int16 if w.element_size() == 2 else torch.int32
                assert torch.equal(a.view(view), w.view(view)), i
    assert api.device_error_word() == 0


@pytest.mark.gpu
def test_debug_build_of_a_serving_step(torch_mod, monkeypatch):
    # pages, appends and chunks of both kinds in the debug-check build: the same bits, nothing recorded
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api, build
    build.build(debug=True)
    results = []
    for lib in (api.load_library(), api.load_debug_library()):
        monkeypatch.setattr(api, "_LIB", lib)
        s, got = Serving(torch, 5, width=40, n_pages=120), []
        for want in ([500, 30, 200], [64, 9, 1], [1, 300, 40], [70, 70, 128]):
            got += [x.clone() for x in s.chunk(*s.inputs(max(want)), ints(torch, *want))]
            before = s.lens.clone()
            s.lens.copy_(s.after), s.free_count.copy_(s.fo), s.seen.add_(s.counts)
            if want[1] == 9:
                before.copy_(s.lens)
                s.lens[0] = 0
                s.seen[0] = 0
                s.free_count.copy_(api.lssar_paged_release(s.table, before, s.lens, s.page, s.free, s.free_count))
        torch.cuda.synchronize()
        assert api.device_error_word() == 0
        results.append(got + [s.k, s.v, s.table, s.lens, s.free_count, s.scores, s.positions])
    for a, b in zip(*results):
        view = torch.int16 if a.element_size() == 2 else torch.int32
        assert torch.equal(a.view(view), b.view(view))


@pytest.mark.gpu
@pytest.mark.parametrize("mode,p", MODES)
def test_nothing_to_attend_and_whole_sequences(torch_mod, mode, p):
    # no rows anywhere: out stays; the lengths themselves as counts: every row of every sequence
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    c = Cache(torch, [0, 5, 131, 0], 2, 64, 16, seed=9)
    q = chunk_q(c, 4, 131)
    out = torch.full((4, 4, 131, 64), 7.0, dtype=c.dt).cuda()
    for lens in (c.lens, c.lens * 0):
        api.lssar_paged_attend(q, c.k, c.v, c.table, lens, counts=ints(torch, 0, 0, 0, 0), p=p, mode=mode, out=out)
        assert api.device_error_word() == 0 and (out == 7.0).all()
    api.lssar_paged_attend(q, *c.args(), counts=c.lens, p=p, mode=mode, out=out)
    assert api.device_error_word() == 0
    check_attend(torch, c, q, c.lens.tolist(), mode, p, [[], range(5), [0, 1, 2, 3, 64, 126, 127, 128, 130], []], got=out)


@pytest.mark.gpu
@pytest.mark.parametrize("d,G", [(64, 1), (128, 1), (64, 4)])
@pytest.mark.parametrize("mode,p", MODES)
def test_non_finite_inputs_stay_with_their_rows(torch_mod, mode, p, d, G):
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    lens, n, s = [700, 300], 600, 400
    rows = [[0, 150, 298, 299], [5, 130, 299]]                # of the first: those before slot s (t attends to 101 + t)
    for value in (float("nan"), float("inf"), -float("inf")):
        # a key: the rows that attend to it and no others
        c = Cache(torch, lens, 1, d, 16, seed=d)
        q, counts = chunk_q(c, G, n), [n, 300]
        c.k[c.table[0, s // 16].long(), 0, s % 16] = value
        out = check_attend(torch, c, q, counts, mode, p, rows)
        first = s - (lens[0] - n)
        assert not out[0, :, first:].isfinite().any() and out[0, :, :first].isfinite().all() and out[1, :, :300].isfinite().all()
        # a query: its row
        c = Cache(torch, lens, 1, d, 16, seed=d)
        q[0, 0, 77] = value
        out = check_attend(torch, c, q, counts, mode, p, rows)
        bad = ~out[:, :, :n].isfinite().all(-1)
        assert bad[0, 0, 77] and bad.sum() == 1
        # a value: no row that lies more than 383 slots before it, no other sequence
        q[0, 0, 77] = 1.0
        c.v[c.table[0, 699 // 16].long(), 0, 699 % 16] = value
        out = check_attend(torch, c, q, counts, mode, p, [[0, 100, 215], [5, 130, 299]])
        assert out[0, :, :216].isfinite().all() and out[1, :, :300].isfinite().all() and not out[0, :, 599].isfinite().any()


@pytest.mark.gpu
@pytest.mark.parametrize("d,half", [(64, False), (128, False), (64, True)])
def test_exact_weights_are_kept_on_request(torch_mod, monkeypatch, d, half):
    # LSSAR rows that meet the bound take the one-exponential softplus, which moves some bits; none do with
    # LSSAR_EXACT_WEIGHTS=1, and the rows are then within the oracle's bound without its share for that form
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    n, count, p = 6000, 200, 15
    c = Cache(torch, [n], 2, d, 64, half=half, seed=d)
    q = chunk_q(c, 2, count)
    run = lambda: api.lssar_paged_attend(q, *c.args(), p=p, mode=MODE_LSSAR)   # noqa: E731
    monkeypatch.delenv("LSSAR_EXACT_WEIGHTS", raising=False)
    default = run()
    monkeypatch.setenv("LSSAR_EXACT_WEIGHTS", "1")
    exact = run()
    monkeypatch.setenv("LSSAR_EXACT_WEIGHTS", "0")
    assert torch.equal(run(), default)
    assert api.device_error_word() == 0
    assert not torch.equal(exact, default)
    half_step = torch.finfo(c.dt).eps / 2
    tiny = 2.0 ** -25 if half else 0.0
    kb, vb, got = po.gather(host(c.k), c.table[0].tolist(), n), po.gather(host(c.v), c.table[0].tolist(), n), host(exact)
    for h in range(2):
        for t in range(0, count, 7):
            i = n - count + t + 1
            ref, err = so.attend_row(host(q[:, h, t]), kb[:i, h], vb[:i, h], MODE_LSSAR, p, half_step)
            err = err - 4e-4 * np.abs(vb[:i, h]).max(axis=0)
            bad = np.abs(got[0, h, t] - ref) - (err + half_step * (np.abs(ref) + err) + tiny)
            assert bad.max() <= 0, (h, t, bad.max(), err.max())


@pytest.mark.gpu
def test_weights_of_an_eviction_are_those_of_decode_steps(torch_mod):
    # a prompt in two chunks leaves the scores at 0; a step of one token through the decode step adds up its weights,
    # and the eviction keeps the tokens that have them
    torch = torch_mod
    s = Serving(torch, 3)
    api, kv = s.api, (s.k, s.v, s.table)
    for n in (40, 30):
        s.chunk(*s.inputs(n), ints(torch, n, n, n))
        s.lens.copy_(s.after), s.free_count.copy_(s.fo), s.seen.add_(s.counts)
        assert (s.scores == 0).all()
    q, k, v = s.inputs(1)
    s.counts, s.free_count = api.lssar_paged_reserve(s.table, s.lens, ints(torch, 1, 1, 1), s.page, s.free, s.free_count)
    q, s.lens = api.lssar_paged_append_rope(q, k, v, *kv, s.lens, s.rotary, counts=s.counts, first_positions=s.seen,
                                            scores=s.scores, positions=s.positions)
    out = api.lssar_paged_decode(q[:, :, 0], *kv, s.lens, p=15, scores=s.scores)
    chunk = api.lssar_paged_attend(q, *kv, s.lens, p=15)[:, :, 0]
    # each is within half a step and its weights' rounding of exact: 2^-8 of the largest |v|, below 5, twice
    assert (out.float() - chunk.float()).abs().max() <= 2 ** -6 * 5
    # two query heads to a key head, whose weights sum to 1: fp32 sums of 71
    total = s.scores.sum(-1)
    assert (total - 2).abs().max() <= 71 * 2.0 ** -23 * 2 + 2.0 ** -12
    want = [[set(host(s.positions)[b, h, np.argsort(-host(s.scores)[b, h, :71], kind="stable")[:20]].astype(int)) for h in range(s.hkv)]
            for b in range(s.B)]
    lens, _, _ = api.lssar_paged_evict(*kv, s.lens, s.scores, s.positions, 20, recent=0, sinks=0)
    assert lens.tolist() == [20] * 3 and api.device_error_word() == 0
    for b in range(s.B):
        for h in range(s.hkv):
            assert set(s.positions[b, h, :20].tolist()) == want[b][h]
