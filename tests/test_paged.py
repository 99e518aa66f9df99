"""The paged key-value cache (append, decode, evict) through the package's
entry points, against the float64 oracle; argument checks on the CPU."""

import ctypes

import numpy as np
import pytest

from lssar_attn_fwd_gb300.inputs import MODE_LSSA, MODE_LSSAR, MODE_SIGMOID_RW, MODE_SOFTMAX, MODE_SOFTMAX_RW
from oracle import paged_oracle as po

MODES = [(MODE_SOFTMAX, 1), (MODE_LSSA, 1), (MODE_LSSAR, 3), (MODE_LSSAR, 15), (MODE_SOFTMAX_RW, 3),
         (MODE_SIGMOID_RW, 15), (MODE_LSSAR, 1), (MODE_LSSAR, 40)]
LENGTH, PAGE = 51, 52      # error word: a bad length, a bad page number


# ---------------------------------------------------------------- argument checks (no GPU)

# far-apart fake addresses, never used: each call has something wrong
KP, VP, TAB, LENS, Q, OUT, SC, SC2, POS, POS2, LO, KN, VN = (i << 40 for i in range(1, 14))


@pytest.fixture(scope="module")
def lib():
    from lssar_attn_fwd_gb300 import api, build
    build.build()
    return api.load_library()


def desc(**kw):
    from lssar_attn_fwd_gb300 import api
    f = dict(k_pages=KP, v_pages=VP, table=TAB, lens=LENS, page_stride=2 * 16 * 64, n_pages=10, max_pages=4,
             page_size=16, B=3, Hkv=2, d=64, dtype=0)
    f.update(kw)
    return api.PagedCacheDesc(**f)


def longs(*v):
    return (ctypes.c_longlong * len(v))(*v)


def append(lib, c, kn=KN, vn=VN, ks=(1024, 512, 64), vs=(1024, 512, 64), n=8, counts=None, first=None, sc=SC, pos=POS, lo=LO):
    return lib.lssar_paged_append(ctypes.byref(c) if c else None, kn, longs(*ks), vn, longs(*vs), n, counts, first, sc, pos, lo, None)


def decode(lib, c, q=Q, qs=(256, 64), out=OUT, H=4, p=3, mode=2, sc=SC, so=SC2):
    return lib.lssar_paged_decode(ctypes.byref(c) if c else None, q, longs(*qs), out, H, p, mode, sc, so, None)


def evict(lib, c, sc=SC, pos=POS, keep=32, recent=8, sinks=4, so=SC2, po_=POS2, lo=LO):
    return lib.lssar_paged_evict(ctypes.byref(c) if c else None, sc, pos, keep, recent, sinks, so, po_, lo, None)


@pytest.mark.parametrize("call", [append, decode, evict])
def test_bad_caches_are_refused(lib, call):
    assert call(lib, None) == -1
    for name in ("k_pages", "v_pages", "table", "lens"):
        assert call(lib, desc(**{name: None})) == -1
    assert call(lib, desc(d=96)) == -3
    assert call(lib, desc(dtype=2)) == -11
    for bad in (dict(B=0), dict(Hkv=0), dict(max_pages=0), dict(max_pages=(1 << 20) + 1), dict(B=1 << 25)):
        assert call(lib, desc(**bad)) == -2, bad
    for bad in (dict(page_size=0), dict(page_size=12), dict(page_size=264), dict(n_pages=0), dict(page_stride=2040),
                dict(page_stride=2048 + 4), dict(page_stride=-2048)):
        assert call(lib, desc(**bad)) == -10, bad
    assert call(lib, desc(k_pages=KP + 8)) == -6
    assert call(lib, desc(table=TAB + 2)) == -6
    # K and V: apart, or slices of one buffer whose pages do not meet
    assert call(lib, desc(v_pages=KP)) == -8
    assert call(lib, desc(v_pages=KP + 4096)) == -8
    assert call(lib, desc(v_pages=KP + 4096, page_stride=4096 - 8)) == -8


def test_bad_appends_are_refused(lib):
    assert append(lib, desc(), lo=None) == -1
    assert append(lib, desc(), kn=None) == -1
    assert append(lib, desc(), n=-1) == -2
    assert append(lib, desc(), ks=(1024, -512, 64)) == -2
    assert append(lib, desc(), ks=(1024, 512, 60)) == -6
    assert append(lib, desc(), vn=VN + 8) == -6
    assert append(lib, desc(), lo=LENS) == -8            # lens is read by every block
    assert append(lib, desc(), sc=POS) == -8
    assert append(lib, desc(), kn=KP + 4096) == -8
    assert append(lib, desc(), counts=LO) == -8
    assert append(lib, desc(), first=LENS, lo=LENS + 4) == -8


def test_bad_decodes_are_refused(lib):
    assert decode(lib, desc(), q=None) == -1
    assert decode(lib, desc(), out=None) == -1
    assert decode(lib, desc(), sc=None) == -1
    assert decode(lib, desc(), so=None) == -1
    assert decode(lib, desc(), H=3) == -2
    assert decode(lib, desc(), H=0) == -2
    assert decode(lib, desc(), H=2 * 129) == -2
    assert decode(lib, desc(B=1 << 10, max_pages=1 << 20, Hkv=16, page_stride=1 << 14), H=16) == -2
    assert decode(lib, desc(), mode=5) == -5
    assert decode(lib, desc(), p=0) == -4
    assert decode(lib, desc(), p=1025) == -4
    assert decode(lib, desc(), qs=(252, 64)) == -6
    assert decode(lib, desc(), out=OUT + 2) == -6
    assert decode(lib, desc(), out=Q) == -8
    assert decode(lib, desc(), out=VP + 2048) == -8
    assert decode(lib, desc(), so=SC + 4) == -8
    assert decode(lib, desc(), so=TAB) == -8


def test_bad_evictions_are_refused(lib):
    for name in ("sc", "pos", "so", "po_", "lo"):
        assert evict(lib, desc(), **{name: None}) == -1, name
    for bad in (dict(keep=0), dict(recent=-1), dict(sinks=-1), dict(recent=29), dict(recent=2 ** 31 - 1, sinks=2 ** 31 - 1)):
        assert evict(lib, desc(), **bad) == -12, bad
    assert evict(lib, desc(), so=SC) == -8               # one in place, the other not
    assert evict(lib, desc(), so=SC + 64) == -8
    assert evict(lib, desc(), lo=LENS) == -8
    assert evict(lib, desc(), po_=SC2) == -8
    assert evict(lib, desc(), lo=POS + 8) == -8


def test_binding_refuses_cpu_tensors():
    import torch
    from lssar_attn_fwd_gb300 import api
    k = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.lssar_paged_decode(k[0, :, 0].unsqueeze(0), k, k.clone(), torch.zeros(1, 2, dtype=torch.int32),
                               torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        api.lssar_paged_decode(k, [], k, k, k)


# ---------------------------------------------------------------- GPU

@pytest.fixture(scope="module")
def torch_mod():
    import torch
    from lssar_attn_fwd_gb300 import api, build
    build.build()
    api.load_library()
    return torch


def host(t):
    return t.detach().double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


class Cache:
    """A pool of pages whose unused slots hold NaN and infinities, handed out in no order."""

    def __init__(self, torch, lens, hkv, d, page, width=None, half=False, seed=0, interleaved=False, equal_keys=False):
        self.torch = torch
        g = torch.Generator().manual_seed(seed)
        self.g, self.B, self.hkv, self.d, self.page = g, len(lens), hkv, d, page
        self.width = width or max(1, -(-max(lens) // page))
        self.dt = torch.float16 if half else torch.bfloat16
        n_pages = self.B * self.width + 2
        order = torch.randperm(n_pages, generator=g)
        table = order[:self.B * self.width].reshape(self.B, self.width)
        both = torch.full((n_pages, 2, hkv, page, d), float("nan"))
        both[::2] = float("inf")
        for b, n in enumerate(lens):
            for i in range(-(-n // page)):
                rows = min(page, n - i * page)
                x = torch.randn(2, hkv, rows, d, generator=g)
                if equal_keys:
                    x[0] = 0.5
                both[table[b, i], :, :, :rows] = x
        both = both.to(self.dt).cuda()
        self.k, self.v = (both[:, 0], both[:, 1]) if interleaved else (both[:, 0].contiguous(), both[:, 1].contiguous())
        # entries past the last page in use are never read: no page number at all
        for b, n in enumerate(lens):
            table[b, -(-n // page):] = -7
        self.table = table.to(torch.int32).cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32).cuda()
        self.cap = self.width * page

    def args(self):
        return self.k, self.v, self.table, self.lens

    def slots(self, scale=1.0):
        return (scale * self.torch.rand(self.B, self.hkv, self.cap, generator=self.g)).cuda()

    def q(self, H):
        return self.torch.randn(self.B, H, self.d, generator=self.g).to(self.dt).cuda()


def check_decode(torch, c, q, mode, p, scores=None, got=None):
    """Decode against the oracle at the oracle's own bounds, plus the output's rounding."""
    from lssar_attn_fwd_gb300 import api
    so = None if scores is None else torch.full_like(scores, -3.0)
    out = api.lssar_paged_decode(q, *c.args(), p=p, mode=mode, scores=scores, scores_out=so) if got is None else got
    assert api.device_error_word() == 0
    lens = c.lens.tolist()
    ref, new, err, new_err = po.paged_decode(host(q), host(c.k), host(c.v), host(c.table), lens, mode, p,
                                             None if scores is None else host(scores))
    half_step = torch.finfo(c.dt).eps / 2
    tiny = 2.0 ** -25 if c.dt == torch.float16 else 0.0       # half a step below fp16's normal range
    bad = np.abs(host(out) - ref) - (err + half_step * (np.abs(ref) + err) + tiny)
    assert bad.max() <= 0, (mode, p, np.unravel_index(bad.argmax(), bad.shape), bad.max(), err.max())
    if scores is not None:
        got = host(so)
        for b, n in enumerate(lens):
            assert (got[b, :, n:] == -3.0).all()
            off = np.abs(got[b, :, :n] - new[b, :, :n]) - new_err[b, :, :n]
            assert off.size == 0 or off.max() <= 0, (mode, p, b, off.max(), new_err[b].max())
    return out, so


LENS_MIX = [0, 1, 2, 3, 4, 5, 8, 15, 16, 17, 63, 64, 65, 127, 129, 200, 257, 700]


@pytest.mark.gpu
@pytest.mark.parametrize("mode,p", MODES)
@pytest.mark.parametrize("d,page,hkv,G,half", [(64, 16, 2, 1, False), (128, 24, 1, 8, False), (64, 8, 1, 3, True),
                                                (128, 256, 2, 2, True), (64, 64, 1, 7, False)])
def test_decode_lengths_and_layouts(torch_mod, mode, p, d, page, hkv, G, half):
    c = Cache(torch_mod, LENS_MIX, hkv, d, page, half=half, seed=d + page, interleaved=page == 24)
    check_decode(torch_mod, c, c.q(hkv * G), mode, p, c.slots(1e-2))


@pytest.mark.gpu
@pytest.mark.parametrize("G", [9, 16, 20, 33])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_large_groups(torch_mod, G, d):
    c = Cache(torch_mod, [300, 1, 0, 77], 2, d, 32, seed=G)
    check_decode(torch_mod, c, c.q(2 * G), MODE_LSSAR, 3, c.slots(1e-2))
    check_decode(torch_mod, c, c.q(2 * G), MODE_SOFTMAX, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,hkv,G,d,page", [([40000], 1, 4, 64, 16), ([9000, 30, 5000], 2, 1, 128, 128),
                                                ([150] * 40, 12, 1, 64, 16), ([1500] * 3 + [3] * 30, 4, 2, 64, 48)])
def test_decode_long_and_many(torch_mod, lens, hkv, G, d, page):
    c = Cache(torch_mod, lens, hkv, d, page, seed=1)
    for mode, p in ((MODE_LSSAR, 15), (MODE_SOFTMAX, 1), (MODE_SOFTMAX_RW, 3)):
        check_decode(torch_mod, c, c.q(hkv * G), mode, p, c.slots(1e-3))


@pytest.mark.gpu
@pytest.mark.parametrize("mode,p", [(MODE_LSSAR, 3), (MODE_SOFTMAX, 1)])
def test_decode_many_sequences(torch_mod, mode, p):
    # more sequences than a warp looks over at once, most of them short or empty
    lens = [(7 * b) % 23 if b % 3 else 0 for b in range(700)]
    lens[0], lens[255], lens[256], lens[699] = 400, 129, 1, 300
    c = Cache(torch_mod, lens, 2, 64, 16, seed=2)
    check_decode(torch_mod, c, c.q(4), mode, p, c.slots(1e-2))


@pytest.mark.gpu
@pytest.mark.parametrize("mode,p", [(MODE_LSSAR, 15), (MODE_SOFTMAX_RW, 3), (MODE_SIGMOID_RW, 2), (MODE_LSSA, 1)])
def test_decode_equal_keys_and_zero_rows(torch_mod, mode, p):
    # equal keys: the uniform row; zero queries and keys: the norm's floor
    c = Cache(torch_mod, [1, 4, 9, 64, 300], 2, 64, 16, seed=3, equal_keys=True)
    q = c.q(4)
    check_decode(torch_mod, c, q, mode, p, c.slots())
    q[:, 1] = 0
    check_decode(torch_mod, c, q, mode, p, c.slots())
    c = Cache(torch_mod, [5, 70], 2, 64, 16, seed=3)
    for b, n in enumerate((5, 70)):
        c.k[c.table[b, (n - 1) // 16].long(), :, (n - 1) % 16] = 0
    check_decode(torch_mod, c, q[:2], mode, p, c.slots())


@pytest.mark.gpu
@pytest.mark.parametrize("n", [40, 300, 5000])
@pytest.mark.parametrize("d,half", [(64, True), (128, False), (128, True)])
def test_decode_keys_away_from_the_query(torch_mod, n, d, half):
    # LSSA: every score far below 0, where log(1 + e^x) is about e^x and down to e^-41
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    c = Cache(torch, [n, 3], 1, d, 16, half=half, seed=n)
    q = c.q(2)
    for b, count in enumerate((n, 3)):
        slot = torch.arange(count)
        away = -q[b, 0].float().cpu() + 0.3 * torch.randn(count, d, generator=c.g)
        c.k[c.table[b].long().cpu()[slot // 16].cuda(), 0, (slot % 16).cuda()] = away.to(c.dt).cuda()
    scores = torch.zeros(2, 1, c.cap, device="cuda")
    out = api.lssar_paged_decode(q, *c.args(), mode=MODE_LSSA, scores=scores)
    assert api.device_error_word() == 0
    for b, count in enumerate((n, 3)):
        kb, vb = (po.gather(host(x), c.table[b].tolist(), count)[:, 0] for x in (c.k, c.v))
        w = po.row_weights(host(q[b]), kb, MODE_LSSA)
        # a weight moves by no more than its score does, d log softplus(x) / dx <= 1, which
        # is |dx| <= (2d + 16) u x_max, u = 2^-24, as in the oracle (sum |q_c k_c| <= |q| |k|) and 4u |x|,
        # and by 2^-16 of itself: series 2^-20, exponential 2^-22, or logarithm 2^-22 of at
        # least 2^-5.5; the sum of weights by as much again
        x_max = po.length_scale(count, d)
        rel = 2 * ((2 * d + 20) * 2.0 ** -24 * x_max + 2.0 ** -16)
        # the value product: 2^-15 and the sum's rounding as in the oracle; in fp16 also half
        # a step of the least weights, 2^-25 against a sum of 2^-1 or more
        e = (rel + 2.0 ** -15 + (count / 4 + 64) * 2.0 ** -24) * w + (2.0 ** -24 if half else 0.0)
        ref = w @ vb
        tol = e @ np.abs(vb)
        tol = tol + torch.finfo(c.dt).eps / 2 * (np.abs(ref) + tol) + (2.0 ** -25 if half else 0.0)
        assert (np.abs(host(out[b]) - ref) <= tol).all()
        got = host(scores[b, 0, :count])
        assert (np.abs(got - w.sum(axis=0)) <= (rel + (count / 16 + 64) * 2.0 ** -24) * w.sum(axis=0)).all()


def keys_below(torch, c, q, b, n, top):
    """Keys of sequence b whose scores against q (one direction) lie from about x = top down to 22 less."""
    d, x1 = c.d, float(po.length_scale(n, c.d))
    unit = q.double() / q.double().norm()
    side = torch.randn(n, d, generator=c.g, dtype=torch.float64)
    side -= (side @ unit)[:, None] * unit
    side /= side.norm(dim=1, keepdim=True)
    low = max(-0.97, (top - 22) / x1)
    cos = low + (top / x1 - low) * torch.rand(n, 1, generator=c.g, dtype=torch.float64)
    k = (d ** 0.5 * (cos * unit + (1 - cos ** 2).sqrt() * side)).to(c.dt).cuda()
    slot = torch.arange(n)
    c.k[c.table[b].long().cpu()[slot // c.page].cuda(), 0, (slot % c.page).cuda()] = k


AWAY = [(300, 64, -8, False), (300, 64, -14, True), (5000, 64, -8, True), (5000, 128, -14, False), (16000, 64, -30, False),
        (20000, 128, -36, True)]


@pytest.mark.gpu
@pytest.mark.parametrize("mode,p", [(MODE_LSSAR, 1), (MODE_LSSAR, 3), (MODE_LSSAR, 15), (MODE_SIGMOID_RW, 1),
                                    (MODE_SIGMOID_RW, 15), (MODE_LSSA, 1)])
@pytest.mark.parametrize("n,d,top,half", AWAY)
def test_decode_rows_of_keys_away_from_the_query(torch_mod, mode, p, n, d, top, half):
    # every score is far below 0, and they differ: the weights do too
    c = Cache(torch_mod, [n, n // 3], 1, d, 16, half=half, seed=n)
    one = torch_mod.randn(2, 1, d, generator=c.g)
    q = (one * torch_mod.tensor([1.0, 2.5, 0.1]).view(1, 3, 1) + 0.01).to(c.dt)
    for b, count in enumerate((n, n // 3)):
        keys_below(torch_mod, c, q[b, 0], b, count, top)
    q = q.cuda()
    for b, count in enumerate((n, n // 3)):
        kb = po.gather(host(c.k), c.table[b].tolist(), count)[:, 0]
        w, e = po.row_weights(host(q[b]), kb, mode, p), po.weight_bound(host(q[b]), kb, mode, p)
        # not uniform by far, and resolved: the comparison can fail
        assert np.abs(w - 1 / count).sum(axis=1).min() > 0.5 and e.sum(axis=1).max() < 0.1
    check_decode(torch_mod, c, q, mode, p, c.slots(1e-3))


@pytest.mark.gpu
@pytest.mark.parametrize("mode,p,log2_weight", [(MODE_SOFTMAX, 1, -25.5), (MODE_SOFTMAX, 1, -24.6), (MODE_SOFTMAX, 1, -20.5),
                                                (MODE_SOFTMAX_RW, 3, -8.0), (MODE_LSSA, 1, -29.0)])
@pytest.mark.parametrize("n,d", [(131071, 64), (9000, 128)])
def test_decode_fp16_of_many_small_weights(torch_mod, mode, p, log2_weight, n, d):
    # one key of a large weight whose value is 0, and many of small ones that make the output
    torch = torch_mod
    c = Cache(torch, [n], 1, d, 128, half=True, seed=1)
    x = torch.zeros(c.cap, d)
    big = n // 3
    q = torch.zeros(1, 1, d)
    if mode == MODE_LSSA:
        # cosines: 0.3 for the one, the others' x = log2_weight ln 2
        q[0, 0, 0] = 4.0
        cos = torch.full((c.cap,), log2_weight * np.log(2) / float(po.length_scale(n, d)))
        cos[big] = 0.3
        x[:, 0], x[:, 1] = 16 * cos, 16 * (1 - cos ** 2).sqrt()
    else:
        q[0, 0, 0] = 16.0
        x[big, 0] = -log2_weight * np.log(2) * d ** 0.5 / 16
        if mode == MODE_SOFTMAX_RW:
            x[1::2, 0] = -40.0                     # half of the keys: no weight at all
            x[big, 0] = -log2_weight * np.log(2) * d ** 0.5 / 16
    pages = c.table[0].long()
    c.k[pages, 0] = x.view(-1, 128, d).to(c.dt).cuda()
    c.v[pages, 0] = (1 + 0.5 * torch.randn(c.cap, d, generator=c.g)).view(-1, 128, d).to(c.dt).cuda()
    c.v[pages[big // 128], 0, big % 128] = 0
    out, _ = check_decode(torch, c, q.to(c.dt).cuda(), mode, p, c.slots(1e-3))
    assert (out != 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("mode,p,log2_weight", [(MODE_SOFTMAX, 1, -25.5), (MODE_SOFTMAX, 1, -24.6), (MODE_SOFTMAX_RW, 3, -8.0)])
def test_decode_fp16_of_many_small_weights_in_one_segment(torch_mod, mode, p, log2_weight):
    # 600 sequences share their pages, so that most rows are summed by one block
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    n, B, d = 9000, 600, 64
    c = Cache(torch, [n], 1, d, 128, half=True, seed=1)
    x = torch.zeros(c.cap, d)
    if mode == MODE_SOFTMAX_RW:
        x[1::2, 0] = -40.0
    x[n // 3, 0] = -log2_weight * np.log(2) * d ** 0.5 / 16
    pages = c.table[0].long()
    c.k[pages, 0] = x.view(-1, 128, d).to(c.dt).cuda()
    c.v[pages, 0] = (1 + 0.5 * torch.randn(c.cap, d, generator=c.g)).view(-1, 128, d).to(c.dt).cuda()
    c.v[pages[n // 3 // 128], 0, n // 3 % 128] = 0
    q = torch.zeros(1, 1, d)
    q[0, 0, 0] = 16.0
    q = q.to(c.dt).cuda()
    out = api.lssar_paged_decode(q.repeat(B, 1, 1), c.k, c.v, c.table.repeat(B, 1), c.lens.repeat(B), p=p, mode=mode)
    assert api.device_error_word() == 0
    ref, _, err, _ = po.paged_decode(host(q), host(c.k), host(c.v), host(c.table), [n], mode, p)
    # as check_decode: the oracle's bound, half a step of fp16, half its least step
    bad = np.abs(host(out) - ref) - (err + 2.0 ** -11 * (np.abs(ref) + err) + 2.0 ** -25)
    assert bad.max() <= 0, (bad.max(), err.max())


@pytest.mark.gpu
@pytest.mark.parametrize("mode,p", [(MODE_SOFTMAX, 1), (MODE_SOFTMAX_RW, 3)])
@pytest.mark.parametrize("size", [300, 2000, 4000, 5600, 30000])
@pytest.mark.parametrize("grows", [False, True])
def test_decode_fp16_of_huge_scores(torch_mod, mode, p, size, grows):
    # scores from 2^20 to 2^33, whose steps pass the weights' range: the best key takes all
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    c = Cache(torch, [390], 1, 64, 16, half=True, seed=size)
    a = 1 - torch.arange(390) / 400
    slot = torch.arange(390)
    pages = c.table[0].long().cpu()[slot // 16].cuda()
    c.k[pages, 0, (slot % 16).cuda()] = (size * (a.flip(0) if grows else a)).view(-1, 1).repeat(1, 64).to(c.dt).cuda()
    q = torch.full((1, 2, 64), float(size)).to(c.dt).cuda()
    out = api.lssar_paged_decode(q, *c.args(), p=p, mode=mode)
    assert api.device_error_word() == 0
    best = 389 if grows else 0
    v = c.v[c.table[0, best // 16].long(), 0, best % 16].float()
    assert ((out[0].float() - v).abs() <= (2.0 ** -15 + 2.0 ** -11) * v.abs() + 2.0 ** -25).all()


@pytest.mark.gpu
def test_offsets_past_32_bits(torch_mod):
    # pages 2^28 + 8 elements apart, the last ones past 2^31 elements: the same bits as close together
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    n_pages, hkv, page, d, far = 10, 2, 16, 64, 2 ** 28 + 8
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(n_pages, hkv, page, d, generator=g).bfloat16().cuda() for _ in range(2))
    pool = torch.empty(n_pages * far, dtype=torch.bfloat16, device="cuda")
    shape, strides = (n_pages, hkv, page, d), (far, page * d, d, 1)
    kf, vf = pool.as_strided(shape, strides), pool.as_strided(shape, strides, 2 ** 27)
    kf.copy_(k)
    vf.copy_(v)
    table = torch.tensor([[9, 0, 8, 2], [7, 1, 6, 3]], dtype=torch.int32).cuda()
    lens = torch.tensor([20, 41], dtype=torch.int32).cuda()
    new = torch.randn(2, 2, hkv, 10, d, generator=g).bfloat16().cuda()
    q = torch.randn(2, 3 * hkv, d, generator=g).bfloat16().cuda()

    def serve(k, v):
        scores = torch.zeros(2, hkv, 4 * page, device="cuda")
        positions = torch.arange(4 * page, dtype=torch.int32).repeat(2, hkv, 1).cuda()
        n = api.lssar_paged_append(new[0], new[1], k, v, table, lens, scores=scores, positions=positions)
        out = api.lssar_paged_decode(q, k, v, table, n, scores=scores)
        n, _, _ = api.lssar_paged_evict(k, v, table, n, scores, positions, 25, recent=5)
        soft = api.lssar_paged_decode(q, k, v, table, n, mode=MODE_SOFTMAX)
        return [n, out, soft, scores, positions, k, v]

    close, apart = serve(k, v), serve(kf, vf)
    assert api.device_error_word() == 0
    assert close[0].tolist() == [25, 25] and close[1].isfinite().all() and close[2].isfinite().all()
    for x, y in zip(close, apart):
        assert torch.equal(x, y)


@pytest.mark.gpu
def test_decode_largest_group(torch_mod):
    c = Cache(torch_mod, [130, 0, 700], 1, 64, 16, seed=6)
    for mode, p in ((MODE_LSSAR, 3), (MODE_SOFTMAX, 1), (MODE_LSSA, 1)):
        check_decode(torch_mod, c, c.q(128), mode, p, c.slots(1e-2))


@pytest.mark.gpu
def test_decode_wide_table_strided_query_and_in_place_scores(torch_mod):
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    c = Cache(torch, [33, 0, 500], 3, 64, 16, width=700, seed=8)
    fused = torch.randn(3, 5, 6, 64, generator=c.g).to(c.dt).cuda()
    q = fused[:, 2]                                   # a slice of a fused projection's output
    assert not q.is_contiguous()
    scores = c.slots(1e-2)
    out, so = check_decode(torch, c, q, MODE_LSSAR, 3, scores)
    before = scores.clone()
    again = api.lssar_paged_decode(q, *c.args(), p=3, mode=MODE_LSSAR, scores=scores)
    assert torch.equal(out, again)
    for b, n in enumerate((33, 0, 500)):
        assert torch.equal(scores[b, :, :n], so[b, :, :n]) and torch.equal(scores[b, :, n:], before[b, :, n:])


@pytest.mark.gpu
def test_decode_equals_dense_decode(torch_mod):
    # a page table that happens to be the dense cache
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    B, H, L, d = 2, 3, 1000, 64
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(*s, generator=g).bfloat16().cuda() for s in ((B, H, d), (B, H, L, d), (B, H, L, d)))
    pages = [x.reshape(B, H, L // 8, 8, d).transpose(1, 2).reshape(-1, H, 8, d).contiguous() for x in (k, v)]
    table = torch.arange(B * L // 8, dtype=torch.int32).reshape(B, -1).cuda()
    for mode, p in MODES:
        dense = api.lssar_attn_decode(q, k, v, p=p, mode=mode)
        paged = api.lssar_paged_decode(q, *pages, table, torch.full((B,), L, dtype=torch.int32).cuda(), p=p, mode=mode)
        # both round a row that fp32 leaves within 1e-3 of exact here (checked above): one step apart at most
        assert (dense.float() - paged.float()).abs().max() <= 2 ** -7 * max(1.0, dense.float().abs().max().item())


@pytest.mark.gpu
def test_decode_bad_lengths_and_pages(torch_mod):
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    c = Cache(torch, [100, 100, 100, 100], 2, 64, 16, seed=4)
    q, scores = c.q(4), c.slots()
    good = api.lssar_paged_decode(q, *c.args())
    for value in (-1, c.cap + 1, 2 ** 31 - 1):
        c.lens[1] = value
        so = scores.clone()
        out = api.lssar_paged_decode(q, *c.args(), scores=scores, scores_out=so)
        assert api.device_error_word() == LENGTH
        assert out[1].isnan().all() and torch.equal(so[1], scores[1])
        assert torch.equal(out[[0, 2, 3]], good[[0, 2, 3]])
    c.lens[1] = 100
    for value in (-1, c.k.shape[0], 2 ** 31 - 1):
        table = c.table.clone()
        table[2, 3] = value
        so = scores.clone()
        out = api.lssar_paged_decode(q, c.k, c.v, table, c.lens, scores=scores, scores_out=so)
        assert api.device_error_word() == PAGE
        assert out[2].isnan().all() and torch.equal(out[[0, 1, 3]], good[[0, 1, 3]])
        assert so[2, :, :100].isnan().all() and not so[[0, 1, 3]].isnan().any()
    assert torch.equal(api.lssar_paged_decode(q, *c.args()), good) and api.device_error_word() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d,page,hkv,n,counts", [(64, 16, 3, 1, None), (128, 24, 2, 50, [0, 50, 17]), (64, 8, 1, 33, [33, 1, 0]),
                                                  (64, 64, 12, 200, [200, 3, 120]), (128, 16, 1, 0, None)])
@pytest.mark.parametrize("half", [False, True])
def test_append(torch_mod, d, page, hkv, n, counts, half):
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    lens = [0, 13, 30]
    c = Cache(torch, [x + n for x in lens], hkv, d, page, width=-(-300 // page), half=half, seed=n)
    # unused pages of the table are no pages
    both = torch.randn(3, n, 2, hkv, d, generator=c.g).to(c.dt).cuda()
    kn, vn = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
    c.lens = torch.tensor(lens, dtype=torch.int32).cuda()
    scores, pos = c.slots(), torch.full((3, hkv, c.cap), -1, dtype=torch.int32).cuda()
    first = torch.tensor([5, 0, 1000], dtype=torch.int32).cuda()
    cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda()
    bits = lambda t: host(t.view(torch.int16))   # noqa: E731
    want = po.paged_append(bits(kn.contiguous()), bits(vn.contiguous()), bits(c.k), bits(c.v), host(c.table), lens,
                           counts or [n] * 3, host(first), host(scores), host(pos))
    if n == 1:
        kn, vn = kn[:, :, 0], vn[:, :, 0]
    new = api.lssar_paged_append(kn, vn, *c.args(), counts=cnt, first_positions=first, scores=scores, positions=pos)
    assert api.device_error_word() == 0
    assert new.tolist() == want[4].tolist() and c.lens.tolist() == lens
    for got, ref in zip((bits(c.k), bits(c.v), host(scores), host(pos)), want):
        assert np.array_equal(got, ref)
    # positions default to the slots
    api.lssar_paged_append(kn, vn, *c.args(), counts=cnt, positions=pos)
    for b in range(3):
        m = counts[b] if counts else n
        assert pos[b, 0, lens[b]:lens[b] + m].tolist() == list(range(lens[b], lens[b] + m))


@pytest.mark.gpu
def test_append_that_does_not_fit_or_names_no_page(torch_mod):
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    c = Cache(torch, [48, 48, 48], 2, 64, 16, seed=6)
    new = torch.randn(3, 2, 5, 64, generator=c.g).to(c.dt).cuda()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()   # noqa: E731
    for lens, counts in ((i32(44, 40, 3), i32(5, 5, 5)), (i32(-1, 40, 3), i32(5, 5, 5)), (i32(3, 40, 3), i32(6, 5, 5)),
                         (i32(3, 40, 3), i32(-1, 5, 5)), (i32(2 ** 31 - 1, 40, 3), i32(5, 5, 5))):
        k = c.k.clone()
        out = api.lssar_paged_append(new, new, k, c.v, c.table, lens, counts=counts)
        assert api.device_error_word() == LENGTH
        assert out.tolist() == [lens[0].item(), 45, 8]
        assert torch.equal(k[c.table[0].long()], c.k[c.table[0].long()])
        assert torch.equal(k[c.table[1, 2].long(), :, 8:13], new[1])
    table = c.table.clone()
    table[1, 2] = c.k.shape[0]
    k = c.k.clone()
    api.lssar_paged_append(new, new, k, c.v, table, i32(0, 30, 3))
    assert api.device_error_word() == PAGE
    assert torch.equal(k[c.table[1, 1].long(), :, 14:], new[1, :, :2]) and torch.equal(k[c.table[1, 2].long()], c.k[c.table[1, 2].long()])


def evict_scores(torch, c, kind):
    s = c.slots()
    if kind == "ties":
        s = (s * 4).floor() * 0.25 - 0.25              # few values, 0 and negatives among them
        s = torch.where((s == 0) & (c.slots() < 0.5), -s, s)
    elif kind == "odd":
        s[c.slots() < 0.2] = float("nan")
        s[c.slots() < 0.2] = float("inf")
        s[c.slots() < 0.2] = -float("inf")
        s[c.slots() < 0.2] = 1e-40
    elif kind == "equal":
        s[:] = 0
    elif kind == "close":
        s = 1 + (s * 8).floor() * 2.0 ** -23
    return s


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["plain", "ties", "odd", "equal", "close"])
@pytest.mark.parametrize("lens,keep,recent,sinks,d,page,hkv", [
    ([0, 1, 40, 41, 42, 100, 333], 41, 0, 0, 64, 16, 2), ([300, 64, 65, 2000], 64, 32, 32, 128, 24, 1),
    ([5000, 4097, 1], 4096, 100, 4, 64, 128, 2), ([700, 3], 1, 1, 0, 64, 8, 1), ([50, 60], 1000, 3, 3, 64, 16, 1),
    ([9000, 3000], 250, 249, 1, 64, 256, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(torch_mod, kind, lens, keep, recent, sinks, d, page, hkv, in_place):
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    c = Cache(torch, lens, hkv, d, page, seed=keep)
    scores = evict_scores(torch, c, kind)
    pos = torch.rand(c.B, hkv, c.cap, generator=c.g).argsort(-1).to(torch.int32).cuda() + 7
    pos[0] = torch.arange(c.cap)
    bits = lambda t: host(t.view(torch.int16))   # noqa: E731
    want = po.paged_evict(bits(c.k), bits(c.v), host(c.table), lens, host(scores), host(pos), keep, recent, sinks)
    if in_place:
        new, so, p2 = api.lssar_paged_evict(*c.args(), scores, pos, keep, recent=recent, sinks=sinks)
        assert so is scores and p2 is pos
    else:
        so, p2 = torch.full_like(scores, -3.0), torch.full_like(pos, -3)
        s0, p0 = scores.clone(), pos.clone()
        new, _, _ = api.lssar_paged_evict(*c.args(), scores, pos, keep, recent=recent, sinks=sinks, scores_out=so, positions_out=p2)
        assert torch.equal(scores.view(torch.int32), s0.view(torch.int32)) and torch.equal(pos, p0)
    assert api.device_error_word() == 0
    assert new.tolist() == want[4].tolist()
    assert np.array_equal(bits(c.k), want[0]) and np.array_equal(bits(c.v), want[1])
    for b, n in enumerate(want[4]):
        assert np.array_equal(host(so)[b, :, :n], want[2][b, :, :n], equal_nan=True)
        assert np.array_equal(host(p2)[b, :, :n], want[3][b, :, :n])
        if not in_place:
            assert (so[b, :, n:] == -3.0).all() and (p2[b, :, n:] == -3).all()


@pytest.mark.gpu
@pytest.mark.parametrize("lens,keep,width", [([300, 90], 64, 10000), ([20000, 3], 5000, 1400), ([20000, 19999], 19000, 1251)])
def test_evict_wide_tables_and_long_rows(torch_mod, lens, keep, width):
    # room for 160000 tokens: keys that do not fit shared memory; rows over several CTAs
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    c = Cache(torch, lens, 1, 64, 16, width=width, seed=keep)
    scores = evict_scores(torch, c, "ties")
    pos = torch.arange(c.cap, dtype=torch.int32).repeat(2, 1, 1).cuda()
    bits = lambda t: host(t.view(torch.int16))   # noqa: E731
    want = po.paged_evict(bits(c.k), bits(c.v), host(c.table), lens, host(scores), host(pos), keep, 30, 2)
    new, _, _ = api.lssar_paged_evict(*c.args(), scores, pos, keep, recent=30, sinks=2)
    assert api.device_error_word() == 0 and new.tolist() == want[4].tolist()
    assert np.array_equal(bits(c.k), want[0]) and np.array_equal(bits(c.v), want[1])
    assert np.array_equal(host(scores), want[2]) and np.array_equal(host(pos), want[3])


@pytest.mark.gpu
def test_evict_many_rows(torch_mod):
    # more rows than fit the GPU at once, each over several CTAs
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    c = Cache(torch, [2300] * 12, 40, 64, 128, seed=9)
    scores = c.slots()
    pos = torch.arange(c.cap, dtype=torch.int32).repeat(12, 40, 1).cuda()
    bits = lambda t: host(t.view(torch.int16))   # noqa: E731
    want = po.paged_evict(bits(c.k), bits(c.v), host(c.table), [2300] * 12, host(scores), host(pos), 1000)
    api.lssar_paged_evict(*c.args(), scores, pos, 1000)
    assert np.array_equal(bits(c.k), want[0]) and np.array_equal(host(scores), want[2]) and np.array_equal(host(pos), want[3])


@pytest.mark.gpu
def test_evict_bad_lengths_and_pages(torch_mod):
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    c = Cache(torch, [90, 90, 90], 2, 64, 16, seed=6)
    scores, pos = c.slots(), torch.arange(c.cap, dtype=torch.int32).repeat(3, 2, 1).cuda()
    lens = c.lens.clone()
    lens[0], lens[2] = -5, c.cap + 1
    k = c.k.clone()
    new, so, _ = api.lssar_paged_evict(k, c.v, c.table, lens, scores, pos, 30, scores_out=scores.clone(), positions_out=pos.clone())
    assert api.device_error_word() == LENGTH
    assert new.tolist() == [-5, 30, c.cap + 1] and torch.equal(so[[0, 2]], scores[[0, 2]])
    assert torch.equal(k[c.table[0].long()].view(torch.int16), c.k[c.table[0].long()].view(torch.int16))
    table = c.table.clone()
    table[1, 5] = -1
    api.lssar_paged_evict(c.k, c.v, table, c.lens, scores, pos, 30, recent=10)     # the newest ten lie in that page
    assert api.device_error_word() == PAGE


@pytest.mark.gpu
@pytest.mark.parametrize("mode,p,G,d,half", [(MODE_LSSAR, 15, 1, 64, False), (MODE_LSSAR, 3, 4, 128, True), (MODE_SOFTMAX, 1, 8, 64, False)])
def test_serving_loop(torch_mod, mode, p, G, d, half):
    # prompts, then decode steps that evict whenever a sequence passes its bound
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    hkv, page, keep, B = 2, 16, 60, 3
    c = Cache(torch, [96] * B, hkv, d, page, half=half, seed=p)
    c.lens = torch.zeros(B, dtype=torch.int32).cuda()
    randn = lambda *s: torch.randn(*s, generator=c.g).to(c.dt).cuda()   # noqa: E731
    scores, pos = torch.zeros(B, hkv, c.cap).cuda(), torch.zeros(B, hkv, c.cap, dtype=torch.int32).cuda()
    counts = torch.tensor([70, 1, 59], dtype=torch.int32).cuda()
    seen = counts.clone()
    c.lens = api.lssar_paged_append(randn(B, hkv, 70, d), randn(B, hkv, 70, d), *c.args(), counts=counts, scores=scores, positions=pos)
    for step in range(12):
        c.lens = api.lssar_paged_append(randn(B, hkv, d), randn(B, hkv, d), *c.args(), first_positions=seen, scores=scores, positions=pos)
        seen += 1
        before = scores.clone()
        q = randn(B, hkv * G, d)
        out = api.lssar_paged_decode(q, *c.args(), p=p, mode=mode, scores=scores)
        ref, so = check_decode(torch, c, q, mode, p, before)
        assert torch.equal(ref, out)
        for b, n in enumerate(c.lens.tolist()):
            assert torch.equal(so[b, :, :n], scores[b, :, :n])
        bits = lambda t: host(t.view(torch.int16))   # noqa: E731
        want = po.paged_evict(bits(c.k), bits(c.v), host(c.table), c.lens.tolist(), host(scores), host(pos), keep, 8, 2)
        c.lens, _, _ = api.lssar_paged_evict(*c.args(), scores, pos, keep, recent=8, sinks=2)
        assert c.lens.tolist() == want[4].tolist()
        assert np.array_equal(bits(c.k), want[0]) and np.array_equal(bits(c.v), want[1])
        assert np.array_equal(host(scores), want[2]) and np.array_equal(host(pos), want[3])
    assert c.lens.tolist() == [60, 13, 60]
    # the protected tokens are still there, in every head
    for b in (0, 2):
        for h in range(hkv):
            at = set(pos[b, h, :60].tolist())
            assert len(at) == 60 and {0, 1} <= at and set(range(int(seen[b]) - 8, int(seen[b]))) <= at


@pytest.mark.gpu
def test_streams_and_graphs(torch_mod):
    # one serving step captured twice (two graphs share the library's pool), both replayed at once on two streams
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    hkv, d, page, keep = 4, 64, 16, 256

    def state(seed):
        c = Cache(torch, [300] * 4, hkv, d, page, seed=seed)
        c.lens.fill_(256)
        return dict(c=c, new=torch.randn(4, hkv, d, generator=c.g).bfloat16().cuda(), q=c.q(8), scores=c.slots(),
                    pos=torch.arange(c.cap, dtype=torch.int32).repeat(4, hkv, 1).cuda(),
                    lens=torch.empty_like(c.lens), after=torch.empty_like(c.lens), out=torch.empty(4, 8, d, dtype=torch.bfloat16).cuda())

    def step(s, stream=None):
        c, kv = s["c"], (s["c"].k, s["c"].v, s["c"].table)
        api.lssar_paged_append(s["new"], s["new"], *kv, c.lens, scores=s["scores"], positions=s["pos"], lens_out=s["lens"], stream=stream)
        api.lssar_paged_decode(s["q"], *kv, s["lens"], p=15, scores=s["scores"], out=s["out"], stream=stream)
        api.lssar_paged_evict(*kv, s["lens"], s["scores"], s["pos"], keep, recent=16, lens_out=s["after"], stream=stream)

    want = [state(1), state(2)]
    for s in want:
        for _ in range(4):
            step(s)
    graphs, got = [], [state(1), state(2)]
    for s in got:
        keep_scores, keep_pos, k, v = s["scores"].clone(), s["pos"].clone(), s["c"].k.clone(), s["c"].v.clone()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(s)
        s["scores"].copy_(keep_scores), s["pos"].copy_(keep_pos), s["c"].k.copy_(k), s["c"].v.copy_(v)
        graphs.append(g)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    third = state(1)
    torch.cuda.synchronize()
    for i in range(4):
        step(third, stream=streams[0] if i % 2 else streams[0].cuda_stream)
    torch.cuda.synchronize()
    assert api.device_error_word() == 0
    bits = lambda t: t.view(torch.int16) if t.dtype == torch.bfloat16 else t   # noqa: E731
    for a, b in ((got[0], want[0]), (got[1], want[1]), (third, want[0])):
        for name in ("scores", "pos", "out", "after", "lens"):
            assert torch.equal(bits(a[name]), bits(b[name])), name
        assert torch.equal(bits(a["c"].k), bits(b["c"].k)) and torch.equal(bits(a["c"].v), bits(b["c"].v))


@pytest.mark.gpu
@pytest.mark.parametrize("d,page,half", [(64, 16, False), (128, 24, True)])
def test_debug_build_checks_fire_nowhere(torch_mod, monkeypatch, d, page, half):
    # the debug-check build (bounds checks that record a code) gives the same bits and records nothing
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api, build
    build.build(debug=True)
    results = []
    for lib in (api.load_library(), api.load_debug_library()):
        monkeypatch.setattr(api, "_LIB", lib)
        c = Cache(torch, LENS_MIX, 2, d, page, half=half, seed=5)
        q, scores, got = c.q(6), c.slots(), []
        for mode, p in MODES:
            so = torch.zeros_like(scores)
            got += [api.lssar_paged_decode(q, *c.args(), p=p, mode=mode, scores=scores, scores_out=so), so]
        pos = torch.arange(c.cap, dtype=torch.int32).repeat(c.B, 2, 1).cuda()
        got += list(api.lssar_paged_evict(*c.args(), scores, pos, 100, recent=9)) + [c.k, c.v]
        torch.cuda.synchronize()
        assert api.device_error_word() == 0
        results.append(got)
    for a, b in zip(*results):
        view = torch.int16 if a.element_size() == 2 else torch.int32
        assert torch.equal(a.view(view), b.view(view))


@pytest.mark.gpu
def test_calls_on_two_streams_at_once(torch_mod):
    # decode steps of two caches, each on a stream of its own, interleaved without any wait between them
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    caches = [Cache(torch, [3000, 17, 900], 4, 64, 16, seed=s) for s in (1, 2)]
    qs = [c.q(8) for c in caches]
    want = [api.lssar_paged_decode(q, *c.args(), p=15) for q, c in zip(qs, caches)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(20):
        for i in (0, 1):
            got[i].append(api.lssar_paged_decode(qs[i], *caches[i].args(), p=15, stream=streams[i]))
    torch.cuda.synchronize()
    assert api.device_error_word() == 0
    for i in (0, 1):
        assert all(torch.equal(x, want[i]) for x in got[i])


@pytest.mark.gpu
def test_results_made_on_another_stream_take_no_block_in_use(torch_mod):
    # Blocks of the results' sizes, just freed on the current stream, are still written by
    # work that is queued there: a call on another stream makes its results elsewhere.
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    c = Cache(torch, [40, 3], 2, 64, 16, seed=3)
    lens = torch.tensor([20, 2], dtype=torch.int32).cuda()
    q, new, scores = c.q(4), c.q(2), c.slots()
    pos = torch.arange(c.cap, dtype=torch.int32).repeat(2, 2, 1).cuda()
    x = torch.randn(4, 2, 3, 100, 64, generator=c.g).bfloat16().cuda()
    ps = [1, 3, 15]
    stats = api.lssar_attn_fwd_train(*x[:3])[1]
    stats_p = api.lssar_attn_fwd_train_heads_p(*x[:3], ps)[1]
    kw = dict(scores_out=scores.clone(), positions_out=pos.clone())
    calls = [lambda s: [api.lssar_paged_decode(q, c.k, c.v, c.table, lens, stream=s)],
             lambda s: [api.lssar_paged_append(new, new, c.k, c.v, c.table, lens, stream=s)],
             lambda s: [api.lssar_paged_evict(c.k, c.v, c.table, lens, scores, pos, 24, stream=s, **kw)[0]],
             lambda s: [api.lssar_attn_fwd(*x[:3], stream=s)],
             lambda s: [api.lssar_attn_fwd_heads_p(*x[:3], ps, stream=s)],
             lambda s: [api.lssar_attn_decode(x[0, :, :, 0].contiguous(), x[1], x[2], stream=s)],
             lambda s: list(api.lssar_attn_fwd_train(*x[:3], stream=s)),
             lambda s: list(api.lssar_attn_fwd_train_heads_p(*x[:3], ps, stream=s)),
             lambda s: list(api.lssar_attn_bwd(*x, stats, stream=s)),
             lambda s: list(api.lssar_attn_bwd_heads_p(*x, stats_p, ps, stream=s))]
    side = torch.cuda.Stream()
    for i, call in enumerate(calls):
        want = call(None)
        torch.cuda.synchronize()
        for stream in (side, side.cuda_stream)[:2 if i < 4 else 1]:
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
def test_append_reads_one_tensor_as_several_arguments(torch_mod):
    # lens as the first positions says what the default does; as the counts, each sequence doubles
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    c = Cache(torch, [8, 3, 0], 2, 64, 16, seed=4)
    new = torch.randn(3, 2, 8, 64, generator=c.g).to(c.dt).cuda()
    results = []
    for kw in (dict(counts=c.lens.clone()), dict(counts=c.lens, first_positions=c.lens)):
        k, v, pos = c.k.clone(), c.v.clone(), torch.full((3, 2, c.cap), -1, dtype=torch.int32).cuda()
        n = api.lssar_paged_append(new, new, k, v, c.table, c.lens, positions=pos, **kw)
        results.append([n, k.view(torch.int16), v.view(torch.int16), pos])
    assert api.device_error_word() == 0 and results[0][0].tolist() == [16, 6, 0]
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_appends_that_read_the_pages_are_refused(lib):
    for at in (KP, KP + 4096, VP + 64):
        assert append(lib, desc(), counts=at) == -8
        assert append(lib, desc(), first=at) == -8
        assert append(lib, desc(), vn=at) == -8


def test_decodes_of_too_many_tiles_are_refused(lib):
    # 2^31 - 2^15 tiles: the last CTA's first one would not fit an int
    c = desc(B=65535, Hkv=1, max_pages=8192, page_stride=1024)
    assert decode(lib, c, qs=(8192, 64), H=128, mode=0, sc=None, so=None) == -2


def test_packed_cache_description_is_the_structure():
    from lssar_attn_fwd_gb300 import api
    values = dict(zip((f[0] for f in api.PagedCacheDesc._fields_), range(1, 13)))
    assert api._CACHE.pack(*values.values()) == bytes(api.PagedCacheDesc(**values))


@pytest.mark.gpu
@pytest.mark.parametrize("G,hkv,d,page,width", [(1, 12, 64, 8, None), (20, 2, 128, 256, None), (3, 1, 64, 24, 700)])
def test_debug_build_of_a_serving_step(torch_mod, monkeypatch, G, hkv, d, page, width):
    # append, decode and eviction in the debug-check build (work items, list, scratch and
    # page indices): the same bits, and nothing recorded
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api, build
    build.build(debug=True)
    results = []
    lens = [0, 1, 255, 256, 700, 1030, 33]
    for lib in (api.load_library(), api.load_debug_library()):
        monkeypatch.setattr(api, "_LIB", lib)
        c = Cache(torch, [n + 40 for n in lens], hkv, d, page, width=width, seed=7)
        c.lens = torch.tensor(lens, dtype=torch.int32).cuda()
        counts = torch.tensor([40, 0, 1, 39, 17, 40, 5], dtype=torch.int32).cuda()
        new, scores = torch.randn(7, hkv, 40, d, generator=c.g).to(c.dt).cuda(), c.slots()
        pos = torch.arange(c.cap, dtype=torch.int32).repeat(7, hkv, 1).cuda()
        c.lens = api.lssar_paged_append(new, new, *c.args(), counts=counts, scores=scores, positions=pos)
        got = [api.lssar_paged_decode(c.q(hkv * G), *c.args(), p=3, mode=mode, scores=scores)
               for mode in (MODE_SOFTMAX, MODE_LSSA, MODE_LSSAR)]
        for keep, recent in ((1000, 10), (200, 200), (3, 0)):
            c.lens, _, _ = api.lssar_paged_evict(*c.args(), scores, pos, keep, recent=recent)
            got.append(c.lens)
        torch.cuda.synchronize()
        assert api.device_error_word() == 0
        results.append(got + [c.k, c.v, scores, pos])
    for a, b in zip(*results):
        view = torch.int16 if a.element_size() == 2 else torch.int32
        assert torch.equal(a.view(view), b.view(view))
