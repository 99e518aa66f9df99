"""Rotary positions (rope, its gradients, and the paged append that turns on the
way) through the package's entry points, against the float64 oracle; argument
checks on the CPU."""

import ctypes

import numpy as np
import pytest

from oracle import serving_oracle as so
from test_paged import KN, KP, LENS, LENGTH, LO, OUT, PAGE, POS, Q, SC, TAB, VN, VP, Cache, desc, host, lib, longs, torch_mod  # noqa: F401

Q2, K2, K2OUT = 20 << 40, 21 << 40, 22 << 40
BANDS = dict(scaling="bands", factor=8.0, original_length=64, low=1.0, high=8.0)
SCALINGS = [dict(), dict(scaling="linear", factor=3.0), dict(scaling="base", factor=8.0), BANDS]


def rotary(**kw):
    from lssar_attn_fwd_gb300 import api
    f = dict(base=10000.0, factor=1.0, low=1.0, high=32.0, original_length=1, rot_dim=64, interleaved=0, scaling=0)
    f.update(kw)
    return api._ROTARY.pack(*f.values())


# ---------------------------------------------------------------- argument checks (no GPU)

def rope(lib, q=Q, qs=(1 << 16, 4096, 64), qo=OUT, H=4, k=K2, ks=(1 << 16, 4096, 64), ko=K2OUT, Hk=2, B=3, L=16, d=64,
         dtype=0, r=None, pos=None, per=0, name="lssar_rope"):
    return getattr(lib, name)(q, longs(*qs), qo, H, k, longs(*ks), ko, Hk, B, L, d, dtype, rotary() if r is None else r, pos, per, None)


@pytest.mark.parametrize("name", ["lssar_rope", "lssar_rope_bwd"])
def test_bad_ropes_are_refused(lib, name):
    call = lambda **kw: rope(lib, name=name, **kw)   # noqa: E731
    for bad in (dict(q=None), dict(qo=None), dict(ko=None)):
        assert call(**bad) == -1, bad
    for bad in (dict(B=0), dict(L=0), dict(H=0), dict(Hk=0), dict(L=(1 << 24) + 1), dict(H=1 << 25), dict(B=1 << 30, L=1 << 20)):
        assert call(**bad) == -2, bad
    assert call(qs=(1 << 16, -64, 64)) == -2
    assert call(d=96) == -3
    assert call(dtype=2) == -11
    for bad in (dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")), dict(rot_dim=8), dict(rot_dim=72),
                dict(rot_dim=128), dict(rot_dim=0), dict(interleaved=2), dict(scaling=4), dict(scaling=-1),
                dict(scaling=1, factor=0.5), dict(scaling=2, factor=float("inf")), dict(scaling=2, factor=1e300, base=1e300),
                dict(scaling=3, factor=2.0, low=-1.0), dict(scaling=3, factor=2.0, low=4.0, high=4.0),
                dict(scaling=3, factor=2.0, original_length=0), dict(scaling=3, factor=2.0, high=float("inf"))):
        assert call(r=rotary(**bad)) == -13, bad
    for bad in (dict(qs=(1 << 16, 4096, 60)), dict(q=Q + 8), dict(qo=OUT + 8), dict(k=K2 + 2), dict(pos=POS + 2)):
        assert call(**bad) == -6, bad
    # outputs over inputs, over one another, over the positions; in place over rows that overlap
    for bad in (dict(qo=Q + 64), dict(qo=K2), dict(ko=OUT), dict(ko=Q), dict(pos=OUT + 64), dict(qo=Q, qs=(1 << 16, 0, 64)),
                dict(qo=Q, qs=(64, 4096, 64)), dict(qo=Q, k=Q + 128), dict(qo=Q, k=Q, ko=Q)):
        assert call(**bad) == -8, bad
    # slices of one buffer [B, L, H + Hk, d] that meet by one head
    st = (16 * 6 * 64, 64, 6 * 64)
    assert call(qo=Q, qs=st, k=Q + 3 * 128, ks=st, ko=Q + 3 * 128) == -8
    assert call(qo=Q, qs=st, k=Q + 5 * 128, ks=st, ko=Q + 5 * 128) == -8


def append_rope(lib, c, q=Q, qs=(1024, 512, 64), qo=OUT, H=4, kn=KN, vn=VN, ks=(1024, 512, 64), n=8, counts=None, first=None,
                sc=SC, pos=POS, lo=LO, r=None):
    return lib.lssar_paged_append_rope(ctypes.byref(c) if c else None, q, longs(*qs), qo, H, kn, longs(*ks), vn, longs(*ks), n,
                                       rotary() if r is None else r, counts, first, sc, pos, lo, None)


def test_bad_turning_appends_are_refused(lib):
    call = lambda **kw: append_rope(lib, desc(), **kw)   # noqa: E731
    assert append_rope(lib, None) == -1
    assert append_rope(lib, desc(d=96)) == -3
    for bad in (dict(lo=None), dict(kn=None), dict(q=None), dict(qo=None)):
        assert call(**bad) == -1, bad
    for bad in (dict(n=-1), dict(H=0), dict(n=1 << 24, H=1 << 10), dict(ks=(1024, -512, 64))):
        assert call(**bad) == -2, bad
    assert call(r=rotary(rot_dim=24)) == -13
    for bad in (dict(qs=(1024, 512, 60)), dict(qo=OUT + 8), dict(vn=VN + 8), dict(first=POS + 2)):
        assert call(**bad) == -6, bad
    for bad in (dict(lo=LENS), dict(sc=POS), dict(kn=KP + 4096), dict(qo=KP), dict(q=VP), dict(qo=KN), dict(qo=Q + 128), dict(qo=TAB),
                dict(qo=SC), dict(counts=OUT), dict(first=OUT), dict(qo=LO), dict(qo=Q, kn=Q + 128, qs=(8 * 384, 64, 384), ks=(8 * 384, 64, 384)),
                dict(qo=Q, qs=(1024, 512, 0)), dict(counts=KP), dict(lo=Q)):
        assert call(**bad) == -8, bad


def test_binding_refuses(torch_cpu=None):
    import torch
    from lssar_attn_fwd_gb300 import api
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.lssar_rope(x, x, api.Rotary(64))
    with pytest.raises(ValueError):
        api.Rotary(64, scaling="other")
    with pytest.raises(TypeError):
        api.lssar_rope([1], None, api.Rotary(64))


# ---------------------------------------------------------------- GPU

def check_rows(torch, got, x, positions, freq, inter, back=False):
    """Turned rows against the oracle, at its bound and half a step of the type."""
    ref, err = so.rope(host(x), positions, freq, inter, back)
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 0.0
    bad = np.abs(host(got) - ref) - (err + torch.finfo(x.dtype).eps / 2 * (np.abs(ref) + err) + tiny)
    assert bad.size == 0 or bad.max() <= 0, bad.max()
    rot = 2 * len(freq)
    assert torch.equal(got[..., rot:].view(torch.int16), x[..., rot:].view(torch.int16))


def make(torch, d, rot, inter, scaling):
    from lssar_attn_fwd_gb300 import api
    return api.Rotary(d, rot_dim=rot, interleaved=inter, **scaling), so.frequencies(rot, **scaling)


@pytest.mark.gpu
@pytest.mark.parametrize("scaling", SCALINGS)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,H,Hk,L,d,rot,half", [(1, 1, 1, 1, 64, 64, False), (2, 12, 4, 33, 64, 16, True), (3, 5, 1, 70, 128, 128, False),
                                                 (2, 2, 3, 129, 128, 48, True), (1, 130, 7, 5, 64, 48, False)])
def test_rope_and_back(torch_mod, scaling, inter, B, H, Hk, L, d, rot, half):
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    g = torch.Generator().manual_seed(L)
    dt = torch.float16 if half else torch.bfloat16
    both = torch.randn(B, L, H + Hk, d, generator=g).to(dt).cuda()
    q, k = both[:, :, :H].transpose(1, 2), both[:, :, H:].transpose(1, 2)
    r, freq = make(torch, d, rot, inter, scaling)
    first = torch.randint(-50, 5000, (B,), generator=g, dtype=torch.int32)
    each = torch.randint(0, 200000, (B, L), generator=g, dtype=torch.int32)
    at = np.arange(L)
    for positions, where in ((None, at[None, None]), (first, first.numpy()[:, None, None] + at), (each, each.numpy()[:, None])):
        dev = None if positions is None else positions.cuda()
        qo, ko = api.lssar_rope(q, k, r, positions=dev)
        assert qo.is_contiguous() and ko.is_contiguous()
        check_rows(torch, qo, q, where, freq, inter)
        check_rows(torch, ko, k, where, freq, inter)
        dq, dk = api.lssar_rope_bwd(q, k, r, positions=dev)
        check_rows(torch, dq, q, where, freq, inter, back=True)
        check_rows(torch, dk, k, where, freq, inter, back=True)
    # q alone, and in place on slices of one buffer: the same bits
    alone, none = api.lssar_rope(q, None, r, positions=dev)
    assert none is None and torch.equal(alone, qo)
    qi, ki = api.lssar_rope(q, k, r, positions=dev, q_out=q, k_out=k)
    assert qi is q and ki is k and torch.equal(q, qo) and torch.equal(k, ko)
    assert api.device_error_word() == 0


@pytest.mark.gpu
def test_rope_far_positions_and_extreme_values(torch_mod):
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    at = [0, 1, -1, 10 ** 6, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 123456789]
    g = torch.Generator().manual_seed(1)
    for d, inter, half in ((64, False, False), (128, True, True)):
        q = torch.randn(len(at), 2, 1, d, generator=g).to(torch.float16 if half else torch.bfloat16).cuda()
        r, freq = make(torch, d, d, inter, {})
        qo, _ = api.lssar_rope(q, None, r, positions=torch.tensor(at, dtype=torch.int32).cuda())
        check_rows(torch, qo, q, np.array(at)[:, None, None], freq, inter)
    # first + t past 2^31 does not wrap
    q = torch.randn(1, 1, 4, 64, generator=g).bfloat16().cuda()
    r, freq = make(torch, 64, 64, False, {})
    qo, _ = api.lssar_rope(q, None, r, positions=torch.tensor([2 ** 31 - 2], dtype=torch.int32).cuda())
    check_rows(torch, qo, q, 2 ** 31 - 2 + np.arange(4)[None, None], freq, False)
    # zeros, subnormals and infinities stay in their pairs
    q = torch.zeros(1, 1, 1, 64)
    q[0, 0, 0, 3], q[0, 0, 0, 5], q[0, 0, 0, 40] = float("inf"), float("nan"), 1e-39
    qo, _ = api.lssar_rope(q.bfloat16().cuda(), None, r, positions=torch.tensor([5], dtype=torch.int32).cuda())
    odd = ~qo[0, 0, 0].isfinite()
    assert odd.nonzero().flatten().tolist() == [3, 5, 35, 37]


@pytest.mark.gpu
def test_rope_gradient_against_differences(torch_mod):
    # the operator is linear: <g, R(x + h e) - R(x)> = h (R^T g)_e, in steps that bf16 holds
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    g = torch.Generator().manual_seed(3)
    r = api.Rotary(64, rot_dim=32, interleaved=True)
    x = torch.zeros(1, 64, 1, 64, dtype=torch.float16)
    x[0, range(64), 0, range(64)] = 1.0                      # head e: the unit vector e
    pos = torch.tensor([77], dtype=torch.int32).cuda()
    y, _ = api.lssar_rope(x.cuda(), None, r, positions=pos)
    dy = torch.randn(1, 1, 1, 64, generator=g).half().cuda()
    dx, _ = api.lssar_rope_bwd(dy, None, r, positions=pos)
    diff = host(y)[0, :, 0] @ host(dy)[0, 0, 0]
    # each of two entries of y rounded by 2^-11, each product by no more; dx by half a step
    assert (np.abs(host(dx)[0, 0, 0] - diff) <= 2.0 ** -11 * 3 * (np.abs(host(y)[0, :, 0]) @ np.abs(host(dy)[0, 0, 0])) + 2.0 ** -24).all()


@pytest.mark.gpu
@pytest.mark.parametrize("mode", [0, 2])
def test_training_step_with_positions(torch_mod, mode):
    # rope, attention, and both gradients back: against the same chain of oracles
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    from oracle import attention_backward, attention_forward
    g = torch.Generator().manual_seed(4)
    B, H, L, d = 1, 2, 130, 64
    q, k, v, dout = (torch.randn(B, H, L, d, generator=g).bfloat16().cuda() for _ in range(4))
    r, freq = make(torch, d, d, False, {})
    qr, kr = api.lssar_rope(q, k, r)
    out, stats = api.lssar_attn_fwd_train(qr, kr, v, p=3, mode=mode)
    dqr, dkr, dv = api.lssar_attn_bwd(qr, kr, v, dout, stats, p=3, mode=mode)
    dq, dk = api.lssar_rope_bwd(dqr, dkr, r)
    assert api.device_error_word() == 0
    # (the attention's tolerance of 2e-2 is for the inputs it gets: rows rounded by rope, 2^-8 of each
    # element, which move scores by up to ln d ln i 2^-7 = 0.16 and re-weighted outputs by more than 2e-2)
    check_rows(torch, qr, q, np.arange(L), freq, False)
    check_rows(torch, kr, k, np.arange(L), freq, False)
    qt, kt = host(qr), host(kr)
    ref = attention_forward(qt, kt, host(v), mode, 3)
    assert np.abs(host(out) - ref).max() <= 2e-2
    gq, gk, gv = attention_backward(qt, kt, host(v), host(dout), mode, 3)
    for got, want in ((dq, so.rope(gq, np.arange(L), freq, back=True)[0]), (dk, so.rope(gk, np.arange(L), freq, back=True)[0]), (dv, gv)):
        # the backward's own tolerance is 2e-2 of the norm; its gradients are rounded once more, by 2^-8
        assert np.linalg.norm(host(got) - want) <= 3e-2 * np.linalg.norm(want)


@pytest.mark.gpu
@pytest.mark.parametrize("d,rot,inter,page,hkv,G,n,counts", [
    (64, 64, False, 16, 3, 1, 1, None), (128, 64, True, 24, 2, 4, 50, [0, 50, 17]), (64, 48, False, 8, 1, 7, 33, [33, 1, 0]),
    (64, 16, True, 64, 12, 1, 200, [200, 3, 120]), (128, 128, False, 16, 1, 2, 0, None)])
@pytest.mark.parametrize("half", [False, True])
def test_append_rope(torch_mod, d, rot, inter, page, hkv, G, n, counts, half):
    # keys, values, scores and positions as rope and then append would leave them; queries as rope
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    lens, H = [0, 13, 30], hkv * G
    c = Cache(torch, [x + n for x in lens], hkv, d, page, width=-(-300 // page), half=half, seed=n)
    fused = torch.randn(3, n, H + 2 * hkv, d, generator=c.g).to(c.dt).cuda().transpose(1, 2)
    q, kn, vn = fused[:, :H], fused[:, H:H + hkv], fused[:, H + hkv:]
    c.lens = torch.tensor(lens, dtype=torch.int32).cuda()
    scores, pos = c.slots(), torch.full((3, hkv, c.cap), -1, dtype=torch.int32).cuda()
    first = torch.tensor([5, 0, 100000], dtype=torch.int32).cuda()
    cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda()
    r, freq = make(torch, d, rot, inter, BANDS)
    for firsts in (first, None):
        at = c.lens if firsts is None else firsts
        k, v, s2, p2 = c.k.clone(), c.v.clone(), scores.clone(), pos.clone()
        if n:
            qr, kr = api.lssar_rope(q, kn, r, positions=at)
            check_rows(torch, qr, q, at.cpu().numpy()[:, None, None] + np.arange(n), freq, inter)
        else:
            qr, kr = q, kn
        want = api.lssar_paged_append(kr, vn, k, v, c.table, c.lens, counts=cnt, first_positions=firsts, scores=s2, positions=p2)
        k3, v3, s3, p3 = c.k.clone(), c.v.clone(), scores.clone(), pos.clone()
        q_out = torch.full((3, H, n, d), 7.0, dtype=c.dt).cuda()
        args = (q, kn, vn) if n != 1 else (q[:, :, 0], kn[:, :, 0], vn[:, :, 0])
        got, new = api.lssar_paged_append_rope(*args, k3, v3, c.table, c.lens, r, counts=cnt, first_positions=firsts, scores=s3,
                                               positions=p3, q_out=q_out if n != 1 else q_out[:, :, 0])
        assert api.device_error_word() == 0 and torch.equal(new, want)
        for a, b in ((k, k3), (v, v3)):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        assert torch.equal(s2, s3) and torch.equal(p2, p3)
        for b in range(3):
            m = counts[b] if counts else n
            assert torch.equal(q_out[b, :, :m], qr[b, :, :m]) and (q_out[b, :, m:] == 7.0).all()
        made, _ = api.lssar_paged_append_rope(q, kn, vn, c.k.clone(), c.v.clone(), c.table, c.lens, r, counts=cnt, first_positions=firsts)
        for b in range(3):
            m = counts[b] if counts else n
            assert torch.equal(made[b, :, :m], qr[b, :, :m]) and (made[b, :, m:] == 0).all()
    if n > 1:
        # in place: a slice of the projection that keys and values are read from
        keep = fused.clone()
        api.lssar_paged_append_rope(q, kn, vn, c.k, c.v, c.table, c.lens, r, counts=cnt, q_out=q)
        assert torch.equal(fused[:, H:], keep[:, H:])
        for b in range(3):
            m = counts[b] if counts else n
            assert torch.equal(q[b, :, :m], qr[b, :, :m]) and torch.equal(fused[b, :, m:], keep[b, :, m:])
        assert torch.equal(c.k.view(torch.int16), k3.view(torch.int16))


@pytest.mark.gpu
def test_append_rope_that_does_not_fit_or_names_no_page(torch_mod):
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    c = Cache(torch, [48, 48, 48], 2, 64, 16, seed=6)
    new = torch.randn(3, 2, 5, 64, generator=c.g).to(c.dt).cuda()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()   # noqa: E731
    r = api.Rotary(64)
    for lens, counts in ((i32(44, 40, 3), i32(5, 5, 5)), (i32(-1, 40, 3), i32(5, 5, 5)), (i32(3, 40, 3), i32(6, 5, 5)),
                         (i32(3, 40, 3), i32(-1, 5, 5)), (i32(2 ** 31 - 1, 40, 3), i32(5, 5, 5))):
        k = c.k.clone()
        q, out = api.lssar_paged_append_rope(new, new, new, k, c.v, c.table, lens, r, counts=counts)
        assert api.device_error_word() == LENGTH
        assert out.tolist() == [lens[0].item(), 45, 8] and (q[0] == 0).all() and (q[1] != 0).any()
        assert torch.equal(k[c.table[0].long()].view(torch.int16), c.k[c.table[0].long()].view(torch.int16))
    table = c.table.clone()
    table[1, 2] = c.k.shape[0]
    k = c.k.clone()
    api.lssar_paged_append_rope(new, new, new, k, c.v, table, i32(0, 30, 3), r)
    assert api.device_error_word() == PAGE
    assert not torch.equal(k[c.table[1, 1].long(), :, 14:], c.k[c.table[1, 1].long(), :, 14:])
    assert torch.equal(k[c.table[1, 2].long()].view(torch.int16), c.k[c.table[1, 2].long()].view(torch.int16))


@pytest.mark.gpu
def test_rope_on_streams_and_in_graphs(torch_mod):
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    r = api.Rotary(64, **BANDS)
    q, k = torch.randn(2, 4, 100, 64).bfloat16().cuda(), torch.randn(2, 2, 100, 64).bfloat16().cuda()
    pos = torch.tensor([3, 9], dtype=torch.int32).cuda()
    want = api.lssar_rope(q, k, r, positions=pos)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        got = api.lssar_rope(q, k, r, positions=pos, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    outs = torch.empty_like(q), torch.empty_like(k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.lssar_rope(q, k, r, positions=pos, q_out=outs[0], k_out=outs[1])
    pos.add_(1)
    g.replay()
    want = api.lssar_rope(q, k, r, positions=pos)
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


@pytest.mark.gpu
def test_outputs_at_the_inputs_address(torch_mod):
    # the input itself turns in place, at its own strides; a tensor of other strides at its address is refused
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    B, H, L, d = 2, 4, 6, 64
    r, g = api.Rotary(d), torch.Generator().manual_seed(8)
    buf = torch.randn(B, L, H, d, generator=g).bfloat16().cuda()
    keep, q = buf.clone(), buf.transpose(1, 2)
    apart = torch.randn(B, H, L, d, generator=g).bfloat16().cuda()
    other = buf.view(B, H, L, d)
    for call in (api.lssar_rope, api.lssar_rope_bwd):
        with pytest.raises(ValueError):
            call(q, None, r, None, other)
        with pytest.raises(ValueError):
            call(apart, q, r, None, None, other)
        with pytest.raises(ValueError):
            call(other, None, r, None, q)
    c = Cache(torch, [20, 20], 2, d, 16, seed=3)
    lens, new = torch.tensor([3, 9], dtype=torch.int32).cuda(), torch.zeros(B, 2, L, d, dtype=torch.bfloat16).cuda()
    for x, y in ((q, other), (other, q)):
        with pytest.raises(ValueError):
            api.lssar_paged_append_rope(x, new, new, c.k, c.v, c.table, lens, r, q_out=y)
    assert torch.equal(buf, keep)
    # the same elements by another view, strides of dimensions of one apart
    want, _ = api.lssar_rope(q[:, :, :1], None, r)
    x = q[:, :, :1]
    y = x.as_strided(x.shape, (x.stride(0), x.stride(1), 8, 1))
    got, _ = api.lssar_rope(x, None, r, q_out=y)
    assert got is y and torch.equal(x, want) and torch.equal(buf[:, 1:], keep[:, 1:])
    # one token, [B, H, d] in place
    step = apart[:, :, 0]
    want, _ = api.lssar_paged_append_rope(step, new[:, :, 0], new[:, :, 0], c.k, c.v, c.table, lens, r)
    got, _ = api.lssar_paged_append_rope(step, new[:, :, 0], new[:, :, 0], c.k, c.v, c.table, lens, r, q_out=step)
    assert got is step and torch.equal(step, want)
    assert api.device_error_word() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n,H,d", [(1, 3, 64), (5, 4, 64), (70, 20, 128)])
def test_append_rope_without_counts_leaves_no_row_unwritten(torch_mod, n, H, d):
    # sequences that do not fit: zeros where the output is apart from q; untouched in place and where counts are given
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    c = Cache(torch, [160, 160, 160, 160], 2, d, 16, seed=6)
    q, new = torch.randn(4, H, n, d, generator=c.g).to(c.dt).cuda(), torch.randn(4, 2, n, d, generator=c.g).to(c.dt).cuda()
    r = api.Rotary(d, rot_dim=48)
    lens = torch.tensor([161 - n, 10, -1, 2 ** 31 - 1], dtype=torch.int32).cuda()
    good = torch.tensor([0, 10, 0, 0], dtype=torch.int32).cuda()
    first = torch.tensor([0, 10, 3, 4], dtype=torch.int32).cuda()
    append = lambda q, lens, **kw: api.lssar_paged_append_rope(q, new, new, c.k.clone(), c.v.clone(), c.table, lens, r,   # noqa: E731
                                                               first_positions=first, **kw)
    want, _ = append(q, good)
    assert api.device_error_word() == 0
    given = torch.full_like(q, 7.0)
    append(q, lens, q_out=given)
    made = []
    for _ in range(4):                        # blocks that held something else
        junk = [torch.full_like(q, 7.0) for _ in range(4)]
        del junk
        made.append(append(q, lens)[0])
    assert api.device_error_word() == LENGTH
    for out in (given, *made):
        assert torch.equal(out[1], want[1]) and (out[[0, 2, 3]] == 0).all()
    x = q.clone()
    append(x, lens, q_out=x)
    assert torch.equal(x[1], want[1]) and torch.equal(x[[0, 2, 3]], q[[0, 2, 3]])
    given.fill_(7.0)
    append(q, lens, counts=torch.full_like(lens, n), q_out=given)
    assert torch.equal(given[1], want[1]) and (given[[0, 2, 3]] == 7.0).all()
    assert api.device_error_word() == LENGTH


def exact_turns(base, rot, c):
    """Turns per position of pair c, as a Fraction of 2^-160."""
    from decimal import Decimal, getcontext
    from fractions import Fraction
    getcontext().prec = 70
    f = (Decimal(base).ln() * Decimal(-2 * c) / Decimal(rot)).exp()
    # pi by Machin's formula
    one = 1 << 220
    atan = lambda x: sum((-1) ** i * (one // ((2 * i + 1) * x ** (2 * i + 1))) for i in range(170))   # noqa: E731
    pi = Fraction(4 * (4 * atan(5) - atan(239)), one)
    return Fraction(f) / (2 * pi)


@pytest.mark.gpu
@pytest.mark.parametrize("base", [10000.0, 1000000.0, 1.25])
@pytest.mark.parametrize("near", [10 ** 6, 2 ** 31 - 2 ** 18])
def test_rope_angles_to_their_bound(torch_mod, base, near):
    # positions whose angle lies next to a half turn, where the output shows it: -sin of what is left
    import math
    from fractions import Fraction
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    d, pairs = 64, 32
    positions, left = [], []
    for c in range(pairs):
        turn = exact_turns(base, d, c)
        t64 = int(turn * 2 ** 64)
        m = near + np.arange(2 ** 18, dtype=np.uint64)
        with np.errstate(over="ignore"):
            phase = (m * np.uint64(t64)).astype(np.uint64) << np.uint64(1)       # modulo half a turn
        off = np.minimum(phase, ~phase).astype(np.float64)
        best = int(m[off.argmin()])
        x = turn * best * 2
        positions.append(best)
        left.append((-1.0 if round(x) % 2 else 1.0, math.sin(math.pi * float(x - round(x)))))
    q = torch.zeros(pairs, 1, 1, d, dtype=torch.float16)
    q[range(pairs), 0, 0, pairs + np.arange(pairs)] = 1.0        # (0, 1) -> (-sin, cos)
    out, _ = api.lssar_rope(q.cuda(), None, api.Rotary(d, base=base), positions=torch.tensor(positions, dtype=torch.int32).cuda())
    got = host(out)[range(pairs), 0, 0, range(pairs)]
    for c, (m, (sign, s)) in enumerate(zip(positions, left)):
        # the angle's bound; the sine's error and the output's half step, relative and absolute
        bound = 2 * math.pi * (m * 2.0 ** -50 + 2.0 ** -25)
        want = -sign * s
        assert abs(got[c] - want) <= bound + (2.0 ** -11 + 2.0 ** -21) * (abs(want) + bound) + 2.0 ** -25, (c, m, got[c], want)
    assert (np.abs([s for _, s in left]) < 0.01).sum() >= 20     # most of them do lie there
