"""Arguments that are no tensors, at the calls of a serving step: refused by type,
before anything is launched."""

import pytest

from test_paged import Cache, torch_mod  # noqa: F401


@pytest.mark.gpu
def test_arguments_that_are_no_tensors(torch_mod):
    torch = torch_mod
    from lssar_attn_fwd_gb300 import api
    c = Cache(torch, [20, 20], 2, 64, 16, seed=3)
    q, new = (torch.zeros(2, h, 3, 64, dtype=c.dt).cuda() for h in (4, 2))
    r = api.Rotary(64)
    i32 = torch.tensor([1, 2], dtype=torch.int32).cuda()
    lens, free, count = i32 * 4, torch.arange(9, dtype=torch.int32).cuda(), torch.tensor([9], dtype=torch.int32).cuda()
    attend = lambda q, **kw: api.lssar_paged_attend(q, *c.args(), **kw)   # noqa: E731
    append = lambda q, k, v, **kw: api.lssar_paged_append_rope(q, k, v, c.k, c.v, c.table, lens, r, **kw)   # noqa: E731
    rope = lambda **kw: api.lssar_rope(q, new, r, **kw)   # noqa: E731
    reserve = lambda counts, **kw: api.lssar_paged_reserve(c.table, lens, counts, 16, free, count, **kw)   # noqa: E731
    release = lambda lens_new, **kw: api.lssar_paged_release(c.table, lens, lens_new, 16, free, count, **kw)   # noqa: E731
    for bad in ([1, 2], 7, i32.cpu().numpy()):
        calls = [lambda: attend(bad), lambda: attend(q, counts=bad), lambda: attend(q, out=bad),
                 lambda: append(bad, new, new), lambda: append(q, bad, new), lambda: append(q, new, bad),
                 lambda: append(q, new, new, q_out=bad), lambda: append(q, new, new, counts=bad),
                 lambda: append(q, new, new, first_positions=bad), lambda: append(q, new, new, scores=bad),
                 lambda: append(q, new, new, positions=bad), lambda: append(q, new, new, lens_out=bad),
                 lambda: rope(positions=bad), lambda: rope(q_out=bad), lambda: rope(k_out=bad),
                 lambda: reserve(bad), lambda: reserve(i32, counts_out=bad), lambda: reserve(i32, free_out=bad),
                 lambda: release(bad), lambda: release(i32, free_out=bad)]
        for i, call in enumerate(calls):
            with pytest.raises(TypeError):
                call()
                raise AssertionError(i)
    assert api.device_error_word() == 0
