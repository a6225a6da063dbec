"""The recurrence's and the state cache's entry points reject bad arguments without launching anything (CPU only: no
call here reaches a kernel)."""
import ctypes

import pytest
import torch

OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16 = 0, 1
# fake, well-separated, 16-byte aligned device addresses: validation never dereferences them
P = [ctypes.c_void_p((i + 1) << 40) for i in range(12)]


def off(p, n=8):
    return ctypes.c_void_p(p.value + n)


def offsets(*v):
    return (ctypes.c_int * len(v))(*v)


def fwd(L, x=P[0], g=P[1], cu=None, S0=P[2], o=P[3], S_T=P[4], B=2, H=3, T=70, d=64, gw=None, dt=F32, rule=0, ws=P[5],
        n=1 << 30):
    return L.efla_scan_fwd(x, g, cu, S0, o, S_T, B, H, T, d, d if gw is None else gw, dt, rule, ws, n, None)


def test_scan_fwd(efla):
    L = efla.lib
    for bad in (dict(B=-1), dict(H=-1), dict(T=-1), dict(d=0), dict(gw=2), dict(rule=7), dict(x=None), dict(g=None),
                dict(o=None), dict(ws=None), dict(n=255), dict(o=P[0]), dict(o=P[1]), dict(S_T=P[3]), dict(ws=P[0]),
                dict(ws=P[4]), dict(S_T=off(P[2], 16)), dict(S_T=P[1]), dict(o=P[5])):
        assert fwd(L, **bad) == INVALID, bad
    for name in ("x", "g", "S0", "o", "S_T", "ws"):
        at = dict(x=P[0], g=P[1], S0=P[2], o=P[3], S_T=P[4], ws=P[5])[name]
        assert fwd(L, **{name: off(at)}) == INVALID, name
    for bad in (dict(dt=2), dict(T=(1 << 30) + 1), dict(d=62), dict(d=4100), dict(d=4, dt=BF16), dict(d=12, dt=BF16), dict(H=1 << 16, B=1 << 16)):
        assert fwd(L, **bad) == UNSUPPORTED, bad
    assert fwd(L, B=0) == OK and fwd(L, H=0) == OK
    need = L.efla_scan_workspace_bytes(2, 3, 70, 64, 64, F32, 0)
    assert need >= 256 and fwd(L, n=need - 1) == INVALID
    assert L.efla_scan_workspace_bytes(2, 3, 70, 62, 62, F32, 0) == 0
    assert L.efla_scan_workspace_bytes(2, 3, 70, 64, 3, F32, 0) == 0
    # packed offsets: from 0, never falling, T in the end
    for cu in (offsets(1, 40, 70), offsets(0, 71, 70), offsets(0, 40, 69), offsets(0, -1, 70)):
        assert fwd(L, cu=cu) == INVALID, list(cu)


def bwd(L, x=P[0], g=P[1], cu=None, S0=P[2], dO=P[3], dST=P[4], dx=P[5], dg=P[6], dS0=P[7], B=2, H=3, T=70, d=64,
        gw=None, dt=F32, rule=0, saved=P[8], ns=1 << 30, ws=P[9], n=1 << 30):
    return L.efla_scan_backward(x, g, cu, S0, dO, dST, dx, dg, dS0, B, H, T, d, d if gw is None else gw, dt, rule, saved,
                                ns, ws, n, None)


def test_scan_backward(efla):
    L = efla.lib
    good = dict(x=P[0], g=P[1], S0=P[2], dO=P[3], dST=P[4], dx=P[5], dg=P[6], dS0=P[7], saved=P[8], ws=P[9])
    for name in good:
        assert bwd(L, **{name: off(good[name])}) == INVALID, name
    for name in ("x", "g", "dO", "dx", "dg", "ws"):
        assert bwd(L, **{name: None}) == INVALID, name
    for out in ("dx", "dg", "dS0", "ws"):            # no output over an input, the saved states or another output
        for other in good:
            if other != out:
                assert bwd(L, **{out: good[other]}) == INVALID, (out, other)
    for bad in (dict(B=-1), dict(T=-1), dict(gw=7), dict(rule=2), dict(n=100), dict(ns=100)):
        assert bwd(L, **bad) == INVALID, bad
    for bad in (dict(dt=5), dict(d=62), dict(d=20, dt=BF16)):
        assert bwd(L, **bad) == UNSUPPORTED, bad
    assert bwd(L, B=0) == OK
    with_states = L.efla_scan_backward_workspace_bytes(2, 3, 70, 64, 64, F32, 0, 1)
    without = L.efla_scan_backward_workspace_bytes(2, 3, 70, 64, 64, F32, 0, 0)
    assert without >= with_states + L.efla_scan_workspace_bytes(2, 3, 70, 64, 64, F32, 0)
    assert bwd(L, saved=None, n=without - 1) == INVALID
    assert bwd(L, cu=offsets(0, 80, 70)) == INVALID


def test_scan_step(efla):
    L = efla.lib
    f = lambda x=P[0], g=P[1], S=P[2], o=P[3], N=4, H=2, d=64, gw=64, dt=F32, rule=0: L.efla_scan_step(
        x, g, S, o, N, H, d, gw, dt, rule, None)
    for name, p in (("x", P[0]), ("g", P[1]), ("S", P[2]), ("o", P[3])):
        assert f(**{name: None}) == INVALID and f(**{name: off(p)}) == INVALID
    assert f(o=P[2]) == INVALID and f(S=P[0]) == INVALID and f(S=P[1]) == INVALID and f(o=P[0]) == INVALID
    assert f(N=-1) == INVALID and f(rule=3) == INVALID and f(gw=3) == INVALID
    assert f(d=66, gw=66) == UNSUPPORTED and f(dt=9) == UNSUPPORTED
    assert f(N=0) == OK and f(H=0) == OK


def test_paged_steps(efla):
    L = efla.lib
    good = dict(x=P[0], g=P[1], pages=P[2], pool=P[3], slots=P[4], source=P[5], o=P[6])

    def f(np=5, ns=6, pb=2 * 64 * 4, N=4, H=2, d=64, gw=64, dt=F32, rule=0, **kw):
        a = {**good, **kw}
        return L.efla_scan_step_paged(a["x"], a["g"], a["pages"], np, ns, a["pool"], pb, a["slots"], a["source"], a["o"],
                                      N, H, d, gw, dt, rule, None)

    deltas = dict(q=P[0], k=P[1], v=P[2], beta=P[3], g=P[4], pages=P[5], pool=P[6], slots=P[7], source=P[8], o=P[9])

    def h(np=5, ns=6, pb=2 * 64 * 64 * 4, N=4, H=2, d=64, dv=None, dt=F32, rule=0, **kw):
        a = {**deltas, **kw}
        return L.efla_recurrent_step_paged(a["q"], a["k"], a["v"], a["beta"], a["g"], a["pages"], np, ns, a["pool"], pb,
                                           a["slots"], a["source"], a["o"], N, H, d, d if dv is None else dv, dt, rule,
                                           None)

    for call, base, optional in ((f, good, ("source",)), (h, deltas, ("source", "g"))):
        for name in base:
            if name not in optional:
                assert call(**{name: None}) == INVALID, name
            assert call(**{name: off(base[name], 2)}) == INVALID, name
        for out in ("pool", "pages", "o"):
            for other in base:
                if other != out:
                    assert call(**{out: base[other]}) == INVALID, (out, other)
        for bad in (dict(np=0), dict(ns=0), dict(np=-3), dict(pb=16), dict(pb=1 << 20 | 8), dict(N=-1), dict(rule=2)):
            assert call(**bad) == INVALID, bad
        assert call(dt=4) == UNSUPPORTED and call(pb=1 << 45) == UNSUPPORTED
        assert call(N=0) == OK
    assert f(d=66, gw=66) == UNSUPPORTED and h(d=96) == UNSUPPORTED and h(dv=128) == UNSUPPORTED


def test_pages(efla):
    L = efla.lib
    assert L.efla_pages_bytes(5, 7) == 4 * (64 + 2 * 7 + 3 * 5)
    assert L.efla_pages_bytes(0, 7) == 0 and L.efla_pages_bytes(5, 0) == 0 and L.efla_pages_bytes(1 << 29, 7) == 0
    nb = L.efla_pages_bytes(5, 7)
    assert L.efla_pages_init(None, nb, 5, 7, None) == INVALID
    assert L.efla_pages_init(P[0], nb - 1, 5, 7, None) == INVALID
    assert L.efla_pages_init(off(P[0]), nb, 5, 7, None) == INVALID
    assert L.efla_pages_init(P[0], nb, 0, 7, None) == INVALID
    assert L.efla_pages_status(None, 0, None) == INVALID and L.efla_pages_status(off(P[0]), 0, None) == INVALID
    assert L.efla_pages_free(P[0], 5, 7, None, 3, None) == INVALID
    assert L.efla_pages_free(P[0], 5, 7, off(P[1], 2), 3, None) == INVALID
    assert L.efla_pages_free(P[0], 5, 7, P[0], 3, None) == INVALID
    assert L.efla_pages_free(P[0], 5, 7, P[1], -1, None) == INVALID
    assert L.efla_pages_free(P[0], 5, 7, None, 0, None) == OK
    for call in (L.efla_pages_fork, L.efla_pages_copy):
        f = lambda pages=P[0], np=5, ns=7, pool=P[1], pb=512, db=256, s=P[2], t=P[3], n=3: call(
            pages, np, ns, pool, pb, db, s, t, n, None)
        for bad in (dict(pages=None), dict(pages=off(P[0])), dict(np=0), dict(ns=-1), dict(pool=off(P[1])), dict(pb=520),
                    dict(db=8), dict(db=0), dict(db=1024), dict(s=None), dict(t=None), dict(s=off(P[2], 2)),
                    dict(t=off(P[3], 1)), dict(n=-1), dict(s=P[0]), dict(t=P[1]), dict(pool=P[0])):
            assert f(**bad) == INVALID, (call, bad)
        assert f(n=0) == OK
    assert L.efla_pages_copy(P[0], 5, 7, None, 512, 256, P[2], P[3], 3, None) == INVALID
    assert L.efla_pages_copy(P[0], 5, 7, P[1], 512, 256, P[2], P[3], 8193, None) == UNSUPPORTED
    g = lambda pages=P[0], np=5, ns=7, pool=P[1], pb=512, db=256: L.efla_pages_compact(pages, np, ns, pool, pb, db, None)
    for bad in (dict(pages=None), dict(pool=None), dict(pool=P[0]), dict(db=24), dict(pb=128), dict(np=0)):
        assert g(**bad) == INVALID, bad
    for call in (L.efla_pages_write, L.efla_pages_read):
        f = lambda pages=P[0], np=5, ns=7, pool=P[1], pb=512, rows=P[2], rb=256, slots=P[3], n=3: call(
            pages, np, ns, pool, pb, rows, rb, slots, n, None)
        for bad in (dict(pages=None), dict(pool=None), dict(rows=None), dict(slots=None), dict(rows=off(P[2])),
                    dict(rb=24), dict(rb=1024), dict(n=-2), dict(rows=P[1]), dict(slots=P[2]), dict(rows=P[0])):
            assert f(**bad) == INVALID, bad
        assert f(n=0) == OK


def test_counts_that_would_overflow(efla):
    """Lists and batches whose counts would pass 32 bits on the way to the device."""
    L = efla.lib
    assert L.efla_pages_free(P[0], 5, 7, P[1], (1 << 31) - 1, None) == INVALID
    assert L.efla_pages_fork(P[0], 5, 7, P[1], 512, 256, P[2], P[3], (1 << 31) - 1, None) == INVALID
    assert L.efla_pages_read(P[0], 5, 7, P[1], 1 << 20, P[2], 1 << 20, P[3], 1 << 24, None) == UNSUPPORTED
    assert L.efla_scan_workspace_bytes(1 << 15, 1 << 15, 1, 64, 1, BF16, 0) == 0
    assert fwd(L, B=1 << 15, H=1 << 15, T=1, S0=None, S_T=None, gw=1) == UNSUPPORTED
    assert L.efla_scan_step(P[0], P[1], P[2], P[3], 1 << 20, 1 << 11, 64, 1, F32, 0, None) == UNSUPPORTED
    assert L.efla_scan_workspace_bytes(1 << 15, 1 << 15, 1, 32, 1, BF16, 0) >= 1 << 37


def test_status_names(efla):
    assert efla.efla_status_string(efla.EFLA_ERR_SLOT) == "EFLA_ERR_SLOT"
    assert efla.efla_status_string(efla.EFLA_ERR_FULL) == "EFLA_ERR_FULL"


def test_binding_checks_its_tensors(efla):
    """Types, shapes, devices and strides are refused before the library is called."""
    x, g = torch.zeros(1, 2, 5, 64), torch.zeros(1, 2, 5, 64)
    for bad in (lambda: efla.efla_scan_fwd(x, g),                               # not on a GPU
                lambda: efla.efla_scan_fwd(x.half(), g),
                lambda: efla.efla_scan_fwd(x[0], g[0]),
                lambda: efla.efla_scan_fwd(x, g[..., :3]),
                lambda: efla.efla_scan_fwd(x, g, cu_seqlens=[0, 5]),
                lambda: efla.efla_scan_fwd(x[0], g[0], cu_seqlens=[]),
                lambda: efla.efla_scan_backward(x, g, x),
                lambda: efla.efla_scan_step(x[0], g, x[0]),
                lambda: efla.efla_scan_step(x[0], g[0], x[0]),
                lambda: efla.EflaPages(torch.zeros(100, dtype=torch.int32), 3, 4)):
        with pytest.raises(ValueError):
            bad()


def test_binding_refuses_rows_on_another_device_than_the_cache(efla):
    class Cache:
        block, n_pages, n_slots = torch.empty(64, dtype=torch.int32, device="meta"), 3, 4

    x, S, slots = torch.zeros(2, 3, 64), torch.zeros(3, 3, 64), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="where the cache is"):
        efla.efla_scan_step_paged(x, x, Cache, S, slots)
    with pytest.raises(ValueError, match="where the cache is"):
        efla.efla_recurrent_step_paged(x, x, x, x[..., 0], Cache, torch.zeros(3, 3, 64, 64), slots)
