"""The refusals of the cache's operators for long contexts, through the C ABI
with buffers that are never touched (all checks come before a launch; no GPU
needed)."""

import ctypes as C
import math

import pytest

from test_kv_host import (BASE, CAPACITY, INVALID, OVERFLOW, OVERLAP, built,  # noqa: F401
                          cache, plan_of, rows, status)

lm = pytest.importorskip("layout_driven_movement_gb300")

ONE = 64 * 8 * 16                     # rows of the cache's heads
Q, OUT, LSE, WS = BASE, BASE * 12, BASE * 9, BASE * 10
TABLE, LENS, W = BASE * 6, BASE * 7, BASE * 14
K, V, KS, VS = BASE * 2, BASE * 3, BASE * 4, BASE * 5


def test_the_cache_lies_where_these_tests_think():
    c = cache()
    assert (c.k, c.v, c.k_scale, c.v_scale) == (K, V, KS, VS)
    assert c.pages == 64


def weigh(store=None, c=None, q=None, out=None, seqs=3, hq=32, table=TABLE,
          stride=9, head=0, pages=9, lens=LENS, window=0, scale=0.1, lse=LSE,
          w=W, wcap=ONE, ws=WS, wsb=1 << 50):
    p = plan_of(store)
    return lm.lib().lm_kv_attend_weigh(
        p.handle, c or cache(), q or rows(Q, ts=4096),
        out or rows(OUT, ts=4096), seqs, hq, table, stride, head, pages, lens,
        window, scale, lse, w, wcap, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    ({"hq": 12}, INVALID), ({"head": -1}, INVALID), ({"w": W + 2}, INVALID),
    ({"wcap": ONE - 1}, CAPACITY), ({"w": K}, OVERLAP), ({"w": V}, OVERLAP),
    ({"w": Q}, OVERLAP), ({"w": OUT}, OVERLAP), ({"w": LSE}, OVERLAP),
    ({"w": LSE - ONE * 4 + 4}, OVERLAP), ({"store": "e4m3", "w": KS}, OVERLAP),
    ({"store": "int8", "w": VS + 4}, OVERLAP), ({"scale": math.nan}, INVALID),
    ({"seqs": -1}, INVALID), ({"window": -1}, INVALID),
    ({"table": None}, INVALID), ({"lens": None}, INVALID),
])
def test_weigh_refusals(kw, want):
    assert weigh(**kw) == want


def shared(store=None, c=None, q=None, out=None, seqs=3, hq=32, st=BASE * 16,
           sstride=5, groups=2, spages=5, sl=BASE * 17, starts=BASE * 18,
           table=TABLE, stride=9, pages=9, lens=LENS, scale=0.1, lse=LSE,
           ws=WS, wsb=1 << 50):
    p = plan_of(store)
    return lm.lib().lm_kv_attend_shared(
        p.handle, c or cache(), q or rows(Q, ts=4096),
        out or rows(OUT, ts=4096), seqs, hq, st, sstride, groups, spages, sl,
        starts, table, stride, pages, lens, scale, lse, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    ({"hq": 0}, INVALID), ({"hq": 12}, INVALID), ({"seqs": -1}, INVALID),
    ({"groups": -1}, INVALID), ({"spages": -1}, INVALID),
    ({"st": None}, INVALID), ({"sl": None}, INVALID),
    ({"starts": None}, INVALID), ({"sstride": 4}, INVALID),
    ({"starts": BASE + 2}, INVALID), ({"scale": math.inf}, INVALID),
    ({"lens": None}, INVALID), ({"table": None}, INVALID),
    ({"lse": LSE + 2}, INVALID), ({"out": rows(OUT, 100)}, CAPACITY),
    ({"out": rows(OUT, ts=1024)}, INVALID),
    ({"out": rows(Q + 256, ts=4096)}, OVERLAP),
    ({"out": rows(K, ts=4096)}, OVERLAP), ({"lse": OUT}, OVERLAP),
    ({"lse": K}, OVERLAP),
    ({"spages": 1 << 28, "sstride": 1 << 28}, OVERFLOW),
    ({"pages": 1 << 28, "stride": 1 << 28}, OVERFLOW),
])
def test_shared_refusals(kw, want):
    assert shared(**kw) == want


def bounds_of(data=BASE * 20, scale=BASE * 21, cap=ONE * 16, scap=64 * 8):
    """(of the plan's 128-element rows: 64 pages x 8 heads x 256 bytes)"""
    return lm._KVBounds(data, scale, cap, scap)


def bound(store=None, c=None, pages=BASE * 22, counts=BASE * 23, n=7, b=None):
    p = plan_of(store)
    return lm.lib().lm_kv_bound(p.handle, c or cache(), pages, counts, n,
                                b or bounds_of(), None)


@pytest.mark.parametrize("kw,want", [
    ({"n": -1}, INVALID), ({"pages": None}, INVALID),
    ({"counts": None}, INVALID), ({"pages": BASE + 2}, INVALID),
    ({"b": bounds_of(None)}, INVALID), ({"b": bounds_of(scale=None)}, INVALID),
    ({"b": bounds_of(BASE * 20 + 8)}, INVALID),
    ({"b": bounds_of(cap=64 * 8 * 256 - 1)}, CAPACITY),
    ({"b": bounds_of(scap=511)}, CAPACITY), ({"b": bounds_of(K)}, OVERLAP),
    ({"b": bounds_of(scale=V)}, OVERLAP),
    ({"b": bounds_of(scale=BASE * 20 + 4)}, OVERLAP),
    ({"store": "e4m3", "b": bounds_of(KS)}, OVERLAP),
    ({"pages": BASE * 20}, OVERLAP), ({"counts": BASE * 21 + 4}, OVERLAP),
])
def test_bound_refusals(kw, want):
    assert bound(**kw) == want


def test_bound_of_nothing():
    assert bound(n=0) == 0 and bound(n=0, pages=None, counts=None) == 0


def select(pages=64, b=None, q=None, seqs=3, hq=32, table=TABLE, stride=9,
           most=9, lens=LENS, keep=4, first=1, last=1, sel=BASE * 24,
           sl=BASE * 25, ws=WS, wsb=3 * 8 * 9 * 4):
    p = plan_of()
    return lm.lib().lm_kv_select(
        p.handle, pages, b or bounds_of(), q or rows(Q, ts=4096),
        seqs, hq, table, stride, most, lens, keep, first, last, sel, sl, ws,
        wsb, None)


@pytest.mark.parametrize("kw,want", [
    ({"hq": 12}, INVALID), ({"seqs": -1}, INVALID), ({"pages": 0}, INVALID),
    ({"keep": 0}, INVALID), ({"first": -1}, INVALID), ({"last": 0}, INVALID),
    ({"first": 4}, INVALID), ({"first": (1 << 31) - 1}, INVALID),
    ({"sel": None}, INVALID), ({"sl": None}, INVALID),
    ({"sel": BASE + 1}, INVALID), ({"table": None}, INVALID),
    ({"lens": None}, INVALID), ({"ws": None}, INVALID),
    ({"ws": WS + 8}, INVALID), ({"wsb": 3 * 8 * 9 * 4 - 1}, CAPACITY),
    ({"pages": 65}, CAPACITY), ({"q": rows(capacity=100)}, CAPACITY),
    ({"sel": BASE * 25 - 4}, OVERLAP), ({"sel": TABLE}, OVERLAP),
    ({"sl": LENS}, OVERLAP), ({"sel": BASE * 20}, OVERLAP),
    ({"sl": BASE * 21}, OVERLAP), ({"ws": Q}, OVERLAP),
    ({"ws": BASE * 24}, OVERLAP), ({"sel": Q}, OVERLAP),
    ({"most": 1 << 28, "stride": 1 << 28, "wsb": 1 << 50}, OVERFLOW),
])
def test_select_refusals(kw, want):
    assert select(**kw) == want


def test_select_of_no_sequences():
    assert select(seqs=0) == 0


def evict(store=None, c=None, w=W, wcap=ONE, table=TABLE, stride=9, seqs=3,
          pages=9, lens=LENS, kt=BASE * 26, kstride=3, kpages=3,
          kl=BASE * 27, keep=48, recent=8, ws=WS, wsb=3 * 8 * 48 * 4):
    p = plan_of(store)
    return lm.lib().lm_kv_evict(p.handle, c or cache(), w, wcap, table,
                                stride, seqs, pages, lens, kt, kstride,
                                kpages, kl, keep, recent, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    ({"w": None}, INVALID), ({"w": W + 2}, INVALID), ({"keep": 0}, INVALID),
    ({"recent": -1}, INVALID), ({"recent": 49}, INVALID),
    ({"seqs": -1}, INVALID), ({"kt": None}, INVALID), ({"kl": None}, INVALID),
    ({"kl": BASE + 1}, INVALID), ({"kstride": 2}, INVALID),
    ({"stride": 8}, INVALID), ({"ws": None}, INVALID),
    ({"wcap": ONE - 1}, CAPACITY), ({"wsb": 3 * 8 * 48 * 4 - 1}, CAPACITY),
    ({"kpages": 2}, CAPACITY), ({"c": cache(pages=65)}, CAPACITY),
    ({"w": K}, OVERLAP), ({"kl": V}, OVERLAP), ({"ws": K}, OVERLAP),
    ({"store": "int8", "w": KS}, OVERLAP), ({"kl": W}, OVERLAP),
    ({"ws": W}, OVERLAP), ({"kl": TABLE}, OVERLAP),
    ({"kl": BASE * 26}, OVERLAP), ({"ws": LENS}, OVERLAP),
    ({"w": TABLE}, OVERLAP), ({"kl": LENS + 4}, OVERLAP),
    ({"pages": 1 << 28, "stride": 1 << 28}, OVERFLOW),
])
def test_evict_refusals(kw, want):
    assert evict(**kw) == want


def test_evict_of_no_sequences():
    assert evict(seqs=0) == 0


def test_workspaces():
    L, p, n = lm.lib(), plan_of(), C.c_int64()
    assert lm.kv_select_workspace(p, 3, 9) == 3 * 8 * 9 * 4
    assert lm.kv_evict_workspace(p, 3, 48) == 3 * 8 * 48 * 4
    assert status(lm.kv_select_workspace, p, -1, 9) == INVALID
    assert status(lm.kv_select_workspace, p, 1, -1) == INVALID
    assert status(lm.kv_select_workspace, p, 1 << 30, 1 << 60) == OVERFLOW
    assert status(lm.kv_evict_workspace, p, -1, 9) == INVALID
    assert status(lm.kv_evict_workspace, p, 1, 0) == INVALID
    for fn in (L.lm_kv_attend_shared_workspace, L.lm_kv_attend_workspace):
        assert fn(None, 1, 8, C.byref(n)) == INVALID
        assert fn(p.handle, 1, 9, C.byref(n)) == INVALID
        assert fn(p.handle, 1, 8, None) == INVALID
    fn = L.lm_kv_attend_weigh_workspace
    assert fn(None, 1, 8, 5, C.byref(n)) == INVALID
    assert fn(p.handle, 1, 8, -1, C.byref(n)) == INVALID
    assert fn(p.handle, 1, 9, 5, C.byref(n)) == INVALID


def test_python_checks_before_the_library():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 3, 128)
    i = torch.zeros(2, dtype=torch.int32)
    plan = plan_of()

    class Stand:
        pass
    c = Stand()
    c.plan, c._p = plan, 0
    for call in (
            lambda: lm.kv_attend(c, x, i, i, x, weights=x),
            lambda: lm.kv_bound(c, i, i, x, x),
            lambda: lm.kv_select(c, x, x, x, i, i, i, i, None),
            lambda: lm.kv_evict(c, x, i, i, i, i, 4, None),
            lambda: lm.kv_attend_shared(c, x, i, i, i, i, i, x, None)):
        with pytest.raises(ValueError):
            call()                                   # not CUDA
    for fn in ("kv_attend_shared", "kv_bound", "kv_select", "kv_evict"):
        with pytest.raises(TypeError):
            getattr(lm._pycall(), fn)(1, 2)
