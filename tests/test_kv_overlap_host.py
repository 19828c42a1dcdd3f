"""Buffers of the paged cache's calls that overlap: refused before a launch
(addresses that nothing dereferences; no GPU needed).  What may lie in one
buffer is tested with its results in test_gpu_kv_overlap.py."""

import pytest

from test_kv_host import (BASE, OVERLAP, built, cache, call_attend,  # noqa: F401
                          call_read, call_write, rows)

lm = pytest.importorskip("layout_driven_movement_gb300")

AT = BASE + (1 << 40)            # where the tests' value outputs lie


def outs(v_at, k=(1024, 128), v=(1024, 128)):
    """k_out at BASE and v_out `v_at` elements on; (token, head) strides."""
    return {"k": rows(BASE, ts=k[0], hs=k[1]),
            "v": rows(BASE + 2 * v_at, ts=v[0], hs=v[1])}


@pytest.mark.parametrize("kw", [
    outs(0), outs(1024), outs(99 * 1024), outs(64), outs(127),
    outs(99 * 1024 + 7 * 128 + 127),
    # one buffer of wider rows: a head too near, from either side
    outs(7 * 128, (2048, 128), (2048, 128)),
    outs(2048 - 7 * 128, (2048, 128), (2048, 128)),
    outs(2048 * 50 + 5 * 128 + 1, (2048, 128), (2048, 128)),
    # every other head, half a head off
    outs(64, (2048, 256), (2048, 256)), outs(192, (2048, 256), (2048, 256)),
    # heads of different distances
    outs(14 * 128, (4096, 256), (4096, 128)),
    outs(7 * 128, (4096, 128), (4096, 256)),
    # heads before tokens
    outs(128, (128, 12800), (128, 12800)),
    outs(12800 * 3, (128, 12800), (128, 12800)),
    outs(12800 - 128, (128, 12800), (128, 12800)),
    # tokens a different distance apart
    outs(1024, (2048, 128), (4096, 128)),
])
def test_read_into_outputs_that_meet(kw):
    assert call_read(**kw) == OVERLAP


def test_read_whatever_the_order_of_the_outputs():
    for at in (64, 1024, 99 * 1024):
        kw = outs(at)
        assert call_read(k=kw["v"], v=kw["k"]) == OVERLAP


KS, VS, ONE = BASE * 4, BASE * 5, 64 * 8 * 16 * 4     # scales, their bytes


@pytest.mark.parametrize("store", ["e4m3", "int8"])
@pytest.mark.parametrize("kw", [
    {"vs": KS + 4}, {"vs": KS + ONE - 4}, {"vs": KS - 4},
    {"ks": BASE * 2 + 64}, {"vs": BASE * 2 - 4},
    {"ks": BASE * 3 + (64 << 14) - 4},           # the last page's last bytes
])
def test_scales_that_meet(store, kw):
    """Each other or a page, in every call."""
    c = cache(**kw)
    assert call_write(store, c) == OVERLAP
    assert call_read(store, c) == OVERLAP
    assert call_attend(store, c) == OVERLAP


def test_rows_that_meet_the_scales():
    for at in (KS, VS - 2, KS + ONE - 2):
        assert call_write("int8", k=rows(at)) == OVERLAP
        assert call_write("e4m3", v=rows(at)) == OVERLAP
        assert call_read("int8", k=rows(at)) == OVERLAP
        assert call_read("e4m3", v=rows(at)) == OVERLAP
        assert call_attend("int8", out=rows(at, ts=4096)) == OVERLAP


@pytest.mark.parametrize("store,at", [
    ("e4m3", KS), ("int8", VS + ONE - 4), (None, BASE * 2), (None, BASE * 3),
    (None, BASE), (None, BASE + 2 * 3 * 4096 - 4),    # the queries
    (None, BASE * 12 - 4), (None, BASE * 12 + 4096)])  # the outputs
def test_lse_that_meets(store, at):
    assert call_attend(store, lse=at) == OVERLAP
