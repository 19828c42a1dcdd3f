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
