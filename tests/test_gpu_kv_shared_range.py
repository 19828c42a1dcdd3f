"""The attention over shared prefixes where the numbers are extreme: scales of
values of any sign and size, no numbers among them, scores far from 0.  Each
against the 64-bit definition on the rows that the cache holds, within the
bounds of test_gpu_kv_shared, unless the test derives its own."""

import math

import pytest

import kv_long_reference as lr
from test_gpu_kv_shared import (BF, HF, Case, built,  # noqa: F401
                                clean_status, ints, space)

torch = pytest.importorskip("torch")
lm = pytest.importorskip("layout_driven_movement_gb300")

pytestmark = pytest.mark.gpu

CODES = ["e4m3", "int8"]


def codes(C, kv):
    """What the held codes stand for under a scale of 1: [pool, page, heads,
    dim] in 64 bits."""
    x = C.P.held[kv]
    if C.P.order == "hnd":
        x = x.transpose(1, 2)
    if C.store == "int8":
        return x.double()
    return lr.e4m3_values().cuda()[x.long()]


def rescale(C, kv, change):
    """Scales of tokens as `change` makes them of the present ones (both
    [pool, heads, page]), and the rows that they give."""
    C.P.scales[kv] = change(C.P.scales[kv]).contiguous()
    C.P.rows[kv] = codes(C, kv) * \
        C.P.scales[kv].double().transpose(1, 2)[..., None]
    return C


@pytest.mark.parametrize("store", CODES)
@pytest.mark.parametrize("dim,order", [(64, "nhd"), (128, "hnd"),
                                       (256, "nhd")])
def test_value_scales_of_any_sign(store, dim, order):
    """Scales of values that are negative, or 0, and every code under them:
    int8's -128 has no opposite of its own type."""
    C = Case([300, 70], [0, 5, 9], [4, 0, 3, 1, 0, 2, 2, 9, 1], 2, 3, dim, 16,
             order, BF, store, seed=dim)
    if store == "int8":
        assert (C.P.held[1] == -128).any()
    g = torch.Generator(device="cuda").manual_seed(1)
    sign = torch.randint(-1, 2, C.P.scales[1].shape, generator=g,
                         device="cuda")
    C.check(*rescale(C, 1, lambda s: s * sign).run())
    C.check(*rescale(C, 1, lambda s: -s.abs()).run())
