"""Attention over the paged cache where the numbers are extreme: values near
the ends of their type's range, scales of every size, codes that are not
numbers, weights far below the largest.  Each against the 64-bit definition on
the rows that the cache holds.

The bounds.  A score of dim products in 32 bits is off by e = (dim + 4) 2^-24
sum |q||k| scale at most, a weight then by the factor 1 + 2e.  A weight meets
its value as two 16-bit parts: the first leaves 2^-8 of it (bfloat16), the
second 2^-8 of that, so 2^-16; its exponential and the sums of up to 2^7 steps
a warp and a few joins, each good to 2^-23, take as much again at most: 2^-15
of sum p |v|.  The result is rounded once to its type."""

import math

import pytest

import kv_reference as kr
from test_gpu_kv import BF, HF, built, clean_status, run_attend  # noqa: F401

torch = pytest.importorskip("torch")
lm = pytest.importorskip("layout_driven_movement_gb300")

pytestmark = pytest.mark.gpu

CODES = ["e4m3", "int8"]


def numbers(P, codes):
    """What held codes stand for under a scale of 1, in 64 bits."""
    if P.store is None:
        return codes.double()
    codes = codes.view(torch.uint8)
    return kr.e4m3_values()[codes.long()] if P.store == "e4m3" else \
        codes.view(torch.int8).double()


def refresh(P):
    """P.rows from the codes and scales as they are now."""
    for kv in range(2):
        x = numbers(P, P.codes[kv])
        if P.store is not None:
            x = x * P.scales[kv].double()[..., None]
        for b, n in enumerate(P.lens):
            ids = P.table[b, :-(-n // P.page)].long()
            P.rows[kv][b] = x[ids].flatten(0, 1)[:n]
    return P


def tokens(P):
    """[pool, page]: whether a sequence's token lies there."""
    used = torch.zeros(P.pool, P.page, dtype=torch.bool)
    for b, n in enumerate(P.lens):
        for j in range(0, n, P.page):
            used[int(P.table[b, j // P.page]), :min(P.page, n - j)] = True
    return used


def check(P, group, q, out, scale=None, rel=2.0 ** -15):
    scale = P.dim ** -0.5 if scale is None else scale
    for b, n in enumerate(P.lens):
        want, _, mag, dot = kr.attend(q[b].double(), P.rows[0][b],
                                      P.rows[1][b], group, scale)
        e = ((P.dim + 4) * 2.0 ** -24 * dot)[:, None]
        bound = (2 * e + rel) * mag + want.abs() * kr.ROUND[P.dtype] * 1.01 \
            + kr.TINY[P.dtype]
        off = (out[b].double() - want).abs()
        assert (off <= bound).all(), (b, n, (off / bound).max())


def aim(P, scores):
    """Keys whose first element is their score (0 elsewhere): with a query of
    1, 0, 0, ... and a softmax scale of 1 the scores are `scores(b, j)`."""
    for b, n in enumerate(P.lens):
        for j in range(n):
            at = int(P.table[b, j // P.page]), j % P.page
            s = scores(b, j)
            P.codes[0][at] = 0
            if P.store is None:
                P.codes[0][at][:, 0] = s
            else:
                one = {"e4m3": 0x38, "int8": 1}[P.store]
                P.codes[0][at][:, 0] = one if s >= 0 else \
                    {"e4m3": 0xb8, "int8": 255}[P.store]
                P.scales[0][at] = abs(s)
    q = torch.zeros(len(P.lens), P.heads, P.dim, dtype=P.dtype)
    q[..., 0] = 1
    return q


# --- values near the top of bfloat16 ----------------------------------------

@pytest.mark.parametrize("lens", [[1, 2, 20, 300], [6000], [2500, 33, 700]],
                         ids=str)
@pytest.mark.parametrize("dim,group", [(64, 1), (128, 4), (256, 9)])
def test_values_near_the_top_of_their_type(lens, dim, group):
    """The weighted mean of finite values is finite, however many there are:
    magnitudes in [2^126, 2^128), of one sign in one head and of either in the
    other."""
    P = kr.Pages(lens, 2, dim, 16, "nhd", BF, None, seed=dim)
    g = torch.Generator().manual_seed(dim)
    x = (1 + torch.rand(P.codes[1].shape, generator=g, dtype=torch.float64))
    x = x * 2.0 ** torch.randint(126, 128, x.shape, generator=g)
    x[:, :, 1] *= torch.randint(0, 2, x[:, :, 1].shape, generator=g) * 2 - 1
    x = x.clamp(-2.0 ** 128 * (1 - 2.0 ** -8), 2.0 ** 128 * (1 - 2.0 ** -8))
    P.codes[1] = torch.where(P.codes[1].isnan(), P.codes[1], x.to(BF))
    refresh(P)
    q, out, lse = run_attend(P, group)
    assert out.isfinite().all()
    check(P, group, q, out)


def test_large_values_under_growing_scores():
    """Every key outweighs the ones before it, so that the reference moves
    again and again under sums that are near the top of the range."""
    P = kr.Pages([700], 1, 64, 16, "nhd", BF, None, seed=1)
    q = aim(P, lambda b, j: j / 4)
    P.codes[1] = torch.where(P.codes[1].isnan(), P.codes[1],
                             P.codes[1].sign() * 2.0 ** 127 * 1.5)
    refresh(P)
    q, out, lse = run_attend(P, 1, q=q, scale=1.0)
    assert out.isfinite().all()
    check(P, 1, q, out, scale=1.0)


# --- scales of every size ---------------------------------------------------

@pytest.mark.parametrize("store", CODES)
@pytest.mark.parametrize("power", [-115, -90, -60, -20, 20, 60, 70, 100, 118])
@pytest.mark.parametrize("dim,group", [(64, 12), (128, 4), (256, 9)])
def test_value_scales_of_every_size(store, power, dim, group):
    """All rows of a head small or large alike, up to the largest that fit."""
    P = kr.Pages([1, 40, 700, 1500], 2, dim, 16, "nhd", BF, store, seed=power)
    P.scales[1] = P.scales[1] * 2.0 ** power
    refresh(P)
    q, out, lse = run_attend(P, group)
    check(P, group, q, out)


@pytest.mark.parametrize("store", CODES)
@pytest.mark.parametrize("size", [1e-37, 1e-25, 1e25, 1.2e38])
def test_rows_that_the_write_takes(store, size):
    """Finite rows, written by kv_write, come out of the attention as the
    definition says for the codes and scales that the cache then holds."""
    P = kr.Pages([33], 2, 64, 16, "nhd", BF, store, seed=3)
    plan = lm.KVPlan(lm.Layout.make(*P.page_layout()), BF, store)
    k, v = (torch.zeros(P.pool, 16, 2, 64, dtype=torch.uint8, device="cuda")
            for _ in range(2))
    scales = [torch.ones(P.pool, 2, 16, device="cuda") for _ in range(2)]
    cache = lm.KVCache(plan, k, v, *scales)
    x = torch.randn(2, 33, 2, 64, generator=torch.Generator().manual_seed(4))
    x[1] = x[1].clamp(-2.5, 2.5) * size
    j = torch.arange(33)
    slots = P.table[0].long()[j // 16] * 16 + j % 16
    lm.kv_write(cache, *x.to(BF).cuda(), slots.cuda())
    for kv, t in enumerate((k, v)):
        P.codes[kv] = t.cpu()
        P.scales[kv] = scales[kv].cpu().transpose(1, 2)
    refresh(P)
    q, out, lse = run_attend(P, 4)
    assert out.isfinite().all() and (out != 0).any()
    check(P, 4, q, out)


@pytest.mark.parametrize("store", CODES)
@pytest.mark.parametrize("order", ["large first", "small first", "mixed"])
@pytest.mark.parametrize("gap", [0, -160])
def test_scales_far_apart_in_one_head(store, order, gap):
    """Values 2^80 (e4m3) or 2^120 (int8) apart in one head: the large ones
    decide where they weigh as much; where their weights vanish (e^-160 of the
    others') the small ones come out as they are."""
    n, far = 400, 40 if store == "e4m3" else 60
    P = kr.Pages([n], 1, 64, 16, "nhd", BF, store, seed=6)
    large = {"large first": lambda j: j < n // 2,
             "small first": lambda j: j >= n // 2,
             "mixed": lambda j: j % 7 == 3}[order]
    q = aim(P, lambda b, j: (gap if large(j) else 0) + (j % 5) / 4)
    for j in range(n):
        at = int(P.table[0, j // 16]), j % 16
        P.scales[1][at] = P.scales[1][at] * 2.0 ** (far if large(j) else -far)
    refresh(P)
    q, out, lse = run_attend(P, 1, q=q, scale=1.0)
    check(P, 1, q, out, scale=1.0)


# --- codes that are not numbers ----------------------------------------------

@pytest.mark.parametrize("code", [127, 255])
@pytest.mark.parametrize("heads,group,dim,order", [
    (2, 4, 64, "nhd"), (2, 9, 64, "nhd"), (2, 4, 128, "hnd"),
    (1, 16, 128, "nhd"), (2, 5, 80, "nhd"), (2, 3, 256, "nhd"),
    (1, 12, 256, "hnd")])
def test_value_codes_that_are_not_numbers(code, heads, group, dim, order):
    """A NaN code makes the element it belongs to NaN in the outputs of its
    key head's queries, as the read back of the same page is, and no other."""
    lens = [1, 20, 64, 130, 700, 90]
    P = kr.Pages(lens, heads, dim, 16, order, BF, "e4m3", seed=dim)
    at = [(0, 0, 0, 3), (1, 19, heads - 1, dim - 1), (2, 0, 0, 16),
          (3, 77, 0, 9), (3, 77, heads - 1, 8), (4, 650, heads - 1, 40),
          (4, 3, 0, 2), (4, 699, 0, 33)]
    bad = torch.zeros(len(lens), heads * group, dim, dtype=torch.bool)
    for b, j, h, d in at:
        P.codes[1][int(P.table[b, j // 16]), j % 16, h, d] = code
        bad[b, h * group:(h + 1) * group, d] = True
    refresh(P)
    q, out, lse = run_attend(P, group)
    assert torch.equal(out.isnan(), bad)
    assert lse.isfinite().all()
    for rows in P.rows[1]:
        rows[rows.isnan()] = 0
    check(P, group, q, torch.where(bad, kr_clean(P, group, q), out.double()))


def kr_clean(P, group, q):
    """The definition on P's rows, [sequences, query heads, dim]."""
    return torch.stack([
        kr.attend(q[b].double(), P.rows[0][b], P.rows[1][b], group,
                  P.dim ** -0.5)[0] for b in range(len(P.lens))])


@pytest.mark.parametrize("code", [127, 255])
def test_key_codes_that_are_not_numbers(code):
    P = kr.Pages([30, 30], 2, 64, 16, "nhd", BF, "e4m3", seed=2)
    P.codes[0][int(P.table[1, 1]), 3, 1, 7] = code
    refresh(P)
    q, out, lse = run_attend(P, 4)
    bad = torch.zeros(2, 8, dtype=torch.bool)
    bad[1, 4:] = True
    assert torch.equal(out.isnan().all(-1), bad)
    assert torch.equal(out.isnan().any(-1), bad)
    assert torch.equal(lse.isnan(), bad)


def test_codes_that_are_not_numbers_past_the_window():
    """Keys that are not seen do not count, whatever they hold."""
    P = kr.Pages([100], 1, 64, 16, "nhd", BF, "e4m3", seed=2)
    q, want, lse = run_attend(P, 2, window=40)
    for j in range(60):
        P.codes[1][int(P.table[0, j // 16]), j % 16, 0, j % 64] = 127
    q, out, lse = run_attend(P, 2, window=40)
    assert torch.equal(out, want) and out.isfinite().all()


# --- weights far below the largest -------------------------------------------

@pytest.mark.parametrize("store,dtype", [(None, HF), (None, BF),
                                         ("e4m3", HF), ("int8", HF)])
@pytest.mark.parametrize("n,drop", [(16, 23.5), (16, 30.0), (64, 12.0),
                                    (3000, 23.0), (3000, 17.0)])
@pytest.mark.parametrize("at", [0, 5])
@pytest.mark.parametrize("sink", [0.0, 2.0 ** -10])
def test_many_weak_keys_beside_a_sink(store, dtype, n, drop, at, sink):
    """One key takes nearly all of the weight and adds nearly nothing; what
    the others, e^drop weaker each, add with values of 2^15 must not be
    lost."""
    P = kr.Pages([n], 2, 64, 16, "nhd", dtype, store, seed=n)
    q = aim(P, lambda b, j: drop if j == at else (j % 8) / 16)
    g = torch.Generator().manual_seed(n)
    page, off = int(P.table[0, at // 16]), at % 16
    if store is None:
        x = (1 + torch.rand(P.codes[1].shape, generator=g)) * 2.0 ** 14
        P.codes[1] = torch.where(P.codes[1].isnan(), P.codes[1], x.to(dtype))
        P.codes[1][page, off] = sink
    else:
        P.codes[1] = torch.where(
            tokens(P)[..., None, None],
            torch.randint(64, 127, P.codes[1].shape, generator=g).byte(),
            P.codes[1])
        P.scales[1] = torch.where(P.scales[1].isnan(), P.scales[1],
                                  torch.full_like(P.scales[1], 2.0 ** 7))
        P.codes[1][page, off] = 8 if sink else 0
        P.scales[1][page, off] = 2.0 ** -10
    refresh(P)
    q, out, lse = run_attend(P, 1, q=q, scale=1.0)
    check(P, 1, q, out, scale=1.0)


@pytest.mark.parametrize("dim,group", [(128, 9), (256, 1), (72, 4)])
def test_weak_keys_among_several_queries(dim, group):
    """The same where the queries of a head weigh the keys differently."""
    P = kr.Pages([200, 17], 2, dim, 16, "nhd", HF, None, seed=dim)
    g = torch.Generator().manual_seed(dim)
    aim(P, lambda b, j: 24.0 if j == 4 else -16.0 if j % 3 else 0.5)
    q = torch.zeros(2, 2 * group, dim, dtype=HF)
    q[..., 0] = torch.linspace(-1, 1, 2 * group)
    x = torch.randn(P.codes[1].shape, generator=g) * 2.0 ** 10
    P.codes[1] = torch.where(P.codes[1].isnan(), P.codes[1], x.to(HF))
    for b in range(2):
        P.codes[1][int(P.table[b, 0]), 4] = 2.0 ** -12
    refresh(P)
    q, out, lse = run_attend(P, group, q=q, scale=1.0)
    check(P, group, q, out, scale=1.0)


@pytest.mark.parametrize("store,dtype,rel", [
    (None, BF, 2.0 ** -15), (None, HF, 2.0 ** -18), ("e4m3", BF, 2.0 ** -15),
    ("int8", HF, 2.0 ** -15)])
def test_weights_keep_their_bits(store, dtype, rel):
    """Values +c and -c that cancel all but fully: what is left is the
    weights' own error.  float16 weights' parts leave 2^-22."""
    n = 64
    P = kr.Pages([n] * 4, 1, 16, 16, "nhd", dtype, store, seed=5)
    r = torch.Generator().manual_seed(8)
    s = [[round(float(x) * 64) / 64 for x in torch.randn(n, generator=r)]
         for _ in range(4)]
    q = aim(P, lambda b, j: s[b][j])
    for b in range(4):
        left = 0.0
        for j in sorted(range(n), key=lambda j: -s[b][j]):
            at = int(P.table[b, j // 16]), j % 16
            sign = -1 if left > 0 else 1
            left += sign * math.exp(s[b][j])
            if store is None:
                P.codes[1][at] = sign * 3.0
            else:
                P.codes[1][at] = {"e4m3": 0x44, "int8": 3}[store] if sign > 0 \
                    else {"e4m3": 0xc4, "int8": 253}[store]
                P.scales[1][at] = 1.0
    refresh(P)
    assert all(r.abs().eq(3).all() for r in P.rows[1])
    q, out, lse = run_attend(P, 1, q=q, scale=1.0)
    check(P, 1, q, out, scale=1.0, rel=rel)
