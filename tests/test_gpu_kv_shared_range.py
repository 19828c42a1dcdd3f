"""The attention over shared prefixes where the numbers are extreme: scales of
values of any sign and size, no numbers among them, scores far from 0.  Each
against the 64-bit definition on the rows that the cache holds, within the
bounds of test_gpu_kv_shared, unless the test derives its own."""

import math

import pytest

import kv_long_reference as lr
import kv_reference as kr
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


@pytest.mark.parametrize("store", CODES)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_value_scales_that_are_no_numbers(store, bad):
    """One key whose value's scale is no number, as a row with one is written:
    the results of its group are none, and the lse, which has nothing to do
    with values, is what it is."""
    for dim in (64, 256):
        C = Case([300, 70], [0, 5, 9], [4, 0, 3, 1, 0, 2, 2, 9, 1], 2, 3, dim,
                 16, "nhd", BF, store, seed=dim)
        page = int(C.P.table[0, 200 // 16])
        C.P.scales[1][page, :, 200 % 16] = bad
        out, lse = C.run()
        assert out[:5].isnan().all()
        C.P.rows[1][page, 200 % 16] = 0
        out[:5] = 0
        for b in range(9):
            k, v = C.rows(b)
            _, wl, _, mag, dot = lr.attend(C.q[b].double(), k, v, 3, dim ** -.5)
            bl = kr.attend_bounds(BF, dim, out[b].double(), wl, mag, dot)[1]
            assert ((lse[b].double() - wl).abs() <= bl).all()
        C.lens, C.q, C.starts = C.lens[5:], C.q[5:], [0, 0, 4]
        C.groups = 2
        table = C.P.table
        C.P.table = torch.cat([table[:2], table[7:]])
        C.P.lens = [300, 70] + C.lens
        C.check(out[5:], lse[5:])


def test_no_numbers_under_a_scale_of_0():
    """0 times a code that is no number is none; an unseen one is not used."""
    C = Case([300], [0, 3], [3] * 3, 1, 2, 64, 16, "nhd", BF, "e4m3")
    page = int(C.P.table[0, 2])
    C.P.scales[1][page, 0, 5] = 0
    C.P.held[1][page, 5, 0, 9] = 0x7f
    last = int(C.P.table[0, 299 // 16])
    C.P.held[1][last, 12:] = 0x7f
    out, lse = C.run()
    assert out[:, :, 9].isnan().all() and not lse.isnan().any()
    assert not out[:, :, :9].isnan().any() and not out[:, :, 10:].isnan().any()


def check_far(C, out, lse, scale=None):
    """Every key's scale is its own, so that a weight's rounding counts relative
    to the largest weight times scale of its row: besides 2^-11 of its own, off
    by 2^-32 of that times the largest code a key."""
    scale = C.dim ** -0.5 if scale is None else scale
    most = {"e4m3": 448.0, "int8": 128.0}[C.store]
    for b in {0, len(C.lens) // 2, len(C.lens) - 1}:     # (all rows are alike)
        k, v = C.rows(b)
        want, wl, p, mag, dot = lr.attend(C.q[b].double(), k, v, C.group, scale)
        bo, bl = kr.attend_bounds(C.dtype, C.dim, want, wl, mag, dot)
        bo += (2.0 ** -11 - 2.0 ** -10 + 2.0 ** -16) * mag
        s = C.row_scales(b).abs()                # [n, heads]
        top = (p.view(C.heads, C.group, -1) * s.T[:, None]).amax(-1)
        bo += (len(v) * 2.0 ** -32 * most * top).reshape(-1, 1)
        assert out[b].isfinite().all(), b
        assert ((out[b].double() - want).abs() <= bo).all(), b
        assert ((lse[b].double() - wl).abs() <= bl).all(), b


class Scaled(Case):
    """A case whose value scales, and where wanted whose scores, are given for
    each token of a prefix (own tokens: none)."""

    def __init__(self, n, seqs, heads, group, dim, store, scales, scores=None,
                 dtype=BF):
        super().__init__([n], [0, seqs], [0] * seqs, heads, group, dim, 16,
                         "nhd", dtype, store, seed=dim)
        self.at = self.P.table[0, :n // 16].long().cuda()
        s = scales.cuda().float().view(-1, 1, 16).expand(-1, heads, -1)

        def change(x):
            x = x.clone()
            x[self.at] = s
            return x
        rescale(self, 1, change)
        if scores is not None:
            one = {"e4m3": 0x38, "int8": 1}[store]
            k = torch.zeros(n // 16, 16, heads, dim, device="cuda",
                            dtype=torch.int64)
            k[..., 0] = one
            self.P.held[0][self.at] = k.to(self.P.held[0].dtype)
            t = scores.cuda().float().view(-1, 1, 16).expand(-1, heads, -1)

            def aim(x):
                x = x.clone()
                x[self.at] = t
                return x
            rescale(self, 0, aim)
            self.q.zero_()
            self.q[..., 0] = 1

    def row_scales(self, b):
        return self.P.scales[1][self.at].double().transpose(1, 2).reshape(
            -1, self.heads)


@pytest.mark.parametrize("store", CODES)
@pytest.mark.parametrize("power", [-140, -126, -112, -64, -33, -32, -1, 0, 1,
                                   47, 90, 112, 118])
def test_value_scales_of_every_size(store, power):
    """Scales about 2^power, those of bands' ends among them; own tokens' as
    the prefix's, so that the two parts are joined."""
    for dim, heads, group, seqs in ((64, 2, 3, 5), (128, 1, 4, 40),
                                    (256, 1, 2, 3)):
        own = 3 if power > -120 else 0       # (lm_kv_attend's range)
        C = Case([700, 130], [0, seqs - 1, seqs], [own] * seqs, heads, group,
                 dim, 16, "nhd", BF, store, seed=dim)
        g = torch.Generator(device="cuda").manual_seed(power)
        by = 2.0 ** torch.randint(-1, 2, C.P.scales[1].shape, generator=g,
                                  device="cuda")
        shift = 2.0 ** (power + 3.0 - (3 if power > 115 else 0))
        rescale(C, 1, lambda s: (s.double().sign() * shift * by / 8).float())
        C.check(*C.run())


@pytest.mark.parametrize("store", CODES)
@pytest.mark.parametrize("order", ["up", "down", "mixed", "steps"])
@pytest.mark.parametrize("lo,hi", [(-140, 118), (-40, 30), (-8, 7)])
def test_value_scales_over_many_bands(store, order, lo, hi):
    """Scales over 2^lo .. 2^hi in one prefix, in tiles that one block has or
    several; equal scores, and scores that make up for the scales, so that the
    largest weight lies where the smallest value does."""
    for n, seqs, dim, heads in ((640, 3, 64, 1), (20480, 3, 64, 4),
                                (2560, 70, 256, 2)):
        e = torch.linspace(lo, hi, n).round()
        if order == "down":
            e = e.flip(0)
        elif order == "mixed":
            e = e[torch.randperm(n, generator=torch.Generator().manual_seed(1))]
        elif order == "steps":
            e = torch.where(torch.arange(n) // 300 % 2 == 0, float(lo),
                            float(hi))
        s = torch.exp2(e.double())
        for lean in (0.0, -0.9, -1.1):
            C = Scaled(n, seqs, heads, 2, dim, store, s, lean * math.log(2) * e)
            check_far(C, *C.run(scale=1.0), scale=1.0)


@pytest.mark.parametrize("store", CODES)
@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 30, 2.0 ** 60])
def test_value_scales_over_many_bands_under_large_scores(store, size):
    """Equal scores of any size, scales that change by 2^70 every 300 tokens: the
    mean of the values, within 2^-11 of each for its weight and as much for the
    rest, and 2^-32 of the largest a key."""
    n = 20480
    e = torch.where(torch.arange(n) // 300 % 2 == 0, -40.0, 30.0)
    C = Scaled(n, 3, 4, 2, 64, store, torch.exp2(e.double()),
               torch.full((n,), size))
    # (of one sign, so that nothing averages out)
    C.P.held[1] = C.P.held[1] & 127
    rescale(C, 1, lambda s: s)
    most = {"e4m3": 448.0, "int8": 128.0}[store]
    for sign in (1.0, -1.0):
        out, lse = C.run(scale=sign)
        assert lse.isfinite().all()
        v = C.rows(0)[1]
        want, mag = (x.mean(0).repeat_interleave(2, 0) for x in (v, v.abs()))
        bound = 2.0 ** -10 * mag + 2.0 ** -32 * most * 2.0 ** 30 \
            + want.abs() * kr.ROUND[BF] * 1.01
        assert ((out.double() - want).abs() <= bound).all()


def stepping(store, dtype, n, heads, seqs, wide):
    """Held keys of two elements, the first a large constant and the second
    larger by one in every `wide` keys of eight times as many, and queries (a,
    1) with a such that scores in units of ln 2 run from 2^24 to 2^26."""
    P = lr.Held([n] + [0] * seqs, heads, 64, 16, "nhd", dtype, store, seed=3)
    x = torch.zeros(P.pool, 16, heads, 64, device="cuda")
    ids = P.table[0, :n // 16].long().cuda()
    step = (torch.arange(n, device="cuda") // wide % 8).view(-1, 16, 1)
    top = 4096.0 if store is None else 64.0
    x[ids, :, :, 0], x[ids, :, :, 1] = top, step.float()
    P.rows[0] = x.double()
    if store is None:
        P.held[0] = x.to(dtype)
    else:
        if store == "int8":
            P.held[0] = x.to(torch.int8)
        else:
            table = lr.e4m3_values().cuda()[:127]
            P.held[0] = torch.searchsorted(table.float(), x.contiguous()).to(
                torch.uint8)
        P.scales[0].fill_(1)
    a = 2.0 ** (24 + 2 * torch.arange(seqs, device="cuda") / seqs)
    q = torch.zeros(seqs, 1, 64, dtype=dtype, device="cuda")
    q[..., 0] = (a / top * math.log(2))[:, None].to(dtype)
    q[..., 1] = 1
    return P, q


@pytest.mark.parametrize("store,dtype", [(None, HF), (None, BF),
                                         ("e4m3", BF), ("int8", BF)], ids=str)
def test_scores_that_grow_by_little_far_from_zero(store, dtype):
    """Scores of 2^24 to 2^26, where a number of 32 bits is 2 or 4 from the
    next, that grow by as much from tile to tile of a block: every result is a
    mean of the values, within the rounding of a weight (2^-8) and its own."""
    n, heads, seqs = 40960, 2, 40
    P, q = stepping(store, dtype, n, heads, seqs, 128)
    cache, plan = P.cache(lm)
    q = q.expand(seqs, heads, 64).contiguous()
    t = P.table.cuda()
    out, lse = torch.empty_like(q), torch.empty(seqs, heads, device="cuda")
    lm.kv_attend_shared(
        cache, q, t[:1], ints([n]), ints([0, seqs]), t[1:], ints([0] * seqs),
        out, space(lm.kv_attend_shared_workspace(plan, seqs, heads)), lse=lse,
        scale=1.0)
    v = P.seq(1, 0)
    assert lse.isfinite().all()
    most = v.abs().amax(0)
    assert (out.double().abs() <= most * (1 + 2.0 ** -6)).all()


def check_far_scores(C, size):
    """Keys of C's first prefix get one score, `size` in units of ln 2, or one
    that is lower by 2^-19 of it or by a half, whichever is more; the values'
    scales differ from key to key.  Own tokens: none.  See
    test_equal_scores_far_from_zero for the bound."""
    n, store, dtype, heads = C.shared[0], C.store, C.dtype, C.heads
    pages = -(-n // 16)
    ids = C.P.table[0, :pages].long().cuda()
    g = torch.Generator(device="cuda").manual_seed(9)
    lower = torch.randint(0, 2, (pages, 16, heads), generator=g,
                          device="cuda").bool()
    x = torch.zeros(C.P.pool, 16, heads, C.dim, dtype=torch.float64,
                    device="cuda")
    x[ids, :, :, 0] = 1
    x[ids, :, :, 1] = torch.where(lower, -1.0, 0.0).double()
    C.P.rows[0] = x
    one, minus = {None: (1, -1), "e4m3": (0x38, 0xb8), "int8": (1, -1)}[store]
    held = torch.zeros(x.shape, dtype=torch.int64, device="cuda")
    held[x > 0], held[x < 0] = one, minus
    if C.P.order == "hnd":
        held = held.transpose(1, 2)
    C.P.held[0] = held.to(C.P.held[0].dtype).contiguous()
    if store is not None:
        C.P.scales[0].fill_(1)
    gap = max(0.5, abs(size) * 2.0 ** -19)
    C.q.zero_()
    C.q[..., 0] = 2.0 ** 9
    C.q[..., 1] = 2.0 ** round(math.log2(gap / abs(size) * 2.0 ** 9))
    scale = torch.tensor(size * math.log(2) / 2 ** 9).item()
    out, lse = C.run(scale=scale)
    half = store is not None or dtype == HF
    step = 2.0 ** -11 if half else 2.0 ** -8
    for b in {0, len(C.lens) // 2, len(C.lens) - 1}:
        k, v = C.rows(b)
        want, wl, p, mag, _ = lr.attend(C.q[b].double(), k, v, C.group, scale)
        bo = (step + 2.0 ** -13) * mag + want.abs() * kr.ROUND[dtype] * 1.01
        if half:
            bo += len(v) * 2.0 ** -35 * v.abs().max()
        assert ((out[b].double() - want).abs() <= bo).all()
        assert ((lse[b].double() - wl).abs() <=
                2.0 ** -14 + wl.abs() * 2.0 ** -22).all()


@pytest.mark.parametrize("store,dtype", [(None, BF), (None, HF), ("e4m3", BF),
                                         ("int8", HF)], ids=str)
@pytest.mark.parametrize("size", [8.0, 900.0, 2.0 ** 12, 2.0 ** 16, 2.0 ** 20,
                                  2.0 ** 25])
@pytest.mark.parametrize("n,heads", [(384, 1), (20480, 4)])
def test_equal_scores_far_from_zero(store, dtype, size, n, heads):
    """Keys of one score, `size` in units of ln 2, and of one that is lower by
    2^-19 of it or by a half, whichever is more, in one block and in many; the
    values' scales differ from key to key.  However far the scores lie from 0,
    weights are what their differences say.  Those are whole numbers of steps of
    32 bits here, and good to 2^-22 of themselves, 2^-17 of 64 at most and so a
    weight to 2^-17.  It is rounded to 11 bits (8 of bfloat16 rows); 2^-13
    covers that of a logarithm beside a reference of up to 2^10, 2^-15, the
    exponentials and the sums."""
    seqs = 3
    check_far_scores(Case([n], [0, seqs], [0] * seqs, heads, 2, 64, 16, "nhd",
                          dtype, store, seed=5), size)


@pytest.mark.parametrize("store,dtype", [(None, BF), (None, HF), ("e4m3", BF),
                                         ("int8", HF)], ids=str)
@pytest.mark.parametrize("dim", [80, 128, 256])
@pytest.mark.parametrize("seqs,group", [(3, 5), (50, 2), (70, 4)])
def test_scores_far_from_zero_of_every_shape(store, dtype, dim, seqs, group):
    """The same for rows of every length, in one tile of rows, in halves of one
    or in several, with a last tile of keys that is not full, and below 0."""
    for n, size in ((700, 2.0 ** 20), (3001, -2.0 ** 14)):
        check_far_scores(Case([n], [0, seqs], [0] * seqs, 2, group, dim, 16,
                              "hnd" if dim == 128 else "nhd", dtype, store,
                              seed=5), size)


@pytest.mark.parametrize("size", [1.0, 2.0 ** 19, 2.0 ** 24, 2.0 ** 27,
                                  2.0 ** 30, 2.0 ** 60])
def test_large_values_under_scores_far_from_zero(size):
    """Values near the top of bfloat16 behind a prefix, under equal scores of
    any size: their mean, within 2^-8 of the values for a weight's rounding."""
    n, seqs = 9000, 40
    top = 2.0 ** 127 * 1.5
    C = Case([n], [0, seqs], [3] * seqs, 1, 2, 64, 16, "nhd", BF, None)
    live = ~C.P.held[0].isnan()
    one = torch.zeros_like(C.P.held[0])
    one[..., 0] = 1
    C.P.held[0] = torch.where(live, one, math.nan)
    C.P.held[1] = torch.where(live, C.P.held[1].sign() * top, math.nan)
    C.P.rows = [x.double() for x in C.P.held]
    C.q.zero_()
    C.q[..., 0] = 1
    for sign in (1, -1):
        out, lse = C.run(scale=sign * size)
        assert out.isfinite().all() and lse.isfinite().all()
        for b in (0, 17, 39):
            want = C.rows(b)[1].mean(0)
            bound = top * (2.0 ** -8 + 2.0 ** -13) + want.abs() * 2.0 ** -8
            assert ((out[b].double() - want).abs() <= bound).all()
