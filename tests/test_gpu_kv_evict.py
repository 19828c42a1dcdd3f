"""The accumulated weights of an attention and the eviction by them, on the GPU
against the definitions in kv_long_reference."""

import math

import pytest

import kv_long_reference as lr
import kv_reference as kr

torch = pytest.importorskip("torch")
lm = pytest.importorskip("layout_driven_movement_gb300")

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    from layout_driven_movement_gb300 import _build
    _build.build()
    lm.lib()


@pytest.fixture(autouse=True)
def clean_status():
    lm.device_status(reset=True)
    yield
    assert lm.device_status(reset=True) == 0


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def space(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def weights_of(P, seed=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(P.pool, P.heads, P.page, generator=g, device="cuda")


def run_weigh(P, q, weights, window=0, workspace=None, table=None):
    cache, plan = P.cache(lm)
    b, hq = q.shape[:2]
    table = P.table if table is None else table
    if workspace is None:
        workspace = space(lm.kv_attend_workspace(plan, b, hq,
                                                 max_pages=table.shape[-1]))
    out, lse = torch.full_like(q, math.nan), torch.empty(b, hq, device="cuda")
    lm.kv_attend(cache, q, table.cuda(), ints(P.lens), out, workspace,
                 lse=lse, weights=weights, window=window)
    return out, lse


def check_weigh(P, q, group, out, lse, before, after, window=0):
    """A weight's score is off by e (as in kv_reference), its sum over the
    group by as much, its exponential and the sums' logarithm by 2^-18 more;
    the addition rounds once."""
    scale = P.dim ** -0.5
    want = before.double()
    room = torch.zeros_like(want)
    for b, n in enumerate(P.lens):
        lo = max(0, n - window) if window else 0
        k, v = (P.seq(kv, b)[lo:] for kv in (0, 1))
        o, wl, p, mag, dot = lr.attend(q[b].double(), k, v, group, scale)
        bo, bl = kr.attend_bounds(P.dtype, P.dim, o, wl, mag, dot)
        assert ((out[b].double() - o).abs() <= bo).all(), b
        if n == 0:
            assert (lse[b] == -math.inf).all()
            continue
        assert ((lse[b].double() - wl).abs() <= bl).all()
        e = (P.dim + 4) * 2.0 ** -24 * dot
        part = p.view(P.heads, group, -1).sum(1)
        err = (p * (4 * e + 2.0 ** -18)[:, None]).view(
            P.heads, group, -1).sum(1)
        j = torch.arange(lo, n)
        page = P.table[b].long()[j // P.page].cuda()
        want[page, :, (j % P.page).cuda()] += part.T
        room[page, :, (j % P.page).cuda()] += err.T + 2.0 ** -24 * part.T
    room += want.abs() * 2.0 ** -23
    assert ((after.double() - want).abs() <= room).all()


CASES = [
    # lens, heads, group, dim, page, order, dtype, store
    ([0, 1, 130, 33, 500], 2, 4, 128, 16, "nhd", BF, None),
    ([5, 0, 300, 1000], 3, 5, 80, 24, "hnd", HF, "int8"),
    ([64, 2, 700], 1, 16, 256, 5, "nhd", BF, "e4m3"),
    ([40, 0, 129], 4, 1, 64, 16, "nhd", HF, None),
    ([40, 0, 129], 2, 20, 64, 1, "nhd", BF, "int8"),
    ([3000, 1, 90], 2, 8, 128, 64, "hnd", BF, "e4m3"),
    ([257], 1, 9, 256, 128, "nhd", HF, None),
    ([10000, 1, 1, 0, 3], 2, 3, 112, 20, "nhd", BF, None),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_weights_add_up(case):
    lens, heads, group, dim, page, order, dtype, store = case
    P = lr.Held(lens, heads, dim, page, order, dtype, store, seed=dim)
    g = torch.Generator().manual_seed(1)
    q = torch.randn(len(lens), heads * group, dim, generator=g).to(
        dtype).cuda()
    for window in (0, 17):
        before = weights_of(P)
        w = before.clone()
        out, lse = run_weigh(P, q, w, window)
        check_weigh(P, q, group, out, lse, before, w, window)
        # what no token names stays as it is, and the outputs are those of a
        # call without weights
        plain = torch.full_like(q, math.nan)
        cache, plan = P.cache(lm)
        ws = space(lm.kv_attend_workspace(plan, *q.shape[:2]))
        lm.kv_attend(cache, q, P.table.cuda(), ints(lens), plain, ws,
                     window=window)
        assert torch.equal(plain, out)


def test_weights_of_pages_that_sequences_share():
    """Two sequences of the same pages: both add.  The order of two additions
    to one number changes its last bit at most."""
    P = lr.Held([100, 100], 2, 64, 16, "nhd", BF, None, seed=3)
    P.table[1] = P.table[0]
    g = torch.Generator().manual_seed(1)
    q = torch.randn(2, 4, 64, generator=g).to(BF).cuda()
    w = torch.zeros(P.pool, 2, 16, device="cuda")
    run_weigh(P, q, w)
    want = torch.zeros(2, 100, dtype=torch.float64, device="cuda")
    for b in (0, 1):
        _, _, p, _, _ = lr.attend(q[b].double(), P.seq(0, b), P.seq(1, b), 2,
                                  64 ** -0.5)
        want += p.view(2, 2, -1).sum(1)
    ids = P.table[0].long().cuda()
    got = w[ids].transpose(0, 1).flatten(1)[:, :100]
    assert ((got.double() - want).abs() <= want * 2.0 ** -16).all()
    assert w.double().sum().item() == pytest.approx(8, abs=1e-4)


def test_weights_of_scores_at_the_ends():
    """All scores -infinity add nothing; a NaN score makes its head's weights
    NaN; a page out of range has none."""
    P = lr.Held([40, 40, 48], 1, 64, 16, "nhd", BF, None, seed=3)
    q = torch.ones(3, 1, 64, dtype=BF, device="cuda")
    rows = P.held[0].view(-1, 64)
    ids = P.table.long()
    for j in range(40):
        rows[ids[0, j // 16] * 16 + j % 16] = 0
        rows[ids[0, j // 16] * 16 + j % 16, 0] = -math.inf
    rows[ids[1, 1] * 16 + 3, 7] = math.nan
    table = P.table.clone()
    table[2, 1] = P.pool
    w = torch.zeros(P.pool, 1, 16, device="cuda")
    out, lse = run_weigh(P, q, w, table=table)
    assert lm.device_status(reset=True) == -12
    assert (lse[0] == -math.inf).all() and (out[0] == 0).all()
    assert (w[ids[0].cuda()] == 0).all()
    assert w[ids[1].cuda()].flatten()[:40].isnan().all()
    assert (w[ids[1].cuda()].flatten()[40:] == 0).all()
    assert w[ids[2, [0, 2]].cuda()].sum().item() == pytest.approx(1, abs=1e-5)
    assert (w[ids[2, 1].cuda()] == 0).all()


@pytest.mark.parametrize("dtype,store", [(BF, None), (HF, None), (BF, "e4m3"),
                                         (HF, "int8")], ids=str)
@pytest.mark.parametrize("size", [1.0, 2.0 ** 16, 2.0 ** 20, 2.0 ** 24,
                                  2.0 ** 25])
def test_weights_of_equal_scores_of_any_size(dtype, store, size):
    """n keys of one score, up to 2^25 about: each has a weight of 1 / n of
    every query.  The score is one product, so equal in all bits; 2^0 is 1, the
    sum is within n 2^-24 (of 2^10 keys at most in runs of a warp's 2^7, so
    2^-16 covers it), and the group's four add up within 2^-22."""
    lens = [1, 3, 40, 700]
    P = lr.Held(lens, 2, 64, 16, "nhd", dtype, store, seed=3)
    P.held[0].zero_()
    P.held[0][..., 0] = {None: 1, "e4m3": 0x38, "int8": 1}[store]
    if store is not None:
        P.scales[0].fill_(1)
    q = torch.zeros(4, 8, 64, dtype=dtype, device="cuda")
    q[:, :, 0] = 1 + torch.arange(8, device="cuda") / 8
    cache, plan = P.cache(lm)
    for sign in (1, -1):
        w = torch.zeros(P.pool, 2, 16, device="cuda")
        ws = space(lm.kv_attend_workspace(plan, 4, 8,
                                          max_pages=P.table.shape[1]))
        lm.kv_attend(cache, q, P.table.cuda(), ints(lens),
                     torch.empty_like(q), ws, weights=w, scale=sign * size)
        for b, n in enumerate(lens):
            ids = P.table[b, :-(-n // 16)].long().cuda()
            got = w[ids].transpose(0, 1).flatten(1).double()
            assert ((got[:, :n] - 4 / n).abs() <= 2.0 ** -15 / n).all()
            assert (got[:, n:] == 0).all()


# --- eviction --------------------------------------------------------------

def expected(P, weights, keep, recent):
    """Per sequence and head the tokens that stay, in order."""
    out = []
    for b, n in enumerate(P.lens):
        ids = P.table[b, :-(-n // P.page)].long().cuda()
        w = weights[ids].transpose(0, 1).flatten(1)[:, :n].cpu().tolist()
        rows = []
        for h in range(P.heads):
            if n <= keep:
                rows.append(list(range(n)))
                continue
            old = lr.choose(w[h][:n - recent] + [0.0], keep - recent + 1, 0, 1)
            rows.append(old[:-1] + list(range(n - recent, n)))
        out.append(rows)
    return out


def check_evict(P, before, held, weights, scales, kept_table, keep, recent,
                kept_lens, untouched=None):
    """`before`: (held, weights, scales) as they were."""
    want = expected(P, before[1], keep, recent)
    tok = (lambda x: x.transpose(1, 2) if P.order == "hnd" else x)
    flat = (lambda x: x.view(torch.uint8) if x.element_size() == 1
            else x.view(torch.int16))
    assert kept_lens.tolist() == [min(n, keep) for n in P.lens]
    hold = [flat(x.clone()) for x in before[0]]
    hw = before[1].clone().view(torch.int32)
    hs = [None if s is None else s.clone().view(torch.int32)
          for s in before[2]]
    for b, n in enumerate(P.lens):
        for h in range(P.heads):
            j = torch.tensor(want[b][h], dtype=torch.long)
            i = torch.arange(len(j))
            sp, so = P.table[b].long()[j // P.page].cuda(), \
                (j % P.page).cuda()
            dp, do = kept_table[b].long().cpu()[i // P.page].cuda(), \
                (i % P.page).cuda()
            for kv in (0, 1):
                tok(hold[kv])[dp, do, h] = tok(flat(before[0][kv]))[sp, so, h]
                if hs[kv] is not None:
                    hs[kv][dp, h, do] = before[2][kv].view(
                        torch.int32)[sp, h, so]
            hw[dp, h, do] = before[1].view(torch.int32)[sp, h, so]
    for kv in (0, 1):
        assert torch.equal(flat(held[kv]), hold[kv])
        if hs[kv] is not None:
            assert torch.equal(scales[kv].view(torch.int32), hs[kv])
    assert torch.equal(weights.view(torch.int32), hw)


EVICT = [
    # lens, heads, dim, page, order, dtype, store, keep, recent
    ([0, 1, 100, 33, 64, 65], 2, 128, 16, "nhd", BF, None, 64, 10),
    ([200, 5, 0, 1000, 129], 3, 80, 24, "hnd", HF, "int8", 128, 0),
    ([300, 2, 77], 1, 256, 5, "nhd", BF, "e4m3", 1, 1),
    ([300, 2, 77], 2, 256, 7, "nhd", BF, None, 76, 76),
    ([3000, 1, 2000], 2, 64, 128, "hnd", HF, "int8", 1999, 100),
    ([12000, 20000], 1, 16, 32, "nhd", BF, None, 700, 5),
    ([500, 400, 300], 5, 72, 1, "nhd", BF, None, 350, 1),
]


@pytest.mark.parametrize("case", EVICT, ids=str)
@pytest.mark.parametrize("in_place", [True, False])
def test_eviction_keeps_the_heaviest(case, in_place):
    lens, heads, dim, page, order, dtype, store, keep, recent = case
    most = -(-min(keep, max(lens)) // page)
    P = lr.Held(lens, heads, dim, page, order, dtype, store, seed=dim,
                spare=2 + len(lens) * most)
    cache, plan = P.cache(lm)
    w = weights_of(P)
    w[w < 0.3] = 0.25                     # many equal ones
    before = ([x.clone() for x in P.held], w.clone(),
              [None if s is None else s.clone() for s in P.scales])
    table = P.table.cuda()
    ws = space(lm.kv_evict_workspace(plan, len(lens), keep))
    ws.fill_(0x7f)
    if in_place:
        kept, ln = table, ints(lens)
        kept_lens = ln
    else:
        kept = P.spare[:len(lens) * most].int().view(len(lens), most).cuda()
        ln, kept_lens = ints(lens), torch.full((len(lens),), 7,
                                               dtype=torch.int32,
                                               device="cuda")
    lm.kv_evict(cache, w, table, ln, kept, kept_lens, keep, ws,
                recent=recent)
    check_evict(P, before, P.held, w, P.scales, kept, keep, recent,
                kept_lens)


@pytest.mark.parametrize("n,keep", [(100000, 30000), (70000, 69999),
                                    (70001, 1)])
def test_eviction_of_long_sequences(n, keep):
    """More tokens than a block's memory holds, in place."""
    P = lr.Held([n], 2, 16, 16, "nhd", BF, None, seed=1)
    cache, plan = P.cache(lm)
    w = weights_of(P)
    w = (w * 50).floor() / 50 if keep < n - 1 else w
    before = ([x.clone() for x in P.held], w.clone(), [None, None])
    kept_lens = ints([0])
    ws = space(lm.kv_evict_workspace(plan, 1, keep))
    table = P.table.cuda()
    lm.kv_evict(cache, w, table, ints([n]), table, kept_lens, keep, ws)
    check_evict(P, before, P.held, w, P.scales, table, keep, 0, kept_lens)


def test_eviction_of_infinite_weights_and_no_numbers():
    P = lr.Held([20], 1, 16, 4, "nhd", BF, None, seed=1)
    cache, plan = P.cache(lm)
    table = P.table.cuda()
    w = torch.zeros(P.pool, 1, 4, device="cuda")
    flat = torch.tensor([0.0, -0.0, 1, -math.inf, math.inf, math.nan, -1, 0.0,
                         -math.nan, 1e-45] + [-2.0] * 10)
    w[P.table[0].long().cuda(), 0] = flat.view(5, 4).cuda()
    before = ([x.clone() for x in P.held], w.clone(), [None, None])
    want = [0, 1, 2, 4, 5, 8, 9]
    kept_lens = ints([0])
    ws = space(lm.kv_evict_workspace(plan, 1, 7))
    lm.kv_evict(cache, w, table, ints([20]), table, kept_lens, 7, ws)
    rows = before[0][0][P.table[0].long().cuda()].view(20, 16)[want]
    got = P.held[0][P.table[0].long().cuda()].view(20, 16)[:7]
    assert torch.equal(got, rows)
    assert kept_lens.item() == 7


def test_eviction_pages_and_lengths_out_of_range():
    P = lr.Held([40, 40, 40], 1, 16, 8, "nhd", BF, None, seed=1)
    cache, plan = P.cache(lm)
    table = P.table.clone()
    table[1, 2] = P.pool
    kept_lens = ints([9, 9, 9])
    w = weights_of(P)
    ws = space(lm.kv_evict_workspace(plan, 3, 32))
    t = table.cuda()
    lm.kv_evict(cache, w, t, ints([-3, 40, 1 << 30]), t, kept_lens, 32, ws)
    # 32 of the 40 lie in pages that are there; the places of page 2 do not
    assert lm.device_status(reset=True) == -12
    assert kept_lens.tolist() == [0, 32, 32]
    # nothing of no sequences, and of tables without pages
    lm.kv_evict(cache, w, t[:0], ints([]), t[:0], ints([]), 32, ws)
    lm.kv_evict(cache, w, t[:, :0], ints([4, 5, 6]), t[:, :0], kept_lens, 32,
                ws)
    assert kept_lens.tolist() == [0, 0, 0]


def test_steps_of_weighing_and_eviction():
    """Decoding steps that weigh, with an eviction when the cache is full: the
    attention after it is that over the rows that stayed, each head's own."""
    lens, heads, group, dim, page = [70, 90, 10], 2, 3, 64, 8
    P = lr.Held(lens, heads, dim, page, "nhd", BF, None, seed=6)
    cache, plan = P.cache(lm)
    g = torch.Generator().manual_seed(1)
    table, ln = P.table.cuda(), ints(lens)
    w = torch.zeros(P.pool, heads, page, device="cuda")
    ws = space(lm.kv_attend_workspace(plan, 3, 6, max_pages=P.most))
    es = space(lm.kv_evict_workspace(plan, 3, 48))
    q = torch.randn(3, 6, dim, generator=g).to(BF).cuda()
    out = torch.empty_like(q)
    lm.kv_attend(cache, q, table, ln, out, ws, weights=w)
    rows = [[P.seq(kv, b).clone() for kv in (0, 1)] for b in range(3)]
    stay = expected(P, w, 48, 4)
    lm.kv_evict(cache, w, table, ln, table, ln, 48, es, recent=4)
    lm.kv_attend(cache, q, table, ln, out, ws, weights=w)
    assert ln.tolist() == [48, 48, 10]
    for b in range(3):
        for h in range(heads):
            part = slice(h * group, (h + 1) * group)
            k, v = (x[stay[b][h]][:, h:h + 1] for x in rows[b])
            want, wl, _, mag, dot = lr.attend(q[b, part].double(), k, v,
                                              group, dim ** -0.5)
            bo, _ = kr.attend_bounds(BF, dim, want, wl, mag, dot)
            assert ((out[b, part].double() - want).abs() <= bo).all()
