"""The bounds of a cache's pages, the choice of pages by them and the attention
over pages of each head's own, on the GPU against the definitions in
kv_long_reference.  Bounds and choices are whole numbers and have to be the
definition's; the attention's bound is kv_reference's."""

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


def page_counts(P):
    """Every page that the sequences name, and how many tokens it holds."""
    pages, counts = [], []
    for b, n in enumerate(P.lens):
        for i in range(-(-n // P.page)):
            pages.append(int(P.table[b, i]))
            counts.append(min(P.page, n - i * P.page))
    return pages, counts


def make_bounds(P, cache):
    bounds = torch.full((P.pool, P.heads, 2, P.dim), 55, dtype=torch.int8,
                        device="cuda")
    scale = torch.full((P.pool, P.heads), 9.0, device="cuda")
    pages, counts = page_counts(P)
    lm.kv_bound(cache, ints(pages), ints(counts), bounds, scale)
    return bounds, scale


def check_bounds(P, bounds, scale, pages, counts):
    x = P.values32()
    for p, n in zip(pages, counts):
        for h in range(P.heads):
            lo, hi, by = lr.bounds(x[p, :n, h])
            assert torch.equal(bounds[p, h, 0].cpu().float(), lo.float())
            assert torch.equal(bounds[p, h, 1].cpu().float(), hi.float())
            assert scale[p, h].item() == by


SHAPES = [
    # heads, group, dim, page, order, dtype, store
    (2, 4, 128, 16, "nhd", BF, None), (3, 1, 64, 5, "hnd", HF, "int8"),
    (1, 8, 256, 24, "nhd", BF, "e4m3"), (2, 5, 80, 1, "nhd", HF, "e4m3"),
    (1, 16, 72, 40, "hnd", HF, None), (4, 2, 112, 64, "hnd", BF, "int8"),
    (5, 9, 8, 7, "nhd", BF, None), (1, 3, 16, 128, "nhd", HF, "int8"),
]


@pytest.mark.parametrize("case", SHAPES, ids=str)
def test_bounds_are_the_definition(case):
    heads, group, dim, page, order, dtype, store = case
    P = lr.Held([0, 1, 3 * page, 2 * page + page // 2, 40], heads, dim, page,
                order, dtype, store, seed=dim)
    cache, plan = P.cache(lm)
    bounds, scale = make_bounds(P, cache)
    pages, counts = page_counts(P)
    check_bounds(P, bounds, scale, pages, counts)
    # the pages that nothing names are as they were
    left = [p for p in range(P.pool) if p not in pages]
    assert (bounds[left] == 55).all() and (scale[left] == 9).all()
    # a page's first tokens, none of them, and pages that are not looked at
    some = pages[:2] + [-1]
    lm.kv_bound(cache, ints(some), ints([0, 1, 5]), bounds, scale)
    check_bounds(P, bounds, scale, some[:2], [0, 1])
    lm.kv_bound(cache, ints(some[:1]), ints([-4]), bounds, scale)
    check_bounds(P, bounds, scale, some[:1], [0])


def test_bounds_of_values_at_the_ends():
    """Powers of two's edges: 127 and the next value above it, the smallest
    and largest numbers, zeros, and keys that are no number."""
    page, dim = 4, 16
    P = lr.Held([page * 9], 1, dim, page, "nhd", BF, None, spare=0)
    top = torch.tensor([127.0, 127.5, 128.0, 63.5, 3.3e38, 1e-40, 0.0,
                        math.inf, math.nan])
    ids = P.table[0].long().cuda()
    x = torch.zeros(9, page, 1, dim)
    x[:, 1, 0, 3] = top
    x[:, 2, 0, 5] = -top / 3
    P.held[0][ids] = x.to(BF).cuda()
    P.rows[0][ids] = x.to(BF).double().cuda()
    cache, plan = P.cache(lm)
    bounds, scale = make_bounds(P, cache)
    pages, counts = page_counts(P)
    x = P.values32()
    for i, (p, n) in enumerate(zip(pages, counts)):
        lo, hi, by = lr.bounds(x[p, :n, 0])
        assert torch.equal(bounds[p, 0, 0].cpu().float(), lo.float())
        assert torch.equal(bounds[p, 0, 1].cpu().float(), hi.float())
        got = scale[p, 0].item()
        assert got == by or (math.isnan(got) and math.isnan(by)), i


@pytest.mark.parametrize("store,dtype", [(None, BF), ("e4m3", BF),
                                         ("int8", HF)], ids=str)
def test_bounds_over_a_wide_range(store, dtype):
    """Keys far smaller than the page's largest, of either sign: a quotient
    that 32 bits do not hold is still below or above 0."""
    page, dim = 4, 16
    P = lr.Held([page * 3], 1, dim, page, "nhd", dtype, store, spare=0)
    ids = P.table[0].long().cuda()
    x = torch.zeros(3, page, 1, dim, dtype=torch.float64)
    big = torch.tensor([2.0 ** 100, 2.0 ** 30, 1.0])
    small = torch.tensor([2.0 ** -60, 2.0 ** -126, 2.0 ** -126])
    # alone in their columns, beside zeros, and beside a small one of the
    # other sign
    for d, s in ((1, 1), (2, -1)):
        x[:, 2, 0, d] = s * small
    x[:, 1, 0, 3], x[:, 2, 0, 3] = small, -small
    x[:, :, 0, 4], x[:, :, 0, 5] = small[:, None], -small[:, None]
    x[:, 0, 0, 0] = big
    if store is None:
        P.held[0][ids] = x.to(dtype).cuda()
    else:
        # one power of two a token: codes of 1 and -1 under its scale
        one = {"e4m3": (0x38, 0xb8), "int8": (1, -1)}[store]
        code = torch.zeros(x.shape, dtype=torch.int64)
        code[x > 0], code[x < 0] = one
        P.held[0][ids] = code.to(P.held[0].dtype).cuda()
        scale = x.abs().amax((-2, -1))
        scale[scale == 0] = 1
        P.scales[0][ids, 0] = scale.float().cuda()
        x = x.sign() * scale[..., None, None]
    P.rows[0][ids] = x.cuda()
    cache, plan = P.cache(lm)
    bounds, scale = make_bounds(P, cache)
    assert (bounds[ids, 0, :, 0] == torch.tensor([0, 64]).cuda()).all()
    check_bounds(P, bounds, scale, *page_counts(P))
    assert (bounds[ids[:2], 0, :, 3] == torch.tensor([-1, 1]).cuda()).all()


def test_bounds_page_out_of_range():
    P = lr.Held([8], 1, 16, 4, "nhd", BF, None)
    cache, plan = P.cache(lm)
    bounds, scale = make_bounds(P, cache)
    before = bounds.clone()
    lm.kv_bound(cache, ints([P.pool, 1 << 30]), ints([4, 4]), bounds, scale)
    assert lm.device_status(reset=True) == -12
    assert torch.equal(before, bounds)


def run_select(P, cache, q, keep, first, last, bounds, scale, lens=None,
               table=None, workspace=None):
    b = len(P.lens)
    selected = torch.full((b, P.heads, keep), 77, dtype=torch.int32,
                          device="cuda")
    out = torch.full((b,), 77, dtype=torch.int32, device="cuda")
    table = P.table if table is None else table
    if workspace is None:
        workspace = space(lm.kv_select_workspace(cache.plan, b,
                                                 table.shape[1]))
        workspace.fill_(0x7f)
    lm.kv_select(cache, q, bounds, scale, table.cuda(),
                 ints(P.lens if lens is None else lens), selected, out,
                 workspace, first=first, last=last)
    return selected, out


def check_select(P, q, keep, first, last, bounds, scale, selected, lens,
                 group):
    bounds, scale = bounds.cpu(), scale.cpu()
    for b, n in enumerate(P.lens):
        m = -(-n // P.page)
        ids = P.table[b, :m].long()
        s = lr.scores(q[b], bounds[ids, :, 0], bounds[ids, :, 1], scale[ids],
                      group)
        for h in range(P.heads):
            want = lr.choose(s[h].tolist(), keep, first, last)
            got = selected[b, h].cpu()
            assert got[:len(want)].tolist() == ids[want].tolist(), (b, h)
            assert (got[len(want):] == -1).all()
        assert lens[b].item() == n - max(0, m - keep) * P.page


@pytest.mark.parametrize("case", SHAPES, ids=str)
@pytest.mark.parametrize("keep,first,last", [(1, 0, 1), (6, 1, 1), (9, 0, 2),
                                             (7, 3, 4)])
def test_choice_and_attention_over_it(case, keep, first, last):
    heads, group, dim, page, order, dtype, store = case
    lens = [0, 1, page * 5, page * 40 - page // 2, page * 33 + 1, page * 7]
    P = lr.Held(lens, heads, dim, page, order, dtype, store, seed=dim + keep,
                drift=1.0)
    cache, plan = P.cache(lm)
    bounds, scale = make_bounds(P, cache)
    g = torch.Generator().manual_seed(keep)
    b, hq = len(lens), heads * group
    wide = torch.randn(b, hq + 1, dim + 8, generator=g).to(dtype).cuda()
    # an aligned slice and one that allows no wide loads
    q = wide[:, :hq, :dim] if keep != 6 else wide[:, 1:, 3:dim + 3]
    selected, sl = run_select(P, cache, q, keep, first, last, bounds, scale)
    check_select(P, q, keep, first, last, bounds, scale, selected, sl, group)
    out, lse = torch.full_like(q, math.nan), torch.empty(b, hq, device="cuda")
    ws = space(lm.kv_attend_workspace(plan, b, hq))
    lm.kv_attend(cache, q, selected, sl, out, ws, lse=lse)
    for i in range(b):
        n = int(sl[i])
        for h in range(heads):
            rows = [P.of(kv, selected[i, h], n)[:, h:h + 1] for kv in (0, 1)]
            part = slice(h * group, (h + 1) * group)
            want, wl, _, mag, dot = lr.attend(q[i, part].double(), *rows,
                                              group, dim ** -0.5)
            bo, bl = kr.attend_bounds(dtype, dim, want, wl, mag, dot)
            assert ((out[i, part].double() - want).abs() <= bo).all()
            if n:
                assert ((lse[i, part].double() - wl).abs() <= bl).all()
            else:
                assert (lse[i, part] == -math.inf).all()


@pytest.mark.parametrize("pages,keep", [(20000, 700), (20000, 19999),
                                        (9000, 9000), (70000, 2048)])
def test_choice_of_many_pages(pages, keep):
    """More pages than a block's memory holds, most of their scores equal to
    others'."""
    page, heads, dim = 2, 2, 16
    P = lr.Held([pages * page - 1, 5], heads, dim, page, "nhd", BF, None,
                seed=4)
    g = torch.Generator(device="cuda").manual_seed(5)
    bounds = torch.randint(-3, 4, (P.pool, heads, 2, dim), generator=g,
                           device="cuda", dtype=torch.int8)
    scale = torch.exp2(torch.randint(-1, 2, (P.pool, heads), generator=g,
                                     device="cuda").float())
    cache, plan = P.cache(lm)
    q = torch.randn(2, heads * 2, dim, generator=g, device="cuda").to(BF)
    q[0, 2:] = q[0, 2:].sign()
    selected, sl = run_select(P, cache, q, keep, 1, 1, bounds, scale)
    check_select(P, q, keep, 1, 1, bounds, scale, selected, sl, 2)


def test_choice_of_equal_scores_and_of_no_numbers():
    """All scores equal: the first pages.  A page whose scale is NaN comes
    first of all, a NaN query makes all pages so."""
    page, heads, dim, n = 4, 1, 32, 50
    P = lr.Held([n * page], heads, dim, page, "nhd", BF, None, seed=4)
    cache, plan = P.cache(lm)
    bounds = torch.ones(P.pool, heads, 2, dim, dtype=torch.int8,
                        device="cuda")
    scale = torch.ones(P.pool, heads, device="cuda")
    q = torch.ones(1, 3, dim, dtype=BF, device="cuda")
    ids = P.table[0].tolist()

    def chosen(q):
        s, sl = run_select(P, cache, q, 5, 0, 1, bounds, scale)
        assert sl.item() == 5 * page
        return [ids.index(i) for i in s[0, 0].tolist()]
    assert chosen(q) == [0, 1, 2, 3, 49]
    scale[ids[20]] = math.nan
    assert chosen(q) == [0, 1, 2, 20, 49]
    bounds[ids[30]] = 7
    assert chosen(q) == [0, 1, 20, 30, 49]
    q[0, 1, 3] = math.inf
    assert chosen(q) == [0, 1, 2, 3, 49]
    q.zero_()
    assert chosen(q) == [0, 1, 2, 20, 49]
    # -0 is 0: products of either sign with bounds of 0
    scale.fill_(1)
    bounds.zero_()
    q.fill_(-1)
    assert chosen(q) == [0, 1, 2, 3, 49]


def test_choice_lengths_and_pages_out_of_range():
    page = 4
    P = lr.Held([40, 40, 40], 2, 16, page, "nhd", BF, None, seed=1)
    cache, plan = P.cache(lm)
    bounds, scale = make_bounds(P, cache)
    q = torch.randn(3, 2, 16, device="cuda").to(BF)
    selected, sl = run_select(P, cache, q, 3, 0, 1, bounds, scale,
                              lens=[-5, 1 << 30, 7])
    assert sl.tolist() == [0, 12, 7]
    assert (selected[0] == -1).all()
    assert selected[1, :, 2].tolist() == [int(P.table[1, 9])] * 2
    table = P.table.clone()
    table[1, 1:9] = torch.tensor([-1, P.pool, 1 << 30, -9, P.pool, P.pool,
                                  P.pool, -1])
    selected, sl = run_select(P, cache, q, 2, 0, 1, bounds, scale, table=table)
    assert lm.device_status(reset=True) == -12
    assert selected[1].tolist() == [[int(table[1, 0]), int(table[1, 9])]] * 2


def test_choice_into_the_longest_list():
    """A list of 2^31 - 1 entries, 9 of them chosen: the rest is -1 to the
    last, and nothing behind or before it is written to."""
    P = lr.Held([9 * 16 - 3], 1, 64, 16, "nhd", BF, None, seed=3)
    cache, plan = P.cache(lm)
    bounds, scale = make_bounds(P, cache)
    keep, room = 2 ** 31 - 1, 1 << 16
    buf = torch.full((keep + 2 * room,), 5, dtype=torch.int32, device="cuda")
    selected = buf[room:room + keep].view(1, 1, keep)
    lens = ints([0])
    q = torch.ones(1, 1, 64, dtype=BF, device="cuda")
    lm.kv_select(cache, q, bounds, scale, P.table.cuda(), ints(P.lens),
                 selected, lens, space(lm.kv_select_workspace(plan, 1, 9)))
    torch.cuda.synchronize()
    assert (buf[:room] == 5).all() and (buf[room + keep:] == 5).all()
    assert lens.item() == P.lens[0]
    assert torch.equal(selected[0, 0, :9], P.table[0].cuda())
    assert selected[0, 0, 9:].max().item() == -1
    assert selected[0, 0, 9:].min().item() == -1


def test_attention_with_a_table_a_head_and_a_window():
    """Heads of different pages, their rows in pairs in one block (the 8-bit
    forms of narrow rows), strides of any size, and a window."""
    for store, dim in ((None, 128), ("int8", 64), ("e4m3", 80)):
        P = lr.Held([130, 300, 64, 0], 4, dim, 16, "nhd", BF, store, seed=dim)
        cache, plan = P.cache(lm)
        g = torch.Generator().manual_seed(3)
        heads, group, b = 4, 2, 4
        wide = torch.full((b, heads + 2, P.most + 3), -3, dtype=torch.int32)
        for i, n in enumerate(P.lens):
            m = -(-n // 16)
            for h in range(heads):
                # the pages of the sequence but the last one in another order
                order = torch.cat([torch.randperm(max(m - 1, 0), generator=g),
                                   torch.arange(max(m - 1, 0), m)])
                wide[i, h, :m] = P.table[i, order]
        table = wide.cuda()[:, :heads, :P.most]
        q = torch.randn(b, heads * group, dim, generator=g).to(BF).cuda()
        for window in (0, 40):
            out = torch.full_like(q, math.nan)
            ws = space(lm.kv_attend_workspace(plan, b, heads * group))
            lm.kv_attend(cache, q, table, ints(P.lens), out, ws,
                         window=window)
            for i, n in enumerate(P.lens):
                lo = max(0, n - window) if window else 0
                for h in range(heads):
                    rows = [P.of(kv, wide[i, h], n)[lo:, h:h + 1]
                            for kv in (0, 1)]
                    part = slice(h * group, (h + 1) * group)
                    want, wl, _, mag, dot = lr.attend(
                        q[i, part].double(), *rows, group, dim ** -0.5)
                    bo, _ = kr.attend_bounds(BF, dim, want, wl, mag, dot)
                    assert ((out[i, part].double() - want).abs() <= bo).all()
