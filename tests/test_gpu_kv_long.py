"""The cache's operators for long contexts together, as a serving program uses
them: written step by step, bounded, chosen from, weighed, evicted, behind a
shared prefix; captured into graphs; over many sequences and groups; at offsets
past 32 bits.  Definitions and bounds are kv_long_reference's and
kv_reference's."""

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


def close(out, q, k, v, group, extra=0.0):
    """One sequence's outputs against the attention over its rows; `extra` is
    the rounding of a weight where attend_bounds has not got it.  Returns the
    weights [heads_q, n] and the bounds of their errors: a score's e, as in
    attend_bounds, in the weight and in the sum, and 2^-18 for the exponential
    and the sum's logarithm."""
    dim = q.shape[-1]
    want, lse, p, mag, dot = lr.attend(q.double(), k, v, group, dim ** -0.5)
    bound, _ = kr.attend_bounds(q.dtype, dim, want, lse, mag, dot)
    assert ((out.double() - want).abs() <= bound + extra * mag).all()
    e = (dim + 4) * 2.0 ** -24 * dot
    return p, p * (4 * e + 2.0 ** -18)[:, None]


def test_decoding_behind_a_shared_prefix():
    """A prefix written once, then steps that write each sequence's token to
    its own pages and attend over both."""
    heads, group, dim, page, seqs, steps = 2, 4, 64, 8, 5, 20
    g = torch.Generator(device="cuda").manual_seed(3)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(BF)
    plan = lm.KVPlan(lm.Layout.parse(f"({page},{heads},{dim}):"
                                     f"({heads * dim},{dim},1)"), BF)
    pool = 40
    kp = torch.full((pool, page, heads, dim), math.nan, dtype=BF,
                    device="cuda")
    vp = kp.clone()
    cache = lm.KVCache(plan, kp, vp)
    n = 83
    prefix = [randn(n, heads, dim) for _ in range(2)]
    shared = ints([list(range(11))])
    slots = torch.arange(n, device="cuda")
    lm.kv_write(cache, *prefix, slots)
    table = ints([[11 + 3 * b + i for i in range(3)] for b in range(seqs)])
    starts = ints([0, seqs])
    ws = space(lm.kv_attend_shared_workspace(plan, seqs, heads * group))
    rows = [[prefix[kv].double() for _ in range(seqs)] for kv in (0, 1)]
    for step in range(steps):
        k, v = randn(seqs, heads, dim), randn(seqs, heads, dim)
        at = table[:, step // page].long() * page + step % page
        lm.kv_write(cache, k, v, at)
        q = randn(seqs, heads * group, dim)
        out = torch.empty_like(q)
        lm.kv_attend_shared(cache, q, shared, ints([n]), starts, table,
                            ints([step + 1] * seqs), out, ws)
        for b in range(seqs):
            rows[0][b] = torch.cat([rows[0][b], k[b:b + 1].double()])
            rows[1][b] = torch.cat([rows[1][b], v[b:b + 1].double()])
            close(out[b], q[b], rows[0][b], rows[1][b], group, 2.0 ** -8)


def test_decoding_over_chosen_pages_with_weights_and_an_eviction():
    """Steps that write a token, renew the bounds of its page, choose pages and
    attend over them, adding up weights; then the cache is evicted to half, its
    bounds are made anew and the steps go on."""
    heads, group, dim, page, seqs = 2, 3, 64, 4, 3
    g = torch.Generator(device="cuda").manual_seed(4)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(BF)
    plan = lm.KVPlan(lm.Layout.parse(f"({page},{heads},{dim}):"
                                     f"({heads * dim},{dim},1)"), BF)
    most, hq = 16, heads * group
    pool = seqs * most
    kp = torch.zeros((pool, page, heads, dim), dtype=BF, device="cuda")
    vp = torch.zeros_like(kp)
    cache = lm.KVCache(plan, kp, vp)
    table = torch.randperm(pool, generator=g, device="cuda").int().view(
        seqs, most)
    lens = [40, 33, 7]
    rows = [[[randn(n, dim) for _ in range(heads)] for n in lens]
            for _ in range(2)]               # kv, sequence, head

    def slot(b, j):
        return int(table[b, j // page]) * page + j % page
    for b, n in enumerate(lens):
        lm.kv_write(cache, torch.stack(rows[0][b], 1).contiguous(),
                    torch.stack(rows[1][b], 1).contiguous(),
                    torch.tensor([slot(b, j) for j in range(n)]).cuda())
    bounds = torch.zeros(pool, heads, 2, dim, dtype=torch.int8, device="cuda")
    scale = torch.ones(pool, heads, device="cuda")
    weights = torch.zeros(pool, heads, page, device="cuda")
    # the weights' sums, and how far off they may be
    total = torch.zeros(2, seqs, heads, most * page, dtype=torch.float64,
                        device="cuda")
    keep = 5
    selected = torch.empty(seqs, heads, keep, dtype=torch.int32,
                           device="cuda")
    sl = torch.empty(seqs, dtype=torch.int32, device="cuda")
    ws = space(lm.kv_attend_workspace(plan, seqs, hq, max_pages=most))
    ss = space(lm.kv_select_workspace(plan, seqs, most))
    es = space(lm.kv_evict_workspace(plan, seqs, 24))

    def all_bounds():
        ids, counts = [], []
        for b, n in enumerate(lens):
            for i in range(-(-n // page)):
                ids.append(int(table[b, i]))
                counts.append(min(page, n - i * page))
        lm.kv_bound(cache, ints(ids), ints(counts), bounds, scale)
    all_bounds()
    for step in range(12):
        if step == 6:                        # the heavier half stays
            lm.kv_evict(cache, weights, table, ints(lens), table, sl, 24, es,
                        recent=4)
            for b, n in enumerate(lens):
                for h in range(heads):
                    w = weights_before[b][h]
                    j = list(range(n)) if n <= 24 else lr.choose(
                        w[:n - 4].tolist() + [0.0], 21, 0, 1)[:-1] + \
                        list(range(n - 4, n))
                    for kv in (0, 1):
                        rows[kv][b][h] = rows[kv][b][h][j]
                    total[:, b, h, :len(j)] = total[:, b, h, j].clone()
                    total[:, b, h, len(j):] = 0
            lens = [min(n, 24) for n in lens]
            assert sl.tolist() == lens
            all_bounds()
        k, v = randn(seqs, heads, dim), randn(seqs, heads, dim)
        lm.kv_write(cache, k, v, torch.tensor(
            [slot(b, n) for b, n in enumerate(lens)]).cuda())
        # a place that an evicted token had still has that one's weight
        for b, n in enumerate(lens):
            weights[int(table[b, n // page]), :, n % page] = 0
        for b in range(seqs):
            for h in range(heads):
                for kv, x in enumerate((k, v)):
                    rows[kv][b][h] = torch.cat([rows[kv][b][h], x[b, h][None]])
        lens = [n + 1 for n in lens]
        last = [int(table[b, (n - 1) // page]) for b, n in enumerate(lens)]
        lm.kv_bound(cache, ints(last), ints([(n - 1) % page + 1
                                             for n in lens]), bounds, scale)
        q = randn(seqs, hq, dim)
        out = torch.empty_like(q)
        lm.kv_select(cache, q, bounds, scale, table, ints(lens), selected, sl,
                     ss, first=1, last=1)
        lm.kv_attend(cache, q, selected, sl, out, ws, weights=weights)
        for b, n in enumerate(lens):
            m = -(-n // page)
            ids = table[b, :m].long()
            part = torch.arange(n, device="cuda") // page
            lo = torch.stack([torch.stack(
                [lr.bounds(rows[0][b][h][part == i].float())[0]
                 for h in range(heads)]) for i in range(m)])
            assert torch.equal(lo.float(), bounds[ids, :, 0].float().cpu())
            s = lr.scores(q[b], bounds[ids, :, 0].cpu(),
                          bounds[ids, :, 1].cpu(), scale[ids].cpu(), group)
            for h in range(heads):
                pages = lr.choose(s[h].tolist(), keep, 1, 1)
                assert selected[b, h, :len(pages)].tolist() == \
                    ids[pages].tolist()
                j = [x for p in pages
                     for x in range(p * page, min(n, (p + 1) * page))]
                kk, vv = (rows[kv][b][h][j].double()[:, None]
                          for kv in (0, 1))
                part_q = q[b, h * group:(h + 1) * group]
                p, err = close(out[b, h * group:(h + 1) * group], part_q, kk,
                               vv, group)
                total[0, b, h, j] += p.sum(0)
                # (group + 1 sums of 32 bits)
                total[1, b, h, j] += err.sum(0) + (group + 1) * 2.0 ** -24 * \
                    total[0, b, h, j]
                got = weights[ids, h].flatten()[:n].double()
                assert ((got - total[0, b, h, :n]).abs() <=
                        total[1, b, h, :n]).all()
        weights_before = [[weights[table[b].long(), h].flatten()
                           for h in range(heads)] for b in range(seqs)]


def test_steps_captured_and_replayed():
    """Bounds, choice and attention with weights in one graph, replayed on new
    queries, and an eviction in another; on a stream of their own as well."""
    P = lr.Held([200, 90, 0, 33], 2, 64, 8, "nhd", BF, "int8", seed=5,
                drift=1.0)
    cache, plan = P.cache(lm)
    table, lens = P.table.cuda(), ints(P.lens)
    bounds = torch.zeros(P.pool, 2, 2, 64, dtype=torch.int8, device="cuda")
    scale = torch.ones(P.pool, 2, device="cuda")
    ids = torch.cat([P.table[b, :-(-n // 8)] for b, n in enumerate(P.lens)])
    counts = [min(8, n - 8 * i) for n in P.lens for i in range(-(-n // 8))]
    weights = torch.zeros(P.pool, 2, 8, device="cuda")
    selected = torch.empty(4, 2, 6, dtype=torch.int32, device="cuda")
    sl, kl = ints([0] * 4), ints([0] * 4)
    q = torch.randn(4, 6, 64, device="cuda").to(BF)
    out = torch.empty_like(q)
    ws = space(lm.kv_attend_workspace(plan, 4, 6, max_pages=P.most))
    ss = space(lm.kv_select_workspace(plan, 4, P.most))
    es = space(lm.kv_evict_workspace(plan, 4, 16))
    cids, ccounts = ids.cuda(), ints(counts)

    def step():
        lm.kv_bound(cache, cids, ccounts, bounds, scale)
        lm.kv_select(cache, q, bounds, scale, table, lens, selected, sl, ss)
        lm.kv_attend(cache, q, selected, sl, out, ws, weights=weights)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (1, 2):
        q.copy_(torch.randn(4, 6, 64).to(BF))
        weights.zero_()
        step()
        torch.cuda.synchronize()
        want = [x.clone() for x in (out, selected, sl, weights)]
        out.zero_()
        weights.zero_()
        selected.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (out, selected, sl, weights)):
            assert torch.equal(a, b)
        out.zero_()
        weights.zero_()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(want, (out, selected, sl, weights)):
            assert torch.equal(a, b)
    before = ([x.clone() for x in P.held], weights.clone(),
              [x.clone() for x in P.scales])
    lm.kv_evict(cache, weights, table, lens, table, kl, 16, es, recent=3)
    torch.cuda.synchronize()
    after = [x.clone() for x in (*P.held, weights, *P.scales)]
    state = (*P.held, weights, *P.scales)
    for x, y in zip(state, (*before[0], before[1], *before[2])):
        x.copy_(y)
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2):
        lm.kv_evict(cache, weights, table, lens, table, kl, 16, es, recent=3)
    for x, y in zip(state, (*before[0], before[1], *before[2])):
        x.copy_(y)
    g2.replay()
    torch.cuda.synchronize()
    for x, y in zip(state, after):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert kl.tolist() == [16, 16, 0, 16]


def test_more_sequences_than_a_warp_counts():
    """700 sequences: weights, and the choice of pages of each."""
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 60, (700,), generator=g).tolist()
    P = lr.Held(lens, 1, 16, 4, "nhd", BF, None, seed=3)
    cache, plan = P.cache(lm)
    q = torch.randn(700, 2, 16, generator=g).to(BF).cuda()
    out = torch.empty_like(q)
    w = torch.zeros(P.pool, 1, 4, device="cuda")
    ws = space(lm.kv_attend_workspace(plan, 700, 2, max_pages=P.most))
    lm.kv_attend(cache, q, P.table.cuda(), ints(lens), out, ws, weights=w)
    some = [0, 31, 32, 500, 699]
    for b in some:
        n = lens[b]
        k, v = P.seq(0, b), P.seq(1, b)
        p, err = close(out[b], q[b], k, v, 2)
        ids = P.table[b, :-(-n // 4)].long().cuda()
        got = w[ids].flatten()[:n].double()
        assert ((got - p.sum(0)).abs() <= err.sum(0) +
                2.0 ** -22 * p.sum(0)).all()
    bounds = torch.zeros(P.pool, 1, 2, 16, dtype=torch.int8, device="cuda")
    scale = torch.ones(P.pool, 1, device="cuda")
    ids = torch.cat([P.table[b, :-(-n // 4)] for b, n in enumerate(lens)])
    counts = [min(4, n - 4 * i) for n in lens for i in range(-(-n // 4))]
    lm.kv_bound(cache, ids.cuda(), ints(counts), bounds, scale)
    selected = torch.empty(700, 1, 5, dtype=torch.int32, device="cuda")
    sl = torch.empty(700, dtype=torch.int32, device="cuda")
    lm.kv_select(cache, q, bounds, scale, P.table.cuda(), ints(lens), selected,
                 sl, space(lm.kv_select_workspace(plan, 700, P.most)))
    for b in some:
        m = -(-lens[b] // 4)
        ids = P.table[b, :m].long()
        s = lr.scores(q[b], bounds[ids, :, 0].cpu(), bounds[ids, :, 1].cpu(),
                      scale[ids].cpu(), 2)
        pages = lr.choose(s[0].tolist(), 5, 0, 1)
        assert selected[b, 0, :len(pages)].tolist() == ids[pages].tolist()


def test_more_groups_than_a_warp_counts():
    """90 groups of one to three sequences, some with no prefix."""
    g = torch.Generator().manual_seed(2)
    sizes = torch.randint(0, 4, (90,), generator=g).tolist()
    shared = torch.randint(0, 300, (90,), generator=g).tolist()
    shared[7] = shared[60] = 0
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + n)
    seqs = starts[-1]
    lens = torch.randint(0, 9, (seqs,), generator=g).tolist()
    P = lr.Held(shared + lens, 1, 64, 8, "nhd", BF, None, seed=3)
    cache, plan = P.cache(lm)
    q = torch.randn(seqs, 3, 64, generator=g).to(BF).cuda()
    out = torch.empty_like(q)
    ws = space(lm.kv_attend_shared_workspace(plan, seqs, 3))
    t = P.table.cuda()
    lm.kv_attend_shared(cache, q, t[:90], ints(shared), ints(starts), t[90:],
                        ints(lens), out, ws)
    of = [i for i, n in enumerate(sizes) for _ in range(n)]
    for b in range(seqs):
        rows = [torch.cat([P.seq(kv, of[b]), P.seq(kv, 90 + b)])
                for kv in (0, 1)]
        close(out[b], q[b], *rows, 3, 2.0 ** -8)


@pytest.mark.parametrize("dim,group,dtype", [(8, 1, BF), (72, 11, HF),
                                             (128, 9, BF), (200, 3, HF),
                                             (256, 16, BF)], ids=str)
def test_choice_by_queries_out_of_line(dim, group, dtype):
    """Queries whose rows allow no wide loads, more of them than a product's
    columns, and rows that end inside a step."""
    P = lr.Held([150, 3, 331], 2, dim, 4, "nhd", dtype, None, seed=3,
                drift=1.0)
    cache, plan = P.cache(lm)
    bounds = torch.zeros(P.pool, 2, 2, dim, dtype=torch.int8, device="cuda")
    scale = torch.ones(P.pool, 2, device="cuda")
    ids = torch.cat([P.table[b, :-(-n // 4)] for b, n in enumerate(P.lens)])
    counts = [min(4, n - 4 * i) for n in P.lens for i in range(-(-n // 4))]
    lm.kv_bound(cache, ids.cuda(), ints(counts), bounds, scale)
    g = torch.Generator().manual_seed(2)
    wide = torch.randn(3, 2 * group, dim + 5, generator=g).to(dtype).cuda()
    q = wide[:, :, 3:3 + dim]
    selected = torch.empty(3, 2, 9, dtype=torch.int32, device="cuda")
    sl = torch.empty(3, dtype=torch.int32, device="cuda")
    lm.kv_select(cache, q, bounds, scale, P.table.cuda(), ints(P.lens),
                 selected, sl, space(lm.kv_select_workspace(plan, 3, P.most)),
                 first=1, last=2)
    for b, n in enumerate(P.lens):
        m = -(-n // 4)
        of = P.table[b, :m].long()
        s = lr.scores(q[b], bounds[of, :, 0].cpu(), bounds[of, :, 1].cpu(),
                      scale[of].cpu(), group)
        for h in range(2):
            pages = lr.choose(s[h].tolist(), 9, 1, 2)
            assert selected[b, h, :len(pages)].tolist() == of[pages].tolist()


@pytest.mark.parametrize("keys", [1, 600, 1300])
def test_a_short_prefix_after_a_long_one(keys):
    """A line of fewer tiles than blocks: what blocks left in the workspace
    that have nothing to do now is nobody's."""
    P = lr.Held([30000, keys, 5, 3], 4, 64, 16, "nhd", BF, None, seed=3)
    cache, plan = P.cache(lm)
    g = torch.Generator().manual_seed(2)
    q = torch.randn(2, 16, 64, generator=g).to(BF).cuda()
    ws = space(lm.kv_attend_shared_workspace(plan, 2, 16))
    t = P.table.cuda()
    out = torch.empty_like(q)
    for first, n in ((0, 30000), (1, keys)):
        lm.kv_attend_shared(cache, q, t[first:first + 1], ints([n]),
                            ints([0, 2]), t[2:], ints([5, 3]), out, ws)
    for b in range(2):
        rows = [torch.cat([P.seq(kv, 1), P.seq(kv, 2 + b)]) for kv in (0, 1)]
        close(out[b], q[b], *rows, 4, 2.0 ** -8)


@pytest.mark.parametrize("dtype,store", [(BF, None), (HF, None), (BF, "int8")],
                         ids=str)
@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 26, 2.0 ** 60])
def test_scores_of_any_size(dtype, store, size):
    """Scores up to 2^60 about (in float16 2^29): all weight lies on each row's
    largest, whose value comes out as it is."""
    if dtype == HF and size > 2.0 ** 29:
        size = 2.0 ** 29
    P = lr.Held([700, 3, 5], 1, 64, 16, "nhd", dtype, store, seed=3)
    cache, plan = P.cache(lm)
    g = torch.Generator().manual_seed(2)
    q = torch.randn(2, 4, 64, generator=g) * 2.0 ** 12
    q = q.to(dtype).cuda()
    out = torch.empty_like(q)
    ws = space(lm.kv_attend_shared_workspace(plan, 2, 4))
    t = P.table.cuda()
    # (a score is 2^12 times some 8)
    scale = size / 2.0 ** 15
    lm.kv_attend_shared(cache, q, t[:1], ints([700]), ints([0, 2]), t[1:],
                        ints([3, 5]), out, ws, scale=scale)
    for b in range(2):
        k, v = (torch.cat([P.seq(kv, 0), P.seq(kv, 1 + b)])[:, 0]
                for kv in (0, 1))
        s = q[b].double() @ k.T * scale
        top, at = s.max(-1)
        s.scatter_(1, at[:, None], -math.inf)
        assert (top - s.amax(-1) > 2.0 ** -14 * top).all()
        assert (top - s.amax(-1) > 40).all()
        want = v[at]
        assert ((out[b].double() - want).abs() <=
                torch.finfo(dtype).eps * want.abs()).all()


def test_two_streams_with_workspaces_of_their_own():
    """The calls of two streams, each with a cache, workspaces and outputs of its
    own, again and again and at once: what each gives alone."""
    def make(seed, store):
        P = lr.Held([3000, 900, 700, 1500, 40], 2, 64, 16, "nhd", BF, store,
                    seed=seed)
        cache, plan = P.cache(lm)
        g = torch.Generator().manual_seed(seed)
        q = torch.randn(4, 8, 64, generator=g).to(BF).cuda()
        t = P.table.cuda()
        lens = ints(P.lens[1:])
        width = t.shape[1]
        out = [torch.empty_like(q) for _ in range(3)]
        bounds = torch.zeros(P.pool, 2, 2, 64, dtype=torch.int8, device="cuda")
        bscale = torch.ones(P.pool, 2, device="cuda")
        selected = torch.empty(4, 2, 9, dtype=torch.int32, device="cuda")
        slens, klens = ints([0] * 4), ints([0] * 4)
        weights = torch.zeros(P.pool, 2, 16, device="cuda")
        spare = [x.clone() for x in P.held]
        wide = lm.KVCache(plan, *spare,
                          *[None if x is None else x.clone() for x in P.scales])
        ws = [space(lm.kv_attend_shared_workspace(plan, 4, 8)),
              space(lm.kv_attend_workspace(plan, 4, 8, max_pages=width)),
              space(lm.kv_select_workspace(plan, 4, width)),
              space(lm.kv_evict_workspace(plan, 4, 500))]
        pages = ints(list(range(P.pool)))
        counts = ints([16] * P.pool)

        def run(stream=None):
            kw = {"stream": stream}
            lm.kv_attend_shared(cache, q, t[:1], ints3000, ints04, t[1:], lens,
                                out[0], ws[0], **kw)
            lm.kv_bound(cache, pages, counts, bounds, bscale, **kw)
            lm.kv_select(cache, q, bounds, bscale, t[1:], lens, selected, slens,
                         ws[2], first=1, last=1, **kw)
            lm.kv_attend(cache, q, selected, slens, out[1], ws[1], **kw)
            lm.kv_attend(cache, q, t[1:], lens, out[2], ws[1],
                         weights=weights, **kw)
            lm.kv_evict(wide, weights, t[1:], lens, t[1:], klens, 500, ws[3],
                        recent=10, **kw)
        ints3000, ints04 = ints([3000]), ints([0, 4])
        results = [*out, bounds, bscale, selected, slens, weights, klens]
        return run, results, weights
    runs = [make(1, None), make(2, "int8")]
    alone = []
    for run, results, weights in runs:
        weights.zero_()
        run()
        torch.cuda.synchronize()
        alone.append([x.clone() for x in results])
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(5):
        for (run, results, weights), stream in zip(runs, streams):
            with torch.cuda.stream(stream):
                weights.zero_()
                for x in results[:3]:
                    x.fill_(7)
            run(stream)
        torch.cuda.synchronize()
        for (_, results, _), want in zip(runs, alone):
            for x, y in zip(results, want):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("store", [None, "e4m3"])
def test_offsets_past_32_bits(store):
    """Pages 3 GB apart: rows that lie past 2^32 elements."""
    heads, dim, page, pages = 1, 64, 16, 4
    held = 2 if store is None else 1
    stride = 3 * 2 ** 30 // held
    plan = lm.KVPlan(lm.Layout.parse("(16,1,64):(64,64,1)"), BF, store,
                     page_stride=stride)
    n = stride * (pages - 1) + page * dim
    kind = BF if store is None else torch.uint8
    k, v = (torch.empty(n, dtype=kind, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(2)
    rows = []
    for x in (k, v):
        part = x.as_strided((pages, page, dim), (stride, dim, 1))
        if store is None:
            part.copy_(torch.randn(pages, page, dim, generator=g,
                                   device="cuda"))
            rows.append(part.double())
        else:
            c = torch.randint(0, 100, part.shape, generator=g, device="cuda")
            part.copy_(c)
            rows.append(kr.e4m3_values().cuda()[c] * 2.0 ** -6)
    scales = [None, None] if store is None else [
        torch.full((pages, 1, page), 2.0 ** -6, device="cuda")
        for _ in range(2)]
    cache = lm.KVCache(plan, k, v, *scales, pages=pages)
    table = ints([[3, 1, 2, 0]])
    order = [3, 1, 2, 0]
    q = torch.randn(2, 2, dim, generator=g, device="cuda").to(BF)
    out = torch.empty_like(q)
    ws = space(lm.kv_attend_shared_workspace(plan, 2, 2))
    lm.kv_attend_shared(cache, q, table, ints([60]), ints([0, 2]),
                        table.repeat(2, 1), ints([5, 0]), out, ws)
    full = [r[order].reshape(-1, 1, dim) for r in rows]
    step = 2.0 ** -8 if store is None else 0.0
    close(out[0], q[0], torch.cat([full[0][:60], full[0][:5]]),
          torch.cat([full[1][:60], full[1][:5]]), 2, step)
    close(out[1], q[1], full[0][:60], full[1][:60], 2, step)
    bounds = torch.zeros(pages, 1, 2, dim, dtype=torch.int8, device="cuda")
    scale = torch.ones(pages, 1, device="cuda")
    lm.kv_bound(cache, ints([3, 2]), ints([16, 16]), bounds, scale)
    for p in (3, 2):
        lo, hi, by = lr.bounds(rows[0][p].float())
        assert torch.equal(bounds[p, 0, 0].float().cpu(), lo.float())
        assert torch.equal(bounds[p, 0, 1].float().cpu(), hi.float())
    w = torch.rand(pages, 1, page, generator=g, device="cuda")
    kept = torch.empty(1, dtype=torch.int32, device="cuda")
    order_w = w[order].flatten()[:60]
    order_w = order_w.tolist()
    j = sorted(sorted(range(60), key=lambda i: (-order_w[i], i))[:20])
    before = [x.as_strided((pages, page, dim), (stride, dim, 1))[order]
              .reshape(-1, dim)[j].clone() for x in (k, v)]
    lm.kv_evict(cache, w, table, ints([60]), table, kept, 20,
                space(lm.kv_evict_workspace(plan, 1, 20)))
    for x, want in zip((k, v), before):
        got = x.as_strided((pages, page, dim), (stride, dim, 1))[order] \
            .reshape(-1, dim)[:20]
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("args", [
    ["--prefix", "300"], ["--prefix", "1", "--store", "e4m3"],
    ["--pages", "5"], ["--pages", "40", "--store", "int8"],
    ["--budget", "64"], ["--budget", "200", "--store", "e4m3"]], ids=str)
def test_the_example_runs(args):
    """examples/decode_cache.py in its long forms: outputs are bfloat16 (2^-8
    of each, half of that in the mean) of the same rows, whose int8 values were
    rounded to bfloat16 on their way back, and a shared token's weight is
    rounded as the output is."""
    import os
    import runpy
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    main = runpy.run_path(os.path.join(root, "examples", "decode_cache.py"))
    assert main["main"](args + ["--steps", "12"]) <= 2.0 ** -7
