"""The paged key-value cache on the GPU against the 64-bit definitions in
kv_reference: rotary positions and their gradient, the quantising write, the
read back and the attention of one new token, at the sizes, strides and
lengths where they can go wrong.  Bounds are derived in kv_reference (or
beside the check) from the roundings that the definitions allow."""

import math

import pytest

import kv_reference as kr

torch = pytest.importorskip("torch")
lm = pytest.importorskip("layout_driven_movement_gb300")

pytestmark = pytest.mark.gpu

BF, HF, FL = torch.bfloat16, torch.float16, torch.float32


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


def range_reported():
    return lm.device_status(reset=True) == -12


# --- rotary positions ------------------------------------------------------

ROPE = [
    # tokens, heads, dim, rot, dtype, interleaved, gap, offset
    (1, 1, 2, 2, BF, False, 0, 0),
    (7, 3, 64, 64, BF, False, 0, 0),
    (33, 5, 128, 128, HF, False, 2, 0),
    (33, 5, 128, 128, BF, True, 0, 0),
    (19, 9, 80, 32, BF, False, 1, 0),      # halves of two chunks, a rest
    (19, 4, 96, 24, HF, False, 0, 0),      # halves that are no whole chunks
    (5, 4, 90, 38, BF, True, 0, 0),        # odd sizes: one element at a time
    (12, 2, 64, 64, FL, False, 0, 0),
    (12, 7, 96, 64, FL, True, 3, 0),
    (11, 6, 128, 64, BF, False, 0, 1),     # misaligned by an element
    (300, 40, 128, 128, BF, False, 8, 0),
]


def rope_inputs(case, seed=3):
    t, h, d, rot, dtype, inter, gap, off = case
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(t * (h + gap) * d + off, generator=g).to(dtype).cuda()
    x = wide[off:].view(t, h + gap, d)[:, :h]
    pos = torch.randint(0, 5000, (t,), generator=g)
    plan = lm.RopePlan(d, rot, interleaved=inter)
    table = torch.empty(5000, rot, device="cuda")
    lm.rope_table(plan, table)
    return x, pos, plan, table


@pytest.mark.parametrize("case", ROPE, ids=str)
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(case, inverse):
    t, h, d, rot, dtype, inter, gap, off = case
    x, pos, plan, table = rope_inputs(case)
    freqs, amp = plan.frequencies()
    assert amp == 1
    want = kr.turn(x.cpu(), pos, freqs, rot, inter, -1.0 if inverse else 1.0)
    bound = kr.turn_bound(x.cpu(), rot, inter, dtype, want)
    out = torch.full((t, h, d), math.nan, dtype=dtype, device="cuda")
    p = pos.cuda() if inverse else pos.int().cuda()
    lm.rope(plan, x, p, table, out, inverse=inverse)
    assert ((out.cpu().double() - want).abs() <= bound).all()
    # in place: the same bits, and the gap between the rows untouched
    y = x.clone(memory_format=torch.preserve_format)
    wide = torch.full((t, h + 1, d), 7.0, dtype=dtype, device="cuda")
    wide[:, :h] = x
    lm.rope(plan, wide[:, :h], p, table, wide[:, :h], inverse=inverse)
    assert torch.equal(wide[:, :h], out)
    assert (wide[:, h] == 7).all()
    assert torch.equal(y, x)


def test_rope_heads_before_tokens_and_broadcast_heads():
    """A [heads, tokens, dim] tensor by its strides, and one head read by
    all (stride 0)."""
    plan = lm.RopePlan(64)
    table = torch.empty(128, 64, device="cuda")
    lm.rope_table(plan, table)
    x = torch.randn(6, 50, 64, device="cuda").to(BF)
    pos = torch.arange(50, device="cuda")
    out = torch.empty(50, 6, 64, dtype=BF, device="cuda")
    lm.rope(plan, x.transpose(0, 1), pos, table, out)
    dense = torch.empty_like(out)
    lm.rope(plan, x.transpose(0, 1).contiguous(), pos, table, dense)
    assert torch.equal(out, dense)
    one = x[:1].transpose(0, 1)
    lm.rope(plan, one.expand(50, 6, 64), pos, table, out)
    lm.rope(plan, one.contiguous(), pos, table, dense[:, :1])
    assert torch.equal(out, dense[:, :1].expand(50, 6, 64))


def test_rope_gradient_against_differences():
    """d sum(w * rope(x)) / dx along random directions: the turn is linear, so
    a central difference in 32 bits is off only by rounding.  With |w|, |x|
    about 1 over n elements the sums carry at most 2 n^0.5 * 2^-20."""
    g = torch.Generator().manual_seed(5)
    plan = lm.RopePlan(32, 24, interleaved=True)
    table = torch.empty(64, 24, device="cuda")
    lm.rope_table(plan, table)
    pos = torch.randint(0, 64, (9,), generator=g).cuda()
    x, w, d = (torch.randn(9, 3, 32, generator=g).cuda() for _ in range(3))
    def f(v):
        out = torch.empty_like(v)
        lm.rope(plan, v, pos, table, out)
        return (out.double() * w.double()).sum()
    dx = torch.empty_like(x)
    lm.rope(plan, w, pos, table, dx, inverse=True)
    slope = (f(x + d) - f(x - d)) / 2
    want = (dx.double() * d.double()).sum()
    assert abs(slope - want) <= 2 * x.numel() ** 0.5 * 2.0 ** -20


def test_rope_table_far_positions_and_scalings():
    for kw in [{}, {"scaling": "linear", "factor": 4.0},
               {"scaling": "ntk", "factor": 8.0},
               {"scaling": "yarn", "factor": 16.0,
                "original_positions": 4096}]:
        plan = lm.RopePlan(128, 96, **kw)
        freqs, amp = plan.frequencies()
        table = torch.empty(131072, 96, device="cuda")
        lm.rope_table(plan, table)
        rows = [0, 1, 4095, 65537, 131071]
        ang = torch.tensor(rows, dtype=torch.float64)[:, None] * \
            torch.tensor(freqs, dtype=torch.float64)
        want = torch.cat([ang.cos() * amp, ang.sin() * amp], 1)
        got = table[rows].cpu().double()
        # one rounding to 32 bits of values up to amp, and 64-bit angles
        assert ((got - want).abs() <= 2.0 ** -24 * 1.01 * amp).all()


def test_rope_position_out_of_the_table():
    plan = lm.RopePlan(64, 32)
    table = torch.empty(10, 32, device="cuda")
    lm.rope_table(plan, table)
    x = torch.randn(4, 2, 64, device="cuda").to(BF)
    out = torch.zeros_like(x)
    lm.rope(plan, x, torch.tensor([0, 10, -1, 9], device="cuda"), table, out)
    assert range_reported()
    assert out[1:3, :, :32].isnan().all() and not out[1:3, :, 32:].isnan().any()
    assert not out[0].isnan().any() and not out[3].isnan().any()


# --- write and read --------------------------------------------------------

def make_cache(P, interleave=False):
    """(cache, plan) over a Pages' buffers; interleaved: one buffer with each
    page's keys followed by its values."""
    plan_args = {}
    if interleave:
        k = P.device(0).flatten(1)
        v = P.device(1).flatten(1)
        both = torch.stack([k, v], 1).contiguous()
        k, v = both[:, 0], both[:, 1]
        plan_args["page_stride"] = both.stride(0)
    else:
        k, v = P.device(0), P.device(1)
    plan = lm.KVPlan(lm.Layout.make(*P.page_layout()), P.dtype, P.store,
                     **plan_args)
    return lm.KVCache(plan, k, v, P.device_scale(0), P.device_scale(1),
                      pages=P.pool), plan


def by_token(P, t):
    t = t.reshape((P.pool, P.page, P.heads, P.dim) if P.order == "nhd"
                  else (P.pool, P.heads, P.page, P.dim)).cpu()
    return t if P.order == "nhd" else t.transpose(1, 2)


WRITE = [
    # tokens, heads, dim, page, order, dtype, store
    (1, 1, 16, 1, "nhd", BF, "e4m3"),
    (37, 8, 128, 16, "nhd", BF, "e4m3"),
    (37, 3, 128, 16, "hnd", HF, "int8"),
    (50, 5, 80, 24, "nhd", HF, "int8"),
    (50, 5, 80, 7, "hnd", BF, "e4m3"),
    (20, 2, 256, 64, "nhd", BF, "int8"),
    (20, 2, 256, 5, "hnd", HF, "e4m3"),
    (33, 4, 72, 3, "nhd", BF, None),
    (33, 4, 128, 16, "hnd", HF, None),
    (9, 1, 8, 2, "hnd", BF, None),
]


@pytest.mark.parametrize("case", WRITE, ids=str)
@pytest.mark.parametrize("fused", [False, True])
def test_write_holds_the_definition(case, fused):
    """Codes and scales of unrotated rows against the format, some slots
    skipped, the rest of the cache untouched."""
    t, heads, dim, page, order, dtype, store = case
    g = torch.Generator().manual_seed(11)
    P = kr.Pages([t], heads, dim, page, order, dtype, store, seed=2)
    cache, plan = make_cache(P, interleave=fused)
    before = [cache.k.clone(), cache.v.clone()]
    wide = torch.randn(t, 2 * heads + 1, dim, generator=g).to(dtype)
    wide[0, 0] = 0                               # a row of zeros
    if t > 3:
        wide[1, 0, 3] = 2.0 ** -20               # tiny and huge rows
        wide[2, 0] *= 1000
        wide[3, :, :] *= 1e-6
    dev = wide.cuda()
    k, v = dev[:, :heads], dev[:, heads:2 * heads]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    slots = torch.randperm(P.pool * page, generator=g)[:t]
    skipped = torch.zeros(t, dtype=torch.bool)
    skipped[4::5] = True
    lm.kv_write(cache, k, v, torch.where(skipped, -1, slots).cuda())
    grid = kr.e4m3_values()
    named = torch.zeros(P.pool, page, dtype=torch.bool)
    for kv, x in enumerate((wide[:, :heads], wide[:, heads:2 * heads])):
        held = by_token(P, (cache.k, cache.v)[kv])
        scales = (cache.k_scale, cache.v_scale)[kv]
        for j in range(t):
            if skipped[j]:
                continue
            p, o = divmod(int(slots[j]), page)
            named[p, o] = True
            if store is None:
                assert torch.equal(held[p, o], x[j])
                continue
            sc = scales[p, :, o].cpu().double()
            for h in range(heads):
                row = x[j, h].double()
                top = float(row.abs().max())
                code = held[p, o, h]
                if store == "e4m3":
                    assert float(sc[h]) == kr.e4m3_scale(top)
                    want = grid[kr.e4m3_nearest(row / sc[h])]
                    assert torch.equal(grid[code.long()], want)
                    assert not grid[code.long()].isnan().any()
                else:
                    s = max(top / 127, 2.0 ** -126) if top else 1.0
                    assert abs(float(sc[h]) - s) <= 2.0 ** -23 * s
                    # two 32-bit roundings of a quotient up to 127
                    q = code.view(torch.int8).double()
                    off = (q - row / s).abs()
                    assert (off <= 0.5 + 127 * 2.0 ** -22).all()
                    assert q.abs().max() <= 127
    for kv in range(2):
        same = by_token(P, (cache.k, cache.v)[kv]).view(torch.uint8)[~named]
        assert torch.equal(same, by_token(P, before[kv]).view(torch.uint8)
                           [~named])


def test_write_rows_that_are_not_finite_are_nan():
    P = kr.Pages([4], 2, 32, 4, "nhd", BF, "e4m3")
    for store in ("e4m3", "int8"):
        P.store = store
        cache, plan = make_cache(P)
        x = torch.ones(4, 2, 32).to(BF)
        x[0, 0, 5], x[1, 1, 31], x[2, 0, 0] = math.inf, math.nan, -math.inf
        lm.kv_write(cache, x.cuda(), torch.ones_like(x).cuda(),
                    torch.arange(4, device="cuda"))
        table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
        out = torch.empty(4, 2, 32, dtype=BF, device="cuda")
        lm.kv_read(cache, table, torch.tensor([4], dtype=torch.int32).cuda(),
                   torch.tensor([0, 4], dtype=torch.int32).cuda(), out,
                   vo := torch.empty_like(out))
        bad = torch.zeros(4, 2, dtype=torch.bool)
        bad[0, 0] = bad[1, 1] = bad[2, 0] = True
        assert torch.equal(out.isnan().all(-1).cpu(), bad)
        assert not out.cpu()[~bad].isnan().any()
        assert not vo.isnan().any()


@pytest.mark.parametrize("store", [None, "e4m3", "int8"])
@pytest.mark.parametrize("rot,inter", [(64, False), (64, True), (40, False),
                                       (20, True)])
def test_write_turns_the_keys(store, rot, inter):
    """Keys turned on their way: the held value is within half a step of the
    64-bit turn (and its 32-bit error); values are not turned."""
    t, heads, dim = 21, 3, 64
    g = torch.Generator().manual_seed(8)
    P = kr.Pages([t], heads, dim, 16, "nhd", BF, store)
    cache, plan = make_cache(P)
    rope = lm.RopePlan(dim, rot, interleaved=inter, base=500.0)
    table = torch.empty(400, rot, device="cuda")
    lm.rope_table(rope, table)
    pos = torch.randint(0, 400, (t,), generator=g)
    x = torch.randn(2, t, heads, dim, generator=g).to(BF)
    slots = torch.arange(t) + 5
    lm.kv_write(cache, x[0].cuda(), x[1].cuda(), slots.cuda(), rope=rope,
                positions=pos.cuda(), table=table)
    want = kr.turn(x[0], pos, rope.frequencies()[0], rot, inter)
    slack = 4 * 2.0 ** -24 * 2 * x[0].double().abs().amax(-1, keepdim=True)
    held = by_token(P, cache.k).reshape(-1, heads, dim)[slots]
    vals = by_token(P, cache.v).reshape(-1, heads, dim)[slots]
    if store is None:
        bound = kr.turn_bound(x[0], rot, inter, BF, want)
        assert ((held.double() - want).abs() <= bound).all()
        assert torch.equal(vals, x[1])
        return
    sc = cache.k_scale.cpu().transpose(1, 2).reshape(-1, heads)[slots]
    sc = sc.double()[..., None]
    if store == "e4m3":
        got = kr.e4m3_values()[held.long()] * sc
        half = torch.maximum(want.abs() * 2.0 ** -4, sc * 2.0 ** -10)
    else:
        got = held.view(torch.int8).double() * sc
        half = sc * (0.5 + 127 * 2.0 ** -22)
    assert ((got - want).abs() <= half + slack * 1.2).all()


def test_write_slot_and_position_out_of_range():
    P = kr.Pages([8], 2, 32, 4, "nhd", BF, None)
    cache, plan = make_cache(P)
    before = cache.k.clone()
    x = torch.ones(2, 2, 32, dtype=BF, device="cuda")
    lm.kv_write(cache, x, x, torch.tensor([P.pool * 4, 1 << 40]).cuda())
    assert range_reported()
    assert torch.equal(before.view(torch.uint8), cache.k.view(torch.uint8))
    rope = lm.RopePlan(32)
    table = torch.ones(3, 32, device="cuda")
    lm.kv_write(cache, x, x, torch.tensor([0, 1]).cuda(), rope=rope,
                positions=torch.tensor([2, 3]).cuda(), table=table)
    assert range_reported()
    k = by_token(P, cache.k).reshape(-1, 2, 32)
    assert not k[0].isnan().any() and k[1].isnan().all()


READ = [
    # lens, heads, dim, page, order, dtype, store, out
    ([1], 1, 16, 1, "nhd", BF, "e4m3", BF),
    ([0, 5, 0, 33, 1], 3, 80, 16, "hnd", HF, "int8", HF),
    ([100, 31, 32, 33, 0], 8, 128, 16, "nhd", BF, "e4m3", BF),
    ([70, 3], 2, 256, 24, "nhd", BF, None, BF),
    ([70, 3], 2, 256, 5, "hnd", HF, "e4m3", FL),
    ([17, 0], 4, 72, 7, "nhd", HF, None, FL),
    ([17, 40], 4, 64, 64, "hnd", BF, "int8", FL),
]


@pytest.mark.parametrize("case", READ, ids=str)
def test_read_gives_every_row(case):
    lens, heads, dim, page, order, dtype, store, to = case
    P = kr.Pages(lens, heads, dim, page, order, dtype, store, seed=4)
    cache, plan = make_cache(P, interleave=heads % 2 == 0)
    starts, at = [0], 0
    for n in lens:
        at += n + 2                       # rows between that nothing names
        starts.append(at)
    wide = torch.full((at, 2 * heads + 1, dim), 5.0, dtype=to, device="cuda")
    k, v = wide[:, :heads], wide[:, heads:2 * heads]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    lm.kv_read(cache, P.table.cuda(), torch.tensor(lens).int().cuda(),
               torch.tensor(starts).int().cuda(), k, v, stream=st)
    st.synchronize()
    for kv, got in enumerate((k.cpu(), v.cpu())):
        for b, n in enumerate(lens):
            want = P.rows[kv][b]
            part = got[starts[b]:starts[b] + n].double()
            # the 32-bit product of code and scale, then the output's type
            u = kr.ROUND[to] + 2.0 ** -24 if store == "int8" else kr.ROUND[to]
            assert ((part - want).abs() <= want.abs() * u * 1.01
                    + kr.TINY[to]).all()
            if store is None and to == dtype:
                assert torch.equal(part, want)
            assert (got[starts[b] + n:starts[b + 1]] == 5).all()
    assert (wide[:, 2 * heads:] == 5).all()


def test_read_bounds():
    """Lengths past the page table or the next sequence's rows, negative
    lengths, page numbers out of range, fewer output rows than tokens."""
    P = kr.Pages([8, 8, 8], 1, 16, 4, "nhd", BF, None)
    cache, plan = make_cache(P)
    table = P.table.clone()
    table[1, 0], table[2, 1] = P.pool, -1
    k = torch.full((22, 1, 16), 5.0, dtype=BF, device="cuda")
    v = k.clone()
    lm.kv_read(cache, table.cuda(), torch.tensor([-3, 8, 1000]).int().cuda(),
               torch.tensor([0, 8, 14, 30]).int().cuda(), k, v)
    assert range_reported()
    for kv, got in enumerate((k.cpu(), v.cpu())):
        assert (got[:8] == 5).all()
        assert (got[8:12] == 0).all()                     # a bad page
        assert torch.equal(got[12:14].double(), P.rows[kv][1][4:6])
        assert torch.equal(got[14:18].double(), P.rows[kv][2][:4])
        assert (got[18:22] == 0).all()                    # a bad page


# --- attention -------------------------------------------------------------

EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300]


def run_attend(P, group, window=0, scale=None, lens=None, q=None, lse=True,
               stream=None, workspace=None, table=None, interleave=False,
               wide=False):
    cache, plan = make_cache(P, interleave)
    n, hq = len(P.lens), P.heads * group
    g = torch.Generator().manual_seed(21)
    if q is None:
        q = torch.randn(n, hq, P.dim, generator=g).to(P.dtype)
    if wide:
        buf = torch.full((n, hq + 3, P.dim + 8), 3.0, dtype=P.dtype).cuda()
        qd, out = buf[:, :hq, :P.dim], torch.full_like(buf, 9.0)
        qd.copy_(q)
        od = out[:, 1:hq + 1, 8:]
    else:
        qd = q.cuda()
        od = torch.full_like(qd, math.nan)
    ld = torch.full((n, hq), math.nan, device="cuda") if lse else None
    if workspace is None:
        workspace = torch.zeros(lm.kv_attend_workspace(plan, n, hq),
                                dtype=torch.uint8, device="cuda")
    ln = torch.tensor(P.lens if lens is None else lens).int().cuda()
    tb = (P.table if table is None else table).cuda()
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    lm.kv_attend(cache, qd, tb, ln, od, workspace, lse=ld, scale=scale,
                 window=window, stream=stream)
    torch.cuda.synchronize()
    if wide:
        mask = torch.ones_like(out, dtype=torch.bool)
        mask[:, 1:hq + 1, 8:] = False
        assert (out[mask] == 9).all()
    return q, od.cpu(), ld.cpu() if lse else None


def check_attend(P, group, q, out, lse, window=0, scale=None, rows=None):
    scale = P.dim ** -0.5 if scale is None else scale
    for b, n in enumerate(P.lens):
        k, v = P.rows[0][b], P.rows[1][b]
        if rows is not None:
            k, v = k[:rows[b]], v[:rows[b]]
        want, wl, mag, dot = kr.attend(q[b].double(), k, v, group, scale,
                                       window)
        bo, bl = kr.attend_bounds(P.dtype, P.dim, want, wl, mag, dot)
        assert ((out[b].double() - want).abs() <= bo).all(), (b, n)
        if lse is not None:
            empty = wl == -math.inf
            assert (lse[b][empty] == -math.inf).all()
            assert ((lse[b].double() - wl).abs() <= bl)[~empty].all(), (b, n)


@pytest.mark.parametrize("store", [None, "e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("heads,group,dim,page,order", [
    (1, 1, 64, 16, "nhd"), (2, 4, 128, 16, "nhd"), (2, 8, 128, 64, "hnd"),
    (3, 5, 80, 24, "hnd"), (1, 16, 128, 1, "nhd"), (2, 9, 64, 5, "nhd"),
    (1, 3, 256, 32, "hnd"), (1, 20, 256, 7, "nhd"), (2, 2, 16, 128, "nhd"),
    (1, 40, 112, 128, "hnd"),
])
def test_attend_lengths(store, dtype, heads, group, dim, page, order):
    P = kr.Pages(EDGES, heads, dim, page, order, dtype, store, seed=dim)
    q, out, lse = run_attend(P, group)
    check_attend(P, group, q, out, lse)


@pytest.mark.parametrize("dim", [8, 24, 72, 200])
def test_attend_dims_of_16_bit_rows(dim):
    P = kr.Pages([40, 0, 129], 2, dim, 12, "nhd", BF, None, seed=dim)
    q, out, lse = run_attend(P, 3)
    check_attend(P, 3, q, out, lse)


@pytest.mark.parametrize("store", [None, "e4m3", "int8"])
@pytest.mark.parametrize("window", [1, 2, 17, 64, 100, 5000])
def test_attend_window(store, window):
    P = kr.Pages(EDGES + [1000], 2, 64, 24, "nhd", BF, store, seed=7)
    q, out, lse = run_attend(P, 4, window=window)
    check_attend(P, 4, q, out, lse, window=window)


@pytest.mark.parametrize("store,dtype", [(None, BF), (None, HF),
                                         ("e4m3", BF), ("int8", HF)])
def test_attend_long_and_ragged(store, dtype):
    """Lengths that many blocks share, among ones that share a block."""
    lens = [20011, 3, 0, 700, 9000, 1, 1, 64, 4097, 0]
    P = kr.Pages(lens, 2, 128, 16, "nhd", dtype, store, seed=9)
    ws = None
    q, out, lse = run_attend(P, 4, workspace=ws)
    check_attend(P, 4, q, out, lse)
    # the same inputs give the same bits, on a stream of one's own too
    q2, out2, lse2 = run_attend(P, 4, q=q, stream=torch.cuda.Stream())
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_attend_many_sequences():
    """More sequences than threads of a block, most of them short."""
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 40, (700,), generator=g).tolist()
    P = kr.Pages(lens, 1, 64, 16, "nhd", BF, None, seed=3)
    q, out, lse = run_attend(P, 2)
    check_attend(P, 2, q, out, lse)


def test_attend_workspace_serves_call_after_call():
    P = kr.Pages([5000, 33], 2, 128, 16, "nhd", BF, None, seed=5)
    cache, plan = make_cache(P)
    ws = torch.zeros(lm.kv_attend_workspace(plan, 2, 8), dtype=torch.uint8,
                     device="cuda")
    outs = [run_attend(P, 4, workspace=ws) for _ in range(3)]
    for q, out, lse in outs:
        check_attend(P, 4, q, out, lse)
        assert torch.equal(out, outs[0][1])
    # another batch through the same workspace
    Q = kr.Pages([1, 900, 70, 2000], 2, 128, 16, "hnd", BF, None, seed=6)
    q, out, lse = run_attend(Q, 4, workspace=ws)
    check_attend(Q, 4, q, out, lse)


@pytest.mark.parametrize("store,dtype,dim,heads,group,order", [
    ("int8", BF, 64, 4, 5, "nhd"), ("e4m3", HF, 64, 2, 12, "nhd"),
    ("e4m3", BF, 80, 6, 4, "nhd"), ("int8", HF, 112, 2, 16, "nhd"),
    ("int8", BF, 64, 3, 5, "nhd"), ("e4m3", BF, 64, 4, 3, "hnd"),
    (None, HF, 256, 1, 9, "nhd"), ("e4m3", HF, 256, 2, 3, "nhd"),
    (None, BF, 64, 1, 1, "hnd"),
])
def test_attend_one_long_sequence(store, dtype, dim, heads, group, order):
    """Heads shared by many blocks (joined in two levels), in pairs where rows
    are narrow and side by side; page sizes a step does and does not divide."""
    for page, n in ((40, 30011), (64, 9000), (1, 2500)):
        P = kr.Pages([n, 100], heads, dim, page, order, dtype, store, seed=n)
        q, out, lse = run_attend(P, group)
        check_attend(P, group, q, out, lse)


def test_attend_one_workspace_for_several_plans():
    """The largest workspace serves every plan, call after call."""
    Ps = [kr.Pages([3000, 40], 2, 64, 16, "nhd", BF, "int8", seed=1),
          kr.Pages([5000], 1, 256, 16, "nhd", HF, None, seed=2),
          kr.Pages([2000, 0, 700], 2, 128, 16, "hnd", BF, "e4m3", seed=3),
          kr.Pages([2500], 2, 64, 16, "nhd", BF, None, seed=4)]
    need = []
    for P in Ps:
        plan = lm.KVPlan(lm.Layout.make(*P.page_layout()), P.dtype, P.store)
        need.append(lm.kv_attend_workspace(plan, len(P.lens), 12 * P.heads))
    ws = torch.zeros(max(need), dtype=torch.uint8, device="cuda")
    for P in Ps + Ps[::-1]:
        q, out, lse = run_attend(P, 12, workspace=ws)
        check_attend(P, 12, q, out, lse)


def test_attend_workspace_too_small():
    P = kr.Pages([50], 1, 64, 16, "nhd", BF, None)
    cache, plan = make_cache(P)
    n = lm.kv_attend_workspace(plan, 1, 2)
    q = torch.zeros(1, 2, 64, dtype=BF, device="cuda")
    args = (cache, q, P.table.cuda(), torch.tensor([50]).int().cuda(),
            torch.zeros_like(q))
    for ws, status in ((torch.zeros(n - 1, dtype=torch.uint8, device="cuda"),
                        -6), (None, -1)):
        with pytest.raises(lm.LayoutMoveError) as e:
            lm.kv_attend(*args, ws)
        assert e.value.status == status


@pytest.mark.parametrize("store", [None, "e4m3", "int8"])
def test_tensors_that_allow_no_wide_accesses(store):
    """Rows that start at odd elements: keys, values, queries and outputs of
    every call, against the same call on aligned copies."""
    P = kr.Pages([37], 3, 48, 5, "nhd", HF, store, seed=6)
    cache, plan = make_cache(P)
    wide = torch.randn(37, 6, 51, device="cuda").to(HF)
    k, v = wide[:, :3, 1:49], wide[:, 3:, 3:51]
    rope = lm.RopePlan(48, 40)
    angles = torch.empty(64, 40, device="cuda")
    lm.rope_table(rope, angles)
    pos = torch.arange(37, device="cuda")
    slots = pos + 2
    pages = torch.arange(P.pool).int()[None].cuda()
    lens, starts = torch.tensor([39]).int().cuda(), \
        torch.tensor([0, 39]).int().cuda()
    got = []
    for a, b in ((k, v), (k.contiguous(), v.contiguous())):
        for turn in ({}, {"rope": rope, "positions": pos, "table": angles}):
            cache.k.fill_(0), cache.v.fill_(0)
            lm.kv_write(cache, a, b, slots, **turn)
            out = torch.full((2, 39, 3, 49), 2.0, dtype=HF, device="cuda")
            dense = torch.empty(2, 39, 3, 48, dtype=HF, device="cuda")
            lm.kv_read(cache, pages, lens, starts, out[0, :, :, 1:],
                       out[1, :, :, 1:])
            lm.kv_read(cache, pages, lens, starts, dense[0], dense[1])
            assert (out[..., 0] == 2).all()
            assert torch.equal(out[:, 2:, :, 1:], dense[:, 2:])
            got.append(dense[:, 2:].clone())
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])
    assert not torch.equal(got[0][0], got[1][0])
    ws = torch.zeros(lm.kv_attend_workspace(plan, 1, 6), dtype=torch.uint8,
                     device="cuda")
    q = torch.randn(1, 6, 49, device="cuda").to(HF)
    odd, even = torch.zeros(1, 6, 49, dtype=HF, device="cuda"), \
        torch.zeros(1, 6, 48, dtype=HF, device="cuda")
    lm.kv_attend(cache, q[:, :, 1:], pages, lens, odd[:, :, 1:], ws)
    lm.kv_attend(cache, q[:, :, 1:].contiguous(), pages, lens, even, ws)
    assert torch.equal(odd[:, :, 1:], even) and (odd[:, :, 0] == 0).all()


def test_write_skips_tokens_whatever_their_position():
    P = kr.Pages([8], 2, 32, 4, "nhd", BF, "e4m3")
    cache, plan = make_cache(P)
    rope = lm.RopePlan(32)
    table = torch.ones(3, 32, device="cuda")
    x = torch.ones(2, 2, 32, dtype=BF, device="cuda")
    before = cache.k.clone()
    lm.kv_write(cache, x, x, torch.tensor([-1, -5]).cuda(), rope=rope,
                positions=torch.tensor([-1, 1 << 40]).cuda(), table=table)
    assert torch.equal(before, cache.k)      # and no status: see clean_status


def test_attend_without_pages():
    P = kr.Pages([0, 0], 2, 64, 16, "nhd", BF, None)
    P.table = torch.zeros(2, 0, dtype=torch.int32)
    q, out, lse = run_attend(P, 3, lens=[5, 0])
    assert (out == 0).all() and (lse == -math.inf).all()


def test_tensors_of_the_wrong_kind_are_refused():
    """What the binding itself checks, on tensors that are on the GPU; nothing
    is launched."""
    P = kr.Pages([20], 2, 64, 16, "nhd", BF, "int8")
    cache, plan = make_cache(P)
    rope = lm.RopePlan(64)
    angles = torch.zeros(8, 64, device="cuda")
    k = torch.zeros(20, 2, 64, dtype=BF, device="cuda")
    slots = torch.arange(20, device="cuda")
    pages, lens = P.table.cuda(), torch.tensor([20]).int().cuda()
    starts = torch.tensor([0, 20]).int().cuda()
    q = torch.zeros(1, 4, 64, dtype=BF, device="cuda")
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    lse = torch.zeros(1, 4, device="cuda")
    wrong = [
        lambda: lm.rope(rope, k, slots, angles, k[:, :1]),
        lambda: lm.rope(rope, k, slots, angles, k.float()),
        lambda: lm.rope(rope, k, slots[:5], angles, k),
        lambda: lm.rope(rope, k, slots.float(), angles, k),
        lambda: lm.rope(rope, k, slots, angles.half(), k),
        lambda: lm.rope(rope, k, slots, angles[:, :32], k),
        lambda: lm.rope(rope, k[..., ::2], slots, angles, k[..., ::2]),
        lambda: lm.rope(rope, k[0], slots, angles, k[0]),
        lambda: lm.kv_write(cache, k.half(), k.half(), slots),
        lambda: lm.kv_write(cache, k[:, :1], k[:, :1], slots),
        lambda: lm.kv_write(cache, k, k[:5], slots),
        lambda: lm.kv_write(cache, k, k, slots.int()),
        lambda: lm.kv_write(cache, k, k, slots, rope=rope),
        lambda: lm.kv_write(cache, k, k.cpu(), slots),
        lambda: lm.kv_read(cache, pages.long(), lens, starts, k, k),
        lambda: lm.kv_read(cache, pages, lens.long(), starts, k, k),
        lambda: lm.kv_read(cache, pages, lens, starts[:1], k, k),
        lambda: lm.kv_read(cache, pages, lens, starts, k, k.float()),
        lambda: lm.kv_read(cache, pages, lens, starts, k, k[:3]),
        lambda: lm.kv_attend(cache, q.half(), pages, lens, q, ws),
        lambda: lm.kv_attend(cache, q, pages[0], lens, q, ws),
        lambda: lm.kv_attend(cache, q, pages.t(), lens, q, ws),
        lambda: lm.kv_attend(cache, q, pages, starts, q, ws),
        lambda: lm.kv_attend(cache, q, pages, lens, q[:, :2], ws),
        lambda: lm.kv_attend(cache, q, pages, lens, q, ws[::2]),
        lambda: lm.kv_attend(cache, q, pages, lens, q, ws, lse=lse[:, :2]),
        lambda: lm.KVCache(plan, cache.k.to(BF), cache.v),
        lambda: lm.KVCache(plan, cache.k, cache.v, cache.k_scale),
        lambda: lm.rope_table(rope, angles[:, ::2]),
    ]
    for i, call in enumerate(wrong):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(i)
    with pytest.raises(lm.LayoutMoveError):    # keys heads do not divide
        lm.kv_attend(cache, q[:, :3], pages, lens, q[:, :3], ws)
    with pytest.raises(lm.LayoutMoveError):    # one buffer for both
        lm.kv_read(cache, pages, lens, starts, k, k)


def test_calls_in_a_graph():
    """A decoding step captured once and replayed with new inputs."""
    P = kr.Pages([60, 7], 2, 64, 16, "nhd", BF, "e4m3", seed=2)
    cache, plan = make_cache(P)
    rope = lm.RopePlan(64)
    table = torch.empty(128, 64, device="cuda")
    lm.rope_table(rope, table)
    x = torch.randn(2, 12, 64, device="cuda").to(BF)
    pos = torch.tensor([59, 6]).cuda()
    slots = torch.stack([P.table[0, 3].long() * 16 + 11,
                         P.table[1, 0].long() * 16 + 6]).cuda()
    pages, lens = P.table.cuda(), torch.tensor(P.lens).int().cuda()
    q, out = torch.empty(2, 8, 64, dtype=BF, device="cuda"), \
        torch.empty(2, 8, 64, dtype=BF, device="cuda")
    ws = torch.zeros(lm.kv_attend_workspace(plan, 2, 8), dtype=torch.uint8,
                     device="cuda")

    def step():
        lm.rope(rope, x[:, :8], pos, table, q)
        lm.kv_write(cache, x[:, 8:10], x[:, 10:], slots, rope=rope,
                    positions=pos, table=table)
        lm.kv_attend(cache, q, pages, lens, out, ws)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            step()
    torch.cuda.synchronize()
    for _ in range(3):
        x.copy_(torch.randn(2, 12, 64, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out)


def test_attend_strides_interleaved_pages_and_no_lse():
    P = kr.Pages([77, 300], 2, 64, 16, "nhd", BF, "int8", seed=8)
    q, out, lse = run_attend(P, 4, interleave=True, wide=True)
    check_attend(P, 4, q, out, lse)
    q2, out2, none = run_attend(P, 4, q=q, lse=False)
    assert torch.equal(out, out2)


def test_attend_in_place():
    P = kr.Pages([77, 3000, 0], 2, 64, 16, "nhd", BF, None, seed=8)
    q, want, _ = run_attend(P, 4)
    cache, plan = make_cache(P)
    ws = torch.zeros(lm.kv_attend_workspace(plan, 3, 8), dtype=torch.uint8,
                     device="cuda")
    x = q.cuda()
    lm.kv_attend(cache, x, P.table.cuda(), torch.tensor(P.lens).int().cuda(),
                 x, ws)
    assert torch.equal(x.cpu(), want)


def test_attend_lengths_beyond_the_table():
    """lens is clipped to the page table's tokens, and to 0 from below."""
    P = kr.Pages([40, 48, 20], 1, 64, 16, "nhd", BF, None, seed=2)
    table = P.table.clone()
    q, out, lse = run_attend(P, 2, lens=[40, 100000, -5])
    check_attend(P, 2, q, out, lse, rows=[40, 48, 0])


def test_attend_page_out_of_range():
    P = kr.Pages([64, 64, 64], 1, 64, 16, "nhd", BF, None, seed=2)
    table = P.table.clone()
    table[1, 2] = P.pool
    table[2, :] = -1
    q, out, lse = run_attend(P, 2, table=table)
    assert range_reported()
    keep = [0, 1, 3]
    for kv in range(2):
        r = P.rows[kv][1]
        P.rows[kv][1] = torch.cat([r[16 * i:16 * i + 16] for i in keep])
        P.rows[kv][2] = P.rows[kv][2][:0]
    check_attend(P, 2, q, out, lse)


@pytest.mark.parametrize("store", [None, "e4m3", "int8"])
def test_attend_extreme_scores(store):
    """Scores hundreds apart, and scales (of the softmax) that flatten or
    turn them."""
    P = kr.Pages([300, 5], 1, 64, 16, "nhd", BF, store, seed=4, mult=20.0)
    for scale in (0.0, 1.0, -0.5, 1e-6):
        q, out, lse = run_attend(P, 4, scale=scale)
        check_attend(P, 4, q, out, lse, scale=scale)


def test_attend_values_of_far_scales():
    """Tokens whose values differ by 10^12 in size, the large ones under
    weights that underflow or not: what is left of the small ones counts."""
    for store in ("e4m3", "int8"):
        P = kr.Pages([200], 1, 64, 16, "nhd", BF, store, seed=4)
        grow = torch.ones(200, dtype=torch.float64)
        grow[::7] = 1e6
        grow[3::7] = 1e-6
        P.rows[1][0] = P.rows[1][0] * grow[:, None, None].float().double()
        for j in range(200):
            p, o = int(P.table[0, j // 16]), j % 16
            P.scales[1][p, o] *= float(grow[j])
        # 32-bit scales: the rows as the cache holds them
        codes = P.codes[1].view(torch.uint8)
        vals = kr.e4m3_values()[codes.long()] if store == "e4m3" else \
            codes.view(torch.int8).double()
        vals = vals * P.scales[1].double()[..., None]
        P.rows[1][0] = torch.stack([
            vals[int(P.table[0, j // 16]), j % 16] for j in range(200)])
        q, out, lse = run_attend(P, 3)
        check_attend(P, 3, q, out, lse)


def test_attend_every_code():
    """A single token's values come back as what their codes stand for, the
    smallest (subnormal) codes beside the largest ones included; keys of all
    codes meet a query that picks one element."""
    for store in ("e4m3", "int8"):
        P = kr.Pages([1] * 64, 1, 256, 1, "nhd", BF, store, seed=4)
        codes = torch.arange(256, dtype=torch.uint8)
        codes[codes % 128 == 127] = 0 if store == "e4m3" else 127
        vals = kr.e4m3_values()[codes.long()] if store == "e4m3" else \
            codes.view(torch.int8).double()
        for b in range(64):
            p = int(P.table[b, 0])
            for kv, sc in ((0, 2.0 ** -5), (1, 2.0 ** (b - 40))):
                P.codes[kv].view(torch.uint8)[p, 0, 0] = codes
                P.scales[kv][p, 0, 0] = sc
                P.rows[kv][b] = (vals * sc)[None, None]
        q = torch.zeros(64, 5, 256, dtype=BF)
        for b in range(64):
            for h in range(4):
                q[b, h, 4 * b + h] = 1.5
        q, out, lse = run_attend(P, 5, q=q, scale=1.0)
        for b in range(64):
            want = P.rows[1][b][0]
            # one rounding of the result, and of 1 / l
            assert ((out[b].double() - want).abs() <=
                    want.abs() * (2.0 ** -8 + 2.0 ** -22)).all()
            s = vals[4 * b:4 * b + 4] * 2.0 ** -5 * 1.5
            # the factor of ln 2 and back: three roundings
            assert ((lse[b, :4].double() - s).abs() <=
                    s.abs() * 2.0 ** -21 + 2.0 ** -24).all()


def test_attend_infinite_and_nan_keys():
    """A key whose score is -infinity weighs nothing; all of them: zeros; a
    NaN key makes its own head group NaN and no other."""
    P = kr.Pages([20, 20, 20, 3], 2, 64, 16, "nhd", BF, None, seed=4)
    q = torch.ones(4, 4, 64).to(BF)
    big = -math.inf
    for b, rows in ((0, [4, 17]), (3, [0, 1, 2])):
        for j in rows:
            P.codes[0][int(P.table[b, j // 16]), j % 16] = big
            P.rows[0][b][j] = big
    P.codes[0][int(P.table[2, 0]), 3, 1, 5] = math.nan
    q, out, lse = run_attend(P, 2, q=q)
    assert out[2, 2:].isnan().all() and lse[2, 2:].isnan().all()
    out[2, 2:], lse[2, 2:] = 0, 0
    keep0 = [j for j in range(20) if j not in (4, 17)]
    for kv in range(2):
        P.rows[kv][0] = P.rows[kv][0][keep0]
        P.rows[kv][3] = P.rows[kv][3][:0]
    for b in (0, 1, 3):
        one = kr.attend(q[b].double(), P.rows[0][b], P.rows[1][b], 2,
                        64 ** -0.5)
        bo, bl = kr.attend_bounds(BF, 64, *one)
        assert ((out[b].double() - one[0]).abs() <= bo).all()
        assert torch.equal(lse[b] == -math.inf, one[1] == -math.inf)
    one = kr.attend(q[2, :2].double(), P.rows[0][2][:, :1],
                    P.rows[1][2][:, :1], 2, 64 ** -0.5)
    bo, bl = kr.attend_bounds(BF, 64, *one)
    assert ((out[2, :2].double() - one[0]).abs() <= bo).all()


@pytest.mark.parametrize("store", [None, "e4m3"])
def test_offsets_past_32_bits(store):
    """A cache whose last pages lie past 2^32 bytes and 2^31 elements."""
    P = kr.Pages([50], 8, 128, 16, "nhd", BF, store, seed=3, spare=0)
    per = 16 * 8 * 128
    pool = (1 << 31) // per + (1 << 31) // per * (store is not None) + 10
    held = BF if store is None else torch.uint8
    k = torch.empty(pool * per, dtype=held, device="cuda")
    v = torch.empty_like(k)
    scales = [None, None]
    if store:
        scales = [torch.ones(pool, 8, 16, device="cuda") for _ in range(2)]
    used = P.pool
    for kv, buf in enumerate((k, v)):
        buf[-used * per:] = P.device(kv).reshape(-1)
        if store:
            scales[kv][-used:] = P.device_scale(kv)
    plan = lm.KVPlan(lm.Layout.make(*P.page_layout()), BF, store)
    cache = lm.KVCache(plan, k, v, *scales)
    assert cache.pages == pool
    table = (P.table.clamp(min=0) + pool - used).cuda()
    lens = torch.tensor([50]).int().cuda()
    q = torch.randn(1, 16, 128).to(BF)
    out, ws = torch.empty(1, 16, 128, dtype=BF, device="cuda"), torch.zeros(
        lm.kv_attend_workspace(plan, 1, 16), dtype=torch.uint8, device="cuda")
    lm.kv_attend(cache, q.cuda(), table, lens, out, ws)
    check_attend(P, 2, q, out.cpu(), None)
    ko = torch.empty(50, 8, 128, dtype=BF, device="cuda")
    vo = torch.empty_like(ko)
    lm.kv_read(cache, table, lens, torch.tensor([0, 50]).int().cuda(), ko, vo)
    assert torch.equal(ko.cpu().double(), P.rows[0][0].to(BF).double())
    # write the rows back to the pages' own slots: nothing changes
    pos = torch.arange(50)
    slots = table[0].cpu().long()[pos // 16] * 16 + pos % 16
    lm.kv_write(cache, ko, vo, slots.cuda())
    lm.kv_read(cache, table, lens, torch.tensor([0, 50]).int().cuda(), vo, ko)
    assert torch.equal(vo.cpu().double(), P.rows[0][0].to(BF).double())


def test_decoding_steps_follow_the_dense_model():
    """Prompt write, then steps of rope -> write -> attend over a growing
    cache, against dense 64-bit attention on the turned keys."""
    g = torch.Generator().manual_seed(2)
    heads, group, dim, page, steps, prompt = 2, 3, 64, 4, 6, 9
    plan = lm.KVPlan(lm.Layout.make([page, heads, dim],
                                    [heads * dim, dim, 1], [1, 1, 1]), BF)
    k = torch.full((12, page, heads, dim), math.nan, dtype=BF, device="cuda")
    cache = lm.KVCache(plan, k, k.clone())
    rope = lm.RopePlan(dim)
    table = torch.empty(64, dim, device="cuda")
    lm.rope_table(rope, table)
    pages = torch.tensor([[7, 2, 11, 0]], dtype=torch.int32)
    ws = torch.zeros(lm.kv_attend_workspace(plan, 1, heads * group),
                     dtype=torch.uint8, device="cuda")
    n = prompt + steps
    x = torch.randn(3, n, heads * group, dim, generator=g).to(BF)
    q, kk, vv = x[0], x[1, :, :heads], x[2, :, :heads]
    pos = torch.arange(n)
    slots = pages[0].long()[pos // page] * page + pos % page
    def put(a, b):
        lm.kv_write(cache, kk[a:b].cuda(), vv[a:b].cuda(), slots[a:b].cuda(),
                    rope=rope, positions=pos[a:b].cuda(), table=table)
    put(0, prompt)
    kt = kr.turn(kk, pos, rope.frequencies()[0], dim, False)
    for j in range(prompt, n):
        put(j, j + 1)
        qt = torch.empty(1, heads * group, dim, dtype=BF, device="cuda")
        lm.rope(rope, q[j:j + 1].cuda(), pos[j:j + 1].cuda(), table, qt)
        out = torch.empty_like(qt)
        lm.kv_attend(cache, qt, pages.cuda(),
                     torch.tensor([j + 1]).int().cuda(), out, ws)
        want, lse, mag, dot = kr.attend(
            kr.turn(q[j:j + 1], pos[j:j + 1], rope.frequencies()[0], dim,
                    False)[0], kt[:j + 1], vv[:j + 1].double(), group,
            dim ** -0.5)
        # keys and queries rounded to bfloat16 after their turn: a score moves
        # by 2 * 2^-8 of its largest terms at most
        bo, _ = kr.attend_bounds(BF, dim, want, lse, mag, dot)
        bo = bo + 4 * 2.0 ** -8 * dot[:, None] * mag
        assert ((out[0].cpu().double() - want).abs() <= bo).all()


@pytest.mark.parametrize("store", [[], ["--store", "e4m3"],
                                   ["--store", "int8"]])
def test_the_example_runs(store):
    """examples/decode_cache.py: its outputs are bfloat16 (2^-8 of each,
    2^-9 in the mean) of the same cached rows, whose int8 values were rounded
    to bfloat16 on their way back."""
    import os
    import runpy
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    main = runpy.run_path(os.path.join(root, "examples", "decode_cache.py"))
    assert main["main"](store + ["--steps", "9"]) <= 2.0 ** -7
