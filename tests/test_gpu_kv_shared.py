"""The attention of sequences that share prefixes, on the GPU against the
attention over both key by key in 64 bits.

A shared weight is rounded once to 16 bits before it meets its value.  bfloat16
has 8 significant bits: a number in [2^n, 2^(n+1)) is held in steps of 2^(n-7),
so rounding is off by half of that, 2^(n-8), at most, 2^-8 of the number;
float16 has 11, so 2^-11 (rows of float16, and codes).  That is no more than as
much of sum p |v| together.  float16 weights, a code's times its scale, below
2^-24 of the largest (of the row's share of the work) are good to 2^-36 of it:
2^-36 max|v| a key, and twice that where the largest code of the largest scale
is not the format's.  A score is off by e as in kv_reference, a weight then by the factor
1 + 2e; 2^-10 covers the exponentials and the sums there, 2^-16 here (the sums
of up to 2^16 positive terms in 32 bits, in runs of 32, are good to 2^-17)."""

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


class Case:
    """Groups' prefixes and sequences' own tokens in one pool."""

    def __init__(self, shared, starts, lens, heads, group, dim, page, order,
                 dtype, store, seed=1, **kw):
        self.P = lr.Held(list(shared) + list(lens), heads, dim, page, order,
                         dtype, store, seed=seed, **kw)
        self.groups, self.shared, self.starts = len(shared), shared, starts
        self.lens, self.heads, self.group, self.dim = lens, heads, group, dim
        self.dtype, self.store = dtype, store
        g = torch.Generator().manual_seed(seed + 50)
        self.q = torch.randn(len(lens), heads * group, dim,
                             generator=g).to(dtype).cuda()
        self.table = self.P.table.cuda()

    def run(self, q=None, out=None, workspace=None, scale=None, stream=None,
            lse=True):
        cache, plan = self.P.cache(lm)
        q = self.q if q is None else q
        out = torch.full_like(q, math.nan) if out is None else out
        ld = torch.full(q.shape[:2], math.nan, device="cuda") if lse else None
        if workspace is None:
            workspace = space(lm.kv_attend_shared_workspace(plan,
                                                            *q.shape[:2]))
        numbers = [ints(x) for x in (self.shared, self.starts, self.lens)]
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        lm.kv_attend_shared(
            cache, q, self.table[:self.groups], *numbers[:2],
            self.table[self.groups:], numbers[2], out, workspace, lse=ld,
            scale=scale, stream=stream)
        torch.cuda.synchronize()
        return out, ld

    def rows(self, b):
        """The keys and values that sequence b sees, in 64 bits."""
        own = [self.P.seq(kv, self.groups + b) for kv in (0, 1)]
        for g in range(self.groups):
            if self.starts[g] <= b < self.starts[g + 1]:
                return [torch.cat([self.P.seq(kv, g), own[kv]])
                        for kv in (0, 1)]
        return own

    def check(self, out, lse, scale=None, q=None):
        q = self.q if q is None else q
        scale = self.dim ** -0.5 if scale is None else scale
        half = self.store is not None or self.dtype == HF
        step = 2.0 ** -11 if half else 2.0 ** -8
        for b in range(len(self.lens)):
            k, v = self.rows(b)
            want, wl, _, mag, dot = lr.attend(q[b].double(), k, v, self.group,
                                              scale)
            bo, bl = kr.attend_bounds(self.dtype, self.dim, want, wl, mag, dot)
            bo += (step - 2.0 ** -10 + 2.0 ** -16) * mag
            if half and len(v):
                bo += len(v) * 2.0 ** -35 * v.abs().max()
            assert ((out[b].double() - want).abs() <= bo).all(), b
            if lse is None:
                continue
            empty = wl == -math.inf
            assert (lse[b][empty] == -math.inf).all()
            assert ((lse[b].double() - wl).abs() <= bl)[~empty].all(), b


SMALL = [
    # shared, starts, lens, heads, group, dim, page, order, dtype, store
    ([40], [0, 2], [5, 0], 1, 1, 64, 16, "nhd", BF, None),
    ([128], [0, 3], [0, 0, 0], 2, 4, 128, 16, "nhd", BF, None),
    ([300, 0, 1], [0, 2, 3, 7], [9, 1, 4, 0, 70, 3, 2], 2, 4, 128, 16, "hnd",
     BF, None),
    ([129, 1000], [1, 3, 5], [7, 3, 0, 2, 40, 11], 3, 5, 80, 24, "nhd", HF,
     None),
    ([257, 64], [0, 17, 20], [3] * 20, 1, 16, 128, 5, "nhd", BF, None),
    ([500], [0, 33], [i % 7 for i in range(33)], 2, 8, 64, 1, "nhd", HF, None),
    ([200, 65, 63], [0, 1, 2, 3], [1, 2, 3], 2, 3, 256, 32, "hnd", BF, None),
    ([300], [0, 50], [2] * 50, 1, 4, 256, 7, "nhd", HF, None),
    ([90, 70], [0, 4, 8], [4] * 8, 2, 2, 8, 16, "nhd", BF, None),
    ([90, 170], [0, 4, 8], [4] * 8, 1, 40, 24, 16, "hnd", HF, None),
    ([400, 130], [0, 3, 9], [4, 0] * 4 + [30], 2, 4, 128, 16, "nhd", BF,
     "e4m3"),
    ([400, 130], [0, 3, 9], [4, 0] * 4 + [30], 2, 4, 128, 64, "hnd", HF,
     "e4m3"),
    ([1000], [0, 40], [i % 5 for i in range(40)], 2, 8, 80, 24, "nhd", BF,
     "int8"),
    ([1000], [0, 40], [i % 5 for i in range(40)], 1, 5, 64, 40, "hnd", HF,
     "int8"),
    ([200, 65], [0, 1, 3], [1, 2, 3], 2, 3, 256, 32, "hnd", BF, "int8"),
    ([200, 65], [0, 1, 3], [1, 2, 3], 1, 9, 240, 3, "nhd", HF, "e4m3"),
    ([100] * 30, list(range(0, 62, 2)), [1] * 60, 1, 2, 112, 20, "nhd", BF,
     None),
    ([7, 5], [0, 0, 0], [3, 2], 1, 2, 64, 4, "nhd", BF, None),
]


@pytest.mark.parametrize("case", SMALL, ids=str)
def test_shared_prefixes(case):
    C = Case(*case)
    out, lse = C.run()
    C.check(out, lse)
    # the same inputs give the same bits, on a stream of one's own too
    out2, lse2 = C.run(stream=torch.cuda.Stream())
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


LONG = [
    ([20011], [0, 40], [33] * 40, 2, 4, 128, 16, "nhd", BF, None),
    ([20011, 5000], [0, 70, 90], [3] * 90, 1, 8, 128, 64, "hnd", BF, "e4m3"),
    ([9000, 3000], [0, 30, 70], [3] * 70, 2, 5, 80, 24, "nhd", HF, None),
    ([12000], [0, 5], [100, 0, 3000, 1, 1], 4, 4, 64, 40, "nhd", HF, "int8"),
    ([6000], [0, 70], [1] * 70, 2, 4, 256, 16, "nhd", BF, None),
    ([60000], [0, 2], [5, 6], 1, 1, 128, 16, "nhd", BF, None),
]


@pytest.mark.parametrize("case", LONG, ids=str)
def test_long_prefixes(case):
    """Prefixes that many blocks share, of rows in one tile or several."""
    C = Case(*case)
    out, lse = C.run()
    C.check(out, lse)


@pytest.mark.parametrize("lens", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256,
                                  257])
def test_prefix_lengths(lens):
    for dim, dtype, store in ((128, BF, None), (256, HF, None),
                              (64, BF, "int8")):
        C = Case([lens], [0, 3], [1, 0, 2], 2, 3, dim, 16, "nhd", dtype, store)
        C.check(*C.run())


def test_rows_of_every_number():
    """1 to 260 rows a key head: one tile of rows or two, in halves or not."""
    for seqs in (1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 130):
        C = Case([300], [0, seqs], [1] * seqs, 1, 2, 64, 16, "nhd", BF, None)
        C.check(*C.run())


def test_strides_in_place_and_no_lse():
    C = Case([300, 20], [0, 3, 5], [5, 0, 40, 1, 2], 2, 4, 64, 16, "nhd", BF,
             None)
    out, lse = C.run()
    n, hq, d = C.q.shape
    wide = torch.full((n, hq + 3, d + 8), 3.0, dtype=BF, device="cuda")
    res = torch.full_like(wide, 9.0)
    for at in (0, 3):                            # 3: no wide loads
        qd = wide[:, 1:hq + 1, at:at + d]
        wide.fill_(3)
        res.fill_(9)
        qd.copy_(C.q)
        od = res[:, 1:hq + 1, at:at + d]
        C.run(q=qd, out=od, lse=False)
        assert torch.equal(od, out)
        od.fill_(9)
        assert (res == 9).all()
    q = C.q.clone()
    C.run(q=q, out=q)
    assert torch.equal(q, out)
    t = C.q.transpose(0, 1).contiguous().transpose(0, 1)
    o, _ = C.run(q=t)
    assert torch.equal(o, out)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scales(scale):
    C = Case([300, 200], [0, 3, 80], [3] * 80, 1, 4, 64, 16, "nhd", BF, None)
    C.check(*C.run(scale=scale), scale=scale)
    C = Case([300, 200], [0, 3, 80], [3] * 80, 1, 4, 64, 16, "nhd", HF, "int8")
    C.check(*C.run(scale=scale), scale=scale)


def test_a_workspace_serves_call_after_call_and_other_calls():
    C = Case([5000, 40], [0, 9, 12], [5] * 12, 2, 4, 128, 16, "nhd", BF, None)
    cache, plan = C.P.cache(lm)
    ws = space(lm.kv_attend_shared_workspace(plan, 12, 8))
    first = C.run(workspace=ws)
    C.check(*first)
    D = Case([900], [0, 3], [5, 2000, 0], 1, 4, 128, 16, "hnd", BF, None)
    D.check(*D.run(workspace=ws))
    out = torch.empty_like(C.q)
    lm.kv_attend(cache, C.q, C.table[2:], ints(C.lens), out, ws)
    again = C.run(workspace=ws)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_no_groups_and_no_pages():
    C = Case([64], [0, 2], [5, 0], 1, 2, 64, 16, "nhd", BF, None)
    cache, plan = C.P.cache(lm)
    ws = space(lm.kv_attend_shared_workspace(plan, 2, 2))
    plain, out = torch.empty_like(C.q), torch.empty_like(C.q)
    lm.kv_attend(cache, C.q, C.table[1:], ints([5, 0]), plain, ws)
    for table, lens, starts in ((C.table[:0], [], [0]),
                                (C.table[:1, :0], [9], [0, 2])):
        out.fill_(7)
        lm.kv_attend_shared(cache, C.q, table, ints(lens), ints(starts),
                            C.table[1:], ints([5, 0]), out, ws)
        assert torch.equal(out, plain)
    out.fill_(7)
    lm.kv_attend_shared(cache, C.q, C.table[:1], ints([0]), ints([0, 2]),
                        C.table[1:, :0], ints([5, 9]), out, ws)
    assert (out == 0).all()


def test_lengths_starts_and_pages_out_of_range():
    """Lengths and starts are clipped; keys of pages that are not there are not
    seen, whatever tile they lie in."""
    C = Case([600], [0, 3], [1, 2, 3], 1, 4, 64, 16, "nhd", BF, None)
    out, lse = C.run()
    C.starts = [-5, 1 << 30]
    C.shared = [600]
    full = C.run()
    assert torch.equal(full[0], out)
    C.starts = [0, 3]
    table = C.table.clone()
    C.table[0, 3:20] = torch.tensor([-1, 1 << 30] * 8 + [C.P.pool],
                                    dtype=torch.int32)
    got, gl = C.run()
    assert lm.device_status(reset=True) == -12
    keep = torch.ones(600, dtype=torch.bool, device="cuda")
    keep[48:320] = False
    for b in range(3):
        k, v = C.rows(b)
        mask = torch.cat([keep, torch.ones(C.lens[b], dtype=torch.bool,
                                           device="cuda")])
        want, wl, _, mag, dot = lr.attend(C.q[b].double(), k[mask], v[mask],
                                          4, 64 ** -0.5)
        bo, bl = kr.attend_bounds(BF, 64, want, wl, mag, dot)
        bo += 2.0 ** -8 * mag
        assert ((got[b].double() - want).abs() <= bo).all()
        assert ((gl[b].double() - wl).abs() <= bl).all()
    C.table = table
    C.shared = [-4]
    none, _ = C.run()
    cache, plan = C.P.cache(lm)
    own = torch.empty_like(C.q)
    lm.kv_attend(cache, C.q, C.table[1:], ints(C.lens), own,
                 space(lm.kv_attend_workspace(plan, 3, 4)))
    # (the join multiplies a mean by l / l: a rounding to the next one of 16
    # bits at most)
    assert ((none.double() - own.double()).abs()
            <= own.double().abs() * 2.0 ** -7).all()


def set_row(C, kv, g, j, row):
    page = int(C.P.table[g, j // C.P.page])
    x = C.P.held[kv]
    (x if C.P.order == "nhd" else x.transpose(1, 2))[page, j % C.P.page] = row
    C.P.rows[kv][page, j % C.P.page] = row.double()


def test_scores_far_apart():
    """Scores that grow along the prefix, so that every tile moves its rows'
    references; one key that outweighs all; none that is below the others."""
    for dtype in (BF, HF):
        C = Case([1000], [0, 40], [2] * 40, 1, 4, 64, 16, "nhd", dtype, None)
        for j in range(1000):
            set_row(C, 0, 0, j, torch.full((1, 64), j / 1000).to(dtype).cuda())
        C.q.fill_(1)
        C.check(*C.run(scale=3.0), scale=3.0)
        C.check(*C.run(scale=-3.0), scale=-3.0)


def test_largest_values_stay_finite():
    top = torch.finfo(BF).max
    C = Case([700], [0, 40], [2] * 40, 1, 4, 64, 16, "nhd", BF, None)
    for j in range(700):
        set_row(C, 1, 0, j, torch.full((1, 64), top).to(BF).cuda())
    C.check(*C.run())


def test_scales_of_values_far_apart():
    """Value scales over 2^-90 .. 2^90 in one prefix, the largest last."""
    C = Case([512], [0, 40], [0] * 40, 1, 4, 64, 16, "nhd", BF, "int8")
    pages = C.P.table[0, :32].long().cuda()
    s = torch.exp2(torch.linspace(-90, 90, 512, device="cuda").round())
    C.P.scales[1][pages, 0] = s.view(32, 16)
    code = C.P.held[1][pages].double()
    C.P.rows[1][pages] = code * s.view(32, 16, 1, 1).double()
    C.check(*C.run())


def test_infinite_scores_and_no_numbers():
    C = Case([300], [0, 40], [3] * 40, 1, 2, 64, 16, "nhd", BF, None)
    C.q.fill_(1)
    row = torch.zeros(1, 64, dtype=BF, device="cuda")
    row[0, 0] = -math.inf
    for j in range(130):                   # a whole tile that is not seen
        set_row(C, 0, 0, j, row)
    C.P.rows[0][C.P.rows[0] == -math.inf] = -1e30     # (times 0 is no number)
    C.check(*C.run())
    set_row(C, 0, 0, 200, row.fill_(math.nan))
    out, lse = C.run()
    assert out.isnan().all() and lse.isnan().all()
    # garbage behind the prefix is not used
    C = Case([300], [0, 40], [3] * 40, 1, 2, 64, 16, "nhd", BF, None)
    assert not C.run()[0].isnan().any()


def test_e4m3_codes_that_are_no_numbers():
    C = Case([300], [0, 3], [3] * 3, 1, 2, 64, 16, "nhd", BF, "e4m3")
    page = int(C.P.table[0, 2])
    C.P.held[1][page, 5, 0, 9] = 0x7f
    out, lse = C.run()
    assert out[:, :, 9].isnan().all() and not lse.isnan().any()
    assert not out[:, :, :9].isnan().any() and not out[:, :, 10:].isnan().any()
    C.P.held[0][page, 5, 0, 9] = 0xff
    out, lse = C.run()
    assert out.isnan().all() and lse.isnan().all()


def test_captured_and_replayed():
    C = Case([3000], [0, 20], [30] * 20, 2, 4, 128, 16, "nhd", BF, None)
    cache, plan = C.P.cache(lm)
    ws = space(lm.kv_attend_shared_workspace(plan, 20, 8))
    out, lse = torch.empty_like(C.q), torch.empty(20, 8, device="cuda")
    args = (cache, C.q, C.table[:1], ints([3000]), ints([0, 20]), C.table[1:],
            ints(C.lens), out, ws)
    lm.kv_attend_shared(*args, lse=lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lm.kv_attend_shared(*args, lse=lse)
    C.q.copy_(C.q.flip(0))
    out.zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    C.check(out, lse)
