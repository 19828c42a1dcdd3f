"""The paged cache's and the rotary plans' host side: plans, frequencies and
every refusal, through the C ABI with buffers that are never touched (all
checks come before a launch; no GPU needed)."""

import ctypes as C
import math

import pytest

lm = pytest.importorskip("layout_driven_movement_gb300")

INVALID, NOT_REP, NOT_INJ, OVERFLOW, CAPACITY, OVERLAP, BUFFER = \
    -1, -3, -4, -5, -6, -7, -11
BF, HF, FL = "torch.bfloat16", "torch.float16", "torch.float32"
BASE = 1 << 40                     # addresses that nothing dereferences


@pytest.fixture(scope="module", autouse=True)
def built():
    from layout_driven_movement_gb300 import _build
    _build.build()
    lm.lib()


def status(fn, *a, **k):
    with pytest.raises(lm.LayoutMoveError) as e:
        fn(*a, **k)
    return e.value.status


def page(text="(16,8,128):(1024,128,1)"):
    return lm.Layout.parse(text)


# --- plans -----------------------------------------------------------------

def test_frequencies_follow_the_formulas():
    n, base = 64, 10000.0
    plain = [base ** (-2 * i / n) for i in range(32)]
    def close(plan, want, amp=1.0):
        f, a = plan.frequencies()
        assert len(f) == len(want)
        assert all(abs(x - y) <= 1e-14 * y for x, y in zip(f, want))
        assert abs(a - amp) < 1e-15
    close(lm.RopePlan(128, n), plain)
    close(lm.RopePlan(128, n, scaling="linear", factor=4.0),
          [f / 4 for f in plain])
    b = base * 8.0 ** (64 / 62)
    close(lm.RopePlan(128, n, scaling="ntk", factor=8.0),
          [b ** (-2 * i / n) for i in range(32)])
    want = []
    for f in plain:
        g = min(1.0, max(0.0, (4096 * f / (2 * math.pi) - 1) / 31))
        want.append((1 - g) * f / 16 + g * f)
    close(lm.RopePlan(128, n, scaling="yarn", factor=16.0,
                      original_positions=4096), want,
          0.1 * math.log(16) + 1)
    # fast pairs keep their turn, slow ones are interpolated
    assert want[0] == plain[0] and want[-1] == plain[-1] / 16


@pytest.mark.parametrize("args,kw", [
    ((1,), {}), ((1026,), {}), ((64, 63), {}), ((64, 66), {}), ((64, 0), {}),
    ((64,), {"base": 1.0}), ((64,), {"base": math.inf}),
    ((64,), {"scaling": "linear", "factor": 0.5}),
    ((64,), {"scaling": "linear", "factor": math.nan}),
    ((64,), {"scaling": "other"}),
    ((64, 2), {"scaling": "ntk", "factor": 2.0}),
    ((64,), {"scaling": "yarn", "factor": 2.0}),
    ((64,), {"scaling": "yarn", "factor": 2.0, "original_positions": 9,
             "beta_fast": 1.0, "beta_slow": 1.0}),
    ((64,), {"scaling": "yarn", "factor": 2.0, "original_positions": 9,
             "beta_slow": -1.0}),
])
def test_rope_plan_refusals(args, kw):
    assert status(lm.RopePlan, *args, **kw) == INVALID


def test_frequencies_buffer():
    p = lm.RopePlan(64)
    f = (C.c_double * 4)()
    assert lm.lib().lm_rope_plan_frequencies(p.handle, f, 4, None) == BUFFER
    assert lm.lib().lm_rope_plan_frequencies(None, f, 4, None) == INVALID


def test_kv_plan_describes_itself():
    d = lm.KVPlan(page("(16,8,80):(80,1280,1)"), HF, "int8").describe()
    assert d == {"page_tokens": 16, "heads": 8, "dim": 80,
                 "page": "(16,8,80):(80,1280,1)", "page_stride": 10240,
                 "elem": "f16", "store": "int8", "held_bytes": 1}
    # the page's cosize, rounded up to 16 bytes of held elements
    assert lm.KVPlan(page("(3,1,24):(24,24,1)"), BF).page_stride == 72
    assert lm.KVPlan(page("(3,2,16):(48,16,1)"), BF, "e4m3").page_stride == 128
    assert lm.KVPlan(page(), BF, page_stride=32768).page_stride == 32768


@pytest.mark.parametrize("text,dtype,store,stride,want", [
    ("(16,8,128):(1024,128,1)", FL, None, 0, INVALID),
    ("(16,8,128):(1024,128,1)", BF, "fp4", 0, INVALID),
    ("(16,8,128):(1024,128,1)", BF, None, 16376, INVALID),     # too small
    ("(16,8,128):(1024,128,1)", BF, None, 16388, NOT_REP),
    ("(16,1024):(1024,1)", BF, None, 0, INVALID),
    ("((4,4),8,128):((1024,4096),128,1)", BF, None, 0, INVALID),
    ("(16,0,128):(1024,128,1)", BF, None, 0, INVALID),
    ("(16,8,264):(2112,264,1)", BF, None, 0, INVALID),
    ("(16,8,128):(1,16,128)", BF, None, 0, NOT_REP),           # dim strided
    ("(16,8,12):(96,12,1)", BF, None, 0, NOT_REP),
    ("(16,8,24):(192,24,1)", BF, "e4m3", 0, NOT_REP),          # 24 bytes
    ("(16,8,16):(132,16,1)", BF, None, 0, NOT_REP),
    ("(16,8,128):(512,128,1)", BF, None, 0, NOT_INJ),
    ("Sw<3,3,3> o (16,8,128):(1024,128,1)", BF, None, 0, NOT_REP),
])
def test_kv_plan_refusals(text, dtype, store, stride, want):
    assert status(lm.KVPlan, page(text), dtype, store, stride) == want


# --- calls -----------------------------------------------------------------

def rows(data=BASE, capacity=1 << 30, ts=1024, hs=128):
    return lm._Rows(data, capacity, ts, hs)


def cache(k=BASE * 2, v=BASE * 3, cap=1 << 20, ks=BASE * 4, vs=BASE * 5,
          scap=1 << 20, pages=64):
    return lm._KVCache(k, v, cap, cap, ks, vs, scap, pages)


def call_rope(plan=None, elem=1, x=None, out=None, tokens=4, heads=8,
              pos=BASE * 6, pb=8, table=BASE * 7, trows=100):
    plan = plan or lm.RopePlan(128)
    return lm.lib().lm_rope(plan.handle, elem, x or rows(),
                            out or rows(BASE * 8), tokens, heads, pos, pb,
                            table, trows, 0, None)


@pytest.mark.parametrize("kw,want", [
    ({"elem": 0}, INVALID), ({"elem": 4}, INVALID), ({"tokens": -1}, INVALID),
    ({"heads": -1}, INVALID), ({"pb": 2}, INVALID), ({"pos": None}, INVALID),
    ({"table": None}, INVALID), ({"trows": -1}, INVALID),
    ({"pos": BASE + 4}, INVALID), ({"table": BASE + 2}, INVALID),
    ({"x": rows(None)}, INVALID), ({"x": rows(BASE + 1)}, INVALID),
    ({"x": rows(ts=-1)}, INVALID), ({"x": rows(capacity=4095)}, CAPACITY),
    ({"out": rows(BASE * 8, 4095)}, CAPACITY),
    ({"out": rows(BASE * 8, ts=0)}, INVALID),
    ({"out": rows(BASE * 8, hs=64)}, INVALID),
    ({"out": rows(BASE * 8, ts=1000)}, INVALID),     # tokens run into heads
    ({"out": rows(BASE + 256)}, OVERLAP),
    ({"out": rows(BASE, ts=2048)}, OVERLAP),
    ({"x": rows(ts=1 << 62)}, OVERFLOW),
])
def test_rope_refusals(kw, want):
    assert call_rope(**kw) == want


def test_rope_of_nothing_is_ok():
    assert call_rope(tokens=0) == 0 and call_rope(heads=0) == 0
    assert lm.lib().lm_rope(None, 1, rows(), rows(), 1, 1, 1, 8, 1, 1, 0,
                            None) == INVALID


def test_rope_table_refusals():
    p = lm.RopePlan(64)
    f = lm.lib().lm_rope_table
    assert f(p.handle, BASE, -1, 10, None) == INVALID
    assert f(p.handle, None, 1, 64, None) == INVALID
    assert f(p.handle, BASE, 2, 127, None) == CAPACITY
    assert f(None, BASE, 1, 64, None) == INVALID
    assert f(p.handle, None, 0, 0, None) == 0


def plan_of(store=None):
    return lm.KVPlan(page(), BF, store)


def call_write(store=None, c=None, k=None, v=None, tokens=4, slots=BASE * 6,
               rope=None, pos=BASE * 7, pb=8, table=BASE * 8, trows=9):
    p = plan_of(store)
    return lm.lib().lm_kv_write(
        p.handle, c or cache(), k or rows(), v or rows(BASE + (1 << 30)),
        tokens, slots, rope.handle if rope else None, pos, pb, table, trows,
        None)


@pytest.mark.parametrize("kw,want", [
    ({"tokens": -1}, INVALID), ({"slots": None}, INVALID),
    ({"slots": BASE + 4}, INVALID), ({"k": rows(None)}, INVALID),
    ({"k": rows(capacity=100)}, CAPACITY),
    ({"v": rows(capacity=100)}, CAPACITY),
    ({"k": rows(BASE * 2 + 64)}, OVERLAP), ({"v": rows(BASE * 3)}, OVERLAP),
    ({"c": cache(k=None)}, INVALID), ({"c": cache(k=BASE * 2 + 8)}, INVALID),
    ({"c": cache(v=BASE * 2)}, OVERLAP), ({"c": cache(pages=0)}, INVALID),
    ({"c": cache(pages=65)}, CAPACITY),
    ({"c": cache(pages=1 << 60)}, OVERFLOW),
    ({"store": "e4m3", "c": cache(ks=None)}, INVALID),
    ({"store": "e4m3", "c": cache(vs=BASE + 2)}, INVALID),
    ({"store": "int8", "c": cache(scap=8191)}, CAPACITY),
    ({"store": "int8", "c": cache(vs=BASE * 4)}, OVERLAP),
    ({"rope": 64}, INVALID), ({"rope": 128, "pos": None}, INVALID),
    ({"rope": 128, "table": None}, INVALID),
    ({"rope": 128, "pb": 1}, INVALID),
])
def test_write_refusals(kw, want):
    kw = dict(kw)
    if "rope" in kw:
        kw["rope"] = lm.RopePlan(kw["rope"])
    assert call_write(**kw) == want


def call_read(store=None, c=None, table=BASE * 6, stride=9, seqs=3, pages=9,
              lens=BASE * 7, starts=BASE * 8, elem=1, k=None, v=None, n=100):
    p = plan_of(store)
    return lm.lib().lm_kv_read(p.handle, c or cache(), table, stride, seqs,
                               pages, lens, starts, elem, k or rows(),
                               v or rows(BASE + (1 << 40)), n, None)


@pytest.mark.parametrize("kw,want", [
    ({"elem": 9}, INVALID), ({"n": -1}, INVALID), ({"table": None}, INVALID),
    ({"lens": None}, INVALID), ({"starts": None}, INVALID),
    ({"seqs": -1}, INVALID), ({"stride": 8}, INVALID),
    ({"table": BASE + 1}, INVALID), ({"starts": BASE + 1}, INVALID),
    ({"pages": 1 << 28, "stride": 1 << 28}, OVERFLOW),
    ({"n": 1 << 31}, OVERFLOW), ({"k": rows(capacity=100)}, CAPACITY),
    ({"k": rows(ts=512)}, INVALID), ({"k": rows(BASE + (1 << 40))}, OVERLAP),
    ({"v": rows(BASE * 3)}, OVERLAP), ({"c": cache(pages=65)}, CAPACITY),
])
def test_read_refusals(kw, want):
    assert call_read(**kw) == want


def test_read_and_write_of_nothing():
    assert call_read(n=0) == 0 and call_read(seqs=0) == 0
    assert call_read(pages=0) == 0 and call_write(tokens=0) == 0


def call_attend(store=None, c=None, q=None, out=None, seqs=3, hq=32,
                table=BASE * 6, stride=9, pages=9, lens=BASE * 7, window=0,
                scale=0.1, lse=BASE * 9, ws=BASE * 10, wsb=0):
    p = plan_of(store)
    return lm.lib().lm_kv_attend(
        p.handle, c or cache(), q or rows(ts=4096),
        out or rows(BASE * 12, ts=4096), seqs, hq, table, stride, pages, lens,
        window, scale, lse, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    ({"hq": 0}, INVALID), ({"hq": 12}, INVALID), ({"hq": 1 << 21}, INVALID), ({"seqs": -1}, INVALID),
    ({"scale": math.inf}, INVALID), ({"scale": math.nan}, INVALID),
    ({"window": -1}, INVALID), ({"table": None}, INVALID),
    ({"lens": None}, INVALID), ({"stride": 3}, INVALID),
    ({"lse": BASE + 2}, INVALID), ({"q": rows(None)}, INVALID),
    ({"q": rows(capacity=100)}, CAPACITY),
    ({"out": rows(BASE * 12, 100)}, CAPACITY),
    ({"out": rows(BASE * 12, ts=1024)}, INVALID),
    ({"out": rows(BASE + 256, ts=4096)}, OVERLAP),
    ({"out": rows(BASE * 2, ts=4096)}, OVERLAP),
    ({"c": cache(pages=65)}, CAPACITY),
    ({"pages": 1 << 28, "stride": 1 << 28}, OVERFLOW),
])
def test_attend_refusals(kw, want):
    assert call_attend(**kw) == want


def test_attend_of_nothing_and_null_handles():
    assert call_attend(seqs=0) == 0
    L = lm.lib()
    n = C.c_int64()
    assert L.lm_kv_attend_workspace(None, 1, 8, C.byref(n)) == INVALID
    p = plan_of()
    assert L.lm_kv_attend_workspace(p.handle, 1, 9, C.byref(n)) == INVALID
    assert L.lm_kv_attend_workspace(p.handle, -1, 8, C.byref(n)) == INVALID
    assert L.lm_kv_attend_workspace(p.handle, 1, 8, None) == INVALID
    L.lm_kv_plan_destroy(None)
    L.lm_rope_plan_destroy(None)
    out = C.c_void_p(1)
    assert L.lm_kv_plan_create(None, 0, 1, 0, C.byref(out)) == INVALID
    assert not out.value
    assert L.lm_kv_plan_create(page().handle, 0, 1, 0, None) == INVALID


def test_python_checks_before_the_library():
    torch = pytest.importorskip("torch")
    plan = lm.RopePlan(64)
    x = torch.zeros(2, 3, 64)
    with pytest.raises(ValueError):
        lm.rope(plan, x, torch.zeros(2), torch.zeros(4, 64), x)   # not CUDA
    with pytest.raises(ValueError):
        lm.rope(plan, None, None, None, None)
    with pytest.raises(ValueError):
        lm.rope(plan, x, torch.zeros(2), torch.zeros(4, 64), x[:1])
    with pytest.raises(ValueError):
        lm.rope_table(plan, torch.zeros(4, 64))
    with pytest.raises(ValueError):
        lm.KVCache(lm.KVPlan(page(), torch.bfloat16), x, x)
    with pytest.raises(ValueError):
        lm.KVPlan(page(), torch.int32)
    for fn in ("rope", "kv_write", "kv_read", "kv_attend"):
        with pytest.raises(TypeError):
            getattr(lm._pycall(), fn)(1, 2)
