"""Outputs of the paged cache's read back that share a buffer but no element:
every form that the refusals (test_kv_overlap_host.py) leave open."""

import pytest

import kv_reference as kr
from test_gpu_kv import BF, built, clean_status, make_cache  # noqa: F401

torch = pytest.importorskip("torch")
lm = pytest.importorskip("layout_driven_movement_gb300")

pytestmark = pytest.mark.gpu


def views(name, n, h, d):
    """(the buffer, k_out, v_out), both [n, h, d]."""
    def full(*shape):
        return torch.full(shape, 5.0, dtype=BF, device="cuda")
    if name == "tokens one after the other":
        b = full(2, n, h, d)
        return b, b[0], b[1]
    if name == "values first":
        b = full(2, n, h, d)
        return b, b[1], b[0]
    if name == "side by side":
        b = full(n, 2, h, d)
        return b, b[:, 0], b[:, 1]
    if name == "every other head":
        b = full(n, h, 2, d)
        return b, b[:, :, 1], b[:, :, 0]
    if name == "within a row":
        b = full(n, h, 2 * d)
        return b, b[..., :d], b[..., d:]
    if name == "heads of different distances":
        b = full(n, 3 * h, d)
        return b, b[:, :2 * h:2], b[:, 2 * h:]
    if name == "heads before tokens":
        b = full(2 * h, n, d)
        return b, b[::2].transpose(0, 1), b[1::2].transpose(0, 1)
    if name == "tokens taken in turn":
        b = full(2 * n, h, d)
        return b, b[::2], b[1::2]
    raise KeyError(name)


@pytest.mark.parametrize("name", [
    "tokens one after the other", "values first", "side by side",
    "every other head", "within a row", "heads of different distances",
    "heads before tokens", "tokens taken in turn"])
@pytest.mark.parametrize("lens,heads", [([9, 20], 4), ([1], 3), ([5], 1)])
def test_read_into_one_buffer(name, lens, heads):
    P = kr.Pages(lens, heads, 32, 8, "nhd", BF, None, seed=2)
    cache, plan = make_cache(P)
    n = sum(lens)
    buf, k, v = views(name, n, heads, 32)
    starts = [sum(lens[:i]) for i in range(len(lens) + 1)]
    lm.kv_read(cache, P.table.cuda(), torch.tensor(lens).int().cuda(),
               torch.tensor(starts).int().cuda(), k, v)
    for kv, got in enumerate((k, v)):
        assert torch.equal(got.cpu().double(), torch.cat(P.rows[kv]))
    rest = int((buf == 5.0).sum())
    assert rest >= buf.numel() - 2 * n * heads * 32


@pytest.mark.parametrize("what", ["lse", "q", "out", "pages", "scales"])
def test_workspace_that_meets(what):
    """Refused before the launch: the buffers are as they were."""
    P = kr.Pages([20], 2, 64, 16, "nhd", BF, "int8", seed=2)
    cache, plan = make_cache(P)
    n = lm.kv_attend_workspace(plan, 1, 4)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    inside = ws[n // 2:n // 2 + 512]
    q = torch.zeros(1, 4, 64, dtype=BF, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(1, 4, device="cuda")
    held = cache
    if what == "lse":
        lse = inside[:16].view(torch.float32).view(1, 4)
    if what == "q":
        q = inside.view(BF).view(1, 4, 64)
    if what == "out":
        out = inside.view(BF).view(1, 4, 64)
    if what == "pages":
        big = ws[n // 2:][:cache.k.numel()].view(cache.k.shape)
        held = lm.KVCache(plan, big, cache.v, cache.k_scale, cache.v_scale)
    if what == "scales":
        big = ws[n // 2:][:cache.v_scale.nbytes].view(torch.float32)
        held = lm.KVCache(plan, cache.k, cache.v, cache.k_scale, big)
    with pytest.raises(lm.LayoutMoveError) as e:
        lm.kv_attend(held, q, P.table.cuda(), torch.tensor([20]).int().cuda(),
                     out, ws, lse=lse)
    assert e.value.status == -7
    assert not ws.any()


def test_scales_beside_the_pages_of_one_buffer():
    """Pages with room between them, scales in the room after the last: taken,
    and right."""
    P = kr.Pages([30], 2, 64, 16, "nhd", BF, "e4m3", seed=3)
    plan = lm.KVPlan(lm.Layout.make(*P.page_layout()), BF, "e4m3",
                     page_stride=2 * 16 * 2 * 64)
    page, scale = 16 * 2 * 64, P.pool * 2 * 16 * 4
    buf = torch.zeros(P.pool * 2 * page + 2 * scale, dtype=torch.uint8,
                      device="cuda")
    pages = buf[:P.pool * 2 * page].view(P.pool, 2, page)
    k, v = pages[:, 0], pages[:, 1]
    ks, vs = buf[P.pool * 2 * page:].view(torch.float32).view(2, -1)
    for kv, (t, s) in enumerate(((k, ks), (v, vs))):
        t.copy_(P.device(kv).reshape(P.pool, page))
        s.copy_(P.device_scale(kv).reshape(-1))
    cache = lm.KVCache(plan, k, v, ks, vs)
    ko, vo = (torch.empty(30, 2, 64, dtype=BF, device="cuda")
              for _ in range(2))
    lm.kv_read(cache, P.table.cuda(), torch.tensor([30]).int().cuda(),
               torch.tensor([0, 30]).int().cuda(), ko, vo)
    for kv, got in enumerate((ko, vo)):
        assert torch.equal(got.cpu(), P.rows[kv][0].to(BF))
