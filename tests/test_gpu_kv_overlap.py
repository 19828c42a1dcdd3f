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
