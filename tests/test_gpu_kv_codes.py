"""Whole-number codes of the cache's write, element by element."""

import pytest

from test_gpu_kv import BF, HF, built, clean_status  # noqa: F401

torch = pytest.importorskip("torch")
lm = pytest.importorskip("layout_driven_movement_gb300")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,size", [
    (HF, 1.0), (HF, 2.0 ** -9), (HF, 7000.0), (BF, 1.0), (BF, 1e-30),
    (BF, 1e30), (BF, 1e37)])
@pytest.mark.parametrize("dim", [16, 80, 256])
def test_whole_number_codes_are_the_formulas(dtype, size, dim):
    """rint(127 x / max|x|), ties to even, of rows that are not turned: among
    16-bit elements exact ties are common (x = max / 2 is one), and the nearest
    other quotient is 2^-12 of a code away from a tie."""
    tokens, heads, page = 640, 4, 16
    g = torch.Generator().manual_seed(dim)
    x = (torch.randn(2, tokens, heads, dim, generator=g) * size).to(dtype)
    # half the largest magnitude, exactly: 63.5
    x[:, :, 0, 1::3] = x[:, :, 0].abs().amax(-1, keepdim=True) / 2
    plan = lm.KVPlan(lm.Layout.make([page, heads, dim], [heads * dim, dim, 1],
                                    [1, 1, 1]), dtype, "int8")
    k, v = (torch.zeros(tokens // page, page, heads, dim, dtype=torch.int8,
                        device="cuda") for _ in range(2))
    scales = [torch.ones(tokens // page, heads, page, device="cuda")
              for _ in range(2)]
    lm.kv_write(lm.KVCache(plan, k, v, *scales), x[0].cuda(), x[1].cuda(),
                torch.arange(tokens, device="cuda"))
    for kv, held in enumerate((k, v)):
        row = x[kv].double()
        want = torch.round(row * 127 / row.abs().amax(-1, keepdim=True))
        assert want.abs().max() == 127
        assert torch.equal(held.cpu().view(tokens, heads, dim).double(), want)
