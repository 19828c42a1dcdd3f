"""The paged cache's Python objects on tensors that are stand-ins (nothing is
read; no GPU needed)."""

import pytest

lm = pytest.importorskip("layout_driven_movement_gb300")


@pytest.fixture(scope="module", autouse=True)
def built():
    from layout_driven_movement_gb300 import _build
    _build.build()
    lm.lib()


class Tensor:
    """What a cache asks of a CUDA tensor."""
    is_cuda = True

    def __init__(self, dtype, *shape, at=1 << 40):
        self.dtype, self.shape, self.at = dtype, shape, at

    def element_size(self):
        return {"uint8": 1, "int8": 1, "float8_e4m3fn": 1, "float8_e5m2": 1,
                "float32": 4}.get(self.dtype.rpartition(".")[2], 2)

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def stride(self):
        out, n = [], 1
        for x in reversed(self.shape):
            out.append(n)
            n *= x
        return tuple(reversed(out))

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at


def cache_of(dtype, store, k, v=None, **kw):
    plan = lm.KVPlan(lm.Layout.parse("(4,2,16):(32,16,1)"), dtype, store)
    scales = [Tensor("torch.float32", 8, 2, 4) for _ in range(2)] if store \
        else [None, None]
    return lm.KVCache(plan, k, k if v is None else v, *scales, **kw)


@pytest.mark.parametrize("dtype,store,held,taken", [
    ("bfloat16", None, "bfloat16", True), ("bfloat16", None, "float16", False),
    ("bfloat16", "same", "int16", False), ("float16", None, "float16", True),
    ("float16", None, "bfloat16", False), ("bfloat16", None, "uint8", False),
    ("bfloat16", "e4m3", "float8_e4m3fn", True),
    ("bfloat16", "e4m3", "uint8", True), ("bfloat16", "e4m3", "int8", False),
    ("bfloat16", "e4m3", "float8_e5m2", False),
    ("bfloat16", "e4m3", "bfloat16", False),
    ("float16", "int8", "int8", True), ("float16", "int8", "uint8", True),
    ("float16", "int8", "float8_e4m3fn", False),
])
def test_pages_are_of_the_plans_type(dtype, store, held, taken):
    """The store's own type, or bytes that stand for it; never another type's
    numbers."""
    right = Tensor("torch." + (dtype if store in (None, "same") else "uint8"),
                   8, 128)
    other = Tensor("torch." + held, 8, 128)
    for k, v in ((other, right), (right, other)):
        if taken:
            assert cache_of("torch." + dtype, store, k, v).pages == 8
        else:
            with pytest.raises(ValueError):
                cache_of("torch." + dtype, store, k, v)


@pytest.mark.parametrize("elements,pages", [
    (8 * 128, 8), (8 * 128 + 1, 8), (8 * 128 + 127, 8), (9 * 128, 9),
    (128, 1), (129, 1)])
def test_pages_that_a_buffer_holds(elements, pages):
    """What a buffer has past its last whole page is no page."""
    k = Tensor("torch.bfloat16", elements)
    assert cache_of("torch.bfloat16", None, k).pages == pages


@pytest.mark.parametrize("elements,pages", [
    (7 * 200 + 128, 8), (7 * 200 + 127, 7), (8 * 200, 8), (7 * 200, 7)])
def test_pages_of_a_stride_above_their_size(elements, pages):
    """The last page needs its own elements, not the gap after them."""
    plan = lm.KVPlan(lm.Layout.parse("(4,2,16):(32,16,1)"), "torch.bfloat16",
                     page_stride=200)
    k = Tensor("torch.bfloat16", elements)
    assert lm.KVCache(plan, k, k).pages == pages
