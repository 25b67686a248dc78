"""KVCache handles as Python objects: subclasses, copies, files, fixed fields (no GPU)."""
import copy
import io

import pytest
import torch

from chunk_wise_hierarchical_landmark_b200 import binding as hb

TENSORS = ("k_pages", "v_pages", "page_table", "lmk", "k_scale", "v_scale", "k_tail", "v_tail")


class Named(hb.KVCache):
    """A user's handle with a field of its own."""

    def __init__(self, *tensors, **kw):
        self.name = "pool"


class Slotted(hb.KVCache):
    __slots__ = ()


def cache(q8=True, cls=hb.KVCache):
    c = hb.alloc_kv_cache(2, 2, 64, 200, q8=q8, device="cpu")
    return cls(*(getattr(c, n) for n in TENSORS))


def pointers(c):
    return [getattr(c._c, n) for n in TENSORS]


def holds_its_tensors(c):
    return pointers(c) == [None if getattr(c, n) is None else getattr(c, n).data_ptr() for n in TENSORS]


@pytest.mark.parametrize("cls", [hb.KVCache, Named, Slotted])
@pytest.mark.parametrize("q8", [True, False])
def test_subclasses(cls, q8):
    c = cache(q8, cls)
    assert type(c) is cls and holds_its_tensors(c) and (c.B, c.Hkv, c.d, c.q8) == (2, 2, 64, q8)
    if cls is Named:
        assert c.name == "pool"
        c.name = "other"  # its own field stays its own
        assert c.name == "other"
    table = c.page_table.clone()
    z = c.replace(page_table=table)
    assert type(z) is cls and z.page_table is table and holds_its_tensors(z)


@pytest.mark.parametrize("cls", [hb.KVCache, Named, Slotted])
def test_fields_are_fixed(cls):
    c = cache(cls=cls)
    for name in TENSORS + ("B", "max_len", "_c"):
        with pytest.raises(AttributeError, match="fixed"):
            setattr(c, name, None)
        with pytest.raises(AttributeError, match="fixed"):
            delattr(c, name)
    assert holds_its_tensors(c)


@pytest.mark.parametrize("cls", [hb.KVCache, Named])
@pytest.mark.parametrize("q8", [True, False])
def test_copies(cls, q8):
    """A copy is a handle of the same tensors; a deep copy and a saved one have tensors
    of their own, and pointers to those."""
    c = cache(q8, cls)
    if cls is Named:
        c.name = "mine"
    s = copy.copy(c)
    assert type(s) is cls and all(getattr(s, n) is getattr(c, n) for n in TENSORS)
    deep = copy.deepcopy(c)
    f = io.BytesIO()
    torch.save(c, f)
    f.seek(0)
    for z in (s, deep, torch.load(f, weights_only=False)):
        assert type(z) is cls and holds_its_tensors(z)
        assert cls is not Named or z.name == "mine"
        for n in TENSORS:
            a, b = getattr(c, n), getattr(z, n)
            assert (a is None and b is None) or torch.equal(a.float(), b.float())
            assert a is None or z is s or a.data_ptr() != b.data_ptr()


def test_tables_past_32_bits_are_refused():
    """The library counts table entries in 32 bits (tensors without memory)."""
    z = dict(device="meta", dtype=torch.bfloat16)
    pages = torch.empty((4, 2, 64, 64), **z)
    for shape in ((1, (1 << 32) + 4), (2, 1 << 30)):
        with pytest.raises(ValueError, match="page_table"):
            hb.KVCache(pages, pages, torch.empty(shape, device="meta", dtype=torch.int32))
