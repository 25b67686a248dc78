"""Which sizes the cache calls take: their own bounds, not those of the prefill
(no GPU: no call here reaches a kernel)."""
import ctypes

import pytest

from chunk_wise_hierarchical_landmark_b200 import binding as hb
from tests.test_kv_cache_host import FAKE, append, cache_struct, decode, lib, params  # noqa: F401

# 2^31 query rows: 64 sequences, 32 heads, room for 1M tokens
WIDE = dict(B=64, Hq=32, Hkv=4, L=1 << 20)


def wide_cache(**kw):
    return cache_struct(max_pages=1 << 14, lmk_rows=1 << 14, num_pages=1 << 10, **kw)


@pytest.mark.parametrize("kw", [WIDE, dict(WIDE, B=2047), dict(WIDE, B=30, L=1 << 24), dict(WIDE, B=2047, L=1 << 24, Hkv=8)])
def test_capacity_does_not_multiply_with_the_heads(lib, kw):  # noqa: F811
    """What stops these calls is the argument left out, or the workspace, not the product B*Hq*L."""
    p = params(**kw)
    pages = kw["L"] // 64
    c = cache_struct(max_pages=pages, lmk_rows=pages, num_pages=1 << 10)
    assert append(lib, p=p, c=c, pos=None) == 1
    assert b"pos is NULL" in lib.hils_last_error()
    rc = decode(lib, p=p, c=c, ws=0)
    if kw["B"] * kw["Hkv"] * pages < 1 << 31:
        assert rc == 3, lib.hils_last_error()
    else:
        assert rc == 2 and b"lmk_rows" in lib.hils_last_error()
    need = lib.hils_workspace_size(ctypes.byref(p), hb.HILS_OP_DECODE_CACHE)
    # at least the landmark scores of every head
    assert need >= 4 * kw["B"] * kw["Hq"] * (pages - 1)


def test_bounds_that_remain(lib):  # noqa: F811
    c = wide_cache()
    assert append(lib, p=params(**dict(WIDE, B=2048)), c=c) == 2      # B*Hq above 65535
    assert decode(lib, p=params(**dict(WIDE, B=2048)), c=c) == 2
    assert lib.hils_workspace_size(ctypes.byref(params(**dict(WIDE, B=2048))), hb.HILS_OP_DECODE_CACHE) == 0
    assert append(lib, p=params(**dict(WIDE, L=(1 << 24) + 1)), c=c) == 2
    # the prefill and the dense decode index by the product
    p = params(**WIDE)
    for op in (hb.HILS_OP_PREFILL, hb.HILS_OP_DECODE):
        assert lib.hils_workspace_size(ctypes.byref(p), op) == 0
    z = ctypes.c_void_p(FAKE)
    assert lib.hils_select(ctypes.byref(p), z, z, z, z, None, None, 0, None) == 2
    assert lib.hils_decode_fwd(ctypes.byref(p), z, z, z, z, z, z, None, z, z, z, 1 << 40, None) == 2
    assert b"2^31" in lib.hils_last_error()
