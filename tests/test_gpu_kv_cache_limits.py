"""The cache operators where a head has nothing left to attend: fusion logits
and token logits of -inf, in every form of the cache and both selections."""
import math

import pytest
import torch

from chunk_wise_hierarchical_landmark_b200 import binding as hb
from tests.kv_cache_ref import C
from tests.test_gpu_kv_cache import BF16, F32, filled, grid, ints, randn

pytestmark = pytest.mark.gpu
FORMS = [(True, BF16), (False, BF16), (True, F32), (False, F32)]


def step(c, q, N, K, **kw):
    return hb.decode_cache(q, c, ints([N]), K, **kw)


def positive_queries(G, d, dtype, seed):
    return grid(randn((1, G, d), seed), dtype).abs().cuda() + 0.0625


@pytest.mark.parametrize("q8,dtype", FORMS)
def test_nan_keys_of_the_own_chunk_are_not_lost(q8, dtype):
    """A NaN among the own chunk's keys reaches out and lse of every head, whether other
    chunks are attended or not."""
    G, d, K = 2, 64, 3
    for n_c in (0, 4):
        c, *_ = filled(1, 1, d, [n_c * C], q8, dtype, seed=725, max_len=n_c * C + 3)
        x = randn((1, 1, 3, d), 726, dtype)
        x[0, 0, 1, 7] = math.nan
        hb.kv_append(c, x.cuda(), x.abs().nan_to_num(1.0).cuda(), ints([n_c * C]))
        got = step(c, positive_queries(G, d, dtype, 727), n_c * C + 3, K, debug_checks=True)
        assert got["out"].isnan().all() and got["lse"].isnan().all()


@pytest.mark.parametrize("q8,dtype", FORMS)
@pytest.mark.parametrize("low", [-1.0])
def test_every_landmark_banned_in_a_long_cache(q8, dtype, low):
    """More than 8192 completed chunks, every landmark -inf: the lowest chunks fill the
    selection with weight 0, lse_lmk is -inf and the own chunk takes all (low:
    its keys; -inf leaves nothing)."""
    d, G, K, chunks, rows = 64, 2, 5, 8200, 3
    N = chunks * C + rows
    ty = torch.float8_e4m3fn if q8 else dtype
    kp = torch.zeros((2, 1, C, d), device="cuda").to(ty)
    own = torch.full((rows, d), low, device="cuda").to(dtype)
    val = randn((rows, d), 730, dtype).cuda()
    table = torch.zeros((1, chunks + 1), dtype=torch.int32, device="cuda")
    table[0, chunks] = 1
    vp, more = kp.clone(), []
    if q8:
        tail = [torch.zeros((1, 2, 1, C, d), dtype=dtype, device="cuda") for _ in range(2)]
        for t, x in zip(tail, (own, val)):
            t[0, chunks % 2, 0, :rows] = x
        more = [torch.ones((2, 1), device="cuda") for _ in range(2)] + tail
    else:
        kp[1, 0, :rows], vp[1, 0, :rows] = own, val
    lmk = torch.full((1, 1, chunks, d), -math.inf, dtype=dtype, device="cuda")
    c = hb.KVCache(kp, vp, table, lmk, *more)
    q = positive_queries(G, d, dtype, 731)
    got = step(c, q, N, K, max_len=N, debug_checks=True)
    assert got["sel_idx"][0].tolist() == [list(range(K))] * G
    assert (got["chunk_w"] == -math.inf).all() and (got["lse_lmk"] == -math.inf).all()
    if low == -math.inf:
        assert not got["out"].any() and (got["lse"] == -math.inf).all()
        return
    # equal logits: the mean of the values, its sums and one rounding of the type
    want = val.double().mean(0)
    tol = torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -18 * val.double().abs().mean(0)
    assert ((got["out"][0].double() - want).abs() <= tol).all()
    lse = -q[0].double().sum(-1) / math.sqrt(d) + math.log(rows)
    assert ((got["lse"][0].double() - lse).abs() <= 2.0 ** -18 * (4 + lse.abs())).all()
