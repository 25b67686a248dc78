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
@pytest.mark.parametrize("d", [64, 128])
def test_own_chunk_without_a_logit_weighs_nothing(q8, dtype, d):
    """Keys of -inf in the whole own chunk: its fusion logit is -inf, its values
    (NaN among them) do not matter and the rest is fused without it, as with keys so
    low that the weight is 0 in 32 bits."""
    G, K, n_c, own = 3, 2, 4, 17
    c, k, v, _ = filled(1, 1, d, [n_c * C], q8, dtype, seed=700 + d, max_len=n_c * C + own)
    q = positive_queries(G, d, dtype, 701)
    got = []
    for low in (-math.inf, -1e4):
        x, y = torch.full((1, 1, own, d), low, dtype=dtype), randn((1, 1, own, d), 702, dtype)
        if low == -math.inf:
            y[0, 0, 3, 5], y[0, 0, 4, 6] = math.inf, math.nan
        hb.kv_append(c, x.cuda(), y.cuda(), ints([n_c * C]))
        got.append(step(c, q, n_c * C + own, K, debug_checks=True))
    for n in got[0]:
        assert torch.equal(got[0][n], got[1][n]), n
    assert got[0]["out"].isfinite().all()
    # nothing but the selected landmarks' logits: the sum of K exponentials
    want = torch.logsumexp(got[0]["chunk_w"].double(), -1)
    assert ((got[0]["lse"].double() - want).abs() <= 2.0 ** -20 * (4 + want.abs())).all()


@pytest.mark.parametrize("q8,dtype", FORMS)
@pytest.mark.parametrize("d", [64, 128])
def test_a_head_with_nothing_left(q8, dtype, d):
    """An own chunk of keys of -inf and no other chunk, or only chunks banned by
    their landmarks: out 0, lse -inf; a sequence beside it is served."""
    G, K = 2, 3
    for n_c in (0, 1, 3, 5):
        N = n_c * C + 9
        c, *_ = filled(2, 1, d, [n_c * C, N], q8, dtype, seed=710 + n_c, max_len=N)
        lm = c.lmk.clone()
        lm[0, :, :n_c] = -math.inf
        c = c.replace(lmk=lm)
        x = torch.full((2, 1, 9, d), -math.inf, dtype=dtype).cuda()
        hb.kv_append(c, x, randn((2, 1, 9, d), 711, dtype).cuda(), ints([n_c * C, 0]), n_new=ints([9, 0]))
        q = positive_queries(G, d, dtype, 712).repeat(2, 1, 1)
        got = hb.decode_cache(q, c, ints([N, N]), K, debug_checks=True)
        assert not got["out"][0].any()
        assert (got["lse"][0] == -math.inf).all() and (got["lse_lmk"][0] == -math.inf).all()
        assert (got["chunk_w"][0] == -math.inf).all()
        assert got["sel_idx"][0].tolist() == [[i if i < n_c else -1 for i in range(K)]] * G
        assert got["out"][1].isfinite().all() and got["out"][1].any() and got["lse"][1].isfinite().all()


@pytest.mark.parametrize("q8,dtype", FORMS)
def test_values_of_a_banned_chunk_do_not_matter(q8, dtype):
    """NaN among the values of a chunk whose landmark logit is -inf."""
    G, d, K, N = 2, 64, 4, 4 * C + 5
    c, *_ = filled(1, 1, d, [N], q8, dtype, seed=720)
    q = positive_queries(G, d, dtype, 721)
    lm = c.lmk.clone()
    lm[0, 0, 2] = -math.inf
    c = c.replace(lmk=lm)
    want = step(c, q, N, K)
    c.v_pages[int(c.page_table[0, 2]), 0, 7] = math.nan
    got = step(c, q, N, K)
    for n in got:
        assert torch.equal(got[n], want[n]), n
    assert got["out"].isfinite().all()


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
@pytest.mark.parametrize("low", [-math.inf, -1.0])
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


@pytest.mark.parametrize("q8,dtype", FORMS)
def test_room_for_a_million_tokens(q8, dtype):
    """64 sequences of 32 heads with room for 2^20 tokens each (2^31 query rows), a
    few hundred of them there: the same as with room for those alone, but for
    the order of the sums of lse_lmk, and in the fp32 8-bit form, whose grid
    follows the capacity, of the merges of a head's K + 1 = 4 chunks: 4 times
    two exponentials of 2^-21 and 2^-22 per unit of their argument (at most the
    range of the logits), in the numerator and in the sum, on both sides."""
    B, H, Hq, d, K, L = 64, 4, 32, 64, 3, 1 << 20
    n = [(37 * b) % 450 for b in range(B)]
    need = 8
    table = torch.full((B, L // C), -1, dtype=torch.int32)
    g = torch.Generator().manual_seed(740)
    table[:, :need] = torch.randperm(B * need, generator=g).view(B, need).to(torch.int32)
    wide = hb.alloc_kv_cache(B, H, d, L, num_pages=B * need, page_table=table.cuda(), q8=q8, dtype=dtype)
    tight = hb.alloc_kv_cache(B, H, d, need * C, num_pages=B * need, page_table=table[:, :need].cuda().contiguous(),
                              q8=q8, dtype=dtype)
    k, v = randn((B, H, 450, d), 741, dtype).cuda(), randn((B, H, 450, d), 742, dtype).cuda()
    q = randn((B, Hq, 1, d), 743, dtype).cuda()
    got = []
    for c in (wide, tight):
        lens = hb.kv_append(c, k, v, ints([0] * B), n_new=ints(n))["seq_lens"]
        r = hb.kv_append(c, k[:, :, :1], v[:, :, :1], lens, q=q, n_rope_pairs=20)
        assert r["seq_lens"].tolist() == [x + 1 for x in n]
        got.append(hb.decode_cache(r["q"].view(B, Hq, d), c, r["seq_lens"], K, debug_checks=True))
    for name in got[0]:
        a, z = got[0][name], got[1][name]
        if name != "lse_lmk" and (not q8 or dtype == BF16 or name in ("sel_idx", "chunk_w")):
            assert torch.equal(a, z), name
            continue
        fin = z != -math.inf
        assert torch.equal(a != -math.inf, fin)
        if name == "lse_lmk":
            assert ((a - z).abs()[fin] <= 2.0 ** -19 * (4 + z.abs()[fin])).all()
            continue
        w = got[0]["chunk_w"]
        span = float(w[w != -math.inf].abs().max()) + float(got[0]["lse"].abs().max())
        tol = 32 * (2.0 ** -21 + 2.0 ** -22 * span)
        assert tol < 2.0 ** -12
        assert ((a - z).abs() <= tol * (float(v.abs().max()) if name == "out" else 1.0)).all(), name


def test_sizes_past_32_bits_are_refused():
    """By the library's own errors; their low 32 bits would be good sizes."""
    c = hb.alloc_kv_cache(1, 2, 64, 256)
    k, q = randn((1, 2, 3, 64), 750, BF16).cuda(), randn((1, 4, 64), 751, BF16).cuda()
    before = c.k_tail.clone()
    for wide in ((1 << 32) + 256, 256 - (1 << 32)):
        for call in (lambda: hb.kv_append(c, k, k, ints([0]), max_len=wide),
                     lambda: hb.decode_cache(q, c, ints([3]), 4, max_len=wide)):
            with pytest.raises(hb.HilsError):
                call()
    for wide in ((1 << 32) + 8, 8 - (1 << 32)):
        with pytest.raises(hb.HilsError):
            hb.kv_append(c, k, k, ints([0]), n_rope_pairs=wide)
    assert torch.equal(c.k_tail, before)


@pytest.mark.parametrize("topk", [65, 1 << 26, (1 << 32) + 8, 8 - (1 << 32)])
def test_a_refused_topk_allocates_nothing_of_its_size(topk):
    c = hb.alloc_kv_cache(1, 2, 64, 256)
    q = randn((1, 4, 64), 752, BF16).cuda()
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    base = torch.cuda.memory_allocated()
    with pytest.raises(hb.HilsError) as e:
        hb.decode_cache(q, c, ints([3]), topk)
    assert e.value.status in (1, 2)
    assert torch.cuda.max_memory_allocated() - base < 1 << 20
