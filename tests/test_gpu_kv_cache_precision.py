"""How many bits the decode step over the 8-bit cache keeps of its probabilities."""
import math

import pytest
import torch

from chunk_wise_hierarchical_landmark_b200 import binding as hb
from tests.kv_cache_ref import C, decode_ref
from tests.test_gpu_kv_cache import BF16, ints

pytestmark = pytest.mark.gpu


def worst_signs(p, half_steps):
    """Signs s of 64 values so that rounding p (times 2^15 over its maximum) to half_steps
    bits moves sum p s as far as it can while the sum itself stays near 0: the 40
    largest rounding errors add up, the others balance the sum."""
    x = p / p.max() * 2.0 ** 15
    ulp = 2.0 ** (torch.floor(torch.log2(x)) - half_steps + 1)
    err = (x / ulp).round() * ulp - x
    s = torch.zeros_like(p)
    order = err.abs().argsort(descending=True)
    s[order[:40]] = torch.sign(err[order[:40]])
    run = float((p * s).sum())
    for j in order[40:][p[order[40:]].argsort(descending=True)]:
        s[j] = -1.0 if run > 0 else 1.0
        run += float(p[j] * s[j])
    s[s == 0] = 1.0
    return s


@pytest.mark.parametrize("d", [64, 128])
def test_probabilities_over_8_bit_blocks_keep_22_bits(d):
    """One selected chunk, whose landmark outweighs the own chunk by e^40, so that out =
    sum p_j v_j with v_j = +-1: signs along the roundings of p to fp16 add these up to
    1e-4 while the sum is near 0 and its own rounding, half a step of bf16, small.

    Tolerance, relative to sum p |v| = 1: a logit is one product (the other
    terms are 0) with 8 roundings of 2^-24 on its way to the exponent; the
    exponent, at most 16, is rounded by 2^-21 and the exponential is good to 2^-22;
    p in two parts of 11 bits to 2^-22; each of these for the numerator and
    for the sum; the sums have 64 terms, two products each: 130 roundings of 2^-24."""
    G, N = 8, C + 1
    g = torch.Generator().manual_seed(810 + d)
    k = torch.zeros((1, 1, C, d))
    k[0, 0, :, 0] = (torch.randperm(C, generator=g) - 32.0) / 32  # rounded to e4m3 below
    kq = k.to(torch.float8_e4m3fn)
    q = torch.zeros((1, G, d))
    q[0, :, 0] = (1.0 + torch.arange(G) / 16.0) * math.sqrt(d) / 8  # logits up to 0.18
    q[0, :, 1] = math.sqrt(d)
    q = q.to(BF16)
    scale = 1.0 / math.sqrt(d)
    lmk = torch.zeros((1, 1, 1, d))
    lmk[..., 1] = 40.0
    v = torch.zeros((1, 1, C, d))
    for h in range(G):
        p = torch.softmax(kq[0, 0].double() @ q[0, h].double() * scale, 0)
        s = worst_signs(p, 11)
        for e in range(h, d, G):
            v[0, 0, :, e] = s if e % 2 else -s
    one, tail = torch.ones((1, 1)), torch.zeros((1, 2, 1, C, d), dtype=BF16)
    c = hb.KVCache(kq.cuda(), v.to(torch.float8_e4m3fn).cuda(), torch.zeros((1, 2), dtype=torch.int32).cuda(),
                   lmk.to(BF16).cuda(), one.cuda(), one.cuda(), tail.cuda(), tail.cuda())
    got = hb.decode_cache(q.cuda(), c, ints([N]), 1, max_len=N)["out"].cpu().double()
    ref = decode_ref(q, [N], None, lmk, lambda b, h, ch: (kq[b, h].double(), v[b, h].double()),
                     lambda b, h, n: (tail[b, 1, h, :n].double(), tail[b, 1, h, :n].double()), 1, scale)
    assert float(ref["spread"].max()) < 0.25 and float((ref["mag"] - 1).abs().max()) < 1e-9
    assert float(ref["out"].abs().min(-1).values.max()) < 2.0 ** -6  # every head has a sum near 0
    tol = 2 * (8 * 2.0 ** -24 * 0.25 + 2.0 ** -21 + 2.0 ** -22 + 2.0 ** -22) + 130 * 2.0 ** -24
    assert ((got - ref["out"]).abs() <= tol + 2.0 ** -8 * ref["out"].abs()).all()


def scaled_twice(v, q, N, K, dtype):
    """The decode of a batch whose values are v, and v times 2^-119 with its out times 2^119."""
    B, H, _, d = v.shape
    g = torch.Generator().manual_seed(831)
    k = torch.randn((B, H, N, d), generator=g).to(dtype).cuda()
    got = []
    for e in (0, -119):
        c = hb.alloc_kv_cache(B, H, d, N, q8=True, dtype=dtype)
        hb.kv_append(c, k, (v.double() * 2.0 ** e).to(dtype), ints([0] * B))
        if e:
            assert 2.0 ** -126 <= float(c.v_scale[c.v_scale > 0].min()) <= 2.0 ** -123
        got.append(hb.decode_cache(q, c, ints([N] * B), K, max_len=N))
    for n in ("sel_idx", "chunk_w", "lse", "lse_lmk"):
        assert torch.equal(got[0][n], got[1][n]), n
    return got[0]["out"].double(), got[1]["out"].double() * 2.0 ** 119


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("coherent", [False, True])
def test_values_near_the_least_scales(d, dtype, coherent):
    """Values times 2^-119 (scales near 2^-126) give the outputs times 2^-119: a power of two
    moves no bit but where intermediate results become subnormal.  What that
    leaves, times 2^119, is 2^-31 for a sum; it may carry a rounding that lay at its
    border to the next step: in fp32 at most 8 of them (the merges of K + 1 = 5
    chunks, two records, a division), each a step, 2^-23, of the largest value; in
    bf16 one more, 2^-7 of out, or 2^-14 where out is subnormal."""
    B, H, G, K, N = 2, 2, 4, 4, 9 * C + 7
    g = torch.Generator().manual_seed(830)
    v = torch.randn((B, H, N, d), generator=g)
    if coherent:
        v = 3.75 + 0.25 * v.tanh()  # the products of a chunk add up
    q = (torch.randn((B, H * G, d), generator=g) / 8).to(dtype).cuda()
    a, z = scaled_twice(v.to(dtype).cuda(), q, N, K, dtype)
    tol = 8 * 2.0 ** -23 * float(v.abs().max())
    tol = tol if dtype != BF16 else 2.0 ** -7 * a.abs() + 2.0 ** -14 + tol
    assert ((a - z).abs() <= tol).all(), float((a - z).abs().max())
