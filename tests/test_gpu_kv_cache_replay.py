"""Steps over long caches as a serving loop makes them: captured, replayed on one
workspace and beside eager calls on another stream, with many more chunks than are
selected; the few-token append's own bounds checks."""
import math

import pytest
import torch

from chunk_wise_hierarchical_landmark_b200 import binding as hb
from tests.kv_cache_ref import C, check_decode
from tests.test_gpu_kv_cache import BF16, F32, ints, make_cache, randn, reference, same, state

pytestmark = pytest.mark.gpu


def running_cache(B, H, d, chunks, q8, dtype, seed):
    """A cache as a long run leaves it: random pages in shuffled places, landmarks, tails."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda shape, ty: torch.randn(shape, generator=g, device="cuda").to(ty)  # noqa: E731
    pages, ty = B * chunks, torch.float8_e4m3fn if q8 else dtype
    table = torch.randperm(pages, generator=g, device="cuda").view(B, chunks).to(torch.int32)
    more = []
    if q8:
        more = [torch.exp2(torch.randint(-2, 2, (pages, H), generator=g, device="cuda").float()) for _ in range(2)]
        more += [rn((B, 2, H, C, d), dtype) for _ in range(2)]
    return hb.KVCache(rn((pages, H, C, d), ty), rn((pages, H, C, d), ty), table, rn((B, H, chunks, d), dtype), *more)


def twin(c):
    return c.replace(**{n: getattr(c, n).clone() for n in
                        ("k_pages", "v_pages", "page_table", "lmk") +
                        (("k_scale", "v_scale", "k_tail", "v_tail") if c.q8 else ())})


@pytest.mark.parametrize("q8,dtype,B,H,G,d,K,chunks", [
    # scores -> selection -> attention -> combine, the list longer than the warps of the
    # grid, so that most of it is shared out by the counter
    (True, BF16, 24, 8, 4, 128, 16, 600), (False, BF16, 24, 8, 4, 64, 16, 600),
    (True, BF16, 3, 4, 8, 64, 64, 2200),
    # the cluster scores its landmarks itself; a list shorter than the warps
    (True, BF16, 2, 2, 4, 128, 5, 300), (False, BF16, 2, 2, 4, 128, 5, 300),
    # the radix select
    (True, BF16, 2, 2, 2, 64, 7, 8300), (True, F32, 2, 2, 2, 64, 7, 700), (False, F32, 2, 2, 2, 64, 7, 700)])
def test_replays_on_one_workspace(q8, dtype, B, H, G, d, K, chunks):
    """Append + decode captured once and replayed with new inputs and lengths, eager calls
    running on another stream meanwhile: the same bits in every output and
    buffer, step for step."""
    L = chunks * C
    eager = running_cache(B, H, d, chunks, q8, dtype, seed=800)
    graphed = twin(eager)
    x = torch.zeros((B, 1, G * H + 2 * H, d), dtype=dtype, device="cuda")
    pos, lens = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")

    def step(c, pos, lens, x):
        r = hb.kv_append(c, x[:, :, G * H:-H].transpose(1, 2), x[:, :, -H:].transpose(1, 2), pos,
                         q=x[:, :, :G * H].transpose(1, 2), n_rope_pairs=20, max_len=L, seq_lens=lens)
        return hb.decode_cache(r["q"].view(B, G * H, d), c, lens, K, max_len=L)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(twin(graphed), pos, lens, x)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(graphed, pos, lens, x)
    gen = torch.Generator().manual_seed(801)
    n_steps = 12
    starts = torch.randint(K * C, L - n_steps, (n_steps, B), generator=gen, dtype=torch.int32)
    starts[0] = L - 1                      # the longest there are
    starts[1, ::2] = 0                     # first tokens beside long sequences
    starts[2] = starts[2] // C * C + C - 1  # every sequence completes a chunk
    starts[6:] = starts[5] + torch.arange(1, n_steps - 5, dtype=torch.int32)[:, None]  # a run of single tokens
    inputs = [randn(tuple(x.shape), 810 + i, dtype).cuda() for i in range(n_steps)]
    starts = starts.cuda()
    torch.cuda.synchronize()
    want, got = [], []
    with torch.cuda.stream(s):
        for i in range(n_steps):
            want.append(step(eager, starts[i], torch.empty_like(pos), inputs[i]))
    for i in range(n_steps):
        x.copy_(inputs[i])
        pos.copy_(starts[i])
        graph.replay()
        got.append({n: t.clone() for n, t in out.items()})
    torch.cuda.synchronize()
    for i in range(n_steps):
        for n in got[i]:
            assert torch.equal(got[i][n], want[i][n]), (i, n)
        assert torch.equal((got[i]["sel_idx"] >= 0).sum(-1)[:, 0].int(), (starts[i] // C).clamp(max=K))
    assert same(state(eager), state(graphed))


@pytest.mark.parametrize("q8,dtype,d", [(True, BF16, 128), (False, BF16, 64), (True, F32, 64), (False, F32, 128)])
def test_serving_run_that_rejects_chunks(q8, dtype, d):
    """Prompts of up to 30 chunks of which 3 are selected, then single tokens across chunk
    borders; every step against the 64-bit model.  Heads whose selection differs may do
    so only where the model's scores lie within the rounding of a score."""
    B, H, G, K, pairs, L = 3, 2, 4, 3, 20, 2100
    c = make_cache(B, H, d, L, q8, dtype, seed=830)
    rope = dict(n_rope_pairs=pairs, max_len=L)
    heads = lambda x: (x[:, :, :G * H].transpose(1, 2), x[:, :, G * H:-H].transpose(1, 2), x[:, :, -H:].transpose(1, 2))  # noqa: E731
    _, k, v = heads(randn((B, 1980, G * H + 2 * H, d), 831, dtype).cuda())
    lens = hb.kv_append(c, k, v, ints([0] * B), n_new=ints([1980, 765, 319]), **rope)["seq_lens"]
    scale = 1.0 / math.sqrt(d)
    for i in range(6):
        q, k, v = heads(randn((B, 1, G * H + 2 * H, d), 840 + i, dtype).cuda())
        r = hb.kv_append(c, k, v, lens, q=q, **rope)
        lens, q = r["seq_lens"], r["q"].view(B, G * H, d)
        got = hb.decode_cache(q, c, lens, K, max_len=L, debug_checks=True)
        ref = reference(c, q, lens.tolist(), K)
        lm, qc = c.lmk.double().cpu(), q.double().cpu()
        alike = (got["sel_idx"].cpu() == ref["sel_idx"]).all(-1)
        for b, h in (~alike).nonzero().tolist():
            n = (int(lens[b]) - 1) // C
            s, m = (lm[b, h // G, :n] @ qc[b, h]) * scale, (lm[b, h // G, :n].abs() @ qc[b, h].abs()) * scale
            a, z = set(got["sel_idx"][b, h].tolist()), set(ref["sel_idx"][b, h].tolist())
            # d products and sums and the scale: (d + 2) roundings of 2^-24 each side
            assert max(float(s[j]) for j in z - a) - min(float(s[j]) for j in a - z) <= 2 * (d + 2) * 2.0 ** -24 * float(m.max())
        pick = alike.nonzero(as_tuple=True)
        assert len(pick[0]) > 0
        check_decode({n: t[pick] for n, t in got.items()}, {n: t[pick] for n, t in ref.items()}, dtype == BF16)
        assert (got["sel_idx"][0] > K).any()  # not simply the first chunks


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("T", [1, 40, 64, 70])
@pytest.mark.parametrize("pos4", [0, 63])
@pytest.mark.parametrize("bad", [-1, "pool", (1 << 31) - 1])
def test_append_bounds_for_few_and_many_tokens(q8, T, pos4, bad):
    """Positions and counts out of bounds, a page outside the pool for a chunk that stays
    partial or becomes complete: nothing is written for them, the queries of a
    refused sequence become 0, the others are served."""
    B, H, Hq, d, L = 6, 2, 4, 64, 256
    k, q = randn((B, H, T, d), 850, BF16).cuda(), randn((B, Hq, T, d), 851, BF16).cuda()
    a, z = (make_cache(B, H, d, L, q8, BF16, seed=852) for _ in range(2))
    page = int(a.page_table[4, 0])
    a.page_table[4, 0] = a.k_pages.shape[0] if bad == "pool" else bad
    before = state(a)
    pos, n = ints([-1, 10, L - T + 1, 30, pos4, 7]), ints([T, T + 1, T, T, T, -1])
    ra = hb.kv_append(a, k, k, pos, n_new=n, q=q, n_rope_pairs=9)
    rz = hb.kv_append(z, k, k, ints([0, 0, 0, 30, pos4, 0]), n_new=ints([0, 0, 0, T, T, 0]), q=q, n_rope_pairs=9)
    assert ra["seq_lens"].tolist() == [0, 10, L - T + 1, 30 + T, pos4 + T, 7]
    assert torch.equal(ra["q"], rz["q"]) and not ra["q"][[0, 1, 2, 5]].any() and ra["q"][3:5].any()
    sa, sz = state(a), state(z)
    for x in ("k_pages", "v_pages") + (("k_scale", "v_scale") if q8 else ()):
        sz[x][page] = before[x][page]
    if not q8:
        sz["lmk"][4, :, 0] = before["lmk"][4, :, 0]  # no page, no landmark
    assert same(sa, sz)
    with pytest.raises(hb.HilsError) as e:
        hb.kv_append(a, k, k, pos, n_new=n, debug_checks=True)
    assert e.value.status == 5
    # the page alone: reported where it is needed (pages: at once, blocks: when the chunk is complete)
    good = ints([0, 0, 0, 30, pos4, 0])
    some = ints([0, 0, 0, T, T, 0])
    if not q8 or pos4 + T >= C:
        with pytest.raises(hb.HilsError) as e:
            hb.kv_append(a, k, k, good, n_new=some, debug_checks=True)
        assert e.value.status == 5
    else:
        hb.kv_append(a, k, k, good, n_new=some, debug_checks=True)
