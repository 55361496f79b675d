"""The 4-bit operators where their ranges end: many new tokens, the most heads
and the longest sums, requests out of range beside others, and calls that share
a cache's workspace in turn."""

import pytest
import torch

import activation_sparse_swiglu_b200 as prox
from tests import decode4_helpers as ref
from tests.test_gpu_decode4 import attend_case, check_attend, gen_of, linear_case, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("lens, Tq, Hkv, G, D, page", [
    ([100, 6, 3, 0], 6, 2, 4, 128, 32), ([40, 700, 17, 16], 17, 1, 5, 64, 16), ([64, 900, 63], 64, 2, 2, 128, 64),
    ([512, 1500, 511], 512, 1, 3, 128, 64), ([130, 300], 130, 1, 2, 256, 16)])
def test_attend_many_new_tokens(lens, Tq, Hkv, G, D, page, dtype):
    """Prompt chunks: more new tokens than a block of rows, contexts that hold
    nothing else, and some shorter than the chunk (a padded batch)."""
    check_attend(prox, *attend_case(prox, lens, Tq, Hkv, G, D, page, dtype, seed=Tq))


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("Hkv, G, D, page", [(1024, 1, 64, 16), (1, 128, 128, 32), (3, 71, 256, 16)])
def test_attend_many_heads(Hkv, G, D, page, dtype):
    lens = [50, 0, 17] if Hkv > 100 else [900, 0, 17]
    check_attend(prox, *attend_case(prox, lens, 1, Hkv, G, D, page, dtype, seed=G))


@pytest.mark.parametrize("dtype", ref.TYPES)
def test_attend_requests_beside_bad_ones(dtype):
    """A length or a table entry out of range sets its bit; the requests beside
    it, inside one warp or split over CTAs, have their results."""
    lens = [70, 20000, 300, 5]
    cache, q, table, ln = attend_case(prox, lens, 1, 2, 4, 64, 16, dtype, seed=60, garbage=False)
    table = torch.where(table < cache.num_pages, table, 0)  # a length cut to the table reads these
    want, _, tol, _ = ref.attend(q, cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, table, ln, 64 ** -0.5)
    for bad_at in (0, 2):
        for n in (-5, 1 << 30, -(1 << 31), (1 << 31) - 1, table.shape[1] * 16 + 1):
            bad = ln.clone()
            bad[bad_at] = n
            got = cache.attend(q, table, bad)
            assert cache.error_word() == prox.DEVERR_LEN
            for b in range(4):
                if b != bad_at:
                    within(got[b], want[b], tol[b])
        for entry in (-1, cache.num_pages, 1 << 30, -(1 << 31), (1 << 31) - 1):
            bad = table.clone()
            bad[bad_at, 1] = entry
            got = cache.attend(q, bad, ln)
            assert cache.error_word() == prox.DEVERR_PAGE
            for b in range(4):
                if b != bad_at:
                    within(got[b], want[b], tol[b])


def test_attend_graphs_that_share_a_cache():
    """Two captured calls on one cache, replayed in turn on one stream between
    eager ones: each leaves the workspace as the next wants it."""
    a = attend_case(prox, [30000, 17, 900], 1, 2, 4, 128, 64, torch.bfloat16, seed=61)
    cache, q, table, lens = a
    q2, lens2 = q.flip(0).contiguous(), lens.clamp(max=600)
    want, want2 = cache.attend(q, table, lens), cache.attend(q2, table, lens2)
    out, out2 = torch.empty_like(q), torch.empty_like(q)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        cache.attend(q, table, lens, out=out)
    with torch.cuda.graph(graphs[1]):
        cache.attend(q2, table, lens2, out=out2)
    for _ in range(10):
        out.zero_(), out2.zero_()
        graphs[0].replay()
        graphs[1].replay()
        mid = cache.attend(q, table, lens2)
        graphs[0].replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(out2, want2)
        assert torch.equal(mid, cache.attend(q, table, lens2))


def test_attend_two_caches_on_two_streams():
    cases = [attend_case(prox, [9000, 40, 0], 1, 2, 4, 128, 32, torch.float16, seed=s) for s in (62, 63)]
    want = [c[0].attend(*c[1:]) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[c[0].attend(*c[1:], stream=s) for c, s in zip(cases, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for pair in got for g, w in zip(pair, want))


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("K, N, B", [(65536, 64, 16), (65536, 2, 1), (65536, 4100, 3), (128, 1 << 20, 16)])
def test_linear4_largest_shapes(K, N, B, dtype):
    codes, scales, x = linear_case(prox, K, N, B, dtype, seed=B)
    want, tol = ref.linear4(x, codes, scales)
    within(prox.Linear4(codes=codes, scales=scales)(x), want, tol)


def test_append_captured_with_padding():
    """A captured append of a fixed number of rows: those behind the step's last
    one (slot -1) leave the cache as it was."""
    cache = prox.KVCache4.zeros(4, 2, 16, 64)
    k = torch.randn((6, 2, 64), device="cuda", generator=gen_of(64))
    slots = torch.full((6,), -1, dtype=torch.int64, device="cuda")
    cache.append(k, k, slots)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.append(k, -k, slots)
    held = torch.full((64,), -1, dtype=torch.int64, device="cuda")
    for step in ([5, 1, 40], [63, 0, 2, 3, 4, 7], [], [6]):
        slots.fill_(-1)
        slots[:len(step)] = torch.tensor(step, dtype=torch.int64, device="cuda")
        graph.replay()
        for row, s in enumerate(step):
            held[s] = row
        rk, rv = cache.read(torch.arange(64, device="cuda"))
        s, c = ref.quantise(k)
        rows = c.float() * s.float()[..., None]
        want = torch.where((held >= 0)[:, None, None], rows[held.clamp(min=0)], 0.0)
        assert torch.equal(rk, want) and torch.equal(rv, -want)
