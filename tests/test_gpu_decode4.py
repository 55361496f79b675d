"""The 4-bit operators on a GPU against plain forms in 64 bits
(tests/decode4_helpers.py), at the sizes, types, strides and masks where they
can go wrong."""

import math
import random

import pytest
import torch

from tests import decode4_helpers as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def prox():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import activation_sparse_swiglu_b200 as p
    return p


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def within(got, want, tol):
    """Elementwise |got - want| <= tol; the worst excess on failure."""
    got = got.double()
    assert got.shape == want.shape
    assert torch.isfinite(got).all()
    off = (got - want).abs()
    bad = off > tol
    assert not bad.any(), (int(bad.sum()), float((off / tol.clamp(min=1e-300)).max()))


# ---- linear4 -----------------------------------------------------------------

def linear_case(prox, K, N, B, dtype, seed=0, spread=1.0):
    g = gen_of(seed)
    codes = ref.random_codes(g, (K, N), "cuda")
    scales = (0.01 * torch.randn((K // 128, N), device="cuda", generator=g).exp()).half()
    x = torch.randn((B, K), device="cuda", generator=g)
    if spread != 1.0:
        x = x * torch.rand((B, K), device="cuda", generator=g).mul(math.log(spread)).exp()
    return codes, scales, x.to(dtype)


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("K, N, B", [
    (128, 2, 1), (128, 16, 1), (256, 34, 3), (512, 1376, 1), (384, 100, 16), (1152, 258, 8), (640, 4098, 5),
    (4096, 6144, 1), (4096, 1030, 9), (2048, 20000, 4), (14336, 512, 2), (28672, 64, 16), (5120, 40002, 16)])
def test_linear4(prox, K, N, B, dtype):
    codes, scales, x = linear_case(prox, K, N, B, dtype, seed=K + N + B)
    lin = prox.Linear4(codes=codes, scales=scales)
    y = lin(x)
    assert y.dtype == dtype and y.shape == (B, N)
    want, tol = ref.linear4(x, codes, scales)
    within(y, want, tol)
    assert torch.equal(lin(x), y)


@pytest.mark.parametrize("B", range(1, 17))
def test_linear4_every_batch(prox, B):
    for dtype in ref.TYPES:
        codes, scales, x = linear_case(prox, 768, 500, B, dtype, seed=B)
        want, tol = ref.linear4(x, codes, scales)
        within(prox.Linear4(codes=codes, scales=scales)(x), want, tol)


def test_linear4_from_weight_equals_packed(prox):
    w = (0.02 * torch.randn((512, 1376), device="cuda", generator=gen_of(1))).to(torch.bfloat16)
    codes, scales = prox.pack_proxy(w)
    x = torch.randn((3, 512), device="cuda", generator=gen_of(2))
    assert torch.equal(prox.Linear4(w)(x), prox.Linear4(codes=codes, scales=scales)(x))


@pytest.mark.parametrize("dtype", ref.TYPES)
def test_linear4_wide_ranges(prox, dtype):
    """Tokens and groups whose magnitudes differ by many orders, zeros, and
    tiny values."""
    codes, scales, x = linear_case(prox, 1024, 96, 4, torch.float32, seed=7, spread=1e3)
    x[0] = 0
    x[1, 128:256] = 0
    x[2] *= 1e-3
    if dtype != torch.float16:
        x[3] *= 1e25
        x[2] *= 1e-30
    x = x.to(dtype)
    want, tol = ref.linear4(x, codes, scales)
    y = prox.Linear4(codes=codes, scales=scales)(x)
    assert torch.equal(y[0], torch.zeros_like(y[0]))
    if dtype == torch.float16:
        within(y, want, tol)
    else:  # in fp32's range: the largest token's values times the tiny scale stay finite
        within(y, want, tol + 2.0 ** -126)


def test_linear4_large_input_at_zero_codes(prox):
    """One input 10^4 times the others of its group, where every code is 0 (a
    byte 0x88): an fp32 result is made of the others, and keeps their bits."""
    codes, scales, x = linear_case(prox, 1024, 96, 3, torch.float32, seed=8)
    x[:, 130] = 1e4
    codes[130] = 0x88
    want, tol = ref.linear4(x, codes, scales)
    within(prox.Linear4(codes=codes, scales=scales)(x), want, tol)


@pytest.mark.parametrize("dtype", ref.TYPES)
def test_linear4_non_finite_token_stays_its_own(prox, dtype):
    codes, scales, x = linear_case(prox, 512, 64, 4, dtype, seed=11)
    clean = prox.Linear4(codes=codes, scales=scales)
    want = clean(x)
    x2 = x.clone()
    x2[1, 5] = float("inf")
    x2[3, 300] = float("nan")
    y = clean(x2)
    assert not torch.isfinite(y[1]).any() and torch.isnan(y[3]).all()
    assert torch.equal(y[0], want[0]) and torch.equal(y[2], want[2])


@pytest.mark.parametrize("dtype", ref.TYPES)
def test_linear4_strides_offsets_and_1d(prox, dtype):
    codes, scales, x = linear_case(prox, 256, 70, 6, dtype, seed=13)
    lin = prox.Linear4(codes=codes, scales=scales)
    want = lin(x)
    # rows of a wider buffer, at an odd offset; out likewise, the rest untouched
    wide = torch.full((6, 300), 7.0, dtype=dtype, device="cuda")
    wide[:, 3:259] = x
    out = torch.full((6, 91), -5.0, dtype=dtype, device="cuda")
    lin.forward(wide[:, 3:259], out=out[:, 11:81])
    assert torch.equal(out[:, 11:81], want)
    assert (out[:, :11] == -5).all() and (out[:, 81:] == -5).all()
    one = lin(x[2])
    assert one.shape == (70,) and torch.equal(one, lin(x[2:3])[0])


def test_linear4_refusals(prox):
    codes, scales, x = linear_case(prox, 256, 64, 2, torch.float32)
    lin = prox.Linear4(codes=codes, scales=scales)
    with pytest.raises(prox.ProxError, match="B=17"):
        lin(torch.zeros(17, 256, device="cuda"))
    with pytest.raises(prox.ProxError, match="B=0"):
        lin(torch.zeros(0, 256, device="cuda"))
    with pytest.raises(ValueError):
        lin(torch.zeros(2, 128, device="cuda"))
    with pytest.raises(ValueError):
        lin(torch.zeros(256, 2, device="cuda").t())
    with pytest.raises(TypeError):
        lin(torch.zeros(2, 256, device="cuda", dtype=torch.float64))
    with pytest.raises(ValueError):
        lin.forward(x, out=torch.empty(2, 64, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError):
        lin.forward(x, out=torch.empty(2, 65, device="cuda"))
    with pytest.raises(ValueError):
        prox.Linear4(codes=codes, scales=scales[:1])
    buf = torch.zeros(2, 256, device="cuda")
    with pytest.raises(prox.ProxError, match="overlap"):
        prox.Linear4(codes=codes, scales=scales).forward(buf, out=buf[:, 100:164])
    lin.close()
    with pytest.raises(RuntimeError):
        lin(x)


def test_linear4_two_streams_and_graph(prox):
    """Calls on one handle overlap on two streams; a captured call replays on
    new inputs."""
    codes, scales, x = linear_case(prox, 2048, 3000, 4, torch.bfloat16, seed=17)
    lin = prox.Linear4(codes=codes, scales=scales)
    x2 = (x.float() * 2).to(x.dtype)
    want, want2 = lin(x), lin(x2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    a, b = [], []
    for _ in range(20):
        a.append(lin.forward(x, stream=s1))
        b.append(lin.forward(x2, stream=s2))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in a) and all(torch.equal(y, want2) for y in b)
    xs, out = x.clone(), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lin.forward(xs, out=out)
    for inp, w in ((x2, want2), (x, want)):
        xs.copy_(inp)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)


@pytest.mark.parametrize("dtype, B", [(torch.float32, 16), (torch.bfloat16, 16), (torch.float32, 7)])
def test_linear4_largest_outputs_with_many_columns(prox, dtype, B):
    """Where x needs several passes and the results of all channels would not
    stay in shared memory: more channels than one launch takes."""
    K, N = 8192, (1 << 19) + 34
    codes, scales, x = linear_case(prox, K, N, B, dtype, seed=21)
    y = prox.Linear4(codes=codes, scales=scales)(x)
    for n0 in list(range(0, N, 1 << 16)) + [N - 34]:
        n1 = min(N, n0 + 2050)
        part = codes[:, n0 // 2:n1 // 2].contiguous(), scales[:, n0:n1].contiguous()
        want, tol = ref.linear4(x, *part)
        within(y[:, n0:n1], want, tol)
    # and everywhere against the same weights in narrow slices
    for n0 in range(0, N, 1 << 17):
        n1 = min(N, n0 + (1 << 17))
        sl = prox.Linear4(codes=codes[:, n0 // 2:n1 // 2].contiguous(), scales=scales[:, n0:n1].contiguous())(x)
        diff = (sl.double() - y[:, n0:n1].double()).norm() / sl.double().norm()
        assert diff <= (2e-6 if dtype == torch.float32 else 2.0 ** -8)
        sl_bad = (sl - y[:, n0:n1]).abs().amax(0) > 0.05 * sl.abs().amax()
        assert not sl_bad.any()


# ---- the cache's rows ----------------------------------------------------------

def new_cache(prox, pages, heads, page, dim):
    return prox.KVCache4.zeros(pages, heads, page, dim)


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("T, H, D, page", [(1, 1, 64, 16), (5, 3, 128, 32), (64, 8, 128, 64), (33, 2, 256, 256),
                                           (700, 4, 64, 128)])
def test_append_and_read(prox, T, H, D, page, dtype):
    g = gen_of(T + D)
    cache = new_cache(prox, T // page * 2 + 3, H, page, D)
    rows = torch.randn((T, 3, H, D), device="cuda", generator=g) * 3
    if T > 4:
        rows[1] = 0
        rows[2] *= 1e-9
        rows[3, :, :, 0] = 700.0
    rows = rows.to(dtype)
    k, v = rows[:, 1], rows[:, 2]
    slots = torch.randperm(cache.num_pages * page, device="cuda", generator=g)[:T].clone()
    if T > 2:
        slots[0] = -1
    before = [t.clone() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
    cache.append(k, v, slots)
    live = slots >= 0
    at = slots[live]
    for x, codes, scales, codes0, scales0 in ((k, cache.k_codes, cache.k_scales, before[0], before[1]),
                                              (v, cache.v_codes, cache.v_scales, before[2], before[3])):
        s, q = ref.quantise(x[live])
        codes0[at // page, :, at % page] = ref.pack(q)
        scales0[at // page, :, at % page] = s
        assert torch.equal(codes, codes0) and torch.equal(scales, scales0)
    for out_type in ref.TYPES:
        for x, got in zip((k, v), cache.read(slots, dtype=out_type)):
            s, q = ref.quantise(x)
            want = (q.float() * s.float()[..., None]).to(out_type)
            want[~live] = 0
            assert got.dtype == out_type and torch.equal(got, want)
    assert cache.error_word() == 0


def test_append_borders_are_exact(prox):
    """Values on and next to the borders between two codes, in fp32 (the
    neighbours of x / S = n + 1/2 differ by one unit in the last place)."""
    D, rows = 128, 512
    g = gen_of(3)
    amax = (torch.rand(rows, device="cuda", generator=g) * 4 + 0.1)
    s = (amax / 7).half().float()
    n = torch.randint(-7, 7, (rows, D), device="cuda", generator=g).float() + 0.5
    x = n * s[:, None]  # exact in fp32
    nudge = torch.randint(-1, 2, (rows, D), device="cuda", generator=g)
    x = torch.where(nudge > 0, torch.nextafter(x, torch.full_like(x, torch.inf)), x)
    x = torch.where(nudge < 0, torch.nextafter(x, torch.full_like(x, -torch.inf)), x)
    x = x.clamp(-amax[:, None], amax[:, None])
    x[:, 0] = amax
    cache = new_cache(prox, rows // 64, 1, 64, D)
    slots = torch.arange(rows, device="cuda")
    k = x[:, None, :].contiguous()
    cache.append(k, -k, slots)
    sw, q = ref.quantise(k)
    assert torch.equal(cache.k_scales.flatten(), sw.flatten())
    assert torch.equal(cache.k_codes.view(rows, 1, D // 2), ref.pack(q))
    assert torch.equal(cache.v_codes.view(rows, 1, D // 2), ref.pack(-q))


def test_append_non_finite_and_strides(prox):
    D = 64
    base = torch.randn((9, 2, 2 * D + 1), device="cuda", generator=gen_of(5))
    base[2, 0, 3] = float("nan")
    base[4, 1, 9] = float("inf")
    k = base[:, :, :D]  # odd row stride: no 16-byte loads
    v = base.flip(0)[:, :, D:2 * D]
    cache = new_cache(prox, 2, 2, 16, D)
    slots = torch.arange(9, device="cuda") + 5
    cache.append(k, v, slots)
    rk, rv = cache.read(slots)
    assert torch.isnan(rk[2, 0]).all() and not torch.isfinite(rk[4, 1]).any()
    ok = torch.ones((9, 2), dtype=torch.bool)
    ok[2, 0] = ok[4, 1] = False
    s, q = ref.quantise(k)
    assert torch.equal(rk[ok], (q.float() * s.float()[..., None])[ok])
    s, q = ref.quantise(v)
    fine = torch.isfinite(v).all(-1)
    assert torch.equal(rv[fine], (q.float() * s.float()[..., None])[fine])


def test_append_slots_past_the_cache(prox):
    cache = new_cache(prox, 2, 1, 16, 64)
    k = torch.ones((3, 1, 64), device="cuda")
    slots = torch.tensor([0, 32, 1 << 40], device="cuda")
    cache.append(k, k, slots)
    assert cache.error_word() == prox.DEVERR_SLOT and cache.error_word() == 0
    rk, _ = cache.read(slots)
    assert cache.error_word() == prox.DEVERR_SLOT
    assert rk[0].ne(0).all() and (rk[1:] == 0).all()
    assert (cache.k_scales.flatten()[1:] == 0).all()
    wide = torch.ones((1, 1, 64), device="cuda").expand(4, 1, 64)  # a row for every token
    cache.append(wide, wide, torch.tensor([1, 2, 3, 4], device="cuda"))
    assert (cache.read(torch.arange(1, 5, device="cuda"))[0] == rk[:1]).all()
    cache.k_scales.view(-1)[1:5] = 0
    cache.append(k[:0], k[:0], slots[:0])
    assert cache.read(slots[:0])[0].shape == (0, 1, 64)
    with pytest.raises(TypeError):
        cache.append(k, k.half(), slots)
    with pytest.raises(TypeError):
        cache.append(k, k, slots.int())
    with pytest.raises(ValueError):
        cache.append(k, k, slots[:2])
    with pytest.raises(ValueError):
        cache.append(k[:, :, :32], k[:, :, :32], slots)
    with pytest.raises(TypeError):
        cache.read(slots, dtype=torch.float64)


# ---- attention -------------------------------------------------------------------

def attend_case(prox, lens, Tq, Hkv, G, D, page, dtype, seed=0, spare_cols=2, garbage=True, sharp=1.0):
    """A cache with scattered pages.  Rows and pages that no request uses hold
    NaN scales, and table entries behind a request's last page are far out of
    range."""
    g = gen_of(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    shape = (pages, Hkv, page)
    kc, vc = (ref.random_codes(g, shape + (D,), "cuda") for _ in range(2))
    ks, vs = ((0.2 * torch.randn(shape, device="cuda", generator=g).mul(0.5).exp()).half() for _ in range(2))
    order = torch.randperm(pages, device="cuda", generator=g).int()
    table = torch.full((len(lens), max(need + [0]) + spare_cols), 1 << 30, dtype=torch.int32, device="cuda")
    unused = torch.ones((pages, page), dtype=torch.bool, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        for j in range(need[b]):
            unused[order[at + j].long(), :min(page, n - j * page)] = False
        at += need[b]
    if garbage:
        m = unused[:, None, :].expand(shape)
        ks[m] = float("nan")
        vs[m] = float("inf")
    q = (sharp * torch.randn((len(lens), Tq, Hkv * G, D), device="cuda", generator=g)).to(dtype)
    cache = prox.KVCache4(kc, ks, vc, vs)
    return cache, q, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def check_attend(prox, cache, q, table, lens, scale=None):
    B, Tq, Hq, D = q.shape
    lse = torch.empty((B, Tq, Hq), device="cuda")
    out = cache.attend(q, table, lens, scale=scale, lse=lse)
    want, wlse, tol, ltol = ref.attend(q, cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, table, lens,
                                       D ** -0.5 if scale is None else scale)
    assert cache.error_word() == 0
    within(out, want, tol)
    empty = torch.isinf(wlse)
    assert torch.equal(lse[empty].double(), wlse[empty])
    within(lse[~empty], wlse[~empty], ltol[~empty])
    again = cache.attend(q, table, lens, scale=scale)
    assert torch.equal(out, again)
    return out


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens, Tq, Hkv, G, page", [
    ([1], 1, 1, 1, 16), ([37], 1, 4, 2, 16), ([0], 1, 2, 3, 32), ([64], 1, 2, 8, 64),
    ([0, 1, 31, 32, 33, 63, 65, 200], 1, 2, 4, 32), ([500, 3, 0, 129], 1, 3, 5, 128),
    ([17, 250, 0, 2], 3, 2, 4, 16), ([1, 2, 300], 4, 1, 16, 64), ([2500], 1, 1, 4, 256), ([700, 90], 5, 2, 7, 64)])
def test_attend(prox, lens, Tq, Hkv, G, page, D, dtype):
    case = attend_case(prox, lens, Tq, Hkv, G, D, page, dtype, seed=sum(lens) + G + D)
    check_attend(prox, *case)


@pytest.mark.parametrize("dtype", ref.TYPES)
def test_attend_long_context_split_over_the_device(prox, dtype):
    """Contexts that many CTAs share, next to short ones."""
    case = attend_case(prox, [70001, 5, 9000, 0, 33], 1, 2, 4, 128, 64, dtype, seed=1)
    check_attend(prox, *case)
    case = attend_case(prox, [40000], 2, 1, 3, 128, 16, dtype, seed=2)
    check_attend(prox, *case)


@pytest.mark.parametrize("dtype", ref.TYPES)
def test_attend_many_short_requests(prox, dtype):
    r = random.Random(5)
    lens = [r.randint(0, 80) for _ in range(300)]
    case = attend_case(prox, lens, 1, 2, 4, 64, 16, dtype, seed=3)
    check_attend(prox, *case)


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("scale, sharp", [(1.0, 3.0), (0.01, 1.0), (-0.2, 1.0), (0.0, 1.0)])
def test_attend_sharp_and_flat_scores(prox, scale, sharp, dtype):
    case = attend_case(prox, [333, 64, 7], 1, 2, 4, 128, 32, dtype, seed=4, sharp=sharp)
    check_attend(prox, *case, scale=scale)


def test_attend_largest_table(prox):
    """The largest batch (its chunk counts take shared memory from the rings)."""
    lens = [(7 * i) % 40 for i in range(8192)]
    case = attend_case(prox, lens, 1, 1, 2, 64, 16, torch.bfloat16, seed=6, garbage=False)
    cache, q, table, ln = case
    out = cache.attend(q, table, ln)
    pick = list(range(0, 8192, 512)) + [8191]
    want, _, tol, _ = ref.attend(q[pick], cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, table[pick],
                                 ln[pick], 64 ** -0.5)
    within(out[pick], want, tol)
    with pytest.raises(prox.ProxError, match="B=8193"):
        cache.attend(torch.zeros((8193, 2, 64), device="cuda"), torch.zeros((8193, 1), dtype=torch.int32, device="cuda"),
                     torch.zeros(8193, dtype=torch.int32, device="cuda"))


def test_attend_offsets_past_32_bits(prox):
    """Rows more than 2^32 bytes into the codes."""
    pages, Hkv, page, D = 1 << 15, 16, 256, 128  # 8.6 GB of K codes and of V codes
    cache = prox.KVCache4.zeros(pages, Hkv, page, D)
    lens = [300, 513]
    T = sum(lens)
    g = gen_of(8)
    # page numbers whose rows start past 2^32 bytes (a page is 256 KB of codes)
    table = torch.tensor([[pages - 1, 20000, 0], [pages - 2, 3, pages - 7]], dtype=torch.int32, device="cuda")
    slots = torch.cat([table[b].long()[torch.arange(n, device="cuda") // page] * page
                       + torch.arange(n, device="cuda") % page for b, n in enumerate(lens)])
    k, v = (torch.randn((T, Hkv, D), device="cuda", generator=g) for _ in range(2))
    cache.append(k, v, slots)
    for x, got in zip((k, v), cache.read(slots)):
        s, qq = ref.quantise(x)
        assert torch.equal(got, qq.float() * s.float()[..., None])
    q = torch.randn((2, 1, 32, D), device="cuda", generator=g)
    check_attend(prox, cache, q, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dtype", ref.TYPES)
def test_attend_masked_rows_may_hold_anything(prox, dtype):
    """A drafted token's NaN scale reaches only the queries that see it."""
    cache, q, table, lens = attend_case(prox, [70], 3, 1, 2, 128, 32, dtype, seed=9)
    want = cache.attend(q, table, lens)
    cache.k_scales[table[0, 2].long(), :, 5] = float("nan")   # token 69: the newest
    cache.v_scales[table[0, 2].long(), :, 5] = float("nan")
    got = cache.attend(q, table, lens)
    assert torch.equal(got[:, :2], want[:, :2]) and torch.isnan(got[:, 2]).all()
    cache.k_scales[table[0, 2].long(), :, 5] = 0.1
    cache.v_scales[table[0, 2].long(), :, 5] = float("inf")
    got = cache.attend(q, table, lens)
    assert torch.equal(got[:, :2], want[:, :2]) and not torch.isfinite(got[:, 2]).any()


def test_attend_non_finite_query_stays_its_own(prox):
    for dtype in ref.TYPES:
        cache, q, table, lens = attend_case(prox, [40, 40], 1, 1, 4, 64, 16, dtype, seed=10)
        want = cache.attend(q, table, lens)
        q2 = q.clone()
        q2[0, 0, 1, 3] = float("nan")
        got = cache.attend(q2, table, lens)
        assert torch.isnan(got[0, 0, 1]).all()
        assert torch.equal(got[1], want[1])
        for h in (0, 2, 3):
            assert torch.isfinite(got[0, 0, h]).all()


def test_attend_strides_3d_and_untouched_surroundings(prox):
    cache, q, table, lens = attend_case(prox, [100, 45, 0], 1, 2, 3, 128, 32, torch.bfloat16, seed=12)
    want = cache.attend(q, table, lens)
    B, _, Hq, D = q.shape
    rows = torch.zeros((B, Hq + 4, D + 1), dtype=q.dtype, device="cuda")  # odd strides
    rows[:, 1:Hq + 1, :D] = q[:, 0]
    assert torch.equal(cache.attend(rows[:, 1:Hq + 1, :D], table, lens), want[:, 0])
    heads_first = q[:, 0].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(cache.attend(heads_first, table, lens), want[:, 0])
    wide = torch.full((B, table.shape[1] + 5), -9, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    assert torch.equal(cache.attend(q, wide[:, :table.shape[1]], lens), want)
    buf = torch.full((B + 2, 1, Hq, D), 3.0, dtype=q.dtype, device="cuda")
    cache.attend(q, table, lens, out=buf[1:B + 1])
    assert torch.equal(buf[1:B + 1], want) and (buf[0] == 3).all() and (buf[B + 1] == 3).all()


def test_attend_bad_pages_and_lengths_are_reported(prox):
    """Entries and lengths out of range: an error bit, other requests intact."""
    cache, q, table, lens = attend_case(prox, [70, 40], 1, 1, 4, 64, 16, torch.float32, seed=13, garbage=False)
    want = cache.attend(q, table, lens)
    for entry in (-1, cache.num_pages, 1 << 30, -(1 << 31)):
        bad = table.clone()
        bad[0, 1] = entry
        got = cache.attend(q, bad, lens)
        assert cache.error_word() == prox.DEVERR_PAGE
        assert torch.equal(got[1], want[1])
    for n in (-5, 1 << 30, -(1 << 31), (1 << 31) - 1):
        ln = lens.clone()
        ln[0] = n
        got = cache.attend(q, table.clamp(max=0), ln)
        assert cache.error_word() == prox.DEVERR_LEN
    assert torch.equal(cache.attend(q, table, lens), want) and cache.error_word() == 0


def test_attend_refusals(prox):
    cache, q, table, lens = attend_case(prox, [20], 1, 2, 2, 64, 16, torch.float16, seed=14)
    with pytest.raises(ValueError):
        cache.attend(q[..., :32], table, lens)
    with pytest.raises(TypeError):
        cache.attend(q.double(), table, lens)
    with pytest.raises(ValueError):
        cache.attend(q, table.long(), lens)
    with pytest.raises(TypeError):
        cache.attend(q, table, lens.long())
    with pytest.raises(ValueError):
        cache.attend(q, table[:0], lens)
    with pytest.raises(prox.ProxError, match="multiple"):
        cache.attend(q[:, :, :3], table, lens)
    with pytest.raises(prox.ProxError, match="finite"):
        cache.attend(q, table, lens, scale=float("inf"))
    with pytest.raises(ValueError):
        cache.attend(q, table, lens, out=torch.empty_like(q).float())
    with pytest.raises(ValueError):
        cache.attend(q, table, lens, lse=torch.empty(1, device="cuda"))
    # rows that share memory could not be told apart
    with pytest.raises(ValueError, match="contiguous rows"):
        cache.attend(q.expand(2, -1, -1, -1), table.expand(2, -1), lens.repeat(2))
    # no columns at all: every length but 0 is out of range
    zero = torch.zeros_like(lens)
    assert (cache.attend(q, table[:, :0], zero) == 0).all() and cache.error_word() == 0
    cache.close()
    with pytest.raises(RuntimeError):
        cache.attend(q, table, lens)


def test_attend_captured_and_replayed(prox):
    """One captured step replays on other lengths: nothing of them is on the host."""
    cache, q, table, lens = attend_case(prox, [3000, 17, 900], 1, 2, 4, 128, 64, torch.bfloat16, seed=15)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    ln = lens.clone()
    cache.attend(q, table, ln, out=out)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        cache.attend(q, table, ln, out=out)
    for new in ([3000, 17, 900], [1, 1, 1], [0, 17, 63], [2999, 0, 512]):
        ln.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, cache.attend(q, table, ln))


# ---- page plans ------------------------------------------------------------------

def run_plan(prox, lens, delta, cols, page, free, count, max_new, commit=False, table=None):
    r = random.Random(sum(lens) + cols)
    B = len(lens)
    if table is None:
        table = [[r.randint(0, 10 ** 6) for _ in range(cols)] for _ in range(B)]
    want = ref.plan(lens, delta, table, free, count, page, max_new)
    dev = lambda x, dt=torch.int32: torch.tensor(x, dtype=dt, device="cuda")  # noqa: E731
    tl, tt, tf, tc = dev(lens), dev(table).reshape(B, cols), dev(free), dev([count])
    for _ in range(1 if commit else 2):  # an uncommitted plan can be made again
        p = prox.plan_pages(tl, dev(delta), tt, tf, tc, page, max_new=max_new, commit=commit)
        ok, wl, wc, wcu, ws, wp, wt, wf = want
        assert int(p.status) == (0 if ok else 1)
        assert p.lens.tolist() == wl and int(p.count) == wc and p.cu.tolist() == wcu
        assert p.slots.tolist() == ws and p.positions.tolist() == wp
        assert tt.tolist() == wt and tf.tolist() == wf
    if commit:
        assert tl.tolist() == wl and int(tc) == wc
    else:
        assert tl.tolist() == lens and int(tc) == count
    return want[0]


@pytest.mark.parametrize("commit", [False, True])
@pytest.mark.parametrize("B, page, longest, most", [(1, 16, 0, 1), (1, 64, 500, 300), (7, 16, 40, 20),
                                                    (64, 64, 4000, 1), (257, 32, 300, 64), (1021, 16, 900, 200),
                                                    (3, 1, 9, 9), (40, 7, 100, 33)])
def test_plan_pages(prox, B, page, longest, most, commit):
    r = random.Random(B + page)
    lens = [r.randint(0, longest) for _ in range(B)]
    delta = [r.choice([r.randint(0, most), r.randint(0, most), -n, -r.randint(0, n)]) for n in lens]
    cols = -(-(longest + most) // page)
    need = sum(-(-n // page) for n in lens)
    spare = sum(-(-max(d, 0) // page) + 1 for d in delta)
    free = list(range(10 ** 6, 10 ** 6 + spare)) + [-7] * need
    assert run_plan(prox, lens, delta, cols, page, free, spare, sum(max(d, 0) for d in delta) + 5, commit)


def test_plan_pages_largest(prox):
    r = random.Random(0)
    lens = [r.randint(0, 40) for _ in range(8192)]
    delta = [r.randint(-n, 9) for n in lens]
    free = list(range(9000)) + [-1] * 30000
    assert run_plan(prox, lens, delta, 4, 16, free, 9000, 50000)


def test_plan_pages_one_long_prompt(prox):
    assert run_plan(prox, [5, 0, 70], [3, 30000, -70], 2000, 16, list(range(3000)), 2000, 30010)


def test_plan_pages_exact_fit_and_refusals(prox):
    free = [4, 9, 2, -1, -1]
    # takes exactly what is free and what the second row returns
    assert run_plan(prox, [0, 32], [64, -32], 4, 16, free, 3, 64)
    assert not run_plan(prox, [0, 32], [64, -16], 3, 16, free, 3, 64)       # past the columns
    assert not run_plan(prox, [0, 32], [64, 16], 4, 16, free, 3, 80)        # too few pages
    assert not run_plan(prox, [0, 32], [64, -32], 4, 16, free, 3, 63)       # too many tokens
    assert not run_plan(prox, [0, 32], [1, -33], 4, 16, free, 3, 64)        # drops more than there is
    assert not run_plan(prox, [0, -1], [1, 5], 4, 16, free, 3, 64)          # a length below 0
    assert not run_plan(prox, [0, 64], [0, -64], 4, 16, free, 3, 64)        # no room to return to
    assert not run_plan(prox, [0, 70], [1, -60], 4, 16, free, 3, 64)        # a length past the columns
    assert not run_plan(prox, [0, 0], [1, 0], 4, 16, free, -1, 64)          # a count below 0
    assert not run_plan(prox, [0, 5], [2 ** 31 - 1, 2 ** 31 - 1], 4, 16, free, 3, 64)
    assert run_plan(prox, [0, 0], [0, 0], 0, 16, [], 0, 0, table=[[], []])


def test_plan_pages_refuses_rows_that_share_memory(prox):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    with pytest.raises(ValueError, match="contiguous rows"):
        prox.plan_pages(i32([0, 0]), i32([1, 1]), i32([[0, 0]]).expand(2, -1), i32([5, 6]), i32([2]), 16, max_new=2)


def test_plan_pages_strided_table_and_max_new_zero(prox):
    wide = torch.full((2, 9), -3, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    p = prox.plan_pages(i32([0, 0]), i32([17, 0]), wide[:, 2:6], i32([5, 6, 7]), i32([3]), 16, max_new=20)
    assert int(p.status) == 0 and wide.tolist() == [[-3, -3, 7, 6, -3, -3, -3, -3, -3], [-3] * 9]
    p = prox.plan_pages(i32([40]), i32([-40]), i32([[1, 2, 3]]), i32([0, 0, 0, 0]), i32([1]), 16, max_new=0)
    assert int(p.status) == 0 and int(p.count) == 4 and p.slots.numel() == 0


# ---- together ---------------------------------------------------------------------

def test_decode_steps_of_a_small_model(prox):
    """Steps of one attention sub-layer as a server makes them: a plan, the
    projections, the rows, the attention and the output projection; requests
    come, go and are rolled back.  Against the plain forms, fed with the
    library's own rows."""
    d, Hq, Hkv, D, page, B = 512, 8, 4, 64, 16, 5
    g = gen_of(20)
    w_qkv, wo = ((0.05 * torch.randn(s, device="cuda", generator=g)).to(torch.bfloat16)
                 for s in ((d, (Hq + 2 * Hkv) * D), (Hq * D, d)))
    qkv_lin, o_lin = prox.Linear4(w_qkv), prox.Linear4(wo)
    cache = prox.KVCache4.zeros(40, Hkv, page, D)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    table = torch.full((B, 8), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(40, dtype=torch.int32, device="cuda")
    count = torch.tensor([40], dtype=torch.int32, device="cuda")
    r = random.Random(2)
    for step in range(12):
        now = lens.tolist()
        # one new token for most; some idle, one rolled back, one finished
        delta = [1] * B
        if step % 4 == 3:
            delta[step % B] = -min(now[step % B], 1 + step)
        if step % 5 == 4:
            delta[(step + 1) % B] = -now[(step + 1) % B]
        plan = prox.plan_pages(lens, torch.tensor(delta, dtype=torch.int32, device="cuda"), table, free, count,
                               page, max_new=B + 2, commit=True)
        assert int(plan.status) == 0
        n_new = sum(x > 0 for x in delta)
        rows = [b for b in range(B) if delta[b] > 0]
        x = torch.randn((n_new, d), device="cuda", generator=g)
        qkv = qkv_lin(x)
        heads = qkv.view(n_new, Hq + 2 * Hkv, D)
        q, k, v = heads[:, :Hq], heads[:, Hq:Hq + Hkv], heads[:, Hq + Hkv:]
        cache.append(k, v, plan.slots[:n_new])
        sub = torch.tensor(rows, device="cuda")
        o = cache.attend(q, table[sub].contiguous(), plan.lens[sub].contiguous())
        y = o_lin(o.reshape(n_new, Hq * D))
        # each stage against its plain form
        want, tol = ref.linear4(x, *prox.pack_proxy(w_qkv))
        within(qkv, want, tol)
        for z, got in zip((k, v), cache.read(plan.slots[:n_new])):
            s, qq = ref.quantise(z)
            assert torch.equal(got, qq.float() * s.float()[..., None])
        want, _, tol, _ = ref.attend(q[:, None], cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales,
                                     table[sub], plan.lens[sub], D ** -0.5)
        within(o[:, None], want, tol)
        want, tol = ref.linear4(o.reshape(n_new, -1), *prox.pack_proxy(wo))
        within(y, want, tol)
    live = sum(-(-n // page) for n in lens.tolist())
    assert int(count) == 40 - live
    pages = [p for b in range(B) for p in table[b, :-(-int(lens[b]) // page)].tolist()] + free[:40 - live].tolist()
    assert sorted(pages) == list(range(40))
    assert cache.error_word() == 0


def test_stack_decodes_through_attention(prox):
    """Stack.decode: three steps of four requests through two layers, each stage
    against the plain forms fed with the library's own input to it, and equal to
    the same calls made one by one."""
    from activation_sparse_swiglu_b200.stack import Stack
    from oracle import prox_oracle as orc
    d, F, Hq, Hkv, D, B, n_layers, page = 256, 512, 4, 2, 64, 4, 2, 16
    g = gen_of(30)
    w = lambda *s: (0.05 * torch.randn(s, device="cuda", generator=g)).to(torch.bfloat16)  # noqa: E731
    ffn = [(w(d, F), w(d, F), w(F, d)) for _ in range(n_layers)]
    qkv, wo = [w(d, (Hq + 2 * Hkv) * D) for _ in range(n_layers)], [w(Hq * D, d) for _ in range(n_layers)]
    seen = []

    def rotate(q, k, positions):
        seen.append(positions.tolist())
        turn = 1.0 - 0.01 * positions.to(q.dtype)[:, None, None]
        return q * turn, k * turn

    def build():
        attn = [prox.Attention4(a, o, Hq, Hkv, D, num_pages=12, page_size=page, rotate=rotate)
                for a, o in zip(qkv, wo)]
        return Stack(ffn, k=F, max_batch=B, attention=attn)

    stack, by_hand = build(), build()
    lens = torch.tensor([0, 15, 31, 2], dtype=torch.int32, device="cuda")
    old = lens.clone()
    table = torch.tensor([[-1, -1, -1], [7, -1, -1], [3, 5, -1], [1, -1, -1]], dtype=torch.int32, device="cuda")
    free, count = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 2, 4, 6, 8, 9, 10, 11], [8]))
    for a, b in zip(stack.attention, by_hand.attention):  # earlier tokens: the same rows in both
        s = torch.cat([table[i, torch.arange(int(n)) // page].long() * page + torch.arange(int(n), device="cuda") % page
                       for i, n in enumerate(old.tolist()) if n])
        k, v = (torch.randn((s.numel(), Hkv, D), device="cuda", generator=g) for _ in range(2))
        a.cache.append(k, v, s)
        b.cache.append(k, v, s)
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    for step in range(3):
        plan = prox.plan_pages(lens, one, table, free, count, page, max_new=B, commit=True)
        assert int(plan.status) == 0 and plan.positions.tolist() == (old + step).tolist()
        x = torch.randn((B, d), device="cuda", generator=g)
        y = stack.decode(x, plan, table)
        h = x
        for li in range(n_layers):
            at = by_hand.attention[li]
            want, tol = ref.linear4(h, *prox.pack_proxy(qkv[li]))
            proj = at.qkv(h)
            within(proj, want, tol)
            heads = proj.view(B, Hq + 2 * Hkv, D)
            q, k = rotate(heads[:, :Hq], heads[:, Hq:Hq + Hkv], plan.positions[:B])
            at.cache.append(k, heads[:, Hq + Hkv:], plan.slots[:B])
            o = at.cache.attend(q, table, plan.lens)
            want, _, tol, _ = ref.attend(q[:, None], at.cache.k_codes, at.cache.k_scales, at.cache.v_codes,
                                         at.cache.v_scales, table, plan.lens, D ** -0.5)
            within(o[:, None], want, tol)
            a = at.out(o.view(B, Hq * D))
            z = prox.rmsnorm(a)
            out = by_hand.layers[li].forward(z)
            for b in range(B):  # k = d_ff and tau 0: the dense FFN
                dense = orc.dense_ffn(z[b].cpu().numpy(), *(t.float().cpu().numpy() for t in ffn[li]))
                got = out[b].double().cpu()
                assert float((got - torch.from_numpy(dense)).norm()) <= 5e-3 * float(torch.from_numpy(dense).norm())
            h = prox.rmsnorm(out)
        assert torch.equal(y, out)
    for a, b in zip(stack.attention, by_hand.attention):
        for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
            assert torch.equal(getattr(a.cache, name), getattr(b.cache, name))
        assert a.cache.error_word() == 0
    stack.close()
    by_hand.close()
    with pytest.raises(RuntimeError):
        Stack(ffn, k=F).decode(x, plan, table)
    with pytest.raises(ValueError):
        Stack(ffn, k=F, attention=[None])
    with pytest.raises(ValueError):
        prox.Attention4(qkv[0], wo[0], 4, 3, D, num_pages=4)
    with pytest.raises(ValueError):
        prox.Attention4(qkv[0], qkv[0], Hq, Hkv, D, num_pages=4)


@pytest.mark.parametrize("raw", [False, True])
def test_decode_step_belongs_to_its_stream(prox, raw):
    """stream= as a torch stream or a raw handle: rotate() runs on it, and the
    tensors the step makes come from its memory, so that what the current
    stream makes and fills meanwhile cannot be theirs."""
    from activation_sparse_swiglu_b200.stack import Stack
    d, F, H, D, B, page = 256, 512, 4, 64, 4, 16
    g = gen_of(31)
    w = lambda *s: (0.05 * torch.randn(s, device="cuda", generator=g)).to(torch.bfloat16)  # noqa: E731
    ffn, qkv, wo = [(w(d, F), w(d, F), w(F, d))], w(d, 3 * H * D), w(H * D, d)
    seen = []

    def rotate(q, k, positions):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return q * 1.5, k * 0.5

    def run(stream):
        attn = prox.Attention4(qkv, wo, H, H, D, num_pages=4, page_size=page, rotate=rotate)
        stack = Stack(ffn, k=F, max_batch=B, attention=[attn])
        table = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
        ones = torch.ones(B, dtype=torch.int32, device="cuda")
        plan = prox.PagePlan(ones, None, None, torch.arange(B, device="cuda") * page, ones - 1, None)
        x = torch.randn((B, d), device="cuda", generator=gen_of(32))
        torch.cuda.synchronize()
        y = stack.decode(x, plan, table, stream=stream)
        trash = [torch.full((B, n), 7.0, device="cuda") for n in (d, d, d, H * D, 3 * H * D)]
        torch.cuda.synchronize()
        del trash
        return y

    side = torch.cuda.Stream()
    want = run(None)
    assert torch.equal(run(side.cuda_stream if raw else side), want)
    assert seen == [torch.cuda.current_stream().cuda_stream, side.cuda_stream]
