"""What inputs of the 4-bit operators must not lose.  Codes enter the products as
integers, so a large 16-bit input costs its small neighbours nothing where its
own codes are 0; query rows have powers of two of their own, so no head costs
another.  Against plain forms in 64 bits, with bounds that count fp32 sums and
each rounding."""

import math

import pytest
import torch

import activation_sparse_swiglu_b200 as prox
from tests import decode4_helpers as ref
from tests.test_gpu_decode4 import attend_case, gen_of, linear_case, within

pytestmark = pytest.mark.gpu
HALVES = [torch.float16, torch.bfloat16]


def linear4(x, codes, scales):
    """y = x W in 64 bits, and the bound on a result's error for 16-bit x: a sum
    of n fp32 terms is off by n 2^-23 of the terms' magnitudes (a group's 8
    tensor core steps, the K / 128 groups' sums with 3 multiplications each, 24
    joins over warps and CTAs); x is exact down to 2^-25 of its group's largest
    magnitude and has a step of 2^-38 of it below; the result is rounded once."""
    K, N = codes.shape[0], scales.shape[1]
    q, s = ref.unpack(codes).double().view(K // 128, 128, N), scales.double()[:, None, :]
    xd = x.double()
    y = xd @ (q * s).view(K, N)
    size = q.abs() * s.abs()
    top = xd.abs().view(-1, K // 128, 128).amax(-1)
    tol = (K // 128 + 8 + 3 + 24) * 2.0 ** -23 * (xd.abs() @ size.view(K, N)) + ref.HALF_STEP[x.dtype] * y.abs()
    tol = tol + 2.0 ** -38 * (top @ size.sum(1))
    return y, tol + (2.0 ** -24 if x.dtype == torch.float16 else 0.0)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("B", [1, 3, 9, 16])
@pytest.mark.parametrize("large, rows", [(1e4, [130]), (6e4, [0, 127, 640]), (1e3, list(range(256, 320)))])
def test_linear4_large_inputs_at_zero_codes(B, large, rows, dtype):
    """Inputs far above their group's others where every code is 0 (a byte 0x88):
    the result is made of the others, and is as good as without them."""
    codes, scales, x = linear_case(prox, 1024, 198, B, torch.float32, seed=B)
    codes[rows] = 0x88
    x[:, rows] = large
    x = x.to(dtype)
    lin = prox.Linear4(codes=codes, scales=scales)
    want, tol = linear4(x, codes, scales)
    within(lin(x), want, tol)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("K, N, B", [(128, 2, 1), (512, 1376, 1), (1152, 258, 8), (640, 4098, 5), (28672, 64, 16),
                                     (4096, 1030, 9), (8192, 3000, 2)])
def test_linear4_sums_are_fp32(K, N, B, dtype):
    codes, scales, x = linear_case(prox, K, N, B, dtype, seed=K + N + B, spread=30.0)
    want, tol = linear4(x, codes, scales)
    within(prox.Linear4(codes=codes, scales=scales)(x), want, tol)


def attend(q, cache, table, lens, scale):
    """Attention in 64 bits and the bound on a result's error for 16-bit q.
    Scores: sums of D products in fp32 (D / 16 tensor core steps), 4 more
    roundings; q is exact down to 2^-25 of its row's largest magnitude and has a
    step of 2^-38 of it below.  Weights: rounded to 11 bits, an exponential good
    to 2^-22.  Outputs: steps of at most 64 rows of 4 tensor core steps each,
    joined at most 12 + 148 times; a weight below 2^-28 of its step's largest has
    a step of 2^-38 of it.  The result is rounded once."""
    B, Tq, Hq, D = q.shape
    Hkv, page = cache.k_scales.shape[1], cache.k_scales.shape[2]
    G = Hq // Hkv
    out = torch.zeros((B, Tq, Hq, D), dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for b, n in enumerate(lens.tolist()):
        ids = table[b, :-(-n // page)].long()
        for h in range(Hkv):
            k, v = ((ref.unpack(c[ids, h]).double() * s[ids, h].double()[..., None]).flatten(0, 1)[:n]
                    for c, s in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)))
            for i in range(Tq):
                m = n - Tq + i + 1
                if m <= 0:
                    continue
                at = (b, i, slice(h * G, (h + 1) * G))
                qd = q[at].double()
                p = torch.softmax(qd @ k[:m].T * scale, -1)
                out[at] = p @ v[:m]
                e = (D / 16 + 6) * 2.0 ** -23 * (qd.abs() @ k[:m].abs().T).amax(-1, keepdim=True)
                e = abs(scale) * (e + 2.0 ** -38 * qd.abs().amax(-1, keepdim=True) * k[:m].abs().sum(-1).max())
                rel = 2 * e + 2.0 ** -11 + 2.0 ** -22 + (m / 16 + 180) * 2.0 ** -23
                tol[at] = rel * (p @ v[:m].abs()) + m * 2.0 ** -38 * v[:m].abs().max() + ref.HALF_STEP[q.dtype] * out[at].abs()
    return out, tol + (2.0 ** -24 if q.dtype == torch.float16 else 0.0)


def check(case, scale=None):
    cache, q, table, lens = case
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    want, tol = attend(q, cache, table, lens, scale)
    within(cache.attend(q, table, lens, scale=scale), want, tol)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens, Tq, Hkv, G, page", [([1, 37], 1, 4, 2, 16), ([200, 3000, 64], 1, 2, 4, 32),
                                                    ([17, 250, 0, 2], 3, 2, 4, 16), ([700, 90], 5, 2, 7, 64)])
def test_attend_sums_are_fp32(lens, Tq, Hkv, G, page, D, dtype):
    check(attend_case(prox, lens, Tq, Hkv, G, D, page, dtype, seed=sum(lens) + D))


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attend_large_query_elements_at_zero_codes(D, dtype):
    """Query elements far above the others where every key's code is 0: the
    scores are made of the others."""
    cache, q, table, lens = attend_case(prox, [300, 64, 5], 2, 2, 3, D, 32, dtype, seed=D)
    for d, large in ((2, 1e4), (D - 1, -3e4)):  # an even and an odd element
        codes = cache.k_codes[..., d // 2]
        cache.k_codes[..., d // 2] = codes & 0xF0 | 0x08 if d % 2 == 0 else codes & 0x0F | 0x80
        q[..., d] = large
    check((cache, q, table, lens))


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("score", [8.0, 16.0])
def test_attend_heavy_row_of_zero_codes(score, D, dtype):
    """A row with nearly all of the weight whose value codes are 0 in one half:
    there the result is made of the other rows."""
    cache, q, table, lens = attend_case(prox, [400, 70], 1, 1, 4, D, 16, dtype, seed=D + 1)
    q.copy_(torch.randn(q.shape, device="cuda", generator=gen_of(1)).sign())  # q . q = D
    for b, j in ((0, 123), (1, 0)):
        page, row = int(table[b, j // 16]), j % 16
        cache.k_codes[page, 0, row] = ref.pack(7 * q[b, 0, 0].long())[None]
        cache.k_scales[page, 0, row] = score / (7.0 * D ** 0.5)  # head 0's score for it
        cache.v_codes[page, 0, row, :D // 4] = 0x88
    check((cache, q, table, lens))


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("small", [1e-3, 1e-4, 1e-5])
def test_attend_small_queries_under_a_large_scale(small, dtype):
    """Queries near the end of fp16's range keep their bits; the scale brings
    their scores to the usual size."""
    for D in (64, 128, 256):
        cache, q, table, lens = attend_case(prox, [300, 33], 1, 2, 4, D, 32, torch.float32, seed=D + 2)
        check((cache, (q * small).to(dtype), table, lens), scale=D ** -0.5 / small)


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("G, Tq, D", [(4, 1, 64), (4, 1, 128), (3, 3, 128), (5, 1, 256)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attend_non_finite_query_leaves_its_block_as_it_was(bad, G, Tq, D, dtype):
    """Every other query of the block has the same bits as without it, queries
    past fp16's range among them."""
    cache, q, table, lens = attend_case(prox, [400, 40], Tq, 1, G, D, 16, dtype, seed=G + D)
    size = 1.0 if dtype == torch.float16 else 2.0 ** 20
    q = q * size
    want = cache.attend(q, table, lens, scale=D ** -0.5 / size)
    assert torch.isfinite(want).all()
    for i, h in ((0, 0), (Tq - 1, G - 1)):
        q2 = q.clone()
        q2[0, i, h, 3] = bad
        got = cache.attend(q2, table, lens, scale=D ** -0.5 / size)
        assert not torch.isfinite(got[0, i, h]).any()
        got[0, i, h] = want[0, i, h]
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ref.TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Tq", [1, 3])
def test_attend_heads_of_very_different_size(Tq, D, dtype):
    """Heads of one group whose queries differ by many orders: each is as good
    as alone, at the scale that brings its scores to the usual size."""
    steps = [0, 8, 16] if dtype == torch.float16 else [0, 20, 40, 60]
    cache, q, table, lens = attend_case(prox, [300, 33], Tq, 2, len(steps), D, 32, torch.float32, seed=D + 3)
    for j, e in enumerate(steps):
        q[:, :, j::len(steps)] *= 2.0 ** -e
    q = q.to(dtype)
    for e in steps:
        scale = D ** -0.5 * 2.0 ** e
        if dtype == torch.float32:
            want, _, tol, _ = ref.attend(q, cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, table, lens,
                                         scale)
        else:
            want, tol = attend(q, cache, table, lens, scale)
        within(cache.attend(q, table, lens, scale=scale), want, tol)


@pytest.mark.parametrize("dtype", ref.TYPES)
def test_attend_zero_queries_beside_others(dtype):
    """A query of zeros weighs all its rows alike, whatever the others are."""
    cache, q, table, lens = attend_case(prox, [300], 1, 1, 4, 128, 32, dtype, seed=5)
    q[:, :, 1] = 0
    q[:, :, 2] *= 1e-4
    for q in (q, torch.zeros_like(q)):
        want, tol = attend(q, cache, table, lens, 128 ** -0.5)  # (for fp32 wider than it need be)
        lse = torch.empty((1, 1, 4), device="cuda")
        within(cache.attend(q, table, lens, lse=lse), want, tol)
        assert abs(float(lse[0, 0, 1]) - math.log(300)) <= 2.0 ** -20
