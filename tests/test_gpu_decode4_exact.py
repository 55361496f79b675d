"""What 16-bit inputs of the 4-bit operators must not lose: codes enter the
products as integers, so a large input costs its small neighbours nothing where
its own codes are 0.  Against plain forms in 64 bits, with bounds that count
fp32 sums and each rounding."""

import pytest
import torch

import activation_sparse_swiglu_b200 as prox
from tests import decode4_helpers as ref
from tests.test_gpu_decode4 import linear_case, within

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
