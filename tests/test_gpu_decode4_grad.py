"""The 4-bit operators give no gradients and say so: an input (or a given
result) whose gradient or tangent a call would drop is refused."""

import pytest
import torch
import torch.autograd.forward_ad as fwd

import activation_sparse_swiglu_b200 as prox
from tests.test_gpu_decode4 import attend_case, linear_case

pytestmark = pytest.mark.gpu


def calls():
    """(name, call of one tensor, that tensor) for each floating argument."""
    codes, scales, x = linear_case(prox, 256, 64, 2, torch.float32)
    lin = prox.Linear4(codes=codes, scales=scales)
    cache, q, table, lens = attend_case(prox, [20], 1, 2, 2, 64, 16, torch.float32, seed=1)
    k, slots = torch.randn((3, 2, 64), device="cuda"), torch.arange(3, device="cuda")
    lse = torch.empty((1, 1, 4), device="cuda")
    return [("x", lambda t: lin(t), x), ("out", lambda t: lin.forward(x, out=t), torch.empty_like(lin(x))),
            ("k", lambda t: cache.append(t, k, slots), k), ("v", lambda t: cache.append(k, t, slots), k),
            ("q", lambda t: cache.attend(t, table, lens), q),
            ("out", lambda t: cache.attend(q, table, lens, out=t), torch.empty_like(q)),
            ("lse", lambda t: cache.attend(q, table, lens, lse=t), lse)]


def test_inputs_that_require_a_gradient():
    for name, call, t in calls():
        g = t.clone().requires_grad_()
        with pytest.raises(RuntimeError, match=f"^{name} carries a gradient"):
            call(g)
        with pytest.raises(RuntimeError, match=f"^{name} carries a gradient"):
            call(g * 1.0)  # not a leaf
        call(g.detach())
        with torch.no_grad():
            call(g)
        with torch.inference_mode():
            call(t.clone())


def test_inputs_with_a_tangent():
    for name, call, t in calls():
        with fwd.dual_level():
            with pytest.raises(RuntimeError, match=f"^{name} carries a gradient"):
                call(fwd.make_dual(t, torch.ones_like(t)))
            call(t)
