"""Raw stream handles of the 4-bit operators' calls: which torch stream a call's
tensors are made on, and that a call on the default stream's handle waits for
what is pending there and is waited for."""

import pytest
import torch

import activation_sparse_swiglu_b200 as prox
from activation_sparse_swiglu_b200 import decode4


@pytest.mark.parametrize("handle, want", [(0, "default"), (1, "default"), (2, 2), (0x7f0012345670, 0x7f0012345670)])
def test_handles_of_the_default_stream_are_the_default_stream(monkeypatch, handle, want):
    """0 and cudaStreamLegacy (1) name the default stream; every other handle is
    an external stream of that pointer."""
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: ("default", device))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr, device: (ptr, device))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    assert decode4.on_stream(handle, "a device") == (want, "a device")


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [0, 1])
def test_decode_step_on_the_default_streams_handle(handle):
    """x arrives on the default stream behind other work; the step on its handle
    uses that x, and the default stream may read the result at once."""
    from activation_sparse_swiglu_b200.stack import Stack
    d, F, H, D, B, page = 256, 512, 4, 64, 4, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    w = lambda *s: (0.05 * torch.randn(s, device="cuda", generator=g)).to(torch.bfloat16)  # noqa: E731
    ffn, qkv, wo = [(w(d, F), w(d, F), w(F, d))], w(d, 3 * H * D), w(H * D, d)
    new = torch.randn((B, d), device="cuda", generator=g)
    seen = []

    def rotate(q, k, positions):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return q * 1.5, k * 0.5

    def run(stream, pending):
        attn = prox.Attention4(qkv, wo, H, H, D, num_pages=4, page_size=page, rotate=rotate)
        stack = Stack(ffn, k=F, max_batch=B, attention=[attn])
        table = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
        ones = torch.ones(B, dtype=torch.int32, device="cuda")
        plan = prox.PagePlan(ones, None, None, torch.arange(B, device="cuda") * page, ones - 1, None)
        x = torch.zeros((B, d), device="cuda")
        torch.cuda.synchronize()
        if pending:
            torch.cuda._sleep(20_000_000)  # some 10 ms
        x.copy_(new)
        y = stack.decode(x, plan, table, stream=stream).clone()
        z = attn.step(x, plan, table, stream=stream).clone()
        torch.cuda.synchronize()
        return y, z

    with torch.cuda.stream(torch.cuda.default_stream()):
        want = run(None, False)
        got = run(handle, True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert seen == [0] * 4


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [0, 1])
def test_calls_on_the_default_streams_handle(handle):
    """Each operator by itself: inputs pending on the default stream."""
    g = torch.Generator(device="cuda").manual_seed(2)
    lin = prox.Linear4((0.05 * torch.randn((256, 512), device="cuda", generator=g)).to(torch.bfloat16))
    cache = prox.KVCache4.zeros(4, 2, 16, 64)
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    real = [torch.randn(s, device="cuda", generator=g) for s in ((2, 256), (40, 2, 64), (1, 4, 64))]
    slots, lens = torch.arange(40, device="cuda"), i32(40)

    def run(stream, pending):
        x, k, q = (torch.zeros_like(t) for t in real)
        delta = i32(0)
        torch.cuda.synchronize()
        if pending:
            torch.cuda._sleep(20_000_000)
        for dst, src in zip((x, k, q), real):
            dst.copy_(src)
        delta.fill_(3)
        y = lin.forward(x, stream=stream)
        cache.append(k, k, slots, stream=stream)
        kv = cache.read(slots, stream=stream)
        o = cache.attend(q, table, lens, stream=stream)
        p = prox.plan_pages(i32(16), delta, table.clone(), i32(5, 6), i32(2), 16, max_new=4, stream=stream)
        out = [t.clone() for t in (y, *kv, o, *p)]
        torch.cuda.synchronize()
        return out

    with torch.cuda.stream(torch.cuda.default_stream()):
        want = run(None, False)
        got = run(handle, True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
