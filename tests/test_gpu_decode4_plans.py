"""Decode steps under plans in which not every request gains a token, and calls
that a step refuses before it has changed anything."""

import pytest
import torch

import activation_sparse_swiglu_b200 as prox
from activation_sparse_swiglu_b200.stack import Stack
from tests.test_gpu_decode4 import gen_of

pytestmark = pytest.mark.gpu
D_MODEL, FF, HQ, HKV, DIM, PAGE = 256, 512, 4, 2, 64, 16


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def build(n_layers, rotate=None, seed=50, max_batch=6):
    g = gen_of(seed)
    w = lambda *s: (0.05 * torch.randn(s, device="cuda", generator=g)).to(torch.bfloat16)  # noqa: E731
    ffn = [(w(D_MODEL, FF), w(D_MODEL, FF), w(FF, D_MODEL)) for _ in range(n_layers)]
    attn = [prox.Attention4(w(D_MODEL, (HQ + 2 * HKV) * DIM), w(HQ * DIM, D_MODEL), HQ, HKV, DIM, num_pages=12,
                            page_size=PAGE, rotate=rotate) for _ in range(n_layers)]
    return Stack(ffn, k=FF, max_batch=max_batch, attention=attn)


def tensors(stack):
    return [t for a in stack.attention for t in (a.cache.k_codes, a.cache.k_scales, a.cache.v_codes, a.cache.v_scales)]


def fill(stack, table, lens, seed):
    g = gen_of(seed)
    slots = torch.cat([table[i].long()[torch.arange(n, device="cuda") // PAGE] * PAGE
                       + torch.arange(n, device="cuda") % PAGE for i, n in enumerate(lens) if n])
    for a in stack.attention:
        k, v = (torch.randn((slots.numel(), HKV, DIM), device="cuda", generator=g) for _ in range(2))
        a.cache.append(k, v, slots)


@pytest.mark.parametrize("deltas", [(1, -20, 1, 0, 1), (0, 1, -3, 1, 0), (-5, 0, 0, -1, 0), (1, 1, 1, 1, 1)])
def test_requests_that_gain_no_token(deltas):
    """Requests that finish, idle or are rolled back between others: each row
    goes to its own request's slot, the others' caches stay, and a request
    without a new token attends to what it has."""
    seen = []

    def rotate(q, k, positions):
        seen.append(positions.tolist())
        turn = 1.0 - 0.01 * positions.to(q.dtype)[:, None, None]
        return q * turn, k * turn

    stack, by_hand = build(2, rotate), build(2)
    now = [5, 20, 16, 31, 0]
    now[0], now[3] = max(now[0], -deltas[0]), max(now[3], -deltas[3])
    table = i32(3, -1, -1, 5, 7, -1, 1, -1, -1, 2, 4, -1, -1, -1, -1).view(5, 3)
    for s in (stack, by_hand):
        fill(s, table, now, 51)
    plan = prox.plan_pages(i32(*now), i32(*deltas), table, i32(0, 6, 8, 9, 0, 0, 0, 0, 0), i32(4), PAGE, max_new=7)
    assert int(plan.status) == 0
    x = torch.randn((5, D_MODEL), device="cuda", generator=gen_of(52))
    y = stack.decode(x, plan, table)
    new = [i for i, d in enumerate(deltas) if d > 0]
    lens = [n + d for n, d in zip(now, deltas)]
    at = torch.tensor(new, device="cuda", dtype=torch.long)
    h = x
    for li, a in enumerate(by_hand.attention):
        heads = a.qkv(h).view(5, HQ + 2 * HKV, DIM)
        q, k = rotate(heads[:, :HQ], heads[:, HQ:HQ + HKV], i32(*(max(n - 1, 0) for n in lens)))
        a.cache.append(k[at].contiguous(), heads[:, HQ + HKV:][at].contiguous(), plan.slots[:len(new)])
        o = a.cache.attend(q, table, plan.lens)
        out = by_hand.layers[li].forward(prox.rmsnorm(a.out(o.view(5, HQ * DIM))))
        if li == 0:  # the sub-layer by itself (same weights) works the plan out too
            twin = build(2)
            fill(twin, table, now, 51)
            twin.attention[0].rotate = rotate
            assert torch.equal(twin.attention[0].step(h, plan, table), a.out(o.view(5, HQ * DIM)))
        h = prox.rmsnorm(out)
    assert torch.equal(y, out)
    assert all(torch.equal(a, b) for a, b in zip(tensors(stack), tensors(by_hand)))
    assert all(p == [max(n - 1, 0) for n in lens] for p in seen)
    rows = plan.per_request()
    assert rows.per_request() is rows
    # by its definition, on the host
    want = [-1] * 5
    for n, i in enumerate(new):
        want[i] = int(table[i, (lens[i] - 1) // PAGE]) * PAGE + (lens[i] - 1) % PAGE
    assert rows.slots.tolist() == want


def test_plan_that_does_not_fit_caches_nothing():
    stack = build(1)
    table = i32(0, 1).view(2, 1)
    fill(stack, table, [16, 3], 53)
    before = [t.clone() for t in tensors(stack)]
    for room in (4, 0):
        plan = prox.plan_pages(i32(16, 3), i32(1, 1), table, i32(5), i32(0), PAGE, max_new=room)
        assert int(plan.status) == 1
        stack.decode(torch.randn((2, D_MODEL), device="cuda"), plan, table)
        assert all(torch.equal(a, b) for a, b in zip(tensors(stack), before))


def test_steps_are_refused_before_they_change_anything():
    stack = build(1, max_batch=2)
    table, lens = torch.arange(3, dtype=torch.int32, device="cuda").view(3, 1), i32(1, 1, 1)
    plan = prox.PagePlan(lens, None, None, torch.arange(3, device="cuda") * PAGE, lens - 1, None)
    two = prox.PagePlan(lens[:2], None, None, plan.slots[:2], plan.positions[:2], None)
    before = [t.clone() for t in tensors(stack)]
    x = torch.randn((3, D_MODEL), device="cuda")
    for bad, kind, args in ((x, ValueError, (plan, table)), (x[:2].half(), TypeError, (two, table[:2])),
                            (x[:2].cpu(), TypeError, (two, table[:2])), (x[0], ValueError, (two, table[:2])),
                            (x[:0], ValueError, (two, table[:2]))):
        for stream in (None, torch.cuda.Stream()):
            with pytest.raises(kind):
                stack.decode(bad, *args, stream=stream)
    assert all(torch.equal(a, b) for a, b in zip(tensors(stack), before))
    stack.decode(x[:2], two, table[:2])
    assert not torch.equal(tensors(stack)[0], before[0])


def test_steps_of_other_sizes_than_their_plan_are_refused():
    """Before a row is cached: fewer or more requests in x, plan or table."""
    stack = build(1)
    table, lens = torch.arange(4, dtype=torch.int32, device="cuda").view(4, 1), i32(1, 1, 1, 1)
    free, count = i32(9, 9, 9, 9), i32(0)
    before = [t.clone() for t in tensors(stack)]
    x = torch.randn((4, D_MODEL), device="cuda")
    by_hand = prox.PagePlan(lens, None, None, torch.arange(4, device="cuda") * PAGE, lens - 1, None)
    for plan in (by_hand, prox.plan_pages(lens, lens, table, free, count, PAGE, max_new=4)):
        for bad in ((x[:3], plan, table), (x[:3], plan, table[:3]), (x, plan, table[:3]), (x[0], plan, table),
                    (x, plan, table[:, 0]), (x, plan._replace(cu=None, slots=plan.slots[:3]), table)):
            for stream in (None, torch.cuda.Stream()):
                with pytest.raises(ValueError):
                    stack.attention[0].step(*bad, stream=stream)
                with pytest.raises(ValueError):
                    stack.decode(*bad, stream=stream)
    assert all(torch.equal(a, b) for a, b in zip(tensors(stack), before))


def test_per_request_in_a_captured_step():
    """A captured step replays on another plan: nothing of it is on the host."""
    stack = build(1)
    table = i32(3, 5, 7).view(3, 1)
    lens, delta, free, count = i32(2, 0, 9), i32(1, 0, 1), i32(0, 0, 0, 0), i32(1)
    x = torch.randn((3, D_MODEL), device="cuda", generator=gen_of(55))

    def step():
        plan = prox.plan_pages(lens, delta, table, free, count, PAGE, max_new=3)
        return stack.decode(x, plan, table)

    fill(stack, table, [2, 0, 9], 56)
    start = [t.clone() for t in tensors(stack)]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    for d in ((1, 0, 1), (0, 0, 1), (1, 0, -9)):
        for t, s in zip(tensors(stack), start):
            t.copy_(s)
        delta.copy_(i32(*d))
        graph.replay()
        torch.cuda.synchronize()
        got, after = y.clone(), [t.clone() for t in tensors(stack)]
        for t, s in zip(tensors(stack), start):
            t.copy_(s)
        want = step()
        assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(after, tensors(stack)))
