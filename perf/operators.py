"""The 4-bit operators of a decode step, case by case: what one call of each
reads, computes and returns, with a plain form in elementary torch operations
beside the library's kernels.

 linear4   y = x W for 1..16 tokens, W held as INT4 codes with one fp16 scale
           per 128 input rows and channel (the format of pack_proxy)
 attend    attention of the newest tokens of each request over a paged cache
           that holds K and V as INT4 codes with one fp16 scale per token and
           head
 append    new K / V rows quantised into that cache at their slots, and read
           back as the values the cache now stands for
 pages     block tables, slots and positions of the tokens that requests gain
           (or drop), pages taken from and returned to a free list

`own` chooses between the plain form (False) and the library's calls (True).
"""

from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
GROUP = 128


# --------------------------------------------------------------------------
# The cases
# --------------------------------------------------------------------------

def listed():
    return [
        # The tiny layer's gate projection for one token: a call that is all
        # latency.
        dict(name="linear4_tiny", op="linear4", K=512, N=1376, B=1, dtype="fp32"),
        # Query, key and value projections (32 + 2 x 8 heads of 128) of the
        # 8B-shaped model, one token in the library's own activation type.
        dict(name="linear4_qkv_8b", op="linear4", K=4096, N=6144, B=1, dtype="fp32"),
        # Down projection of the 70B-shaped layer for a small batch: long sums.
        dict(name="linear4_down_70b", op="linear4", K=28672, N=8192, B=5, dtype="bf16"),
        # An output head over a large vocabulary, a full batch.
        dict(name="linear4_head", op="linear4", K=5120, N=131072, B=16, dtype="fp16"),
        # One request a few tokens into its answer, the tiny model's heads.
        dict(name="attend_short", op="attend", B=1, Tq=1, Hkv=4, G=2, D=64, page=16, longest=37,
             spread="full", dtype="fp32", lens_seed=1),
        # A serving batch of the 8B-shaped model: ragged lengths, some requests
        # with nothing cached.
        dict(name="attend_batch_8b", op="attend", B=64, Tq=1, Hkv=8, G=4, D=128, page=64,
             longest=8191, spread="ragged", dtype="bf16", lens_seed=2),
        # One very long context of the 14B-shaped model in fp32 activations.
        dict(name="attend_long_14b", op="attend", B=1, Tq=1, Hkv=8, G=5, D=128, page=64,
             longest=131071, spread="full", dtype="fp32", lens_seed=3),
        # Four drafted tokens per request checked at once, 70B-shaped heads.
        dict(name="attend_draft_70b", op="attend", B=16, Tq=4, Hkv=8, G=8, D=128, page=16,
             longest=6001, spread="ragged", dtype="fp16", lens_seed=4),
        # The rows of one decode step of a batch: one token per request.
        dict(name="append_step", op="append", T=64, Hkv=8, D=128, page=64, pages=512,
             skipped=3, dtype="fp32"),
        # The rows of a prompt chunk, with the padding that a fixed-size chunk
        # carries.
        dict(name="append_prompt", op="append", T=16000, Hkv=8, D=128, page=64, pages=512,
             skipped=133, dtype="bf16"),
        # A decode step of 64 requests, a few of them finished.
        dict(name="pages_step", op="pages", B=64, page=64, cols=128, longest=8000, most=1,
             dropped=3, plan_seed=1),
        # Prompts admitted to a large batch: many tokens at once.
        dict(name="pages_admit", op="pages", B=1021, page=16, cols=640, longest=9000, most=200,
             dropped=90, plan_seed=2),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["linear4", "linear4", "attend", "attend", "append", "pages"])
    if op == "linear4":
        while True:
            K, N = GROUP * _log_int(rng, 1, 224), 2 * _log_int(rng, 8, 65536)
            if K * N <= 5120 * 131072:
                return dict(op=op, K=K, N=N, B=rng.randint(1, 16), dtype=rng.choice(list(DTYPES)))
    if op == "attend":
        while True:
            c = dict(op=op, B=_log_int(rng, 1, 256), Tq=rng.choice([1, 1, 1, 2, 3, 5]),
                     Hkv=rng.choice([1, 2, 4, 8, 10]), G=rng.choice([1, 2, 3, 4, 5, 8, 16]),
                     D=rng.choice([64, 128, 128, 256]), page=rng.choice([16, 32, 64, 128]),
                     longest=_log_int(rng, 1, 131071), spread=rng.choice(["full", "ragged"]),
                     dtype=rng.choice(list(DTYPES)), lens_seed=rng.randrange(1 << 30))
            if c["B"] * (c["longest"] + 128) * c["Hkv"] * c["D"] <= 131072 * 8 * 128 * 2 \
                    and c["Tq"] * c["G"] * c["longest"] * c["B"] * c["Hkv"] <= 1 << 26:
                return c
    if op == "append":
        while True:
            c = dict(op=op, T=_log_int(rng, 1, 16000), Hkv=rng.choice([1, 2, 4, 8, 10]),
                     D=rng.choice([64, 128, 256]), page=rng.choice([16, 32, 64, 128]),
                     dtype=rng.choice(list(DTYPES)))
            if c["T"] * c["Hkv"] * c["D"] <= 16000 * 8 * 128:
                c["pages"] = -(-c["T"] // c["page"]) * 2 + rng.randint(0, 9)
                c["skipped"] = rng.randint(0, c["T"] // 4)
                return c
    B = _log_int(rng, 1, 1021)
    page, longest, most = rng.choice([16, 32, 64, 128]), _log_int(rng, 1, 9000), _log_int(rng, 1, 200)
    return dict(op="pages", B=B, page=page, cols=-(-(longest + most) // page), longest=longest,
                most=most, dropped=rng.randint(0, B // 4), plan_seed=rng.randrange(1 << 30))


def _lens(c):
    r = random.Random(c["lens_seed"])
    if c["spread"] == "full":
        return [c["longest"]] * c["B"]
    return [0 if r.random() < 0.05 else r.randint(1, c["longest"]) for _ in range(c["B"])]


def _plan(c):
    """lens and deltas of a pages case: most requests gain tokens, `dropped`
    of them finish and return everything, a few lose their newest tokens."""
    r = random.Random(c["plan_seed"])
    lens = [r.randint(0, c["longest"]) for _ in range(c["B"])]
    delta = [r.randint(1, c["most"]) for _ in range(c["B"])]
    for i in r.sample(range(c["B"]), c["dropped"]):
        delta[i] = -lens[i]
    for i in range(0, c["B"], 17):
        if delta[i] > 0 and lens[i] > 8:
            delta[i] = -r.randint(0, 8)
    return lens, delta


def _ceil(a, b):
    return -(-a // b)


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    return {"linear4": _prepare_linear4, "attend": _prepare_attend, "append": _prepare_append,
            "pages": _prepare_pages}[case["op"]](dict(case), gen)


def _codes(gen, shape):
    """Packed codes of normally distributed values: q + 8 with q in [-7, 7],
    two per byte."""
    n = torch.empty(shape[:-1] + (shape[-1] // 2, 2), dtype=torch.float16, device="cuda")
    n.normal_(0.0, 2.5, generator=gen)
    n = n.round_().clamp_(-7, 7).add_(8).to(torch.uint8)
    return n[..., 0] | (n[..., 1] << 4)


def _scales(gen, shape, mid):
    s = torch.empty(shape, dtype=torch.float32, device="cuda")
    return (mid * s.normal_(0.0, 0.3, generator=gen).exp_()).to(torch.float16)


def _prepare_linear4(c, gen):
    K, N, B = c["K"], c["N"], c["B"]
    codes = _codes(gen, (K, N))
    scales = _scales(gen, (K // GROUP, N), 0.02 / 2.5)
    # activations as the decode step meets them: heavy tails, a few channels
    # with outliers
    x = torch.empty((B, K), dtype=torch.float32, device="cuda").normal_(0.0, 1.0, generator=gen)
    x = x * torch.empty_like(x).exponential_(1.0, generator=gen).sqrt_()
    x[:, torch.randint(0, K, (max(1, K // 200),), device="cuda", generator=gen)] *= 30.0
    s = dict(op="linear4", x=x.to(DTYPES[c["dtype"]]), codes=codes, scales=scales)
    if own:
        import activation_sparse_swiglu_b200 as prox
        s["layer"] = prox.Linear4(codes=codes, scales=scales)
    return s


def _new_cache(c, gen, pages, filled):
    shape = (pages, c["Hkv"], c["page"])
    if filled:
        k, v = _codes(gen, shape + (c["D"],)), _codes(gen, shape + (c["D"],))
        ks, vs = _scales(gen, shape, 0.4), _scales(gen, shape, 0.3)
    else:
        k, v = (torch.full(shape + (c["D"] // 2,), 0x88, dtype=torch.uint8, device="cuda")
                for _ in range(2))
        ks, vs = (torch.zeros(shape, dtype=torch.float16, device="cuda") for _ in range(2))
    s = dict(k=k, ks=ks, v=v, vs=vs)
    if own:
        import activation_sparse_swiglu_b200 as prox
        s["cache"] = prox.KVCache4(k, ks, v, vs)
    return s


def _prepare_attend(c, gen):
    lens = _lens(c)
    need = [_ceil(n, c["page"]) for n in lens]
    cols = max(1, max(need))
    pages = sum(need) + 3
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    # row b holds its own pages; the entries behind them are never used
    start = torch.tensor([0] + need, dtype=torch.int64).cumsum(0)[:-1]
    at = start[:, None] + torch.arange(cols)[None, :]
    used = torch.arange(cols)[None, :] < torch.tensor(need)[:, None]
    table = torch.where(used.cuda(), order[at.clamp(max=pages - 1).cuda()], -1).to(torch.int32)
    q = torch.empty((c["B"], c["Tq"], c["Hkv"] * c["G"], c["D"]), dtype=torch.float32,
                    device="cuda").normal_(0.0, 1.0, generator=gen).to(DTYPES[c["dtype"]])
    return dict(op="attend", q=q, table=table.contiguous(),
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                scale=1.0 / math.sqrt(c["D"]), **_new_cache(c, gen, pages, True))


def _prepare_append(c, gen):
    dt = DTYPES[c["dtype"]]
    # K and V as the projections leave them: slices of one row per token
    rows = torch.empty((c["T"], 3, c["Hkv"], c["D"]), dtype=torch.float32, device="cuda")
    rows = rows.normal_(0.0, 1.0, generator=gen).to(dt)
    slots = torch.randperm(c["pages"] * c["page"], device="cuda", generator=gen)[:c["T"]].clone()
    gone = torch.randperm(c["T"], device="cuda", generator=gen)[:c["skipped"]]
    slots[gone] = -1
    return dict(op="append", k_new=rows[:, 1], v_new=rows[:, 2], slots=slots,
                **_new_cache(c, gen, c["pages"], False))


def _prepare_pages(c, gen):
    lens, delta = _plan(c)
    need = [_ceil(n, c["page"]) for n in lens]
    wanted = sum(max(0, _ceil(n + d, c["page"]) - _ceil(n, c["page"])) for n, d in zip(lens, delta))
    pages = sum(need) + wanted + 5
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    start = torch.tensor([0] + need, dtype=torch.int64).cumsum(0)[:-1]
    at = start[:, None] + torch.arange(c["cols"])[None, :]
    used = torch.arange(c["cols"])[None, :] < torch.tensor(need)[:, None]
    table = torch.where(used.cuda(), order[at.clamp(max=pages - 1).cuda()], -1).to(torch.int32)
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free[:pages - sum(need)] = order[sum(need):]
    new = sum(max(0, d) for d in delta)
    return dict(op="pages", lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                delta=torch.tensor(delta, dtype=torch.int32, device="cuda"),
                table=table.contiguous(), free=free,
                count=torch.tensor([pages - sum(need)], dtype=torch.int32, device="cuda"),
                page=c["page"], room=new + 7)


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------

def run(state):
    return {"linear4": _run_linear4, "attend": _run_attend, "append": _run_append,
            "pages": _run_pages}[state["op"]](state)


def _unpack(codes):
    """Packed bytes [..., n / 2] as fp32 integers q [..., n]."""
    lo = (codes & 15).to(torch.float32)
    hi = (codes >> 4).to(torch.float32)
    return torch.stack((lo, hi), dim=-1).flatten(-2) - 8.0


def _run_linear4(s):
    if own:
        return s["layer"].forward(s["x"])
    K, N = s["codes"].shape[0], s["scales"].shape[1]
    w = _unpack(s["codes"]).view(K // GROUP, GROUP, N) * s["scales"].float()[:, None, :]
    return (s["x"].float() @ w.view(K, N)).to(s["x"].dtype)


def _run_attend(s):
    q = s["q"]
    if own:
        return s["cache"].attend(q, s["table"], s["lens"], scale=s["scale"])
    B, Tq, Hq, D = q.shape
    Hkv, page = s["ks"].shape[1], s["ks"].shape[2]
    table = s["table"].long().clamp(min=0)
    rows = table.shape[1] * page

    def values(codes, scales):  # [B, Hkv, rows, D]
        x = _unpack(codes[table]) * scales[table].float()[..., None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, rows, D)

    q5 = q.float().view(B, Tq, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    sc = (q5 @ values(s["k"], s["ks"]).transpose(-1, -2)) * s["scale"]
    sc = sc.view(B, Hkv, Tq, Hq // Hkv, rows)
    last = s["lens"].long()[:, None] - Tq + torch.arange(Tq, device=q.device)[None, :]
    seen = torch.arange(rows, device=q.device)[None, None, :] <= last[:, :, None]
    seen = seen[:, None, :, None, :]
    sc = sc.masked_fill(~seen, -torch.inf)
    top = sc.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (sc - top).exp()
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, 0.0)
    o = p.view(B, Hkv, -1, rows) @ values(s["v"], s["vs"])
    o = o.view(B, Hkv, Tq, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Tq, Hq, D)
    return o.to(q.dtype)


def _quantise(x):
    """Scales fp16 [T, H] and integers q [T, H, D] of rows x, symmetric: the
    scale is the largest magnitude over 7, rounded to fp16, the code x / scale
    rounded half to even.  In 64 bits, so that no rounding before the last one
    moves a value across a border."""
    x = x.double()
    s = (x.abs().amax(-1) / 7.0).to(torch.float16)
    q = (x / s.double()[..., None]).round().clamp(-7, 7)
    return s, torch.where(s[..., None] > 0, q, 0.0)


def _run_append(s):
    slots, dt = s["slots"], s["k_new"].dtype
    if own:
        s["cache"].append(s["k_new"], s["v_new"], slots)
        return s["cache"].read(slots, dtype=dt)
    page = s["ks"].shape[2]
    held = slots >= 0
    at = slots.clamp(min=0)
    # a skipped row writes what its place already holds
    p, r = at // page, at % page
    out = []
    for codes, scales, rows in ((s["k"], s["ks"], s["k_new"]), (s["v"], s["vs"], s["v_new"])):
        sc, q = _quantise(rows)
        n = (q + 8).to(torch.uint8)
        packed = n[..., 0::2] | (n[..., 1::2] << 4)
        live = held.nonzero().squeeze(1)
        codes[p[live], :, r[live]] = packed[live]
        scales[p[live], :, r[live]] = sc[live]
        back = _unpack(codes[p, :, r]) * scales[p, :, r].float()[..., None]
        out.append(torch.where(held[:, None, None], back, 0.0).to(dt))
    return tuple(out)


def _run_pages(s):
    if own:
        import activation_sparse_swiglu_b200 as prox
        r = prox.plan_pages(s["lens"], s["delta"], s["table"], s["free"], s["count"], s["page"],
                            max_new=s["room"])
        return {"lens": r.lens, "count": r.count, "cu": r.cu, "slots": r.slots,
                "positions": r.positions, "table": s["table"], "free": s["free"],
                "status": r.status}
    lens, delta, table, free, page = s["lens"], s["delta"], s["table"], s["free"], s["page"]
    dev, cols, room = lens.device, table.shape[1], s["room"]
    to = lens + delta
    have, need = (lens + page - 1) // page, (to + page - 1) // page
    gain, drop = (need - have).clamp(min=0), (have - need).clamp(min=0)
    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    at_new = torch.cat((zero, delta.clamp(min=0).cumsum(0)))
    at_gain, at_drop = gain.cumsum(0) - gain, drop.cumsum(0) - drop
    c0 = s["count"].long()
    c1 = c0 + drop.sum()
    c2 = c1 - gain.sum()
    bad = ((lens < 0) | (to < 0) | (need > cols)).any() | (c2 < 0) | (c1 > free.numel()) \
        | (at_new[-1] > room)
    # dropped pages onto the free list, in request order
    col = torch.arange(cols, device=dev)[None, :]
    out = (col >= need[:, None]) & (col < have[:, None]) & ~bad
    i, j = out.nonzero(as_tuple=True)
    free[c0 + at_drop[i] + j - need[i]] = table[i, j]
    # pages for the gained columns, from the list's end
    into = (col >= have[:, None]) & (col < need[:, None]) & ~bad
    i, j = into.nonzero(as_tuple=True)
    table[i, j] = free[c1 - 1 - (at_gain[i] + j - have[i])]
    n = torch.arange(room, device=dev)
    req = (torch.searchsorted(at_new, n, right=True) - 1).clamp(max=lens.numel() - 1)
    live = (n < at_new[-1]) & ~bad
    pos = torch.where(live, lens[req] + n - at_new[req], -1)
    where = pos.clamp(min=0)
    slots = table[req, (where // page).clamp(max=cols - 1)].long() * page + where % page
    return {"lens": torch.where(bad, lens, to), "count": torch.where(bad, c0, c2).to(torch.int32),
            "cu": torch.where(bad, 0, at_new).to(torch.int32), "slots": torch.where(live, slots, -1),
            "positions": pos.to(torch.int32), "table": table, "free": free,
            "status": bad.to(torch.int32).reshape(1)}


# --------------------------------------------------------------------------
# What a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    c = case
    size = {"fp32": 4, "bf16": 2, "fp16": 2}.get(c.get("dtype"), 0)
    if c["op"] == "linear4":
        K, N, B = c["K"], c["N"], c["B"]
        return {"bytes": K * N // 2 + K // GROUP * N * 2 + B * (K + N) * size, "flops": 2 * B * K * N}
    if c["op"] == "attend":
        lens, Hq = _lens(c), c["Hkv"] * c["G"]
        tokens = sum(lens)
        pages = sum(_ceil(n, c["page"]) for n in lens)
        seen = sum(max(0, n - c["Tq"] + i + 1) for n in lens for i in range(c["Tq"]))
        return {"bytes": tokens * c["Hkv"] * (c["D"] + 4) + 2 * c["B"] * c["Tq"] * Hq * c["D"] * size
                + 4 * (pages + c["B"]), "flops": 4 * seen * Hq * c["D"]}
    if c["op"] == "append":
        rows = (c["T"] - c["skipped"]) * c["Hkv"] * 2
        # values in, codes and scales written and read, values out
        return {"bytes": rows * (c["D"] * size + 2 * (c["D"] // 2 + 2))
                + c["T"] * c["Hkv"] * 2 * c["D"] * size + 8 * c["T"], "flops": 4 * rows * c["D"]}
    lens, delta = _plan(c)
    new = sum(max(0, d) for d in delta)
    pages = sum(abs(_ceil(n + d, c["page"]) - _ceil(n, c["page"])) for n, d in zip(lens, delta))
    return {"bytes": 16 * c["B"] + 12 * new + 8 * pages + 16, "flops": 10 * c["B"] + 5 * new}


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------

def _values64(codes, scales):
    """[rows, D/2] bytes and [rows] scales as float64 [rows, D]."""
    v = torch.empty((codes.shape[0], codes.shape[1] * 2), dtype=torch.float64, device=codes.device)
    v[:, 0::2] = (codes % 16).double() - 8
    v[:, 1::2] = torch.div(codes, 16, rounding_mode="floor").double() - 8
    return v * scales.double()[:, None]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear4":
        x, (K, half) = s["x"].double(), s["codes"].shape
        out = torch.zeros((x.shape[0], 2 * half), dtype=torch.float64, device=x.device)
        for g in range(K // GROUP):
            blk = s["codes"][g * GROUP:(g + 1) * GROUP]
            xs = x[:, g * GROUP:(g + 1) * GROUP]
            sc = s["scales"][g].double()
            out[:, 0::2] += (xs @ ((blk % 16).double() - 8)) * sc[0::2]
            out[:, 1::2] += (xs @ (torch.div(blk, 16, rounding_mode="floor").double() - 8)) * sc[1::2]
        return out
    if case["op"] == "attend":
        q = s["q"].double()
        B, Tq, Hq, D = q.shape
        G, page = case["G"], case["page"]
        out = torch.zeros((B, Tq, Hq, D), dtype=torch.float64, device=q.device)
        for b, n in enumerate(_lens(case)):
            ids = s["table"][b, :_ceil(n, page)].long()
            for h in range(case["Hkv"] if n else 0):
                k = _values64(s["k"][ids, h].flatten(0, 1)[:n], s["ks"][ids, h].flatten()[:n])
                v = _values64(s["v"][ids, h].flatten(0, 1)[:n], s["vs"][ids, h].flatten()[:n])
                for i in range(Tq):
                    m = n - Tq + i + 1
                    if m > 0:
                        z = q[b, i, h * G:(h + 1) * G] @ k[:m].T * s["scale"]
                        out[b, i, h * G:(h + 1) * G] = torch.softmax(z, -1) @ v[:m]
        return out
    if case["op"] == "append":
        back = []
        for rows in (s["k_new"], s["v_new"]):
            x = rows.double()
            sc = (x.abs().amax(-1, keepdim=True) / 7).to(torch.float16).double()
            y = torch.where(sc > 0, torch.round(x / sc).clamp(-7, 7) * sc, 0.0)
            y[s["slots"] < 0] = 0
            back.append(y)
        return tuple(back)
    return None
