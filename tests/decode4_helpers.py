"""Plain 64-bit forms of the 4-bit operators, and what their results may be
off by, for the tests of the library's kernels.

A rounding to a type of precision eps is off by at most eps / 2 of the value;
a sum of n fp32 terms by n 2^-23 of the terms' magnitudes (2^-24 a rounding,
twice that where a tensor core truncates).
"""

from __future__ import annotations

import torch

HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TYPES = [torch.float32, torch.float16, torch.bfloat16]


def unpack(codes):
    """uint8 [..., n / 2] -> int64 q [..., n]."""
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long() - 8


def pack(q):
    n = (q + 8).to(torch.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4)


def random_codes(gen, shape, device):
    """All sixteen codes, -8 among them."""
    return torch.randint(0, 256, tuple(shape[:-1]) + (shape[-1] // 2,), dtype=torch.uint8,
                         device=device, generator=gen)


def linear4(x, codes, scales):
    """y = x W in 64 bits, and the bound on a result's error."""
    K, N = codes.shape[0], scales.shape[1]
    q, s = unpack(codes).double().view(K // 128, 128, N), scales.double()[:, None, :]
    w = (q * s).view(K, N)
    xd = x.double()
    y = xd @ w
    # For 16-bit inputs the sums run over codes q + 8 and start from -8 sum x:
    # terms of up to (|q| + 16) |x| S.  The groups' sums are added one after the
    # other, after at most 8 tensor core steps and 3 multiplications; warps and
    # CTAs join 16 + 8 parts; the start value is a sum of 128 values over 7 levels.
    wide = x.dtype == torch.float32
    size = (q.abs() + (0 if wide else 16)) * s.abs()
    mag = xd.abs() @ size.view(K, N)
    n = K // 128 + 8 + 3 + 24 + 7
    tol = n * 2.0 ** -23 * mag + HALF_STEP[x.dtype] * y.abs()
    # fp32 inputs carry 22 bits; what lies below 2^-25 of its group's largest
    # magnitude has an absolute step of 2^-38 of it (2^-39 off, hi and lo)
    if wide:
        tol = tol + 2.0 ** -22 * mag
    top = xd.abs().view(-1, K // 128, 128).amax(-1)
    tol = tol + 2.0 ** -38 * (top @ size.sum(1))
    # the tensor core aligns subnormal codes at 2^-14: each of a group's 8 steps
    # is off by up to 2^-16 of a code step of the largest x
    if not wide:
        tol = tol + 8 * 2.0 ** -16 * (top @ s.squeeze(1).abs())
    if x.dtype == torch.float16:
        tol = tol + 2.0 ** -24  # below fp16's normal range a step is 2^-24
    return y, tol


def quantise(x):
    """Scales fp16 [...] and integers [..., D] of rows x, by the documented rule."""
    # the fp32 quotient by way of 64 bits (torch divides fp32 tensors by a
    # number as a product with its reciprocal, which is not the quotient): a
    # binary fraction over 7 has period 3, so 53 bits never sit on a border of 24
    s = (x.double().abs().amax(-1) / 7.0).float().to(torch.float16)
    q = (x.double() / s.double()[..., None]).round().clamp(-7, 7)
    q = torch.where(s[..., None] > 0, q, torch.zeros_like(q))
    return s, q.nan_to_num(0.0).long()


def attend(q, k_codes, k_scales, v_codes, v_scales, table, lens, scale):
    """(out, lse, bound on out's error, bound on lse's), in 64 bits, one request
    and kv head after the other."""
    B, Tq, Hq, D = q.shape
    Hkv, page = k_scales.shape[1], k_scales.shape[2]
    G = Hq // Hkv
    out = torch.zeros((B, Tq, Hq, D), dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    lse = torch.full((B, Tq, Hq), -torch.inf, dtype=torch.float64, device=q.device)
    lse_tol = torch.zeros_like(lse)
    wide = q.dtype == torch.float32
    for b in range(B):
        n = int(lens[b])
        ids = table[b, :-(-n // page)].long()
        for h in range(Hkv if n > 0 else 0):
            ks, vs = k_scales[ids, h].flatten()[:n].double(), v_scales[ids, h].flatten()[:n].double()
            kq = unpack(k_codes[ids, h]).flatten(0, 1)[:n].double()
            vq = unpack(v_codes[ids, h]).flatten(0, 1)[:n].double()
            k, v = kq * ks[:, None], vq * vs[:, None]
            # for 16-bit queries the sums run over codes q + 8 and start from
            # -8 times the other factor's sum: terms of up to |q| + 16
            more = 0 if wide else 16
            k_mag, v_mag = (kq.abs() + more) * ks[:, None], (vq.abs() + more) * vs[:, None]
            for i in range(Tq):
                m = n - Tq + i + 1
                if m <= 0:
                    continue
                qd = q[b, i, h * G:(h + 1) * G].double()
                z = qd @ k[:m].T * scale
                p = torch.softmax(z, -1)
                o = p @ v[:m]
                out[b, i, h * G:(h + 1) * G] = o
                lse[b, i, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
                # a score: at most D / 16 tensor core steps, 2 multiplications,
                # the difference to the maximum; fp32 queries carry 22 bits.  For
                # 16-bit queries a step is off by up to 2^-14 of a code step of
                # the largest factor (subnormal codes are aligned at 2^-14)
                t = (qd.abs() @ k_mag[:m].T * abs(scale)).amax(-1, keepdim=True)
                e_t = (D / 16 + 6) * 2.0 ** -23 * t
                if not wide:
                    e_t = e_t + (D / 16) * 2.0 ** -14 * abs(scale) * qd.abs().amax(-1, keepdim=True) * ks[:m].abs().max()
                # a probability's weight is rounded to 11 bits (fp32: 22), ex2
                # is good to 2^-22; the sums run over steps of at most 64 rows
                # (m / 32 bounds their number), each of at most 5 tensor core
                # steps, and are joined at most 12 + 148 times
                e_w = (2.0 ** -21 if wide else 2.0 ** -11) + 2.0 ** -22
                e_s = (m / 32 + 170) * 2.0 ** -23
                # weights below 2^-28 of the largest lose bits: 2^-39 of it each
                floor = m * 16 * vs[:m].abs().max() * 2.0 ** -38
                tol[b, i, h * G:(h + 1) * G] = ((2 * e_t + e_w + e_s) * (p @ v[:m].abs()) + 6 * 2.0 ** -23 * (p @ v_mag[:m])
                                                + floor + HALF_STEP[q.dtype] * o.abs())
                if not wide:  # 5 tensor core steps per step of rows
                    tol[b, i, h * G:(h + 1) * G] += 5 * 2.0 ** -14 * (p @ vs[:m].abs())[:, None]
                if q.dtype == torch.float16:
                    tol[b, i, h * G:(h + 1) * G] += 2.0 ** -24
                lse_tol[b, i, h * G:(h + 1) * G] = (e_t.squeeze(-1) + (m / 32 + 170) * 2.0 ** -23
                                                    + 2.0 ** -22 * (1 + lse[b, i, h * G:(h + 1) * G].abs()))
    return out, lse, tol, lse_tol


def plan(lens, delta, table, free, count, page, max_new):
    """plan_pages in plain Python on lists: (ok, lens, count, cu, slots,
    positions, table, free)."""
    lens, delta, table, free = list(lens), list(delta), [list(r) for r in table], list(free)
    cols = len(table[0]) if table else 0
    to = [a + d for a, d in zip(lens, delta)]
    have, need = [-(-a // page) for a in lens], [-(-a // page) for a in to]
    taken = sum(max(0, n - h) for n, h in zip(need, have))
    back = sum(max(0, h - n) for n, h in zip(need, have))
    new = sum(max(0, d) for d in delta)
    ok = (min(lens) >= 0 and min(to) >= 0 and max(need) <= cols and max(have) <= cols
          and 0 <= count and count + back <= len(free) and taken <= count + back and new <= max_new)
    if not ok:
        return False, lens, count, [0] * (len(lens) + 1), [-1] * max_new, [-1] * max_new, table, free
    at = count
    for i in range(len(lens)):
        for j in range(need[i], have[i]):
            free[at] = table[i][j]
            at += 1
    for i in range(len(lens)):
        for j in range(have[i], need[i]):
            at -= 1
            table[i][j] = free[at]
    slots, pos, cu = [], [], [0]
    for i in range(len(lens)):
        for p in range(lens[i], to[i]):
            slots.append(table[i][p // page] * page + p % page)
            pos.append(p)
        cu.append(len(slots))
    pad = [-1] * (max_new - len(slots))
    return True, to, at, cu, slots + pad, pos + pad, table, free
