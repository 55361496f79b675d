"""Sizes at which the 4-bit operators' 32-bit counters end: refused on the host,
before any device work."""

import ctypes

import pytest

from activation_sparse_swiglu_b200 import _lib
from tests.test_decode4_cpu import OK, plan_args, refused

ECUDA = 3


@pytest.mark.parametrize("max_new", [(1 << 30) + 1, (1 << 31) - (1 << 16), (1 << 31) - 1])
def test_plan_pages_more_new_tokens_than_32_bits_count(max_new):
    """A CTA steps through token numbers by up to 2^16: past 2^31 they turned
    negative, and slots were written there."""
    refused(_lib.lib.prox_plan_pages(*plan_args(max_new=max_new)), "max_new")


class Cache(ctypes.Structure):
    """struct prox_kv4 of csrc/decode4.h, of a device that does not exist: a call
    whose arguments pass ends at the check of the device."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "ks", "v", "vs")]
                + [(n, ctypes.c_int) for n in ("pages", "heads", "page", "D", "device", "num_sms")]
                + [(n, ctypes.c_void_p) for n in ("err", "part", "warp_part", "arrived", "base")]
                + [("bytes", ctypes.c_size_t)])


def attend(heads=8, page=64, dim=128, q_heads=8, B=1, Tq=1, q=1 << 40, out=1 << 41, lse=None, table=1 << 42, cols=4,
           lens=1 << 43, dtype=0, strides=None):
    cache = Cache(pages=4, heads=heads, page=page, D=dim, device=-1, num_sms=148)
    st = strides or (Tq * q_heads * dim, q_heads * dim, dim)
    return _lib.lib.prox_kv4_attend(ctypes.byref(cache), q, *st, q_heads, B, Tq, table, cols, cols, lens, 1.0, out, lse,
                                    dtype, None)


def passes(status):
    """The arguments were taken: the call ended at the device."""
    assert status != OK
    assert status == ECUDA or "lives on device -1" in _lib.last_error(), _lib.last_error()


@pytest.mark.parametrize("B, page, cols", [(8192, 256, 1 << 15), (8192, 16, 1 << 19), (4097, 64, 1 << 18)])
def test_attend_more_rows_than_32_bits_count(B, page, cols):
    """Units of 32 rows of all requests are numbered in 32 bits: past 2^31 (tables
    whose requests share pages, or lengths out of range, which are cut to the
    table) the kernel took heads and rows that are not there."""
    refused(attend(heads=1, q_heads=1, page=page, B=B, cols=cols), "B * cols")
    passes(attend(heads=1, q_heads=1, page=page, B=B // 2 - 1, cols=cols))


Q, ROW = 1 << 40, 8 * 128  # the queries' address; values of a request's queries


@pytest.mark.parametrize("dtype, size", [(0, 4), (1, 2), (2, 2)])
def test_attend_results_over_its_inputs(dtype, size):
    """Requests are read and written in an order of the device's own: results in
    another place of the queries' memory would reach queries not yet read."""
    def call(**kw):
        return attend(B=3, q=Q, dtype=dtype, **kw)
    one = ROW * size
    for out in (Q + one, Q - one, Q + 16, Q + 3 * one - 16, Q - 3 * one + 16):
        refused(call(out=out), "overlap q")
    for out in (Q, Q + 3 * one, Q - 3 * one):  # in place, right behind, right before
        passes(call(out=out))
    # rows of a wider buffer: in place no more; the queries' gaps are free for lse
    wide = (2 * ROW, ROW, 128)
    refused(call(out=Q, strides=wide), "overlap q")
    passes(call(lse=Q + one, strides=wide))
    refused(call(lse=Q + one - 4, strides=wide), "overlap q")
    refused(call(lse=Q + 2 * one - 92, strides=wide), "overlap q")
    passes(call(lse=Q + 2 * one - 96, strides=wide))  # 3 x 8 values up to the next request
    # heads in front of requests (a transposed buffer), and a stride below 0
    refused(call(out=Q + 23 * 128 * size, strides=(128, 128, 3 * 128)), "overlap q")
    passes(call(out=Q + 24 * 128 * size, strides=(128, 128, 3 * 128)))
    refused(call(out=Q - 2 * one, strides=(-ROW, ROW, 128)), "overlap q")
    passes(call(out=Q + one, strides=(-ROW, ROW, 128)))


def test_attend_results_over_each_other_and_the_plan():
    out, n = 1 << 41, 3 * ROW * 4
    for kw in (dict(lse=out + n - 4), dict(lse=out - 92), dict(lens=out + n - 12), dict(table=out - 44),
               dict(lse=(1 << 43) - 92), dict(lse=(1 << 42) + 44)):
        refused(attend(B=3, out=out, **kw), "each other")
    for kw in (dict(lse=out + n), dict(lse=out - 96), dict(lens=out + n), dict(table=out - 48),
               dict(lse=(1 << 43) - 96), dict(lse=(1 << 42) + 48)):
        passes(attend(B=3, out=out, **kw))


@pytest.mark.gpu
def test_attend_in_place_and_shifted_views():
    import torch
    import activation_sparse_swiglu_b200 as prox
    from tests.test_gpu_decode4 import attend_case
    for dtype in (torch.float32, torch.bfloat16):
        # contexts inside a warp, over warps and over CTAs; two row blocks a head
        cache, q, table, lens = attend_case(prox, [5, 40000, 0, 300, 64, 7000], 3, 2, 7, 128, 32, dtype, seed=40)
        want = cache.attend(q, table, lens)
        buf = torch.zeros((8, *q.shape[1:]), dtype=dtype, device="cuda")
        for at in (0, 2):
            with pytest.raises(prox.ProxError, match="overlap q"):
                cache.attend(buf[1:7].copy_(q), table, lens, out=buf[at:at + 6])
        assert torch.equal(cache.attend(buf[1:7], table, lens, out=buf[1:7]), want)
        assert torch.equal(buf[1:7], want)
