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
