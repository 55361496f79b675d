"""The 4-bit operators' argument checks, on the CPU: the library refuses bad
calls on the host before any device work, and the binding refuses what the C
ABI cannot see."""

import ctypes

import pytest
import torch

import activation_sparse_swiglu_b200 as prox
from activation_sparse_swiglu_b200 import _lib

EINVAL, OK = 1, 0
P16 = ctypes.c_void_p(1 << 20)  # never dereferenced


def refused(status, word):
    assert status == EINVAL
    assert word in _lib.last_error(), _lib.last_error()


@pytest.mark.parametrize("d_in, d_out, word", [
    (0, 64, "d_in"), (100, 64, "d_in"), (-128, 64, "d_in"), (65664, 64, "d_in"),
    (128, 0, "d_out"), (128, 63, "d_out"), (128, -2, "d_out"), (128, (1 << 20) + 2, "d_out")])
def test_linear4_shapes(d_in, d_out, word):
    h = ctypes.c_void_p(0)
    refused(_lib.lib.prox_linear4_create(P16, P16, d_in, d_out, None, ctypes.byref(h)), word)
    refused(_lib.lib.prox_linear4_create_bf16(P16, d_in, d_out, None, ctypes.byref(h)), word)
    assert not h.value


def test_linear4_pointers_and_handles():
    h = ctypes.c_void_p(0)
    lib = _lib.lib
    refused(lib.prox_linear4_create(None, P16, 128, 64, None, ctypes.byref(h)), "NULL")
    refused(lib.prox_linear4_create(P16, ctypes.c_void_p(17), 128, 64, None, ctypes.byref(h)), "aligned")
    refused(lib.prox_linear4_create_bf16(ctypes.c_void_p(18), 128, 64, None, ctypes.byref(h)), "aligned")
    refused(lib.prox_linear4_create(P16, P16, 128, 64, None, None), "out_host")
    refused(lib.prox_linear4_forward(None, P16, 128, P16, 64, 1, 0, None), "NULL")
    assert lib.prox_linear4_destroy(None) == OK


@pytest.mark.parametrize("pages, heads, page, dim, word", [
    (0, 8, 64, 128, "num_pages"), (4, 0, 64, 128, "n_heads"), (4, 8, 8, 128, "page_size"),
    (4, 8, 48, 128, "page_size"), (4, 8, 512, 128, "page_size"), (4, 8, 64, 96, "head_dim"),
    (4, 8, 64, 512, "head_dim")])
def test_kv4_shapes(pages, heads, page, dim, word):
    h = ctypes.c_void_p(0)
    refused(_lib.lib.prox_kv4_create(P16, P16, P16, P16, pages, heads, page, dim, ctypes.byref(h)), word)


def test_kv4_pointers_and_handles():
    h = ctypes.c_void_p(0)
    lib = _lib.lib
    odd = ctypes.c_void_p((1 << 20) + 8)
    refused(lib.prox_kv4_create(odd, P16, P16, P16, 4, 8, 64, 128, ctypes.byref(h)), "16-byte")
    refused(lib.prox_kv4_create(P16, odd, P16, P16, 4, 8, 64, 128, ctypes.byref(h)), "32-byte")
    refused(lib.prox_kv4_create(P16, P16, P16, None, 4, 8, 64, 128, ctypes.byref(h)), "32-byte")
    refused(lib.prox_kv4_create(P16, P16, P16, P16, 4, 8, 64, 128, None), "out_host")
    refused(lib.prox_kv4_append(None, P16, P16, 1, 1, 1, 1, P16, 1, 0, None), "NULL")
    refused(lib.prox_kv4_read(None, P16, 1, P16, P16, 0, None), "NULL")
    refused(lib.prox_kv4_attend(None, P16, 1, 1, 1, 8, 1, 1, P16, 4, 4, P16, 1.0, P16, None, 0, None), "NULL")
    refused(lib.prox_kv4_error(None, None, None), "NULL")
    assert lib.prox_kv4_destroy(None) == OK


def plan_args(**kw):
    a = dict(lens=P16, delta=P16, B=4, page=64, table=P16, stride=8, cols=8, free=P16, cap=9, count=P16,
             lens_out=ctypes.c_void_p(2 << 20), count_out=P16, cu=P16, slots=P16, pos=P16, max_new=4, status=P16)
    a.update(kw)
    return list(a.values()) + [None]


@pytest.mark.parametrize("kw, word", [
    (dict(B=0), "B=0"), (dict(B=8193), "B=8193"), (dict(page=0), "page_size"), (dict(cols=-1), "cols"),
    (dict(stride=7), "table_stride"), (dict(B=8000, cols=1 << 20, stride=1 << 20), "2^31"),
    (dict(cap=-1), "free_cap"), (dict(max_new=-1), "max_new"), (dict(lens=None), "NULL"),
    (dict(status=ctypes.c_void_p(2)), "aligned"), (dict(table=None), "table"), (dict(free=None), "free_pages"),
    (dict(slots=ctypes.c_void_p(4)), "slots"), (dict(lens_out=P16), "alias")])
def test_plan_pages_arguments(kw, word):
    refused(_lib.lib.prox_plan_pages(*plan_args(**kw)), word)


def test_binding_refuses_host_tensors_and_wrong_types():
    with pytest.raises(ValueError, match="either"):
        prox.Linear4()
    with pytest.raises(ValueError, match="either"):
        prox.Linear4(codes=torch.zeros(128, 32, dtype=torch.uint8))
    with pytest.raises(TypeError, match="bfloat16"):
        prox.Linear4(torch.zeros(128, 64, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="codes"):
        prox.Linear4(codes=torch.zeros(128, 32, dtype=torch.uint8), scales=torch.zeros(1, 64))
    z = torch.zeros(2, 4, 64, 64, dtype=torch.uint8)
    s = torch.zeros(2, 4, 64, dtype=torch.float16)
    with pytest.raises(TypeError, match="k_codes"):
        prox.KVCache4(z, s, z, s)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError, match="lens"):
        prox.plan_pages(i, i, torch.zeros(4, 8, dtype=torch.int32), i, i[:1], 64, max_new=4)
    for lens in (i, [0]):  # refused as without a stream
        with pytest.raises(TypeError, match="lens"):
            prox.plan_pages(lens, i, torch.zeros(4, 8, dtype=torch.int32), i, i[:1], 64, max_new=4, stream=1)
