"""Sizes at which the 4-bit operators' 32-bit counters end: refused on the host,
before any device work."""

import ctypes

import pytest

from activation_sparse_swiglu_b200 import _lib
from tests.test_decode4_cpu import plan_args, refused


@pytest.mark.parametrize("max_new", [(1 << 30) + 1, (1 << 31) - (1 << 16), (1 << 31) - 1])
def test_plan_pages_more_new_tokens_than_32_bits_count(max_new):
    """A CTA steps through token numbers by up to 2^16: past 2^31 they turned
    negative, and slots were written there."""
    refused(_lib.lib.prox_plan_pages(*plan_args(max_new=max_new)), "max_new")
