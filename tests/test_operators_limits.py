"""Limits of the operators' host code, without a GPU."""
import ctypes

import pytest

import block_scaled_grouped_gb300 as bsgg
from block_scaled_grouped_gb300 import build as bsgg_build

P = ctypes.c_void_p(4096)        # never dereferenced: refused first


@pytest.fixture(scope="module", autouse=True)
def lib():
    bsgg_build.build()
    return bsgg.lib()


@pytest.mark.parametrize("slots", [2 ** 30 + 1, 2 ** 31 - 1])
def test_sort_refuses_more_slots_than_rows_can_be(lib, slots):
    assert lib.bsgg_sort_tokens(slots, 4, 2 ** 30, P, None, P, P, P, None, None, P, None, None) == 2
