"""Sizes at which the tree attention's 32-bit positions would end: refused before a launch."""
import ctypes

import pytest

import attention_forward_13_gb300 as A
from attention_forward_13_gb300 import _lib

P = 1 << 12  # (an address that is aligned, never read)


def tree(page, width, B=1, T=1, Hq=1, Hkv=1):
    return A.library().attn_fwd_paged_tree(P, P, P, P, P, P, None, None, P, None, B, T, Hq, Hkv, 64, 1, page, 9, width, P,
                                           1 << 40, ctypes.byref(_lib.attn_opts()), None)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_tables_of_almost_2_31_keys(page):
    """A tile of 128 keys that starts below the last key has to end below 2^31."""
    most = (2 ** 31 - 256) // page
    for width in (2 ** 31 // page - 1, most + 1):
        if width > most:
            assert tree(page, width) == 2, width
    assert tree(page, 2 ** 31 // page) == 2
