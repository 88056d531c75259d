"""Lengths that no cache holds (within a page of 2^31, far past the table, below
zero) in the cache's upkeep: nothing is read outside a sequence's table row."""
import ctypes
import os
import subprocess

import pytest
import torch

import attention_forward_13_gb300 as A
from tests._parity import no_device_error

gpu = pytest.mark.gpu

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_forward_13_gb300", "csrc")
TOP = 2 ** 31 - 1


@pytest.fixture(scope="module")
def pages_lib(tmp_path_factory):
    """The kernels' own page arithmetic, compiled for the host."""
    d = tmp_path_factory.mktemp("pages")
    src = d / "pages.cpp"
    src.write_text('#include "pages.h"\n'
                   'extern "C" int pages_of(int len, int lg) { return attn::pages_of(len, lg); }\n'
                   'extern "C" int held_pages(int len, int lg, int m) { return attn::held_pages(len, lg, m); }\n')
    out = d / "pages.so"
    subprocess.run(["g++", "-O2", "-shared", "-fPIC", "-ftrapv", "-I", CSRC, "-o", str(out), str(src)], check=True)
    return ctypes.CDLL(str(out))


@pytest.mark.parametrize("log2", [4, 5, 6, 7, 8])
def test_page_counts_of_any_length(pages_lib, log2):
    page = 1 << log2
    lens = [0, 1, page - 1, page, page + 1, 3 * page, TOP - 2 * page, TOP - page, TOP - page + 1, TOP - 1, TOP]
    for n in lens:
        want = -(-n // page)
        assert pages_lib.pages_of(n, log2) == want, n
        for most in (1, 7, want - 1, want, want + 1, TOP):
            if most > 0:
                assert pages_lib.held_pages(n, log2, most) == min(want, most)
    for n in (-1, -page, -TOP - 1):
        assert pages_lib.held_pages(n, log2, 7) == 0


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@gpu
@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("length", [TOP, TOP - 2, TOP - 15, 1 << 30, 3 * 256 + 1])
def test_upkeep_with_a_length_past_the_table(page, length):
    """Two columns; sequence 1 says it holds far more.  It counts as holding its whole row."""
    num, width = 8, 2
    pools = [torch.randint(0, 100, (num, page, 1, 8), dtype=torch.int16, device="cuda").view(torch.float16)
             for _ in range(2)]
    before = [p.clone() for p in pools]
    table, refs = i32([[0, 1], [2, 3], [4, 5]]), i32([1, 1, 1, 1, 1, 1, 0, 0])
    lens = [page + 3, length, 2 * page - 1]
    # More tokens for it: an error, and nothing changes.
    t, l, r, f = A.attn_cache_reserve(*pools, table, i32(lens), refs, i32([0, 5, 0]))
    assert f.item() == -num - 1 and l.tolist() == lens and torch.equal(r, refs) and torch.equal(t, table)
    assert A.attn_device_error() == 1 << 25
    # Taken over as it is, shared, dropped.
    t, l, r = A.attn_cache_reorder(table, i32(lens), refs, i32([1, 1]), page)
    assert t.tolist() == [[2, 3], [2, 3]] and l.tolist() == [length] * 2
    assert r.tolist() == [0, 0, 2, 2, 0, 0, 0, 0]
    # The last two rows are its tree, of which the first stays: lengths end at the table's.
    l, r = A.attn_cache_accept(*pools, table, i32(lens), refs, i32([[0]] * 3), i32([1] * 3), i32([2] * 3))
    assert l.tolist() == [page + 2, 2 * page - 1, 2 * page - 2]
    assert torch.equal(r, refs)
    t, r, m = A.attn_cache_compact(*pools, table, i32(lens), refs)
    assert torch.equal(t, table) and torch.equal(r, refs) and m.tolist() == [0, 1, 2, 3, 4, 5, -1, -1]
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(pools, before))
    no_device_error()
