"""Outputs that share memory with inputs are refused where a kernel writes one while others read the other: the host's
search (csrc/overlap.h) against every pair of rows, and the calls that must be refused.  (Nothing here launches anything:
what the search lets through is asked of the search alone.)"""
import ctypes
import os
import random
import subprocess

import pytest
import torch

import attention_forward_13_gb300 as A
from tests.test_serving_checks import P, S, linear

HERE = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include "overlap.h"
extern "C" int overlaps(int64_t a, int64_t b, const int64_t* x, const int64_t* y, int64_t width) {
  using attn::Extent;
  auto e = [&](int64_t at, const int64_t* v) {
    return Extent{reinterpret_cast<const void*>(at), {v[3], v[4], v[5]}, {v[0], v[1], v[2]}, width};
  };
  return attn::overlap(e(a, x), e(b, y));
}
"""


@pytest.fixture(scope="module")
def search(tmp_path_factory):
    d = tmp_path_factory.mktemp("overlap")
    src, lib = str(d / "o.cpp"), str(d / "o.so")
    open(src, "w").write(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", os.path.join(HERE, "attention_forward_13_gb300", "csrc"),
                    src, "-o", lib], check=True)
    fn = ctypes.CDLL(lib).overlaps
    fn.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64]
    row = ctypes.c_int64 * 6
    return lambda a, b, x, y, w: fn(a, b, row(*x), row(*y), w)


def elements(base, x, width):
    n, s = x[:3], x[3:]
    return {base // 2 + i * s[0] + j * s[1] + k * s[2] + e for i in range(n[0]) for j in range(n[1]) for k in range(n[2])
            for e in range(width)}


def layouts(rng, H):
    """Dense, heads next to each other, a slice of wider rows, packed."""
    B, L, d = rng.randint(1, 3), rng.randint(1, 6), 8
    wide = H + rng.randint(0, 4)
    return (B, H, L), rng.choice([(H * L * d, L * d, d), (L * wide * d, d, wide * d), (L * wide * d, 2 * d, 2 * wide * d),
                                  (8 * rng.randint(1, 60), 8 * rng.randint(1, 60), 8 * rng.randint(1, 60))]), d


def test_against_all_pairs(search):
    rng = random.Random(3)
    yes = 0
    for _ in range(4000):
        n, s, d = layouts(rng, rng.randint(1, 4))
        m, t, _ = layouts(rng, rng.randint(1, 4))
        if rng.random() < 0.5:
            t = s
        a, b = 1 << 20, (1 << 20) + 16 * rng.randint(-40, 40)
        want = not elements(a, n + s, d).isdisjoint(elements(b, m + t, d))
        assert search(a, b, n + s, m + t, d) == want, (n, s, m, t, b - a)
        yes += want
    assert 500 < yes < 3500


def test_parts_of_one_projection(search):
    """Slices of one buffer do not overlap however long it is, and neighbours of a head do from one element on."""
    B, L, H, d = 4, 1 << 20, 96, 128
    x = (B, 32, L, L * H * d, d, H * d)
    assert not search(1 << 40, (1 << 40) + 2 * 32 * d, x, x, d) and not search(1 << 40, (1 << 40) + 2 * 64 * d, x, x, d)
    assert search(1 << 40, (1 << 40) + 2 * 32 * d - 16, x, x, d) and search(1 << 40, (1 << 40) + 2 * 31 * d, x, x, d)
    far = (1 << 40) + 2 * B * L * H * d
    assert not search(1 << 40, far, x, x, d) and search(1 << 40, far - 2 * 65 * d, x, x, d)


OVER = dict(B=1, Hq=2, Hkv=2, L=8, s=S(4096, 64, 128))  # rows of 2 heads next to each other: 2048 bytes


@pytest.mark.parametrize("form", ["dense", "packed", "step"])
@pytest.mark.parametrize("x", ["q", "k", "v"])
def test_linear_output_over_an_input(form, x):
    a = dict(q=1 << 20, k=1 << 21, v=1 << 22, o=1 << 23, **OVER)
    for by in (0, 16, -16, 128):
        assert linear(form, **{**a, x: a["o"] + by}) == 1


def test_states_over_each_other():
    n = 2 * 64 * 64 * 4
    for by in (16, -16, n - 16, 16 - n):
        assert linear(q=1 << 20, k=1 << 21, v=1 << 22, o=1 << 23, si=1 << 24, so=(1 << 24) + by, **OVER) == 1


def rope(q, qo, k, ko, s=S(4096, 64, 128), so=None):
    from attention_forward_13_gb300 import _lib
    o = _lib.attn_rope_opts(P, 64, 0, 0, 0.0)
    so = so or s
    return A.library().attn_rope(q, qo, k, ko, P, 0, 1, 8, 2, 2, 64, 1, s, so, s, so, ctypes.byref(o), None)


def test_rope_outputs():
    a, b, c, d = (1 << n for n in range(20, 24))
    for by in (16, -16, 128):
        assert rope(a, a + by, b, c) == 1 and rope(a, c, b, b + by) == 1       # its own input, but not in place
        assert rope(a, b + by, b, c) == 1 and rope(a, d, b, a + by) == 1       # the other one
        assert rope(a, c, b, c + by) == 1                                      # the two outputs
    assert rope(a, a, b, d, so=S(4096, 512, 64)) == 1                          # in place, but other rows
    assert rope(a, a, b, a) == 1


def test_append_output():
    from attention_forward_13_gb300 import _lib
    o, s = _lib.attn_rope_opts(P, 64, 0, 0, 0.0), S(0, 64, 128)

    def call(q, qo, k, v, so=s):
        return A.library().attn_cache_append(q, qo, k, v, 1 << 26, 1 << 27, P, P, 8, 2, 2, 64, 1, 16, 9, s, so, s, s,
                                             ctypes.byref(o), None)
    a, b, c = (1 << n for n in range(20, 23))
    assert call(a, a + 16, b, c) == 1 and call(a, b, b, c) == 1 and call(a, c + 128, b, c) == 1
    assert call(a, a, b, c, S(0, 512, 64)) == 1


@pytest.mark.gpu
def test_parts_of_one_buffer_stay_allowed():
    """q, k, v and o side by side in one buffer, and a rotation in place there."""
    N, H, d = 300, 2, 64
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    buf = torch.randn(N, 4 * H, d, generator=gen, device="cuda").bfloat16()
    q, k, v, o = buf.split(H, 1)
    g = torch.tensor([-0.1, -0.5], device="cuda")
    f = A.attn_rope_freqs(d)
    want_q, want_k = A.attn_rope(q.contiguous(), k.contiguous(), f)
    A.attn_rope(q, k, f, q_out=q, k_out=k)
    assert torch.equal(q, want_q) and torch.equal(k, want_k)
    cu = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    want, _ = A.attn_linear_fwd_varlen(*(x.contiguous() for x in (q, k, v)), cu, 200, g)
    A.attn_linear_fwd_varlen(q, k, v, cu, 200, g, o=o)
    assert torch.equal(o, want)
    state = torch.zeros(N, H, d, d, device="cuda")
    want = A.attn_linear_step(*(x.contiguous() for x in (q, k, v)), g, state.clone())
    A.attn_linear_step(q, k, v, g, state, o=o)
    assert torch.equal(o, want)
