"""Window bounds as wide as an int: the same bits as the unbounded side, wherever a row's
diagonal lies (before the first key, behind the last), with and without first tokens."""
import numpy as np
import pytest
import torch

import attention_forward_13_gb300 as A
from attention_forward_13_gb300 import inputs
from tests import _masked as M
from tests._parity import check, cuda, f64, no_device_error

gpu = pytest.mark.gpu

TOP = 2 ** 31 - 1
WIDE = [(TOP, 0), (TOP, -1), (TOP, TOP), (-1, TOP), (TOP - 5, 3), (60, TOP), (5, TOP - 1)]
IDS = ["%d_%d" % w for w in WIDE]


def unbounded(window):
    return tuple(-1 if w > 1 << 29 else w for w in window)


@gpu
@pytest.mark.parametrize("window", WIDE, ids=IDS)
@pytest.mark.parametrize("Lq,Lk", [(300, 300), (700, 90), (90, 700)])
@pytest.mark.parametrize("keep", [0, 3, 150])
def test_dense(window, Lq, Lk, keep):
    for d, dt in ((64, "f16"), (128, "bf16")):
        inp = inputs.dense(1, 4, 2, Lq, Lk, d, dt, seed=Lq + d)
        for top in (False, True):
            o, lse = A.attn_fwd(cuda(inp.q), cuda(inp.k), cuda(inp.v), window=window, top_left=top, sink_tokens=keep)
            seen = M.band(Lq, Lk, *unbounded(window), sink_tokens=keep, top_left=top)
            ro, rl = M.attend(f64(inp.q[0]), np.repeat(f64(inp.k[0]), 2, 0), np.repeat(f64(inp.v[0]), 2, 0), seen,
                              1 / np.sqrt(d))
            torch.cuda.synchronize()
            check(o[0], lse[0], ro, rl, "dense %s top %s" % (window, top))
    no_device_error()


@gpu
@pytest.mark.parametrize("window", WIDE, ids=IDS)
@pytest.mark.parametrize("Lq", [1, 4, 70])  # decode, and the chunked prefill
@pytest.mark.parametrize("keep", [0, 3, 150])
def test_paged(window, Lq, keep):
    lens = [0, 1, 3, 69, 500, 1300]  # some shorter than the queries
    inp = inputs.paged(lens, Lq, 8, 2, 128, 64, 40, seed=Lq)
    args = [cuda(x) for x in (inp.q, inp.k_pool, inp.v_pool, inp.block_table, inp.seqlens_k)]
    o, lse = A.attn_fwd_paged(*args, window=window, sink_tokens=keep)
    torch.cuda.synchronize()
    for b, L in enumerate(lens):
        seen = M.band(Lq, L, *unbounded(window), sink_tokens=keep)
        k, v = (M.paged_rows(f64(p), inp.block_table[b].tolist(), L, 64).transpose(1, 0, 2)
                for p in (inp.k_pool, inp.v_pool))
        ro, rl = M.attend(f64(inp.q[b]).transpose(1, 0, 2), np.repeat(k, 4, 0), np.repeat(v, 4, 0), seen, 128 ** -0.5)
        check(o[b].transpose(0, 1), lse[b], ro, rl, "paged %s" % (window,))
    no_device_error()


@gpu
@pytest.mark.parametrize("keep", [0, 3, 150])
def test_tree(keep):
    inp = inputs.paged([0, 1, 40, 500, 1300], 24, 8, 2, 128, 64, 40, seed=9)
    args = [cuda(x) for x in (inp.q, inp.k_pool, inp.v_pool, inp.block_table, inp.seqlens_k)]
    mask, depth = A.attn_tree_mask(torch.arange(-1, 23, dtype=torch.int32, device="cuda").repeat(5, 1))
    want = A.attn_fwd_paged_tree(*args, mask)
    got = A.attn_fwd_paged_tree(*args, mask, tree_depth=depth, window=(TOP, -1), sink_tokens=keep)
    # (a window masks other tiles too; what is kept and its order are the same)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    no_device_error()


def test_pages_and_schedule_of_wide_windows():
    """Host arithmetic: the widest bounds count as the unbounded side."""
    W = A.attn_paged_window_pages
    assert W(4, 64, 100, window=(TOP, -1)) == 100 and W(4, 64, 100, window=(TOP, TOP), sink_tokens=TOP) == 100
    for Lq, Lk in ((4096, 4096), (4096, 1000)):
        for wide, plain in (((TOP, 0), (-1, 0)), ((300, TOP), (300, -1))):
            assert A.attn_dense_schedule(2, 8, Lq, Lk, 100, window=wide) == \
                A.attn_dense_schedule(2, 8, Lq, Lk, 100, window=plain)
