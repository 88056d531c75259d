"""NaN that a row sees comes out of it: rows with a NaN query, key or value among what
they see give NaN (as the formula does), the other rows what they gave before."""
import numpy as np
import pytest
import torch

import attention_forward_13_gb300 as A
from attention_forward_13_gb300 import inputs
from tests._parity import cuda, no_device_error

pytestmark = pytest.mark.gpu

# B, keys, T, Hq, Hkv, d, page, dtype, cap, sink: one stream pair, two query tiles, cut and whole units
CASES = [
    (1, 3000, 5, 8, 2, 128, 64, "bf16", 0.0, False),
    (2, 300, 16, 8, 2, 64, 16, "f16", 30.0, True),
    (1, 2000, 70, 16, 4, 128, 64, "bf16", 0.0, True),
    (48, 200, 3, 32, 8, 64, 32, "f16", 0.0, False),
    (40, 400, 40, 32, 8, 128, 64, "bf16", 20.0, False),
]


def nan_rows(o, lse):
    """(rows whose O is all NaN, rows with some NaN, rows with NaN LSE), as [B, T, Hq]."""
    return o.isnan().all(-1), o.isnan().any(-1), lse.isnan().transpose(1, 2)


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
@pytest.mark.parametrize("where", ["q", "k", "v"])
def test_tree(case, where):
    B, L, T, Hq, Hkv, d, page, dt, cap, sink = case
    g = Hq // Hkv
    npages = B * -(-L // page)
    inp = inputs.paged([L] * B, T, Hq, Hkv, d, page, npages, dtype=dt, seed=L + T, softcap=cap, with_sink=sink)
    parents = torch.full((B, T), -1, dtype=torch.int32)  # node i > 1 follows node 0; node 1 a root of its own
    parents[:, 2:] = 0
    mask, _ = A.attn_tree_mask(cuda(parents))
    q, kp, vp = cuda(inp.q), cuda(inp.k_pool), cuda(inp.v_pool)
    args = (cuda(inp.block_table), cuda(inp.seqlens_k), mask)
    kw = dict(softcap=cap, sink=cuda(inp.sink))
    want, wlse = A.attn_fwd_paged_tree(q, kp, vp, *args, **kw)
    b, hk = B - 1, Hkv - 1
    bad = torch.zeros(B, T, Hq, dtype=torch.bool, device="cuda")
    if where == "q":
        q[b, 2, 1, 3] = float("nan")
        bad[b, 2, 1] = True
    else:  # node 0's row: nodes 0 and 2 .. see it, node 1 does not
        pos = L - T
        row = int(inp.block_table[b, pos // page]), pos % page
        (kp if where == "k" else vp)[row[0], row[1], hk, 5] = float("nan")
        bad[b, 0, hk * g:] = True
        bad[b, 2:, hk * g:] = True
    o, lse = A.attn_fwd_paged_tree(q, kp, vp, *args, **kw)
    torch.cuda.synchronize()
    whole, some, l = nan_rows(o, lse)
    if where == "v":  # that column alone, and the weights are what they were
        # (in it a row that does not see the node but reads its tile gets 0 * NaN)
        assert o[..., 5].isnan()[bad].all() and torch.equal(lse, wlse)
        other = torch.arange(d, device="cuda") != 5
        assert torch.equal(o[..., other], want[..., other])
    else:
        assert torch.equal(whole, bad) and torch.equal(some, bad) and torch.equal(l, bad)
        assert torch.equal(o[~bad], want[~bad]) and torch.equal(lse.transpose(1, 2)[~bad], wlse.transpose(1, 2)[~bad])
    no_device_error()


@pytest.mark.parametrize("many", [False, True])
def test_window_decode(many):
    """The same of single tokens under a window with first tokens, on both its kernels."""
    B, Hkv = (60, 8) if many else (2, 2)
    inp = inputs.paged([400] * B, 1, 4 * Hkv, Hkv, 128, 64, 7 * B, dtype="bf16", seed=5)
    q = cuda(inp.q)
    args = (cuda(inp.k_pool), cuda(inp.v_pool), cuda(inp.block_table), cuda(inp.seqlens_k))
    kw = dict(causal=True, window=(100, -1), sink_tokens=4, num_splits=1)
    want, wlse = A.attn_fwd_paged(q, *args, **kw)
    assert ("chain" in A.attn_last_kernel_name()) == many
    q[1, 0, 6, 9] = float("nan")
    o, lse = A.attn_fwd_paged(q, *args, **kw)
    bad = torch.zeros(B, 1, 4 * Hkv, dtype=torch.bool, device="cuda")
    bad[1, 0, 6] = True
    whole, some, l = nan_rows(o, lse)
    assert torch.equal(whole, bad) and torch.equal(some, bad)
    assert torch.equal(o[~bad], want[~bad])
    if many:
        assert torch.equal(l, bad)
    no_device_error()
