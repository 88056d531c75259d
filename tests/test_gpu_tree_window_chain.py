"""A window in the tree attention bounds the keys before the nodes; among the nodes a row
sees what its mask says.  So a chain of drafted tokens equals the same tokens as a
causal chunk under the window (attn_fwd_paged) as long as no path is longer than
the window, and beyond that once the bits of the ancestors that lie further above
than the window are cleared."""
import pytest
import torch

import attention_forward_13_gb300 as A
from attention_forward_13_gb300 import inputs
from tests import _masked as M
from tests._parity import check, cuda, f64, no_device_error
from tests.test_gpu_tree import pack, plain_masks

import numpy as np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,left", [(5, 4), (5, 100), (24, 10), (24, 0), (70, 33)])
@pytest.mark.parametrize("keep", [0, 6])
def test_chain(T, left, keep):
    lens = [T, T + 3, 300, 1000]
    inp = inputs.paged(lens, T, 8, 2, 128, 64, 40, seed=T)
    args = [cuda(x) for x in (inp.q, inp.k_pool, inp.v_pool, inp.block_table, inp.seqlens_k)]
    parents = torch.arange(-1, T - 1, dtype=torch.int32).repeat(4, 1)
    mask, depth = A.attn_tree_mask(cuda(parents))
    sees, dep = plain_masks(parents, [T] * 4)
    near = sees & ((dep[:, :, None] - dep[:, None, :]) <= left)
    if T <= left + 1:
        assert (near == sees).all()
    else:
        # First tokens stay visible: those among the nodes, where nothing lies before them.
        base = np.array(lens)[:, None, None] - T
        near |= sees & (base + np.arange(T)[None, None, :] < keep)
        mask = cuda(pack(near))
    o, lse = A.attn_fwd_paged_tree(*args, mask, tree_depth=depth, window=(left, -1), sink_tokens=keep)
    want, wlse = A.attn_fwd_paged(*args, causal=True, window=(left, -1), sink_tokens=keep)
    for b, L in enumerate(lens):
        seen = M.band(T, L, left, 0, sink_tokens=keep)
        k, v = (M.paged_rows(f64(p), inp.block_table[b].tolist(), L, 64).transpose(1, 0, 2)
                for p in (inp.k_pool, inp.v_pool))
        ro, rl = M.attend(f64(inp.q[b]).transpose(1, 0, 2), np.repeat(k, 4, 0), np.repeat(v, 4, 0), seen, 128 ** -0.5)
        check(o[b].transpose(0, 1), lse[b], ro, rl, "tree")
        check(want[b].transpose(0, 1), wlse[b], ro, rl, "chunk")
    no_device_error()
