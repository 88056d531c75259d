"""Tree attention of one sequence over a long cache with few kv heads: the unit of a kv
head is cut into a piece for every CTA (or every second), all merged in one pass."""
import math

import pytest
import torch

import attention_forward_13_gb300 as A
from attention_forward_13_gb300 import inputs
from tests._parity import check, cuda, no_device_error
from tests.test_gpu_tree import plain_masks, random_parents, reference

pytestmark = pytest.mark.gpu

CASES = [
    # keys, T, Hq, Hkv, d, page, dtype, cap, sink
    (160_000, 4, 8, 1, 64, 256, "bf16", 0.0, False),    # two streams, a piece per CTA
    (163_001, 24, 8, 1, 128, 64, "f16", 0.0, True),     # two query tiles
    (150_017, 1, 16, 2, 128, 16, "bf16", 30.0, True),   # two units
    (700, 3, 4, 1, 64, 16, "f16", 0.0, False),          # a few short pieces
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_one_sequence(case):
    import numpy as np
    L, T, Hq, Hkv, d, page, dt, cap, sink = case
    inp = inputs.paged([L], T, Hq, Hkv, d, page, -(-L // page) + 3, dtype=dt, seed=T + d, softcap=cap, with_sink=sink)
    parents = random_parents(np.random.default_rng(T), 1, T)
    sees, depth = plain_masks(parents, [T])
    ro, rl = reference(inp, sees, depth, [T], 1 / math.sqrt(d), cap)
    mask, _ = A.attn_tree_mask(cuda(parents))
    need = A.attn_tree_workspace_bytes(T, Hq, Hkv, d)
    space = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN, and notes that name no unit
    args = (cuda(inp.q), cuda(inp.k_pool), cuda(inp.v_pool), cuda(inp.block_table), cuda(inp.seqlens_k), mask)
    kw = dict(softcap=cap, sink=cuda(inp.sink), workspace=space)
    o, lse = A.attn_fwd_paged_tree(*args, **kw)
    torch.cuda.synchronize()
    no_device_error()
    check(o, lse, ro, rl, "one sequence")
    for _ in range(20):  # the same bits, whatever the order the CTAs ran in
        o2, lse2 = A.attn_fwd_paged_tree(*args, **kw)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    no_device_error()
