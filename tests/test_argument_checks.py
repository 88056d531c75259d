"""The entry points check what their kernels take for granted before anything is
launched: types, shapes, layouts.  (CPU tensors: a call that passes the checks
would fail later.)"""
import pytest
import torch

import attention_forward_13_gb300 as A


def args(**kw):
    a = dict(q=torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16), k=torch.zeros(5, 16, 2, 64, dtype=torch.bfloat16),
             v=torch.zeros(5, 16, 2, 64, dtype=torch.bfloat16), table=torch.zeros(2, 3, dtype=torch.int32),
             lens=torch.ones(2, dtype=torch.int32))
    a.update(kw)
    return [a[n] for n in ("q", "k", "v", "table", "lens")]


BAD = {
    "table of int64": (args(table=torch.zeros(2, 3, dtype=torch.int64)), {}),
    "lengths of int64": (args(lens=torch.ones(2, dtype=torch.int64)), {}),
    "a table row short": (args(table=torch.zeros(1, 3, dtype=torch.int32)), {}),
    "a flat table": (args(table=torch.zeros(6, dtype=torch.int32)), {}),
    "a length short": (args(lens=torch.ones(1, dtype=torch.int32)), {}),
    "a strided table": (args(table=torch.zeros(2, 6, dtype=torch.int32)[:, ::2]), {}),
    "pools of another type": (args(k=torch.zeros(5, 16, 2, 64, dtype=torch.float16)), {}),
    "a smaller v pool": (args(v=torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)), {}),
    "another head dimension": (args(q=torch.zeros(2, 1, 4, 128, dtype=torch.bfloat16)), {}),
    "o of another type": (args(), dict(o=torch.zeros(2, 1, 4, 64))),
    "o of another shape": (args(), dict(o=torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16))),
    "a short lse": (args(), dict(lse=torch.zeros(2, 3, 1))),
    "lse of bf16": (args(), dict(lse=torch.zeros(2, 4, 1, dtype=torch.bfloat16))),
}


@pytest.mark.parametrize("name", BAD)
@pytest.mark.parametrize("fn", [A.attn_fwd_paged, A.attn_fwd_paged_noalloc], ids=["paged", "noalloc"])
def test_refused(name, fn):
    a, kw = BAD[name]
    with pytest.raises(ValueError):
        fn(*a, num_splits=2, **kw)


@pytest.mark.parametrize("workspace", [torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(1 << 20, dtype=torch.bfloat16),
                                       torch.zeros(1 << 12)[::2], torch.zeros(64, 64)])
def test_workspace_refused(workspace):
    """It is counted and cut in floats."""
    with pytest.raises(ValueError, match="workspace"):
        A.attn_fwd_paged(*args(), num_splits=2, workspace=workspace)


Q4, K4 = torch.zeros(2, 4, 8, 64, dtype=torch.float16), torch.zeros(2, 2, 9, 64, dtype=torch.float16)
DENSE = {
    "v of another length": ((Q4, K4, K4[:, :, :8]), {}),
    "k of another type": ((Q4, K4.bfloat16(), K4.bfloat16()), {}),
    "k of another head dimension": ((Q4, torch.zeros(2, 2, 9, 128, dtype=torch.float16),
                                     torch.zeros(2, 2, 9, 128, dtype=torch.float16)), {}),
    "k of fewer batches": ((Q4, K4[:1], K4[:1]), {}),
    "a bias of fewer keys": ((Q4, K4, K4), dict(bias=torch.zeros(1, 1, 8, 8, dtype=torch.float16))),
    "a bias of fewer rows": ((Q4, K4, K4), dict(bias=torch.zeros(2, 4, 7, 9, dtype=torch.float16))),
    "a bias of fewer heads": ((Q4, K4, K4), dict(bias=torch.zeros(2, 2, 8, 9, dtype=torch.float16))),
    "o of another type": ((Q4, K4, K4), dict(o=Q4.float())),
    "o of another shape": ((Q4, K4, K4), dict(o=Q4[:, :, :7])),
    "a short lse": ((Q4, K4, K4), dict(lse=torch.zeros(2, 4, 7))),
    "a strided lse": ((Q4, K4, K4), dict(lse=torch.zeros(2, 4, 16)[..., ::2])),
}


@pytest.mark.parametrize("name", DENSE)
def test_dense_refused(name):
    a, kw = DENSE[name]
    with pytest.raises(ValueError):
        A.attn_fwd(*a, **kw)


CU = torch.tensor([0, 3, 8], dtype=torch.int32)
Q3, K3 = torch.zeros(8, 4, 64, dtype=torch.float16), torch.zeros(9, 2, 64, dtype=torch.float16)
PACKED = {
    "fewer key sequences": ((Q3, K3, K3, CU, CU[:2], 5), {}),
    "v of another length": ((Q3, K3, K3[:8], CU, CU, 5), {}),
    "k of another type": ((Q3, K3.bfloat16(), K3.bfloat16(), CU, CU, 5), {}),
    "o of another shape": ((Q3, K3, K3, CU, CU, 5), dict(o=torch.zeros(8, 2, 64, dtype=torch.float16))),
    "a short lse": ((Q3, K3, K3, CU, CU, 5), dict(lse=torch.zeros(4, 7))),
}


@pytest.mark.parametrize("name", PACKED)
def test_packed_refused(name):
    a, kw = PACKED[name]
    with pytest.raises(ValueError):
        A.attn_fwd_varlen(*a, **kw)
