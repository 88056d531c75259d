"""Windows whose first tokens stay visible with e4m3 inputs: packed sequences, shared kv
heads, first tokens in the band's first tile and in tiles of their own, scales.
Tolerances as in _parity.check_e4m3."""
import math

import numpy as np
import pytest
import torch

import attention_forward_13_gb300 as A
from attention_forward_13_gb300 import inputs
from tests import _masked as M
from tests._parity import check_e4m3, cuda, f64, no_device_error

pytestmark = pytest.mark.gpu

CASES = [
    # lens_q, lens_k, Hq, Hkv, causal, window, keep, sink, scale_o
    ([300, 1, 129, 0, 513], None, 4, 2, True, (64, -1), 4, False, None),
    ([700, 130], [900, 400], 4, 4, False, (100, 20), 150, True, 2.0),
    ([5, 260], [700, 3], 8, 1, True, (16, -1), 60, False, 0.5),
    ([385], [385], 2, 2, False, (0, 0), 1, True, None),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
@pytest.mark.parametrize("packed", [True, False])
def test_parity(case, packed):
    lq, lk, Hq, Hkv, causal, win, keep, with_sink, so = case
    lk = lq if lk is None else lk
    g, scale = Hq // Hkv, 1 / math.sqrt(128)
    inp = inputs.varlen(lq, lk, Hq, Hkv, 128, "e4m3", seed=sum(lq))
    sink = torch.randn(Hq, device="cuda") if with_sink else None
    kw = dict(causal=causal, window=win, sink_tokens=keep, sink=sink, scale_o=so)
    if packed:
        o, lse = A.attn_fwd_varlen(cuda(inp.q), cuda(inp.k), cuda(inp.v), cuda(inp.cu_seqlens_q),
                                   cuda(inp.cu_seqlens_k), inp.max_seqlen_q, **kw)
    cq, ck = inp.cu_seqlens_q.tolist(), inp.cu_seqlens_k.tolist()
    for b in range(len(lq)):
        if lq[b] == 0:
            continue
        q, k, v = (x[c[b]:c[b + 1]].transpose(0, 1) for x, c in ((inp.q, cq), (inp.k, ck), (inp.v, ck)))
        if packed:
            ob, lb = o[cq[b]:cq[b + 1]].transpose(0, 1), lse[:, cq[b]:cq[b + 1]]
        else:
            ob, lb = (x[0] for x in A.attn_fwd(*(cuda(x.contiguous()[None]) for x in (q, k, v)), **kw))
        seen = M.band(lq[b], lk[b], win[0], 0 if causal else win[1], sink_tokens=keep)
        ro, rl = M.attend(f64(q), np.repeat(f64(k), g, 0), np.repeat(f64(v), g, 0), seen, scale, 0.0,
                          None if sink is None else f64(sink))
        vmax = float(np.abs(f64(v)).max()) if lk[b] else 0.0
        check_e4m3(ob, lb, ro * (so or 1.0), rl, "sequence %d" % b, min_exact=0.9, o_scale=so or 1.0, vmax=vmax)
    no_device_error()
