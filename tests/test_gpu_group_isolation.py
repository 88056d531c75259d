"""Group mode: a sequence's results depend on its own rows alone.  K and V rows of its
neighbours, and packed rows behind the last sequence, may hold NaN or infinity."""
import pytest
import torch

import attention_forward_13_gb300 as A
from tests._parity import no_device_error

pytestmark = pytest.mark.gpu

OPTS = [dict(), dict(causal=True), dict(window=(40, 5)), dict(causal=True, window=(100, -1), sink_tokens=4),
        dict(causal=True, window=(30, -1), sink_tokens=150), dict(causal=True, softcap=20.0),
        dict(causal=True, window=(60, -1), sink_tokens=5, softcap=30.0), dict(causal=True, alibi=True)]
KINDS = [(64, torch.float16), (128, torch.bfloat16), (128, torch.float8_e4m3fn)]


@pytest.mark.parametrize("opts", OPTS, ids=[str(i) for i in range(len(OPTS))])
@pytest.mark.parametrize("d,dt", KINDS, ids=["f16", "bf16", "e4m3"])
def test_neighbours(opts, d, dt):
    opts = dict(opts)
    if dt is torch.float8_e4m3fn and (opts.get("softcap") or opts.get("alibi")):
        pytest.skip("not built")
    Hq, Hkv = 4, 2
    if opts.pop("alibi", False):
        opts["alibi_slopes"] = torch.tensor([0.5, 0.25, 0.1, 0.01], device="cuda")
    lens = [300, 1, 129, 77, 128, 400, 0, 19]
    extra = 200  # rows behind the last sequence
    g = torch.Generator(device="cuda").manual_seed(d)
    n = sum(lens) + extra
    q, k, v = (torch.randn(n, h, d, generator=g, device="cuda").to(dt) for h in (Hq, Hkv, Hkv))
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")
    want, wlse = A.attn_fwd_varlen(q, k, v, cu, cu, 400, **opts)
    bad = torch.full_like(k.float(), float("nan"))
    if dt is not torch.float8_e4m3fn:
        bad[::2] = float("inf")
    for odd in (0, 1):  # every second sequence's keys and values, and the rows behind the last
        kk, vv = k.float(), v.float()
        for b in range(len(lens)):
            if b % 2 == odd:
                kk[cu[b]:cu[b + 1]], vv[cu[b]:cu[b + 1]] = bad[cu[b]:cu[b + 1]], bad[cu[b]:cu[b + 1]]
        kk[cu[-1]:], vv[cu[-1]:] = bad[cu[-1]:], bad[cu[-1]:]
        o, lse = A.attn_fwd_varlen(q, kk.to(dt), vv.to(dt), cu, cu, 400, **opts)
        for b in range(len(lens)):
            if b % 2 != odd:
                s = slice(int(cu[b]), int(cu[b + 1]))
                assert torch.equal(o[s].float(), want[s].float()), (odd, b)
                assert torch.equal(lse[:, s], wlse[:, s]), (odd, b)
    no_device_error()
