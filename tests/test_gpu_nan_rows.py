"""NaN that a row sees comes out of it, O and LSE, on the dense, packed, paged and split
paths; an LSE of -inf says that a row has seen nothing, and a merge by LSE leaves such
parts out."""
import pytest
import torch

import attention_forward_13_gb300 as A
from attention_forward_13_gb300 import inputs
from tests._parity import cuda, no_device_error

pytestmark = pytest.mark.gpu

NAN = float("nan")


def same_but(o, lse, want, wlse, bad):
    """Rows of `bad` are NaN, the others the bits they were.  o [..., d], the rest [...]."""
    assert o.float().isnan()[bad].all() and lse.isnan()[bad].all()
    assert torch.equal(o[~bad].float(), want[~bad].float()) and torch.equal(lse[~bad], wlse[~bad])


OPTS = [dict(), dict(causal=True), dict(window=(70, 3), sink_tokens=2), dict(causal=True, softcap=20.0),
        dict(causal=True, sink=True), dict(alibi=True), dict(bias=True), dict(window=(30, 0), sink_tokens=9, sink=True)]


@pytest.mark.parametrize("opts", OPTS, ids=[str(i) for i in range(len(OPTS))])
@pytest.mark.parametrize("d,dt", [(64, "f16"), (128, "bf16")])
def test_dense(opts, d, dt):
    opts = dict(opts)
    Hq, Hkv, L = 4, 2, 300
    inp = inputs.dense(1, Hq, Hkv, L, L, d, dt, seed=d)
    q, k, v = cuda(inp.q), cuda(inp.k), cuda(inp.v)
    if opts.pop("sink", None):
        opts["sink"] = torch.randn(Hq, device="cuda")
    if opts.pop("alibi", None):
        opts["alibi_slopes"] = torch.rand(Hq, device="cuda")
    if opts.pop("bias", None):
        opts["bias"] = torch.randn(1, 1, L, 304, device="cuda").to(q.dtype)[..., :L]
    want, wlse = A.attn_fwd(q, k, v, **opts)
    q2 = q.clone()
    q2[0, 1, 150, 3] = q2[0, 2, 0, 0] = q2[0, 3, 299, d - 1] = NAN
    bad = torch.zeros(1, Hq, L, dtype=torch.bool, device="cuda")
    bad[0, 1, 150] = bad[0, 2, 0] = bad[0, 3, 299] = True
    same_but(*A.attn_fwd(q2, k, v, **opts), want, wlse, bad)
    k2 = k.clone()
    k2[0, 1, 0, 5] = NAN  # key 0 of kv head 1: the causal rows and those whose window reaches it
    i = torch.arange(L, device="cuda")
    sees = torch.ones(L, dtype=torch.bool, device="cuda")
    if "window" in opts and not opts.get("sink_tokens"):
        sees = i <= opts["window"][0]
    bad = torch.zeros(1, Hq, L, dtype=torch.bool, device="cuda")
    bad[0, 2:] = sees
    same_but(*A.attn_fwd(q, k2, v, **opts), want, wlse, bad)
    no_device_error()


def test_fp8_and_packed():
    Hq, L, d = 2, 200, 128
    q, k, v = (torch.randn(2 * L, Hq, d, device="cuda") for _ in range(3))
    cu = torch.tensor([0, L, 2 * L], dtype=torch.int32, device="cuda")
    for dt in (torch.bfloat16, torch.float8_e4m3fn):
        args = [x.to(dt) for x in (q, k, v)]
        want, wlse = A.attn_fwd_varlen(*args, cu, cu, L, causal=True)
        q2 = q.clone()
        q2[L + 7, 1, 2] = NAN
        o, lse = A.attn_fwd_varlen(q2.to(dt), *args[1:], cu, cu, L, causal=True)
        bad = torch.zeros(2 * L, Hq, dtype=torch.bool, device="cuda")
        bad[L + 7, 1] = True
        same_but(o, lse.t(), want, wlse.t(), bad)
    no_device_error()


@pytest.mark.parametrize("Lq", [1, 4, 40])  # decode; the chunked prefill
@pytest.mark.parametrize("splits", [0, 1, 2, 5])
@pytest.mark.parametrize("opts", [dict(), dict(sink=True, causal=True), dict(causal=True, window=(200, -1), sink_tokens=5)],
                         ids=["plain", "sink", "window"])
def test_paged(Lq, splits, opts):
    opts = dict(opts)
    inp = inputs.paged([500, 333], Lq, 8, 2, 128, 32, 40, dtype="bf16", seed=Lq)
    if opts.pop("sink", None):
        opts["sink"] = torch.randn(8, device="cuda")
    q, kp, vp, bt, sl = (cuda(x) for x in (inp.q, inp.k_pool, inp.v_pool, inp.block_table, inp.seqlens_k))
    want, wlse = A.attn_fwd_paged(q, kp, vp, bt, sl, num_splits=splits, **opts)
    q2 = q.clone()
    q2[1, Lq - 1, 6, 9] = NAN
    bad = torch.zeros(2, Lq, 8, dtype=torch.bool, device="cuda")
    bad[1, Lq - 1, 6] = True
    o, lse = A.attn_fwd_paged(q2, kp, vp, bt, sl, num_splits=splits, **opts)
    same_but(o, lse.transpose(1, 2), want, wlse.transpose(1, 2), bad)
    k2 = kp.clone()
    k2[bt[0, 0].item(), 3, 1, 4] = NAN  # key 3 of sequence 0, kv head 1: one split's
    bad = torch.zeros(2, Lq, 8, dtype=torch.bool, device="cuda")
    bad[0, :, 4:] = True
    o, lse = A.attn_fwd_paged(q, k2, vp, bt, sl, num_splits=splits, **opts)
    same_but(o, lse.transpose(1, 2), want, wlse.transpose(1, 2), bad)
    no_device_error()


def test_combine():
    """A part with a NaN LSE makes the row NaN; parts of -inf are left out; all of them: empty."""
    S, B, H, L, d = 5, 1, 2, 3, 64
    o, lse = torch.randn(S, B, H, L, d, device="cuda"), torch.randn(S, B, H, L, device="cuda")
    lse[3, 0, 0, 1] = float("-inf")
    lse[2, 0, 1, 2] = NAN
    o[2, 0, 1, 2] = NAN
    lse[:, 0, 1, 0] = NAN
    lse[:, 0, 0, 2] = float("-inf")
    for sink in (None, torch.randn(H, device="cuda")):
        out, l = A.attn_splitkv_combine(o, lse, sink=sink)
        for h, i in ((1, 2), (1, 0)):
            assert out[0, i, h].isnan().all() and l[0, h, i].isnan()
        assert not out[0, 2, 0].any() and torch.equal(l[0, 0, 2], torch.tensor(float("-inf"), device="cuda")
                                                     if sink is None else sink[0])
        assert out[0, :2, 0].isfinite().all() and l[0, 0, :2].isfinite().all() and l[0, 1, 1].isfinite()
    no_device_error()
