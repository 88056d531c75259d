"""What attn_rope, attn_cache_slots, attn_cache_append and the linear attention entry points refuse before anything is
launched, in C (addresses that nothing dereferences) and in Python (CPU tensors)."""
import ctypes
import math

import pytest
import torch

import attention_forward_13_gb300 as A
from attention_forward_13_gb300 import _lib

P = 1 << 12
S = _lib.attn_strides
OK = S(4096, 64, 64)


def rope(lib=None, **kw):
    a = dict(q=P, qo=P, k=P, ko=P, pos=P, stride=0, B=1, L=8, Hq=2, Hkv=2, d=64, dtype=1, s=OK, rot=64, freq=P, scale=0.0)
    a.update(kw)
    o = _lib.attn_rope_opts(a["freq"], a["rot"], 0, 0, a["scale"])
    s = a["s"]
    return A.library().attn_rope(a["q"], a["qo"], a["k"], a["ko"], a["pos"], a["stride"], a["B"], a["L"], a["Hq"],
                                 a["Hkv"], a["d"], a["dtype"], s, s, s, s, ctypes.byref(o), None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(qo=None), 1), (dict(ko=None), 1), (dict(q=P + 2), 1), (dict(pos=P + 2), 1),
    (dict(d=60), 2), (dict(d=520), 2), (dict(d=0), 1), (dict(rot=66), 1), (dict(rot=3), 1), (dict(rot=-2), 1),
    (dict(freq=None), 1), (dict(freq=P + 4), 1), (dict(scale=-1.0), 1), (dict(scale=math.nan), 1),
    (dict(scale=math.inf), 1), (dict(dtype=2), 2), (dict(dtype=7), 1), (dict(B=-1), 1), (dict(L=-1), 1), (dict(Hq=-1), 1),
    (dict(s=S(4096, 64, 60)), 1), (dict(s=S(4096, 0, 64)), 1), (dict(B=2, s=S(0, 64, 64)), 1), (dict(stride=-1), 1),
    (dict(B=1 << 20, L=1 << 12), 2), (dict(Hq=60000, Hkv=6000), 2),
    (dict(B=0), 0), (dict(L=0), 0), (dict(Hq=0, Hkv=0), 0)])
def test_rope(kw, status):
    assert rope(**kw) == status


def test_rope_needs_options():
    assert A.library().attn_rope(P, P, P, P, P, 0, 1, 8, 2, 2, 64, 1, OK, OK, OK, OK, None, None) == 1


def append(**kw):
    a = dict(q=P, qo=P, k=P, v=P, kp=P, vp=P, slots=P, pos=P, n=4, Hq=2, Hkv=2, d=64, dtype=1, page=16, pages=9, s=OK,
             rot=64, inverse=0)
    a.update(kw)
    o = _lib.attn_rope_opts(P, a["rot"], 0, a["inverse"], 0.0)
    s = a["s"]
    return A.library().attn_cache_append(a["q"], a["qo"], a["k"], a["v"], a["kp"], a["vp"], a["slots"], a["pos"], a["n"],
                                         a["Hq"], a["Hkv"], a["d"], a["dtype"], a["page"], a["pages"], s, s, s, s,
                                         ctypes.byref(o), None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(kp=None), 1), (dict(vp=P + 8), 1), (dict(slots=None), 1),
    (dict(pos=None), 1), (dict(page=48), 2), (dict(page=0), 1), (dict(pages=0), 1), (dict(inverse=1), 2), (dict(n=-1), 1),
    (dict(Hkv=0), 1), (dict(d=100), 2), (dict(dtype=2), 2), (dict(pages=1 << 28), 2), (dict(s=S(0, 64, 0)), 1),
    (dict(n=0), 0)])
def test_append(kw, status):
    assert append(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(table=None), 1), (dict(cu=None), 1), (dict(slots=None), 1), (dict(n=-1), 1), (dict(page=48), 2), (dict(B=9000), 2),
    (dict(pages=0), 1), (dict(B=-1), 1), (dict(slots=P + 2), 1)])
def test_slots(kw, status):
    a = dict(table=P, slots=P, cu=P, B=2, n=4, pages=9, page=16)
    a.update(kw)
    assert A.library().attn_cache_slots(a["table"], P, P, a["slots"], P, a["cu"], P, a["B"], a["n"], 3, a["pages"],
                                        a["page"], None) == status


def linear(form="dense", **kw):
    a = dict(q=P, k=P, v=P, o=2 * P, cu=P, g=P, si=P, so=P, index=None, n=1, B=1, Hq=2, Hkv=2, L=8, total=8, d=64, dtype=1,
             s=OK, scale=0.0, work=P, size=1 << 30)
    a.update(kw)
    lib, s = A.library(), [a["s"]] * 4
    if form == "dense":
        return lib.attn_linear_fwd(a["q"], a["k"], a["v"], a["o"], a["g"], a["si"], a["so"], a["index"], a["n"], a["B"],
                                   a["Hq"], a["Hkv"], a["L"], a["d"], a["dtype"], *s, a["scale"], a["work"], a["size"], None)
    if form == "packed":
        return lib.attn_linear_fwd_varlen(a["q"], a["k"], a["v"], a["o"], a["cu"], a["g"], a["si"], a["so"], a["index"],
                                          a["n"], a["B"], a["total"], a["L"], a["Hq"], a["Hkv"], a["d"], a["dtype"], *s,
                                          a["scale"], a["work"], a["size"], None)
    return lib.attn_linear_step(a["q"], a["k"], a["v"], a["o"], a["g"], a["si"], a["index"], a["n"], a["B"], a["Hq"],
                                a["Hkv"], a["d"], a["dtype"], *s, a["scale"], None)


@pytest.mark.parametrize("form", ["dense", "packed", "step"])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(o=None), 1), (dict(v=P + 2), 1), (dict(g=None), 1), (dict(g=P + 1), 1), (dict(si=P + 4), 1),
    (dict(n=0), 1), (dict(B=3, n=2), 1), (dict(index=P + 2), 1), (dict(Hq=3), 1), (dict(Hkv=0), 1), (dict(d=96), 2),
    (dict(dtype=2), 2), (dict(dtype=9), 1), (dict(scale=math.nan), 1), (dict(B=-1), 1), (dict(B=0), 0),
    (dict(B=70000, n=70000), 2), (dict(s=S(4096, 60, 64)), 1), (dict(o=P), 1)])
def test_linear(form, kw, status):
    assert linear(form, **kw) == status


def test_linear_lengths():
    assert linear(L=-1) == 1 and linear("packed", L=-1) == 1 and linear("packed", total=-1) == 1
    assert linear("packed", cu=None) == 1
    assert linear("step", si=None) == 1
    assert linear(s=S(4096, 64, 60)) == 1


# ------------------------------------------------------------------- Python
bf = dict(dtype=torch.bfloat16)
Q, K = torch.zeros(5, 4, 64, **bf), torch.zeros(5, 2, 64, **bf)
Q4, K4 = torch.zeros(2, 4, 5, 64, **bf), torch.zeros(2, 2, 5, 64, **bf)
F = torch.ones(32, dtype=torch.float64)
I5 = torch.zeros(5, dtype=torch.int32)


@pytest.mark.parametrize("a,kw", [
    ((Q, K.half(), F), {}), ((Q, K[:4], F), {}), ((Q4, K, F), {}), ((Q4, K4[:1], F), {}), ((Q, K, F.float()), {}),
    ((Q, K, torch.ones(33, dtype=torch.float64)), {}), ((Q, K, F[::2]), {}), ((Q, K, F, I5.long()), {}),
    ((Q, K, F, I5[:4]), {}), ((Q4, K4, F, torch.zeros(3, 5, dtype=torch.int32)), {}), ((Q, K, F), dict(q_out=Q4)),
    ((Q, K, F), dict(k_out=Q)), ((Q, None, F), dict(k_out=K)), ((Q[0], None, F), {})])
def test_rope_python(a, kw):
    with pytest.raises(ValueError):
        A.attn_rope(*a, **kw)


POOL = torch.zeros(3, 16, 2, 64, **bf)


@pytest.mark.parametrize("kw", [
    dict(v=K[:4]), dict(v=K.half()), dict(k_pool=POOL.half()), dict(k_pool=POOL[:2]), dict(k_pool=POOL[..., :32]),
    dict(k_pool=POOL[:, ::2], v_pool=POOL[:, ::2]), dict(slots=I5.long()), dict(slots=I5[:3]), dict(positions=I5[:3]), dict(q=Q[:4]),
    dict(q=Q.half()), dict(q=None, q_out=Q), dict(positions=None), dict(inv_freq=F.float())])
def test_append_python(kw):
    a = dict(k=K, v=K, k_pool=POOL, v_pool=POOL, slots=I5, q=Q, inv_freq=F, positions=I5)
    a.update(kw)
    with pytest.raises(ValueError):
        A.attn_cache_append(**a)


def test_slots_python():
    t = torch.zeros(2, 3, dtype=torch.int32)
    n = torch.ones(2, dtype=torch.int32)
    for a in [(t, n, n, 1 << 30, 16, 9), (t, n.long(), n, 4, 16, 9), (t, n, n[:1], 4, 16, 9), (t.long(), n, n, 4, 16, 9), (t, n, n, -1, 16, 9)]:
        with pytest.raises(ValueError):
            A.attn_cache_slots(*a)


G4 = torch.zeros(4)
ST = torch.zeros(2, 4, 64, 64)
I2 = torch.zeros(2, dtype=torch.int32)


@pytest.mark.parametrize("kw", [
    dict(k=K4[:1]), dict(v=K4.half()), dict(log_decay=G4[:2]), dict(log_decay=G4.double()), dict(state=ST[:1]),
    dict(state=ST.half()), dict(state=ST.transpose(0, 1)), dict(state=torch.zeros(2, 2, 64, 64)), dict(state_out=ST[:1]),
    dict(state_index=I2.long(), state=ST), dict(state_index=I2), dict(state_index=I2[:1], state=ST), dict(o=Q4[:1]),
    dict(state=ST, state_index=I2, state_out=torch.zeros(3, 4, 64, 64))])
def test_linear_python(kw):
    a = dict(q=Q4, k=K4, v=K4, log_decay=G4)
    a.update(kw)
    with pytest.raises(ValueError):
        A.attn_linear_fwd(**a)


def test_linear_packed_and_step_python():
    cu = torch.tensor([0, 2, 5], dtype=torch.int32)
    for kw in (dict(cu_seqlens=cu.long()), dict(k=K[:4], v=K[:4]), dict(state=ST[:1]), dict(cu_seqlens=cu[:0])):
        with pytest.raises(ValueError):
            A.attn_linear_fwd_varlen(**{**dict(q=Q, k=K, v=K, cu_seqlens=cu, max_seqlen=3, log_decay=G4), **kw})
    for kw in (dict(k=K[:4], v=K[:4]), dict(state=ST), dict(o=Q[:4]), dict(log_decay=G4[:1])):
        with pytest.raises(ValueError):
            A.attn_linear_step(**{**dict(q=Q, k=K, v=K, log_decay=G4, state=torch.zeros(5, 4, 64, 64)), **kw})


def test_linear_workspace():
    """None where heads fill the GPU or sequences are short; else a state for every piece of each head."""
    W = A.attn_linear_workspace_bytes
    assert W(2, 32, 8192, 2 * 8192, 128) == 0 and W(1, 16, 128, 128, 128) == 0 and W(0, 4, 100, 0, 64) == 0
    assert W(1, 16, 2048, 2048, 128) == 4 * 16 * 128 * 128 * 4
    assert W(1, 1, 1 << 20, 1 << 20, 64) == 16 * 64 * 64 * 4        # at most 16 pieces
    assert W(60000, 1, 100000, 200000, 64) == 0                      # a grid's third dimension
    # the buffer a call needs is the one this says, whatever the lengths
    assert linear(B=1, Hq=16, Hkv=16, L=2048, d=128, n=1, s=S(1 << 24, 2048 * 128, 128), work=None) == 1
    assert linear(B=1, Hq=16, Hkv=16, L=2048, d=128, n=1, s=S(1 << 24, 2048 * 128, 128), size=1000) == 1
