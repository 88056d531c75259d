"""Calls with a stream by argument: what they allocate and copy on the way belongs to that
stream, as under torch.cuda.stream.  (On the current one, the memory could still be in
use by work queued there, be handed out again while the call's kernels run, and
copies would not be ordered before them.)"""
import pytest
import torch

import attention_forward_13_gb300 as A
from attention_forward_13_gb300 import inputs
from tests._parity import cuda, no_device_error

pytestmark = pytest.mark.gpu


def calls():
    inp = inputs.dense(1, 4, 2, 64, 64, 64, "bf16", seed=1)
    q, k, v = cuda(inp.q), cuda(inp.k), cuda(inp.v)
    pin = inputs.paged([300, 70], 1, 4, 2, 64, 16, 30, seed=2)
    pg = [cuda(x) for x in (pin.q, pin.k_pool, pin.v_pool, pin.block_table, pin.seqlens_k)]
    cu = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    flat = [x[0].transpose(0, 1).contiguous() for x in (q, k, v)]
    part = torch.randn(3, 1, 4, 2, 64, device="cuda"), torch.randn(3, 1, 4, 2, device="cuda")
    strided = part[0].transpose(3, 4).contiguous().transpose(3, 4)
    sink = torch.randn(8, device="cuda")[::2]  # (made contiguous by the call)
    return {
        "dense": lambda **k_: A.attn_fwd(q, k, v, causal=True, sink=sink, **k_),
        "varlen": lambda **k_: A.attn_fwd_varlen(*flat, cu, cu, 64, sink=sink, **k_),
        "paged": lambda **k_: A.attn_fwd_paged(*pg, num_splits=3, sink=sink, **k_),
        "window": lambda **k_: A.attn_fwd_paged(*pg, num_splits=2, causal=True, window=(99, -1), sink_tokens=4, **k_),
        "noalloc": lambda **k_: A.attn_fwd_paged_noalloc(*pg, num_splits=3, sink=sink, **k_),
        "combine": lambda **k_: A.attn_splitkv_combine(strided, part[1], sink=sink, **k_),
    }


NAMES = ["dense", "varlen", "paged", "window", "noalloc", "combine"]


@pytest.mark.parametrize("name", NAMES)
def test_allocations_are_the_streams_own(name, monkeypatch):
    call = calls()[name]
    want = call()
    torch.cuda.synchronize()
    s, made = torch.cuda.Stream(), []
    empty, contiguous = torch.empty, torch.Tensor.contiguous
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (made.append(torch.cuda.current_stream()), empty(*a, **k))[1])
    monkeypatch.setattr(torch.Tensor, "contiguous",
                        lambda t, *a: (made.append(torch.cuda.current_stream()) if t.dim() == 1 else None,
                                       contiguous(t, *a))[1])
    got = call(stream=s)
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert made and all(x == s for x in made), made
    assert torch.cuda.current_stream() != s
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    no_device_error()


@pytest.mark.parametrize("name", NAMES)
def test_nothing_waits_for_or_disturbs_the_current_stream(name):
    """With the current stream held for a while: the call is done when its stream is, and a
    tensor freed on the current stream keeps its contents for what is queued there."""
    call = calls()[name]
    want = call()
    call(stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    shapes = [(t.shape, t.dtype) for t in want] + [((3 * 2 * 4 * 65,), torch.float32)]
    old = [torch.full(sh, 7, dtype=dt, device="cuda") for sh, dt in shapes]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # a tenth of a second
    seen = [t.clone() for t in old]  # queued behind it
    del old
    got = call(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip([g.clone() for g in got], want))
    torch.cuda.synchronize()
    for t in seen:
        assert (t == 7).all()
    no_device_error()


def test_stream_as_a_positional_argument():
    inp = inputs.dense(1, 2, 2, 64, 64, 64, "f16", seed=1)
    q, k, v = cuda(inp.q), cuda(inp.k), cuda(inp.v)
    want = A.attn_fwd(q, k, v, None, True, True, 0.2, 5.0, None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = A.attn_fwd(q, k, v, None, True, True, 0.2, 5.0, None, s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
