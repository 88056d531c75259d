"""A serving loop over a ragged batch: pages reserved, tokens placed, keys rotated into the cache, softmax attention over
the pages, linear attention over the packed rows and token by token.  Eagerly, on streams, and captured."""
import math

import pytest
import torch

import attention_forward_13_gb300 as A
from tests._linear_plain import check, with_bounds
from tests._parity import no_device_error

pytestmark = pytest.mark.gpu
HQ, HKV, D, PAGE = 8, 2, 128, 16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Loop:
    """Two layers' worth of state for B sequences: a paged cache and linear states."""

    def __init__(self, B, pages=160, width=24):
        self.B = B
        self.kp, self.vp = (torch.zeros(pages, PAGE, HKV, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.table, self.lens, self.refs = i32([[-1] * width] * B), i32([0] * B), i32([0] * pages)
        self.states = torch.zeros(B + 2, HQ, D, D, device="cuda")
        self.index = i32(list(range(B))[::-1])
        self.f = A.attn_rope_freqs(D)
        self.g = -(2.0 ** -torch.arange(1, HQ + 1, device="cuda").float())

    def place(self, add, tokens):
        self.table, self.lens, self.refs, free = A.attn_cache_reserve(self.kp, self.vp, self.table, self.lens, self.refs, add)
        return A.attn_cache_slots(self.table, self.lens, add, tokens, PAGE, self.kp.shape[0])


def test_prompts_then_tokens():
    """Prompts of 70, 1, 0 and 200 tokens, then three steps of one token each, against dense attention over all tokens
    so far (with rotated keys) and the linear recurrence."""
    torch.manual_seed(3)
    lens = [70, 1, 0, 200]
    B, steps = len(lens), 3
    loop = Loop(B)
    full = [torch.randn(n + steps, HQ + 2 * HKV, D, device="cuda").bfloat16() for n in lens]
    cu = [sum(lens[:i]) for i in range(B + 1)]
    pad = 9
    x = torch.cat([f[:n] for f, n in zip(full, lens)] + [torch.full((pad, HQ + 2 * HKV, D), math.nan, device="cuda").bfloat16()])
    slots, pos, cu_t, seq = loop.place(i32(lens), cu[-1] + pad)
    assert cu_t.tolist() == cu and seq.tolist()[-pad:] == [-1] * pad
    q, k, v = x.split([HQ, HKV, HKV], 1)
    qr = A.attn_cache_append(k, v, loop.kp, loop.vp, slots, q=q, inv_freq=loop.f, positions=pos)
    kr, _ = A.attn_rope(k.contiguous(), None, loop.f, pos)
    o, _ = A.attn_fwd_varlen(qr, kr, v, cu_t, cu_t, max(lens), causal=True)
    lin, pool = A.attn_linear_fwd_varlen(q, k, v, cu_t, max(lens), loop.g, state=loop.states, state_index=loop.index)
    assert pool is loop.states
    outs, louts = [[o[cu[b]:cu[b + 1]]] for b in range(B)], [[lin[cu[b]:cu[b + 1]]] for b in range(B)]
    one = i32([1] * B)
    for t in range(steps):
        slots, pos, cu_t, _ = loop.place(one, B)
        assert pos.tolist() == [n + t for n in lens] and cu_t.tolist() == list(range(B + 1))
        q, k, v = torch.stack([f[n + t] for f, n in zip(full, lens)]).split([HQ, HKV, HKV], 1)
        qr = A.attn_cache_append(k, v, loop.kp, loop.vp, slots, q=q, inv_freq=loop.f, positions=pos)
        o, _ = A.attn_fwd_paged(qr[:, None], loop.kp, loop.vp, loop.table, loop.lens)
        lo = A.attn_linear_step(q, k, v, loop.g, loop.states, state_index=loop.index)
        for b in range(B):
            outs[b].append(o[b])
            louts[b].append(lo[b][None])
    for b, n in enumerate(lens):
        q, k, v = full[b].split([HQ, HKV, HKV], 1)
        pos = torch.arange(n + steps, dtype=torch.int32, device="cuda")
        qr, kr = A.attn_rope(q.contiguous(), k.contiguous(), loop.f, pos)
        Q, K, V = (t.double().transpose(0, 1) for t in (qr, kr.repeat_interleave(HQ // HKV, 1), v.repeat_interleave(HQ // HKV, 1)))
        s = Q @ K.transpose(1, 2) / math.sqrt(D)
        s = s.masked_fill(pos[:, None] < pos, -math.inf)
        want = (torch.softmax(s, -1) @ V).transpose(0, 1)
        assert (torch.cat(outs[b]).double() - want).abs().max() <= 2e-2
        lw = with_bounds(*(t.transpose(0, 1) for t in (q, k.repeat_interleave(HQ // HKV, 1), v.repeat_interleave(HQ // HKV, 1))),
                         loop.g, 1 / math.sqrt(D))
        check(torch.cat(louts[b]).transpose(0, 1), loop.states[loop.index[b]], lw, b)
    assert not loop.states[B:].any()
    no_device_error()


def serve(loop, x, add, f):
    """One captured step: everything from the lengths in device memory on."""
    slots, pos, cu, _ = A.attn_cache_slots(loop.table, loop.lens, add, x.shape[0], PAGE, loop.kp.shape[0])
    q, k, v = x.split([HQ, HKV, HKV], 1)
    qr = A.attn_cache_append(k, v, loop.kp, loop.vp, slots, q=q, inv_freq=f, positions=pos)
    qq, kk = A.attn_rope(q, k, f, pos)
    lin, _ = A.attn_linear_fwd_varlen(qq, kk, v, cu, x.shape[0], loop.g, state=loop.states, state_index=loop.index)
    step = A.attn_linear_step(qq[:loop.B], kk[:loop.B], v[:loop.B], loop.g, loop.states[:loop.B])
    return slots, qr, qq, kk, lin, step, loop.kp, loop.vp, loop.states


@pytest.mark.parametrize("lens", [[40, 3], [700, 900, 30]])
def test_captured(lens):
    """Captured once, replayed with other contents, two graphs of the same calls in flight one after the other."""
    torch.manual_seed(5)
    loop = Loop(len(lens), width=70, pages=300)
    loop.place(i32(lens), sum(lens))
    add = i32(lens)
    x = torch.randn(sum(lens), HQ + 2 * HKV, D, device="cuda").bfloat16()
    start = torch.randn_like(loop.states)
    serve(loop, x, add, loop.f)  # (loads the kernels)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = serve(loop, x, add, loop.f)
        graphs.append((g, out))
    for seed in (1, 2):
        torch.manual_seed(seed)
        x.copy_(torch.randn(x.shape, device="cuda"))
        loop.states.copy_(start)
        want = [t.clone() for t in serve(loop, x, add, loop.f)]
        for g, out in graphs:
            loop.states.copy_(start)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))
    no_device_error()


def test_streams():
    """Two calls at once on two streams, each with what it allocates on its own."""
    torch.manual_seed(6)
    loops = [Loop(2, width=70, pages=300) for _ in range(2)]
    data = []
    for i, loop in enumerate(loops):
        loop.place(i32([600, 150 + i]), 750 + i)
        data.append((torch.randn(750 + i, HQ + 2 * HKV, D, device="cuda").bfloat16(), i32([600, 150 + i])))
    want = []
    for loop, (x, add) in zip(loops, data):
        want.append([t.clone() for t in serve(loop, x, add, loop.f)])
        loop.states.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in loops]
    for _ in range(4):
        got = []
        for s, loop, (x, add) in zip(streams, loops, data):
            with torch.cuda.stream(s):
                loop.states.zero_()
                got.append(serve(loop, x, add, loop.f))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    no_device_error()


def test_stream_by_argument():
    """stream=s is the call under torch.cuda.stream(s)."""
    q = torch.randn(1, 4, 300, 64, device="cuda").half()
    g = -torch.ones(4, device="cuda")
    f = A.attn_rope_freqs(64)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    a = A.attn_linear_fwd(q, q, q, g, stream=s)
    b = A.attn_rope(q, q, f, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, A.attn_linear_fwd(q, q, q, g)))
    assert all(torch.equal(x, y) for x, y in zip(b, A.attn_rope(q, q, f)))
    no_device_error()
