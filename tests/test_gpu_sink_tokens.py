"""GPU parity of the sliding window whose first tokens stay visible
(attn_opts.sink_tokens) against the definition in 64 bits: dense, group mode,
paged decode with splits, chunked prefill; first tokens that end inside a tile
or a page, reach into the band, or exceed the sequence; rows the right bound
leaves without any of them; the pages between them and the band, which are never
read.  Tolerances as in _parity.py (one output rounding plus the kernel's own
2e-2 budget; LSE 1e-3)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import attention_forward_13_gb300 as A
from attention_forward_13_gb300 import _lib, inputs
from tests import _masked as M
from tests._parity import check, check_e4m3, cuda, f64, no_device_error

gpu = pytest.mark.gpu


def _dense_ref(q, k, v, keep, scale, cap=0.0, sink=None, bias=None):
    g = q.shape[1] // k.shape[1]
    outs = [M.attend(f64(q[b]), np.repeat(f64(k[b]), g, 0), np.repeat(f64(v[b]), g, 0), keep, scale, cap,
                     None if sink is None else f64(sink), bias) for b in range(q.shape[0])]
    return np.stack([o for o, _ in outs]), np.stack([l for _, l in outs])


DENSE = [
    # B, Hq, Hkv, Lq, Lk, d, dtype, causal, window, keep, cap, sink, top_left
    (1, 2, 2, 700, 700, 128, "bf16", True, (100, -1), 4, 0.0, False, False),
    (1, 4, 2, 900, 900, 64, "f16", True, (64, -1), 130, 0.0, True, False),    # ends in tile 1
    (2, 8, 2, 513, 513, 128, "bf16", False, (30, 20), 1, 0.0, False, False),   # packed heads
    (1, 2, 1, 300, 1300, 64, "bf16", True, (200, -1), 256, 30.0, True, False),  # Lq < Lk
    (1, 2, 2, 900, 300, 128, "bf16", True, (64, -1), 40, 0.0, False, False),   # Lq > Lk: keyless rows
    (1, 2, 2, 600, 600, 128, "f16", True, (0, -1), 5000, 0.0, False, False),   # more than the keys
    (1, 3, 3, 385, 385, 64, "bf16", False, (0, 0), 3, 0.0, True, False),       # the diagonal and 3
    (1, 2, 2, 500, 400, 128, "bf16", False, (50, 10), 7, 0.0, False, True),    # top-left, rows past the keys
    (1, 16, 1, 200, 200, 128, "bf16", True, (16, -1), 2, 0.0, False, False),   # 16 heads per tile
    (1, 1, 1, 1, 1, 64, "f16", True, (0, -1), 1, 0.0, False, False),
    # first tokens in the band's first tile: whole multiples of 8 and not, the most and one more
    (1, 2, 2, 1000, 1000, 128, "bf16", True, (150, -1), 8, 0.0, False, False),
    (1, 8, 2, 1111, 1111, 64, "f16", True, (255, -1), 63, 30.0, True, False),
    (2, 4, 4, 777, 1500, 128, "bf16", True, (301, -1), 64, 0.0, True, False),
    (1, 2, 1, 900, 900, 128, "bf16", True, (200, -1), 65, 0.0, False, False),
    (1, 2, 2, 640, 640, 64, "bf16", False, (100, 200), 17, 0.0, False, False),
    (1, 2, 2, 500, 900, 128, "f16", False, (40, 3), 33, 0.0, False, True),
    (1, 1, 1, 2000, 2000, 64, "bf16", True, (0, -1), 1, 0.0, False, False),
]


@gpu
@pytest.mark.parametrize("case", DENSE, ids=[str(i) for i in range(len(DENSE))])
def test_dense(case):
    B, Hq, Hkv, Lq, Lk, d, dt, causal, win, keep, cap, sink, tl = case
    inp = inputs.dense(B, Hq, Hkv, Lq, Lk, d, dt, seed=7 + Lq + keep, softcap=cap, with_sink=sink)
    o, lse = A.attn_fwd(cuda(inp.q), cuda(inp.k), cuda(inp.v), causal=causal, softcap=cap,
                        sink=cuda(inp.sink), window=win, top_left=tl, sink_tokens=keep)
    torch.cuda.synchronize()
    assert "_window_keep_" in A.attn_last_kernel_name() or "topleft" in A.attn_last_kernel_name()
    seen = M.band(Lq, Lk, win[0], 0 if causal else win[1], keep, tl)
    ro, rl = _dense_ref(inp.q, inp.k, inp.v, seen, 1 / math.sqrt(d), cap, inp.sink)
    check(o, lse, ro, rl, "dense")
    no_device_error()


@gpu
def test_dense_strides_alibi_and_bias():
    """Non-contiguous inputs, ALiBi (the first tokens keep their true distance) and an
    elementwise bias."""
    d, L, H = 128, 420, 4
    inp = inputs.dense(1, H, H, L, L, d, "bf16", seed=5)
    q, k, v = (cuda(x).transpose(1, 2).contiguous().transpose(1, 2) for x in (inp.q, inp.k, inp.v))
    seen = M.band(L, L, 60, 0, 33)
    slopes = torch.tensor([2.0 ** -(h + 3) for h in range(H)])
    o, lse = A.attn_fwd(q, k, v, causal=True, window=(60, -1), sink_tokens=33, alibi_slopes=cuda(slopes))
    ro, rl = _dense_ref(inp.q, inp.k, inp.v, seen, 1 / math.sqrt(d), bias=M.alibi_bias(slopes.numpy(), L, L))
    check(o, lse, ro, rl, "alibi")
    bias = torch.randn(1, H, L, 424, generator=torch.Generator().manual_seed(2)).bfloat16()
    o, lse = A.attn_fwd(q, k, v, causal=True, window=(60, -1), sink_tokens=33, bias=cuda(bias)[..., :L])
    ro, rl = _dense_ref(inp.q, inp.k, inp.v, seen, 1 / math.sqrt(d), bias=f64(bias[0, :, :, :L]))
    check(o, lse, ro, rl, "bias")
    no_device_error()


@gpu
def test_more_first_tokens_than_any_cache_holds():
    inp = inputs.paged([700, 90], 1, 8, 2, 64, 16, 60, seed=3)
    args = [cuda(x) for x in (inp.q, inp.k_pool, inp.v_pool, inp.block_table, inp.seqlens_k)]
    a = A.attn_fwd_paged(*args, causal=True, window=(5, -1), sink_tokens=0x7fffffff)
    ro, rl = _paged_ref(inp, 5, 10 ** 6, 0.0, 64)
    check(*a, ro, rl, "all")
    q = cuda(inputs.dense(1, 2, 2, 300, 300, 64, "bf16", seed=1).q)
    b = A.attn_fwd(q, q, q, causal=True, window=(5, -1), sink_tokens=0x7fffffff)
    ro, rl = _dense_ref(q.cpu(), q.cpu(), q.cpu(), M.band(300, 300, -1, 0), 1 / 8)
    check(*b, ro, rl, "dense")
    no_device_error()


@gpu
def test_fp8():
    inp = inputs.dense(1, 2, 2, 600, 600, 128, "e4m3", seed=21)
    o, lse = A.attn_fwd(cuda(inp.q), cuda(inp.k), cuda(inp.v), causal=True, window=(90, -1), sink_tokens=4)
    ro, rl = _dense_ref(inp.q, inp.k, inp.v, M.band(600, 600, 90, 0, 4), 1 / math.sqrt(128))
    check_e4m3(o, lse, ro, rl, "fp8", min_exact=0.9, vmax=float(inp.v.float().abs().max()))
    no_device_error()


VARLEN = [
    # lens_q, lens_k, Hq, Hkv, d, dtype, causal, window, keep
    ([1, 0, 130, 257, 500], None, 4, 2, 128, "bf16", True, (64, -1), 4),
    ([5, 100, 64], [300, 100, 1], 2, 2, 64, "f16", False, (32, 16), 140),
    ([513, 1, 129], [513, 1000, 0], 8, 2, 128, "bf16", False, (200, 0), 1),
    ([700, 3, 1025], [900, 400, 1025], 4, 4, 64, "f16", True, (130, -1), 60),
]


@gpu
@pytest.mark.parametrize("case", VARLEN, ids=[str(i) for i in range(len(VARLEN))])
def test_varlen(case):
    lq, lk, Hq, Hkv, d, dt, causal, win, keep = case
    lk = lk if lk is not None else lq
    inp = inputs.varlen(lq, lk, Hq, Hkv, d, dt, seed=sum(lq) + 5)
    o, lse = A.attn_fwd_varlen(cuda(inp.q), cuda(inp.k), cuda(inp.v), cuda(inp.cu_seqlens_q),
                               cuda(inp.cu_seqlens_k), inp.max_seqlen_q, causal=causal, window=win,
                               sink_tokens=keep)
    torch.cuda.synchronize()
    cq, ck = inp.cu_seqlens_q.tolist(), inp.cu_seqlens_k.tolist()
    for b in range(len(lq)):
        if lq[b] == 0:
            continue
        qs, ks = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        seen = M.band(lq[b], lk[b], win[0], 0 if causal else win[1], keep)
        q, k, v = (x.transpose(0, 1)[None] for x in (inp.q[qs], inp.k[ks], inp.v[ks]))
        ro, rl = _dense_ref(q, k, v, seen, 1 / math.sqrt(d))
        check(o[qs].transpose(0, 1)[None], lse[None, :, qs], ro, rl, f"sequence {b}")
    no_device_error()


PAGED = [
    # lens, Lq, Hq, Hkv, d, page, splits, dtype, window, keep, cap, sink
    ([1, 64, 700], 1, 8, 2, 128, 64, 1, "bf16", 100, 4, 0.0, False),
    ([1, 64, 700, 3000], 1, 8, 2, 128, 64, 3, "bf16", 100, 70, 0.0, True),     # two sink pages
    ([0, 17, 3000], 1, 8, 2, 128, 16, 0, "f16", 500, 40, 0.0, False),          # auto splits
    ([50, 1290], 4, 8, 2, 128, 32, 2, "bf16", 40, 1, 0.0, False),              # Lq * g = 16
    ([90, 911], 2, 4, 4, 64, 128, 4, "bf16", 0, 300, 0.0, False),
    ([4096, 130], 1, 16, 1, 128, 256, 5, "bf16", 1000, 3, 30.0, True),         # MQA, big pages
    ([600, 257, 33], 33, 8, 2, 128, 32, 0, "bf16", 100, 5, 0.0, False),        # chunked prefill
    ([1000, 129], 129, 6, 2, 64, 16, 0, "f16", 37, 200, 0.0, True),            # ... group of 3
    ([777, 400], 300, 4, 4, 128, 256, 0, "bf16", 64, 130, 0.0, False),
]


def _paged_ref(inp, win, keep, cap, d):
    page, outs = inp.page_size, []
    Lq, Hq = inp.q.shape[1], inp.q.shape[2]
    g = Hq // inp.k_pool.shape[2]
    for b, L in enumerate(inp.seqlens_k.tolist()):
        k, v = (M.paged_rows(f64(p), inp.block_table[b].tolist(), L, page).transpose(1, 0, 2)
                for p in (inp.k_pool, inp.v_pool))
        outs.append(M.attend(f64(inp.q[b]).transpose(1, 0, 2), np.repeat(k, g, 0), np.repeat(v, g, 0),
                             M.band(Lq, L, win, 0, keep), 1 / math.sqrt(d), cap,
                             None if inp.sink is None else f64(inp.sink)))
    return np.stack([o.transpose(1, 0, 2) for o, _ in outs]), np.stack([l for _, l in outs])


@gpu
@pytest.mark.parametrize("case", PAGED, ids=[str(i) for i in range(len(PAGED))])
def test_paged_with_the_hole_freed(case):
    """The pages between the first tokens and the window are taken out of the table (-1)
    and the rows behind each sequence's end hold NaN: neither is read."""
    lens, Lq, Hq, Hkv, d, page, splits, dt, win, keep, cap, sink = case
    npages = sum(-(-L // page) for L in lens) + 5
    inp = inputs.paged(lens, Lq, Hq, Hkv, d, page, npages, dtype=dt, seed=len(lens) + page + keep,
                       softcap=cap, with_sink=sink)
    ro, rl = _paged_ref(inp, win, keep, cap, d)
    bt = inp.block_table.clone()
    kp, vp = inp.k_pool.clone(), inp.v_pool.clone()
    for b, L in enumerate(lens):
        held = -(-L // page)
        if L % page:
            kp[bt[b, held - 1], L % page:] = float("nan")
            vp[bt[b, held - 1], L % page:] = float("nan")
        first = max(0, L - Lq - win) // page
        bt[b, -(-keep // page):first] = -1
        bt[b, held:] = -1
    args = (cuda(inp.q), cuda(kp), cuda(vp), cuda(bt), cuda(inp.seqlens_k))
    kw = dict(causal=True, softcap=cap, sink=cuda(inp.sink), window=(win, -1), sink_tokens=keep)
    o, lse = A.attn_fwd_paged(*args, num_splits=splits, **kw)
    torch.cuda.synchronize()
    no_device_error()
    check(o, lse, ro, rl, "paged")
    o2, lse2 = A.attn_fwd_paged_noalloc(*args, num_splits=splits, **kw)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    no_device_error()


MANY = [
    # B, longest, Lq, Hq, Hkv, d, page, dtype, window, keep, cap, sink: enough (sequence, kv head)
    # pairs for whole ones to be dealt to the SMs
    (40, 700, 1, 16, 8, 64, 16, "f16", 100, 40, 0.0, False),
    (64, 900, 1, 24, 8, 128, 64, "bf16", 256, 4, 0.0, True),
    (160, 300, 4, 8, 2, 64, 32, "bf16", 33, 1, 30.0, True),     # four queries, shorter sequences too
    (256, 200, 2, 16, 2, 64, 128, "f16", 0, 130, 0.0, False),   # 8 heads a pair, the most sequences
    (320, 90, 1, 2, 1, 64, 16, "bf16", 20, 3, 0.0, False),      # more: the other kernel
]


@gpu
@pytest.mark.parametrize("case", MANY, ids=[str(i) for i in range(len(MANY))])
def test_paged_with_many_sequences(case):
    B, most, Lq, Hq, Hkv, d, page, dt, win, keep, cap, sink = case
    rng = np.random.default_rng(B)
    lens = [0, 1, Lq, max(0, Lq - 1), most] + [int(x) for x in rng.integers(0, most + 1, B - 5)]
    npages = sum(-(-L // page) for L in lens) + 5
    inp = inputs.paged(lens, Lq, Hq, Hkv, d, page, npages, dtype=dt, seed=B + page, softcap=cap, with_sink=sink)
    ro, rl = _paged_ref(inp, win, keep, cap, d)
    bt, kp, vp = inp.block_table.clone(), inp.k_pool.clone(), inp.v_pool.clone()
    for b, L in enumerate(lens):
        held = -(-L // page)
        if L % page:
            kp[bt[b, held - 1], L % page:] = float("nan")
            vp[bt[b, held - 1], L % page:] = float("nan")
        bt[b, -(-keep // page):max(0, L - Lq - win) // page] = -1
        bt[b, held:] = -1
    args = (cuda(inp.q), cuda(kp), cuda(vp), cuda(bt), cuda(inp.seqlens_k))
    kw = dict(causal=True, softcap=cap, sink=cuda(inp.sink), window=(win, -1), sink_tokens=keep)
    o, lse = A.attn_fwd_paged(*args, **kw)
    assert ("chain" in A.attn_last_kernel_name()) == (B <= 256)
    torch.cuda.synchronize()
    no_device_error()
    check(o, lse, ro, rl, "many")
    o2, lse2 = A.attn_fwd_paged_noalloc(*args, **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o3, lse3 = A.attn_fwd_paged(*args, num_splits=2, **kw)  # the splitting kernel
    assert "decode" in A.attn_last_kernel_name()
    check(o3, lse3, ro, rl, "split")
    no_device_error()


@gpu
def test_zero_and_unbounded_are_what_they_were():
    """sink_tokens without a left bound, and 0 with one, give the bits of the call without it."""
    inp = inputs.dense(1, 4, 4, 700, 700, 128, "bf16", seed=8)
    q, k, v = cuda(inp.q), cuda(inp.k), cuda(inp.v)
    for kw in (dict(causal=True), dict(causal=True, window=(90, -1)), dict(window=(-1, 3))):
        a = A.attn_fwd(q, k, v, **kw)
        n = A.attn_last_kernel_name()
        b = A.attn_fwd(q, k, v, sink_tokens=0 if kw.get("window", (-1,))[0] >= 0 else 9, **kw)
        assert A.attn_last_kernel_name() == n
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    no_device_error()


def test_refusals_and_split_layout():
    lib = A.library()
    p, st = 1 << 12, _lib.attn_strides(1024, 512, 64)
    o = _lib.attn_opts()
    o.use_window, o.window_left, o.window_right, o.sink_tokens = 1, 8, -1, -1
    assert lib.attn_fwd(p, p, p, p, None, 1, 2, 2, 8, 8, 64, 1, st, st, st, st, ctypes.byref(o), None) == 1
    assert lib.attn_fwd_paged(p, p, p, p, p, p, None, 1, 1, 8, 2, 128, 1, 64, 4, 2, 1, None, None,
                              ctypes.byref(o), None) == 1
    W = A.attn_paged_window_pages
    assert W(1, 64, 100, window=(255, -1), sink_tokens=1) == 4 + 1 + 1
    assert W(1, 64, 100, window=(255, -1), sink_tokens=65) == 4 + 1 + 2
    assert W(1, 64, 100, sink_tokens=65) == 100
    assert W(1, 64, 6, window=(255, -1), sink_tokens=640) == 6


def test_schedule_counts_the_first_tokens():
    """The static schedule places every item once, with first tokens as without."""
    for keep in (0, 4, 300):
        s = A.attn_dense_schedule(2, 8, 4096, 4096, 100, causal=True, window=(500, -1), sink_tokens=keep)
        got = sorted(i for c in s for i in c)
        assert got == list(range(len(got))) and len(got) == 2 * 8 * 16
