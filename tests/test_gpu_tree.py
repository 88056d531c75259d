"""Attention for a tree of drafted tokens over the paged cache (attn_tree_mask,
attn_fwd_paged_tree) against the definition in 64 bits: node counts from one to
several query blocks, group sizes that do not divide a tile, ragged node counts,
no token before the tree, empty sequences, masks that leave a row nothing, bits
past a sequence's nodes, windows with first tokens, lengths that cut tiles and
pages anywhere.  Tolerances as in _parity.py (one output rounding plus 2e-2; LSE
1e-3)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import attention_forward_13_gb300 as A
from attention_forward_13_gb300 import _lib, inputs
from tests import _masked as M
from tests._parity import check, cuda, f64, no_device_error

gpu = pytest.mark.gpu


def random_parents(rng, B, T, reach=9):
    return torch.tensor([[-1 if i == 0 else int(rng.integers(max(-1, i - reach), i)) for i in range(T)]
                         for _ in range(B)], dtype=torch.int32).reshape(B, T)


def plain_masks(parents, lens):
    """sees [B, T, T] and depth [B, T] by walking up from every node."""
    B, T = parents.shape
    sees, depth = np.zeros((B, T, T), bool), np.zeros((B, T), int)
    for b in range(B):
        for i in range(min(T, lens[b])):
            j = i
            while j >= 0:
                sees[b, i, j] = True
                j = int(parents[b, j])
            depth[b, i] = sees[b, i].sum() - 1
    return sees, depth


def pack(sees):
    """Bits -> int32 words, node j at bit j % 32 of word j / 32."""
    B, T, N = sees.shape
    W = -(-T // 32)
    bits = np.zeros((B, T, W * 32), np.uint64)
    bits[:, :, :N] = sees
    words = (bits.reshape(B, T, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    return torch.from_numpy(words.view(np.int32).copy())


@gpu
@pytest.mark.parametrize("B,T,reach", [(1, 1, 1), (3, 2, 1), (2, 16, 4), (5, 31, 9), (2, 33, 1), (1, 64, 64),
                                       (2, 100, 5), (1, 1023, 1), (2, 1024, 20)])
def test_masks(B, T, reach):
    rng = np.random.default_rng(B * T)
    parents = random_parents(rng, B, T, reach)
    lens = [T] * B if B == 1 else [int(rng.integers(0, T + 1)) for _ in range(B)]
    mask, depth = A.attn_tree_mask(cuda(parents), cuda(torch.tensor(lens, dtype=torch.int32)))
    sees, want = plain_masks(parents, lens)
    assert torch.equal(mask.cpu(), pack(sees)) and np.array_equal(depth.cpu().numpy(), want)
    mask2, _ = A.attn_tree_mask(cuda(parents))
    assert torch.equal(mask2.cpu(), pack(plain_masks(parents, [T] * B)[0]))
    no_device_error()


@gpu
def test_bad_parents_are_reported_and_read_as_roots():
    parents = torch.tensor([[-1, 0, 2, 7, -5, 3]], dtype=torch.int32)
    mask, depth = A.attn_tree_mask(cuda(parents))
    assert A.attn_device_error() == 1 << 24
    fixed = torch.tensor([[-1, 0, -1, -1, -1, 3]], dtype=torch.int32)
    sees, want = plain_masks(fixed, [6])
    assert torch.equal(mask.cpu(), pack(sees)) and np.array_equal(depth.cpu().numpy(), want)


def reference(inp, sees, depth, lens, scale, cap=0.0, window=-1, keep=0):
    """lens: drafted nodes per sequence."""
    page, outs = inp.page_size, []
    T, Hq = inp.q.shape[1], inp.q.shape[2]
    g = Hq // inp.k_pool.shape[2]
    for b, L in enumerate(inp.seqlens_k.tolist()):
        n = min(lens[b], L)
        base = L - n
        seen = np.zeros((T, L), bool)
        j = np.arange(base)
        for i in range(n):
            seen[i, :base] = True if window < 0 else (j >= base + depth[b, i] - window) | (j < keep)
        seen[:n, base:] = sees[b, :n, :n]
        k, v = (M.paged_rows(f64(p), inp.block_table[b].tolist(), L, page).transpose(1, 0, 2)
                for p in (inp.k_pool, inp.v_pool))
        q = np.nan_to_num(f64(inp.q[b]).transpose(1, 0, 2))
        outs.append(M.attend(q, np.repeat(k, g, 0), np.repeat(v, g, 0), seen, scale, cap,
                             None if inp.sink is None else f64(inp.sink)))
    return np.stack([o.transpose(1, 0, 2) for o, _ in outs]), np.stack([l for _, l in outs])


CASES = [
    # prefix lengths, T, Hq, Hkv, d, page, dtype, ragged, cap, sink, window, keep
    ([100], 1, 1, 1, 64, 16, "bf16", False, 0.0, False, -1, 0),
    ([2000], 16, 32, 8, 128, 64, "bf16", False, 0.0, False, -1, 0),
    ([0, 5, 127, 128, 129, 700], 8, 8, 2, 128, 64, "bf16", False, 0.0, False, -1, 0),
    ([1, 300, 64], 61, 6, 2, 64, 16, "f16", False, 30.0, True, -1, 0),        # group of 3
    ([900, 40], 33, 28, 4, 128, 32, "bf16", True, 0.0, True, -1, 0),          # group of 7
    ([513, 0, 20], 64, 8, 2, 128, 64, "f16", True, 0.0, False, -1, 0),        # two query tiles
    ([333], 200, 4, 4, 64, 256, "bf16", False, 0.0, False, -1, 0),            # group of 1, two blocks
    ([70, 1500], 130, 16, 1, 128, 128, "bf16", True, 0.0, False, -1, 0),      # MQA: many blocks
    ([3000, 1, 640], 7, 8, 2, 128, 64, "bf16", False, 0.0, False, 100, 4),    # window, first tokens
    ([1000, 260, 90], 40, 8, 4, 64, 16, "f16", True, 30.0, True, 17, 200),
    ([5000], 3, 8, 8, 128, 256, "bf16", False, 0.0, False, 0, 300),
    ([4000] * 3, 90, 4, 1, 128, 32, "bf16", False, 0.0, False, 1000, 0),
    ([130] * 40 + [0] * 3, 5, 4, 2, 64, 64, "bf16", True, 0.0, True, -1, 0),  # units smaller than a share
    ([17, 4], 5, 96, 1, 64, 16, "f16", False, 0.0, False, -1, 0),             # 96 heads on one kv head
]


def build(case):
    pre, T, Hq, Hkv, d, page, dt, ragged, cap, sink, window, keep = case
    rng = np.random.default_rng(sum(pre) + T)
    B = len(pre)
    nodes = [int(rng.integers(0, T + 1)) if ragged else T for _ in range(B)]
    lens = [p + n for p, n in zip(pre, nodes)]
    npages = sum(-(-L // page) for L in lens) + 5
    inp = inputs.paged(lens, T, Hq, Hkv, d, page, npages, dtype=dt, seed=T + d + page, softcap=cap,
                       with_sink=sink)
    parents = random_parents(rng, B, T)
    sees, depth = plain_masks(parents, nodes)
    return inp, nodes, parents, sees, depth


@gpu
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_parity(case):
    """Also: rows behind the sequences hold NaN, queries of unused nodes hold NaN, and the
    table names no page the call has no business reading."""
    pre, T, Hq, Hkv, d, page, dt, ragged, cap, sink, window, keep = case
    inp, nodes, parents, sees, depth = build(case)
    ro, rl = reference(inp, sees, depth, nodes, 1 / math.sqrt(d), cap, window, keep)
    q, kp, vp, bt = inp.q.clone(), inp.k_pool.clone(), inp.v_pool.clone(), inp.block_table.clone()
    for b, L in enumerate(inp.seqlens_k.tolist()):
        held = -(-L // page)
        q[b, nodes[b]:] = float("nan")
        if L % page:
            kp[bt[b, held - 1], L % page:] = float("nan")
            vp[bt[b, held - 1], L % page:] = float("nan")
        if window >= 0:
            bt[b, -(-keep // page):max(0, L - nodes[b] - window) // page] = -1
        bt[b, held:] = -1
    tl = cuda(torch.tensor(nodes, dtype=torch.int32)) if ragged else None
    mask, dep = A.attn_tree_mask(cuda(parents), tl)
    kw = dict(tree_lens=tl, softcap=cap, sink=cuda(inp.sink), tree_depth=dep,
              window=(window, -1) if window >= 0 else None, sink_tokens=keep)
    args = (cuda(q), cuda(kp), cuda(vp), cuda(bt), cuda(inp.seqlens_k), mask)
    o, lse = A.attn_fwd_paged_tree(*args, **kw)
    torch.cuda.synchronize()
    no_device_error()
    check(o, lse, ro, rl, "tree")
    o2, lse2 = A.attn_fwd_paged_tree(*args, **kw)  # the same bits every time
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@gpu
def test_streams_strided_views_and_a_shared_workspace():
    """Two streams with a workspace each; a workspace kept from call to call; outputs given;
    the masks of one tree shape read by sequences of other lengths."""
    case = ([1500, 40, 333], 33, 8, 2, 128, 64, "bf16", False, 0.0, False, -1, 0)
    inp, nodes, parents, sees, depth = build(case)
    ro, rl = reference(inp, sees, depth, nodes, 1 / math.sqrt(128))
    args = [cuda(x) for x in (inp.q, inp.k_pool, inp.v_pool, inp.block_table, inp.seqlens_k)]
    mask, dep = A.attn_tree_mask(cuda(parents))
    need = A.attn_tree_workspace_bytes(33, 8, 2, 128)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in streams]  # NaN patterns
    torch.cuda.synchronize()
    outs = []
    for i in range(8):
        s = streams[i % 2]
        kw = dict(workspace=spaces[i % 2]) if i < 4 else {}
        outs.append(A.attn_fwd_paged_tree(*args, mask, stream=s, **kw))
    torch.cuda.synchronize()
    no_device_error()
    check(*outs[0], ro, rl, "stream")
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])
    o, lse = torch.empty_like(args[0]), torch.empty_like(outs[0][1])
    A.attn_fwd_paged_tree(*args, mask, o=o, lse=lse)
    assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])
    o, none = A.attn_fwd_paged_tree(*args, mask, lse=False)
    assert none is None and torch.equal(o, outs[0][0])
    no_device_error()


@gpu
def test_many_units_are_dealt_whole():
    """Units enough per SM for whole ones to be dealt (and far too many of them): the same
    answer as the definition, every row written."""
    for B, Hkv, T, most in ((60, 8, 5, 400), (250, 2, 3, 300), (40, 16, 70, 260)):
        rng = np.random.default_rng(B)
        case = ([int(x) for x in rng.integers(0, most, B)], T, 2 * Hkv, Hkv, 64, 32, "f16", True, 0.0, False, -1, 0)
        inp, nodes, parents, sees, depth = build(case)
        ro, rl = reference(inp, sees, depth, nodes, 1 / 8)
        tl = cuda(torch.tensor(nodes, dtype=torch.int32))
        mask, _ = A.attn_tree_mask(cuda(parents), tl)
        o = torch.full_like(cuda(inp.q), float("nan"))
        lse = torch.full((B, 2 * Hkv, T), float("nan"), device="cuda")
        A.attn_fwd_paged_tree(cuda(inp.q), cuda(inp.k_pool), cuda(inp.v_pool), cuda(inp.block_table),
                              cuda(inp.seqlens_k), mask, tree_lens=tl, o=o, lse=lse)
        torch.cuda.synchronize()
        no_device_error()
        check(o, lse, ro, rl, f"B {B}")


@gpu
@pytest.mark.parametrize("B", [257, 385, 900])  # past the order's 256, past a block's threads, past two
def test_many_sequences(B):
    rng = np.random.default_rng(B)
    case = ([int(x) for x in rng.integers(0, 200, B)], 4, 2, 1, 64, 16, "f16", True, 0.0, False, -1, 0)
    inp, nodes, parents, sees, depth = build(case)
    ro, rl = reference(inp, sees, depth, nodes, 1 / 8)
    tl = cuda(torch.tensor(nodes, dtype=torch.int32))
    mask, _ = A.attn_tree_mask(cuda(parents), tl)
    o, lse = A.attn_fwd_paged_tree(cuda(inp.q), cuda(inp.k_pool), cuda(inp.v_pool), cuda(inp.block_table),
                                   cuda(inp.seqlens_k), mask, tree_lens=tl)
    torch.cuda.synchronize()
    no_device_error()
    check(o, lse, ro, rl, f"B {B}")


@gpu
def test_pages_past_32_bits():
    """The same sequences in a small pool and at the end of one of 40000 pages (2.6e9 elements,
    5 GB each): the same bits, and the same after the pool has been closed up."""
    page, Hkv, d, num, T = 64, 8, 128, 40000, 6
    inp = inputs.paged([700, 65, 1300], T, 4 * Hkv, Hkv, d, page, 40, seed=3)
    parents = cuda(torch.tensor([[-1, 0, 0, 1, 3, 2]] * 3, dtype=torch.int32))
    mask, depth = A.attn_tree_mask(parents)
    lens = cuda(inp.seqlens_k)

    def run(kp, vp, table):
        tree = A.attn_fwd_paged_tree(cuda(inp.q), kp, vp, table, lens, mask, tree_depth=depth)
        win = A.attn_fwd_paged_tree(cuda(inp.q), kp, vp, table, lens, mask, tree_depth=depth, window=(200, -1),
                                    sink_tokens=5)
        one = A.attn_fwd_paged(cuda(inp.q[:, :1].contiguous()), kp, vp, table, lens, window=(200, -1), causal=True,
                               sink_tokens=5)
        chunk = A.attn_fwd_paged(cuda(inp.q), kp, vp, table, lens, window=(200, -1), causal=True, sink_tokens=5)
        return tree + win + one + chunk

    small = cuda(inp.k_pool), cuda(inp.v_pool)
    want = run(*small, cuda(inp.block_table))
    pools = [torch.empty(num, page, Hkv, d, dtype=inp.q.dtype, device="cuda") for _ in range(2)]
    for big, x in zip(pools, small):
        big[num - 40:] = x
    table = cuda(inp.block_table) + (num - 40)
    assert all(torch.equal(x, y) for x, y in zip(run(*pools, table), want))
    refs = torch.zeros(num, dtype=torch.int32, device="cuda")
    for row, n in zip(table.tolist(), inp.seqlens_k.tolist()):
        refs[row[:-(-n // page)]] += 1
    table, refs, _ = A.attn_cache_compact(*pools, table, lens, refs)
    assert int(table.max()) < 40
    assert all(torch.equal(x, y) for x, y in zip(run(*pools, table.clamp(min=0)), want))
    no_device_error()


@gpu
def test_bad_pages_are_reported_not_followed():
    case = ([300, 64], 4, 8, 2, 64, 64, "bf16", False, 0.0, False, -1, 0)
    inp, nodes, parents, sees, depth = build(case)
    bt = cuda(inp.block_table)
    bt[0, 2], bt[1, 0] = -7, 1 << 30
    mask, _ = A.attn_tree_mask(cuda(parents))
    o, lse = A.attn_fwd_paged_tree(cuda(inp.q), cuda(inp.k_pool), cuda(inp.v_pool), bt, cuda(inp.seqlens_k), mask)
    assert A.attn_device_error() == 1 << 22 and torch.isfinite(o.float()).all()
    sl = cuda(inp.seqlens_k).clone()
    sl[0], sl[1] = 1 << 30, -5  # lengths past the table, and below zero
    bt = cuda(inp.block_table)
    o, lse = A.attn_fwd_paged_tree(cuda(inp.q), cuda(inp.k_pool), cuda(inp.v_pool), bt, sl, mask)
    torch.cuda.synchronize()
    A.attn_device_error()
    assert not o[1].any() and torch.isneginf(lse[1]).all()


def test_refusals_before_a_launch():
    """Host-side checks of the tree entry points (no GPU needed)."""
    lib = A.library()
    p = 1 << 12

    def tree(opts=None, **k):
        a = dict(q=p, k=p, mask=p, depth=None, o=p, B=2, T=8, Hq=8, Hkv=2, d=128, dt=1, page=64, num=9, w=4,
                 ws=p, wb=1 << 30)
        a.update(k)
        o = _lib.attn_opts()
        for name, v in (opts or {}).items():
            setattr(o, name, v)
        return lib.attn_fwd_paged_tree(a["q"], a["k"], p, p, p, a["mask"], None, a["depth"], a["o"], None, a["B"],
                                       a["T"], a["Hq"], a["Hkv"], a["d"], a["dt"], a["page"], a["num"], a["w"],
                                       a["ws"], a["wb"], ctypes.byref(o), None)

    assert tree(B=0) == 0 and tree(T=0) == 0
    assert tree(Hq=9) == 1 and tree(q=None) == 1 and tree(k=p + 8) == 1 and tree(mask=p + 1) == 1
    assert tree(dt=2) == 1 and tree(d=96) == 2 and tree(page=8) == 2 and tree(T=1025) == 2
    assert tree(Hq=258, Hkv=2) == 2
    assert tree(ws=None) == 1 and tree(ws=p + 4) == 1
    need = A.attn_tree_workspace_bytes(8, 8, 2, 128)
    assert need > 0 and tree(wb=need - 1) == 1
    assert tree({"causal": 1}) == 2 and tree({"top_left": 1}) == 2 and tree({"alibi_slopes": p}) == 2
    assert tree({"bias": p}) == 2
    assert tree({"use_window": 1, "window_left": 4, "window_right": 0}, depth=p) == 2
    assert tree({"use_window": 1, "window_left": 4, "window_right": -1}) == 1     # depths are missing
    assert tree({"sink_tokens": -1}) == 1
    assert A.attn_tree_workspace_bytes(40, 8, 2, 128) > need  # two query tiles
    assert lib.attn_tree_mask(p, None, p, None, 2, 1025, None) == 2
    assert lib.attn_tree_mask(p, None, None, None, 2, 8, None) == 1
    assert lib.attn_tree_mask(p + 2, None, p, None, 2, 8, None) == 1
    assert lib.attn_tree_mask(None, None, None, None, 0, 8, None) == 0


def test_python_checks():
    q = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16)
    kp = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    bt, sl = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    mask = torch.zeros(2, 4, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        A.attn_fwd_paged_tree(q, kp.half(), kp.half(), bt, sl, mask)
    with pytest.raises(ValueError):
        A.attn_fwd_paged_tree(q, kp, kp, bt, sl.long(), mask)
    with pytest.raises(ValueError):
        A.attn_fwd_paged_tree(q, kp, kp, bt, sl, mask[:, :3])
    with pytest.raises(ValueError):
        A.attn_fwd_paged_tree(q, kp, kp, bt[:1], sl, mask)
    with pytest.raises(ValueError):
        A.attn_tree_mask(torch.zeros(2, 4))
