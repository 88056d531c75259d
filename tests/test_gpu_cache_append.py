"""Slot maps and the write into the pages: integers and moved rows have to be equal, rotated ones what attn_rope gives."""
import random

import pytest
import torch

import attention_forward_13_gb300 as A
from tests._parity import no_device_error

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def slots_plain(table, lens, add, N, page):
    slots, positions, seq, cu = [], [], [], [0]
    for b, (n, m) in enumerate(zip(lens, add)):
        for p in range(n - m, n):
            slots.append(table[b][p // page] * page + p % page)
            positions.append(p)
            seq.append(b)
        cu.append(cu[-1] + m)
    rest = N - len(slots)
    return [slots + [-1] * rest, positions + [0] * rest, cu, seq + [-1] * rest]


def state(seed, B, page, hi, most, pad=0):
    rng = random.Random(seed)
    add = [rng.choice([0, 1, rng.randint(0, most)]) for _ in range(B)]
    lens = [rng.randint(0, hi) + m for m in add]
    width = max([1] + [-(-n // page) for n in lens])
    pages = sum(-(-n // page) for n in lens) + 5
    order = list(range(pages))
    rng.shuffle(order)
    table = []
    for n in lens:
        held = -(-n // page)
        table.append([order.pop() for _ in range(held)] + [-7] * (width - held))
    return table, lens, add, sum(add) + pad, pages


@pytest.mark.parametrize("B,page,hi,most,pad", [(1, 16, 0, 1, 0), (1, 64, 5, 3000, 9), (7, 16, 100, 40, 0), (64, 64, 900, 1, 0),
                                                (300, 32, 50, 60, 500), (1000, 128, 300, 9, 1), (8192, 16, 3, 2, 77),
                                                (513, 256, 600, 300, 0)])
def test_slots(B, page, hi, most, pad):
    table, lens, add, N, pages = state(B + page, B, page, hi, most, pad)
    got = A.attn_cache_slots(i32(table), i32(lens), i32(add), N, page, pages)
    for name, g, w in zip(("slots", "positions", "cu", "sequence"), got, slots_plain(table, lens, add, N, page)):
        assert g.tolist() == w, name
    no_device_error()


def test_no_new_tokens_and_no_sequences():
    got = A.attn_cache_slots(i32([[0], [1]]), i32([3, 4]), i32([0, 0]), 3, 16, 2)
    assert [x.tolist() for x in got] == [[-1] * 3, [0] * 3, [0] * 3, [-1] * 3]
    got = A.attn_cache_slots(i32([[0], [1]]), i32([3, 4]), i32([0, 0]), 0, 16, 2)
    assert got[2].tolist() == [0, 0, 0] and got[0].numel() == 0
    got = A.attn_cache_slots(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), i32([]), i32([]), 2, 16, 2)
    assert [x.tolist() for x in got] == [[-1] * 2, [0] * 2, [0], [-1] * 2]
    no_device_error()


@pytest.mark.parametrize("table,lens,add,N,slots,cu", [
    ([[0], [1]], [3, 4], [-2, 2], 4, [18, 19, -1, -1], [0, 0, 2]),                 # a negative count
    ([[0], [1]], [3, 4], [3, 4], 5, [0, 1, 2, 16, 17], [0, 3, 5]),                 # more than there is room for
    ([[0], [9]], [3, 4], [1, 2], 3, [2, -1, -1], [0, 1, 3]),                       # a page outside the pool
    ([[0], [-1]], [3, 4], [1, 2], 3, [2, -1, -1], [0, 1, 3]),
    ([[0], [1]], [3, 18], [1, 4], 5, [2, 30, 31, -1, -1], [0, 1, 5]),              # past the table's row
    ([[0], [1]], [2, 4], [3, 1], 4, [-1, 0, 1, 19], [0, 3, 4]),                    # more new tokens than tokens
    ([[0], [1]], [3, 4], [2 ** 31 - 1, 2 ** 31 - 1], 2, [-1, -1], [0, 2, 2]),      # counts whose sum leaves 32 bits
    ([[0], [1]], [-2 ** 31, 4], [1, 1], 2, [-1, 19], [0, 1, 2])])
def test_bad_entries_are_left_out_and_reported(table, lens, add, N, slots, cu):
    got = A.attn_cache_slots(i32(table), i32(lens), i32(add), N, 16, 2)
    assert got[0].tolist() == slots and got[2].tolist() == cu
    assert A.attn_device_error() == 1 << 25


DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,Hq,Hkv,page,n", [(128, 128, 32, 8, 64, 64), (64, 32, 6, 2, 16, 300), (64, 0, 4, 4, 32, 77),
                                                 (64, 22, 3, 1, 16, 130), (128, 128, 0, 2, 256, 9), (96, 48, 5, 5, 128, 1),
                                                 (80, 6, 10, 2, 16, 501)])
def test_append(d, rot, Hq, Hkv, page, n, interleaved, dt):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n)
    pages = 2 * n // page + 3
    qkv = torch.randn(n, Hq + 2 * Hkv, d, generator=gen, device="cuda").to(DT[dt])
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    kp, vp = (torch.randn(pages, page, Hkv, d, generator=gen, device="cuda").to(DT[dt]) for _ in range(2))
    slots = torch.randperm(pages * page, generator=gen, device="cuda")[:n].to(torch.int32)
    slots[::7] = -1  # padding
    pos = torch.randint(0, 1 << 20, (n,), generator=gen, device="cuda").to(torch.int32)
    f = A.attn_rope_freqs(rot) if rot else None
    qr, kr = q.contiguous(), k.contiguous()
    if rot:
        kr, _ = A.attn_rope(kr, None, f, pos, interleaved=interleaved, scale=0.9)
        if Hq:
            qr, _ = A.attn_rope(qr, None, f, pos, interleaved=interleaved, scale=0.9)
    want = [kp.clone(), vp.clone()]
    at = slots.long()
    for pool, rows in zip(want, (kr, v)):
        pool.view(-1, Hkv, d)[at[at >= 0]] = rows[at >= 0]
    out = A.attn_cache_append(k, v, kp, vp, slots, q=q if Hq else None, inv_freq=f, positions=pos, interleaved=interleaved,
                              scale=0.9)
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    assert out is None if not Hq else torch.equal(out, qr)
    if Hq:  # and in place
        out = A.attn_cache_append(k, v, kp, vp, slots, q=q, inv_freq=f, positions=pos, interleaved=interleaved, scale=0.9,
                                  q_out=q)
        assert out is q and torch.equal(q, qr) and torch.equal(kp, want[0])
    no_device_error()


@pytest.mark.parametrize("rot", [64, 10])
def test_slots_outside_the_pool_are_reported(rot):
    kp, vp = torch.zeros(2, 16, 1, 64, device="cuda").half(), torch.zeros(2, 16, 1, 64, device="cuda").half()
    k = torch.ones(5, 1, 64, device="cuda").half()
    A.attn_cache_append(k, k, kp, vp, i32([0, 32, -2, 31, 2 ** 31 - 1]), inv_freq=A.attn_rope_freqs(rot), positions=i32([0] * 5))
    assert vp.view(32, 64).sum(1).nonzero().view(-1).tolist() == [0, 31]
    assert A.attn_device_error() == 1 << 25


def test_long_pools():
    """Rows past 32 bits of elements."""
    pages, page, H, d = 70000, 64, 8, 64  # 2.3e9 elements a pool
    kp = torch.zeros(pages, page, H, d, dtype=torch.float16, device="cuda")
    vp = torch.zeros_like(kp)
    k = torch.randn(3, H, d, device="cuda").half()
    slots = [5, pages * page - 1, pages * page // 2]
    A.attn_cache_append(k, -k, kp, vp, i32(slots))
    for i, s in enumerate(slots):
        assert torch.equal(kp.view(-1, H, d)[s], k[i]) and torch.equal(vp.view(-1, H, d)[s], -k[i])
    assert int((kp != 0).sum()) == int((k != 0).sum())
    no_device_error()
