"""Linear attention with a decay per head against the recurrence in 64 bits (tests/_linear_plain.py has the bounds)."""
import math

import pytest
import torch

import attention_forward_13_gb300 as A
from tests._linear_plain import check, with_bounds
from tests._parity import no_device_error

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def decays(H, strong=1.0):
    h = torch.arange(1, H + 1, dtype=torch.float32, device="cuda")
    return -strong * 2.0 ** (-8.0 * h / H)


def make(seed, B, L, Hq, Hkv, d, dt, state=True):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    q = randn(gen, B, Hq, L, d).to(dt)
    k, v = randn(gen, B, Hkv, L, d).to(dt), randn(gen, B, Hkv, L, d).to(dt)
    return q, k, v, (randn(gen, B, Hq, d, d) * 3 if state else None)


def plain(q, k, v, g, scale, state):
    """Per batch element: what with_bounds says."""
    r = q.shape[1] // k.shape[1]
    return [with_bounds(q[b], k[b].repeat_interleave(r, 0), v[b].repeat_interleave(r, 0), g, scale,
                        None if state is None else state[b]) for b in range(q.shape[0])]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L", [1, 2, 63, 127, 128, 129, 255, 256, 300, 641])
def test_dense(L, d, dt):
    q, k, v, state = make(L * d, 2, L, 4, 2, d, DT[dt], state=L % 2 == 1)
    g = decays(4)
    o, S = A.attn_linear_fwd(q, k, v, g, state=state)
    for b, want in enumerate(plain(q, k, v, g, 1 / math.sqrt(d), state)):
        check(o[b], S[b], want, (L, d, dt, b))
    no_device_error()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("strong", [0.0, 0.05, 8.0, 40.0, 400.0, math.inf])
@pytest.mark.parametrize("d", [64, 128])
def test_decays(strong, d, dt):
    """None, weak ones, some that leave a few tokens, and -inf: the token's own term alone."""
    q, k, v, state = make(7, 1, 333, 4, 4, d, DT[dt])
    g = decays(4, strong) if strong < math.inf else torch.full((4,), -math.inf, device="cuda")
    o, S = A.attn_linear_fwd(q, k, v, g, state=state, scale=0.37)
    check(o[0], S[0], plain(q, k, v, g, 0.37, state)[0], strong)
    if strong == math.inf:
        last = k[0, :, -1, :, None].double() * v[0, :, -1, None, :].double()
        assert (S[0].double() - last).abs().max() <= 1e-6 * last.abs().max()
    no_device_error()


def test_growing_states_within_range():
    q, k, v, state = make(8, 1, 200, 2, 2, 64, torch.bfloat16)
    g = torch.tensor([0.01, 0.002], device="cuda")
    o, S = A.attn_linear_fwd(q, k, v, g, state=state)
    # (g > 0: e^(g n) up to e^2 here; the bound's argument for the exponents' rounding holds within that factor)
    o64, S64, do, dS = plain(q, k, v, g, 0.125, state)[0]
    check(o[0], S[0], (o64, S64, 2 * do, 2 * dS))
    no_device_error()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (6, 2), (5, 5), (8, 1), (40, 8)])
def test_heads(Hq, Hkv):
    q, k, v, state = make(Hq, 1, 150, Hq, Hkv, 128, torch.bfloat16)
    g = decays(Hq)
    o, S = A.attn_linear_fwd(q, k, v, g, state=state)
    check(o[0], S[0], plain(q, k, v, g, 1 / math.sqrt(128), state)[0])
    no_device_error()


@pytest.mark.parametrize("B,L,H", [(1, 2000, 1), (1, 4111, 3), (3, 1500, 2), (2, 1025, 20)])
@pytest.mark.parametrize("dt,d", [("bf16", 128), ("f16", 64)])
def test_long(B, L, H, dt, d):
    """Few heads over long sequences: work split along the sequence."""
    q, k, v, state = make(L, B, L, H, H, d, DT[dt])
    g = decays(H, 0.25)
    o, S = A.attn_linear_fwd(q, k, v, g, state=state)
    for b, want in enumerate(plain(q, k, v, g, 1 / math.sqrt(d), state)):
        check(o[b], S[b], want, (b,))
    no_device_error()


LENS = [[5], [0], [0, 0, 0], [1, 0, 700, 128, 0, 33], [129, 64, 1, 1, 255, 900, 2], [300] * 9,
        [(37 * i * i) % 391 for i in range(30)], [i % 4 for i in range(140)], [1100] + [3] * 5]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("dt,d", [("bf16", 128), ("f16", 64), ("f16", 128)])
def test_packed(lens, dt, d):
    B, H, total = len(lens), 6, sum(lens)
    q, k, v, state = make(total + d, 1, total + 40, H, 3, d, DT[dt])
    q, k, v = (x[0].transpose(0, 1).contiguous() for x in (q, k, v))
    k[total:], v[total:], q[total:] = math.nan, math.nan, math.nan  # rows of nobody
    state = state.repeat(B, 1, 1, 1) * torch.arange(1, B + 1, device="cuda")[:, None, None, None]
    cu = torch.tensor([sum(lens[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
    g = decays(H)
    o = torch.full_like(q, 7.0)
    out, S = A.attn_linear_fwd_varlen(q, k, v, cu, max(lens), g, state=state, o=o)
    assert out is o and (o[total:] == 7.0).all()
    for b, n in enumerate(lens):
        i = int(cu[b])
        x = [t[i:i + n].transpose(0, 1)[None] for t in (q, k, v)]
        want = plain(*x, g, 1 / math.sqrt(d), state[b:b + 1])[0]
        check(o[i:i + n].transpose(0, 1), S[b], want, (b, n))
        if n == 0:
            assert torch.equal(S[b], state[b])
    no_device_error()


def test_a_sequence_does_not_see_its_neighbours():
    """NaN in one packed sequence reaches none of the others."""
    q, k, v, state = make(3, 1, 500, 2, 2, 64, torch.float16)
    q, k, v = (x[0].transpose(0, 1).contiguous() for x in (q, k, v))
    cu = torch.tensor([0, 100, 333, 500], dtype=torch.int32, device="cuda")
    g = decays(2)
    want, S = A.attn_linear_fwd_varlen(q, k, v, cu, 233, g)
    for x in (q, k, v):
        x[100:333] = math.nan
    got, T = A.attn_linear_fwd_varlen(q, k, v, cu, 233, g)
    for a, b in ((0, 100), (333, 500)):
        assert torch.equal(got[a:b], want[a:b])
    assert torch.equal(T[0], S[0]) and torch.equal(T[2], S[2])
    no_device_error()


@pytest.mark.parametrize("L", [130, 2100])
def test_strides_and_layouts(L):
    """Heads next to each other ([B,L,H,d] seen as [B,H,L,d]), slices of one projection, an o of its own strides."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    B, H, d = 2, 3, 64
    qkv = randn(gen, B, L, 3 * H, d).bfloat16()
    q, k, v = (x.transpose(1, 2) for x in qkv.split(H, 2))
    wide = torch.zeros(B, L, H, 2 * d, dtype=torch.bfloat16, device="cuda")
    g = decays(H)
    o, S = A.attn_linear_fwd(q, k, v, g, o=wide[..., d:].transpose(1, 2))
    want, T = A.attn_linear_fwd(*(x.contiguous() for x in (q, k, v)), g)
    assert torch.equal(o, want) and torch.equal(S, T) and (wide[..., :d] == 0).all()
    no_device_error()


@pytest.mark.parametrize("L", [256, 2048])
@pytest.mark.parametrize("cut", [1, 128, 200])
def test_chunks_continue_each_other(L, cut):
    """A prompt in two calls, the state carried over in place, is near the prompt in one (each within its bound)."""
    q, k, v, state = make(11, 1, L, 2, 2, 128, torch.bfloat16)
    g = decays(2)
    pool = state.clone()
    o1, p1 = A.attn_linear_fwd(*(x[:, :, :cut] for x in (q, k, v)), g, state=pool, state_out=pool)
    assert p1 is pool
    o2, _ = A.attn_linear_fwd(*(x[:, :, cut:] for x in (q, k, v)), g, state=pool, state_out=pool)
    want = plain(q, k, v, g, 1 / math.sqrt(128), state)[0]
    check(torch.cat((o1, o2), 2)[0], pool[0], want)
    no_device_error()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv", [(1, 1, 1), (3, 6, 2), (20, 16, 16), (70, 32, 8)])
def test_step(B, Hq, Hkv, d, dt):
    q, k, v, state = make(B, B, 1, Hq, Hkv, d, DT[dt])
    g = decays(Hq)
    want = plain(q, k, v, g, 0.2, state)
    S = state.clone()
    o = A.attn_linear_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], g, S, scale=0.2)
    for b in range(B):
        check(o[b][:, None], S[b], want[b], b)
    no_device_error()


def test_steps_follow_the_prompt():
    """A prompt, then token after token, is the longer prompt."""
    q, k, v, _ = make(5, 2, 140, 4, 4, 64, torch.float16, state=False)
    g = decays(4)
    o, S = A.attn_linear_fwd(*(x[:, :, :130] for x in (q, k, v)), g)
    rows = [o]
    for t in range(130, 140):
        rows.append(A.attn_linear_step(q[:, :, t], k[:, :, t], v[:, :, t], g, S)[:, :, None])
    got = torch.cat(rows, 2)
    for b, want in enumerate(plain(q, k, v, g, 0.125, None)):
        check(got[b], S[b], want)
    no_device_error()


@pytest.mark.parametrize("form", ["dense", "packed", "step"])
def test_index(form):
    """States of a pool by index: -1 starts from zero and is kept nowhere, other rows stay as they were."""
    B, H, d, L = 4, 3, 64, 1 if form == "step" else 150
    q, k, v, _ = make(21, B, L, H, H, d, torch.bfloat16)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    pool = randn(gen, 7, H, d, d)
    before = pool.clone()
    index = torch.tensor([5, -1, 0, 6], dtype=torch.int32, device="cuda")
    g = decays(H)
    start = torch.stack([before[i] if i >= 0 else torch.zeros_like(before[0]) for i in index.tolist()])
    want = plain(q, k, v, g, 0.125, start)
    o = run_form(form, q, k, v, g, pool, index)
    for b, i in enumerate(index.tolist()):
        check(o[b], pool[i] if i >= 0 else None, want[b], b)
    for i in (1, 2, 3, 4):
        assert torch.equal(pool[i], before[i])
    no_device_error()


def run_form(form, q, k, v, g, pool, index):
    B, H, L, d = q.shape
    if form == "dense":
        o, out = A.attn_linear_fwd(q, k, v, g, state=pool, state_index=index)
        assert out is pool
        return o
    if form == "step":
        return A.attn_linear_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], g, pool, state_index=index)[:, :, None]
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * L
    flat = [x.transpose(1, 2).reshape(B * L, -1, d).contiguous() for x in (q, k, v)]
    o, out = A.attn_linear_fwd_varlen(*flat, cu, L, g, state=pool, state_index=index)
    assert out is pool
    return o.view(B, L, H, d).transpose(1, 2)


@pytest.mark.parametrize("form", ["dense", "packed", "step"])
@pytest.mark.parametrize("index", [[2, 7], [2, -2], [2, 2], [2, 1 << 30]])
def test_bad_index(form, index):
    """Out of range, or named twice: the row is run from zero, kept nowhere, and reported."""
    L = 1 if form == "step" else 131
    q, k, v, _ = make(22, 2, L, 2, 2, 64, torch.float16)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(10)
    pool = randn(gen, 7, 2, 64, 64)
    before = pool.clone()
    g = decays(2)
    want = plain(q, k, v, g, 0.125, torch.stack((before[2], torch.zeros_like(before[0]))))
    o = run_form(form, q, k, v, g, pool, torch.tensor(index, dtype=torch.int32, device="cuda"))
    check(o[0], pool[2], want[0])
    check(o[1], None, want[1])
    for i in (0, 1, 3, 4, 5, 6):
        assert torch.equal(pool[i], before[i])
    assert A.attn_device_error() == 1 << 25


def test_no_state_kept():
    q, k, v, state = make(30, 1, 260, 2, 2, 64, torch.bfloat16)
    g = decays(2)
    o, S = A.attn_linear_fwd(q, k, v, g, state=state, state_out=False)
    want, _ = A.attn_linear_fwd(q, k, v, g, state=state)
    assert S is None and torch.equal(o, want)
    no_device_error()


@pytest.mark.parametrize("L,H", [(700, 3), (2300, 2)])
def test_same_every_time(L, H):
    q, k, v, state = make(31, 2, L, H, H, 128, torch.bfloat16)
    g = decays(H)
    first = A.attn_linear_fwd(q, k, v, g, state=state)
    for _ in range(5):
        again = A.attn_linear_fwd(q, k, v, g, state=state)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    no_device_error()


def test_empty():
    q, k, v, state = make(32, 2, 0, 2, 2, 64, torch.bfloat16)
    g = decays(2)
    o, S = A.attn_linear_fwd(q, k, v, g, state=state)
    assert o.shape == (2, 2, 0, 64) and torch.equal(S, state)
    _, S = A.attn_linear_fwd(q, k, v, g)
    assert not S.any()
    o, S = A.attn_linear_fwd(q[:0], k[:0], v[:0], g)
    assert S.shape == (0, 2, 64, 64)
    no_device_error()


@pytest.mark.parametrize("size_q,size_v,g", [(60.0, 1e-3, 0.01), (0.002, 1e-2, 0.3), (15.0, 30.0, 1.0), (1.0, 200.0, 0.0)])
def test_fp16_ranges(size_q, size_v, g):
    """Weights and states far above and below what fp16 holds, where o itself fits it: scores up to 10^6, states up to
    10^5 (no decay, keys and values that agree)."""
    q, k, v, _ = make(41, 1, 700, 2, 2, 128, torch.float16, state=False)
    q, k, v = q * size_q, k.abs() * size_q, v.abs() * size_v
    g = torch.full((2,), -g, device="cuda")
    o64, S64, do, dS = plain(q, k, v, g, 1.0, None)[0]
    most = float(o64.abs().max())
    scale = min(1.0, 2e4 / most) if size_q > 50 else 100.0 / most
    o, S = A.attn_linear_fwd(q, k, v, g, scale=scale)
    check(o[0], S[0], plain(q, k, v, g, scale, None)[0])
    if size_q > 50:
        assert torch.matmul(q[0].float(), k[0].float().transpose(1, 2)).abs().max() * scale > 65504
    if size_v == 200.0:
        assert S.abs().max() > 65504
    no_device_error()


def test_index_without_states():
    """Nothing to look up: the index says nothing."""
    q, k, v, _ = make(42, 2, 140, 2, 2, 64, torch.bfloat16, state=False)
    g = decays(2)
    o, S = A.attn_linear_fwd(q, k, v, g, state_out=False, state_index=torch.tensor([9, 9], dtype=torch.int32, device="cuda"))
    want, _ = A.attn_linear_fwd(q, k, v, g)
    assert S is None and torch.equal(o, want)
    no_device_error()


@pytest.mark.parametrize("form", ["dense", "step"])
def test_outputs_over_inputs_refused(form):
    q, k, v, state = make(43, 2, 1 if form == "step" else 140, 2, 2, 64, torch.bfloat16)
    g = decays(2)
    for x in (q, k, v):
        with pytest.raises(A.AttnError):
            if form == "dense":
                A.attn_linear_fwd(q, k, v, g, o=x)
            else:
                A.attn_linear_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], g, state, o=x[:, :, 0])
    no_device_error()


def test_packed_without_rows():
    """No rows at all: the states are handed on."""
    e = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    state = torch.randn(3, 2, 64, 64, device="cuda")
    o, S = A.attn_linear_fwd_varlen(e, e, e, cu, 0, decays(2), state=state)
    assert o.shape == e.shape and torch.equal(S, state)
    no_device_error()


def test_lengths_past_the_given_most():
    """max_seqlen below a sequence's length costs balance, not results; cu_seqlens past the rows are cut there."""
    q, k, v, _ = make(44, 1, 1500, 2, 2, 64, torch.bfloat16, state=False)
    q, k, v = (x[0].transpose(0, 1).contiguous() for x in (q, k, v))
    g = decays(2)
    cu = torch.tensor([0, 1500], dtype=torch.int32, device="cuda")
    want, S = A.attn_linear_fwd_varlen(q, k, v, cu, 1500, g)
    for most, ends in ((600, [0, 1500]), (1500, [0, 1 << 30]), (2000, [0, 1500, 1499])):
        c = torch.tensor(ends, dtype=torch.int32, device="cuda")
        o, T = A.attn_linear_fwd_varlen(q, k, v, c, most, g)
        x = [t.transpose(0, 1)[None] for t in (q, k, v)]
        check(o.transpose(0, 1), T[0], plain(*x, g, 0.125, None)[0], (most, ends))
        if len(ends) == 3:
            assert not T[1].any()
    no_device_error()
