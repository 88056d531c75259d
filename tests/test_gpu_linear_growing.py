"""Linear attention with decays above 1 (log_decay > 0), as long as e^(128 g) and the results fit: against the recurrence
in 64 bits (tests/_linear_bounds.py has the bounds)."""
import math

import pytest
import torch

import attention_forward_13_gb300 as A
from tests._linear_bounds import bounds, check
from tests._parity import no_device_error

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def make(seed, H, L, d, dt, state=False):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    q, k, v = (torch.randn(1, H, L, d, generator=gen, device="cuda").to(dt) for _ in range(3))
    return q, k, v, torch.randn(1, H, d, d, generator=gen, device="cuda") if state else None


def run(q, k, v, g, state=None, states=True, most=2e4):
    """The call with a scale that keeps o below `most`, and what it should give."""
    o1 = bounds(q[0], k[0], v[0], g, 1.0, None if state is None else state[0])[0]
    scale = 2.0 ** math.floor(math.log2(most / float(o1.abs().max())))
    want = bounds(q[0], k[0], v[0], g, scale, None if state is None else state[0])
    o, S = A.attn_linear_fwd(q, k, v, g, state=state, state_out=states, scale=scale)
    return o[0], None if S is None else S[0], want


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L", [3, 40, 97, 128])
@pytest.mark.parametrize("g", [0.03, 0.05, 0.08, 0.3])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_weights_of_a_chunk(dt, g, L, d):
    """e^(g (i - j)) makes the weights of far tokens any multiple of their scores."""
    q, k, v, _ = make(L + d, 2, L, d, DT[dt])
    o, _, want = run(q, k, v, torch.tensor([g, g / 2], device="cuda"), states=False)
    check(o, None, want, (dt, g, L, d))
    no_device_error()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L", [1, 40, 128, 129, 300, 384])
@pytest.mark.parametrize("g", [0.01, 0.05, 0.08])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_states(dt, g, L, d):
    """Over several chunks, from a state and from none, and from chunk to chunk in place."""
    q, k, v, state = make(L + d, 2, L, d, DT[dt], state=True)
    g = torch.tensor([g, -0.02], device="cuda")
    for s in (state, None):
        o, S, want = run(q, k, v, g, s)
        check(o, S, want, (dt, L, d))
    no_device_error()


def test_the_first_tokens_are_padding():
    """Zeros at the front, which the largest weights meet."""
    q, k, v, _ = make(5, 2, 300, 64, torch.float16)
    for x in (k, v):
        x[:, :, :120] = 0
    o, S, want = run(q, k, v, torch.tensor([0.05, 0.1], device="cuda"))
    check(o, S, want)
    no_device_error()


def split(B, H, L, d):
    """Whether the call is cut into pieces along the sequence."""
    return A.attn_linear_workspace_bytes(B, H, L, B * L, d) > 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L", [700, 1200, 2050])
@pytest.mark.parametrize("g", [0.002, 0.01, 0.02])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_cut_sequences(dt, g, L, d):
    """Pieces of 256 tokens and more, whose states are summed up first."""
    assert split(1, 2, L, d)
    q, k, v, state = make(L + d, 2, L, d, DT[dt], state=True)
    g = torch.tensor([g, g / 3], device="cuda")
    for s in (state, None):
        o, S, want = run(q, k, v, g, s)
        check(o, S, want, (dt, g, L, d))
    no_device_error()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_cut_sequences_whose_first_tokens_are_padding(dt):
    """e^(g n) of a whole piece is past fp32's range, the results are not: there is nothing at the front for it to multiply."""
    H, L, d, g = 2, 8192, 64, 0.3
    assert A.attn_linear_workspace_bytes(1, H, L, L, d) == 16 * H * d * d * 4 and L // 16 * 0.25 > math.log(3.4e38) > g * 128
    q, k, v, _ = make(9, H, L, d, DT[dt])
    for x in (k, v):
        x[:, :, :L - 100] = 0
    o, S, want = run(q, k, v, torch.tensor([g, 0.25], device="cuda"))
    check(o, S, want, dt)
    no_device_error()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_cut_in_place_and_packed(dt):
    """A pool's states in place, short sequences beside a cut one, decays on both sides of 1."""
    lens, H, d = [5, 1500, 130], 2, 128
    total = sum(lens)
    q, k, v, _ = make(13, H, total, d, DT[dt])
    q, k, v = (x[0].transpose(0, 1).contiguous() for x in (q, k, v))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(14)
    pool = torch.randn(6, H, d, d, generator=gen, device="cuda")
    before, index = pool.clone(), [4, 0, 5]
    g = torch.tensor([0.01, -0.01], device="cuda")
    cu = torch.tensor([0, 5, 1505, 1635], dtype=torch.int32, device="cuda")
    parts = [[x[cu[b]:cu[b + 1]].transpose(0, 1) for x in (q, k, v)] for b in range(3)]
    most = max(float(bounds(*x, g, 1.0, before[i])[0].abs().max()) for x, i in zip(parts, index))
    scale = 2.0 ** math.floor(math.log2(2e4 / most))
    o, _ = A.attn_linear_fwd_varlen(q, k, v, cu, 1500, g, state=pool, scale=scale,
                                    state_index=torch.tensor(index, dtype=torch.int32, device="cuda"))
    for b, i in enumerate(index):
        check(o[cu[b]:cu[b + 1]].transpose(0, 1), pool[i], bounds(*parts[b], g, scale, before[i], piece=384), (dt, b))
    for i in (1, 2, 3):
        assert torch.equal(pool[i], before[i])
    no_device_error()
