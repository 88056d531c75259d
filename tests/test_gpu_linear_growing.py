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
