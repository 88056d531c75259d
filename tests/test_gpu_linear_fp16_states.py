"""fp16 states keep their bits whatever the size of v: against the recurrence in 64 bits, within bounds in proportion to the
inputs (tests/_linear_bounds.py), and as a whole."""
import math

import pytest
import torch

import attention_forward_13_gb300 as A
from tests._linear_bounds import bounds, check, piece
from tests._parity import no_device_error

pytestmark = pytest.mark.gpu


def make(seed, H, L, d, size, dt=torch.float16):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    q, k, v = (torch.randn(1, H, L, d, generator=gen, device="cuda") for _ in range(3))
    return q.to(dt), k.to(dt), (v * size).to(dt)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L", [1, 77, 128, 300, 1100])
@pytest.mark.parametrize("size", [1e4, 100.0, 1.0, 1e-2, 1e-3, 1e-4, 1e-5])
def test_states_of_small_and_large_values(size, L, d):
    """Every term by itself is within 2^-21 of it and 2^-36 of |k|, so for v ~ 10^-4 the whole state within 2^-19."""
    q, k, v = make(L + d, 2, L, d, size)
    g = torch.tensor([-0.01, -0.3], device="cuda")
    scale = 1 / math.sqrt(d) * (1e-4 if size > 1e3 else 1.0)
    want = bounds(q[0], k[0], v[0], g, scale, piece=piece(1, 2, L, d))
    o, S = A.attn_linear_fwd(q, k, v, g, scale=scale)
    check(o[0], S[0], want, (size, L, d))
    # Signs are random: the roundings of sums and pieces are some 2^-22 of the norm, and 2^-36 |k| against |v k| some 2^-22
    # where v is 10^-4 (2^-13.3), but the last token alone stands against a whole piece's where the decay is e^-0.3: 2^-19.
    if size >= 1e-4:
        rel = ((S[0].double() - want[1]).norm() / want[1].norm()).item()
        assert rel <= 2.0 ** -19, rel
    no_device_error()


@pytest.mark.parametrize("size", [1e4, 1.0, 1e-3])
def test_old_tokens_count_where_the_new_have_no_keys(size):
    """The last 100 tokens' keys are 0: what is left are terms of weight e^(-100 g) and less."""
    q, k, v = make(3, 3, 128, 64, size)
    k[:, :, 28:] = 0
    g = torch.tensor([-0.05, -0.1, -0.2], device="cuda")
    scale = 0.125 * min(1.0, 1 / size)
    want = bounds(q[0], k[0], v[0], g, scale)
    o, S = A.attn_linear_fwd(q, k, v, g, scale=scale)
    check(o[0], S[0], want, size)
    rel = (S[0].double() - want[1]).norm(dim=(1, 2)) / want[1].norm(dim=(1, 2))
    assert (rel <= 2.0 ** -32 / (size * torch.exp(100 * g.double())) + 2.0 ** -20).all(), rel
    no_device_error()


@pytest.mark.parametrize("size_q,size_v,g", [(60.0, 1e-3, 0.01), (0.002, 1e-2, 0.3), (15.0, 30.0, 1.0), (1.0, 200.0, 0.0)])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_ranges(dt, size_q, size_v, g):
    """Scores up to 10^6 and states from 10^-5 to 10^5, within bounds in proportion to them."""
    q, k, v = make(41, 2, 700, 128, size_v, dt)
    q, k, v = q * size_q, k.abs() * size_q, v.abs()
    g = torch.full((2,), -g, device="cuda")
    most = float(bounds(q[0], k[0], v[0], g, 1.0)[0].abs().max())
    scale = min(1.0, 2e4 / most) if size_q > 50 else 100.0 / most
    o, S = A.attn_linear_fwd(q, k, v, g, scale=scale)
    check(o[0], S[0], bounds(q[0], k[0], v[0], g, scale, piece=piece(1, 2, 700, 128)), (size_q, size_v))
    no_device_error()
