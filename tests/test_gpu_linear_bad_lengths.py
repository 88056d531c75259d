"""Packed linear attention with cu_seqlens that no batch has: whatever the entries, no row outside the packed tensors is
read or written, and a sequence without a valid range has no tokens."""
import pytest
import torch

import attention_forward_13_gb300 as A
from tests._parity import no_device_error

LOW, HIGH = -2 ** 31, 2 ** 31 - 1


def rows_of(first, last, total):
    """A sequence's range by the rules, in numbers without a width."""
    return (0, 0) if first < 0 or last <= first or first >= total else (first, min(last, total))


def wrapped(x):
    return (x + 2 ** 31) % 2 ** 32 - 2 ** 31


def test_the_difference_of_two_ints_may_not_be_taken_first():
    """Where the end is far below the start, end - start wraps round to a long sequence."""
    assert wrapped(min(LOW, 300) - 1) == HIGH and rows_of(1, LOW, 300) == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("cu", [[1, LOW], [200, LOW], [200, LOW + 100, 130], [LOW, HIGH], [0, HIGH], [299, HIGH, LOW],
                                [300, 400], [-5, 100, 40], [HIGH, LOW, 300]], ids=str)
def test_wrong_ranges(cu, dt):
    B, H, d, total = len(cu) - 1, 2, 64, 300
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    q, k, v = (torch.randn(total, H, d, generator=gen, device="cuda").to(dt) for _ in range(3))
    state = torch.randn(B, H, d, d, generator=gen, device="cuda")
    g = torch.tensor([-0.3, -0.01], device="cuda")
    room = torch.full((3 * total, H, d), 7.0, dtype=dt, device="cuda")  # rows before and behind those of the call
    o, S = A.attn_linear_fwd_varlen(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), total, g, state=state,
                                    o=room[total:2 * total])
    kept = torch.ones(total, dtype=torch.bool, device="cuda")
    for b in range(B):
        first, last = rows_of(cu[b], cu[b + 1], total)
        if first == last:
            assert torch.equal(S[b], state[b])
            continue
        kept[first:last] = False
        x = [t[first:last].transpose(0, 1)[None] for t in (q, k, v)]
        want, T = A.attn_linear_fwd(*x, g, state=state[b:b + 1])
        assert (o[first:last].float() - want[0].transpose(0, 1).float()).abs().max() <= 0.02 * want.abs().max()
        assert (S[b] - T[0]).norm() <= 1e-5 * T.norm()
    assert (o[kept] == 7.0).all() and (room[:total] == 7.0).all() and (room[2 * total:] == 7.0).all()
    no_device_error()
