"""The two 16-bit pieces of a term f v of a linear-attention state, by the kernel's steps in exact arithmetic with its
roundings: within 3 h^2 of the term in bf16 (h = 2^-8: f = f1 + f2 with |f2| <= h f, rounded again: h^2; the first piece is within
h of f1 v, so that the second is at most 2 h of the term and rounded by h of that), and in fp16 within 2^-22 and the 32-bit
product's 2^-24, or 2^-36."""
import pytest
import torch


def weights(gen, n, low):
    return torch.exp2(-low * torch.rand(n, generator=gen)).float()


@pytest.mark.parametrize("low", [0.01, 1.0, 20.0])
def test_bf16(low):
    gen = torch.Generator().manual_seed(1)
    worst = 0.0
    for _ in range(40):
        f, v = weights(gen, 1 << 15, low), (1 + torch.rand(1 << 15, generator=gen)).bfloat16()
        f1 = f.bfloat16()
        f2 = (f - f1.float()).bfloat16()
        hi = (v.double() * f1.double()).bfloat16()
        rest = v.double() * f1.double() - hi.double()
        assert torch.equal(rest.bfloat16().double(), rest)  # exact
        lo = (v.double() * f2.double() + rest).bfloat16()
        term = f.double() * v.double()
        worst = max(worst, ((hi.double() + lo.double() - term).abs() / term).max().item())
    assert 2.0 ** -17 < worst <= 3 * 2.0 ** -16


@pytest.mark.parametrize("size", [3e4, 1.0, 1e-3, 1e-5, 6e-8])
@pytest.mark.parametrize("low", [0.01, 1.0, 40.0])
def test_fp16(low, size):
    gen = torch.Generator().manual_seed(2)
    for _ in range(20):
        f, v = weights(gen, 1 << 15, low), ((1 + torch.rand(1 << 15, generator=gen)) * size).half()
        hi = (v.float() * f).half()
        up = (v.float() * (f * 2048)).double() - 2048 * hi.double()
        assert torch.equal(up.float().double(), up)  # exact in 32 bits
        lo = up.half()
        assert lo.isfinite().all()
        term = f.double() * v.double()
        err = (hi.double() + lo.double() / 2048 - term).abs()
        assert (err <= (2.0 ** -22 + 2.0 ** -24) * term + 2.0 ** -36).all()
