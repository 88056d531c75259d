"""The two 16-bit pieces of a term f v of a linear-attention state, by the kernel's steps in exact arithmetic with its
roundings: in fp16 within 2^-22 of the term and the 32-bit product's 2^-24, or 2^-36."""
import pytest
import torch


def weights(gen, n, low):
    return torch.exp2(-low * torch.rand(n, generator=gen)).float()


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
