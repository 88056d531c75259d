"""Rotations with a factor: `inverse` with the same factor is the transpose (the gradient), with its reciprocal the inverse.

An output is m (x c - y s) in 32 bits, rounded once.  The angle is off by 2^-23 at most at these positions (a 32-bit
argument: 2^-32 of a turn cut, 2^-25 of a half turn rounded), sincospi by 2 steps of 2^-24, the scaled c and s, the products
and the sum by four more: below 2^-21 m (|x| + |y|)."""
import pytest
import torch

import attention_forward_13_gb300 as A
from tests._parity import no_device_error
from tests.test_gpu_rope import check, rotated

pytestmark = pytest.mark.gpu


def randn(seed, dt, *shape):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda").to(dt)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scale", [1.25, 0.5, 1.3466])
@pytest.mark.parametrize("rot", [64, 30])
@pytest.mark.parametrize("interleaved", [False, True])
def test_transpose_and_inverse(interleaved, rot, scale, dt):
    x, g = randn(1, dt, 2, 3, 50, 64), randn(2, dt, 2, 3, 50, 64)
    f = A.attn_rope_freqs(rot)
    pos = torch.arange(1000, 1050, dtype=torch.int32, device="cuda")
    at = pos.expand(2, 50)[:, None]
    h = torch.finfo(dt).eps / 2
    y, _ = A.attn_rope(x, None, f, pos, interleaved=interleaved, scale=scale)
    check(y, rotated(x, at, f, interleaved, scale=scale), x)
    # <g, R x> = <R^T g, x>, with R x in 64 bits and the kernel's R^T g, rounded once
    back, _ = A.attn_rope(g, None, f, pos, interleaved=interleaved, inverse=True, scale=scale)
    check(back, rotated(g, at, f, interleaved, inverse=True, scale=scale), g)
    Rx, _ = rotated(x, at, f, interleaved, scale=scale)
    left, right = (g.double().cpu() * Rx).sum(), (back.double() * x.double()).sum().cpu()
    assert abs(left - right) <= h * 1.01 * (back.double().abs() * x.double().abs()).sum().cpu()
    # the inverse: two roundings, of y (scaled by m, at most m (|x| + |x'|)) and of the result
    z, _ = A.attn_rope(y, None, f, pos, interleaved=interleaved, inverse=True, scale=1 / scale)
    most = 2 * x.double().abs().amax()
    assert (z.double() - x.double()).abs().max() <= (2 * h + h) * 1.01 * most + 2.0 ** -20 * most
    # with the same factor the pairs come back m^2 times as long
    w, _ = A.attn_rope(y, None, f, pos, interleaved=interleaved, inverse=True, scale=scale)
    assert (w[..., :rot].double() - scale ** 2 * x[..., :rot].double()).abs().max() <= scale ** 2 * (4 * h * 1.01 + 2.0 ** -19) * most
    no_device_error()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_append_rotates_by_the_same_factor(dt):
    N, H, d, m = 37, 2, 64, 1.3466
    k, v, q = randn(3, dt, N, H, d), randn(4, dt, N, H, d), randn(5, dt, N, 4, d)
    kp, vp = torch.zeros(5, 16, H, d, dtype=dt, device="cuda"), torch.zeros(5, 16, H, d, dtype=dt, device="cuda")
    slots = (torch.randperm(80)[:N]).to(torch.int32).cuda()
    pos = torch.arange(500, 500 + N, dtype=torch.int32, device="cuda")
    f = A.attn_rope_freqs(d)
    out = A.attn_cache_append(k, v, kp, vp, slots, q=q, inv_freq=f, positions=pos, scale=m)
    wq, wk = A.attn_rope(q, k, f, pos, scale=m)
    assert torch.equal(out, wq) and torch.equal(kp.view(80, H, d)[slots.long()], wk)
    assert torch.equal(vp.view(80, H, d)[slots.long()], v)
    no_device_error()
