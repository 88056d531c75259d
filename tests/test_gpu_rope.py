"""Rotary positions against complex products in 64 bits.  An output is x c - y s in 32 bits, rounded once: half a step
of the type relative to it, and 2^-21 (|x| + |y|) for the angle (its fixed-point form cut to 32 bits of a turn: 2^-31 of a half
turn, times pi), sincospi's error (2 steps) and three roundings."""
import math

import pytest
import torch

import attention_forward_13_gb300 as A
from tests._parity import no_device_error

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def rotated(x, pos, f, interleaved, inverse=False, scale=1.0):
    """x [..., d], pos broadcastable to x's leading dimensions.  fp64 (values, most error before the output's rounding)."""
    y = x.double().cpu()
    r = 2 * f.numel()
    head = y[..., :r].unflatten(-1, (r // 2, 2)) if interleaved else torch.stack((y[..., :r // 2], y[..., r // 2:r]), -1)
    a = pos.double().cpu()[..., None] * f.cpu() * (-1.0 if inverse else 1.0)
    c, s = torch.cos(a) * scale, torch.sin(a) * scale
    z = torch.stack((head[..., 0] * c - head[..., 1] * s, head[..., 1] * c + head[..., 0] * s), -1)
    m = (head.abs().sum(-1, keepdim=True) * abs(scale)).expand(z.shape)
    join = (lambda t: t.flatten(-2)) if interleaved else (lambda t: torch.cat((t[..., 0], t[..., 1]), -1))
    return torch.cat((join(z), y[..., r:]), -1), torch.cat((join(m), torch.zeros_like(y[..., r:])), -1)


def check(got, want, x):
    v, m = want
    eps = torch.finfo(x.dtype).eps / 2
    tiny = torch.finfo(x.dtype).smallest_normal * eps
    err = (got.double().cpu() - v).abs()
    assert (err <= eps * v.abs() + 2.0 ** -21 * m * (1 + eps) + tiny * (m > 0)).all(), err.max()


def dense(B, H, L, d, dt, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(B, H, L, d, generator=gen, device="cuda").to(dt)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (128, 32), (64, 48), (64, 2), (80, 20), (96, 50), (128, 126), (8, 8),
                                   (512, 512), (512, 510), (24, 16), (64, 0)])
def test_dense(d, rot, interleaved, dt):
    B, L = 2, 37
    q, k = dense(B, 5, L, d, DT[dt]), dense(B, 2, L, d, DT[dt], 1)
    f = A.attn_rope_freqs(rot) if rot else torch.zeros(0, dtype=torch.float64, device="cuda")
    pos = torch.arange(L, dtype=torch.int32, device="cuda")
    for given, p in ((None, pos.expand(B, L)), (pos * 3 + 5, (pos * 3 + 5).expand(B, L)),
                     (torch.stack((pos, 900 - pos)), torch.stack((pos, 900 - pos)))):
        qo, ko = A.attn_rope(q, k, f, given, interleaved=interleaved, scale=1.0 if given is None else 1.25)
        for x, y in ((q, qo), (k, ko)):
            check(y, rotated(x, p[:, None], f, interleaved, scale=1.0 if given is None else 1.25), x)
            assert torch.equal(y[..., rot:], x[..., rot:])
    no_device_error()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [64, 34])
@pytest.mark.parametrize("far", [10 ** 6, 2 ** 30, 2 ** 31 - 100, -5, -2 ** 31])
def test_far_positions(far, rot, interleaved):
    """Angles keep their accuracy wherever the position lies (the fp64 angle itself is within 2^-53 * 2^31 of a turn)."""
    q = dense(1, 3, 64, 64, torch.float16)
    pos = (torch.arange(64) + far).to(torch.int32).cuda()
    f = A.attn_rope_freqs(rot)
    qo, none = A.attn_rope(q, None, f, pos, interleaved=interleaved)
    assert none is None
    check(qo, rotated(q, pos[None, None], f, interleaved), q)
    no_device_error()


@pytest.mark.parametrize("rot", [64, 30])
@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse(rot, interleaved):
    """Turning back: the transpose of the rotation, which is its gradient, and (to two roundings) the input again."""
    x = dense(2, 3, 50, 64, torch.bfloat16)
    f = A.attn_rope_freqs(rot)
    pos = torch.arange(1000, 1050, dtype=torch.int32, device="cuda")
    y, _ = A.attn_rope(x, None, f, pos, interleaved=interleaved)
    z, _ = A.attn_rope(y, None, f, pos, interleaved=interleaved, inverse=True)
    check(z, rotated(y, pos.expand(2, 50)[:, None], f, interleaved, inverse=True), y)
    h = torch.finfo(torch.bfloat16).eps / 2
    pairs = x.double().abs().amax()
    assert (z.double() - x.double()).abs().max() <= (2 * h * math.sqrt(2) + h) * 2 * pairs
    # The gradient against differences, in 64 bits through the tested formula: <g, R x> = <R^T g, x>.
    g = dense(2, 3, 50, 64, torch.bfloat16, 5)
    back, _ = A.attn_rope(g, None, f, pos, interleaved=interleaved, inverse=True)
    Rx, _ = rotated(x, pos.expand(2, 50)[:, None], f, interleaved)
    left, right = (g.double().cpu() * Rx).sum(), (back.double() * x.double()).sum().cpu()
    assert abs(left - right) <= h * 1.01 * (back.double().abs() * x.double().abs()).sum().cpu()
    no_device_error()


@pytest.mark.parametrize("rot", [64, 32, 18])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n", [1, 2, 300])
def test_packed_in_place_and_slices(n, interleaved, rot):
    """Rows of one projection's output, rotated where they stand; what lies beside them stays."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n)
    qkv = torch.randn(n, 9, 64, generator=gen, device="cuda").bfloat16()
    before = qkv.clone()
    q, k, v = qkv.split([5, 2, 2], 1)
    pos = torch.randint(0, 5000, (n,), generator=gen, device="cuda").to(torch.int32)
    f = A.attn_rope_freqs(rot)
    want = A.attn_rope(q.contiguous(), k.contiguous(), f, pos, interleaved=interleaved)
    got = A.attn_rope(q, k, f, pos, interleaved=interleaved, q_out=q, k_out=k)
    assert got[0] is q and all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(v, before[:, 7:])
    check(want[0], rotated(before[:, :5], pos[:, None].expand(n, 5), f, interleaved), q)
    no_device_error()


def test_relative_positions():
    """q . k depends on the difference of the positions alone, near and far (within the two roundings)."""
    q, k = dense(1, 1, 1, 128, torch.float16), dense(1, 1, 1, 128, torch.float16, 1)
    f = A.attn_rope_freqs(128)
    at = lambda a: torch.tensor([a], dtype=torch.int32, device="cuda")  # noqa: E731
    dots = []
    for base in (0, 17, 10 ** 6, 2 * 10 ** 9):
        a, _ = A.attn_rope(q, None, f, at(base + 40))
        b, _ = A.attn_rope(k, None, f, at(base))
        dots.append((a.double() * b.double()).sum().item())
    most = 2 * 2.0 ** -11 * (q.double().norm() * k.double().norm()).item() * 1.5
    assert max(dots) - min(dots) <= 2 * most
    no_device_error()


@pytest.mark.parametrize("L,H", [(1, 1), (1, 300), (5000, 3), (257, 64)])
def test_sizes(L, H):
    q = dense(1, H, L, 64, torch.bfloat16)
    f = A.attn_rope_freqs(64)
    y, _ = A.attn_rope(q, None, f)
    check(y, rotated(q, torch.arange(L)[None, None], f, False), q)
    no_device_error()


def test_empty():
    f = A.attn_rope_freqs(64)
    e = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    q, k = A.attn_rope(e, e[:, :2], f)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
