"""Rotary frequencies (host only), from their definitions in Python floats, and what is refused."""
import ctypes
import math

import pytest

import attention_forward_13_gb300 as A


def freqs(r, *a, **k):
    return A.attn_rope_freqs(r, *a, device="cpu", **k).tolist()


def near(got, want):
    assert len(got) == len(want)
    assert all(abs(g - w) <= 1e-14 * w for g, w in zip(got, want)), (got, want)


PLAIN = [10000.0 ** (-i / 32) for i in range(32)]


def test_plain():
    near(freqs(64), PLAIN)
    near(freqs(2), [1.0])
    near(freqs(6, base=500000.0), [1.0, 500000.0 ** (-1 / 3), 500000.0 ** (-2 / 3)])


def test_linear_is_interpolated_positions():
    near(freqs(64, scaling="linear", factor=8.0), [f / 8 for f in PLAIN])


def test_base_divides_the_slowest_by_the_factor_and_keeps_the_fastest():
    got = freqs(64, scaling="base", factor=4.0)
    assert got[0] == 1.0 and abs(got[-1] - PLAIN[-1] / 4) < 1e-14
    assert all(a > b for a, b in zip(got, got[1:]))


@pytest.mark.parametrize("slow,fast,factor", [(1.0, 32.0, 16.0), (1.0, 4.0, 8.0)])
def test_parts(slow, fast, factor):
    want = []
    for f in PLAIN:
        turns = 8192 * f / (2 * math.pi)
        w = 0.0 if turns <= slow else 1.0 if turns >= fast else (turns - slow) / (fast - slow)
        want.append(w * f + (1 - w) * f / factor)
    got = freqs(64, scaling="parts", factor=factor, original_len=8192, slow_turns=slow, fast_turns=fast)
    near(got, want)
    assert got[0] == 1.0 and abs(got[-1] - PLAIN[-1] / factor) < 1e-14


def test_ramp():
    got = freqs(64, scaling="ramp", factor=16.0, original_len=4096, slow_turns=1.0, fast_turns=32.0)
    # turns(i) = 4096 / 2 pi * 10000^(-i / 32) is 32 at i = 10.46 and 1 at i = 22.51
    low, high = 10, 23
    want = []
    for i, f in enumerate(PLAIN):
        slowed = min(1.0, max(0.0, (i - low) / (high - low)))
        want.append(f * (1 - slowed) + f / 16 * slowed)
    near(got, want)


def test_a_factor_of_one_changes_nothing():
    for s in ("linear", "base", "parts", "ramp"):
        near(freqs(64, scaling=s, factor=1.0, original_len=4096), PLAIN)


@pytest.mark.parametrize("kw", [dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=-2), dict(base=1.0),
                                dict(base=math.inf), dict(base=math.nan), dict(scaling="linear", factor=0.5),
                                dict(scaling="linear", factor=math.nan), dict(scaling="parts", factor=2.0),
                                dict(scaling="parts", factor=2.0, original_len=100, slow_turns=4.0, fast_turns=4.0),
                                dict(scaling="ramp", factor=2.0, original_len=100, slow_turns=0.0),
                                dict(rotary_dim=2, scaling="base", factor=2.0)])
def test_refused(kw):
    with pytest.raises(A.AttnError):
        A.attn_rope_freqs(**{**dict(rotary_dim=64, device="cpu"), **kw})


def test_unknown_scaling_refused():
    with pytest.raises(ValueError):
        A.attn_rope_freqs(64, scaling="other", device="cpu")
    assert A.library().attn_rope_freqs(64, 1e4, 7, 1.0, 0.0, 0.0, 0.0, (ctypes.c_double * 32)()) == 1
    assert A.library().attn_rope_freqs(64, 1e4, 0, 1.0, 0.0, 0.0, 0.0, None) == 1
