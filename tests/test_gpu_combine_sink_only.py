"""A merged row whose parts have all seen nothing: O is 0, and its LSE is the sink's to the bit (there is nothing to add
to it), -inf without a sink."""
import numpy as np
import pytest
import torch

import attention_forward_13_gb300 as A
from tests._parity import no_device_error


def sinks(n):
    x = np.random.default_rng(4).standard_normal(n).astype(np.float32) * 3
    x[:4] = 0.0, -1.3946, 1e4, -1e4
    return x


def test_the_way_through_log2_units_is_not_exact():
    """x log2(e) ln(2) in 32 bits is often a neighbour of x."""
    x = sinks(512)
    y = (x * np.float32(1.4426950408889634)) * np.float32(0.6931471805599453)
    assert (x != y).mean() > 0.1


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S", [1, 5, 40])
def test_lse_is_the_sink(S, d):
    H = 512
    sink = torch.from_numpy(sinks(H)).cuda()
    o, lse = torch.randn(S, 1, H, 2, d, device="cuda"), torch.randn(S, 1, H, 2, device="cuda")
    lse[..., 0] = float("-inf")
    out, got = A.attn_splitkv_combine(o, lse, sink=sink)
    assert not out[0, 0].any() and torch.equal(got[0, :, 0], sink)
    want = torch.logsumexp(torch.cat((lse[:, 0, :, 1].double(), sink[None].double())), 0)
    assert ((got[0, :, 1].double() - want).abs() <= 1e-5 * (1 + want.abs())).all()
    out, got = A.attn_splitkv_combine(o, lse)
    assert not out[0, 0].any() and (got[0, :, 0] == float("-inf")).all() and got[0, :, 1].isfinite().all()
    no_device_error()
