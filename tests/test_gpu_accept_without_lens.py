"""attn_cache_accept without tree_lens, as the C interface has it: every sequence's last
T positions are its nodes."""
import pytest
import torch

import attention_forward_13_gb300 as A
from tests._parity import no_device_error

gpu = pytest.mark.gpu


def state(device):
    g = torch.Generator().manual_seed(3)
    pools = [torch.randint(0, 1 << 15, (2, 9, 16, 2, 8), dtype=torch.int16, generator=g).view(torch.float16).to(device)
             for _ in range(2)]
    ints = [torch.tensor(x, dtype=torch.int32, device=device) for x in
            ([[0, 1, 2], [5, 4, -1], [7, -1, -1], [8, -1, -1]], [40, 20, 3, 0], [1, 1, 1, 0, 1, 1, 0, 1, 1])]
    path = torch.tensor([[0, 2, 4], [1, 3, 4], [0, 2, 0], [0, 0, 0]], dtype=torch.int32, device=device)
    lens = torch.tensor([3, 2, 2, 0], dtype=torch.int32, device=device)
    return pools, ints, path, lens


def test_it_is_an_argument_check_that_refuses():
    pools, ints, path, lens = state("cpu")
    with pytest.raises(ValueError, match="T"):  # neither
        A.attn_cache_accept(*pools, *ints, path, lens)
    with pytest.raises(ValueError, match="CUDA"):  # fine, but for the device
        A.attn_cache_accept(*pools, *ints, path, lens, None, T=5)
    with pytest.raises(ValueError, match="T"):
        A.attn_cache_accept(*pools, *ints, path, lens, T=-1)


@gpu
@pytest.mark.parametrize("T", [3, 5, 24])
def test_the_same_as_with_equal_lens(T):
    want_pools, ints, path, lens = state("cuda")
    want = A.attn_cache_accept(*want_pools, *ints, path, lens, torch.full_like(lens, T))
    bits = A.attn_device_error()  # (a path that leaves a short tree is an error, with both)
    for kw in (dict(tree_lens=None, T=T), dict(T=T)):
        pools, ints, path, lens = state("cuda")
        got = A.attn_cache_accept(*pools, *ints, path, lens, **kw)
        assert A.attn_device_error() == bits
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(pools, want_pools))


@gpu
def test_lens_past_t_are_cut_to_it():
    want_pools, ints, path, lens = state("cuda")
    want = A.attn_cache_accept(*want_pools, *ints, path, lens, torch.full_like(lens, 5))
    pools, ints, path, lens = state("cuda")
    got = A.attn_cache_accept(*pools, *ints, path, lens, torch.full_like(lens, 900), T=5)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(pools, want_pools))
    no_device_error()
