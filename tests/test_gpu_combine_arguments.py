"""attn_splitkv_combine with partials in other layouts, and what it refuses."""
import pytest
import torch

import attention_forward_13_gb300 as A
from tests._parity import no_device_error

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("S,B,H,L,d", [(3, 2, 4, 5, 64), (2, 1, 8, 1, 128), (7, 3, 2, 16, 64)])
def test_strided_partials(S, B, H, L, d):
    """Both made contiguous by the call: their copies stay apart, and alive until the kernel
    has read them."""
    g = torch.Generator(device="cuda").manual_seed(S)
    o, lse = torch.randn(S, B, H, L, d, device="cuda", generator=g), torch.randn(S, B, H, L, device="cuda", generator=g)
    want = A.attn_splitkv_combine(o, lse, dtype=torch.float16)
    so = o.transpose(0, 4).contiguous().transpose(0, 4)
    sl = lse.transpose(0, 3).contiguous().transpose(0, 3)
    assert not so.is_contiguous() and (L == 1 or not sl.is_contiguous())
    for _ in range(5):
        got = A.attn_splitkv_combine(so, sl, dtype=torch.float16)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # A doubled copy of lse alone, as large as o's: it may not land on o's.
    wide = torch.randn(S, B, H, L, 2 * d, device="cuda", generator=g)[..., ::2]
    want = A.attn_splitkv_combine(wide.contiguous(), lse)
    got = A.attn_splitkv_combine(wide, lse[..., None].expand(S, B, H, L, 2)[..., 0].transpose(0, 1).contiguous()
                                 .transpose(0, 1))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    no_device_error()


def test_copies_are_held_until_the_call(monkeypatch):
    """No copy dies before the library is called (its memory could go to the next copy)."""
    import weakref
    refs, alive = [], []
    contiguous = torch.Tensor.contiguous

    def noted(t, *a):
        out = contiguous(t, *a)
        refs.append(weakref.ref(out))
        return out

    class Lib:
        def attn_splitkv_combine(self, *a):
            alive.append([r() is not None for r in refs])
            return 0

    monkeypatch.setattr(torch.Tensor, "contiguous", noted)
    monkeypatch.setattr(A, "library", lambda: Lib())
    monkeypatch.setattr(A, "_stream", lambda s: 0)
    o, lse = torch.zeros(2, 1, 3, 64, 4).transpose(3, 4), torch.zeros(2, 1, 4, 3).transpose(2, 3)
    A.attn_splitkv_combine(o, lse)
    assert len(refs) == 2 and alive == [[True, True]]


@pytest.mark.parametrize("bad", [
    dict(o_partial=torch.zeros(2, 1, 3, 4, 64, dtype=torch.bfloat16)),
    dict(lse_partial=torch.zeros(2, 1, 3, 4, dtype=torch.float64)),
    dict(lse_partial=torch.zeros(2, 1, 3, 3)),
    dict(lse_partial=torch.zeros(1, 1, 3, 4)),
    dict(o=torch.zeros(1, 3, 4, 64, dtype=torch.bfloat16)),
    dict(o=torch.zeros(1, 4, 3, 128, dtype=torch.bfloat16)[..., ::2]),
    dict(lse=torch.zeros(1, 3, 3)),
    dict(lse=torch.zeros(1, 3, 4, dtype=torch.bfloat16)),
])
def test_refused(bad):
    kw = dict(o_partial=torch.zeros(2, 1, 3, 4, 64), lse_partial=torch.zeros(2, 1, 3, 4))
    kw.update(bad)
    with pytest.raises(ValueError):
        A.attn_splitkv_combine(**kw)
