"""The factor on rotated elements: 0 is refused in Python, also what is 0 in 32 bits (the C options' 0
stands for 1)."""
import pytest

import attention_forward_13_gb300 as A
from tests.test_serving_checks import F, I5, K, K4, POOL, Q, Q4


@pytest.mark.parametrize("scale", [0.0, 0, -0.0, 1e-50])
def test_no_scale_of_zero(scale):
    for a in ((Q, K), (Q4, K4), (Q, None)):
        with pytest.raises(ValueError, match="scale"):
            A.attn_rope(*a, F, scale=scale)
    with pytest.raises(ValueError, match="scale"):
        A.attn_cache_append(K, K, POOL, POOL, I5, q=Q, inv_freq=F, positions=I5, scale=scale)


def test_others_come_to_the_device():
    with pytest.raises(ValueError, match="CUDA"):
        A.attn_rope(Q, K, F, scale=0.5)
