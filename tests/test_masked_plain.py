"""The 64-bit masked attention the newer GPU tests compare with, against the C
oracle where both apply, and its own extremes."""
import numpy as np
import pytest

import oracle
from tests import _masked as M


@pytest.mark.parametrize("case", [
    # Lq, Lk, causal, window, cap, sink, top_left
    (5, 9, True, (-1, -1), 0.0, False, False),
    (9, 5, True, (2, -1), 0.0, True, False),
    (7, 7, False, (1, 2), 3.0, True, False),
    (6, 8, False, (0, 0), 0.0, False, True),
])
def test_matches_the_oracle(case):
    Lq, Lk, causal, win, cap, sink, tl = case
    rng = np.random.default_rng(Lq * Lk)
    H, d = 3, 8
    q, k, v = rng.normal(size=(H, Lq, d)), rng.normal(size=(H, Lk, d)), rng.normal(size=(H, Lk, d))
    sk = rng.normal(size=H) if sink else None
    right = 0 if causal else win[1]
    o, lse = M.attend(q, k, v, M.band(Lq, Lk, win[0], right, 0, tl), 0.3, cap, sk)
    ro, rl = oracle.attn_dense(q[None], k[None], v[None], 0.3, causal, cap, sk, window=win, top_left=tl)
    assert np.allclose(o, ro[0], rtol=1e-12, atol=1e-12)
    fin = np.isfinite(rl[0])
    assert np.array_equal(np.isfinite(lse), fin) and np.allclose(lse[fin], rl[0][fin], rtol=1e-12)


def test_alibi_matches_the_oracle():
    rng = np.random.default_rng(3)
    q, k, v = (rng.normal(size=(2, 6, 8)) for _ in range(3))
    sl = np.array([0.5, 0.125])
    o, lse = M.attend(q, k, v, M.band(6, 6, 2, 0), 0.3, bias=M.alibi_bias(sl, 6, 6))
    ro, rl = oracle.attn_dense(q[None], k[None], v[None], 0.3, True, window=(2, -1), alibi=sl)
    assert np.allclose(o, ro[0], rtol=1e-12, atol=1e-12) and np.allclose(lse, rl[0], rtol=1e-12)


def test_first_tokens():
    """Enough first tokens make a left window the plain causal mask; none make it the band; in
    between exactly the listed keys come back, never past the right bound."""
    assert np.array_equal(M.band(9, 9, 2, 0, 9), M.band(9, 9, -1, 0))
    assert np.array_equal(M.band(9, 9, 2, 0, 0), M.band(9, 9, 2, 0))
    keep = M.band(6, 6, 1, 0, 2)
    want = [[1, 0, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0], [1, 1, 1, 0, 0, 0], [1, 1, 1, 1, 0, 0],
            [1, 1, 0, 1, 1, 0], [1, 1, 0, 0, 1, 1]]
    assert np.array_equal(keep.astype(int), want)
