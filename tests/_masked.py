"""Attention in 64 bits under an arbitrary visibility table: the definition the
tests of the window-with-first-tokens and tree forms compare with.  Plain numpy,
S and P materialised; shares nothing with the library (test_masked_plain.py pins
it against the C oracle where both apply)."""
import numpy as np


def attend(q, k, v, keep, scale, softcap=0.0, sink=None, bias=None):
    """q [H, R, d], k/v [H, N, d] (kv heads already repeated), keep [R, N] or [H, R, N]
    bool, sink [H] or None, bias [H, R, N] added to the scaled score (natural-log
    units) -> o [H, R, d], lse [H, R].  A row that keeps nothing gives 0 and -inf (or
    its sink)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    keep = np.broadcast_to(keep, (q.shape[0], q.shape[1], k.shape[1]))
    s = scale * np.einsum("hrd,hnd->hrn", q, k)
    if softcap > 0:
        s = softcap * np.tanh(s / softcap)
    if bias is not None:
        s = s + bias
    s = np.where(keep, s, -np.inf)
    m = s.max(-1, initial=-np.inf)
    if sink is not None:
        m = np.maximum(m, np.asarray(sink, np.float64)[:, None])
    ms = np.where(np.isneginf(m), 0.0, m)
    p = np.exp(s - ms[..., None])
    z = p.sum(-1)
    if sink is not None:
        z = z + np.exp(np.asarray(sink, np.float64)[:, None] - ms)
    vz = np.where(keep.any((0, 1))[None, :, None], v, 0.0)  # rows nobody sees may hold anything
    o = np.einsum("hrn,hnd->hrd", p, vz) / np.where(z > 0, z, 1.0)[..., None]
    with np.errstate(divide="ignore"):
        lse = np.where(z > 0, ms + np.log(z), -np.inf)
    return o, lse


def band(Lq, Lk, left, right, sink_tokens=0, top_left=False):
    """keep[i, j] of the causal / window mask with the first sink_tokens keys visible
    left of it (negative bounds: unbounded)."""
    diag = np.arange(Lq)[:, None] + (0 if top_left else Lk - Lq)
    j = np.arange(Lk)[None, :]
    keep = np.ones((Lq, Lk), bool)
    if right >= 0:
        keep &= j <= diag + right
    if left >= 0:
        keep &= (j >= diag - left) | (j < sink_tokens)
    return keep


def alibi_bias(slopes, Lq, Lk, top_left=False):
    diag = np.arange(Lq)[:, None] + (0 if top_left else Lk - Lq)
    return -np.asarray(slopes, np.float64)[:, None, None] * np.abs(diag - np.arange(Lk)[None, :])


def paged_rows(pool, table_row, L, page):
    """Rows 0 .. L-1 of one sequence of a pool [pages, page, H, d] (numpy or torch)."""
    n = -(-L // page)
    ids = np.asarray(table_row[:n], np.int64)
    x = pool[ids]
    return x.reshape(-1, *x.shape[2:])[:L]
