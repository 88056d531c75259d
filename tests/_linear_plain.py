"""Linear attention with a decay per head, token by token in 64 bits, and how far a kernel of 16-bit products may be from
it.

The chunked kernel rounds two things to the input type on the way to o (the weights q_i . k_j e^(g (i-j)) within a
chunk, and the state before it), each by at most half a step h = eps / 2 relative to its value, and o itself:
    |do| <= h (A + |o|) + 32-bit terms,   A = the same recurrence on |q|, |k|, |v| and the state's magnitude.
(A rounded weight moves o_i by at most h |w_ij v_j|; a rounded state element by h |q_r S_rc|: both sums are at most A,
and the two cover different tokens, so that together they are at most h A.)  The state's own sum takes e^(g n) v in two pieces of the input
type, the second rounded: h^2 relative to each term, plus 32-bit sums.  32 bits: products of
a chunk are summed by the tensor core in steps of 16 tokens or elements, each step rounding (or cutting) within 2^-23 of the
sum of magnitudes, 8 steps at d = 128 and a chunk of 128; the decays' exponents are rounded to 2^-24, which moves e^(g n) by at
most 2^-24 |g n| e^(g n) < 2^-24 relative to the undecayed term, so that summed over tokens it stays below 2^-22 A; one
rounding per chunk for the carried state: c 2^-24 over c chunks.  Together below (64 + c) 2^-23 A."""
import torch


def recurrence(q, k, v, g, state=None):
    """q, k, v [H, L, d] (k, v repeated for shared heads), g [H]; state [H, d, d].  fp64 (o without the scale, S)."""
    H, L, d = q.shape
    q, k, v, w = q.double(), k.double(), v.double(), torch.exp(g.double())[:, None, None]
    S = torch.zeros(H, d, d, dtype=torch.float64, device=q.device) if state is None else state.double().clone()
    o = torch.empty(H, L, d, dtype=torch.float64, device=q.device)
    for t in range(L):
        S = S * w + k[:, t, :, None] * v[:, t, None, :]
        o[:, t] = (q[:, t, :, None] * S).sum(1)
    return o, S


def with_bounds(q, k, v, g, scale, state=None):
    """(o, S, most |do|, most |dS|) in fp64."""
    o, S = recurrence(q, k, v, g, state)
    A, M = recurrence(q.abs(), k.abs(), v.abs(), g, None if state is None else state.abs())
    h = torch.finfo(q.dtype).eps / 2
    tiny = torch.finfo(q.dtype).smallest_normal * torch.finfo(q.dtype).eps  # half a step below the normal numbers, and more
    f32 = (64 + (q.shape[1] + 127) // 128) * 2.0 ** -23
    o = o * scale
    # Weights and decayed values below the normal numbers are rounded to multiples of `tiny` (fp16): against |v|, |k| of
    # at most 16 here, and 128 of them.
    low = tiny * 16 * 128
    return o, S, h * (A * scale + o.abs()) + f32 * A * scale + tiny + low, (h * h + f32) * M + 1e-30 + low


def check(o, S, want, what=""):
    o64, S64, do, dS = want
    worst = ((o.double() - o64).abs() / do).max().item() if o.numel() else 0.0
    assert torch.isfinite(o).all() and worst <= 1.0, (what, "o", worst)
    if S is not None:
        assert torch.isfinite(S).all()
        w = ((S.double() - S64).abs() / dS).max().item()
        assert w <= 1.0, (what, "state", w)
    # The bound above allows for every rounding going the same way; random signs do not.
    if o.numel() >= 1 << 14:
        h = torch.finfo(o.dtype).eps / 2
        rel = ((o.double() - o64).norm() / o64.norm()).item()
        assert rel <= 3 * h, (what, "norm of o", rel / h)
