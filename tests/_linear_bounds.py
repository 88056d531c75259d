"""How far the chunked linear attention kernel may be from the recurrence in 64 bits, with every allowance in
proportion to the inputs (nothing absolute but the subnormal numbers of o's own type), and for decays above 1 too.

h = eps / 2 is half a step of the 16-bit type, w = e^g, A and M the recurrences of o and S on magnitudes.
o:  weights and the state before a chunk are rounded to 16 bits, each h of its own value, and o itself: h (A + |o|).
    In fp16 both are scaled by powers of two and may fall among the subnormal numbers (half a step 2^-25): a row's weights
    where its largest score lies at 2^10 or more, so by 2^-35 of that score against the sum of |v| (decays above 1: its
    largest weight at 2^14 w^-15 or more, so by 2^-39 w^15 of that); the state where its largest element lies at 2^14 or more, so by 2^-39 of that element against the sum of |q|,
    times up to w^128 if that is above 1.
S:  the terms e^(g n) v come in two 16-bit pieces.  bf16: 3 h^2 of each term (the weight's rest, at most h of it, is
    rounded by h of itself, and the second piece, at most 2 h of the term, by h of that).  fp16: the second piece, at most
    2^-11 of the term and exact before, is rounded to 2^-11 of itself, and the term was to 2^-24; it is held at 2^11 of
    its size, so that below the normal numbers it is off by 2^-25 2^-11 = 2^-36.  That meets |k| whatever the weight was, n counting the tokens to the end of a chunk of
    128, or of a piece where the sequence is cut (piece: at least that many tokens), and decays from there on; decays above
    1 are counted from a chunk's start, so that the state then grows by up to w^128.
32 bits: (64 + c) 2^-23 of the magnitudes over c chunks for the sums, and 2 |g| L 2^-23 for the decays' exponents where
    these do not make up for themselves (above 1)."""
import torch


def bounds(q, k, v, g, scale, state=None, piece=128):
    """q, k, v [H, L, d] (k, v repeated for shared heads), g fp32 [H], state [H, d, d] -> fp64 (o, S, |do|, |dS|)."""
    f16 = q.dtype is torch.float16
    h = torch.finfo(q.dtype).eps / 2
    H, L, d = q.shape
    q, k, v, g = q.double(), k.double(), v.double(), g.double()
    w = torch.exp(g)[:, None, None]
    S = torch.zeros(H, d, d, dtype=torch.float64, device=q.device) if state is None else state.double().clone()
    M, now, before = S.abs(), torch.zeros_like(S), torch.zeros_like(S)
    grown = torch.exp(128 * g.clamp(min=0))[:, None, None]
    o, A, top = torch.empty_like(q), torch.empty_like(q), torch.empty(H, L, dtype=torch.float64, device=q.device)
    most = S.abs().amax((1, 2))
    for t in range(L):
        top[:, t] = most
        kt, vt, qt = k[:, t, :, None], v[:, t, None, :], q[:, t, :, None]
        S, M = S * w + kt * vt, M * w + kt.abs() * vt.abs()
        before, now = before * w, now + kt.abs() * 2.0 ** -36
        if (t + 1) % piece == 0 or t == L - 1:
            before, now = before + now * grown, torch.zeros_like(now)
        o[:, t], A[:, t] = (qt * S).sum(1), (qt.abs() * M).sum(1)
        most = torch.maximum(most, S.abs().amax((1, 2)))
    f32 = ((64 + (L + 127) // 128 + 2 * g.clamp(min=0) * L) * 2.0 ** -23)[:, None, None]
    do = h * (A * scale + o.abs() * scale) + f32 * A * scale + torch.finfo(torch.float16 if f16 else torch.bfloat16).smallest_normal * h
    dS = (2.0 ** -21 if f16 else 3 * h * h) * M + f32 * M + 1e-35
    if f16:
        i = torch.arange(L, device=q.device)
        best = torch.zeros(H, L, dtype=torch.float64, device=q.device)
        for a in range(0, L, 128):  # scores within a chunk
            n = i[a:a + 128]
            span = (n[:, None] - n).clamp(min=0)
            sc = torch.matmul(q[:, n], k[:, n].transpose(1, 2)).abs() * torch.exp(g.clamp(min=0)[:, None, None] * span)
            best[:, n] = torch.where(n[:, None] >= n, sc, 0.0).amax(2)
        low = torch.where(g > 0, 2.0 ** -39 * torch.exp(15 * g), 2.0 ** -35)[:, None, None]
        do += low * best[..., None] * scale * v.abs().cumsum(1)
        do += 2.0 ** -39 * (top * q.abs().sum(2))[..., None] * scale * grown
        dS += before
    return o * scale, S, do, dS


def piece(B, H, L, d):
    """Tokens of a cut sequence's pieces, at most (128 where it is not cut)."""
    import attention_forward_13_gb300 as A
    pieces = A.attn_linear_workspace_bytes(B, H, L, B * L, d) // (B * H * d * d * 4)
    chunks = (L + 127) // 128
    return 128 * (-(-chunks // (pieces - 1)) if pieces > 1 else 1)


def check(o, S, want, what=""):
    o64, S64, do, dS = want
    if o is not None:
        assert torch.isfinite(o).all(), (what, "o")
        worst = ((o.double() - o64).abs() / do).max().item()
        assert worst <= 1.0, (what, "o", worst)
    if S is not None:
        assert torch.isfinite(S).all(), (what, "state")
        worst = ((S.double() - S64).abs() / dS).max().item()
        assert worst <= 1.0, (what, "state", worst)
