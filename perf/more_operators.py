"""Cases for what a serving step runs around the attention over a ragged batch: where
each new token goes in the paged cache (slots and positions from the requests' lengths),
rotary positions, the rotated keys and the values written into the pages, and linear
attention with a decay per head (whole prompts in chunks, single tokens by recurrence).

`own` false: the operators in plain torch, 32-bit arithmetic (angles in 64), rounded once
at the end.  `own` true: the same through the library's entry points.  Both take the state
`prepare` makes and return the same outputs.

Packed tokens: sequence b owns rows cu[b] .. cu[b+1]-1.  A cache row's slot is
page * page_size + row in the page; -1 marks a padding token.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# --------------------------------------------------------------------------- cases
def _slots(name, B, lo, hi, add_lo, add_hi, page, pad):
    """B sequences with lo..hi cached tokens and add_lo..add_hi new ones; pad: room for more tokens."""
    return dict(name=name, kind="slots", B=B, lo=lo, hi=hi, add_lo=add_lo, add_hi=add_hi, page=page, pad=pad)


def _rope(name, form, B, L, Hq, Hkv, d, rot, dtype, interleaved, first, factor, inverse=False):
    """form dense: [B,H,L,d]; packed: B sequences of 1..L tokens.  Positions start at `first`."""
    return dict(name=name, kind="rope", form=form, B=B, L=L, Hq=Hq, Hkv=Hkv, d=d, rot=rot, dtype=dtype,
                interleaved=interleaved, first=first, factor=factor, inverse=inverse)


def _append(name, B, lo, hi, add_lo, add_hi, Hq, Hkv, d, rot, page, dtype, interleaved, pages, pad):
    return dict(name=name, kind="append", B=B, lo=lo, hi=hi, add_lo=add_lo, add_hi=add_hi, Hq=Hq, Hkv=Hkv, d=d,
                rot=rot, page=page, dtype=dtype, interleaved=interleaved, pages=pages, pad=pad)


def _linear(name, form, B, L, Hq, Hkv, d, dtype, state, strong=1.0):
    """form dense, packed or step; state: the call starts from a state; strong scales the decays' logarithms."""
    return dict(name=name, kind="linear", form=form, B=B, L=L, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, state=state,
                strong=strong)


def listed():
    return [
        # one decode step of the paged serving batch: a new token each, the smallest call
        _slots("slots_decode64", 64, 512, 8192, 1, 1, 64, 0),
        # a step that admits 256 ragged prompts into a cache of small pages, token count padded for a graph
        _slots("slots_prompts256", 256, 0, 900, 1, 500, 16, 1000),
        # the long grouped-query prompt, dense layout, whole heads rotated in halves
        _rope("rope_prompt_8192", "dense", 2, 8192, 32, 8, 128, 128, "bf16", False, 0, 1.0),
        # packed sequences far into a long context: pairs side by side, a quarter of the head, scaled by parts
        _rope("rope_far_odd", "packed", 16, 257, 24, 8, 64, 16, "f16", True, 1000003, 32.0),
        # the decode step's write into the cache, queries rotated on the way
        _append("append_decode64", 64, 512, 8192, 1, 1, 32, 8, 128, 128, 64, "bf16", False, 9000, 0),
        # chunked prefill: 512 tokens of each of 8 sequences
        _append("append_chunks", 8, 0, 3584, 512, 512, 32, 8, 128, 128, 64, "bf16", False, 1024, 0),
        # ragged chunks with padding, small pages, half of the head rotated in pairs, 3 heads per kv head
        _append("append_odd", 13, 0, 700, 1, 333, 24, 8, 64, 32, 16, "f16", True, 1200, 77),
        # a long prompt through a linear layer, the final state kept for decoding
        _linear("linear_prompt_8192", "dense", 2, 8192, 32, 32, 128, "bf16", False),
        # one user's next chunk: few heads, the state carried over
        _linear("linear_one_2048", "dense", 1, 2048, 16, 16, 128, "bf16", True),
        # packed prompts of odd lengths, d = 64, strong decays, shared kv heads
        _linear("linear_packed_odd", "packed", 16, 3001, 16, 4, 64, "f16", True, 4.0),
        # one token of one user
        _linear("step_one_user", "step", 1, 1, 16, 16, 128, "bf16", True),
        # one decode step of a 64-sequence batch
        _linear("step_decode64", "step", 64, 1, 32, 32, 128, "bf16", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["slots", "rope", "rope", "append", "append", "linear", "linear", "linear"])
    dtype, d, page = rng.choice(["bf16", "f16"]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128, 256])
    Hkv, g, mixed = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8]), rng.random() < 0.5
    if kind == "slots":
        hi, add = _log(rng, 1, 9000), _log(rng, 1, 500)
        c = _slots("", _log(rng, 1, 256), rng.randrange(0, hi), hi, rng.choice([0, 1, add]), add, page,
                   rng.randrange(0, 300))
    elif kind == "rope":
        d = rng.choice([64, 80, 96, 128])
        rot = rng.choice([d, d, d // 2, 32, 2 * rng.randrange(1, d // 2)])
        c = _rope("", rng.choice(["dense", "packed"]), _log(rng, 1, 8), _log(rng, 1, 2048), Hkv * g, Hkv, d, rot,
                  dtype, mixed, rng.choice([0, _log(rng, 1, 2000000)]), rng.choice([1.0, 1.0, 4.0, 32.0]),
                  rng.random() < 0.3)
    elif kind == "append":
        B, hi, add = _log(rng, 1, 64), _log(rng, 1, 2000), rng.choice([1, 1, _log(rng, 2, 300)])
        rot = rng.choice([0, d, d, d // 2, 2 * rng.randrange(1, d // 2)])
        c = _append("", B, rng.randrange(0, hi), hi, rng.randrange(1, add + 1), add, Hkv * g, Hkv, d, rot, page, dtype,
                    mixed, B * ((hi + add + page - 1) // page) + rng.randrange(1, 40), rng.randrange(0, 40))
    else:
        form = rng.choice(["dense", "packed", "step"])
        B = _log(rng, 1, 64 if form == "step" else 8)
        L = 1 if form == "step" else _log(rng, 1, 2500)
        g = min(g, 4)
        c = _linear("", form, B, L, Hkv * g, Hkv, d, dtype, form == "step" or rng.random() < 0.6,
                    rng.choice([0.0, 0.25, 1.0, 4.0, 40.0]))
    return {k: v for k, v in c.items() if k != "name"}


# --------------------------------------------------------------------------- inputs
def _randn(gen, shape, dtype):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat, n = out.view(-1), out.numel()
    for s in range(0, n, 1 << 27):
        e = min(n, s + (1 << 27))
        flat[s:e] = torch.randn(e - s, generator=gen, device="cuda")
    return out


def _i32(rows):
    return torch.tensor(rows, dtype=torch.int32, device="cuda")


def _frequencies(c):
    """Angle per position of each pair, fp64: base 10000; with a factor, pairs of fewer than one turn in
    4096 positions are slowed by it, those of over 32 keep their pace, between them linearly in the turns."""
    f = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])
    if c.get("factor", 1.0) != 1.0:
        keep = ((4096 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
        f = f * keep + f / c["factor"] * (1 - keep)
    return f.cuda()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed * 7919 + 29)
    pick = random.Random(6)  # packed lengths stay, so that the packed tensors keep their shapes
    s = {"case": c}
    B = c["B"]
    if c["kind"] in ("slots", "append"):
        add = [pick.randint(c["add_lo"], c["add_hi"]) for _ in range(B)]
        lens = [rng.randint(c["lo"], c["hi"]) + n for n in add]
        held = [-(-n // c["page"]) for n in lens]
        s["pages"] = c["pages"] if c["kind"] == "append" else B * max(1, -(-(c["hi"] + c["add_hi"]) // c["page"]))
        order = list(range(s["pages"]))
        rng.shuffle(order)
        width, rows, at = max(1, -(-(c["hi"] + c["add_hi"]) // c["page"])), [], 0
        for n in held:
            rows.append(order[at:at + n] + [0] * (width - n))
            at += n
        s["block_table"], s["seqlens"], s["add"] = _i32(rows), _i32(lens), _i32(add)
        s["tokens"] = sum(add) + c["pad"]
        if c["kind"] == "slots":
            return s
        slots, positions = [], []
        for row, n, m in zip(rows, lens, add):
            for p in range(n - m, n):
                slots.append(row[p // c["page"]] * c["page"] + p % c["page"])
                positions.append(p)
        N = s["tokens"]
        s["slots"], s["positions"] = _i32(slots + [-1] * c["pad"]), _i32(positions + [0] * c["pad"])
        # one projection's output, q, k and v side by side, as a layer hands them over
        qkv = _randn(gen, (N, c["Hq"] + 2 * c["Hkv"], c["d"]), DTYPES[c["dtype"]])
        s["q"], s["k"], s["v"] = qkv.split([c["Hq"], c["Hkv"], c["Hkv"]], 1)
        for name in ("k_pool", "v_pool"):
            s[name] = _randn(gen, (c["pages"], c["page"], c["Hkv"], c["d"]), DTYPES[c["dtype"]])
        s["inv_freq"] = _frequencies(c) if c["rot"] else None
        return s
    dt, L = DTYPES[c["dtype"]], c["L"]
    if c["form"] == "packed":
        lens = [pick.randint(1, L) for _ in range(B)]
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["lens"], s["cu"], s["longest"] = lens, _i32(cu), max(lens)
        shape = lambda H: (cu[-1], H, c["d"])  # noqa: E731
    else:
        shape = (lambda H: (B, H, c["d"])) if c["form"] == "step" else (lambda H: (B, H, L, c["d"]))
    s["q"], s["k"] = _randn(gen, shape(c["Hq"]), dt), _randn(gen, shape(c["Hkv"]), dt)
    if c["kind"] == "rope":
        start = [c["first"] + rng.randrange(0, 1000) for _ in range(B)]
        if c["form"] == "packed":
            s["positions"] = _i32([a + i for a, n in zip(start, s["lens"]) for i in range(n)])
        else:
            s["positions"] = _i32([list(range(a, a + L)) for a in start])
        s["inv_freq"] = _frequencies(c)
        return s
    s["v"] = _randn(gen, shape(c["Hkv"]), dt)
    s["scale"] = 1.0 / math.sqrt(c["d"])
    # decays from e^-0.7 down to e^-0.004 a token, over the heads
    h = torch.arange(1, c["Hq"] + 1, dtype=torch.float64)
    s["log_decay"] = (-c["strong"] * 2.0 ** (-8.0 * h / c["Hq"])).float().cuda()
    s["state"] = torch.randn(B, c["Hq"], c["d"], c["d"], generator=gen, device="cuda") if c["state"] else None
    return s


# --------------------------------------------------------------------------- one pass
def run(state):
    return (_own if own else _plain)[state["case"]["kind"]](state)


def _own_slots(s):
    import attention_forward_13_gb300 as A
    slots, positions, cu, sequence = A.attn_cache_slots(s["block_table"], s["seqlens"], s["add"], s["tokens"],
                                                        s["case"]["page"], s["pages"])
    return {"slots": slots, "positions": positions, "cu": cu, "sequence": sequence}


def _own_rope(s):
    import attention_forward_13_gb300 as A
    c = s["case"]
    q, k = A.attn_rope(s["q"], s["k"], s["inv_freq"], s["positions"], interleaved=c["interleaved"],
                       inverse=c["inverse"])
    return {"q": q, "k": k}


def _own_append(s):
    import attention_forward_13_gb300 as A
    q = A.attn_cache_append(s["k"], s["v"], s["k_pool"], s["v_pool"], s["slots"], q=s["q"], inv_freq=s["inv_freq"],
                            positions=s["positions"], interleaved=s["case"]["interleaved"])
    return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _own_linear(s):
    import attention_forward_13_gb300 as A
    c = s["case"]
    if c["form"] == "step":
        o = A.attn_linear_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], scale=s["scale"])
        return {"o": o, "state": s["state"]}
    if c["form"] == "dense":
        o, state = A.attn_linear_fwd(s["q"], s["k"], s["v"], s["log_decay"], state=s["state"], scale=s["scale"])
    else:
        o, state = A.attn_linear_fwd_varlen(s["q"], s["k"], s["v"], s["cu"], s["longest"], s["log_decay"],
                                            state=s["state"], scale=s["scale"])
    return {"o": o, "state": state}


_own = {"slots": _own_slots, "rope": _own_rope, "append": _own_append, "linear": _own_linear}


# --------------------------------------------------------------------------- plain forms
def _plain_slots(s):
    page, N = s["case"]["page"], s["tokens"]
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), s["add"].long().cumsum(0)])
    t = torch.arange(N, device="cuda")
    b = (t[:, None] >= cu[1:]).sum(1)
    real = b < s["case"]["B"]
    b = b.clamp(max=s["case"]["B"] - 1)
    pos = torch.where(real, s["seqlens"].long()[b] - s["add"].long()[b] + t - cu[b], 0)
    slots = torch.where(real, s["block_table"].long()[b, pos // page] * page + pos % page, -1)
    return {"slots": slots.to(torch.int32), "positions": pos.to(torch.int32), "cu": cu.to(torch.int32),
            "sequence": torch.where(real, b, -1).to(torch.int32)}


def _turned(x, angle, interleaved):
    """x [..., d] with its first pairs turned by angle [..., pairs] (fp64; broadcast over heads)."""
    r = 2 * angle.shape[-1]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    f = x.float()
    y = torch.empty_like(f)
    a = slice(0, r, 2) if interleaved else slice(0, r // 2)
    b = slice(1, r, 2) if interleaved else slice(r // 2, r)
    y[..., a] = f[..., a] * cos - f[..., b] * sin
    y[..., b] = f[..., b] * cos + f[..., a] * sin
    y[..., r:] = f[..., r:]
    return y.to(x.dtype)


def _plain_rope(s):
    c = s["case"]
    angle = s["positions"].double()[..., None] * s["inv_freq"]
    angle = (-angle if c["inverse"] else angle).unsqueeze(1)  # one angle for all heads
    return {"q": _turned(s["q"], angle, c["interleaved"]), "k": _turned(s["k"], angle, c["interleaved"])}


def _plain_append(s):
    c = s["case"]
    q, k = s["q"].clone(memory_format=torch.contiguous_format), s["k"]
    if c["rot"]:
        angle = (s["positions"].double()[:, None] * s["inv_freq"]).unsqueeze(1)
        q, k = _turned(q, angle, c["interleaved"]), _turned(k, angle, c["interleaved"])
    n = s["tokens"] - c["pad"]
    at = s["slots"][:n].long()
    s["k_pool"].view(-1, c["Hkv"], c["d"])[at] = k[:n]
    s["v_pool"].view(-1, c["Hkv"], c["d"])[at] = s["v"][:n]
    return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _chunked(q, k, v, g, state, scale, lens):
    """q, k, v [B,H,L,d] fp32, zero past lens [B]; g [H].  Chunks of 128 tokens: products within a chunk, the
    chunks' own states, and those carried on by a triangle of decays.  Returns o and the states after lens."""
    B, H, L, d = q.shape
    C = 128
    n = -(-L // C)
    pad = lambda x: torch.nn.functional.pad(x, (0, 0, 0, n * C - L)).view(B, H, n, C, d)  # noqa: E731
    q, k, v = pad(q), pad(k), pad(v)
    i = torch.arange(C, device="cuda")
    span = (i[:, None] - i).clamp(min=0).double()
    within = torch.where(i[:, None] >= i, torch.exp(g.double()[:, None, None] * span), 0.0).float()
    o = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * within[:, None], v)
    ahead = torch.exp(g.double()[:, None] * (C - 1 - i)).float()[:, None, :, None]
    own_state = torch.matmul((k * ahead).transpose(-1, -2), v)  # [B,H,n,d,d]
    m = torch.arange(n + 1, device="cuda")
    over = torch.exp(g.double()[:, None, None] * (C * (m[:, None] - 1 - m[:n]).clamp(min=0)).double())
    carry = torch.where(m[:, None] > m[:n], over, 0.0).float()  # [H, n + 1, n]
    states = torch.matmul(carry, own_state.view(B, H, n, d * d))
    if state is not None:
        first = torch.exp(g.double()[:, None] * (C * m)).float()
        states = states + first[:, :, None] * state.reshape(B, H, 1, d * d)
    states = states.view(B, H, n + 1, d, d)
    since = torch.exp(g.double()[:, None] * (i + 1)).float()[:, None, :, None]
    o = o + torch.matmul(q * since, states[:, :, :n])
    # the state after a sequence's last token: from its last chunk's start, that chunk's tokens added
    last = ((lens - 1) // C).clamp(min=0)
    rest = lens - last * C  # 0 .. C tokens of it
    b = torch.arange(B, device="cuda")
    back = (rest[:, None] - 1 - i)[:, None]  # [B, 1, C]
    w = torch.where(back >= 0, torch.exp(g.double()[:, None] * back.clamp(min=0).double()), 0.0).float()
    final = torch.matmul((k[b, :, last] * w[..., None]).transpose(-1, -2), v[b, :, last])
    final = final + torch.exp(g.double() * rest[:, None]).float()[:, :, None, None] * states[b, :, last]
    return o.reshape(B, H, n * C, d)[:, :, :L] * scale, final


def _plain_linear(s):
    c = s["case"]
    r = c["Hq"] // c["Hkv"]
    if c["form"] == "step":
        k, v = (s[x].float().repeat_interleave(r, 1) for x in "kv")
        s["state"].mul_(torch.exp(s["log_decay"].double()).float()[:, None, None]).add_(k[..., :, None] * v[..., None, :])
        o = (s["q"].float()[..., :, None] * s["state"]).sum(-2) * s["scale"]
        return {"o": o.to(s["q"].dtype), "state": s["state"]}
    if c["form"] == "dense":
        q = s["q"].float()
        k, v = (s[x].float().repeat_interleave(r, 1) for x in "kv")
        lens = torch.full((c["B"],), c["L"], device="cuda")
        o, final = _chunked(q, k, v, s["log_decay"], s["state"], s["scale"], lens)
        return {"o": o.to(s["q"].dtype), "state": final}
    cu, n = s["cu"].long(), s["longest"]
    lens = cu[1:] - cu[:-1]
    i = torch.arange(n, device="cuda")
    inside = i < lens[:, None]
    at = torch.where(inside, cu[:-1, None] + i, 0)
    rows = lambda x: torch.where(inside[..., None, None], x[at].float(), 0.0).transpose(1, 2)  # noqa: E731
    q = rows(s["q"])
    k, v = (rows(s[x]).repeat_interleave(r, 1) for x in "kv")
    o, final = _chunked(q, k, v, s["log_decay"], s["state"], s["scale"], lens)
    return {"o": o.transpose(1, 2)[inside].to(s["q"].dtype), "state": final}


_plain = {"slots": _plain_slots, "rope": _plain_rope, "append": _plain_append, "linear": _plain_linear}


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["kind"] in ("slots", "append"):
        pick = random.Random(6)
        add = [pick.randint(c["add_lo"], c["add_hi"]) for _ in range(c["B"])]
        N, real = sum(add) + c["pad"], sum(add)
        if c["kind"] == "slots":
            touched = sum(-(-n // c["page"]) for n in add)
            return {"bytes": 4.0 * (2 * c["B"] + touched + 3 * N + c["B"] + 1), "flops": 0.0}
        row = 2.0 * c["d"]
        pairs = c["rot"] // 2
        return {"bytes": row * (2 * N * c["Hq"] + 4 * real * c["Hkv"]) + 4.0 * (real + N) + 8.0 * pairs,
                "flops": 6.0 * pairs * (N * c["Hq"] + real * c["Hkv"])}
    tokens = c["B"] * c["L"]
    if c["form"] == "packed":
        pick = random.Random(6)
        tokens = sum(pick.randint(1, c["L"]) for _ in range(c["B"]))
    row, heads = 2.0 * c["d"], c["Hq"] + c["Hkv"]
    if c["kind"] == "rope":
        return {"bytes": 2 * row * tokens * heads + 4.0 * tokens + 4.0 * c["rot"], "flops": 3.0 * c["rot"] * tokens * heads}
    states = c["B"] * c["Hq"] * c["d"] * c["d"] * 4.0 * (2 if c["state"] else 1)
    # an update and a product with the state for every token: 2 d^2 multiply-adds
    return {"bytes": 2 * row * tokens * heads + states, "flops": 4.0 * tokens * c["Hq"] * c["d"] ** 2}


# --------------------------------------------------------------------------- in 64 bits, from the definition
def _rotated64(x, positions, f, interleaved, inverse):
    """The pairs as complex numbers times e^{i position f}; x [..., d], positions as x without its last dimension."""
    r, y = 2 * f.numel(), x.double()
    head = y[..., :r].reshape(*y.shape[:-1], r // 2, 2) if interleaved else \
        torch.stack((y[..., :r // 2], y[..., r // 2:r]), -1)
    angle = positions.double()[..., None] * f * (-1.0 if inverse else 1.0)
    z = torch.view_as_real(torch.view_as_complex(head.contiguous()) * torch.polar(torch.ones_like(angle), angle))
    z = z.reshape(*y.shape[:-1], r) if interleaved else torch.cat((z[..., 0], z[..., 1]), -1)
    return torch.cat((z, y[..., r:]), -1)


def _recurrence(q, k, v, decay, state, scale):
    """Token by token: q [H,L,d], k, v [H,L,d] in fp64."""
    o = torch.empty_like(q)
    S = state.double().clone()
    for t in range(q.shape[1]):
        S = S * decay + k[:, t, :, None] * v[:, t, None, :]
        o[:, t] = torch.matmul(q[:, t, None, :], S)[:, 0]
    return o * scale, S


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["kind"] == "slots":
        table, slots, positions, sequence, cu = s["block_table"].tolist(), [], [], [], [0]
        for b, (n, m) in enumerate(zip(s["seqlens"].tolist(), s["add"].tolist())):
            for p in range(n - m, n):
                slots.append(table[b][p // c["page"]] * c["page"] + p % c["page"])
                positions.append(p)
                sequence.append(b)
            cu.append(cu[-1] + m)
        rest = [0] * (s["tokens"] - len(slots))
        return {"slots": _i32(slots + [-1] * len(rest)), "positions": _i32(positions + rest), "cu": _i32(cu),
                "sequence": _i32(sequence + [-1] * len(rest))}
    if c["kind"] == "rope":
        at = s["positions"].unsqueeze(1)
        return {x: _rotated64(s[x], at.expand(s[x].shape[:-1]), s["inv_freq"], c["interleaved"], c["inverse"])
                for x in "qk"}
    if c["kind"] == "append":
        q, k = s["q"].double(), s["k"].double()
        if c["rot"]:
            at = s["positions"][:, None]
            q, k = (_rotated64(s[x], at.expand(s[x].shape[:-1]), s["inv_freq"], c["interleaved"], False) for x in "qk")
        out = {"q": q, "k_pool": s["k_pool"].double(), "v_pool": s["v_pool"].double()}
        n = s["tokens"] - c["pad"]
        at = s["slots"][:n].long()
        page, row = at // c["page"], at % c["page"]
        out["k_pool"][page, row], out["v_pool"][page, row] = k[:n], s["v"][:n].double()
        return out
    r = c["Hq"] // c["Hkv"]
    decay = torch.exp(s["log_decay"].double())[:, None, None]
    state = s["state"] if s["state"] is not None else torch.zeros(c["B"], c["Hq"], c["d"], c["d"], device="cuda")
    if c["form"] == "packed":
        o, final, at = [], [], 0
        for b, n in enumerate(s["lens"]):
            q, k, v = (s[x][at:at + n].double().transpose(0, 1) for x in "qkv")
            a, z = _recurrence(q, k.repeat_interleave(r, 0), v.repeat_interleave(r, 0), decay, state[b], s["scale"])
            o.append(a.transpose(0, 1))
            final.append(z)
            at += n
        return {"o": torch.cat(o), "state": torch.stack(final)}
    q, k, v = (s[x].double().view(c["B"], -1, c["L"], c["d"]) for x in "qkv")
    k, v = k.repeat_interleave(r, 1), v.repeat_interleave(r, 1)
    H = c["B"] * c["Hq"]
    o, final = _recurrence(*(x.reshape(H, c["L"], c["d"]) for x in (q, k, v)), decay.repeat(c["B"], 1, 1),
                           state.reshape(H, c["d"], c["d"]), s["scale"])
    return {"o": o.view(s["q"].shape), "state": final.view(c["B"], c["Hq"], c["d"], c["d"])}
