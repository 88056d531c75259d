"""Cases for the serving operators around the paged K/V cache: attention for a
tree of drafted tokens, attention with a sliding window whose first tokens stay
visible, and the upkeep of the cache's pages (forking, reserving with
copy-on-write, keeping the accepted tokens, compacting).

`own` false: the operators in plain torch, 32-bit arithmetic, rounded once at
the end.  `own` true: the same through the library's entry points.  Both take
the state `prepare` makes and return the same outputs.

Block tables: sequence b holds the first ceil(seqlens[b] / page) entries of its
row; page_refs[p] counts the table entries that hold page p (0: free).
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# --------------------------------------------------------------------------- cases
def _tree(name, B, T, Hq, Hkv, d, page, dtype, lo, hi, pages, softcap=0.0, sink=False, window=-1,
          keep=0):
    return dict(name=name, kind="tree", B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, page=page, dtype=dtype,
                lo=lo, hi=hi, pages=pages, softcap=softcap, sink=sink, window=window, keep=keep)


def _window(name, form, B, Lq, Hq, Hkv, d, page, dtype, lo, hi, pages, window, keep, softcap=0.0,
            sink=False):
    return dict(name=name, kind="window", form=form, B=B, Lq=Lq, Hq=Hq, Hkv=Hkv, d=d, page=page,
                dtype=dtype, lo=lo, hi=hi, pages=pages, window=window, keep=keep, softcap=softcap,
                sink=sink)


def _cache(name, kind, B, layers, page, Hkv, d, dtype, lo, hi, pages, T=0, most=0):
    return dict(name=name, kind=kind, B=B, layers=layers, page=page, Hkv=Hkv, d=d, dtype=dtype,
                lo=lo, hi=hi, pages=pages, T=T, most=most)


def listed():
    return [
        # one user's chat with a small draft tree: the verification step is pure latency
        _tree("tree_one_user", 1, 16, 32, 8, 128, 64, "bf16", 2000, 2000, 256),
        # the paged serving batch (64 sequences, 10240-page pool), every user with a 64-node tree
        _tree("tree_batch64", 64, 64, 32, 8, 128, 64, "bf16", 512, 8128, 10240),
        # odd everything: 3 heads per kv head, 61 nodes, 16-token pages, d = 64, capped scores, sink
        _tree("tree_odd", 7, 61, 24, 8, 64, 16, "f16", 1, 3001, 1600, softcap=30.0, sink=True),
        # long prompt through a sliding-window layer that keeps its first 4 tokens
        _window("window_prefill_8192", "dense", 2, 8192, 32, 8, 128, 0, "bf16", 8192, 8192, 0, 1023, 4),
        # packed prompts of odd lengths in one launch, d = 64, capped scores
        _window("window_varlen_odd", "varlen", 16, 0, 16, 16, 64, 0, "f16", 1, 2047, 0, 200, 5,
                softcap=30.0, sink=True),
        # single-token decode of a batch whose cache holds sink pages and a 1024-key window
        _window("window_decode_batch64", "paged", 64, 1, 32, 8, 128, 64, "bf16", 512, 8192, 10240,
                1023, 64),
        # after verification: the accepted path's rows made contiguous, one layer, few users
        _cache("accept_few", "accept", 4, 1, 64, 8, 128, "bf16", 100, 3000, 256, T=16, most=6),
        # the same for a 64-sequence batch over 16 layers of cache at once
        _cache("accept_batch64", "accept", 64, 16, 64, 8, 128, "bf16", 64, 1024, 1280, T=64, most=12),
        # one beam-search step: four beams of one prompt re-ordered, then room for a token each
        _cache("fork_beams", "fork", 4, 1, 64, 8, 128, "bf16", 700, 700, 128, T=1),
        # a 64-sequence batch re-ordered over 16 layers: the shared last pages are copied
        _cache("fork_batch64", "fork", 64, 16, 64, 8, 128, "bf16", 64, 900, 1536, T=3),
        # a small pool's holes closed, odd page bytes (96 columns of 3 heads)
        _cache("compact_small", "compact", 9, 1, 16, 3, 96, "f16", 1, 500, 300),
        # a large pool, half of it free, closed up before the pool is cut to size
        _cache("compact_pool4096", "compact", 64, 1, 64, 8, 128, "bf16", 512, 3500, 4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["tree", "tree", "window", "window", "accept", "fork", "compact"])
    d, page, dtype = rng.choice([64, 128]), rng.choice([16, 32, 64, 128, 256]), rng.choice(["bf16", "f16"])
    Hkv = rng.choice([1, 2, 4, 8])
    if kind == "tree":
        T, g = _log(rng, 1, 130), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        if Hkv * g > 64:
            g = 4
        B, hi = _log(rng, 1, 48), _log(rng, 8, 6000)
        lo = rng.randrange(0, hi)
        capped = rng.random() < 0.3
        return _case_without_name(_tree("", B, T, Hkv * g, Hkv, d, page, dtype, lo, hi,
                                        B * ((hi + T + page - 1) // page) + rng.randrange(1, 40),
                                        30.0 if capped else 0.0, rng.random() < 0.3,
                                        _log(rng, 1, 2000) if rng.random() < 0.3 else -1,
                                        rng.randrange(0, 70)))
    if kind == "window":
        form = rng.choice(["dense", "varlen", "paged", "paged"])
        g, win, keep = rng.choice([1, 2, 3, 4, 8]), _log(rng, 1, 2000), _log(rng, 1, 200)
        capped = rng.random() < 0.3
        if form == "paged":
            B, hi = _log(rng, 1, 48), _log(rng, 8, 8000)
            Lq = rng.choice([1, 1, 2, 3, rng.randrange(4, 300)])
            return _case_without_name(_window("", form, B, Lq, Hkv * g, Hkv, d, page, dtype,
                                              rng.randrange(1, hi), hi, B * ((hi + page - 1) // page) + 7,
                                              win, keep, 30.0 if capped else 0.0, rng.random() < 0.3))
        B, hi = _log(rng, 1, 6), _log(rng, 1, 2500)
        return _case_without_name(_window("", form, B, hi if form == "dense" else 0, Hkv * g, Hkv, d, 0,
                                          dtype, hi if form == "dense" else 1, hi, 0, win, keep,
                                          30.0 if capped else 0.0, rng.random() < 0.3))
    B, layers, hi = _log(rng, 1, 64), rng.choice([1, 1, 2, 5]), _log(rng, 8, 1500)
    d = rng.choice([64, 80, 96, 128])
    need = B * ((hi + 70 + page - 1) // page)
    if kind == "accept":
        T = _log(rng, 1, 64)
        return _case_without_name(_cache("", kind, B, layers, page, Hkv, d, dtype, rng.randrange(1, hi + 1),
                                         hi, need + rng.randrange(1, 30), T, rng.randrange(1, min(T, 16) + 1)))
    if kind == "fork":
        return _case_without_name(_cache("", kind, B, layers, page, Hkv, d, dtype, rng.randrange(1, hi + 1),
                                         hi, need + B + rng.randrange(1, 30), rng.choice([1, 1, 3, 17])))
    return _case_without_name(_cache("", kind, B, 1, page, Hkv, d, dtype, rng.randrange(1, hi + 1), hi,
                                     2 * need + rng.randrange(1, 50)))


def _case_without_name(c):
    return {k: v for k, v in c.items() if k != "name"}


# --------------------------------------------------------------------------- inputs
def _ints(seed, c):
    """The case's host-side integers, from the seed alone (packed sequences keep their lengths, so that the
    packed tensors keep their shapes)."""
    rng = random.Random(seed * 7919 + 13)
    pick = random.Random(4) if c.get("form") == "varlen" else rng
    lens = [pick.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    return rng, lens


def _randn(gen, shape, dtype):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat, n = out.view(-1), out.numel()
    for s in range(0, n, 1 << 27):
        e = min(n, s + (1 << 27))
        flat[s:e] = torch.randn(e - s, generator=gen, device="cuda")
    return out


def _i32(rows):
    return torch.tensor(rows, dtype=torch.int32, device="cuda")


def _table(rng, lens, page, pages, width=None):
    held = [-(-n // page) for n in lens]
    order = list(range(pages))
    rng.shuffle(order)
    width = max([1] + held) if width is None else width
    rows, at = [], 0
    for n in held:
        rows.append(order[at:at + n] + [0] * (width - n))
        at += n
    return rows


def _parents(rng, T):
    """A draft tree in index order: node 0 follows the last token, later nodes mostly extend recent ones."""
    return [-1] + [rng.randrange(max(-1, i - 9), i) for i in range(1, T)]


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng, lens = _ints(seed, c)
    dt = DTYPES[c["dtype"]]
    s = {"case": c, "page": c["page"]}
    if c["kind"] in ("tree", "window"):
        s["scale"] = 1.0 / math.sqrt(c["d"])
        s["sink"] = torch.randn(c["Hq"], generator=gen, device="cuda") if c["sink"] else None
    if c["kind"] == "tree":
        lens = [n + c["T"] for n in lens]  # the drafted tokens' K/V are in the cache already
        s["parents"] = _i32([_parents(rng, c["T"]) for _ in lens])
        Lq = c["T"]
    elif c["kind"] == "window":
        Lq = c["Lq"]
    if c["kind"] == "tree" or c.get("form") == "paged":
        s["q"] = _randn(gen, (c["B"], Lq, c["Hq"], c["d"]), dt)
        s["block_table"] = _i32(_table(rng, lens, c["page"], c["pages"]))
        s["seqlens"] = _i32(lens)
        for name in ("k_pool", "v_pool"):
            s[name] = _randn(gen, (c["pages"], c["page"], c["Hkv"], c["d"]), dt)
        return s
    if c["kind"] == "window" and c["form"] == "dense":
        s["q"] = _randn(gen, (c["B"], c["Hq"], Lq, c["d"]), dt)
        for name in "kv":
            s[name] = _randn(gen, (c["B"], c["Hkv"], Lq, c["d"]), dt)
        return s
    if c["kind"] == "window":  # packed sequences
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["cu"], s["longest"], s["lens"] = _i32(cu), max(lens), lens
        s["q"] = _randn(gen, (cu[-1], c["Hq"], c["d"]), dt)
        for name in "kv":
            s[name] = _randn(gen, (cu[-1], c["Hkv"], c["d"]), dt)
        return s
    # ------------------------------------------------------------- cache upkeep
    B, T, page = c["B"], c["T"], c["page"]
    width = -(-(c["hi"] + T) // page) + 1
    if c["kind"] == "accept":
        lens = [n + T for n in lens]
        path, path_lens = [], []
        for _ in lens:
            n = rng.randint(0, c["most"])
            path.append(sorted(rng.sample(range(T), n)) + [0] * (c["most"] - n))
            path_lens.append(n)
        s["path"], s["path_lens"] = _i32(path), _i32(path_lens)
        s["tree_lens"] = _i32([T] * B)
    if c["kind"] == "fork":
        s["index"] = _i32([rng.choice([b, rng.randrange(B), rng.randrange(B)]) for b in range(B)])
        s["add"] = _i32([T] * B)
    rows = _table(rng, lens, page, c["pages"], width)
    refs = [0] * c["pages"]
    for row, n in zip(rows, lens):
        for p in row[:-(-n // page)]:
            refs[p] += 1
    s["block_table"], s["seqlens"], s["refs"] = _i32(rows), _i32(lens), _i32(refs)
    shape = (c["pages"], page, c["Hkv"], c["d"])
    shape = shape if c["layers"] == 1 else (c["layers"],) + shape
    for name in ("k_pool", "v_pool"):
        s[name] = _randn(gen, shape, dt)
    return s


# --------------------------------------------------------------------------- one pass
def run(state):
    return (_own if own else _plain)[state["case"]["kind"]](state)


def _own_tree(s):
    import attention_forward_13_gb300 as A
    c = s["case"]
    mask, depth = A.attn_tree_mask(s["parents"])
    window = (c["window"], -1) if c["window"] >= 0 else None
    o, lse = A.attn_fwd_paged_tree(s["q"], s["k_pool"], s["v_pool"], s["block_table"], s["seqlens"],
                                   mask, tree_depth=depth, scale=s["scale"], softcap=c["softcap"],
                                   sink=s["sink"], window=window,
                                   sink_tokens=c["keep"] if window else 0)
    return {"o": o, "lse": lse, "mask": mask, "depth": depth}


def _own_window(s):
    import attention_forward_13_gb300 as A
    c = s["case"]
    kw = dict(causal=True, scale=s["scale"], softcap=c["softcap"], sink=s["sink"],
              window=(c["window"], -1), sink_tokens=c["keep"])
    if c["form"] == "dense":
        o, lse = A.attn_fwd(s["q"], s["k"], s["v"], **kw)
    elif c["form"] == "varlen":
        o, lse = A.attn_fwd_varlen(s["q"], s["k"], s["v"], s["cu"], s["cu"], s["longest"], **kw)
    else:
        o, lse = A.attn_fwd_paged(s["q"], s["k_pool"], s["v_pool"], s["block_table"], s["seqlens"], **kw)
    return {"o": o, "lse": lse}


def _own_accept(s):
    import attention_forward_13_gb300 as A
    lens, refs = A.attn_cache_accept(s["k_pool"], s["v_pool"], s["block_table"], s["seqlens"],
                                     s["refs"], s["path"], s["path_lens"], s["tree_lens"])
    return {"seqlens": lens, "refs": refs, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _own_fork(s):
    import attention_forward_13_gb300 as A
    table, lens, refs = A.attn_cache_reorder(s["block_table"], s["seqlens"], s["refs"], s["index"],
                                             s["page"])
    table, lens, refs, free = A.attn_cache_reserve(s["k_pool"], s["v_pool"], table, lens, refs, s["add"])
    return {"table": table, "seqlens": lens, "refs": refs, "free": free, "k_pool": s["k_pool"],
            "v_pool": s["v_pool"]}


def _own_compact(s):
    import attention_forward_13_gb300 as A
    table, refs, page_map = A.attn_cache_compact(s["k_pool"], s["v_pool"], s["block_table"],
                                                 s["seqlens"], s["refs"])
    return {"table": table, "refs": refs, "map": page_map, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


_own = {"tree": _own_tree, "window": _own_window, "accept": _own_accept, "fork": _own_fork,
        "compact": _own_compact}


# --------------------------------------------------------------------------- plain forms
def _attend(q, k, v, keep, scale, cap, sink, dtype):
    """Rows q [..., H, R, d] against k, v [..., H, N, d] where keep [..., 1 or H, R, N]; sink [..., H, 1]."""
    x = torch.matmul(q.float() * scale, k.float().transpose(-1, -2))
    if cap > 0:
        x = cap * torch.tanh(x / cap)
    x = torch.where(keep, x, -math.inf)
    m = x.amax(-1)
    if sink is not None:
        m = torch.maximum(m, sink)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m[..., None])
    z = p.sum(-1)
    if sink is not None:
        z = z + torch.exp(sink - m)
    o = torch.matmul(p, v.float()) / torch.where(z > 0, z, 1.0)[..., None]
    return o.to(dtype), torch.where(z > 0, m + torch.log(z), -math.inf)


def _gathered(s):
    """The sequences' keys and values [B, Hkv, N, d] in position order, rows past a sequence's end zero."""
    c, table = s["case"], s["block_table"].long()
    N = table.shape[1] * c["page"]
    j = torch.arange(N, device="cuda")
    inside = (j < s["seqlens"].long()[:, None])[:, None, :, None]
    both = []
    for name in ("k_pool", "v_pool"):
        x = s[name][table].reshape(c["B"], N, c["Hkv"], c["d"]).transpose(1, 2)
        both.append(torch.where(inside, x, torch.zeros((), dtype=x.dtype, device="cuda")))
    return both[0], both[1], j


def _grouped(x, Hkv):
    """[B, L, Hq, d] -> [B, Hkv, g * L, d], the rows of a kv head by head and position."""
    B, L, Hq, d = x.shape
    return x.view(B, L, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, (Hq // Hkv) * L, d)


def _ungrouped(o, lse, B, L, Hq, Hkv):
    g, d = Hq // Hkv, o.shape[-1]
    o = o.view(B, Hkv, g, L, d).permute(0, 3, 1, 2, 4).reshape(B, L, Hq, d)
    return o, lse.view(B, Hkv, g, L).reshape(B, Hq, L).contiguous()


def _sink_rows(s, L):
    """The sink logit of every grouped row, [Hkv, g * L]."""
    c = s["case"]
    return None if s["sink"] is None else s["sink"].view(c["Hkv"], -1, 1).expand(-1, -1, L).reshape(c["Hkv"], -1)


def _tree_relations(parents):
    """Which nodes a node sees (itself and what it descends from), and how many lie above it."""
    B, T = parents.shape
    i = torch.arange(T, device="cuda")
    sees = (parents[:, :, None] == i).float() + (i[:, None] == i).float()
    for _ in range(max(1, math.ceil(math.log2(max(2, T))))):
        sees = torch.minimum(torch.matmul(sees, sees), torch.ones((), device="cuda"))
    return sees > 0, (sees.sum(-1) - 1).to(torch.int32)


def _plain_tree(s):
    c = s["case"]
    B, T, g = c["B"], c["T"], c["Hq"] // c["Hkv"]
    sees, depth = _tree_relations(s["parents"])
    W = -(-T // 32)
    bits = torch.zeros(B, T, W * 32, dtype=torch.int64, device="cuda")
    bits[:, :, :T] = sees.long()
    words = (bits.view(B, T, W, 32) << torch.arange(32, device="cuda")).sum(-1)
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    k, v, j = _gathered(s)
    base = s["seqlens"].long() - T
    node = j - base[:, None]  # [B, N]: index in the tree, negative for the tokens before it
    keep = (node < 0)[:, None, :].expand(B, T, -1)
    if c["window"] >= 0:
        at = base[:, None] + depth.long()
        keep = keep & ((j >= at[:, :, None] - c["window"]) | (j < c["keep"]))
    drafted = torch.gather(sees, 2, node.clamp(0, T - 1)[:, None, :].expand(B, T, -1))
    keep = keep | (drafted & ((node >= 0) & (node < T))[:, None, :])
    keep = keep[:, None].expand(B, g, T, -1).reshape(B, 1, g * T, -1)
    o, lse = _attend(_grouped(s["q"], c["Hkv"]), k, v, keep, s["scale"], c["softcap"], _sink_rows(s, T),
                     s["q"].dtype)
    o, lse = _ungrouped(o, lse, B, T, c["Hq"], c["Hkv"])
    return {"o": o, "lse": lse, "mask": words, "depth": depth}


def _plain_window(s):
    c = s["case"]
    B, g = c["B"], c["Hq"] // c["Hkv"]
    if c["form"] == "paged":
        k, v, j = _gathered(s)
        Lq = c["Lq"]
        at = s["seqlens"].long()[:, None] - Lq + torch.arange(Lq, device="cuda")
        keep = (j <= at[:, :, None]) & ((j >= at[:, :, None] - c["window"]) | (j < c["keep"]))
        keep = keep[:, None].expand(B, g, Lq, -1).reshape(B, 1, g * Lq, -1)
        o, lse = _attend(_grouped(s["q"], c["Hkv"]), k, v, keep, s["scale"], c["softcap"],
                         _sink_rows(s, Lq), s["q"].dtype)
        o, lse = _ungrouped(o, lse, B, Lq, c["Hq"], c["Hkv"])
        return {"o": o, "lse": lse}
    if c["form"] == "dense":
        q, k, v, spans = s["q"], s["k"], s["v"], None
        n = c["Lq"]
        i = torch.arange(n, device="cuda")
        keep = (i <= i[:, None]) & ((i >= i[:, None] - c["window"]) | (i < c["keep"]))
        sink = None if s["sink"] is None else s["sink"][:, None]
        o, lse = _attend(q, k.repeat_interleave(g, 1), v.repeat_interleave(g, 1), keep, s["scale"],
                         c["softcap"], sink, q.dtype)
        return {"o": o, "lse": lse}
    o, lse, at = [], [], 0
    sink = None if s["sink"] is None else s["sink"][:, None]
    for n in s["lens"]:
        q, k, v = (s[x][at:at + n].transpose(0, 1) for x in "qkv")
        i = torch.arange(n, device="cuda")
        keep = (i <= i[:, None]) & ((i >= i[:, None] - c["window"]) | (i < c["keep"]))
        a, b = _attend(q, k.repeat_interleave(g, 0), v.repeat_interleave(g, 0), keep, s["scale"],
                       c["softcap"], sink, q.dtype)
        o.append(a.transpose(0, 1))
        lse.append(b)
        at += n
    return {"o": torch.cat(o), "lse": torch.cat(lse, 1)}


def _holds(lens, page, width):
    """[B, width]: which entries of a table with these lengths hold a page."""
    return torch.arange(width, device="cuda") < ((lens.long() + page - 1) // page)[:, None]


def _count(table, held, pages):
    """How many held entries of the table name each page."""
    n = torch.zeros(pages, dtype=torch.int32, device="cuda")
    return n.index_add_(0, table.long().clamp(0, pages - 1).view(-1), held.to(torch.int32).view(-1))


def _layered(pool):
    return pool if pool.dim() == 5 else pool[None]


def _plain_accept(s):
    c = s["case"]
    B, page, table = c["B"], c["page"], s["block_table"].long()
    lens, tree, n = s["seqlens"].long(), s["tree_lens"].long(), s["path_lens"].long()
    base = lens - tree
    i = torch.arange(s["path"].shape[1], device="cuda")
    taken = i < n[:, None]
    to = base[:, None] + i
    fro = torch.where(taken, base[:, None] + s["path"].long(), to)
    rows = lambda at: torch.gather(table, 1, at // page) * page + at % page  # noqa: E731
    to, fro = rows(to).view(-1), rows(fro).view(-1)
    for name in ("k_pool", "v_pool"):
        pool = _layered(s[name])
        flat = pool.view(pool.shape[0], pool.shape[1] * page, c["Hkv"], c["d"])
        flat[:, to] = flat[:, fro]
    new = base + n
    width = table.shape[1]
    dropped = _holds(lens, page, width) & ~_holds(new, page, width)
    refs = s["refs"] - _count(table, dropped, s["refs"].numel())
    return {"seqlens": new.to(torch.int32), "refs": refs, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _free_list(refs):
    """The free pages in rising order, and their number."""
    free = refs == 0
    pages = refs.numel()
    at = torch.where(free, torch.cumsum(free, 0) - 1, pages)
    out = torch.zeros(pages + 1, dtype=torch.int64, device="cuda")
    out[at] = torch.arange(pages, device="cuda")
    return out, free.sum()


def _plain_fork(s):
    page, pages = s["page"], s["refs"].numel()
    old, index = s["block_table"], s["index"].long()
    width = old.shape[1]
    lens = s["seqlens"][index]
    held = _holds(lens, page, width)
    table = torch.where(held, old[index], -1)
    refs = s["refs"] + _count(table, held, pages) - _count(old, _holds(s["seqlens"], page, width), pages)
    # room for the new tokens; a partly filled last page that others hold too is copied first
    n, add = lens.long(), s["add"].long()
    has, want = (n + page - 1) // page, (n + add + page - 1) // page
    last = torch.gather(table.long(), 1, (has - 1).clamp(0)[:, None])[:, 0]
    part = (n % page != 0) & (add > 0)
    same = (last[:, None] == last) & part[:, None] & part
    b = torch.arange(n.numel(), device="cuda")
    before = (same & (b < b[:, None])).sum(1)  # lower sequences that leave the page first
    copied = part & (refs.long()[last.clamp(0)] - before > 1)
    need = want - has + copied
    start = torch.cumsum(need, 0) - need
    free, count = _free_list(refs)
    col = torch.arange(width, device="cuda")
    first = has - copied.long()
    fresh = (col >= first[:, None]) & (col < want[:, None])
    page_of = free[(start[:, None] + col - first[:, None]).clamp(0, pages - 1)]
    grown = torch.where(fresh, page_of, table.long()).to(torch.int32)
    new = torch.where(copied, torch.gather(grown.long(), 1, first.clamp(0)[:, None])[:, 0], last)
    for name in ("k_pool", "v_pool"):
        pool = _layered(s[name])
        src, dst = torch.where(copied, last, new), new
        pool[:, dst] = pool[:, src]
    out = refs + _count(grown, fresh, pages) - _count(last[:, None], copied[:, None], pages)
    return {"table": grown, "seqlens": (n + add).to(torch.int32), "refs": out,
            "free": (count - need.sum()).to(torch.int32).view(1), "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _plain_compact(s):
    c = s["case"]
    refs, table = s["refs"], s["block_table"]
    pages = refs.numel()
    p = torch.arange(pages, device="cuda")
    live = refs > 0
    n = live.sum()
    hole, moved = ~live & (p < n), live & (p >= n)
    spare = torch.full((), pages, device="cuda")
    src = torch.zeros(pages + 1, dtype=torch.int64, device="cuda")
    src[torch.where(moved, torch.cumsum(moved, 0) - 1, spare)] = p
    dst = torch.zeros(pages + 1, dtype=torch.int64, device="cuda")
    dst[torch.where(hole, torch.cumsum(hole, 0) - 1, spare)] = p
    come = torch.where(hole, src[(torch.cumsum(hole, 0) - 1).clamp(0)], p)  # what each page holds afterwards
    go = torch.where(moved, dst[(torch.cumsum(moved, 0) - 1).clamp(0)], torch.where(live, p, -1))
    for name in ("k_pool", "v_pool"):
        pool = _layered(s[name])
        pool.copy_(pool[:, come])
    held = _holds(s["seqlens"], c["page"], table.shape[1])
    out = torch.where(held, go[table.long().clamp(0, pages - 1)], -1).to(torch.int32)
    after = torch.where(p < n, refs[come], 0)
    return {"table": out, "refs": after, "map": go.to(torch.int32), "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


_plain = {"tree": _plain_tree, "window": _plain_window, "accept": _plain_accept, "fork": _plain_fork,
          "compact": _plain_compact}


# --------------------------------------------------------------------------- what a pass cannot do without
def _mean_kept(n_rows, total, window, keep):
    """Pairs (row, key) kept by a causal window with visible first tokens: rows are the last n_rows of total."""
    pairs = 0
    for i in range(total - n_rows, total):
        lo = max(0, i - window)
        pairs += i + 1 - lo + min(keep, lo)
    return pairs


def work(case):
    c = case
    rng, lens = _ints(1, c)
    eb = 2
    if c["kind"] == "tree":
        rows = c["B"] * c["T"] * c["Hq"]
        total, pairs = 0, 0
        for n in lens:
            first = 0 if c["window"] < 0 else max(0, n - c["window"])
            seen = n - first + (min(c["keep"], first) if c["window"] >= 0 else 0)
            total += seen + c["T"]
            pairs += c["T"] * seen + 4 * c["T"]
        return {"bytes": total * c["Hkv"] * c["d"] * 2 * eb + rows * c["d"] * 2 * eb + rows * 4,
                "flops": 4.0 * pairs * c["Hq"] * c["d"]}
    if c["kind"] == "window":
        if c["form"] == "paged":
            pairs = sum(_mean_kept(min(c["Lq"], n), n, c["window"], c["keep"]) for n in lens)
            seen = 0
            for n in lens:
                first = max(0, n - c["Lq"] - c["window"])
                seen += n - first + min(c["keep"], first)
            rows = c["B"] * c["Lq"] * c["Hq"]
        else:
            pairs = sum(_mean_kept(n, n, c["window"], c["keep"]) for n in lens)
            seen = sum(lens)
            rows = seen * c["Hq"]
        return {"bytes": seen * c["Hkv"] * c["d"] * 2 * eb + rows * c["d"] * 2 * eb + rows * 4,
                "flops": 4.0 * pairs * c["Hq"] * c["d"]}
    token = c["Hkv"] * c["d"] * 2 * eb * c["layers"]
    small = 4 * (2 * c["pages"] + 2 * sum(-(-n // c["page"]) for n in lens))
    if c["kind"] == "accept":
        return {"bytes": 2 * token * c["B"] * c["most"] / 2 + small, "flops": 0}
    if c["kind"] == "fork":  # about half of the sequences come to share a partly filled page
        return {"bytes": 2 * token * c["page"] * max(1, c["B"] // 2) + small, "flops": 0}
    held = sum(-(-n // c["page"]) for n in lens)
    move = held * (1 - held / c["pages"])  # live pages beyond the first `held`, on average
    return {"bytes": 2 * token * c["page"] * move + small, "flops": 0}


# --------------------------------------------------------------------------- 64 bits
def _rows64(q, k, v, keep, scale, cap, sink):
    """One head: q [R, d], k/v [N, d], keep [R, N] in 64 bits."""
    x = (q @ k.T) * scale
    if cap > 0:
        x = cap * torch.tanh(x / cap)
    x = x.masked_fill(~keep, -math.inf)
    if sink is not None:
        x = torch.cat([x, sink.double().expand(x.shape[0], 1)], 1)
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
    p = p if sink is None else p[:, :-1]
    return p @ v, lse


def _exact_seq(c, s, b, q, k, v, keep):
    """All heads of one sequence: q [L, Hq, d], k/v [N, Hkv, d], keep [L, N] -> o [L, Hq, d], lse [Hq, L]."""
    g = c["Hq"] // c["Hkv"]
    used = keep.any(0)
    k, v, keep = k[used].double(), v[used].double(), keep[:, used]
    o, lse = [], []
    for h in range(c["Hq"]):
        a, z = _rows64(q[:, h].double(), k[:, h // g], v[:, h // g], keep, s["scale"], c["softcap"],
                       None if s["sink"] is None else s["sink"][h])
        o.append(a)
        lse.append(z)
    return torch.stack(o, 1), torch.stack(lse)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["kind"] == "tree":
        o, lse, masks, depths = [], [], [], []
        parents, T = s["parents"].tolist(), c["T"]
        for b in range(c["B"]):
            n = int(s["seqlens"][b])
            base = n - T
            sees = torch.zeros(T, T, dtype=torch.bool)
            depth = []
            for i, p in enumerate(parents[b]):
                if p >= 0:
                    sees[i] = sees[p]
                sees[i, i] = True
                depth.append(depth[p] + 1 if p >= 0 else 0)
            keep = torch.ones(T, n, dtype=torch.bool)
            keep[:, base:] = sees
            if c["window"] >= 0:
                j = torch.arange(base)
                at = base + torch.tensor(depth)
                keep[:, :base] = (j >= at[:, None] - c["window"]) | (j < c["keep"])
            ids = s["block_table"][b, :-(-n // c["page"])].long()
            k, v = (s[x][ids].reshape(-1, c["Hkv"], c["d"])[:n] for x in ("k_pool", "v_pool"))
            a, z = _exact_seq(c, s, b, s["q"][b], k, v, keep.cuda())
            o.append(a)
            lse.append(z)
            words = []
            for i in range(T):
                row = [0] * -(-T // 32)
                for m in sees[i].nonzero().view(-1).tolist():
                    row[m // 32] |= 1 << (m % 32)
                words.append([x - (1 << 32) if x >= 1 << 31 else x for x in row])
            masks.append(words)
            depths.append(depth)
        return {"o": torch.stack(o), "lse": torch.stack(lse), "mask": _i32(masks), "depth": _i32(depths)}
    if c["kind"] == "window":
        if c["form"] == "dense":
            seqs = [(c["Lq"], *(s[x][b].transpose(0, 1) for x in "qkv")) for b in range(c["B"])]
        elif c["form"] == "varlen":
            seqs, at = [], 0
            for n in s["lens"]:
                seqs.append((n, *(s[x][at:at + n] for x in "qkv")))
                at += n
        else:
            seqs = []
            for b in range(c["B"]):
                n = int(s["seqlens"][b])
                ids = s["block_table"][b, :-(-n // c["page"])].long()
                k, v = (s[x][ids].reshape(-1, c["Hkv"], c["d"])[:n] for x in ("k_pool", "v_pool"))
                seqs.append((n, s["q"][b], k, v))
        o, lse = [], []
        for b, (n, q, k, v) in enumerate(seqs):
            L, parts = q.shape[0], []
            for r in range(0, L, 1024):  # blocks of rows against the keys some row of them keeps
                i = torch.arange(r, min(r + 1024, L), device="cuda")[:, None] + (n - L)
                j = torch.arange(n, device="cuda")
                keep = (j <= i) & ((j >= i - c["window"]) | (j < c["keep"]))
                parts.append(_exact_seq(c, s, b, q[r:r + 1024], k, v, keep))
            o.append(torch.cat([p[0] for p in parts]))
            lse.append(torch.cat([p[1] for p in parts], 1))
        if c["form"] == "varlen":
            return {"o": torch.cat(o), "lse": torch.cat(lse, 1)}
        o = torch.stack(o)
        return {"o": o.transpose(1, 2) if c["form"] == "dense" else o, "lse": torch.stack(lse)}
    # ------------------------------------------------- cache upkeep: the whole numbers, on the host
    page = c["page"]
    table, lens, refs = s["block_table"].tolist(), s["seqlens"].tolist(), s["refs"].tolist()
    pages = lambda n: -(-n // page)  # noqa: E731
    if c["kind"] == "accept":
        tree, took = s["tree_lens"].tolist(), s["path_lens"].tolist()
        for b, n in enumerate(lens):
            new = n - tree[b] + took[b]
            for p in table[b][pages(new):pages(n)]:
                refs[p] -= 1
            lens[b] = new
        return {"seqlens": _i32(lens), "refs": _i32(refs), "k_pool": None, "v_pool": None}
    if c["kind"] == "fork":
        index, add, width = s["index"].tolist(), s["add"].tolist(), len(table[0])
        rows = [table[i][:pages(lens[i])] for i in index]
        for row in rows:
            for p in row:
                refs[p] += 1
        for b, n in enumerate(lens):
            for p in table[b][:pages(n)]:
                refs[p] -= 1
        lens = [lens[i] for i in index]
        free = iter([p for p, r in enumerate(refs) if r == 0])
        left, out = sum(r == 0 for r in refs), list(refs)
        for b, row in enumerate(rows):
            if lens[b] % page and add[b] > 0 and refs[row[-1]] > 1:
                refs[row[-1]] -= 1
                out[row[-1]] -= 1
                row.pop()
            while len(row) < pages(lens[b] + add[b]):
                row.append(next(free))
                out[row[-1]] += 1
                left -= 1
            row += [-1] * (width - len(row))
        return {"table": _i32(rows), "seqlens": _i32([n + a for n, a in zip(lens, add)]), "refs": _i32(out),
                "free": _i32([left]), "k_pool": None, "v_pool": None}
    n = sum(r > 0 for r in refs)
    holes = iter([p for p in range(n) if refs[p] == 0])
    go = [(-1 if r == 0 else p if p < n else next(holes)) for p, r in enumerate(refs)]
    after = [0] * len(refs)
    for p, to in enumerate(go):
        if to >= 0:
            after[to] = refs[p]
    rows = [[go[p] if i < pages(lens[b]) else -1 for i, p in enumerate(row)] for b, row in enumerate(table)]
    return {"table": _i32(rows), "refs": _i32(after), "map": _i32(go), "k_pool": None, "v_pool": None}
