"""Upkeep of the paged cache (attn_cache_reorder, _reserve, _accept, _compact) against
the rules on Python lists: every table entry, count, length and pool byte is
compared.  Then a run of all of them with the tree attention, as a serving loop
uses them, eager, captured and on a side stream."""
import math

import numpy as np
import pytest
import torch

import attention_forward_13_gb300 as A
from tests import _cache_plain as P
from tests import _masked as M
from tests._parity import check, f64, no_device_error

gpu = pytest.mark.gpu


class Cache:
    """A random cache state on the host and on the GPU."""

    def __init__(self, rng, lens, page, spare, width=None, layers=1, Hkv=2, d=64, dtype=torch.bfloat16,
                 forks=0):
        held = [P.pages(n, page) for n in lens]
        self.page, self.num = page, sum(held) + spare
        order = rng.permutation(self.num).tolist()
        self.rows, at = [], 0
        for n in held:
            self.rows.append(order[at:at + n])
            at += n
        self.lens = list(lens)
        self.refs = [0] * self.num
        for row in self.rows:
            for p in row:
                self.refs[p] += 1
        if forks:  # some sequences share everything with another
            index = [int(rng.integers(0, len(lens))) if rng.random() < forks else b for b in range(len(lens))]
            self.rows, self.lens, self.refs = P.reorder(self.rows, self.lens, self.refs, index, page)
        self.width = max([1] + [len(r) for r in self.rows]) if width is None else width
        shape = (layers, self.num, page, Hkv, d)
        self.pools = [torch.randint(0, 256, shape + (dtype.itemsize,), dtype=torch.uint8,
                                    generator=torch.Generator().manual_seed(int(rng.integers(1 << 30))))
                      for _ in range(2)]
        self.dtype, self.layers = dtype, layers

    def table(self, junk=0):
        return torch.tensor([r + [junk] * (self.width - len(r)) for r in self.rows],
                            dtype=torch.int32).reshape(-1, self.width)

    def gpu(self):
        pools = [p.cuda().view(self.dtype).squeeze(-1) for p in self.pools]
        if self.layers == 1:
            pools = [p[0] for p in pools]
        ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (self.lens, self.refs)]
        return pools, self.table(junk=1 << 20).cuda(), ints[0], ints[1]

    def np_pools(self):
        return [p.numpy().copy().reshape(*p.shape[:3], -1) for p in self.pools]


def raw(pool, like):
    return pool.contiguous().view(torch.uint8).cpu().numpy().reshape(like.shape)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def same_table(got, rows):
    want = [r + [-1] * (got.shape[1] - len(r)) for r in rows]
    assert got.tolist() == want


STATES = [
    # lens, page, spare, layers, Hkv, d, dtype, forks
    ([5], 16, 3, 1, 1, 64, torch.bfloat16, 0.0),
    ([100, 1, 0, 257, 64], 64, 9, 1, 8, 128, torch.bfloat16, 0.6),
    ([33, 500, 17, 16, 31, 2], 16, 40, 3, 3, 80, torch.float16, 0.5),
    ([700, 513, 0, 256], 256, 4, 2, 2, 64, torch.float8_e4m3fn, 0.3),
    ([7 * (i % 13) for i in range(300)], 32, 300, 1, 1, 64, torch.bfloat16, 0.4),
    ([20000, 3, 19999], 16, 3000, 1, 1, 16, torch.float16, 0.0),
    ([300] * 40, 16, 9000, 1, 1, 8, torch.float16, 0.0),   # more pages than one counting range
    ([40000, 7] * 20, 16, 300, 1, 1, 8, torch.float16, 0.2),  # a table that several CTAs write
]
IDS = [str(i) for i in range(len(STATES))]


def make(state, seed, **kw):
    lens, page, spare, layers, Hkv, d, dtype, forks = state
    return Cache(np.random.default_rng(seed), lens, page, spare, layers=layers, Hkv=Hkv, d=d, dtype=dtype,
                 forks=forks, **kw)


@gpu
@pytest.mark.parametrize("state", STATES, ids=IDS)
def test_reorder(state):
    rng = np.random.default_rng(3)
    c = make(state, 1)
    B = len(c.lens)
    _, table, lens, refs = c.gpu()
    for n in (B, 1, 2 * B, 0):
        index = [int(rng.integers(-1, B)) for _ in range(n)]
        t, l, r = A.attn_cache_reorder(table, lens, refs, i32(index), c.page)
        rows, wl, wr = P.reorder(c.rows, c.lens, c.refs, index, c.page)
        assert l.tolist() == wl and r.tolist() == wr
        same_table(t, rows)
    no_device_error()


@gpu
@pytest.mark.parametrize("state", STATES, ids=IDS)
def test_reserve(state):
    rng = np.random.default_rng(4)
    c = make(state, 2)
    c.width += 20
    pools, table, lens, refs = c.gpu()
    B = len(c.lens)
    for most in (1, 40):
        add = [int(rng.integers(0, most + 1)) for _ in range(B)]
        host = c.np_pools()
        rows, wl, wr, free = P.reserve(host, c.rows, c.lens, c.refs, add, c.page, c.width)
        t, l, r, f = A.attn_cache_reserve(*pools, table, lens, refs, i32(add))
        assert f.tolist() == [free] and l.tolist() == wl and r.tolist() == wr
        same_table(t, rows)
        for pool, want in zip(pools, host):
            assert np.array_equal(raw(pool, want), want)
        if free >= 0:  # go on from the new state
            c.rows, c.lens, c.refs = rows, wl, wr
            c.pools = [torch.from_numpy(h.reshape(p.shape)) for h, p in zip(host, c.pools)]
            table, lens, refs = t, l, r
    no_device_error()


@gpu
def test_reserve_is_all_or_nothing():
    c = make(STATES[1], 5)
    c.width += 30
    pools, table, lens, refs = c.gpu()
    before = [p.clone() for p in pools]
    t, l, r, f = A.attn_cache_reserve(*pools, table, lens, refs, i32([1, 1, 1500, 1, 1]))
    want = P.reserve(c.np_pools(), c.rows, c.lens, c.refs, [1, 1, 1500, 1, 1], c.page, c.width)
    assert f.item() == want[3] and -c.num <= f.item() < 0
    same_table(t, c.rows)
    assert l.tolist() == c.lens and r.tolist() == c.refs
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(pools, before))
    no_device_error()
    t, l, r, f = A.attn_cache_reserve(*pools, table, lens, refs, i32([0, 0, 64 * 40, 0, 0]))  # outgrows its row
    assert f.item() == -c.num - 1 and l.tolist() == c.lens and r.tolist() == c.refs
    assert A.attn_device_error() == 1 << 25


@gpu
@pytest.mark.parametrize("state", STATES, ids=IDS)
def test_accept(state):
    rng = np.random.default_rng(6)
    c = make(state[:-1] + (0.0,), 7)
    pools, table, lens, refs = c.gpu()
    most = 0
    tree = [int(rng.integers(0, min(n, 70) + 1)) for n in c.lens]
    path = []
    for t in tree:
        path.append(sorted(rng.choice(t, size=int(rng.integers(0, t + 1)), replace=False).tolist()))
        most = max(most, len(path[-1]))
    host = c.np_pools()
    wl, wr = P.accept(host, c.rows, c.lens, c.refs, path, tree, c.page)
    padded = i32([p + [1 << 20] * (most - len(p)) for p in path]).reshape(len(path), most)
    l, r = A.attn_cache_accept(*pools, table, lens, refs, padded, i32([len(p) for p in path]), i32(tree))
    assert l.tolist() == wl and r.tolist() == wr
    for pool, want in zip(pools, host):
        assert np.array_equal(raw(pool, want), want)
    no_device_error()


@gpu
def test_accept_ends_a_bad_path():
    c = make(STATES[1][:-1] + (0.0,), 8)
    pools, table, lens, refs = c.gpu()
    tree = [8, 1, 0, 8, 8]
    path = [[1, 3, 3, 4], [0, 5, 0, 0], [0, 0, 0, 0], [2, -1, 5, 6], [0, 2, 9, 0]]
    good = [[1, 3], [0], [], [2], [0, 2]]
    host = c.np_pools()
    wl, wr = P.accept(host, c.rows, c.lens, c.refs, good, tree, c.page)
    l, r = A.attn_cache_accept(*pools, table, lens, refs, i32(path), i32([4, 2, 1, 4, 4]), i32(tree))
    assert l.tolist() == wl and r.tolist() == wr
    assert np.array_equal(raw(pools[0], host[0]), host[0])
    assert A.attn_device_error() == 1 << 25


@gpu
@pytest.mark.parametrize("state", STATES, ids=IDS)
def test_compact(state):
    c = make(state, 9)
    rng = np.random.default_rng(10)
    for p in rng.integers(0, c.num, 3):  # pages that something outside the table holds
        c.refs[int(p)] += 2
    pools, table, lens, refs = c.gpu()
    host = c.np_pools()
    rows, wr, go = P.compact(host, c.rows, c.lens, c.refs, c.page)
    t, r, m = A.attn_cache_compact(*pools, table, lens, refs)
    assert r.tolist() == wr and m.tolist() == go
    same_table(t, rows)
    live = sum(x > 0 for x in wr)
    for pool, want in zip(pools, host):  # what free pages hold is nobody's business
        assert np.array_equal(raw(pool, want)[:, :live], want[:, :live])
    no_device_error()


@gpu
@pytest.mark.parametrize("num", [1, 9, 8191, 8192, 8193, 20000])  # around what one block's registers hold
@pytest.mark.parametrize("live", [0.0, 0.03, 0.5, 0.97, 1.0])
def test_compact_pool_sizes(num, live):
    rng = np.random.default_rng(num)
    refs = [int(rng.integers(1, 4)) if rng.random() < live else 0 for _ in range(num)]
    pools = [torch.from_numpy(rng.integers(0, 1 << 15, (num, 16, 1, 8)).astype(np.int16)).view(torch.float16).cuda()
             for _ in range(2)]
    host = [pool.view(torch.uint8).cpu().numpy().reshape(1, num, 16, -1).copy() for pool in pools]
    held = [p for p in range(num) if refs[p] > 0][-3:]
    rows, wr, go = P.compact(host, [held], [16 * len(held)], refs, 16)
    table = i32([held + [1 << 20] * (4 - len(held))])
    t, r, m = A.attn_cache_compact(*pools, table, i32([16 * len(held)]), i32(refs))
    assert r.tolist() == wr and m.tolist() == go
    same_table(t, rows)
    n = sum(x > 0 for x in wr)
    for pool, want in zip(pools, host):
        assert np.array_equal(raw(pool, want)[:, :n], want[:, :n])
    no_device_error()


@gpu
@pytest.mark.parametrize("B", [1025, 2600, 8192])  # past one block of threads; the most there may be
def test_many_sequences(B):
    rng = np.random.default_rng(B)
    c = Cache(rng, [int(n) for n in rng.integers(0, 70, B)], 16, 2 * B, Hkv=1, d=8, dtype=torch.float16)
    c.width += 2
    pools, table, lens, refs = c.gpu()
    index = [int(i) for i in rng.integers(-1, B, B)]  # (about a third share their pages)
    table, lens, refs = A.attn_cache_reorder(table, lens, refs, i32(index), c.page)
    rows, wl, wr = P.reorder(c.rows, c.lens, c.refs, index, c.page)
    assert lens.tolist() == wl and refs.tolist() == wr
    same_table(table, rows)
    add = [int(n) for n in rng.integers(0, 9, B)]
    host = c.np_pools()
    rows, wl, wr, free = P.reserve(host, rows, wl, wr, add, c.page, c.width)
    assert free >= 0
    table, lens, refs, f = A.attn_cache_reserve(*pools, table, lens, refs, i32(add))
    assert f.tolist() == [free] and lens.tolist() == wl and refs.tolist() == wr
    same_table(table, rows)
    for pool, want in zip(pools, host):
        assert np.array_equal(raw(pool, want), want)
    path = [sorted(rng.permutation(n)[:int(rng.integers(0, n + 1))].tolist()) for n in add]
    width = max(len(x) for x in path)
    wl, wr = P.accept(host, rows, wl, wr, path, add, c.page)
    lens, refs = A.attn_cache_accept(*pools, table, lens, refs, i32([x + [0] * (width - len(x)) for x in path]),
                                     i32([len(x) for x in path]), i32(add))
    assert lens.tolist() == wl and refs.tolist() == wr
    for pool, want in zip(pools, host):
        assert np.array_equal(raw(pool, want), want)
    no_device_error()


@gpu
def test_a_cache_without_sequences():
    """Pages that only something outside the table holds."""
    refs = i32([0, 2, 0, 0, 1, 1])
    pools = [torch.arange(6 * 16 * 8, dtype=torch.float16, device="cuda").view(6, 16, 1, 8) + i for i in (0, 1)]
    before = [p.clone() for p in pools]
    table, lens, none = i32([]).view(0, 4), i32([]), i32([])
    t, l, r = A.attn_cache_reorder(table, lens, refs, none, 16)
    assert t.shape == (0, 4) and torch.equal(r, refs)
    t, l, r, f = A.attn_cache_reserve(*pools, table, lens, refs, none)
    assert f.item() == 3 and torch.equal(r, refs)
    l, r = A.attn_cache_accept(*pools, table, lens, refs, i32([]).view(0, 2), none, none)
    assert torch.equal(r, refs)
    t, r, m = A.attn_cache_compact(*pools, table, lens, refs)
    assert r.tolist() == [1, 2, 1, 0, 0, 0] and m.tolist() == [-1, 1, -1, -1, 0, 2]
    for new, old in zip(pools, before):
        assert torch.equal(new[:3], old[[4, 1, 5]])
    no_device_error()


@gpu
def test_two_streams_at_once():
    """Calls on two streams, named by argument, with nothing ordering them: each its own state."""
    caches = [make(STATES[1], 20 + i) for i in range(2)]
    for c in caches:
        c.width += 4
    streams = [torch.cuda.Stream() for _ in caches]
    states = [c.gpu() for c in caches]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for c, s, (pools, table, lens, refs) in zip(caches, streams, states):
            t, l, r = A.attn_cache_reorder(table, lens, refs, i32(list(range(len(c.lens)))[::-1]), c.page, stream=s)
            got.append((t, l, r))
    torch.cuda.synchronize()
    for i, (t, l, r) in enumerate(got):
        c = caches[i % 2]
        rows, wl, wr = P.reorder(c.rows, c.lens, c.refs, list(range(len(c.lens)))[::-1], c.page)
        same_table(t, rows)
        assert l.tolist() == wl and r.tolist() == wr
    no_device_error()


@gpu
def test_bad_indices_are_reported_not_followed():
    c = make(STATES[1], 11)
    _, table, lens, refs = c.gpu()
    t, l, r = A.attn_cache_reorder(table, lens, refs, i32([7, 0, -2]), c.page)
    rows, wl, wr = P.reorder(c.rows, c.lens, c.refs, [-1, 0, -1], c.page)
    same_table(t, rows)
    assert l.tolist() == wl and r.tolist() == wr and A.attn_device_error() == 1 << 25
    pools, table, lens, refs = c.gpu()
    table[0, 0] = c.num  # a held entry outside the pool
    t, r, m = A.attn_cache_compact(*pools, table, lens, refs)
    assert t[0, 0].item() == -1 and A.attn_device_error() == 1 << 25


class Model:
    """Every sequence's K and V rows on the host, beside the cache on the GPU."""

    def __init__(self, B, Hkv, d):
        self.k, self.v = [torch.zeros(0, Hkv, d) for _ in range(B)], [torch.zeros(0, Hkv, d) for _ in range(B)]


def write_rows(pool, table, lens, rows, page):
    """The new tokens' rows into their places: rows [B, n, Hkv, d] behind position lens - n."""
    n = rows.shape[1]
    pos = lens.long()[:, None] - n + torch.arange(n, device="cuda")
    slot = torch.gather(table.long(), 1, pos // page) * page + pos % page
    pool.view(-1, *pool.shape[2:])[slot.view(-1)] = rows.reshape(-1, *rows.shape[2:])


@gpu
@pytest.mark.parametrize("mode", ["eager", "graph", "stream"])
def test_speculative_decoding_run(mode):
    """Fork, reserve, write drafts, mask, tree attention, accept, compact, several rounds: each
    attention against the definition on the host's own copy of the rows."""
    B, T, Hq, Hkv, d, page, num, width, Amax = 4, 9, 8, 2, 64, 16, 160, 24, 4
    rng = np.random.default_rng(12)
    gen = torch.Generator().manual_seed(5)
    bf = lambda *s: torch.randn(*s, generator=gen).bfloat16()  # noqa: E731
    prompt = [37, 3, 64, 90]
    kp, vp = (torch.full((num, page, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    lens, refs = i32([0] * B), i32([0] * num)
    host_k, host_v = [], []
    # the prompts, one reserve for all
    table, lens, refs, free = A.attn_cache_reserve(kp, vp, table, lens, refs, i32(prompt))
    assert free.item() == num - sum(P.pages(n, page) for n in prompt)
    for b, n in enumerate(prompt):
        k, v = bf(1, n, Hkv, d), bf(1, n, Hkv, d)
        for pool, x in ((kp, k), (vp, v)):
            write_rows(pool, table[b:b + 1], lens[b:b + 1], x.cuda(), page)
        host_k.append(k[0])
        host_v.append(v[0])
    side = torch.cuda.Stream() if mode == "stream" else torch.cuda.current_stream()

    # one captured step's inputs and state
    st = dict(index=i32([0] * B), k=torch.empty(B, T, Hkv, d, dtype=torch.bfloat16, device="cuda"),
              v=torch.empty(B, T, Hkv, d, dtype=torch.bfloat16, device="cuda"),
              q=torch.empty(B, T, Hq, d, dtype=torch.bfloat16, device="cuda"),
              parents=i32([[-1] * T] * B), path=i32([[0] * Amax] * B), n=i32([0] * B), tree=i32([T] * B),
              add=i32([T] * B), table=table, lens=lens, refs=refs)

    def step():
        t, l, r = A.attn_cache_reorder(st["table"], st["lens"], st["refs"], st["index"], page)
        t, l, r, f = A.attn_cache_reserve(kp, vp, t, l, r, st["add"])
        write_rows(kp, t, l, st["k"], page)
        write_rows(vp, t, l, st["v"], page)
        mask, depth = A.attn_tree_mask(st["parents"])
        o, lse = A.attn_fwd_paged_tree(st["q"], kp, vp, t, l, mask, tree_depth=depth)
        l, r = A.attn_cache_accept(kp, vp, t, l, r, st["path"], st["n"], st["tree"])
        t, r, m = A.attn_cache_compact(kp, vp, t, l, r)
        for name, x in (("table", t), ("lens", l), ("refs", r)):
            st[name].copy_(x)
        return o, lse, f

    graph = None
    for rnd in range(4):
        index = [0, 1, 2, 3] if rnd == 0 else [int(rng.integers(0, B)) for _ in range(B)]
        k, v, q = bf(B, T, Hkv, d), bf(B, T, Hkv, d), bf(B, T, Hq, d)
        parents = [[-1] + [int(rng.integers(-1, i)) for i in range(1, T)] for _ in range(B)]
        path, n = [], []
        for b in range(B):  # from a random node up to its root
            x, up = int(rng.integers(0, T)), []
            while x >= 0:
                up.append(x)
                x = parents[b][x]
            up = up[::-1][:Amax] if rnd != 2 or b else []
            n.append(len(up))
            path.append(up + [0] * (Amax - len(up)))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for name, x in (("index", index), ("parents", parents), ("path", path), ("n", n)):
                st[name].copy_(torch.tensor(x, dtype=torch.int32))
            for name, x in (("k", k), ("v", v), ("q", q)):
                st[name].copy_(x)
            if mode != "graph":
                o, lse, f = step()
            else:
                if graph is None:
                    keep = {x: st[x].clone() for x in ("table", "lens", "refs")}
                    pools = kp.clone(), vp.clone()
                    step()  # (loads the kernels)
                    torch.cuda.synchronize()
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph):
                        o, lse, f = step()
                    for x in keep:
                        st[x].copy_(keep[x])
                    kp.copy_(pools[0])
                    vp.copy_(pools[1])
                graph.replay()
        torch.cuda.synchronize()
        no_device_error()
        assert f.item() >= 0
        host_k = [torch.cat([host_k[i], k[b]]) for b, i in enumerate(index)]
        host_v = [torch.cat([host_v[i], v[b]]) for b, i in enumerate(index)]
        for b in range(B):
            L = len(host_k[b])
            seen = np.ones((T, L), bool)
            for i in range(T):
                seen[i, L - T:] = False
                x = i
                while x >= 0:
                    seen[i, L - T + x] = True
                    x = parents[b][x]
            kk, vv = (np.repeat(f64(x).transpose(1, 0, 2), Hq // Hkv, 0) for x in (host_k[b], host_v[b]))
            ro, rl = M.attend(f64(q[b]).transpose(1, 0, 2), kk, vv, seen, 1 / math.sqrt(d))
            check(o[b].transpose(0, 1), lse[b], ro, rl, f"round {rnd} sequence {b}")
            rows = torch.cat([torch.arange(L - T), torch.tensor(path[b][:n[b]], dtype=torch.long) + L - T])
            host_k[b], host_v[b] = host_k[b][rows], host_v[b][rows]
        # the cache holds exactly those rows, at the pool's front
        assert st["lens"].tolist() == [len(x) for x in host_k]
        r = st["refs"].tolist()
        live = sum(x > 0 for x in r)
        assert all(x > 0 for x in r[:live]) and not any(r[live:])
        tab = st["table"].tolist()
        for b in range(B):
            got = M.paged_rows(kp.cpu(), tab[b], len(host_k[b]), page)
            assert torch.equal(got, host_k[b])
    # the window with first tokens reads the same cache
    q1 = bf(B, 1, Hq, d).cuda()
    o, lse = A.attn_fwd_paged(q1, kp, vp, st["table"], st["lens"], causal=True, window=(20, -1), sink_tokens=3)
    for b in range(B):
        L = len(host_k[b])
        kk, vv = (np.repeat(f64(x).transpose(1, 0, 2), Hq // Hkv, 0) for x in (host_k[b], host_v[b]))
        ro, rl = M.attend(f64(q1[b]).transpose(1, 0, 2), kk, vv, M.band(1, L, 20, 0, 3), 1 / math.sqrt(d))
        check(o[b].transpose(0, 1), lse[b], ro, rl, "window")
    no_device_error()


def test_refusals_before_a_launch():
    """Bad sizes, pointers and overlaps are refused on the host (no GPU needed)."""
    lib = A.library()
    p, q, r = 1 << 12, 1 << 13, 1 << 14

    def reorder(**k):
        a = dict(t=p, to=q, l=p, lo=q, refs=p, ro=q, idx=r, B=4, n=4, w=8, num=16, page=64)
        a.update(k)
        return lib.attn_cache_reorder(a["t"], a["l"], a["refs"], a["idx"], a["to"], a["lo"], a["ro"], a["B"],
                                      a["n"], a["w"], a["num"], a["page"], None)

    assert reorder(B=-1) == 1 and reorder(w=0) == 1 and reorder(num=0) == 1
    assert reorder(page=48) == 2 and reorder(B=9000) == 2 and reorder(num=1 << 30, page=256) == 2
    assert reorder(t=None) == 1 and reorder(idx=p + 2) == 1 and reorder(to=p) == 1 and reorder(lo=p) == 1

    def reserve(**k):
        a = dict(k=p, v=p, to=q, lo=q, ro=q, add=r, free=r, B=4, w=8, num=16, page=64, layers=1, row=256)
        a.update(k)
        return lib.attn_cache_reserve(a["k"], a["v"], p, p, p, a["add"], a["to"], a["lo"], a["ro"], a["free"],
                                      a["B"], a["w"], a["num"], a["page"], a["layers"], a["row"], None)

    assert reserve(row=24) == 1 and reserve(row=0) == 1 and reserve(layers=0) == 1
    assert reserve(k=p + 8) == 1 and reserve(v=None) == 1 and reserve(add=None) == 1 and reserve(free=None) == 1
    assert reserve(to=p) == 1 and reserve(lo=p) == 1 and reserve(ro=p) == 1
    assert reserve(page=8) == 2

    def accept(**k):
        a = dict(k=p, path=r, pl=r, lo=q, B=4, A=3, T=8, w=8, num=16, page=64, row=256)
        a.update(k)
        return lib.attn_cache_accept(a["k"], p, p, p, p, a["path"], a["pl"], None, a["lo"], q, a["B"], a["A"],
                                     a["T"], a["w"], a["num"], a["page"], 1, a["row"], None)

    assert accept(A=-1) == 1 and accept(T=-1) == 1 and accept(path=None) == 1 and accept(pl=None) == 1
    assert accept(lo=p) == 1 and accept(row=8) == 1

    def compact(**k):
        a = dict(to=q, ro=q, m=r, ws=r, B=4, row=256)
        a.update(k)
        return lib.attn_cache_compact(p, p, p, p, p, a["to"], a["ro"], a["m"], a["ws"], a["B"], 8, 16, 64, 1,
                                      a["row"], None)

    assert compact(to=p) == 1 and compact(ro=p) == 1 and compact(m=None) == 1 and compact(ws=None) == 1
    assert compact(row=17) == 1


def test_python_checks():
    t, n, r = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    k = torch.zeros(5, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        A.attn_cache_reorder(t, n, r, torch.zeros(2), 16)
    with pytest.raises(ValueError):
        A.attn_cache_reserve(k, k[:4], t, n, r, n)
    with pytest.raises(ValueError):
        A.attn_cache_reserve(k, k, t, n, r[:4], n)
    with pytest.raises(ValueError):
        A.attn_cache_accept(k, k, t, n, r, torch.zeros(3, 4, dtype=torch.int32), n, n)
    with pytest.raises(ValueError):
        A.attn_cache_compact(k, k.transpose(1, 2), t, n, r)
