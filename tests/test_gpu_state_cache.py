"""The state cache's pages and the decode steps on them, on the GPU: lists and pages exactly as on the CPU's lists,
the steps against fp64 within state_mirror's bounds."""
import pytest
import torch

from state_mirror import EULER, EXACT, Cache, delta_step, half_step, scan, step
from test_gpu_scan import DT, close

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Both:
    """The library's cache and the CPU's, driven with the same calls."""

    def __init__(self, efla, n_pages, n_slots, shape=(8,), dtype=torch.float32, gap=0, seed=0):
        self.efla = efla
        gen = torch.Generator().manual_seed(seed)
        big = torch.randn(n_pages, 8 + gap + torch.Size(shape).numel(), generator=gen).to(dtype)
        self.whole = big.cuda()
        self.at = 8         # 16 bytes of bf16, 32 of fp32 before the data
        n = torch.Size(shape).numel()
        view = lambda t: t[:, self.at:self.at + n].unflatten(1, shape)
        self.pool = view(self.whole)
        self.edge = big
        self.n = n
        self.pages = efla.new_pages(n_pages, n_slots)
        self.ref = Cache(n_pages, n_slots, view(big))

    def fork(self, source, dest, copy=True):
        self.efla.efla_pages_fork(self.pages, self.pool if copy else None, ints(source), ints(dest))
        self.ref.fork(source, dest, copy)

    def copy(self, source, dest):
        self.efla.efla_pages_copy(self.pages, self.pool, ints(source), ints(dest))
        self.ref.copy(source, dest)

    def free(self, slots):
        self.efla.efla_pages_free(self.pages, ints(slots))
        self.ref.free(slots)

    def compact(self):
        self.efla.efla_pages_compact(self.pages, self.pool)
        self.ref.compact()

    def check(self, error=None):
        e = self.efla
        want = e.EFLA_ERR_SLOT if self.ref.slot_error else e.EFLA_ERR_FULL if self.ref.full_error else e.EFLA_OK
        assert e.efla_pages_status(self.pages, clear=True) == want and (error is None or error == want)
        assert e.efla_pages_status(self.pages) == e.EFLA_OK
        self.ref.slot_error = self.ref.full_error = False
        assert self.pages.table.tolist() == self.ref.table
        assert self.pages.owner.tolist() == self.ref.owner
        assert torch.equal(self.pool.cpu(), self.ref.pool)
        got = self.whole.cpu()      # what lies between the pages' data is as it was
        assert torch.equal(got[:, :self.at], self.edge[:, :self.at])
        assert torch.equal(got[:, self.at + self.n:], self.edge[:, self.at + self.n:])
        # the scratch is zero again, the move list aside
        claims = self.pages.block[64 + self.pages.n_slots + self.pages.n_pages:][:self.pages.n_slots]
        assert int(claims.abs().sum()) == 0


def test_new_cache_is_empty(efla, cuda):
    for n_pages, n_slots in ((1, 1), (3, 70), (1500, 3)):
        p = efla.new_pages(n_pages, n_slots)
        assert p.table.tolist() == [-1] * n_slots and p.owner.tolist() == [-1] * n_pages
        assert efla.efla_pages_status(p) == efla.EFLA_OK


@pytest.mark.parametrize("shape,dtype,gap", [((4,), torch.float32, 0), ((2, 36), torch.float32, 12),
                                             ((3, 520), torch.bfloat16, 8), ((5003 * 4,), torch.float32, 0)])
def test_fork_free_compact_copy(efla, cuda, shape, dtype, gap):
    b = Both(efla, 9, 12, shape, dtype, gap)
    b.fork([-1, -1, -1, -1, -1], [3, 0, 7, 11, 5])     # zeroed pages
    b.check()
    b.efla.efla_pages_write(b.pages, b.pool, torch.arange(5, device="cuda").reshape(-1, *[1] * len(shape)).expand(5, *shape).to(dtype).contiguous(), ints([3, 0, 7, 11, 5]))
    for i, s in enumerate([3, 0, 7, 11, 5]):
        b.ref.pool[b.ref.table[s]] = i
    b.check()
    b.fork([3, 3, -1], [1, 2, 9])
    b.check()
    b.free([0, -1, 7, 1])
    b.check()
    b.compact()
    b.check()
    b.fork([11, 2], [6, 8])
    b.check()
    b.copy([11, 3, 5, -1], [3, 11, 6, 8])               # an exchange, a copy, a clearing
    b.check()
    b.copy([6, 6, 6], [6, -1, 2])
    b.check()
    b.compact()
    b.check()
    b.free([2, 3, 5, 6, 8, 9, 11])
    b.check()
    b.compact()
    b.check(efla.EFLA_OK)


def test_wrong_entries_touch_nothing(efla, cuda):
    b = Both(efla, 6, 8, (16,))
    b.fork([-1, -1, -1], [0, 1, 2])
    b.check(efla.EFLA_OK)
    b.fork([0, 0, 5, 99, -7, 0, 0], [1, 4, 5, 6, 6, 8, -5])   # taken, fine, source empty, out of range, ...
    b.check(efla.EFLA_ERR_SLOT)
    b.fork([1, 2], [7, 7])                                     # the same slot twice: the first
    b.check(efla.EFLA_ERR_SLOT)
    b.fork([4], [4])                                           # a destination that is in use
    b.check(efla.EFLA_ERR_SLOT)
    b.copy([0, 1, 5, 2, 1], [1, 1, 0, 99, 5])                  # named twice, source empty, out of range, empty
    b.check(efla.EFLA_ERR_SLOT)
    b.free([5, 99, -3, 0, 0])
    b.check(efla.EFLA_ERR_SLOT)
    b.fork([-1] * 8, [0, 3, 5, 6, -1, -1, -1, -1])             # 4 wanted, 2 left
    b.check(efla.EFLA_ERR_FULL)
    rows = torch.randn(4, 16)
    efla.efla_pages_write(b.pages, b.pool, rows.cuda(), ints([1, 99, 1, 6]))
    b.ref.write(rows, [1, 99, 1, 6])
    b.check(efla.EFLA_ERR_SLOT)
    out = torch.full((4, 16), 7.0, device="cuda")
    efla.efla_pages_read(b.pages, b.pool, ints([1, 6, -1, 1]), rows=out)
    assert efla.efla_pages_status(b.pages, clear=True) == efla.EFLA_ERR_SLOT
    assert torch.equal(out[0].cpu(), rows[0]) and torch.equal(out[3].cpu(), rows[0])
    assert float(out[1].min()) == 7 and float(out[2].min()) == 7
    b.check(efla.EFLA_OK)


def test_random_calls(efla, cuda):
    import random
    r = random.Random(5)
    # lists and caches below and above what one launch plans (256 entries, 4096 pages)
    for n_pages, n_slots, rounds in ((37, 50, 12), (1100, 1200, 12), (4096, 300, 6), (4500, 5000, 6)):
        b = Both(efla, n_pages, n_slots, (12,), seed=n_pages)
        for _ in range(rounds):
            pick = lambda k: [r.randrange(-1, n_slots) for _ in range(k)]
            k = r.choice([1, 5, n_slots // 2, n_slots + 30])
            b.fork(pick(k), pick(k))
            b.copy(pick(k), pick(k))
            b.free(pick(n_slots // 3))
            if r.random() < 0.5:
                b.compact()
            b.check()


def test_copy_of_many_pairs(efla, cuda):
    """As many pairs as one call takes: a rotation of all slots."""
    n = 8192
    b = Both(efla, n, n, (20,))
    b.fork([-1] * n, list(range(n)), copy=False)
    order = torch.randperm(n, generator=torch.Generator().manual_seed(1)).tolist()
    b.copy(order, list(range(n)))
    b.check(efla.EFLA_OK)
    with pytest.raises(efla.EflaError):
        efla.efla_pages_copy(b.pages, b.pool, ints([0] * (n + 1)), ints([1] * (n + 1)))


def filled(efla, n_pages, n_slots, live, shape, seed=0):
    """A cache whose first `live` slots hold scattered pages of random states."""
    b = Both(efla, n_pages, n_slots, shape, seed=seed)
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()[:live]
    for s, p in enumerate(order):
        b.ref.table[s], b.ref.owner[p] = p, s
    b.pages.table.copy_(ints(b.ref.table))
    b.pages.owner.copy_(ints(b.ref.owner))
    return b


def step_case(N, H, d, dtype, seed, per_channel=True):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    q, k, v = r(N, H, d) * d ** -0.5, r(N, H, d) * d ** -0.5, r(N, H, d)
    x = r(N, H, d)
    g = -torch.exp(-2.0 + r(N, H))
    gx = -torch.exp(-2.0 + r(N, H, d)) if per_channel else g
    return dict(q=q.to(dtype), k=k.to(dtype), v=v.to(dtype), beta=torch.sigmoid(r(N, H)).to(dtype), g=g,
                x=x.to(dtype), gx=gx)


def pages_of(ref, slots, source=None):
    """(rows that run, the pages they write, the entering states) by the rules of the header."""
    source = slots if source is None else source
    rows = []
    for n, s in enumerate(slots):
        if s == -1 or not 0 <= s < len(ref.table) or ref.table[s] < 0 or s in slots[:n]:
            continue
        src = source[n]
        if src != s and src != -1 and (not 0 <= src < len(ref.table) or ref.table[src] < 0 or src in slots):
            continue
        rows.append((n, ref.table[s], None if src == -1 else ref.pool[ref.table[src]].clone()))
    return rows


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["delta", "gated", "scan", "scan shared"])
@pytest.mark.parametrize("N,H,d", [(1, 1, 64), (7, 3, 64), (5, 16, 128), (40, 2, 128), (150, 3, 128), (333, 3, 64), (160, 7, 64)])
@pytest.mark.parametrize("rule", [EXACT, EULER])
def test_paged_steps(efla, cuda, N, H, d, kind, dtype, rule):
    shape = (H, d, d) if kind in ("delta", "gated") else (H, d)
    b = filled(efla, N + 6, N + 4, N + 3, shape, seed=N + d)
    c = step_case(N, H, d, DT[dtype], N + d, kind != "scan shared")
    dv = {n: t.cuda() for n, t in c.items()}
    slots = torch.randperm(N + 3, generator=torch.Generator().manual_seed(N)).tolist()[:N]
    if N > 4:
        slots[2] = -1
    marker = torch.full((N, H, d), 3.0, dtype=DT[dtype], device="cuda")
    for sources in (None, [s if n % 3 else -1 for n, s in enumerate(slots)]):
        o = marker.clone()
        src = None if sources is None else ints(sources)
        if kind in ("delta", "gated"):
            efla.efla_recurrent_step_paged(dv["q"], dv["k"], dv["v"], dv["beta"], b.pages, b.pool, ints(slots),
                                           source=src, g=dv["g"] if kind == "gated" else None, o=o, rule=rule)
        else:
            efla.efla_scan_step_paged(dv["x"], dv["gx"], b.pages, b.pool, ints(slots), source=src, o=o, rule=rule)
        assert efla.efla_pages_status(b.pages) == efla.EFLA_OK
        rows = pages_of(b.ref, slots, sources)
        assert len(rows) == sum(s != -1 for s in slots)
        after = b.pool.cpu()
        for n, page, S in rows:
            S = torch.zeros(shape) if S is None else S
            at = slice(n, n + 1)
            if kind in ("delta", "gated"):
                ov, Sv, oe, Se = delta_step(c["q"][at], c["k"][at], c["v"][at], c["beta"][at],
                                            c["g"][at] if kind == "gated" else None, S[None], rule)
            else:
                Sv, Se = step(c["x"][at], c["gx"][at], S[None], rule)
                ov, oe = Sv, Se
            close(o[at], (ov, oe), f"o of row {n}")
            close(after[page][None], (Sv, Se), f"state of row {n}")
            b.ref.pool[page] = after[page]
        assert torch.equal(after, b.ref.pool)                       # every other page as it was
        for n, s in enumerate(slots):
            if s == -1:
                assert torch.equal(o[n], marker[n])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,H,d", [(130, 7, 128), (480, 7, 64)])
def test_paged_delta_step_of_many_rows(efla, cuda, N, H, d, dtype):
    """Enough heads that every block takes many: rows from their own page, from another one and from a zero state in
    turn, and heads that do not fill a block's last piece of a row."""
    b = filled(efla, N + 9, N + 8, N + 8, (H, d, d), seed=d)
    c = step_case(N, H, d, DT[dtype], d)
    slots = torch.randperm(N, generator=torch.Generator().manual_seed(N)).tolist()
    source = [-1 if n % 3 == 0 else s if n % 3 == 1 else N + n % 8 for n, s in enumerate(slots)]
    dv = {n: t.cuda() for n, t in c.items()}
    o = efla.efla_recurrent_step_paged(dv["q"], dv["k"], dv["v"], dv["beta"], b.pages, b.pool, ints(slots),
                                       source=ints(source), g=dv["g"])
    assert efla.efla_pages_status(b.pages) == efla.EFLA_OK
    rows = pages_of(b.ref, slots, source)
    assert len(rows) == N
    S = torch.stack([torch.zeros(H, d, d) if s is None else s for _, _, s in rows])
    ov, Sv, oe, Se = delta_step(c["q"], c["k"], c["v"], c["beta"], c["g"], S, EXACT)
    close(o, (ov, oe), "o")
    pages = [p for _, p, _ in rows]
    after = b.pool.cpu()
    close(after[pages], (Sv, Se), "states")
    others = [p for p in range(N + 9) if p not in pages]
    assert torch.equal(after[others], b.ref.pool[others])


@pytest.mark.parametrize("H", [2, 150])
@pytest.mark.parametrize("kind", ["delta", "scan"])
def test_paged_steps_refuse_rows(efla, cuda, kind, H):
    """Rows that would be wrong or race are left out whole; the others are what they would be alone."""
    N, d = 9, 64
    shape = (H, d, d) if kind == "delta" else (H, d)
    b = filled(efla, 14, 12, 10, shape)
    c = {n: t.cuda() for n, t in step_case(N, H, d, torch.float32, 1).items()}

    def run(slots, source, pool):
        o = torch.full((N, H, d), 3.0, device="cuda")
        src = None if source is None else ints(source)
        if kind == "delta":
            efla.efla_recurrent_step_paged(c["q"], c["k"], c["v"], c["beta"], b.pages, pool, ints(slots), source=src, o=o)
        else:
            efla.efla_scan_step_paged(c["x"], c["gx"], b.pages, pool, ints(slots), source=src, o=o)
        return o

    #        fine twice  none  range  below  fine  reads a written one, reads an empty one, fine from another
    slots = [4, 4, 11, 12, -2, 5, 6, 7, 8]
    source = [4, 4, 11, 12, -2, -1, 4, 10, 9]
    fine = {0: (4, 4), 5: (5, -1), 8: (8, 9)}
    pool = b.pool.clone()
    o = run(slots, source, pool)
    assert efla.efla_pages_status(b.pages, clear=True) == efla.EFLA_ERR_SLOT
    alone = b.pool.clone()
    oa = run([s if n in fine else -1 for n, s in enumerate(slots)], source, alone)
    assert efla.efla_pages_status(b.pages) == efla.EFLA_OK
    assert torch.equal(pool, alone) and torch.equal(o, oa)
    for n in range(N):
        assert (float((o[n] - 3).abs().max()) == 0) == (n not in fine)
    written = [b.ref.table[s] for s, _ in fine.values()]
    for p in range(14):
        assert torch.equal(pool[p], b.pool[p]) == (p not in written)


def test_paged_step_is_the_dense_step(efla, cuda):
    N, H, d = 6, 4, 128
    b = filled(efla, 8, 8, 8, (H, d, d))
    c = {n: t.cuda() for n, t in step_case(N, H, d, torch.bfloat16, 3).items()}
    slots = [5, 0, 7, 2, 1, 3]
    S = torch.stack([b.pool[b.ref.table[s]] for s in slots]).contiguous()
    o1 = efla.efla_recurrent_step_gated(c["q"], c["k"], c["v"], c["beta"], c["g"], S)
    o2 = efla.efla_recurrent_step_paged(c["q"], c["k"], c["v"], c["beta"], b.pages, b.pool, ints(slots), g=c["g"])
    S2 = torch.stack([b.pool[b.ref.table[s]] for s in slots])
    # the same formulas in the same precision: a few roundings apart
    assert float((S - S2).abs().max()) <= 1e-5 and float((o1.float() - o2.float()).abs().max()) <= 2e-2


def test_full_cache_many_entries(efla, cuda):
    """More entries than free pages, by both planners: the first entries get them."""
    for n_pages, n in ((10, 100), (300, 600), (5000, 5200)):
        b = Both(efla, n_pages, n, (4,))
        b.fork([-1] * n, list(range(n)))
        b.check(efla.EFLA_ERR_FULL)
        b.free(list(range(0, n_pages, 3)))
        b.compact()
        b.check(efla.EFLA_OK)


def test_other_streams(efla, cuda):
    """Calls on streams of their own, with outputs that they allocate."""
    N, H, d = 6, 2, 64
    b = filled(efla, 8, 8, 8, (H, d, d))
    v = filled(efla, 8, 8, 8, (H, d))
    c = {n: t.cuda() for n, t in step_case(N, H, d, torch.float32, 3).items()}
    slots = ints([5, 0, -1, 2, 1, 3])
    want = None
    for stream in (None, torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        pool, vec = b.pool.clone(), v.pool.clone()
        torch.cuda.synchronize()
        o1 = efla.efla_recurrent_step_paged(c["q"], c["k"], c["v"], c["beta"], b.pages, pool, slots, stream=stream)
        o2 = efla.efla_scan_step_paged(c["x"], c["gx"], v.pages, vec, slots, stream=stream)
        rows = efla.efla_pages_read(v.pages, vec, slots, stream=stream)
        torch.cuda.synchronize()
        got = (o1, o2, rows, pool, vec)
        want = want or got
        assert all(torch.equal(x, y) for x, y in zip(want, got))
        assert float(o1[2].abs().max()) == 0 and float(rows[2].abs().max()) == 0


def test_far_pages(efla, cuda):
    """Pages past 2^32 bytes of the pool."""
    H, d = 2, 64
    words = (1 << 30) // 4
    pool = torch.zeros(6, words, device="cuda")
    pages = efla.new_pages(6, 6)
    efla.efla_pages_fork(pages, None, ints([-1] * 6), ints([0, 1, 2, 3, 4, 5]))
    layer = pool[:, 1024:1024 + H * d].unflatten(1, (H, d))
    x, g = torch.randn(1, H, d, device="cuda"), -torch.rand(1, H, d, device="cuda")
    efla.efla_scan_step_paged(x, g, pages, layer, ints([5]))
    h, bound = step(x.cpu(), g.cpu(), torch.zeros(1, H, d))
    close(layer[5][None], (h, bound))
    assert float(pool[:5].abs().max()) == 0 and float(pool[5, :1024].abs().max()) == 0
    efla.efla_pages_copy(pages, layer, ints([5]), ints([4]))
    assert torch.equal(layer[4], layer[5])
    efla.efla_pages_free(pages, ints([0, 1, 2, 3]))
    efla.efla_pages_compact(pages, pool)
    assert pages.table.tolist() == [-1, -1, -1, -1, 0, 1]
    assert torch.equal(layer[0], layer[4]) and torch.equal(layer[1], layer[5])
    del pool


def test_captured_server_tick(efla, cuda):
    """Free, compact, fork and a step in one graph, replayed on new lists: the same as the eager calls."""
    H, d = 2, 64
    b = filled(efla, 24, 20, 16, (H, d, d), seed=4)
    c = {n: t.cuda() for n, t in step_case(6, H, d, torch.float32, 8).items()}
    lists = {n: ints([-1] * 6) for n in ("gone", "source", "slots")}
    o = torch.zeros(6, H, d, device="cuda")

    def tick(pages, pool, o):
        efla.efla_pages_free(pages, lists["gone"])
        efla.efla_pages_compact(pages, pool)
        efla.efla_pages_fork(pages, pool, lists["source"], lists["gone"])
        efla.efla_recurrent_step_paged(c["q"], c["k"], c["v"], c["beta"], pages, pool, lists["slots"], o=o)

    # the graph's and the eager caches have buffers of their own
    pages2, pool2, o2 = efla.EflaPages(b.pages.block.clone(), 24, 20), b.pool.clone(), torch.zeros_like(o)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        tick(efla.EflaPages(b.pages.block.clone(), 24, 20), b.pool.clone(), torch.zeros_like(o))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tick(b.pages, b.pool, o)
    for gone, source, slots in (([1, 2, 3, -1, -1, -1], [0, 0, 9, -1, -1, -1], [1, 2, 3, 15, -1, 4]),
                                ([15, 14, 0, 1, 2, 3], [4, 5, 6, 7, -1, 8], [0, 1, 2, 3, 14, 15]),
                                ([4, -1, 5, -1, -1, -1], [1, -1, 1, -1, -1, -1], [4, 5, -1, -1, -1, -1])):
        for n, v in zip(("gone", "source", "slots"), (gone, source, slots)):
            lists[n].copy_(ints(v))
        graph.replay()
        tick(pages2, pool2, o2)
        torch.cuda.synchronize()
        assert torch.equal(b.pages.table, pages2.table) and torch.equal(b.pages.owner, pages2.owner)
        assert torch.equal(b.pool, pool2) and torch.equal(o, o2)
        assert efla.efla_pages_status(b.pages) == efla.EFLA_OK == efla.efla_pages_status(pages2)
    del graph


def test_a_server_of_a_hybrid_layer_pair(efla, cuda):
    """The operators together: packed prefill of a delta-rule layer and a per-channel layer, their final states into
    one cache whose pages hold both, forks, decode, departures and compaction; every step against fp64 from the
    cache's own states, and the scan layer's whole streams against one fp64 run."""
    H, d, dt = 2, 64, torch.float32
    lengths = [70, 1, 133, 40]
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    gen = torch.Generator().manual_seed(12)
    r = lambda *s: torch.randn(*s, generator=gen)
    T = cu[-1]
    q, k, v = r(H, T, d) * d ** -0.5, r(H, T, d) * d ** -0.5, r(H, T, d)
    beta, x, gx = torch.sigmoid(r(H, T)), r(H, T, d), -torch.exp(-2 + r(H, T, d))
    cud = lambda t: t.cuda()
    _, SM = efla.efla_chunk_fwd_varlen(cud(q), cud(k), cud(v), cud(beta), cu)
    _, SV = efla.efla_scan_fwd(cud(x), cud(gx), cu_seqlens=cu)
    words = H * d * d + H * d
    pool = torch.zeros(8, words, device="cuda")
    matrix, vector = pool[:, :H * d * d].unflatten(1, (H, d, d)), pool[:, H * d * d:].unflatten(1, (H, d))
    pages = efla.new_pages(8, 8)
    efla.efla_pages_fork(pages, None, ints([-1] * 4), ints([0, 1, 2, 3]))
    efla.efla_pages_write(pages, matrix, SM, ints([0, 1, 2, 3]))
    efla.efla_pages_write(pages, vector, SV, ints([0, 1, 2, 3]))
    assert torch.equal(efla.efla_pages_read(pages, vector, ints([2, 0])), SV[[2, 0]])
    history = {s: (x[:, cu[s]:cu[s + 1]], gx[:, cu[s]:cu[s + 1]]) for s in range(4)}

    def token(rows, seed):
        c = step_case(len(rows), H, d, dt, seed)
        table, before = pages.table.tolist(), pool.clone()
        dv = {n: t.cuda() for n, t in c.items()}
        o1 = efla.efla_recurrent_step_paged(dv["q"], dv["k"], dv["v"], dv["beta"], pages, matrix, ints(rows), g=dv["g"])
        o2 = efla.efla_scan_step_paged(dv["x"], dv["gx"], pages, vector, ints(rows))
        for n, s in enumerate(rows):
            if s < 0:
                continue
            at = slice(n, n + 1)
            S = before[table[s], :H * d * d].reshape(1, H, d, d).cpu()
            ov, Sv, oe, Se = delta_step(c["q"][at], c["k"][at], c["v"][at], c["beta"][at], c["g"][at], S)
            close(o1[at], (ov, oe))
            close(matrix[table[s]][None], (Sv, Se))
            hx, hg = history[s]
            history[s] = (torch.cat([hx, c["x"][n][:, None]], 1), torch.cat([hg, c["gx"][n][:, None]], 1))
            ref = scan(history[s][0][None], history[s][1][None])
            close(o2[n][None], tuple(t[:, :, -1] for t in ref["o"]))

    token([3, 1, -1, 0, 2], 1)
    efla.efla_pages_fork(pages, pool, ints([2, 2]), ints([6, 7]))
    history[6], history[7] = history[2], history[2]
    token([0, 1, 2, 3, 6, 7], 2)
    efla.efla_pages_free(pages, ints([1, 2]))
    efla.efla_pages_compact(pages, pool)
    assert sorted(p for p in pages.table.tolist() if p >= 0) == [0, 1, 2, 3]
    token([7, 3, 6, 0], 3)
    efla.efla_pages_copy(pages, pool, ints([7, 6]), ints([6, 7]))
    history[6], history[7] = history[7], history[6]
    token([6, 7], 4)
    assert efla.efla_pages_status(pages) == efla.EFLA_OK
