"""The cases that the gated linear recurrence and the state cache are measured on.

Operators: the per-channel gated linear recurrence (forward over dense and packed batches, a training step, one token
on paged states), the delta-rule decode step on paged states, and the operations on the cache's pages.  `own` chooses
between the plain form (elementary torch operations in fp32) and the library's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EMPTY = -1       # an empty slot of the table, a free page, a padded entry of a list of slots
HEADER = 64      # int32 words before the table in the cache's block


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one short prompt of a small model, one decay per head: latency
        dict(name="scan short prompt", op="scan", B=1, H=2, T=257, d=64, dtype="f32", per_channel=False, exact=False,
             state=False, packed=False, train=False, mix=1),
        # prefill of a batch at the 1.3B layer shape, one decay per channel
        dict(name="scan layer prefill", op="scan", B=4, H=16, T=2048, d=128, dtype="bf16", per_channel=True,
             exact=True, state=False, packed=False, train=False, mix=1),
        # one long document continued from a state: only 16 streams, so time itself has to be split
        dict(name="scan long document", op="scan", B=1, H=16, T=32768, d=128, dtype="bf16", per_channel=True,
             exact=True, state=True, packed=False, train=False, mix=1),
        # prefill of 24 requests of mixed lengths (some empty), packed without padding
        dict(name="scan packed requests", op="scan", B=24, H=16, T=16381, d=128, dtype="bf16", per_channel=True,
             exact=True, state=True, packed=True, train=False, mix=5),
        # a layer's training step: forward and gradients
        dict(name="train layer", op="scan", B=4, H=16, T=2048, d=128, dtype="bf16", per_channel=True, exact=True,
             state=False, packed=False, train=True, mix=1),
        # a training step in fp32 with one decay per head (its gradient summed over the channels) and an odd length
        dict(name="train shared decay", op="scan", B=2, H=16, T=4095, d=64, dtype="f32", per_channel=False,
             exact=True, state=True, packed=False, train=True, mix=1),
        # one token for a full serving batch, vector states in pages
        dict(name="scan step batch", op="scan_step", N=256, slots=288, pages=300, H=16, d=128, dtype="bf16",
             per_channel=True, exact=True, idle=0),
        # one token for a few sequences of a padded batch: latency
        dict(name="scan step few", op="scan_step", N=4, slots=8, pages=9, H=4, d=64, dtype="f32", per_channel=False,
             exact=False, idle=1),
        # one delta-rule token for the full decode batch, matrix states in pages
        dict(name="step paged batch", op="step", N=256, slots=288, pages=300, H=16, d=128, dtype="f32", gated=False,
             exact=True, idle=0),
        # one gated delta-rule token for a few sequences of a padded batch
        dict(name="step paged few", op="step", N=12, slots=16, pages=20, H=16, d=128, dtype="bf16", gated=True,
             exact=True, idle=3),
        # between two tokens: finished sequences leave, the cache is compacted, new ones fork from kept prompts
        dict(name="cache tick", op="tick", live=256, slots=288, pages=384, moved=24, words=16 * 128 * 128),
        # beams take over their parents' vector states, all at once
        dict(name="cache beams", op="beams", live=61, slots=64, pages=80, n=48, words=16 * 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "train", "train", "scan_step", "step", "tick", "beams"])
    dtype = rng.choice(["bf16", "f32"])
    if op in ("scan", "train"):
        packed, d = rng.random() < 0.4, rng.choice([8, 40, 64, 64, 80, 128, 128, 128, 136, 192, 256])
        B, H = (_log(rng, 1, 40), _log(rng, 1, 16)) if packed else (_log(rng, 1, 8), _log(rng, 1, 16))
        room = (22_000_000 if op == "train" or dtype == "f32" else 50_000_000) // (H * d * (1 if packed else B))
        return dict(op="scan", B=B, H=H, T=_log(rng, 1, min(32768, room)), d=d, dtype=dtype,
                    per_channel=rng.random() < 0.6, exact=rng.random() < 0.7, state=rng.random() < 0.5, packed=packed,
                    train=op == "train", mix=rng.randrange(1 << 20))
    if op in ("scan_step", "step"):
        N = _log(rng, 1, 240)
        slots, idle = N + rng.randrange(40), rng.randrange(1 + N // 4)
        c = dict(op=op, N=N, slots=slots, pages=slots + rng.randrange(20), H=_log(rng, 1, 16), dtype=dtype,
                 exact=True, idle=idle)
        if op == "step":
            return dict(c, d=rng.choice([64, 128]), gated=rng.random() < 0.5)
        return dict(c, d=rng.choice([8, 64, 80, 128, 136, 256]), per_channel=rng.random() < 0.6)
    if op == "tick":
        live = _log(rng, 12, 240)
        return dict(op=op, live=live, slots=live + rng.randrange(30), pages=live + rng.randrange(1, 120),
                    moved=rng.randint(1, live // 4), words=4 * _log(rng, 64, 65536))
    live = _log(rng, 4, 400)
    return dict(op=op, live=live, slots=live + rng.randrange(30), pages=live + rng.randrange(1, 80),
                n=rng.randint(1, live), words=4 * _log(rng, 16, 8192))


def _offsets(case):
    """The packed batch's offsets: B lengths whose logarithms are spread evenly, a few of them empty, T in all."""
    gen = torch.Generator().manual_seed(case["mix"])
    N, T = case["B"], case["T"]
    share = torch.exp(4.0 * torch.rand(N, generator=gen, dtype=torch.float64))
    share[torch.rand(N, generator=gen) < 0.1] = 0.0
    share[-1] = max(float(share[-1]), 1.0)
    cu = [0] + [int(v) for v in torch.floor(share.cumsum(0) / share.sum() * T).tolist()]
    cu[-1] = T
    return cu


def _active(case):
    return case["N"] - case["idle"]


def work(case):
    if case["op"] == "scan":
        es = 2 if case["dtype"] == "bf16" else 4
        Z, d = case["H"] * (1 if case["packed"] else case["B"]), case["d"]
        n = Z * case["T"] * d                                         # elements
        ng = n if case["per_channel"] else n // d
        ns = case["B"] * case["H"] * d * 4                            # states
        byt = n * es + ng * 4 + n * es + ns * (2 if case["state"] else 1)
        if case["train"]:                                             # dO, x and g in; dx, dg, dS0 out
            byt += 2 * n * es + ng * 4 + n * 4 + ng * 4 + ns * 2 + (ns if case["state"] else 0)
        return {"bytes": byt, "flops": n * (24 if case["train"] else 8)}
    if case["op"] in ("scan_step", "step"):
        es, n, H, d = (2 if case["dtype"] == "bf16" else 4), _active(case), case["H"], case["d"]
        if case["op"] == "scan_step":
            return {"bytes": n * H * (d * (2 * es + 8) + (d if case["per_channel"] else 1) * 4),
                    "flops": n * H * d * 8}
        return {"bytes": n * H * (d * d * 8 + d * 4 * es + es + (4 if case["gated"] else 0)),
                "flops": n * H * d * d * 8}
    pages = 2 * case["moved"] if case["op"] == "tick" else case["n"]  # moved pages: read once and written once
    return {"bytes": 2 * pages * case["words"] * 4 + 4 * (case["slots"] + case["pages"]), "flops": 0}


# ---------------------------------------------------------------- inputs
def _decay(shape, gen):
    """Log-decays of memories that last from about one token to a few thousand."""
    return -torch.exp(-3.0 + 1.5 * torch.randn(shape, generator=gen, device=DEV)).clamp_(3e-4, 30.0)


def _cache(case, live, gen):
    """The block of a cache whose slots 0 .. live - 1 hold scattered pages: header, table, owners, scratch."""
    slots, pages = case["slots"], case["pages"]
    block = torch.zeros(HEADER + 2 * slots + 3 * pages, dtype=torch.int32, device=DEV)
    block[HEADER:HEADER + slots + pages] = EMPTY
    at = torch.randperm(pages, generator=gen, device=DEV)[:live].int()
    block[HEADER:HEADER + live] = at
    block[HEADER + slots + at.long()] = torch.arange(live, dtype=torch.int32, device=DEV)
    return block


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def rand(*shape, dtype=torch.float32, scale=1.0):
        return (scale * torch.randn(shape, generator=gen, device=DEV)).to(dtype)

    st = {"case": case}
    if case["op"] == "scan":
        B, H, T, d, dt = case["B"], case["H"], case["T"], case["d"], DTYPES[case["dtype"]]
        lead = (H, T) if case["packed"] else (B, H, T)
        st["x"] = rand(*lead, d, dtype=dt)
        st["g"] = _decay(lead + ((d,) if case["per_channel"] else ()), gen)
        st["S0"] = rand(B, H, d) if case["state"] else None
        st["cu"] = _offsets(case) if case["packed"] else None
        if case["packed"]:   # first and last tokens of the sequences that have any
            some = [n for n in range(B) if st["cu"][n + 1] > st["cu"][n]]
            st["which"] = torch.tensor(some, device=DEV)
            st["first"] = torch.tensor([st["cu"][n] for n in some], device=DEV)
            st["last"] = torch.tensor([st["cu"][n + 1] - 1 for n in some], device=DEV)
        if case["train"]:
            st["dO"] = rand(*lead, d, dtype=dt)
            st["dS_T"] = rand(B, H, d) if case["state"] else None
    elif case["op"] in ("scan_step", "step"):
        N, H, d, dt = case["N"], case["H"], case["d"], DTYPES[case["dtype"]]
        st["block"] = _cache(case, case["slots"], gen)
        slots = torch.randperm(case["slots"], generator=gen, device=DEV)[:N].int()
        slots[_active(case):] = EMPTY
        st["slots"] = slots
        st["o"] = torch.zeros(N, H, d, dtype=dt, device=DEV)
        if case["op"] == "scan_step":
            st["x"] = rand(N, H, d, dtype=dt)
            st["g"] = _decay((N, H, d) if case["per_channel"] else (N, H), gen)
            st["pool"] = rand(case["pages"], H, d)
        else:
            st["q"], st["k"] = (rand(N, H, d, dtype=dt, scale=d ** -0.5) for _ in range(2))
            st["v"] = rand(N, H, d, dtype=dt)
            st["beta"] = torch.sigmoid(rand(N, H)).to(dt)
            st["g"] = _decay((N, H), gen) if case["gated"] else None
            st["pool"] = rand(case["pages"], H, d, d, scale=0.1)
    else:
        live = case["live"]
        st["block"] = _cache(case, live, gen)
        st["pool"] = rand(case["pages"], case["words"])
        order = torch.randperm(live, generator=gen, device=DEV).int()
        if case["op"] == "tick":   # two groups of sequences that end and start again in turn, from kept ones
            m = case["moved"]
            st["groups"] = [order[:m].contiguous(), order[m:2 * m].contiguous()]
            kept = order[2 * m:]
            st["sources"] = [kept[torch.randint(0, live - 2 * m, (m,), generator=gen, device=DEV)] for _ in range(2)]
            st["tick"] = 0
        else:
            st["dest"] = order[:case["n"]].contiguous()
            st["source"] = order[torch.randint(0, live, (case["n"],), generator=gen, device=DEV)]
    return st


# ---------------------------------------------------------------- the plain forms
def _gates(g, exact):
    """a = e^g, the write gate w, and w's derivative; those of the exact flow are (e^g - 1) / g and its derivative."""
    a = torch.exp(g)
    if not exact:
        return a, torch.ones_like(g), torch.zeros_like(g)
    r = g.double()      # the derivative's difference cancels near 0
    w = torch.where(r.abs() < 1e-4, 1 + r / 2 + r * r / 6, torch.expm1(r) / r)
    dw = torch.where(r.abs() < 1e-3, 0.5 + r / 3 + r * r / 8, (torch.exp(r) - w) / r)
    return a, w.float(), dw.float()


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from zero, by doubling the reach of every row's sum."""
    k = 1
    while k < b.shape[1]:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _streams(st):
    """The batch as streams [Z, T, d] that restart at tokens `first` from the rows of S0 [Z, R, d]."""
    case = st["case"]
    T, d = case["T"], case["d"]
    x = st["x"].float().reshape(-1, T, d)
    g = st["g"].reshape(-1, T, d if case["per_channel"] else 1)
    if case["packed"]:
        first, last, which = st["first"], st["last"], st["which"]
    else:
        first, last, which = (torch.full((1,), v, device=DEV) for v in (0, T - 1, 0))
    return x, g, first, last, which


def _rows(state, case, which):
    """States [B, H, d] as the streams' rows [Z, R, d] (zero where there is none)."""
    if case["packed"]:
        return state.transpose(0, 1)[:, which]
    return state.reshape(-1, 1, case["d"])


def _plain_scan(st):
    case = st["case"]
    B, H, d = case["B"], case["H"], case["d"]
    x, g, first, last, which = _streams(st)
    zero = torch.zeros(B, H, d, device=DEV)
    S0 = zero if st["S0"] is None else st["S0"]
    a, w, dw = _gates(g, case["exact"])
    s0 = _rows(S0, case, which)
    A, b = a.expand_as(x).clone(), w * x
    b[:, first] += A[:, first] * s0
    A[:, first] = 0
    h = _scan(A, b)

    def states(rows, rest):
        if not case["packed"]:
            return rows.reshape(B, H, d)
        out = rest.clone()
        out[which] = rows.transpose(0, 1)
        return out

    out = [h.to(st["x"].dtype).reshape(st["x"].shape), states(h[:, last], S0)]
    if not case["train"]:
        return out
    dST = zero if st["dS_T"] is None else st["dS_T"]
    u = st["dO"].float().reshape(x.shape).clone()
    u[:, last] += _rows(dST, case, which)
    c = torch.cat([A[:, 1:], torch.zeros_like(A[:, :1])], 1)    # A is zero where a sequence starts
    G = _scan(c.flip(1), u.flip(1)).flip(1)
    prev = torch.cat([h[:, :1], h[:, :-1]], 1)
    prev[:, first] = s0
    dg = G * (a * prev + dw * x)
    dg = dg if case["per_channel"] else dg.sum(-1)
    return out + [(w * G).reshape(st["x"].shape), dg.reshape(st["g"].shape), states((a * G)[:, first], dST)]


def _plain_scan_step(st):
    case, n = st["case"], _active(st["case"])
    at = st["block"][HEADER + st["slots"][:n].long()].long()
    g = st["g"][:n] if case["per_channel"] else st["g"][:n, :, None]
    a, w, _ = _gates(g, case["exact"])
    h = a * st["pool"][at] + w * st["x"][:n].float()
    st["pool"][at] = h
    st["o"][:n] = h.to(st["o"].dtype)
    return [st["o"], st["pool"]]


def _plain_step(st):
    case, n = st["case"], _active(st["case"])
    at = st["block"][HEADER + st["slots"][:n].long()].long()
    q, k, v = (st[name][:n].float() for name in ("q", "k", "v"))
    beta = st["beta"][:n].float()
    lam = (k * k).sum(-1)
    g = st["g"][:n] if case["gated"] else torch.zeros_like(beta)

    def phi(y):   # (1 - e^-y) / y
        y = y.double()
        return torch.where(y.abs() < 1e-4, 1 - y / 2 + y * y / 6, -torch.expm1(-y) / y).float()

    alpha, abar = beta * phi(beta * lam), beta * phi(beta * lam - g)
    dec = torch.exp(g)
    S = st["pool"][at]
    r = (k[..., None] * S).sum(-2)
    wr = (dec * alpha)[..., None] * r - abar[..., None] * v
    S = dec[..., None, None] * S - k[..., None] * wr[..., None, :]
    st["pool"][at] = S
    st["o"][:n] = (q[..., None] * S).sum(-2).to(st["o"].dtype)
    return [st["o"], st["pool"]]


def _cache_views(st):
    """The cache's table (slot -> page) and owners (page -> slot): views of its block."""
    case = st["case"]
    table = st["block"][HEADER:HEADER + case["slots"]]
    return table, st["block"][HEADER + case["slots"]:HEADER + case["slots"] + case["pages"]]


def _plain_tick(st):
    pool = st["pool"]
    table, owner = _cache_views(st)
    gone, source = st["groups"][st["tick"]].long(), st["sources"][st["tick"]].long()
    st["tick"] ^= 1
    # the finished sequences' pages are free
    owner[table[gone].long()] = EMPTY
    table[gone] = EMPTY
    # the k-th page in use behind the live count moves into the k-th free page before it
    used = owner >= 0
    live = st["case"]["live"] - st["case"]["moved"]
    holes, late = torch.nonzero(~used[:live])[:, 0], live + torch.nonzero(used[live:])[:, 0]
    pool[holes] = pool[late]
    table[owner[late].long()] = holes.int()
    owner[holes] = owner[late]
    owner[late] = EMPTY
    # new sequences get the lowest free pages, with copies of their prompts' states
    fresh = torch.nonzero(owner < 0)[:gone.numel(), 0]
    pool[fresh] = pool[table[source].long()]
    table[gone] = fresh.int()
    owner[fresh] = gone.int()
    return [pool, table, owner]


def _plain_beams(st):
    table, _ = _cache_views(st)
    st["pool"][table[st["dest"].long()].long()] = st["pool"][table[st["source"].long()].long()]
    return [st["pool"]]


PLAIN = {"scan": _plain_scan, "scan_step": _plain_scan_step, "step": _plain_step, "tick": _plain_tick,
         "beams": _plain_beams}


# ---------------------------------------------------------------- the library's calls
def _library(st):
    import delta_rule_linear_02_b200 as efla

    case = st["case"]
    rule = efla.EFLA_RULE_EXACT if case.get("exact", True) else efla.EFLA_RULE_EULER
    if case["op"] == "scan":
        if not case["train"]:
            return efla.efla_scan_fwd(st["x"], st["g"], S0=st["S0"], cu_seqlens=st["cu"], rule=rule)
        o, S_T, saved = efla.efla_scan_fwd_save(st["x"], st["g"], S0=st["S0"], cu_seqlens=st["cu"], rule=rule)
        dx, dg, dS0 = efla.efla_scan_backward(st["x"], st["g"], st["dO"], S0=st["S0"], dS_T=st["dS_T"], saved=saved,
                                              cu_seqlens=st["cu"], rule=rule)
        return [o, S_T, dx, dg, dS0]
    pages = efla.EflaPages(st["block"], case["pages"], case["slots"])
    if case["op"] == "scan_step":
        efla.efla_scan_step_paged(st["x"], st["g"], pages, st["pool"], st["slots"], o=st["o"], rule=rule)
        return [st["o"], st["pool"]]
    if case["op"] == "step":
        efla.efla_recurrent_step_paged(st["q"], st["k"], st["v"], st["beta"], pages, st["pool"], st["slots"],
                                       g=st["g"], o=st["o"], rule=rule)
        return [st["o"], st["pool"]]
    if case["op"] == "beams":
        efla.efla_pages_copy(pages, st["pool"], st["source"], st["dest"])
        return [st["pool"]]
    gone, source = st["groups"][st["tick"]], st["sources"][st["tick"]]
    st["tick"] ^= 1
    efla.efla_pages_free(pages, gone)
    efla.efla_pages_compact(pages, st["pool"])
    efla.efla_pages_fork(pages, st["pool"], source, gone)
    return [st["pool"], pages.table, pages.owner]


def run(state):
    if own:
        return _library(state)
    return PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_scan(st):
    """Token by token, each sequence from its own state."""
    case = st["case"]
    B, H, T, d = case["B"], case["H"], case["T"], case["d"]
    shape = st["x"].shape
    x = st["x"].double().reshape(-1, T, d).transpose(0, 1).contiguous()             # [T, Z, d]
    g = st["g"].double().reshape(-1, T, d if case["per_channel"] else 1).transpose(0, 1).contiguous()
    a, w = g.exp(), torch.ones_like(g)
    if case["exact"]:
        w = torch.where(g == 0, torch.ones_like(g), torch.expm1(g) / g)
    cu = st["cu"] if case["packed"] else [0, T]
    S0 = torch.zeros(B, H, d, dtype=torch.float64, device=DEV) if st["S0"] is None else st["S0"].double()
    begin = S0 if case["packed"] else S0.reshape(1, B * H, d)
    finish = begin.clone()
    wx = w * x
    h = torch.empty_like(x)
    for n in range(len(cu) - 1):
        now = begin[n]
        for t in range(cu[n], cu[n + 1]):
            now = torch.addcmul(wx[t], a[t], now, out=h[t])
        if cu[n + 1] > cu[n]:
            finish[n] = now
    out = [h.transpose(0, 1).reshape(shape), finish.reshape(B, H, d)]
    if not case["train"]:
        return out
    up = st["dO"].double().reshape(-1, T, d).transpose(0, 1)
    G = torch.empty_like(x)
    dS = torch.zeros_like(begin) if st["dS_T"] is None else st["dS_T"].double().reshape(begin.shape).clone()
    prev = torch.empty_like(h)
    for n in range(len(cu) - 1):
        flow = dS[n]
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            torch.add(up[t], flow, out=G[t])
            flow = a[t] * G[t]
        if cu[n + 1] > cu[n]:
            dS[n] = flow
            prev[cu[n]] = begin[n]
            prev[cu[n] + 1:cu[n + 1]] = h[cu[n]:cu[n + 1] - 1]
    dw = torch.zeros_like(g)
    if case["exact"]:
        dw = torch.where(g.abs() < 1e-3, 0.5 + g / 3 + g ** 2 / 8 + g ** 3 / 30, (a - w) / g)
    dg = G * (a * prev + dw * x)
    dg = dg.transpose(0, 1) if case["per_channel"] else dg.sum(-1).transpose(0, 1)
    return out + [(w * G).transpose(0, 1).reshape(shape), dg.reshape(st["g"].shape), dS.reshape(B, H, d)]


def _exact_steps(st):
    """One token in 64 bits, row by row of the batch."""
    case = st["case"]
    pool, o = st["pool"].double(), st["o"].double()
    at = st["block"][HEADER:].tolist()
    slots = st["slots"].tolist()
    for n in range(_active(case)):
        page = at[slots[n]]
        S = pool[page]
        if case["op"] == "scan_step":
            g = st["g"][n].double()
            g = g if case["per_channel"] else g[:, None]
            S = g.exp() * S + (torch.expm1(g) / g if case["exact"] else 1.0) * st["x"][n].double()
            o[n] = S
        else:
            q, k, v, beta = (st[name][n].double() for name in ("q", "k", "v", "beta"))
            lam = (k * k).sum(-1)
            g = st["g"][n].double() if case["gated"] else torch.zeros_like(lam)
            y = beta * lam - g
            alpha, abar = -torch.expm1(-beta * lam) / lam, -beta * torch.expm1(-y) / y
            kS = torch.einsum("hi,hij->hj", k, S)
            S = g.exp()[:, None, None] * (S - alpha[:, None, None] * torch.einsum("hi,hj->hij", k, kS))
            S = S + abar[:, None, None] * torch.einsum("hi,hj->hij", k, v)
            o[n] = torch.einsum("hi,hij->hj", q, S)
        pool[page] = S
    return [o, pool]


def _exact_pages(st):
    """The pages moved one by one on lists."""
    case, pool = st["case"], st["pool"].double()
    table, owner = (v.tolist() for v in _cache_views(st))
    if case["op"] == "beams":
        before = pool.clone()
        for i, j in zip(st["source"].tolist(), st["dest"].tolist()):
            pool[table[j]] = before[table[i]]
        return [pool]
    gone, source = st["groups"][0].tolist(), st["sources"][0].tolist()
    for s in gone:
        owner[table[s]], table[s] = EMPTY, EMPTY
    hole = 0
    live = sum(s >= 0 for s in owner)
    for page in range(live, case["pages"]):
        if owner[page] < 0:
            continue
        while owner[hole] >= 0:
            hole += 1
        pool[hole] = pool[page]
        owner[hole], table[owner[page]], owner[page] = owner[page], hole, EMPTY
    for i, s in zip(source, gone):
        page = owner.index(EMPTY)
        pool[page] = pool[table[i]]
        owner[page], table[s] = s, page
    return [pool] + [torch.tensor(v, dtype=torch.int32, device=DEV) for v in (table, owner)]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "scan":
        return _exact_scan(st)
    return _exact_steps(st) if case["op"] in ("scan_step", "step") else _exact_pages(st)
