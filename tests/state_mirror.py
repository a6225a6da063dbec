"""Plain fp64 implementations of the per-channel gated recurrence, the decode steps and the state cache's pages,
with the first-order error bounds that the fp32 kernels are held to.

Bounds.  u = 2^-24 is fp32's rounding.  A token's new state h = a h' + w x takes: a's error (expf: 1 ulp = 2 u, and as
much again for the products over a chunk), w's (below 4 u: one expf, one difference, one division; or a polynomial
whose cut is below u) and three roundings (w x, the sum, the product over a chunk).  So with M = |a| M' + |w x| (the
sum of the terms' sizes) each token adds at most 11 u M to the error, and the error of h is at most 11 u K with
K = |a| K' + M.  STEP = 12 leaves the rest for second order.  The reverse recurrence has the same form.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
STEP = 12          # roundings that one token adds, see above
EXACT, EULER = 0, 1


def half_step(dtype) -> float:
    """Largest relative error of one rounding to `dtype`."""
    return 0.0 if dtype == torch.float64 else torch.finfo(dtype).eps / 2


def gates(g, rule):
    """e^g, phi(g) = (e^g - 1) / g and phi'(g) in fp64 (Euler: e^g, 1, 0)."""
    a = g.exp()
    if rule == EULER:
        return a, torch.ones_like(g), torch.zeros_like(g)
    near = g.abs() < 1e-2
    safe = torch.where(near, torch.ones_like(g), g)
    series = 1 + g / 2 + g ** 2 / 6 + g ** 3 / 24 + g ** 4 / 120 + g ** 5 / 720
    slope = 0.5 + g / 3 + g ** 2 / 8 + g ** 3 / 30 + g ** 4 / 144 + g ** 5 / 840
    w = torch.where(near, series, torch.expm1(safe) / safe)
    dw = torch.where(near, slope, (a - w) / safe)
    dead = torch.isinf(g) & (g < 0)
    return a, torch.where(dead, 0.0, w), torch.where(dead, 0.0, dw)


def sequences(shape, cu):
    """(n, z rows as an index, first, last + 1) of every sequence; streams are [Z, T]."""
    return [(0, 0, shape[1])] if cu is None else [(n, cu[n], cu[n + 1]) for n in range(len(cu) - 1)]


def scan(x, g, S0=None, cu=None, rule=EXACT, dO=None, dS_T=None):
    """Forward, and with dO backward.  Returns {name: (value, bound)} of o, S_T and dx, dg, dS0 in fp64, bounds
    without the rounding to the output's type."""
    packed, d = cu is not None, x.shape[-1]
    shared = g.dim() < x.dim()
    H = x.shape[0] if packed else x.shape[1]
    B = len(cu) - 1 if packed else x.shape[0]
    T = x.shape[-2]
    xs = x.double().reshape(-1, T, d)
    gs = g.double().reshape(-1, T, 1 if shared else d).expand(xs.shape)
    Z = xs.shape[0]

    def rows(state):      # [B,H,d] -> [n][Z,d]
        s = torch.zeros(B, H, d, dtype=torch.float64) if state is None else state.double()
        return [s[n] for n in range(B)] if packed else [s.reshape(Z, d)]

    def back(rows_):      # the reverse
        return torch.stack(rows_) if packed else rows_[0].reshape(B, H, d)

    a, w, dw = gates(gs, rule)
    s0 = rows(S0)
    h, prev, Kprev, Mprev = (torch.zeros_like(xs) for _ in range(4))
    Kh = torch.zeros_like(xs)
    hT, KT = [r.clone() for r in s0], [torch.zeros_like(r) for r in s0]
    wx = w * xs
    for n, y0, y1 in sequences(xs.shape[:2], cu):
        now, M, K = s0[n], s0[n].abs(), torch.zeros_like(s0[n])
        for t in range(y0, y1):
            prev[:, t], Kprev[:, t], Mprev[:, t] = now, K, M
            now = a[:, t] * now + wx[:, t]
            M = a[:, t] * M + wx[:, t].abs()
            K = a[:, t] * K + M
            h[:, t], Kh[:, t] = now, K
        hT[n], KT[n] = now, K
    e = STEP * U
    out = {"o": (h.reshape(x.shape), e * Kh.reshape(x.shape)), "S_T": (back(hT), e * back(KT))}
    if dO is None:
        return out
    up, dst = dO.double().reshape(xs.shape), rows(dS_T)
    G, MG, KG = (torch.zeros_like(xs) for _ in range(3))
    d0, k0 = [r.clone() for r in dst], [torch.zeros_like(r) for r in dst]
    for n, y0, y1 in sequences(xs.shape[:2], cu):
        flow, M, K = dst[n], dst[n].abs(), torch.zeros_like(dst[n])
        for t in range(y1 - 1, y0 - 1, -1):
            G[:, t] = up[:, t] + flow
            M = up[:, t].abs() + M
            K = K + M
            MG[:, t], KG[:, t] = M, K
            flow, M, K = a[:, t] * G[:, t], a[:, t] * M, a[:, t] * (K + M)
        d0[n], k0[n] = flow, K
    # dg: G and h' with their errors, and phi' (its difference leaves at most 24 u), three roundings more
    terms = a * Mprev + (dw * xs).abs()
    dg = G * (a * prev + dw * xs)
    kg = KG * terms + MG * (a * Kprev + 3 * terms)
    if shared:            # the sum over the channels: four in a lane, five steps over a warp, a few strips
        kg = (kg + 2 * MG * terms).sum(-1)
        dg = dg.sum(-1)
    out["dx"] = ((w * G).reshape(x.shape), e * (w * (KG + MG)).reshape(x.shape))
    out["dg"] = (dg.reshape(g.shape), e * kg.reshape(g.shape))
    out["dS0"] = (back(d0), e * back(k0))
    return out


def step(x, g, S, rule=EXACT):
    """One token: (o, S) and the bound of both."""
    gg = g.double()[..., None].expand(x.shape) if g.dim() < x.dim() else g.double()
    a, w, _ = gates(gg, rule)
    h = a * S.double() + w * x.double()
    return h, STEP * U * (a * S.double().abs() + (w * x.double()).abs())


def delta_step(q, k, v, beta, g, S, rule=EXACT):
    """One token of the (gated) delta-rule recurrence in fp64: o, S and their bounds.

    r = k^T S and p = q^T S are sums of d products: four or two in a thread, then at most 13 partial sums: 18 u of the
    terms' sizes.  lambda and c the same; the gates add 6 u; the update three roundings.  40 u covers each term."""
    q, k, v, beta, S = (t.double() for t in (q, k, v, beta, S))
    lam = (k * k).sum(-1)
    gg = torch.zeros_like(lam) if g is None else g.double()
    if rule == EULER:
        alpha = abar = beta
    else:
        phi = lambda y: torch.where(y.abs() < 1e-6, 1 - y / 2 + y * y / 6, -torch.expm1(-y) / torch.where(y == 0, 1.0, y))
        alpha, abar = beta * phi(beta * lam), beta * phi(beta * lam - gg)
    dec = gg.exp()
    r = torch.einsum("nhi,nhij->nhj", k, S)
    w = (dec * alpha)[..., None] * r - abar[..., None] * v
    new = dec[..., None, None] * S - k[..., None] * w[..., None, :]
    o = torch.einsum("nhi,nhij->nhj", q, new)
    rm = torch.einsum("nhi,nhij->nhj", k.abs(), S.abs())
    wm = (dec * alpha)[..., None] * rm + abar[..., None] * v.abs()
    sm = dec[..., None, None] * S.abs() + k.abs()[..., None] * wm[..., None, :]
    om = dec[..., None] * torch.einsum("nhi,nhij->nhj", q.abs(), S.abs()) + (q * k).abs().sum(-1)[..., None] * wm
    return o, new, 40 * U * om, 40 * U * sm


class Cache:
    """The state cache on lists."""

    def __init__(self, n_pages, n_slots, pool):
        self.table, self.owner, self.pool = [-1] * n_slots, [-1] * n_pages, pool.clone()
        self.slot_error = self.full_error = False

    def _page(self, s):
        return self.table[s] if 0 <= s < len(self.table) else -1

    def fork(self, source, dest, copy=True):
        named, plan = set(), []
        for s, t in zip(source, dest):
            if t == -1:
                continue
            first = t not in named
            named.add(t)
            ok = first and 0 <= t < len(self.table) and self.table[t] == -1 and (s == -1 or self._page(s) >= 0)
            if ok:
                plan.append((t, self._page(s) if s != -1 else -1))
            else:
                self.slot_error = True
        before = self.pool.clone()
        for t, page in plan:
            if -1 not in self.owner:
                self.full_error = True
                continue
            p = self.owner.index(-1)
            self.owner[p], self.table[t] = t, p
            if copy:
                self.pool[p] = before[page] if page >= 0 else 0

    def copy(self, source, dest):
        named, before = set(), self.pool.clone()
        for s, t in zip(source, dest):
            if t == -1:
                continue
            first = t not in named
            named.add(t)
            if first and self._page(t) >= 0 and (s == -1 or self._page(s) >= 0):
                self.pool[self.table[t]] = before[self._page(s)] if s != -1 else 0
            else:
                self.slot_error = True

    def free(self, slots):
        for s in slots:
            if s == -1:
                continue
            if self._page(s) < 0:
                self.slot_error = True
            else:
                self.owner[self.table[s]], self.table[s] = -1, -1

    def compact(self):
        live = sum(o >= 0 for o in self.owner)
        holes = [p for p in range(live) if self.owner[p] < 0]
        late = [p for p in range(live, len(self.owner)) if self.owner[p] >= 0]
        for to, frm in zip(holes, late):
            self.pool[to] = self.pool[frm]
            self.table[self.owner[frm]], self.owner[to], self.owner[frm] = to, self.owner[frm], -1

    def write(self, rows, slots):
        named = set()
        for i, s in enumerate(slots):
            if s == -1:
                continue
            if s in named or self._page(s) < 0:
                self.slot_error = True
            else:
                self.pool[self.table[s]] = rows[i]
            named.add(s)
