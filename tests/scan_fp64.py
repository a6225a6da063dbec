"""The per-channel gated recurrence in fp64 on any device, with first-order error bounds of the fp32 kernels that follow
their gates (csrc/efla_scan.cuh).

u = 2^-24.  A token takes h' to h = a h' + w x.  On the term a h' it adds a's error, at most 5 u for |g| < 1 and
(2.8 + 1.25 |g|) u elsewhere (2^-22.5 of the power, |g| 1.22 u of its rounded argument), a rounding of a product of decays,
one of the sum that the token is first part of, one of the state that is written, and a third of those of the runs that are
put together (a run has four tokens; a tile's, a cluster's and a turn's sums follow): 5 + 6 u, beyond |g| = 2 1.25 u more
per unit of |g|.  On w x: 6 u of w (g up to 2) and 5 roundings.  So c = 12 + 1.25 max(|g| - 2, 0) times u for the one and 12 u for
the other cover both, and the reverse recurrence c' = a (dO + c) alike.
"""
import torch

U = 2.0 ** -24
EXACT, EULER = 0, 1


def gates(g, rule):
    """a, w, w' by expm1 and, where a difference would cancel, by the series of the difference."""
    a = g.exp()
    if rule == EULER:
        return a, torch.ones_like(g), torch.zeros_like(g)
    near = g.abs() < 0.05
    safe = torch.where(near, torch.ones_like(g), g)
    term, w, slope = torch.ones_like(g), torch.ones_like(g), torch.full_like(g, 0.5)
    for n in range(1, 10):      # g^n / (n + 1)!, and n g^(n - 1) / (n + 1)! its derivative
        slope = slope if n == 1 else slope + n * term / (n + 1)
        term = term * g / (n + 1)
        w = w + term
    return a, torch.where(near, w, torch.expm1(safe) / safe), torch.where(near, slope, (a - torch.expm1(safe) / safe) / safe)


def reference(x, g, S0, dO, dS_T, cu=None, rule=EXACT):
    """{o, S_T, dx, dg, dS0: (value, bound)}, streams [.., T, d] from states [B, H, d] (none of them None)."""
    packed, T, d = cu is not None, x.shape[-2], x.shape[-1]
    shared = g.dim() < x.dim()
    B, H = S0.shape[:2]
    xs, up = x.double().reshape(-1, T, d), dO.double().reshape(-1, T, d)
    gs = g.double().reshape(-1, T, 1 if shared else d)
    a, w, dw = gates(gs, rule)
    far = 1.25 * (gs.abs() - 2).clamp_min(0)
    ca = 12 + far
    rows = (lambda s: list(s.double())) if packed else (lambda s: [s.double().reshape(-1, d)])
    back = (lambda r: torch.stack(r)) if packed else (lambda r: r[0].reshape(B, H, d))
    seqs = [(n, cu[n], cu[n + 1]) for n in range(B)] if packed else [(0, 0, T)]
    h, K, prev, Kprev, Mprev, G, KG, MG = (torch.zeros_like(xs) for _ in range(8))
    S, SK, D, DK = rows(S0), [torch.zeros_like(r) for r in rows(S0)], rows(dS_T), [torch.zeros_like(r) for r in rows(S0)]
    for n, y0, y1 in seqs:
        now, k, m = S[n], SK[n], S[n].abs()
        for t in range(y0, y1):
            prev[:, t], Kprev[:, t], Mprev[:, t] = now, k, m
            wx = w[:, t] * xs[:, t]
            k = a[:, t] * (k + ca[:, t] * m) + 12 * wx.abs()
            now, m = a[:, t] * now + wx, a[:, t] * m + wx.abs()
            h[:, t], K[:, t] = now, k
        S[n], SK[n] = now, k
        now, k, m = D[n], DK[n], D[n].abs()
        for t in range(y1 - 1, y0 - 1, -1):
            m = up[:, t].abs() + m
            k = k + m
            G[:, t], KG[:, t], MG[:, t] = up[:, t] + now, k, m
            now, k, m = a[:, t] * G[:, t], a[:, t] * (k + ca[:, t] * m), a[:, t] * m
        D[n], DK[n] = now, k
    # dg = G (a h' + w' x): w' to 24 u, three roundings
    e, terms = a * prev + dw * xs, a * Mprev + (dw * xs).abs()
    dg, kg = G * e, KG * terms + MG * (a * Kprev + (36 + far) * terms)
    if shared:      # over the channels: two additions in a lane, five over a warp, one for every 32 channels
        kg = (kg + (7 + (d + 31) // 32) * MG * terms).sum(-1)
        dg = dg.sum(-1)
    out = dict(o=(h.reshape(x.shape), K.reshape(x.shape)), S_T=(back(S), back(SK)),
               dx=((w * G).reshape(x.shape), (w * (KG + 12 * MG)).reshape(x.shape)),
               dg=(dg.reshape(g.shape), kg.reshape(g.shape)), dS0=(back(D), back(DK)))
    return {name: (v, U * b) for name, (v, b) in out.items()}


def compare(got, ref, name=""):
    """|got - ref| <= bound for every element; bf16 outputs with half a step of the result on top."""
    val, bound = ref
    assert got.shape == val.shape, name
    if got.dtype == torch.bfloat16:
        bound = bound + torch.finfo(got.dtype).eps / 2 * (val.abs() + bound)
    bad = ~((got.double() - val).abs() <= bound + 1e-37)
    if bad.any():
        at = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, first at {at}: {float(got[at])!r}, "
                             f"fp64 {float(val[at])!r}, bound {float(bound[at]):.3e}")
