"""The per-channel gated recurrence against fp64 in the launch shapes that its large calls take: strips of 32, 64 and 128
channels, each by single blocks and by clusters over several turns, of several heads, of one, and of a part of one; and
offsets past 32 bits."""
import pytest
import torch

from scan_fp64 import EULER, EXACT, compare, reference

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}

# (heads, tokens, channels) by the width of a strip, whether single blocks or clusters take it, and what a strip holds
SHAPES = [
    # 32 channels, single blocks of several turns: parts of wide heads, one head, four heads (the last strip not full)
    (64, 1100, 128), (77, 300, 80), (296, 300, 32), (999, 300, 8),
    # 32 channels, clusters of several turns
    (50, 700, 80), (77, 1500, 32), (333, 700, 16), (5, 1900, 136),
    # 64 channels, single blocks
    (77, 200, 192), (296, 200, 64), (701, 200, 32), (999, 300, 16),
    # 64 channels, clusters
    (20, 1500, 256), (77, 1500, 64), (333, 1500, 16),
    # 128 channels, single blocks: a layer's heads and more
    (148, 130, 256), (296, 300, 128), (444, 260, 128), (999, 100, 32), (60, 500, 1032),
    # 128 channels, clusters
    (200, 300, 256), (77, 300, 128), (50, 300, 80), (99, 300, 64), (701, 400, 16),
]


def inputs(H, T, d, dtype, per_channel, cu=None, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    B = 1 if cu is None else len(cu) - 1
    lead = (B, H, T) if cu is None else (H, T)
    g = -torch.exp(-2.5 + 1.5 * r(*lead, *((d,) if per_channel else ())))
    return dict(x=r(*lead, d).to(dtype), g=g, S0=r(B, H, d), dO=r(*lead, d).to(dtype), dS_T=r(B, H, d))


def check(efla, c, cu=None, rule=EXACT):
    o, S_T, saved = efla.efla_scan_fwd_save(c["x"], c["g"], S0=c["S0"], cu_seqlens=cu, rule=rule)
    dx, dg, dS0 = efla.efla_scan_backward(c["x"], c["g"], c["dO"], S0=c["S0"], dS_T=c["dS_T"], saved=saved, cu_seqlens=cu,
                                          rule=rule)
    assert efla.efla_workspace_status(saved) == efla.EFLA_OK
    got = dict(o=o, S_T=S_T, dx=dx, dg=dg, dS0=dS0)
    for name, ref in reference(**c, cu=cu, rule=rule).items():
        compare(got[name], ref, name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("per_channel", [True, False])
@pytest.mark.parametrize("H,T,d", SHAPES)
def test_dense(efla, cuda, H, T, d, per_channel, dtype):
    check(efla, inputs(H, T, d, DT[dtype], per_channel, seed=H + d))


@pytest.mark.parametrize("per_channel", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,d", [(64, 128), (444, 128), (999, 16), (150, 192), (20, 256), (77, 64)])
def test_packed(efla, cuda, H, d, dtype, per_channel):
    cu = [0]
    for n in (1, 40, 0, 128, 3, 97, 0, 0, 260, 5):
        cu.append(cu[-1] + n)
    check(efla, inputs(H, cu[-1], d, DT[dtype], per_channel, cu=cu, seed=d), cu)


@pytest.mark.parametrize("H,T,d", [(64, 300, 128), (444, 100, 128), (5, 700, 136), (999, 70, 16)])
def test_euler_rule(efla, cuda, H, T, d):
    check(efla, inputs(H, T, d, torch.bfloat16, True, seed=3), rule=EULER)


@pytest.mark.parametrize("H,d", [(16400, 128), (10930, 192)])
def test_offsets_past_32_bits(efla, cuda, H, d):
    """More than 2^31 elements of x, dO, g and every gradient, so more than 2^32 bytes of each; values everywhere, the
    first, a middle and the last streams against fp64.  Heads that a strip divides, and wider ones."""
    T = 1024
    gen = torch.Generator(device="cuda").manual_seed(d)
    new = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="cuda")
    x, dO = (new(1, H, T, d, dtype=torch.bfloat16).normal_(generator=gen) for _ in range(2))
    g = new(1, H, T, d).uniform_(-1.5, 0, generator=gen)
    S0, dS_T = (new(1, H, d).normal_(generator=gen) for _ in range(2))
    assert x.numel() > 2 ** 31
    o, S_T, saved = efla.efla_scan_fwd_save(x, g, S0=S0)
    dx, dg, dS0 = efla.efla_scan_backward(x, g, dO, S0=S0, dS_T=dS_T, saved=saved)
    assert efla.efla_workspace_status(saved) == efla.EFLA_OK
    for at in (0, 1, H // 2, H - 2, H - 1):
        s = slice(at, at + 1)
        ref = reference(x[:, s], g[:, s], S0[:, s], dO[:, s], dS_T[:, s])
        for name, t in dict(o=o, S_T=S_T, dx=dx, dg=dg, dS0=dS0).items():
            compare(t[:, s], ref[name], f"{name} of stream {at}")
    del x, dO, g, o, dx, dg, saved
    torch.cuda.empty_cache()
