"""Growth (g > 0) where a cluster of blocks walks a stream: the decays of any 32 consecutive tokens multiply to less than
fp32's largest value, those of 64 do not.  The results are still those of one token after the other, zero and tiny
states among them.

Bounds: state_mirror's.  Here |g| <= 2, and a's error is at most (2.8 + 1.25 * 2) u = 5.3 u (efla_scan.cuh), w's 6 u of
w x: with three roundings and the products' one each, below the 11 u a token that state_mirror counts.
"""
import pytest
import torch

from state_mirror import scan
from test_gpu_scan import check, close, dev, inputs, run_both

pytestmark = pytest.mark.gpu

TINY = 1e-30


def calm(inp, before, growing, per_token):
    """Nothing but the entering state up to the end of the growth [before, before + growing); decays behind it."""
    g, x, dO = inp["g"], inp["x"], inp["dO"]
    t = torch.arange(x.shape[-2])
    axis = (slice(None),) * (x.dim() - 2)
    grows = (t >= before) & (t < before + growing)
    after = (t >= before + growing) & (t < before + 2 * growing)
    g[(*axis, t < before)] = 0.0
    g[(*axis, grows)] = per_token
    g[(*axis, after)] = -per_token
    x[(*axis, t < before + growing)] = 0
    dO.mul_(TINY)
    return inp


@pytest.mark.parametrize("per_channel", [True, False])
@pytest.mark.parametrize("state", ["none", "zero", "tiny"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,before,per_token", [(257, 64, 1.4), (600, 128, 2.0), (1000, 45, 1.9)])
def test_growth_in_a_cluster(efla, cuda, T, before, per_token, dtype, state, per_channel):
    inp = inputs(1, 3, T, 64, {"f32": torch.float32, "bf16": torch.bfloat16}[dtype], per_channel, state=state != "none",
                 seed=T)
    calm(inp, before, 64, per_token)
    if state != "none":
        inp["S0"].mul_(TINY if state == "tiny" else 0)
        inp["dS_T"].mul_(TINY)
    got = check(efla, inp)
    assert all(torch.isfinite(v).all() for v in got.values() if v is not None)
    if state != "tiny":
        assert float(got["o"][:, :, :before + 64].abs().max()) == 0
    again = run_both(efla, inp, saved=False)
    assert all(torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("per_channel", [True, False])
def test_growth_in_packed_sequences(efla, cuda, per_channel):
    """Growing runs at the begin, in the middle and across a tile of several sequences; short ones between them."""
    lengths = [70, 333, 0, 5, 200, 128, 1, 90]
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    inp = inputs(len(lengths), 2, cu[-1], 128, torch.float32, per_channel, cu=cu, seed=2)
    inp["S0"].mul_(TINY)
    inp["dS_T"].mul_(TINY)
    inp["dO"].mul_(TINY)
    # (token 186 of sequence 1 is token 256 of the batch: the begin of a tile)
    for n, at in ((1, 0), (1, 186), (4, 60), (5, 64)):
        a = cu[n] + at
        inp["x"][:, cu[n]:a + 64] = 0
        inp["g"][:, cu[n]:a] = 0
        inp["g"][:, a:a + 64] = 1.5
        inp["g"][:, a + 64:min(a + 128, cu[n + 1])] = -1.5
    got = check(efla, inp, cu)
    assert all(torch.isfinite(v).all() for v in got.values())


def test_growth_of_what_cancels(efla, cuda):
    """The first token's input takes the entering state away: what is left of either alone would pass fp32's range."""
    inp = inputs(1, 3, 600, 64, torch.float32, False, seed=3)
    calm(inp, 128, 64, 1.4)
    inp["S0"].fill_(-1.0)
    inp["dS_T"].mul_(TINY)
    g = inp["g"][:, :, 128].double()
    inp["x"][:, :, 128] = (g.exp() * g / torch.expm1(g)).float()[..., None]
    d = dev(inp)
    o, S_T, saved = efla.efla_scan_fwd_save(d["x"], d["g"], S0=d["S0"])
    assert efla.efla_workspace_status(saved) == efla.EFLA_OK
    assert torch.isfinite(o).all() and torch.isfinite(S_T).all()
    ref = scan(inp["x"], inp["g"], inp["S0"])       # (its bound is of the size of the terms, about 1e35)
    close(o, ref["o"])
    close(S_T, ref["S_T"])


@pytest.mark.parametrize("per_channel", [True, False])
def test_non_finite_values_in_a_cluster(efla, cuda, per_channel):
    """Infinities and NaN of the inputs, where the parts of a pair are no longer sent as one."""
    inp = inputs(1, 3, 900, 64, torch.float32, per_channel, seed=4)
    clean = run_both(efla, inp)
    inp["x"][0, 1, 300, 5] = float("nan")
    inp["x"][0, 0, 700, 9] = float("inf")
    got = run_both(efla, inp)
    assert torch.isnan(got["o"][0, 1, 300:, 5]).all()
    assert not torch.isfinite(got["o"][0, 0, 700, 9])
    touched = torch.zeros(1, 3, 64, dtype=torch.bool)
    touched[0, 1, 5] = touched[0, 0, 9] = True
    for name in ("o", "dx"):
        same = (got[name] == clean[name]).cpu()
        assert same.permute(0, 1, 3, 2)[~touched].all(), name
    assert torch.equal(got["o"][:, :, :300], clean["o"][:, :, :300])
