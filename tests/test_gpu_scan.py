"""The per-channel gated recurrence on the GPU (forward, backward, one token) against fp64, elementwise.

Every comparison is |kernel - fp64| <= bound, the first-order error bound that state_mirror derives for fp32 arithmetic
and, for bf16 outputs, half a step of the result on top.
"""
import pytest
import torch

from state_mirror import EULER, EXACT, half_step, scan, step

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def close(got, ref, name=""):
    val, bound = ref
    got64 = got.double().cpu()
    bound = bound + half_step(got.dtype) * (val.abs() + bound) if got.dtype == torch.bfloat16 else bound + 1e-37
    bad = ~((got64 - val).abs() <= bound)
    assert got64.shape == val.shape
    if bad.any():
        at = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, first at {at}: {float(got64[at])!r}, "
                             f"fp64 {float(val[at])!r}, bound {float(bound[at]):.3e}")


def inputs(B, H, T, d, dtype, per_channel, cu=None, state=True, seed=0, spread=1.5):
    gen = torch.Generator().manual_seed(seed)
    lead = (H, T) if cu is not None else (B, H, T)
    r = lambda *s: torch.randn(*s, generator=gen)
    g = -torch.exp(-2.5 + spread * r(*lead, *((d,) if per_channel else ())))
    out = dict(x=r(*lead, d).to(dtype), g=g, S0=r(B, H, d) if state else None, dO=r(*lead, d).to(dtype),
               dS_T=r(B, H, d) if state else None)
    return out


def dev(inp):
    return {k: (None if v is None else v.cuda()) for k, v in inp.items()}


def run_both(efla, inp, cu=None, rule=EXACT, saved=True):
    """Forward and backward on the GPU: every output by name."""
    d = dev(inp)
    o, S_T, keep = efla.efla_scan_fwd_save(d["x"], d["g"], S0=d["S0"], cu_seqlens=cu, rule=rule)
    assert efla.efla_workspace_status(keep) == efla.EFLA_OK
    dx, dg, dS0 = efla.efla_scan_backward(d["x"], d["g"], d["dO"], S0=d["S0"], dS_T=d["dS_T"], cu_seqlens=cu,
                                          saved=keep if saved else None, rule=rule)
    torch.cuda.synchronize()
    return dict(o=o, S_T=S_T, dx=dx, dg=dg, dS0=dS0)


def check(efla, inp, cu=None, rule=EXACT, saved=True):
    got = run_both(efla, inp, cu, rule, saved)
    ref = scan(inp["x"], inp["g"], inp["S0"], cu, rule, inp["dO"], inp["dS_T"])
    for name, r in ref.items():
        close(got[name], r, name)
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("per_channel", [True, False])
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64, 65, 257])
def test_lengths(efla, cuda, T, per_channel, dtype):
    check(efla, inputs(2, 3, T, 64, DT[dtype], per_channel, seed=T))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("per_channel", [True, False])
@pytest.mark.parametrize("B,H,d", [(1, 1, 8), (1, 5, 8), (2, 3, 16), (1, 2, 40), (1, 3, 80), (2, 1, 128), (1, 2, 136),
                                   (1, 1, 192), (1, 2, 256), (1, 1, 1032)])
def test_widths(efla, cuda, B, H, d, per_channel, dtype):
    check(efla, inputs(B, H, 100, d, DT[dtype], per_channel, seed=d))


def test_width_of_one_vector_fp32(efla, cuda):
    check(efla, inputs(3, 7, 45, 4, torch.float32, True))
    check(efla, inputs(3, 7, 45, 12, torch.float32, False))


@pytest.mark.parametrize("per_channel", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_euler_rule_and_no_state(efla, cuda, dtype, per_channel):
    check(efla, inputs(2, 2, 130, 64, DT[dtype], per_channel, state=False, seed=3), rule=EULER)


@pytest.mark.parametrize("per_channel", [True, False])
def test_long_memory(efla, cuda, per_channel):
    """Decays near one over some thousand tokens: many chunks carry into each other."""
    inp = inputs(1, 2, 5003, 64, torch.float32, per_channel, seed=8)
    inp["g"] = inp["g"] * 1e-2
    check(efla, inp)


MIX = [1, 31, 0, 32, 33, 64, 200, 0, 0, 7, 130, 2]


def offsets(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return cu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("per_channel", [True, False])
@pytest.mark.parametrize("lengths", [MIX, [100], [0, 0, 5], [1] * 70, [500, 0, 1]], ids=str)
def test_packed(efla, cuda, lengths, per_channel, dtype):
    cu = offsets(lengths)
    inp = inputs(len(lengths), 3, cu[-1], 64, DT[dtype], per_channel, cu=cu, seed=11)
    got = check(efla, inp, cu)
    for n, length in enumerate(lengths):
        if length == 0:      # an empty sequence passes its state and its gradient through
            assert torch.equal(got["S_T"][n].cpu(), inp["S0"][n])
            assert torch.equal(got["dS0"][n].cpu(), inp["dS_T"][n])


@pytest.mark.parametrize("per_channel", [True, False])
def test_packed_many_sequences(efla, cuda, per_channel):
    """More sequences than a launch carries the offsets of, most of them short or empty, many in one tile."""
    lengths = [(7 * i) % 11 if i % 3 else 0 for i in range(400)] + [0] * 50 + [300]
    cu = offsets(lengths)
    inp = inputs(len(lengths), 2, cu[-1], 64, torch.bfloat16, per_channel, cu=cu, seed=12)
    got = check(efla, inp, cu)
    again = run_both(efla, inp, cu, saved=False)
    assert all(torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("count", [255, 256])
def test_captured_packed_batch(efla, cuda, count):
    """A captured call replayed after its list is gone; offsets that it would have to copy from there are refused."""
    lengths = [(5 * i) % 7 for i in range(count)]
    cu = offsets(lengths)
    inp = inputs(count, 2, cu[-1], 64, torch.float32, True, cu=cu, seed=13)
    want, t = run_both(efla, inp, cu), dev(inp)
    graph = torch.cuda.CUDAGraph()

    def train(cu):
        o, S_T, saved = efla.efla_scan_fwd_save(t["x"], t["g"], S0=t["S0"], cu_seqlens=cu)
        dx, dg, dS0 = efla.efla_scan_backward(t["x"], t["g"], t["dO"], S0=t["S0"], dS_T=t["dS_T"], saved=saved,
                                              cu_seqlens=cu)
        return dict(o=o, S_T=S_T, dx=dx, dg=dg, dS0=dS0)

    if count > 255:
        with pytest.raises(efla.EflaError) as refused, torch.cuda.graph(graph):
            train(list(cu))
        assert refused.value.status == efla.EFLA_ERR_INVALID_ARG
        graph = torch.cuda.CUDAGraph()
    pinned = torch.tensor(cu, dtype=torch.int32).pin_memory()
    with torch.cuda.graph(graph):
        out = train(list(cu) if count <= 255 else pinned)
    for _ in range(2):
        for v in out.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], want[k]) for k in want)


def test_change_of_formula(efla, cuda):
    """Decays on both sides of |g| = 1, where the gates change their formula, and next to it."""
    inp = inputs(1, 2, 160, 64, torch.float32, True, seed=6)
    edge = torch.tensor([1.0, 1.0 - 2.0 ** -24, 1.0 + 2.0 ** -23, 0.9999, 1.0001, 0.5, 2.0, 1e-7])
    inp["g"] = -edge[torch.randint(0, len(edge), inp["g"].shape, generator=torch.Generator().manual_seed(6))]
    check(efla, inp)
    inp["g"][:, :, ::2] *= -1           # growth and decay in turn
    check(efla, inp)


def test_packed_without_states(efla, cuda):
    cu = offsets(MIX)
    check(efla, inputs(len(MIX), 2, cu[-1], 128, torch.bfloat16, True, cu=cu, state=False), cu, rule=EULER)


@pytest.mark.parametrize("per_channel", [True, False])
def test_backward_without_saved_states_is_the_same_bits(efla, cuda, per_channel):
    for cu in (None, offsets(MIX)):
        B, T = (2, 300) if cu is None else (len(MIX), cu[-1])
        inp = inputs(B, 2, T, 64, torch.bfloat16, per_channel, cu=cu)
        a, b = run_both(efla, inp, cu), run_both(efla, inp, cu, saved=False)
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_same_bits_on_every_call(efla, cuda):
    d = dev(inputs(1, 16, 3000, 128, torch.bfloat16, True))
    first = None
    for _ in range(20):
        o, S_T, saved = efla.efla_scan_fwd_save(d["x"], d["g"], S0=d["S0"])
        out = (o, S_T, *efla.efla_scan_backward(d["x"], d["g"], d["dO"], S0=d["S0"], dS_T=d["dS_T"], saved=saved))
        first = first or out
        assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_resets_and_extreme_decays(efla, cuda):
    """g = -inf forgets all; very long and very short memories; g around the change of formula at 1/2."""
    inp = inputs(1, 2, 200, 64, torch.float32, True, seed=5)
    g = inp["g"]
    g[:, :, 50] = float("-inf")
    g[:, :, 51, ::2] = float("-inf")
    g[:, :, 100] = -80.0
    g[:, :, 120] = 0.0
    g[:, :, 121] = -1e-30
    g[:, :, 122] = -0.5
    g[:, :, 123] = -0.4999999
    g[:, :, 124] = -20.0
    g[:, :, 125] = 0.3          # growth is allowed
    g[:, :, 126] = 0.7
    got = check(efla, inp)
    assert torch.equal(got["o"][:, :, 50], torch.zeros_like(got["o"][:, :, 50]))
    g[:] = float("-inf")        # every token forgets: nothing is left
    got = check(efla, inp)
    assert float(got["o"].abs().max()) == 0 and float(got["dx"].abs().max()) == 0


@pytest.mark.parametrize("per_channel", [True, False])
def test_growth(efla, cuda, per_channel):
    """g > 0: a state that grows by up to e^2 a token, e^78 in all, and its gradients."""
    inp = inputs(1, 3, 39, 64, torch.float32, per_channel, seed=8)
    inp["g"].uniform_(1.5, 2.0, generator=torch.Generator().manual_seed(8))
    check(efla, inp)


def test_non_finite_inputs_stay_in_their_channel(efla, cuda):
    inp = inputs(1, 2, 100, 64, torch.float32, True)
    clean = run_both(efla, inp)
    inp["x"][0, 1, 40, 5] = float("nan")
    inp["x"][0, 0, 70, 9] = float("inf")
    got = run_both(efla, inp)
    assert torch.isnan(got["o"][0, 1, 40:, 5]).all() and torch.isinf(got["o"][0, 0, 70:, 9]).all()
    touched = torch.zeros(1, 2, 64, dtype=torch.bool)
    touched[0, 1, 5] = touched[0, 0, 9] = True
    for name in ("o", "dx", "dg"):
        same = (got[name] == clean[name]).cpu()
        assert same.permute(0, 1, 3, 2)[~touched].all(), name
    assert torch.equal(got["o"][:, :, :40], clean["o"][:, :, :40])


@pytest.mark.parametrize("per_channel", [True, False])
def test_packed_sequences_do_not_touch_each_other(efla, cuda, per_channel):
    """NaN and infinities of one sequence stay in it, forward and back, wherever its ends lie in the tiles."""
    cu = offsets([70, 5, 3, 1, 90, 64, 128, 30, 300, 2])
    inp = inputs(10, 2, cu[-1], 64, torch.float32, per_channel, cu=cu)
    clean = run_both(efla, inp, cu)
    for n in (0, 2, 4, 6, 8):
        for name in ("x", "dO"):
            inp[name][:, cu[n]:cu[n + 1]] = float("nan")
        inp["S0"][n], inp["dS_T"][n] = float("inf"), float("nan")
    got = run_both(efla, inp, cu)
    for n in (1, 3, 5, 7, 9):
        for name in ("o", "dx", "dg"):
            assert torch.equal(got[name][:, cu[n]:cu[n + 1]], clean[name][:, cu[n]:cu[n + 1]]), (n, name)
        assert torch.equal(got["S_T"][n], clean["S_T"][n]) and torch.equal(got["dS0"][n], clean["dS0"][n])
    assert torch.isnan(got["o"][:, cu[4]:cu[5]]).all() and torch.isnan(got["dx"][:, cu[4]:cu[5]]).all()


def test_backward_against_differences(efla, cuda):
    """The loss's directional derivatives by central differences of the fp64 forward."""
    inp = inputs(1, 2, 70, 16, torch.float32, True, seed=2)
    got = run_both(efla, inp)
    gen = torch.Generator().manual_seed(9)

    def loss(x, g, S0):
        r = scan(x, g, S0)
        return float((r["o"][0] * inp["dO"].double()).sum() + (r["S_T"][0] * inp["dS_T"].double()).sum())

    for key, grad in (("x", "dx"), ("g", "dg"), ("S0", "dS0")):
        args = {k: inp[k].double() for k in ("x", "g", "S0")}
        v = torch.randn(args[key].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        hi, lo = dict(args), dict(args)
        hi[key], lo[key] = args[key] + h * v, args[key] - h * v
        want = (loss(**hi) - loss(**lo)) / (2 * h)
        have = float((got[grad].double().cpu() * v).sum())
        # the difference's own error is of order h^2 and 1e-16 / h; the sum has 2240 terms of error ~1e-6
        assert abs(have - want) <= 1e-4 * (1 + float((got[grad].double().cpu() * v).abs().sum())) / 10


def test_state_in_place_and_carry(efla, cuda):
    """S_T may be S0; two halves give the whole."""
    inp = inputs(2, 2, 300, 64, torch.float32, True)
    d = dev(inp)
    o, S_T = efla.efla_scan_fwd(d["x"], d["g"], S0=d["S0"])
    S = d["S0"].clone()
    o2, _ = efla.efla_scan_fwd(d["x"], d["g"], S0=S, S_T=S)
    assert torch.equal(o, o2) and torch.equal(S, S_T)
    cut = lambda t, a, b: t[:, :, a:b].contiguous()
    oa, Sa = efla.efla_scan_fwd(cut(d["x"], 0, 131), cut(d["g"], 0, 131), S0=d["S0"])
    ob, Sb = efla.efla_scan_fwd(cut(d["x"], 131, 300), cut(d["g"], 131, 300), S0=Sa)
    ref = scan(inp["x"], inp["g"], inp["S0"])
    close(torch.cat([oa, ob], 2), ref["o"])
    close(Sb, ref["S_T"])


def test_empty_calls(efla, cuda):
    x, g, S0 = torch.zeros(2, 3, 0, 64).cuda(), torch.zeros(2, 3, 0, 64).cuda(), torch.randn(2, 3, 64).cuda()
    o, S_T = efla.efla_scan_fwd(x, g, S0=S0)
    assert o.numel() == 0 and torch.equal(S_T, S0)
    _, S_T = efla.efla_scan_fwd(x, g)
    assert float(S_T.abs().max()) == 0
    dx, dg, dS0 = efla.efla_scan_backward(x, g, x, S0=S0, dS_T=S0)
    assert torch.equal(dS0, S0)
    x = torch.zeros(3, 0, 64).cuda()
    o, S_T = efla.efla_scan_fwd(x, x, S0=S0, cu_seqlens=[0, 0, 0])
    assert torch.equal(S_T, S0)


def test_workspace_reuse_across_shapes_and_garbage(efla, cuda):
    """A workspace left with anything in it, or used by a call of another shape, changes nothing."""
    ws = torch.full((1 << 22,), 0xA5, dtype=torch.uint8, device="cuda")
    for T, H, d in ((300, 2, 64), (77, 3, 128), (2000, 1, 64), (33, 2, 64), (700, 20, 128)):
        inp = inputs(1, H, T, d, torch.float32, True, seed=T)
        dd = dev(inp)
        o, S_T = efla.efla_scan_fwd(dd["x"], dd["g"], S0=dd["S0"], workspace=ws)
        ref = scan(inp["x"], inp["g"], inp["S0"])
        close(o, ref["o"])
        close(S_T, ref["S_T"])
    assert efla.efla_workspace_status(ws) == efla.EFLA_OK


def test_streams_and_graphs(efla, cuda):
    """Two calls at once on two streams; a captured training step replayed on new inputs."""
    a, b = dev(inputs(1, 4, 3001, 128, torch.bfloat16, True, seed=1)), dev(inputs(1, 4, 2500, 128, torch.bfloat16, True, seed=2))
    want = [efla.efla_scan_fwd(t["x"], t["g"], S0=t["S0"]) for t in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, t in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(efla.efla_scan_fwd(t["x"], t["g"], S0=t["S0"]))
        torch.cuda.synchronize()
        for (o, S), (o2, S2) in zip(want, got):
            assert torch.equal(o, o2) and torch.equal(S, S2)
    # a stream as an argument, an object or an address; what the calls allocate is theirs until they have run
    for stream in (streams[0], streams[1].cuda_stream):
        outs = [efla.efla_scan_fwd(a["x"], a["g"], S0=a["S0"], stream=stream) for _ in range(3)]
        _, _, saved = efla.efla_scan_fwd_save(a["x"], a["g"], S0=a["S0"], stream=stream)
        grads = efla.efla_scan_backward(a["x"], a["g"], a["dO"], S0=a["S0"], dS_T=a["dS_T"], saved=saved, stream=stream)
        for _ in range(20):
            torch.empty(1 << 22, device="cuda").fill_(float("nan"))      # would land in memory freed too early
        torch.cuda.synchronize()
        assert all(torch.equal(o2, want[0][0]) and torch.equal(S2, want[0][1]) for o2, S2 in outs)
        ref = efla.efla_scan_backward(a["x"], a["g"], a["dO"], S0=a["S0"], dS_T=a["dS_T"])
        assert all(torch.equal(u, v) for u, v in zip(grads, ref))
    t = {k: v.clone() for k, v in a.items()}

    def train():
        o, S_T, saved = efla.efla_scan_fwd_save(t["x"], t["g"], S0=t["S0"])
        return (o, S_T, *efla.efla_scan_backward(t["x"], t["g"], t["dO"], S0=t["S0"], dS_T=t["dS_T"], saved=saved))

    with torch.cuda.stream(streams[0]):
        train()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = train()
    other = dev(inputs(1, 4, 3001, 128, torch.bfloat16, True, seed=3))
    for src in (other, a, other):
        for k in t:
            t[k].copy_(src[k])
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in out]
        assert all(torch.equal(u, v) for u, v in zip(got, train()))
    del graph


def test_offsets_past_32_bits(efla, cuda):
    """More than 2^31 elements and 2^32 bytes of g in one call: the last stream against fp64."""
    B, H, T, d = 1, 33, 512 * 1024, 128
    x = torch.zeros(B, H, T, d, dtype=torch.bfloat16, device="cuda")
    g = torch.full((B, H, T), -0.01, device="cuda")
    gen = torch.Generator().manual_seed(4)
    tail = torch.randn(300, d, generator=gen).bfloat16()
    x[0, H - 1, T - 300:] = tail.cuda()
    o, S_T = efla.efla_scan_fwd(x, g)
    ref = scan(tail[None, None], torch.full((1, 1, 300), -0.01))
    close(S_T[:, H - 1:], ref["S_T"])
    close(o[:, H - 1:, T - 300:], ref["o"])
    assert float(o[:, :H - 1].abs().max()) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("per_channel", [True, False])
@pytest.mark.parametrize("N,H,d", [(1, 1, 8), (3, 4, 64), (5, 16, 128), (2, 3, 136), (300, 1, 40)])
@pytest.mark.parametrize("rule", [EXACT, EULER])
def test_step(efla, cuda, N, H, d, per_channel, dtype, rule):
    gen = torch.Generator().manual_seed(N + d)
    S = torch.randn(N, H, d, generator=gen)
    Sd = S.cuda()
    for _ in range(3):
        x = torch.randn(N, H, d, generator=gen).to(DT[dtype])
        g = -torch.exp(-2.0 + 1.5 * torch.randn(N, H, *((d,) if per_channel else ()), generator=gen))
        h, bound = step(x, g, Sd.cpu(), rule)
        o = efla.efla_scan_step(x.cuda(), g.cuda(), Sd, rule=rule)
        close(Sd, (h, bound))
        close(o, (h, bound))


def test_steps_continue_a_forward(efla, cuda):
    inp = inputs(2, 3, 60, 64, torch.float32, True)
    d = dev(inp)
    ref = scan(inp["x"], inp["g"], inp["S0"])
    _, S = efla.efla_scan_fwd(d["x"][:, :, :50].contiguous(), d["g"][:, :, :50].contiguous(), S0=d["S0"])
    for t in range(50, 60):
        o = efla.efla_scan_step(d["x"][:, :, t].contiguous(), d["g"][:, :, t].contiguous(), S)
        close(o, tuple(v[:, :, t] for v in ref["o"]))
    close(S, ref["S_T"])
