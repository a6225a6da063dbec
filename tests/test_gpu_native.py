"""The binding's native way against its Python way (an explicit stream takes the latter): the same bits, the same
refusals, and that ordinary calls take it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture
def data(efla, cuda):
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s, dtype=torch.float32: torch.randn(*s, generator=gen, device="cuda").to(dtype)
    N, H, d, slots = 5, 3, 64, 9
    pages = efla.new_pages(12, slots)
    pool = torch.zeros(12, H, d, device="cuda")
    mats = torch.zeros(12, H, d, d, device="cuda")
    all_slots = torch.arange(slots, dtype=torch.int32, device="cuda")
    efla.efla_pages_fork(pages, None, torch.full_like(all_slots, -1), all_slots)
    pool.copy_(r(12, H, d))
    mats.copy_(0.1 * r(12, H, d, d))
    bf = torch.bfloat16
    return dict(x=r(N, H, d, dtype=bf), g=-r(N, H, d).abs(), gs=-r(N, H).abs(), S=r(N, H, d), pages=pages, pool=pool, mats=mats,
                slots=torch.tensor([4, -1, 0, 8, 2], dtype=torch.int32, device="cuda"),
                source=torch.tensor([4, 3, -1, 7, 5], dtype=torch.int32, device="cuda"),
                q=0.1 * r(N, H, d), k=0.1 * r(N, H, d), v=r(N, H, d), beta=torch.sigmoid(r(N, H)),
                X=r(2, H, 70, d, dtype=bf), G=-r(2, H, 70).abs(), dO=r(2, H, 70, d, dtype=bf), S0=r(2, H, d), dS_T=r(2, H, d))


def both_ways(call, *state):
    """call(stream) natively and through Python, from the same state tensors: the results and states of both."""
    before = [t.clone() for t in state]
    outs = []
    for stream in (None, torch.cuda.current_stream()):
        for t, b in zip(state, before):
            t.copy_(b)
        out = call(stream)
        outs.append([t.clone() for t in (out if isinstance(out, tuple) else (out,)) if t is not None] +
                    [t.clone() for t in state])
    torch.cuda.synchronize()
    assert len(outs[0]) == len(outs[1])
    for a, b in zip(*outs):
        assert a.dtype == b.dtype and torch.equal(a, b)


def test_same_as_the_python_way(efla, data):
    D, pages = data, data["pages"]
    both_ways(lambda s: efla.efla_scan_step(D["x"], D["g"], D["S"], stream=s), D["S"])
    both_ways(lambda s: efla.efla_scan_step(D["x"], D["gs"], D["S"], stream=s, rule=efla.EFLA_RULE_EULER), D["S"])
    for source in (None, D["source"]):
        both_ways(lambda s: efla.efla_scan_step_paged(D["x"], D["g"], pages, D["pool"], D["slots"], source=source, stream=s),
                  D["pool"])
        for g in (None, D["gs"]):
            both_ways(lambda s: efla.efla_recurrent_step_paged(D["q"], D["k"], D["v"], D["beta"], pages, D["mats"],
                                                               D["slots"], source=source, g=g, stream=s), D["mats"])
    lists = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 5, -1], [1, 2, 3])]
    both_ways(lambda s: efla.efla_pages_copy(pages, D["mats"], *lists, stream=s), D["mats"], pages.block)
    both_ways(lambda s: efla.efla_pages_free(pages, lists[1], stream=s), pages.block)
    both_ways(lambda s: efla.efla_pages_compact(pages, D["mats"], stream=s), D["mats"], pages.block)
    both_ways(lambda s: efla.efla_pages_fork(pages, D["mats"], *lists, stream=s), D["mats"], pages.block)
    for cu in (None, [0, 20, 20, 140], torch.tensor([0, 20, 20, 140], dtype=torch.int32)):
        X, G, dO = (D[k] if cu is None else D[k].flatten(0, 0).transpose(0, 1).reshape(3, 140, *D[k].shape[3:]).contiguous()
                    for k in ("X", "G", "dO"))
        S0, dS_T = (D[k] if cu is None else torch.cat([D[k], D[k][:1]]) for k in ("S0", "dS_T"))
        for want in (True, False):
            both_ways(lambda s: efla.efla_scan_fwd(X, G, S0=S0, cu_seqlens=cu, want_state=want, stream=s))
        saved = efla.efla_scan_fwd_save(X, G, S0=S0, cu_seqlens=cu)[2]
        for keep in (saved, None):
            both_ways(lambda s: efla.efla_scan_backward(X, G, dO, S0=S0, dS_T=dS_T, saved=keep, cu_seqlens=cu, stream=s))
        both_ways(lambda s: efla.efla_scan_backward(X, G, dO, cu_seqlens=cu, want_dS0=False, stream=s))
    assert efla.efla_pages_status(pages) == efla.EFLA_OK


def test_ordinary_calls_take_it(efla, data):
    D, pages, n, e = data, data["pages"], efla._native, efla.lib.entries
    block = (pages.block, pages.n_pages, pages.n_slots)
    assert n.scan_step(e, D["x"], D["g"], D["S"], None, 0) is not None
    assert n.scan_step_paged(e, D["x"], D["g"], *block, D["pool"], D["slots"], None, None, 0) is not None
    assert n.recurrent_step_paged(e, D["q"], D["k"], D["v"], D["beta"], *block, D["mats"], D["slots"], None, None, None, 0) \
        is not None
    assert n.scan_fwd(e, D["X"], D["G"], D["S0"], None, None, None, None, True, 0) is not None
    assert n.scan_fwd(e, D["X"][0], D["G"][0], None, [0, 5, 70], None, None, None, True, 0) is not None
    assert n.scan_backward(e, D["X"], D["G"], D["dO"], None, None, None, None, True, 0) is not None
    assert n.pages_compact(e, *block, D["pool"]) == 0
    layer = torch.zeros(12, 4, 3, 64, device="cuda")[:, 2]          # a layer of a larger pool
    assert n.scan_step_paged(e, D["x"], D["g"], *block, layer, D["slots"], None, None, 0) is not None
    # not ordinary: the Python layer's
    assert n.scan_step(e, D["x"].cpu(), D["g"], D["S"], None, 0) is None
    assert n.scan_step(e, D["x"], D["g"], D["S"].transpose(0, 1), None, 0) is None
    assert n.scan_step(e, D["x"], D["g"], D["S"], None, None) is None
    assert n.scan_step(None, D["x"], D["g"], D["S"], None, 0) is None
    assert n.scan_step(e, D["x"]) is None


def test_refusals_on_the_gpu(efla, data):
    D, pages = data, data["pages"]
    half = torch.zeros(2, 3, 70, 64, dtype=torch.float16, device="cuda")
    strided = D["X"].transpose(1, 2)
    for bad in (lambda: efla.efla_scan_fwd(half, D["G"]),
                lambda: efla.efla_scan_fwd(strided, D["G"]),
                lambda: efla.efla_scan_fwd(D["X"], D["G"].double()),
                lambda: efla.efla_scan_fwd(D["X"], D["G"][:, :, :5]),
                lambda: efla.efla_scan_fwd(D["X"], D["G"], S0=D["S0"][:1]),
                lambda: efla.efla_scan_fwd(D["X"], D["G"], o=D["X"].float()),
                lambda: efla.efla_scan_fwd(D["X"], D["G"].cpu()),
                lambda: efla.efla_scan_backward(D["X"], D["G"], D["dO"].float()),
                lambda: efla.efla_scan_step(D["x"], D["g"], D["S"][:4]),
                lambda: efla.efla_scan_step_paged(D["x"], D["g"], pages, D["pool"][:11], D["slots"]),
                lambda: efla.efla_scan_step_paged(D["x"], D["g"], pages, D["pool"], D["slots"].long()),
                lambda: efla.efla_scan_step_paged(D["x"], D["g"], pages, D["pool"], D["slots"], source=D["source"][:3]),
                lambda: efla.efla_scan_step_paged(D["x"], D["g"], pages, D["pool"].bfloat16(), D["slots"]),
                lambda: efla.efla_recurrent_step_paged(D["q"], D["k"], D["v"], D["beta"], pages, D["pool"], D["slots"]),
                lambda: efla.efla_pages_copy(pages, D["mats"], D["slots"], D["slots"][:2]),
                lambda: efla.efla_pages_free(pages, D["slots"].float()),
                lambda: efla.efla_pages_compact(pages, D["mats"][:3])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(efla.EflaError) as small:
        efla.efla_scan_fwd(D["X"], D["G"], workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    assert small.value.status == efla.EFLA_ERR_INVALID_ARG
    with pytest.raises(efla.EflaError) as inside:      # the states' input inside the output
        efla.efla_scan_step(D["S"], D["g"], D["S"])
    assert inside.value.status == efla.EFLA_ERR_INVALID_ARG
    with pytest.raises(efla.EflaError) as offsets:
        efla.efla_scan_fwd(D["X"][0], D["G"][0], cu_seqlens=[0, 30, 20, 70])
    assert offsets.value.status == efla.EFLA_ERR_INVALID_ARG
    with pytest.raises(efla.EflaError):
        efla.efla_scan_fwd(D["X"], D["G"], rule=7)
    assert efla.efla_pages_status(pages) == efla.EFLA_OK


def test_runs_of_calls_without_waiting(efla, data):
    """Calls that each need the one before, of the library and of PyTorch in turn, queued at once: the bits of the same
    calls with a wait after each."""
    D, pages = data, data["pages"]
    ones = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    zero = torch.full_like(ones, -1)
    x = D["x"][:3].contiguous()
    state = (D["pool"], D["mats"], pages.block)
    before = [t.clone() for t in state]

    def run(wait):
        for t, b in zip(state, before):
            t.copy_(b)
        done, X = [], D["X"].clone()
        mark = (lambda *t: (done.extend(t), torch.cuda.synchronize())) if wait else (lambda *t: done.extend(t))
        for i in range(40):
            o = efla.efla_scan_step_paged(x, D["g"][:3].contiguous(), pages, D["pool"], ones)
            mark(o)
            oo, S_T, saved = efla.efla_scan_fwd_save(X, D["G"], S0=D["S0"])
            mark(oo, S_T)
            grads = efla.efla_scan_backward(X, D["G"], oo, S0=D["S0"], saved=saved)
            mark(*grads)
            X = torch.tanh(grads[0]).to(X.dtype)
            r = efla.efla_recurrent_step_paged(D["q"], D["k"], D["v"], D["beta"], pages, D["mats"], D["slots"])
            mark(r)
            efla.efla_pages_free(pages, ones)
            mark()
            efla.efla_pages_compact(pages, D["mats"])
            mark()
            efla.efla_pages_fork(pages, D["mats"], zero if i % 3 == 0 else zero + 5, ones)
            mark()
            efla.efla_pages_copy(pages, D["mats"], ones.flip(0), ones)
            mark(efla.efla_pages_read(pages, D["mats"], ones))
            D["mats"].mul_(0.9)
        torch.cuda.synchronize()
        return [t.clone() for t in (*done, *state)]

    want, got = run(True), run(False)
    assert len(want) == len(got) and all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    for t, b in zip(state, before):
        t.copy_(b)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        o = efla.efla_scan_step_paged(x, D["g"][:3].contiguous(), pages, D["pool"], ones)
        efla.efla_pages_free(pages, ones)
        efla.efla_pages_compact(pages, D["mats"])
        efla.efla_pages_fork(pages, D["mats"], zero + 5, ones)
        r = efla.efla_recurrent_step_paged(D["q"], D["k"], D["v"], D["beta"], pages, D["mats"], D["slots"])
    for t, b in zip(state, before):
        t.copy_(b)
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    captured = [t.clone() for t in (o, r, *state)]
    for t, b in zip(state, before):
        t.copy_(b)
    for _ in range(20):
        o = efla.efla_scan_step_paged(x, D["g"][:3].contiguous(), pages, D["pool"], ones)
        efla.efla_pages_free(pages, ones)
        efla.efla_pages_compact(pages, D["mats"])
        efla.efla_pages_fork(pages, D["mats"], zero + 5, ones)
        r = efla.efla_recurrent_step_paged(D["q"], D["k"], D["v"], D["beta"], pages, D["mats"], D["slots"])
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, (o, r, *state)))
    assert efla.efla_pages_status(pages) == efla.EFLA_OK


@pytest.mark.parametrize("packed", [False, True])
def test_states_in_place_through_queued_calls(efla, cuda, packed):
    """A prompt in pieces, each from the state that the one before left in the same memory, queued at once."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    B, H, T, d = 3, 4, 1500, 128
    cu = [0, 700, 700, T] if packed else None
    lead = (H, T) if packed else (B, H, T)
    x = torch.randn(*lead, d, generator=gen, device="cuda")
    g = -0.01 * torch.rand(*lead, d, generator=gen, device="cuda")
    S0 = torch.randn(B, H, d, generator=gen, device="cuda")

    def run(wait):
        S, out = S0.clone(), []
        for _ in range(60):
            out.append(efla.efla_scan_fwd(x, g, S0=S, S_T=S, cu_seqlens=cu)[0][..., -1, :].clone() if wait else
                       efla.efla_scan_fwd(x, g, S0=S, S_T=S, cu_seqlens=cu)[0])
            if wait:
                torch.cuda.synchronize()
        return [o if wait else o[..., -1, :].clone() for o in out] + [S]

    want, got = run(True), run(False)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_two_streams_that_wait_for_each_other(efla, cuda):
    """Calls on two streams that need each other's results through events, queued at once, and the same captured."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x, g, S0 = r(2, 4, 900, 64), -0.1 * r(2, 4, 900).abs(), r(2, 4, 64)
    xt, gt = r(2, 4, 64), -0.1 * r(2, 4, 64).abs()
    other = torch.cuda.Stream()
    S = S0.clone()

    def turn():      # here: a prompt's piece; there: a token on its state; here again: the next piece
        main = torch.cuda.current_stream()
        efla.efla_scan_fwd(x, g, S0=S, S_T=S)
        other.wait_stream(main)
        with torch.cuda.stream(other):
            o = efla.efla_scan_step(xt, gt, S)
            torch.mul(S, 0.5, out=S)
            o2 = efla.efla_scan_step(xt, gt, S)
        main.wait_stream(other)
        out = efla.efla_scan_fwd(x, g, S0=S, S_T=S)[0]
        return o, o2, out

    def run(wait):
        S.copy_(S0)
        keep = []
        for _ in range(30):
            keep.append(turn())
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return [t.clone() for ts in keep for t in ts] + [S.clone()]

    want, got = run(True), run(False)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = turn()
    S.copy_(S0)
    for _ in range(30):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*outs, S), want[-4:]))
