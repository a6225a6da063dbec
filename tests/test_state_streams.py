"""Calls on a stream of their own: what they allocate belongs to that stream.  On the CPU with tensors that have no memory,
on the GPU behind work that the current stream has still queued for the memory it gave back."""
import contextlib
import types

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.utils._python_dispatch import TorchDispatchMode

MADE = ("empty", "empty_like", "new_empty", "zeros", "zeros_like", "new_zeros", "empty_strided", "new_empty_strided")


class Allocations(TorchDispatchMode):
    """Every allocation, with the stream that was current."""

    def __init__(self):
        super().__init__()
        self.stream, self.seen = None, []

    def __torch_dispatch__(self, func, types_, args=(), kwargs=None):
        name = func.overloadpacket.__name__
        if name in MADE:
            self.seen.append((name, self.stream))
        return func(*args, **(kwargs or {}))


@pytest.fixture
def calls(efla, monkeypatch):
    log, handed = Allocations(), []

    @contextlib.contextmanager
    def on(stream):
        before, log.stream = log.stream, stream
        yield
        log.stream = before

    ok = lambda *a: 0
    monkeypatch.setattr(efla, "lib", types.SimpleNamespace(
        efla_scan_workspace_bytes=lambda *a: 512, efla_scan_backward_workspace_bytes=lambda *a: 512,
        efla_pages_bytes=lambda n, m: 4 * (64 + 2 * m + 3 * n), efla_scan_fwd=ok, efla_scan_backward=ok, efla_scan_step=ok,
        efla_scan_step_paged=ok, efla_recurrent_step_paged=ok, efla_pages_init=ok, efla_pages_read=ok))
    monkeypatch.setattr(efla, "_call", lambda *a: None)
    monkeypatch.setattr(efla, "_tensor", lambda *a: 0)
    monkeypatch.setattr(efla, "_pool", lambda pool, *a: (0, 1024, 1024))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: ("current", str(device)))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("default", str(device)))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device=None: (raw, str(device)))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: handed.append((tuple(t.shape), s)))
    return efla, log, handed


@pytest.mark.parametrize("stream,want", [(1 << 20, (1 << 20, "cuda:1")), (0, ("default", "cuda:1")),
                                         (types.SimpleNamespace(cuda_stream=96), (96, "cuda:1"))], ids=str)
def test_allocations_are_made_on_the_calls_stream(calls, stream, want):
    efla, log, handed = calls
    with FakeTensorMode(allow_non_fake_inputs=True):
        new = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="cuda:1")
        x, S0, pool, mats = new(2, 3, 5, 64), new(2, 3, 64), new(4, 3, 64), new(4, 3, 64, 64)
        slots = new(2, dtype=torch.int32)
        with log:
            pages = efla.new_pages(4, 4, device="cuda:1", stream=stream)
            o, S_T, saved = efla.efla_scan_fwd_save(x, x, S0=S0, stream=stream)
            grads = efla.efla_scan_backward(x, x, x, S0=S0, saved=saved, stream=stream)
            results = [pages.block, o, S_T, saved, *grads, efla.efla_scan_step(S0, S0, S0, stream=stream),
                       efla.efla_scan_step_paged(S0, S0, pages, pool, slots, stream=stream),
                       efla.efla_recurrent_step_paged(S0, S0, S0, S0[..., 0], pages, mats, slots, stream=stream),
                       efla.efla_pages_read(pages, pool, slots, stream=stream)]
    assert len(log.seen) >= 12 and {s for _, s in log.seen} == {want}, log.seen
    assert all((tuple(t.shape), ("current", "cuda:1")) in handed for t in results)


def test_without_a_stream_the_current_one_is_taken(calls):
    efla, log, handed = calls
    with FakeTensorMode(allow_non_fake_inputs=True):
        x = torch.empty(2, 3, 64, device="cuda:1")
        with log:
            efla.efla_pages_read(efla.new_pages(4, 4, device="cuda:1"), x, torch.empty(2, device="cuda:1"))
    assert log.seen and all(s is None for _, s in log.seen) and not handed


@pytest.mark.gpu
def test_memory_that_the_current_stream_still_writes(efla, cuda):
    """The current stream has given a tensor back and will still fill it: a call on another stream does not get it."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(2, 4, 700, 64, generator=gen, device="cuda")
    g, S0 = -0.1 * torch.rand(2, 4, 700, 64, generator=gen, device="cuda"), torch.randn(2, 4, 64, generator=gen, device="cuda")
    slots = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    busy = torch.randn(4096, 4096, device="cuda")
    pages = efla.new_pages(2, 2)
    efla.efla_pages_fork(pages, None, torch.full_like(slots, -1), slots)

    def run(stream):
        o, S_T, saved = efla.efla_scan_fwd_save(x, g, S0=S0, stream=stream)
        grads = efla.efla_scan_backward(x, g, x, S0=S0, dS_T=S0, saved=saved, stream=stream)
        step = efla.efla_scan_step(S0, S0, S0.clone(), stream=stream)
        fresh = efla.new_pages(3, 5, stream=stream)
        rows = efla.efla_pages_read(pages, S0, slots, stream=stream)
        return [o, S_T, *grads, step, fresh.block[64:], rows]

    want = run(None)
    nbytes = sorted({t.untyped_storage().nbytes() for t in want} | {efla.efla_scan_workspace_bytes(2, 4, 700, 64, 64, torch.float32)})
    other = torch.cuda.Stream()
    for stream in (other, other.cuda_stream):
        torch.cuda.synchronize()
        other.wait_stream(torch.cuda.current_stream())
        S = S0.clone()                                  # (the step's own state is the caller's to order)
        torch.cuda.synchronize()
        given_back = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in nbytes for _ in range(4)]
        for _ in range(20):
            busy @ busy                                 # tens of milliseconds before the fills
        for t in given_back:
            t.fill_(0xFF)
        del given_back, t
        o, S_T, saved = efla.efla_scan_fwd_save(x, g, S0=S0, stream=stream)
        grads = efla.efla_scan_backward(x, g, x, S0=S0, dS_T=S0, saved=saved, stream=stream)
        step = efla.efla_scan_step(S0, S0, S, stream=stream)
        fresh = efla.new_pages(3, 5, stream=stream)
        rows = efla.efla_pages_read(pages, S0, slots, stream=stream)
        torch.cuda.synchronize()
        got = [o, S_T, *grads, step, fresh.block[64:], rows]
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert efla.efla_workspace_status(saved) == efla.EFLA_OK
