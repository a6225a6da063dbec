"""Calls without a token or without a stream: the workspace's error word is that of the call, whatever was there before."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def garbage(n):
    return torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("packed", [False, True])
def test_no_tokens(efla, cuda, packed):
    B, H, d = 3, 2, 64
    cu = [0] * (B + 1) if packed else None
    x = torch.zeros((H, 0, d) if packed else (B, H, 0, d), device="cuda")
    S0 = torch.randn(B, H, d, device="cuda")
    ws = garbage(4096)
    for S in (S0, None):
        for given in (ws, None):
            _, S_T, saved = efla.efla_scan_fwd_save(x, x, S0=S, cu_seqlens=cu, saved=given)
            if given is None:      # memory that held something else
                saved.fill_(0xA5)
                _, S_T, saved = efla.efla_scan_fwd_save(x, x, S0=S, cu_seqlens=cu, saved=saved)
            assert efla.efla_workspace_status(saved) == efla.EFLA_OK
            assert torch.equal(S_T, torch.zeros_like(S0) if S is None else S)
            ws.fill_(0xA5)
    # the states in place, or not wanted: the word is cleared all the same
    S = S0.clone()
    efla.efla_scan_fwd(x, x, S0=S, S_T=S, cu_seqlens=cu, workspace=ws)
    assert efla.efla_workspace_status(ws) == efla.EFLA_OK and torch.equal(S, S0)
    ws.fill_(0xA5)
    efla.efla_scan_fwd(x, x, S0=S, cu_seqlens=cu, workspace=ws, want_state=False)
    assert efla.efla_workspace_status(ws) == efla.EFLA_OK
    saved = efla.efla_scan_fwd_save(x, x, S0=S0, cu_seqlens=cu)[2]
    for keep in (saved, None):
        for want in (True, False):
            ws.fill_(0xA5)
            dS0 = efla.efla_scan_backward(x, x, x, S0=S0, dS_T=S0, saved=keep, cu_seqlens=cu, want_dS0=want, workspace=ws)[2]
            assert efla.efla_workspace_status(ws) == efla.EFLA_OK
            assert dS0 is None or torch.equal(dS0, S0)


@pytest.mark.parametrize("B,H", [(0, 3), (2, 0)])
def test_no_streams(efla, cuda, B, H):
    x = torch.zeros(B, H, 5, 64, device="cuda")
    held = [garbage(n) for n in (256, 512, 1024, 4096) for _ in range(8)]      # what new memory may hold
    del held
    o, S_T, saved = efla.efla_scan_fwd_save(x, x)
    assert o.shape == x.shape and S_T.shape == (B, H, 64)
    assert efla.efla_workspace_status(saved) == efla.EFLA_OK
    dx, dg, dS0 = efla.efla_scan_backward(x, x, x, saved=saved)
    assert dx.shape == dg.shape == x.shape and dS0.shape == (B, H, 64)
