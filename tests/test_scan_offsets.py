"""Offsets of packed batches that are not whole numbers of 32 bits are refused, not cut to size (CPU only)."""
import pytest
import torch


@pytest.mark.parametrize("cu", [[0, 2.5, 5], [0.0, 5.0], torch.tensor([0.0, 2.9, 5.0]), torch.tensor([0, 2 ** 32 + 2, 5]),
                                torch.tensor([0, -2 ** 32, 5]), [0, 2 ** 31, 5], torch.tensor([False, True]), [[0, 5]], [5]],
                         ids=str)
def test_refused(efla, cu):
    x = torch.zeros(2, 5, 64)
    for call in (lambda: efla.efla_scan_fwd(x, x, cu_seqlens=cu),
                 lambda: efla.efla_scan_fwd_save(x, x, cu_seqlens=cu),
                 lambda: efla.efla_scan_backward(x, x, x, cu_seqlens=cu)):
        with pytest.raises(ValueError, match="cu_seqlens"):
            call()


@pytest.mark.parametrize("cu", [[0, 2, 5], (0, 2, 5), torch.tensor([0, 2, 5]), torch.tensor([0, 2, 5], dtype=torch.int16),
                                torch.tensor([0, 9, 2, 9, 5, 9], dtype=torch.int32)[::2]], ids=str)
def test_taken(efla, cu):
    x = torch.zeros(2, 5, 64)
    got = efla._scan_shape(x, x, cu)[-1]
    assert got.dtype == torch.int32 and got.is_contiguous() and got.tolist() == [0, 2, 5]
