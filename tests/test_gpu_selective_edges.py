"""The selective scan's gradients where there are no channels."""
import pytest
import torch

import fft_long_convolution_flashconv_amd as pkg
from parity_util import device

pytestmark = pytest.mark.gpu


def test_no_channels():
    """Without channels B and C have gradients all the same: sums over no channels."""
    dev = device()
    junk = torch.full((3, 2, 4, 5), 7.0, device=dev)
    del junk  # (what the gradients' memory may hold)
    u, A = torch.empty(3, 0, 5, device=dev), torch.empty(0, 4, device=dev)
    Bm, C = torch.randn(3, 2, 4, 5).to(dev), torch.randn(3, 2, 4, 5).to(dev)
    y, saved = pkg.selective_scan(u, u, A, Bm, C, return_saved=True)
    g = pkg.selective_scan_bwd(u, u, A, Bm, C, u, saved)
    assert y.shape == u.shape and g.du.shape == u.shape and g.dA.shape == A.shape
    assert g.dB.shape == Bm.shape and g.dC.shape == C.shape and not g.dB.any() and not g.dC.any()
