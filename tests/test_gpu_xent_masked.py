"""Linear cross entropy: what tokens without a loss hold, and upstream gradients of unlike size."""
import pytest
import torch

import fft_long_convolution_flashconv_amd as pkg
import lm_reference as ref
from parity_util import device, say

pytestmark = pytest.mark.gpu
DT = ref.DT


# (T, D, V): widths with and without padding, tiles of every fp32 side, several per side
@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,D,V", [(3, 2, 5), (70, 64, 300), (300, 65, 2000), (1100, 128, 1300)])
def test_ignored_tokens_may_hold_anything(io, T, D, V):
    """NaN and infinity in x of tokens without a loss: the other tokens' gradients are as if those were not there."""
    say("xent masked x", io, T, D, V)
    g = torch.Generator().manual_seed(T + D)
    x = torch.randn(T, D, generator=g).to(DT[io])
    w = (torch.randn(V, D, generator=g) * (2.0 / D ** 0.5)).to(DT[io])
    labels = torch.randint(0, V, (T,), generator=g)
    labels[::3], labels[-1] = -100, V + 1
    off = (labels < 0) | (labels >= V)
    bad = x.clone()
    bad[off] = torch.tensor([float("nan"), float("inf"), -float("inf")]).to(DT[io]).repeat(D)[:D]
    dloss = torch.rand(T, generator=g) + 0.5
    dev = device()
    loss, lse = pkg.linear_xent(bad.to(dev), w.to(dev), labels.to(dev), return_lse=True)
    dx, dw = pkg.linear_xent_bwd(bad.to(dev), w.to(dev), labels.to(dev), lse, dloss.to(dev))
    assert not dx[off.to(dev)].any() and not loss[off.to(dev)].any()
    lx, lw = ref.leaf(x), ref.leaf(w)
    (ref.linear_xent(lx, lw, labels)[0] * dloss.double()).sum().backward()
    ref.close(dx, lx.grad, io, roundings=2, what="dx")
    ref.close(dw, lw.grad, io, roundings=2, what="dw")
