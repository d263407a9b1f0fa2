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


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
def test_an_infinite_gradient_stays_with_its_token(io):
    """dx of the other tokens is what it is without it, also where theirs are large."""
    T, D, V = 40, 64, 200
    g = torch.Generator().manual_seed(8)
    x = torch.randn(T, D, generator=g).to(DT[io])
    w = (torch.randn(V, D, generator=g) * (2.0 / D ** 0.5)).to(DT[io])
    labels = torch.randint(0, V, (T,), generator=g)
    dloss = 100.0 * (torch.rand(T, generator=g) + 0.5)
    dloss[3], dloss[7] = float("inf"), float("nan")
    dev = device()
    _, lse = pkg.linear_xent(x.to(dev), w.to(dev), labels.to(dev), return_lse=True)
    dx, _ = pkg.linear_xent_bwd(x.to(dev), w.to(dev), labels.to(dev), lse, dloss.to(dev))
    finite = torch.isfinite(dloss)
    lx = ref.leaf(x[finite])
    (ref.linear_xent(lx, w.double(), labels[finite])[0] * dloss[finite].double()).sum().backward()
    ref.close(dx[finite.to(dev)], lx.grad, io, roundings=2, what="dx")
    assert not torch.isfinite(dx[~finite.to(dev)]).any(dim=1).all()


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
def test_upstream_gradients_of_unlike_size(io):
    """|dloss| from 2^12 down to 2^-8: dx of every token by itself, and dw of the labels that only small ones have.

    G is held in fp16 as a share of the largest |dloss| times 2^15, so its entries are off by up to 2^-40 of the largest,
    beside the half ulp of the type; over V entries of a row and w's of like size these add up to sqrt(V) 2^-40 of it."""
    T, D, V = 63, 64, 1000
    say("xent unlike dloss", io)
    g = torch.Generator().manual_seed(9)
    x = torch.randn(T, D, generator=g).to(DT[io])
    w = (torch.randn(V, D, generator=g) * (2.0 / D ** 0.5)).to(DT[io])
    labels = torch.randperm(V, generator=g)[:T]
    dloss = 2.0 ** torch.linspace(12, -8, T)
    dev = device()
    _, lse = pkg.linear_xent(x.to(dev), w.to(dev), labels.to(dev), return_lse=True)
    dx, dw = pkg.linear_xent_bwd(x.to(dev), w.to(dev), labels.to(dev), lse, dloss.to(dev))
    lx, lw = ref.leaf(x), ref.leaf(w)
    (ref.linear_xent(lx, lw, labels)[0] * dloss.double()).sum().backward()
    for t in range(T):
        extra = V ** 0.5 * 2.0 ** -40 * float(dloss.max() / dloss[t]) if io == "f16" else 0.0
        ref.close(dx[t], lx.grad[t], io, roundings=2, what="dx %d" % t, extra=extra)
    ref.close(dw, lw.grad, io, roundings=2, what="dw")
