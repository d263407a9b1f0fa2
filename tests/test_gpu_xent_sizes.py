"""Linear cross entropy at sizes that reach every tile side and several pieces of the vocabulary, against 64 bits."""
import pytest
import torch

import fft_long_convolution_flashconv_amd as pkg
import lm_reference as ref
from parity_util import device, say
from xent_sizes import SIZES

pytestmark = pytest.mark.gpu
CASES = [(io, s) for kind, ios in (("16", ("f16", "bf16")), ("f32", ("f32",))) for io in ios for s, _ in SIZES[kind]]


def _definition(x, w, labels, dloss):
    """loss, lse, dx, dw and the largest logit in 64 bits on the GPU, some of the vocabulary at a time."""
    T, V = x.shape[0], w.shape[0]
    on = (labels >= 0) & (labels < V)
    step = max(1, (1 << 27) // T)
    parts, hit, big = [], x.new_zeros(T), 0.0
    for v in range(0, V, step):
        z = torch.mm(x, w[v:v + step].t().contiguous())
        parts.append(torch.logsumexp(z, 1))
        here = on & (labels >= v) & (labels < v + step)
        hit[here] = z[here, labels[here] - v]
        big = max(big, float(z.abs().max()))
    lse = torch.logsumexp(torch.stack(parts, 1), 1)
    dx, dw, g = torch.zeros_like(x), torch.empty_like(w), torch.where(on, dloss, torch.zeros_like(dloss))[:, None]
    for v in range(0, V, step):
        z = torch.exp(torch.mm(x, w[v:v + step].t().contiguous()) - lse[:, None])
        here = on & (labels >= v) & (labels < v + step)
        z[here, labels[here] - v] -= 1.0
        z *= g
        dx += torch.mm(z, w[v:v + step])
        dw[v:v + step] = torch.mm(z.t().contiguous(), x)
    return torch.where(on, lse - hit, torch.zeros_like(lse)), lse, dx, dw, big


@pytest.mark.parametrize("io,size", CASES, ids=lambda v: v if isinstance(v, str) else "%dx%dx%d" % v)
def test_sizes(io, size):
    T, D, V = size
    say("xent sizes", io, size)
    dev = device()
    g = torch.Generator(device=dev).manual_seed(T + D)
    x = torch.randn(T, D, generator=g, device=dev).to(ref.DT[io])
    w = (torch.randn(V, D, generator=g, device=dev) * (3.0 / D ** 0.5)).to(ref.DT[io])
    labels = torch.randint(0, V, (T,), generator=g, device=dev)
    labels[1::5], labels[2] = -100, V + 5
    labels[0], labels[-1] = 0, V - 1
    # unscaled, gradients of 16-bit floats would fall below fp16's normal numbers: as a training scales its loss
    dloss = (torch.rand(T, generator=g, device=dev) + 0.1) * (1024.0 if io == "f16" else 1.0 / T)
    loss, lse = pkg.linear_xent(x, w, labels, return_lse=True)
    dx, dw = pkg.linear_xent_bwd(x, w, labels, lse, dloss)
    rl, rs, rx, rw, big = _definition(x.double(), w.double(), labels, dloss.double())
    # absolute: the logits' own rounding, fp32 sums of products of the logits' size
    reach = float((x.double().norm(dim=1).max() * w.double().norm(dim=1).max()).item()) + 1.0
    assert (lse.double() - rs).abs().max().item() <= 4e-6 * reach
    assert (loss.double() - rl).abs().max().item() <= 8e-6 * reach
    extra = 2.0 ** -22 * big
    ref.close(dx, rx.cpu(), io, roundings=2, what="dx", extra=extra)
    ref.close(dw, rw.cpu(), io, roundings=2, what="dw", extra=extra)
    on = (labels >= 0) & (labels < V)
    assert not dx[~on].any()
