"""Linear cross entropy (h3conv_linear_xent, _bwd) against its 64-bit definition."""
import pytest
import torch

import fft_long_convolution_flashconv_amd as pkg
import lm_reference as ref
from parity_util import device, say

pytestmark = pytest.mark.gpu
DT = ref.DT

# (T, D, V)
CASES = [(1, 1, 1), (1, 64, 2), (3, 8, 127), (5, 33, 128), (127, 64, 129), (128, 96, 300), (130, 65, 1000),
         (257, 200, 513), (64, 768, 2049)]


def _make(io, T, D, V, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, D, generator=g).to(DT[io])
    w = (torch.randn(V, D, generator=g) * (3.0 / D ** 0.5)).to(DT[io])
    labels = torch.randint(0, V, (T,), generator=g)
    if T > 2:
        labels[1] = -100
        labels[2] = V + 5          # outside the vocabulary: no loss
    labels[-1] = V - 1
    dloss = torch.rand(T, generator=g) + 0.1
    return x, w, labels, dloss


def _check(io, x, w, labels, dloss, tag=""):
    dev = device()
    gx, gw, gl = x.to(dev), w.to(dev), labels.to(dev)
    loss, lse = pkg.linear_xent(gx, gw, gl, return_lse=True)
    dx, dw = pkg.linear_xent_bwd(gx, gw, gl, lse, dloss.to(dev))
    torch.cuda.synchronize()
    rx, rw = ref.leaf(x), ref.leaf(w)
    rl, rs = ref.linear_xent(rx, rw, labels)
    (rl * torch.nan_to_num(dloss.double(), 0.0, 0.0, 0.0)).sum().backward()
    # absolute: the logits' own rounding, fp32 sums of products of the logits' size
    size = float((x.double().norm(dim=1).max() * w.double().norm(dim=1).max()).item()) + 1.0
    assert (lse.double().cpu() - rs).abs().max().item() <= 4e-6 * size, tag
    assert (loss.double().cpu() - rl).abs().max().item() <= 8e-6 * size, tag
    wide = 2.0 ** -22 * float((rx.detach() @ rw.detach().t()).abs().max())
    ref.close(dx, rx.grad, io, roundings=2, what="dx" + tag, extra=wide)
    ref.close(dw, rw.grad, io, roundings=2, what="dw" + tag, extra=wide)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,D,V", CASES)
def test_linear_xent(io, T, D, V):
    say("linear_xent", io, T, D, V)
    _check(io, *_make(io, T, D, V, 7))


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
def test_ignored_tokens_carry_nothing(io):
    """All tokens ignored; and NaN in the upstream gradient of ignored tokens."""
    dev = device()
    x, w, labels, dloss = _make(io, 40, 64, 200, 3)
    loss, lse = pkg.linear_xent(x.to(dev), w.to(dev), torch.full((40,), -100).to(dev), return_lse=True)
    dx, dw = pkg.linear_xent_bwd(x.to(dev), w.to(dev), torch.full((40,), -100).to(dev), lse, dloss.to(dev))
    assert bool((loss == 0).all()) and bool((dx == 0).all()) and bool((dw == 0).all())
    dloss[1] = float("nan")
    dloss[2] = float("inf")
    _check(io, x, w, labels, dloss)
    loss = pkg.linear_xent(x.to(dev), w.to(dev), labels.to(dev), ignore_index=int(labels[5]))
    assert float(loss[5]) == 0.0


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
def test_wide_logits_and_tiny_gradients(io):
    """Logits of some hundred in magnitude; a mean over many tokens under a loss scale of one."""
    x, w, labels, dloss = _make(io, 96, 64, 700, 5)
    _check(io, x, (w.float() * 20).to(DT[io]), labels, dloss, " wide")
    # unscaled, fp16 gradients would fall below its normal numbers: scale the loss as training does
    _check(io, x, w, labels, dloss * (1e-6 if io != "f16" else 1024.0), " scaled")


def test_pieces_of_the_vocabulary():
    """A vocabulary in several pieces (their size goes by the workspace bound) against one."""
    dev = device()
    T, D, V = 16400, 64, 20000  # two pieces in 32 bits, one in 16
    g = torch.Generator(device=dev).manual_seed(1)
    x, w = torch.randn(T, D, generator=g, device=dev), torch.randn(V, D, generator=g, device=dev) * 0.3
    labels = torch.randint(0, V, (T,), generator=g, device=dev)
    loss, lse = pkg.linear_xent(x, w, labels, return_lse=True)
    dloss = torch.rand(T, generator=g, device=dev) / T
    dx, dw = pkg.linear_xent_bwd(x, w, labels, lse, dloss)
    p = torch.exp((x.double() @ w.double().t()) - lse.double()[:, None])
    p[torch.arange(T, device=dev), labels] -= 1.0
    p *= dloss.double()[:, None]
    ref.close(dx, (p @ w.double()).cpu(), what="dx")
    ref.close(dw, torch.mm(p.t().contiguous(), x.double()).cpu(), what="dw")


def test_xent_differences():
    dev = device()
    x, w, labels, dloss = _make("f32", 20, 17, 50, 9)
    loss, lse = pkg.linear_xent(x.to(dev), w.to(dev), labels.to(dev), return_lse=True)
    dx, dw = pkg.linear_xent_bwd(x.to(dev), w.to(dev), labels.to(dev), lse, dloss.to(dev))
    f = lambda a: (ref.linear_xent(a["x"], a["w"], labels)[0] * dloss.double()).sum()
    dot, diff, size = ref.directional(f, dict(x=x.double(), w=w.double()), dict(x=dx, w=dw), 5)
    assert abs(dot - diff) <= 1e-5 * size + 1e-7


def test_xent_empty():
    dev = device()
    x, w, l = torch.empty(0, 8, device=dev), torch.randn(5, 8).to(dev), torch.empty(0, dtype=torch.int64, device=dev)
    loss, lse = pkg.linear_xent(x, w, l, return_lse=True)
    dx, dw = pkg.linear_xent_bwd(x, w, l, lse, lse)
    assert loss.shape == (0,) and dx.shape == (0, 8) and bool((dw == 0).all())


def test_xent_same_bits_and_other_stream():
    dev = device()
    x, w, labels, dloss = (t.to(dev) for t in _make("bf16", 300, 128, 3001, 2))

    def once():
        loss, lse = pkg.linear_xent(x, w, labels, return_lse=True)
        return (loss, lse) + pkg.linear_xent_bwd(x, w, labels, lse, dloss)

    one = once()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        two = once()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_xent_refusals():
    dev = device()
    x, w, labels, dloss = (t.to(dev) for t in _make("f32", 4, 8, 10, 1))
    with pytest.raises(ValueError):
        pkg.linear_xent(x, w.half(), labels)
    with pytest.raises(ValueError):
        pkg.linear_xent(x, w[:, :4].contiguous(), labels)
    with pytest.raises(ValueError):
        pkg.linear_xent(x, w, labels.int())
    with pytest.raises(ValueError):
        pkg.linear_xent(x, w.t(), labels)
    with pytest.raises(ValueError):
        pkg.linear_xent_bwd(x, w, labels, dloss, dloss[:3].contiguous())
    with pytest.raises(TypeError):
        pkg.linear_xent_bwd(x, w, labels, None, dloss)


@pytest.mark.parametrize("T,D,V", [(512, 64, 9000), (300, 40, 4545), (130, 128, 12300)])
def test_gradient_ranges(T, D, V):
    """dx of few tokens and few columns over many rows: summed over ranges of the vocabulary."""
    _check("bf16", *_make("bf16", T, D, V, 21))


# fp32: tiles of both sizes, with rows, columns and sums that end inside a vector
@pytest.mark.parametrize("T,D,V", [(1, 1, 1), (2, 3, 3), (5, 2, 700), (33, 67, 3), (67, 35, 36), (64, 4, 65),
                                   (1025, 130, 1030), (40, 1100, 1050)])
def test_fp32_tiles(T, D, V):
    say("linear_xent fp32", T, D, V)
    _check("f32", *_make("f32", T, D, V, T + D + V))


# 16-bit: tiles of every side, sums over the vocabulary and over the tokens in ranges of their own
@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("T,D,V", [(1, 1, 1), (40, 64, 20000), (2500, 70, 130), (1100, 130, 513), (700, 320, 5000),
                                   (2100, 96, 4200), (300, 65, 33000)])
def test_16bit_tiles(io, T, D, V):
    say("linear_xent 16-bit", io, T, D, V)
    _check(io, *_make(io, T, D, V, T + D + V))


@pytest.mark.parametrize("T,D,V", [(40, 70, 20000), (33, 3, 9001), (130, 257, 12345)])
def test_fp32_ranges(T, D, V):
    """fp32: sums of dx over the vocabulary in ranges of their own."""
    say("linear_xent fp32 ranges", T, D, V)
    _check("f32", *_make("f32", T, D, V, T + D + V))
