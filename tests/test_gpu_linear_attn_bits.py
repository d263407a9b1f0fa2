"""How many bits linear attention keeps of what multiplies its inputs again: the state, and the weights of steps close by.

Outputs that are rounded to 16 bits hide that, unless larger terms cancel in them: here each output is the difference of
a full-length number (a state, or a decayed product) and its first 13 or so bits, which later steps take away again."""
import pytest
import torch

import fft_long_convolution_flashconv_amd as pkg
from parity_util import device, say

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def cut(x, dtype):
    """x in two parts of the type, the second of 4 bits, that come to it within 2^-12 of it."""
    first = x.to(dtype)
    e = torch.floor(torch.log2((x - first.double()).abs().clamp(min=2.0 ** -60))) - 3
    return first, ((x - first.double()) / 2 ** e).round().mul(2 ** e).to(dtype)


def check(y, x, parts, io):
    """y is x without its parts.  Weights and states keep 22 bits, an error of 2^-22 of x at most; the sum of three
    products, and the factor of the state or of the products, are rounded in fp32, at most eight times half a step."""
    want = x - sum(p.double() for p in parts)
    err, bound = (y.double().cpu() - want).abs(), HALF_ULP[io] * want.abs() + (2.0 ** -22 + 8 * 2.0 ** -24) * x.abs()
    assert bool((err <= bound + 2.0 ** -25).all()), "error over bound: %.2f" % (err / bound).max().item()


@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("H,dv", [(4, 64), (2, 128)])
def test_state(io, H, dv):
    """The state that enters, less steps that take its first bits away."""
    say("linear_attn bits of a state", io, H, dv)
    gen = torch.Generator().manual_seed(2)
    S = torch.rand(1, H, 1, dv, generator=gen) + 1.0
    parts = cut(S[:, :, 0].double(), DT[io])
    v = torch.stack([-p for p in parts], 1)  # [1,2,H,dv]
    one = torch.ones(1, 2, H, 1, dtype=DT[io])
    y = pkg.linear_attn(one.to(device()), one.to(device()), v.to(device()), torch.zeros(H, device=device()),
                        x_in=S.to(device()))
    check(y[:, 1], S[:, :, 0].double(), parts, io)


@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("H,dv", [(4, 64), (2, 128)])
def test_weights(io, H, dv):
    """A decayed product, less steps that take its first bits away."""
    say("linear_attn bits of weights", io, H, dv)
    g = torch.zeros(1, 3, H)
    g[0, 1] = torch.linspace(-0.9, -0.1, H)
    w = torch.exp(g[:, 1].double())
    first, second = cut(w, DT[io])
    k = torch.stack([torch.ones_like(first), -first, -second], 1)[..., None]
    one = torch.ones(1, 3, H, 1, dtype=DT[io])
    v = torch.ones(1, 3, H, dv, dtype=DT[io])
    y = pkg.linear_attn(one.to(device()), k.to(device()), v.to(device()), g.to(device()))
    wide = [t[..., None].expand(1, H, dv) for t in (w, first, second)]
    # (e^g in fp32 is within 2^-23 of it: an exponent of two of at most 2, rounded once, and the function's last place)
    check(y[:, 2], wide[0], wide[1:], io)
