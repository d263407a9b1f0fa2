"""Linear attention whose states grow by more than fp32 holds over a segment, and shrink again: the factors over any 64
steps and every state are within fp32, and so is every result.

Rows are cut into segments of several chunks, the states of which are joined (in place where there are few segments, by a
launch of their own where there are many).  The growth is e^96 over 128 steps that lie in one segment, from states of
1e-6 and less; the upstream gradients are large where the states are small and the other way round, so that the gradients'
states pass through the same range."""
import pytest
import torch

import fft_long_convolution_flashconv_amd as pkg
import layer_reference as lref
import lm_reference as ref
from parity_util import device, say

pytestmark = pytest.mark.gpu
DT = ref.DT
RAMP, RATE = 128, 0.75

# B, N, H, dim, first step that grows, first that shrinks
CASES = [(8, 1024, 12, 8, 256, 640),    # forward 8 segments of 128 steps, backward 2 of 512
         (2, 4096, 32, 4, 768, 2432)]   # forward 11 segments of 384, backward 4 of 1024
IDS = ["in_place", "joined"]


def decays(N, H, up, down):
    g = torch.zeros(N)
    g[up:up + RAMP], g[down:down + RAMP] = RATE, -RATE
    return g[:, None].repeat(1, H)


def parts(N, up, down):
    """Steps of states of one size: before, between and behind the two ramps."""
    return (slice(0, up), slice(up + RAMP, down), slice(down + RAMP, N))


def make(io, case, seed):
    B, N, H, d, up, down = case
    gen = torch.Generator().manual_seed(seed)

    def n(*s, std=1.0, dtype=DT[io]):
        return (torch.randn(*s, generator=gen) * std).to(dtype)

    g = decays(N, H, up, down)
    size = torch.exp(torch.cumsum(g.double(), 0))[None, :, :, None]  # of the states, over what they begin with
    a = dict(q=n(B, N, H, d), k=n(B, N, H, d), v=n(B, N, H, d, std=1e-7), g=g.expand(B, N, H).contiguous(),
             x_in=n(B, H, d, d, std=1e-7, dtype=torch.float32))
    a["dy"] = (1e12 * torch.randn(B, N, H, d, generator=gen, dtype=torch.float64) / size).to(DT[io])
    a["dx_out"] = n(B, H, d, d, std=1e12, dtype=torch.float32)
    # the first sequence has no state at all until all growth is behind it
    a["v"][0, :up + RAMP] = 0
    a["x_in"][0] = 0
    return a


def gpu(a):
    return {k: v.to(device()) for k, v in a.items()}


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_growth_forward(io, case):
    say("linear_attn growth", io, case)
    a = make(io, case, 1)
    d = gpu(a)
    y, xo = pkg.linear_attn(d["q"], d["k"], d["v"], d["g"], x_in=d["x_in"], return_state=True)
    ry, rx = lref.linear_attn(*(a[k].double() for k in ("q", "k", "v", "g")), 1.0, a["x_in"].double())
    ref.close(xo, rx, what="x_out")
    for at in parts(case[1], *case[4:]):
        ref.close(y[:, at], ry[:, at], io, what="y of steps %s" % at)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_growth_forward_f16(case):
    """Half's range does not hold what is read from the large states: nothing is read from them."""
    say("linear_attn growth f16", case)
    B, N, H, dim, up, down = case
    a = make("f16", case, 2)
    gen = torch.Generator().manual_seed(3)
    a["k"], a["v"] = ((torch.randn(B, N, H, dim, generator=gen) * std).half() for std in (2.0 ** -13, 2.0 ** -20))
    a["v"][0, :up + RAMP] = 0
    a["x_in"] *= 0.03
    a["q"][:, up:down + RAMP] = 0
    d = gpu(a)
    y, xo = pkg.linear_attn(d["q"], d["k"], d["v"], d["g"], scale=2.0 ** 24, x_in=d["x_in"], return_state=True)
    ry, rx = lref.linear_attn(*(a[k].double() for k in ("q", "k", "v", "g")), 2.0 ** 24, a["x_in"].double())
    ref.close(xo, rx, what="x_out")
    ref.close(y[:, :up], ry[:, :up], "f16", what="y before")
    ref.close(y[:, down + RAMP:], ry[:, down + RAMP:], "f16", what="y behind")
    assert not y[:, up:down + RAMP].any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_growth_backward(io, case):
    say("linear_attn growth backward", io, case)
    a = make(io, case, 5)
    d = gpu(a)
    o = pkg.linear_attn_bwd(d["q"], d["k"], d["v"], d["g"], d["dy"], x_in=d["x_in"], dx_out=d["dx_out"])
    leaf = {k: ref.leaf(a[k]) for k in ("q", "k", "v", "g", "x_in")}
    y, xo = lref.linear_attn(leaf["q"], leaf["k"], leaf["v"], leaf["g"], 1.0, leaf["x_in"])
    ((y * a["dy"].double()).sum() + (xo * a["dx_out"].double()).sum()).backward()
    ref.close(o.dx_in, leaf["x_in"].grad, what="dx_in")
    for name, got in (("q", o.dq), ("k", o.dk), ("v", o.dv)):
        for at in parts(case[1], *case[4:]):
            ref.close(got[:, at], leaf[name].grad[:, at], io, what="d%s of steps %s" % (name, at))
    terms = ((a["q"].double() * leaf["q"].grad).sum(-1).square().sum() + (a["k"].double() * leaf["k"].grad).sum(-1).square().sum()).sqrt()
    lref.close_dg(o.dg, leaf["g"].grad, terms.item(), case[1])
