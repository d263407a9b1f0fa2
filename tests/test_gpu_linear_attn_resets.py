"""Gradients of the decays where steps start the state anew (documents packed into one row): each document's are as
accurate as its own terms, whatever stands behind it in the row."""
import pytest
import torch

import fft_long_convolution_flashconv_amd as pkg
import layer_reference as lref
import lm_reference as ref
from parity_util import device, say

pytestmark = pytest.mark.gpu
DT = ref.DT
H, D = 2, 16

# N, steps that start anew, lengths, a state on both sides
CASES = [(512, [256], None, False), (512, [256], None, True), (300, [0, 299], None, True), (200, [70, 71, 73, 150], [200, 71], True),
         (2500, [5, 1023, 1024, 1025, 2048, 2300], [2500, 2049], True), (1100, [1], [1100, 0], False)]


def make(io, case, seed, strength):
    N, resets, lengths, state = case
    gen = torch.Generator().manual_seed(seed)

    def n(*s, dtype=DT[io]):
        return torch.randn(*s, generator=gen).to(dtype)

    a = dict(q=n(2, N, H, D), k=n(2, N, H, D), v=n(2, N, H, D), g=-strength * n(2, N, H, dtype=torch.float32).abs(),
             dy=n(2, N, H, D, dtype=torch.float32))
    edges = [0, *resets, N]
    for i, (lo, hi) in enumerate(zip(edges, edges[1:])):  # documents of very different size
        a["dy"][:, lo:hi] *= [1.0, 1e4, 1e-2, 1e2][i % 4]
    a["dy"] = a["dy"].to(DT[io])
    for t in resets:
        a["g"][:, t] = float("-inf") if t % 2 else -1e5
    if state:
        a["x_in"], a["dx_out"] = n(2, H, D, D, dtype=torch.float32), n(2, H, D, D, dtype=torch.float32)
    return a


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("strength", [0.02, 0.3])
@pytest.mark.parametrize("case", CASES, ids=["N%d_%d%s" % (c[0], len(c[1]), "_state" if c[3] else "") for c in CASES])
def test_resets(io, strength, case):
    say("linear_attn resets", io, strength, case)
    N, resets, lengths, state = case
    a = make(io, case, 3, strength)
    dev = {k: t.to(device()) for k, t in a.items()}
    o = pkg.linear_attn_bwd(dev["q"], dev["k"], dev["v"], dev["g"], dev["dy"], scale=0.25, x_in=dev.get("x_in"),
                            dx_out=dev.get("dx_out"),
                            lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=device()))
    leaf = {k: ref.leaf(t) for k, t in a.items() if k not in ("dy", "dx_out")}
    with torch.no_grad():
        leaf["g"].clamp_(min=-1e4)  # (its factor is zero in 64 bits too)
    y, xo = lref.linear_attn(leaf["q"], leaf["k"], leaf["v"], leaf["g"], 0.25, leaf.get("x_in"), lengths)
    s = (y * a["dy"].double()).sum()
    if state:
        s = s + (xo * a["dx_out"].double()).sum()
    s.backward()
    for t in resets:
        assert not o.dg[:, t].any()
    edges = sorted({0, *resets, N})
    for lo, hi in zip(edges, edges[1:]):
        at = slice(lo, hi)
        terms = sum((leaf[n].double() * leaf[n].grad)[:, at].sum(-1).square().sum() for n in ("q", "k")).sqrt().item()
        lref.close_dg(o.dg[:, at], leaf["g"].grad[:, at], terms, hi - lo, what="dg of steps %d to %d" % (lo, hi))


def test_resets_of_heads():
    """A decay per head that always starts anew has no gradient."""
    a = {k: t.to(device()) for k, t in make("f32", CASES[0], 4, 0.1).items()}
    g = torch.tensor([-0.05, float("-inf")], device=device())
    o = pkg.linear_attn_bwd(a["q"], a["k"], a["v"], g, a["dy"])
    assert float(o.dg[1]) == 0.0 and float(o.dg[0]) != 0.0
    one = pkg.linear_attn_bwd(*(a[n][:, :, :1].contiguous() for n in ("q", "k", "v")), g[:1].contiguous(),
                              a["dy"][:, :, :1].contiguous())
    assert torch.equal(one.dg, o.dg[:1])


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("N", [300, 1500])
def test_decays_of_heads(io, N, state):
    """A decay per head: what its steps' gradients are off by adds up.  A step's products lose about 2^-22 of their size
    (sums of 16, each of factors of 22 bits or more), 2^-21 with what the states lose; step t's is counted t + 1 times,
    less its share of the correction, (N + 1) / 2 times: sqrt(N^3 / 12) of a step's, N / sqrt(12) of their norm, and
    sqrt(12) times that at most."""
    say("linear_attn decays of heads", io, N, state)
    a = make(io, (N, [], None, state), 5, 0.1)
    a["g"] = torch.tensor([-0.01, -0.2])
    dev = {k: t.to(device()) for k, t in a.items()}
    o = pkg.linear_attn_bwd(dev["q"], dev["k"], dev["v"], dev["g"], dev["dy"], x_in=dev.get("x_in"), dx_out=dev.get("dx_out"))
    leaf = {k: ref.leaf(t) for k, t in a.items() if k not in ("dy", "dx_out")}
    y, xo = lref.linear_attn(leaf["q"], leaf["k"], leaf["v"], leaf["g"], 1.0, leaf.get("x_in"))
    s = (y * a["dy"].double()).sum()
    if state:
        s = s + (xo * a["dx_out"].double()).sum()
    s.backward()
    terms = sum((leaf[n].double() * leaf[n].grad).sum(-1).square().sum((0, 1)) for n in ("q", "k")).sqrt()
    err = (o.dg.double().cpu() - leaf["g"].grad).abs()
    bound = N * 2.0 ** -21 * terms + 2.0 ** -23 * leaf["g"].grad.abs()
    assert bool((err <= bound).all()), "errors %s, bounds %s" % (err.tolist(), bound.tolist())
