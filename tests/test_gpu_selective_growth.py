"""Selective scan with states that grow (A > 0, or negative steps): zero and small states stay what they are where the
factor of many steps passes the largest float."""
import pytest
import torch

import fft_long_convolution_flashconv_amd as pkg
import lm_reference as ref
from parity_util import device, say

pytestmark = pytest.mark.gpu
DT = ref.DT

# The exponent of a factor carries a few roundings (rate times log2 e, the sum over steps, their product), each up to
# 2^-24 of it: of the exponents up to 100 that finite states here meet, 4 x 100 x 2^-24.
EXTRA = 4 * 100 * 2.0 ** -24

# (B, H, N, S, where the fast steps are): 16 lanes per row, 64, modes over four waves, one row over four waves
SHAPES = [(1, 3, 200, 2, (20, 180)), (1, 600, 150, 1, (10, 140)), (1, 3, 700, 2, (40, 600)), (2, 4, 700, 5, (40, 600)),
          (1, 2, 8300, 3, (300, 8100)), (1, 2, 9000, 16, (300, 8800))]


def _check(got, want, io, what):
    ref.close(got, want, io, what=what, extra=EXTRA)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: "B%d_H%d_N%d_S%d" % c[:4])
def test_zero_states_stay_zero(io, softplus, shape):
    """Mode 0 grows by e^100 and more over the fast steps, where its state and its gradient are zero: B of it is zero
    before them, C after.  The other modes decay.  Without softplus some rows take the opposite signs of step and A."""
    B, H, N, S, (lo, hi) = shape
    say("growth", io, softplus, shape)
    g = torch.Generator().manual_seed(B + H + N + S)
    t = DT[io]

    def r(*s):
        return torch.randn(*s, generator=g)

    d = torch.full((B, H, N), 0.004)
    d[..., lo:hi] = 200.0 / (hi - lo)
    A = -torch.arange(0, S).float().repeat(H, 1) - 0.5
    A[:, 0] = 1.0
    if not softplus:
        d[:, ::2] *= -1.0
        A[::2] *= -1.0
        dt = d.to(t)
    else:
        dt = torch.log(torch.expm1(d.double())).to(t)
    Bm, C = r(B, 1, S, N), r(B, 1, S, N)
    Bm[:, :, 0, :hi] = 0.0
    C[:, :, 0, lo:] = 0.0
    u, z, dy, D, dx_out = r(B, H, N).to(t), r(B, H, N).to(t), r(B, H, N).to(t), r(H), r(B, H, S)
    Bm, C = Bm.to(t), C.to(t)
    x_in = r(B, H, S)
    x_in[..., 0] = 0.0
    dx_out[..., 0] = 0.0
    dev = device()
    a = [v.to(dev) for v in (u, dt, A, Bm, C)]
    k = dict(D=D.to(dev), z=z.to(dev), softplus=softplus)
    y, xo, saved = pkg.selective_scan(*a, x_in=x_in.to(dev), return_state=True, return_saved=True, **k)
    o = pkg.selective_scan_bwd(*a, dy.to(dev), saved, dx_out=dx_out.to(dev), **k)
    torch.cuda.synchronize()
    leaves = [ref.leaf(v) for v in (u, dt, A, Bm, C, D, z, x_in)]
    lu, ld, lA, lB, lC, lD, lz, lx = leaves
    ry, ro = ref.selective_scan(lu, ld, lA, lB, lC, lD, lz, None, softplus, lx, None)
    ((ry * dy.double()).sum() + (ro * dx_out.double()).sum()).backward()
    _check(y, ry, io, "y")
    _check(xo, ro, "f32", "x_out")
    for name, got, leaf, kind in zip(("du", "ddt", "dB", "dC", "dz", "dx_in"), (o.du, o.ddt, o.dB, o.dC, o.dz, o.dx_in),
                                     (lu, ld, lB, lC, lz, lx), (io, io, io, io, io, "f32")):
        _check(got, leaf.grad, kind, name)
    for name, got in (("dA", o.dA), ("dD", o.dD)):
        assert bool(torch.isfinite(got).all()), name


@pytest.mark.parametrize("N,down,up", [(250, (0, 80), (80, 250)), (1000, (0, 300), (300, 1000)),
                                       (8200, (10, 2500), (2500, 8190))])
def test_small_states_grow(N, down, up):
    """A state of one falls by e^-40 and then grows by e^95: the second factor alone passes the largest float."""
    say("small states", N)
    dev = device()
    dt = torch.zeros(1, 2, N)
    dt[..., down[0]:down[1]] = -40.0 / (down[1] - down[0])
    dt[..., up[0]:up[1]] = 95.0 / (up[1] - up[0])
    u, A = torch.zeros(1, 2, N), torch.ones(2, 1)
    Bm, C, x_in = torch.ones(1, 1, 1, N), torch.ones(1, 1, 1, N), torch.tensor([[[1.0], [-2.0]]])
    y, xo = pkg.selective_scan(*(v.to(dev) for v in (u, dt, A, Bm, C)), softplus=False, x_in=x_in.to(dev),
                               return_state=True)
    ry, ro = ref.selective_scan(*(v.double() for v in (u, dt, A, Bm, C)), None, None, None, False, x_in.double(), None)
    _check(y, ry, "f32", "y")
    _check(xo, ro, "f32", "x_out")
    # every step by itself: small ones are not hidden by the largest
    rel = ((y.double().cpu() - ry).abs() / ry.abs()).max().item()
    assert rel <= 1e-5 + EXTRA, rel
