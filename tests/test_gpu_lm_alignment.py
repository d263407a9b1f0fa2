"""The convolution and the scan on tensors that start at any element (slices of larger buffers, rows of odd lengths):
the same bits as on aligned ones."""
import pytest
import torch

import fft_long_convolution_flashconv_amd as pkg
import lm_reference as ref
from parity_util import device, say

pytestmark = pytest.mark.gpu


def _at(t, off):
    """A contiguous copy of t that starts ``off`` elements after an aligned address."""
    if t is None:
        return None
    buf = torch.empty(t.numel() + off + 8, device=t.device, dtype=t.dtype)
    v = buf[off:off + t.numel()].view(t.shape)
    v.copy_(t)
    assert v.is_contiguous() and v.data_ptr() % 16 == (off * t.element_size()) % 16
    return v


def _normal(io, seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s, dtype=ref.DT[io]: torch.randn(*s, generator=g).to(dtype).to(device())


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("off", [1, 3, 7])
def test_short_conv(io, off):
    say("alignment short_conv", io, off)
    r = _normal(io, off)
    B, H, N, W = 2, 5, 531, 4
    t = dict(x=r(B, H, N), dy=r(B, H, N), x_in=r(B, H, W - 1), dx_out=r(B, H, W - 1), w=r(H, W, dtype=torch.float32),
             bias=r(H, dtype=torch.float32), lengths=torch.tensor([N, 300], dtype=torch.int32, device=device()))

    def run(t, out):
        y, last = pkg.short_conv(t["x"], t["w"], bias=t["bias"], x_in=t["x_in"], lengths=t["lengths"], return_state=True,
                                 out=out)
        g = pkg.short_conv_bwd(t["x"], t["w"], t["dy"], bias=t["bias"], x_in=t["x_in"], lengths=t["lengths"],
                               dx_out=t["dx_out"])
        tok, pool = t["x"][:, :, 0].contiguous(), t["x_in"].clone()
        s = pkg.short_conv_step(_at(tok, off) if out is not None else tok, t["w"], pool, bias=t["bias"])
        return (y, last, s, pool) + tuple(g)

    a = run(t, None)
    b = run({k: _at(v, off) for k, v in t.items()}, _at(torch.zeros_like(t["x"]), off))
    assert all(torch.equal(p, q) for p, q in zip(a, b))


# 16 modes: the aligned form reads rates in vectors, the other one by one; sums of the same products in the same order
@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,S", [(7, 16), (130, 16), (531, 16), (531, 5), (9001, 16)])
def test_selective(io, N, S):
    say("alignment selective", io, N, S)
    r = _normal(io, N + S)
    B, H, G, f32 = 2, 6, 2, torch.float32
    t = dict(u=r(B, H, N), dt=r(B, H, N), A=-r(H, S, dtype=f32).abs(), Bm=r(B, G, S, N), C=r(B, G, S, N), dy=r(B, H, N),
             D=r(H, dtype=f32), z=r(B, H, N), dt_bias=r(H, dtype=f32) - 2.0, x_in=r(B, H, S, dtype=f32),
             dx_out=r(B, H, S, dtype=f32), lengths=torch.tensor([N, max(N - 3, 0)], dtype=torch.int32, device=device()))

    def run(t):
        a = [t[k] for k in ("u", "dt", "A", "Bm", "C")]
        k = dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"])
        y, x, saved = pkg.selective_scan(*a, x_in=t["x_in"], lengths=t["lengths"], return_state=True, return_saved=True, **k)
        o = pkg.selective_scan_bwd(*a, t["dy"], saved, lengths=t["lengths"], dx_out=t["dx_out"], **k)
        return (y, x, saved), o

    base, g0 = run(t)
    for off in (1, 3):
        odd, g1 = run({k: _at(v, off) for k, v in t.items()})
        assert all(torch.equal(p, q) for p, q in zip(base, odd)), off
        for name, p, q in zip(g0._fields, g0, g1):
            # du, ddt, dz of 16 modes: within the rounding of fp32 sums (see above), then of the type
            ref.close(q, p.double().cpu(), io if q.dtype != f32 else "f32", what="%s %d" % (name, off))
    tok = {k: (v[..., 0].contiguous() if k in ("u", "dt", "Bm", "C", "z") else v) for k, v in t.items()}

    def step(t):
        pool = _at(t["x_in"], 1 if t is not tok else 0)
        y = pkg.selective_step(t["u"], t["dt"], t["A"], t["Bm"], t["C"], pool, D=t["D"], z=t["z"], dt_bias=t["dt_bias"])
        return y, pool

    p, q = step(tok), step({k: _at(v, 1) for k, v in tok.items()})
    assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])
