"""Every path that the new layers' kernels choose by size, type or alignment, against the definitions or the path beside it."""
import pytest
import torch

import fft_long_convolution_flashconv_amd as pkg
import layer_reference as lref
import lm_reference as ref
from parity_util import device, say

pytestmark = pytest.mark.gpu
IOS = ["f32", "f16", "bf16"]

# (B, N, H, dk, dv): rows in few segments and in many, of one and of several chunks each; every width of the state's
# tiles, whole units and odd
LONG = [(1, 2000, 1, 32, 32), (1, 4100, 2, 64, 64), (2, 1500, 3, 64, 128), (1, 3000, 2, 128, 128), (1, 1100, 1, 256, 256),
        (1, 1100, 1, 136, 64), (1, 2300, 2, 37, 70), (1, 700, 1, 129, 131)]


def _inputs(io, B, N, H, dk, dv, seed=1):
    gen = torch.Generator().manual_seed(seed)

    def n(*s, dtype=ref.DT[io], std=1.0):
        return (torch.randn(*s, generator=gen) * std).to(dtype)

    return dict(q=n(B, N, H, dk), k=n(B, N, H, dk), v=n(B, N, H, dv), g=-0.05 * n(B, N, H, dtype=torch.float32).abs(),
                x_in=n(B, H, dk, dv, dtype=torch.float32), dy=n(B, N, H, dv), dx_out=n(B, H, dk, dv, dtype=torch.float32))


def _quadratic(d, scale):
    """y, x_out and the gradients in 64 bits on the GPU: all pairs of steps at once, by automatic differentiation."""
    p = {k: v.to(device()).double() for k, v in d.items()}
    leaf = {k: p[k].requires_grad_(True) for k in ("q", "k", "v", "g", "x_in")}
    G = torch.cumsum(leaf["g"], 1).transpose(1, 2)                       # [B,H,N]
    q, k, v = (leaf[n].transpose(1, 2).contiguous() for n in ("q", "k", "v"))
    N = q.shape[2]
    low = torch.ones(N, N, dtype=torch.bool, device=q.device).tril()
    w = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], torch.full((), float("-inf"), dtype=torch.float64, device=q.device)))
    y = scale * (torch.matmul(torch.matmul(q, k.transpose(2, 3).contiguous()) * w, v) + torch.matmul(q * torch.exp(G)[..., None], leaf["x_in"]))
    end = torch.exp(G[..., -1:, None]) * leaf["x_in"] + torch.matmul((k * torch.exp(G[..., -1:] - G)[..., None]).transpose(2, 3).contiguous(), v)
    y = y.transpose(1, 2)
    ((y * p["dy"]).sum() + (end * p["dx_out"]).sum()).backward()
    return y.detach().cpu(), end.detach().cpu(), {n: t.grad.cpu() for n, t in leaf.items()}


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("B,N,H,dk,dv", LONG)
def test_long_rows(io, B, N, H, dk, dv):
    say("long rows", io, B, N, H, dk, dv)
    d = _inputs(io, B, N, H, dk, dv)
    ry, rx, rg = _quadratic(d, 0.2)
    g = {k: v.to(device()) for k, v in d.items()}
    y, x = pkg.linear_attn(g["q"], g["k"], g["v"], g["g"], 0.2, x_in=g["x_in"], return_state=True)
    ref.close(y, ry, io, what="y")
    ref.close(x, rx, what="x_out")
    o = pkg.linear_attn_bwd(g["q"], g["k"], g["v"], g["g"], g["dy"], 0.2, x_in=g["x_in"], dx_out=g["dx_out"])
    for name, got in (("q", o.dq), ("k", o.dk), ("v", o.dv)):
        ref.close(got, rg[name], io, what="d" + name)
    ref.close(o.dx_in, rg["x_in"], what="dx_in")
    terms = ((d["q"].double() * rg["q"]).sum(-1).square().sum() + (d["k"].double() * rg["k"]).sum(-1).square().sum()).sqrt().item()
    lref.close_dg(o.dg, rg["g"], terms, N)


@pytest.mark.parametrize("io", IOS)
def test_lengths_across_segments(io):
    """Rows that end in every segment, at its borders and before the first: each is what it is alone."""
    say("lengths across segments", io)
    N, H, d = 1300, 2, 64
    lengths = [1300, 0, 1, 63, 64, 65, 640, 641, 1299]
    a = _inputs(io, len(lengths), N, H, d, d, 2)
    g = {k: v.to(device()) for k, v in a.items()}
    for b, n in enumerate(lengths):
        for k in ("q", "k", "v", "g", "dy"):
            g[k][b, n:] = float("nan")
    ln = torch.tensor(lengths, dtype=torch.int32, device=device())
    y, x = pkg.linear_attn(g["q"], g["k"], g["v"], g["g"], x_in=g["x_in"], lengths=ln, return_state=True)
    o = pkg.linear_attn_bwd(g["q"], g["k"], g["v"], g["g"], g["dy"], x_in=g["x_in"], lengths=ln, dx_out=g["dx_out"])
    for b, n in enumerate(lengths):
        one = {k: (v[b:b + 1, :n] if k not in ("x_in", "dx_out") else v[b:b + 1]).contiguous() for k, v in g.items()}
        y1, x1 = pkg.linear_attn(one["q"], one["k"], one["v"], one["g"], x_in=one["x_in"], return_state=True)
        o1 = pkg.linear_attn_bwd(one["q"], one["k"], one["v"], one["g"], one["dy"], x_in=one["x_in"], dx_out=one["dx_out"])
        ref.close(y[b:b + 1, :n], y1.double().cpu(), io, roundings=2, what="y")
        ref.close(x[b:b + 1], x1.double().cpu(), what="x")
        assert not y[b, n:].any() and not o.dq[b, n:].any() and not o.dk[b, n:].any() and not o.dv[b, n:].any() and not o.dg[b, n:].any()
        for name in ("dq", "dk", "dv"):
            ref.close(getattr(o, name)[b:b + 1, :n], getattr(o1, name).double().cpu(), io, roundings=2, what=name)
        ref.close(o.dx_in[b:b + 1], o1.dx_in.double().cpu(), what="dx_in")


@pytest.mark.parametrize("io", IOS)
def test_slices_at_dwords(io):
    """Slices that begin at a dword but at no unit of 16 bytes, tokens a multiple of dwords apart: the windows' path."""
    say("slices at dwords", io)
    B, N, H, d = 2, 130, 2, 32
    off, ld = 2, 3 * H * d + 6
    wide = torch.randn(B, N, ld, generator=torch.Generator().manual_seed(3)).to(ref.DT[io]).to(device())
    q, k, v = (wide[..., off + i * H * d:off + (i + 1) * H * d].unflatten(-1, (H, d)) for i in range(3))
    g, dy = torch.full((H,), -0.03, device=device()), torch.randn(B, N, H, d).to(ref.DT[io]).to(device())
    for a, b in ((pkg.linear_attn(q, k, v, g, return_state=True), pkg.linear_attn(q.contiguous(), k.contiguous(), v.contiguous(), g, return_state=True)),
                 (pkg.linear_attn_bwd(q, k, v, g, dy), pkg.linear_attn_bwd(q.contiguous(), k.contiguous(), v.contiguous(), g, dy))):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("D,groups", [(48, 1), (512, 8), (768, 12), (1600, 1), (2560, 20), (3600, 1), (4096, 2), (6000, 1), (16256, 127), (16380, 4)])
@pytest.mark.parametrize("off", [0, 1, 2])
def test_norm_at_any_element(io, D, groups, off):
    """Rows at a unit, at a dword and at any element, forward and backward."""
    say("norm at any element", io, D, groups, off)
    _norm_against_definition(io, 3, D, groups, off)


# heads of whole vectors that are not a power of two of them, of one to 64 and more; rows of whole dwords that are not
# whole vectors; rows that are not whole dwords in 16 bits
@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("T,D,groups", [(5, 48, 2), (7, 768, 8), (3, 1536, 64), (2, 2560, 32), (3, 3600, 10), (2, 1040, 2),
                                        (1, 1008, 2), (4, 1050, 1), (3, 1050, 5), (2, 2, 1), (9, 6, 3), (3, 14, 1), (2, 4002, 1),
                                        (2, 9002, 1), (1, 16382, 1), (3, 1031, 1), (2, 15, 5), (2, 8040, 15)])
def test_norm_heads_and_row_ends(io, T, D, groups):
    say("norm heads and row ends", io, T, D, groups)
    _norm_against_definition(io, T, D, groups, 0)


def _norm_against_definition(io, T, D, groups, off):
    dev = device()
    gen = torch.Generator().manual_seed(D + off)
    flat = [torch.randn(T * D + 2, generator=gen).to(ref.DT[io]).to(dev) for _ in range(5)]
    f, res, z, dr, dy = (t[off:off + T * D].view(T, D) for t in flat)
    w = [torch.randn(D, generator=gen).to(dev) for _ in range(3)]
    k = dict(res=res, gate=z, w_out=w[0], scale=w[1], w_in=w[2], groups=groups)
    r, y = pkg.block_norm(f, **k)
    o = pkg.block_norm_bwd(f, dr, dy, **k)
    leaf = {n: ref.leaf(t) for n, t in dict(f=f, **{a: b for a, b in k.items() if a != "groups"}).items()}
    rr, ry = lref.block_norm(**leaf, groups=groups)
    ((rr * dr.double().cpu()).sum() + (ry * dy.double().cpu()).sum()).backward()
    ref.close(r, rr, io, what="r")
    ref.close(y, ry, io, what="y")
    for name, got in zip(("f", "res", "gate", "w_out", "scale", "w_in"), o):
        ref.close(got, leaf[name].grad, "f32" if name in ("w_out", "scale", "w_in") else io, what="d" + name)


def test_two_calls_at_once():
    """Calls on two streams, each with buffers of its own, give what they give one after another."""
    say("two calls at once")
    sets = [{k: v.to(device()) for k, v in _inputs("bf16", 2, 900, 4, 64, 64, s).items()} for s in (1, 2)]

    def work(d):
        a = (d["q"], d["k"], d["v"], d["g"])
        return (*pkg.linear_attn(*a, return_state=True), *pkg.linear_attn_bwd(*a, d["dy"]))

    want = [work(d) for d in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = []
        for s, d in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(work(d))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for a, b in zip(got, want) for x, y in zip(a, b))


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("D", [8, 7, 512, 520, 1030])
def test_embed_many_of_one_and_few_of_all(io, D):
    """Ids of more entries than one unit, exactly one, one more and none, side by side, whose units they share."""
    say("embed units", io, D)
    counts = [33, 0, 32, 64, 1, 65, 0, 0, 100, 31, 32, 1, 200, 2, 0, 40]
    gen = torch.Generator().manual_seed(D)
    tok = torch.cat([torch.full((n,), i) for i, n in enumerate(counts)])
    tok = tok[torch.randperm(len(tok), generator=gen)]
    dy = torch.randn(len(tok), D, generator=gen).to(ref.DT[io])
    dw = pkg.embed_bwd(tok.to(device()), dy.to(device()), len(counts), scale=0.7)
    want = torch.zeros(len(counts), D, dtype=torch.float64).index_add_(0, tok, dy.double()) * 0.7
    ref.close(dw, want, io, what="dw")


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("D", [14, 50, 1050, 1031, 1537])
def test_norm_leaves_what_is_behind(io, D):
    """What lies behind the last row, which ends inside a vector, stays as it was."""
    say("norm leaves what is behind", io, D)
    T, dev, t = 5, device(), ref.DT[io]
    f, w = torch.randn(T, D, device=dev).to(t), torch.randn(D, device=dev)
    flat = [torch.full((T * D + 16,), 3.0, dtype=t, device=dev) for _ in range(2)]
    pkg.block_norm(f, w_in=w, out=tuple(x[:T * D].view(T, D) for x in flat))
    r, y = pkg.block_norm(f, w_in=w)
    for x, want in zip(flat, (r, y)):
        assert torch.equal(x[:T * D].view(T, D), want) and bool((x[T * D:] == 3.0).all())
