"""The norms around a block (h3conv_block_norm, _bwd) against their 64-bit definition."""
import pytest
import torch

import fft_long_convolution_flashconv_amd as pkg
import layer_reference as lref
import lm_reference as ref
from parity_util import device, say

pytestmark = pytest.mark.gpu
IOS = ["f32", "f16", "bf16"]
ALL = ("res", "gate", "w_out", "scale", "w_in")

# (T, D, groups, what is given)
CASES = [
    (1, 1, 1, ALL), (3, 8, 1, ALL), (5, 7, 7, ALL), (2, 9, 3, ("gate", "w_out")),
    (4, 64, 8, ALL), (3, 201, 3, ALL), (7, 201, 1, ("res", "w_in")), (33, 512, 1, ALL), (6, 513, 1, ALL),
    (5, 768, 12, ALL), (9, 768, 1, ("w_in",)), (3, 1000, 8, ALL), (4, 1024, 2, ("res", "w_out", "w_in")),
    (3, 1537, 1, ALL), (2, 1600, 50, ALL), (4, 2560, 1, ALL), (3, 2560, 40, ("gate", "w_out")), (3, 2560, 10, ALL),
    (2, 4100, 1, ALL), (3, 5001, 3, ALL), (2, 6145, 1, ALL), (2, 8192, 64, ALL), (2, 9000, 9, ALL), (1, 16384, 1, ALL),
    (1500, 40, 5, ALL), (5000, 16, 1, ("res", "scale")), (600, 130, 1, ("gate",)),
]


def make(io, case, seed):
    T, D, groups, given = case
    gen = torch.Generator().manual_seed(seed)

    def n(*s, dtype=ref.DT[io], std=1.0, mean=0.0):
        return (torch.randn(*s, generator=gen) * std + mean).to(dtype)

    f32 = torch.float32
    every = dict(res=n(T, D, std=2.0), gate=n(T, D), w_out=n(D, dtype=f32, std=0.3, mean=1.0),
                 scale=n(D, dtype=f32, std=0.3, mean=0.5), w_in=n(D, dtype=f32, std=0.3, mean=1.0))
    a = dict(f=n(T, D, std=0.7), **{k: v if k in given else None for k, v in every.items()})
    return a, n(T, D), n(T, D) if "w_in" in given else None


def gpu(d):
    return {k: None if v is None else v.to(device()) for k, v in d.items()}


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("case", CASES, ids=lambda c: "T%d_D%d_g%d_%d" % (*c[:3], len(c[3])))
def test_block_norm(io, case):
    say("block_norm", io, case)
    a, dr, dy = make(io, case, 3)
    g = gpu(a)
    out = pkg.block_norm(**g, groups=case[2], eps=1e-5)
    o = pkg.block_norm_bwd(g["f"], dr.to(device()), None if dy is None else dy.to(device()),
                           **{k: g[k] for k in ALL}, groups=case[2], eps=1e-5)
    torch.cuda.synchronize()
    leaf = {k: ref.leaf(v) for k, v in a.items()}
    r, y = lref.block_norm(**leaf, groups=case[2], eps=1e-5)
    if y is None:
        ref.close(out, r, io, what="r")
        (r * dr.double()).sum().backward()
    else:
        ref.close(out[0], r, io, what="r")
        ref.close(out[1], y, io, what="y")
        ((r * dr.double()).sum() + (y * dy.double()).sum()).backward()
    for name, got in zip(("f",) + ALL, o):
        if a[name] is None:
            assert got is None, name
        else:
            # (a norm over one channel is its sign: df is a difference of equal terms)
            one = name == "f" and case[1] == case[2]
            if one:
                assert (got.double().cpu() - leaf[name].grad).abs().max() <= 1e-5 * (1.0 / a["f"].double().abs().min()), name
            else:
                ref.close(got, leaf[name].grad, "f32" if name in ("w_out", "scale", "w_in") else io, what="d" + name)


@pytest.mark.parametrize("given", [ALL, ("res", "w_in"), ("gate", "w_out")])
def test_block_norm_differences(given):
    """The gradients as directional derivatives of the definition."""
    case = (4, 24, 3, given)
    a, dr, dy = make("f32", case, 5)
    g = gpu(a)
    o = pkg.block_norm_bwd(g["f"], dr.to(device()), None if dy is None else dy.to(device()), **{k: g[k] for k in ALL},
                           groups=3)

    def fn(x):
        r, y = lref.block_norm(**{k: x.get(k) for k in ("f",) + ALL}, groups=3)
        return (r * dr.double()).sum() + (0 if y is None else (y * dy.double()).sum())

    args = {k: v.double() for k, v in a.items() if v is not None}
    dot, diff, size = ref.directional(fn, args, dict(zip(("f",) + ALL, o)), 5)
    assert abs(dot - diff) <= 1e-5 * size + 1e-7


@pytest.mark.parametrize("io", IOS)
def test_block_norm_one_upstream(io):
    """Either upstream gradient alone, and neither."""
    a, dr, dy = make(io, (9, 130, 1, ALL), 6)
    g, dev = gpu(a), device()
    k = {n: g[n] for n in ALL}
    for up in ("dr", "dy", None):
        o = pkg.block_norm_bwd(g["f"], dr.to(dev) if up == "dr" else None, dy.to(dev) if up == "dy" else None, **k)
        leaf = {n: ref.leaf(v) for n, v in a.items()}
        r, y = lref.block_norm(**leaf)
        if up is None:
            assert all(not t.any() for t in o)
            continue
        (r * dr.double()).sum().backward() if up == "dr" else (y * dy.double()).sum().backward()
        for name, got in zip(("f",) + ALL, o):
            want = leaf[name].grad if leaf[name].grad is not None else torch.zeros_like(leaf[name])
            ref.close(got, want, "f32" if name in ("w_out", "scale", "w_in") else io, what="d" + name)


def test_block_norm_rows_apart():
    """A row of NaN, of infinities or of zeros changes no other row; a row of zeros is finite."""
    a, _, _ = make("f16", (5, 96, 4, ALL), 7)
    g = gpu(a)
    r, y = pkg.block_norm(**g, groups=4)
    for bad in (float("nan"), float("inf"), 0.0):
        f = g["f"].clone()
        f[2] = bad
        r2, y2 = pkg.block_norm(**{**g, "f": f}, groups=4)
        keep = [0, 1, 3, 4]
        assert torch.equal(r[keep], r2[keep]) and torch.equal(y[keep], y2[keep])
        assert bad != 0.0 or bool(torch.isfinite(y2).all())


def test_block_norm_any_element_and_empty():
    """Tensors that start at any element; no rows."""
    dev = device()
    for io in ("f16", "f32"):
        flat = torch.randn(3 * 50 + 1).to(ref.DT[io]).to(dev)
        w = torch.randn(51).to(dev)
        a = pkg.block_norm(flat[1:].view(3, 50), w_in=w[1:])
        b = pkg.block_norm(flat[1:].view(3, 50).clone(), w_in=w[1:].clone())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    e = torch.empty(0, 50, device=dev)
    r, y = pkg.block_norm(e, w_in=w[1:].clone())
    assert r.shape == y.shape == (0, 50)
    o = pkg.block_norm_bwd(e, e, e, w_in=w[1:].clone(), scale=w[:50].clone())
    assert o.df.shape == (0, 50) and not o.dw_in.any() and not o.dscale.any()


def test_block_norm_graph_streams_and_bits():
    """Captured and replayed with other values, on another stream, twice: the same bits."""
    say("block_norm graph")
    dev = device()
    a, dr, dy = make("bf16", (700, 320, 5, ALL), 8)
    g, dr, dy = gpu(a), dr.to(dev), dy.to(dev)

    def work():
        return (*pkg.block_norm(**g, groups=5), *pkg.block_norm_bwd(g["f"], dr, dy, **{k: g[k] for k in ALL}, groups=5))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = work()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(first, work()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    gen = torch.Generator().manual_seed(1)
    for i in range(4):
        for t in (g["f"], g["res"], g["gate"], dr, dy):
            t.copy_(torch.randn(t.shape, generator=gen).to(dev))
        graph.replay()
        want = work()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)), i


def test_block_norm_refusals():
    dev = device()
    f, w = torch.randn(4, 12).to(dev), torch.randn(12).to(dev)
    for bad in (dict(f=f.t()), dict(res=f.half()), dict(w_in=w.half()), dict(w_out=torch.randn(11).to(dev)), dict(groups=5),
                dict(groups=0), dict(gate=f[:3])):
        with pytest.raises(ValueError):
            pkg.block_norm(**{**dict(f=f, w_in=w), **bad})
    with pytest.raises(ValueError):
        pkg.block_norm_bwd(f, f, f)                          # dy without a w_in
    with pytest.raises(pkg.H3ConvError):
        pkg.block_norm(f, w_in=w, eps=-1.0)
    with pytest.raises(pkg.H3ConvError):
        pkg.block_norm(f, w_in=w, out=(f, torch.empty_like(f)))
    with pytest.raises(pkg.H3ConvError):
        pkg.block_norm(torch.randn(1, 16385).to(dev))        # more than MAX_NORM
