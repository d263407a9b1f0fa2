"""The embedding (h3conv_embed, _bwd) against its 64-bit definition."""
import pytest
import torch

import fft_long_convolution_flashconv_amd as pkg
import layer_reference as lref
import lm_reference as ref
from parity_util import device, say

pytestmark = pytest.mark.gpu
IOS = ["f32", "f16", "bf16"]

# (T, D, V, tokens: "any", "few" (of 3 ids), "one" id, "skew" (most are one id), "out" (most outside the table))
CASES = [
    (1, 1, 1, "any"), (5, 7, 3, "any"), (64, 8, 1, "any"), (63, 33, 200, "any"), (300, 96, 50, "any"),
    (1000, 64, 1009, "any"), (1000, 65, 1009, "skew"), (2000, 16, 5, "one"), (777, 520, 70, "few"), (500, 40, 300, "out"),
    (4097, 24, 3000, "any"), (9000, 12, 70000, "skew"), (5000, 768, 50021, "any"), (20000, 8, 257, "skew"),
    (33000, 4, 40000, "few"), (300, 1, 5, "few"), (70, 2561, 9, "any"),
]


def make(io, case, seed):
    T, D, V, kind = case
    gen = torch.Generator().manual_seed(seed)
    tok = torch.randint(0, V, (T,), generator=gen)
    few = torch.randint(0, V, (3,), generator=gen)
    if kind == "few":
        tok = few[torch.randint(0, 3, (T,), generator=gen)]
    elif kind == "one":
        tok[:] = few[0]
    elif kind == "skew":
        tok[torch.rand(T, generator=gen) < 0.6] = few[0]
    elif kind == "out":
        bad = torch.tensor([-1, -100, V, V + 7, 1 << 40, -(1 << 62)])
        out = torch.rand(T, generator=gen) < 0.7
        tok[out] = bad[torch.randint(0, len(bad), (int(out.sum()),), generator=gen)]
    t = ref.DT[io]
    return tok, torch.randn(V, D, generator=gen).to(t), torch.randn(T, D, generator=gen).to(t)


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("case", CASES, ids=lambda c: "T%d_D%d_V%d_%s" % c)
def test_embed(io, case):
    say("embed", io, case)
    tok, w, dy = make(io, case, 3)
    T, D, V, _ = case
    dev = device()
    dy[(tok < 0) | (tok >= V)] = float("nan")  # (tokens outside the table add nothing)
    y = pkg.embed(tok.to(dev), w.to(dev), scale=1.7)
    dw = pkg.embed_bwd(tok.to(dev), dy.to(dev), V, scale=1.7)
    torch.cuda.synchronize()
    # one product in fp32, rounded: the scale itself is rounded to fp32 as well
    ref.close(y, lref.embed(tok, w.double(), 1.7), io, what="y")
    on = (tok >= 0) & (tok < V)
    want = torch.zeros(V, D, dtype=torch.float64).index_add_(0, tok[on], dy[on].double()) * 1.7
    ref.close(dw, want, io, what="dw")
    count = torch.bincount(tok[on], minlength=V)
    assert not dw.cpu()[count == 0].any()
    assert torch.equal(dw, pkg.embed_bwd(tok.to(dev), dy.to(dev), V, scale=1.7)), "the same bits"
    # rows by themselves: each no further off than its own sum allows (n terms in fp32, then one rounding)
    size = torch.zeros(V, D, dtype=torch.float64).index_add_(0, tok[on], dy[on].double().abs()) * 1.7
    off = (dw.double().cpu() - want).abs()
    n = count.clamp(min=1).double()[:, None]
    bound = size * (n + 2) * 2.0 ** -24 + want.abs() * (ref.HALF_ULP[io] + 2.0 ** -23) + (2.0 ** -25 if io == "f16" else 0)
    assert bool((off <= bound * 1.01).all())


def test_embed_gradient_is_that_of_the_lookup():
    """<dw, v> is the change of <y, dy> along v, for any direction v (the lookup is linear)."""
    tok, w, dy = make("f32", (400, 33, 60, "out"), 4)
    dev = device()
    v = torch.randn(60, 33, generator=torch.Generator().manual_seed(1))
    dw = pkg.embed_bwd(tok.to(dev), dy.to(dev), 60, scale=0.5)
    change = (pkg.embed(tok.to(dev), v.to(dev), scale=0.5).double() * dy.to(dev).double()).sum().item()
    dot = (dw.double().cpu() * v.double()).sum().item()
    assert abs(dot - change) <= 1e-6 * (dw.norm() * v.norm().to(dev)).item()


def test_embed_shapes_and_empty():
    dev = device()
    w = torch.randn(10, 6).to(dev)
    tok = torch.randint(0, 10, (3, 4)).to(dev)
    y = pkg.embed(tok, w)
    assert y.shape == (3, 4, 6) and torch.equal(y, w[tok])
    assert pkg.embed_bwd(tok, y, 10).shape == (10, 6)
    none = torch.zeros(0, dtype=torch.int64, device=dev)
    assert pkg.embed(none, w).shape == (0, 6)
    assert not pkg.embed_bwd(none, w[:0], 10).any()
    assert pkg.embed_bwd(tok, y, 0).shape == (0, 6)
    one = torch.tensor(3, device=dev)
    assert torch.equal(pkg.embed(one, w), w[3])
    flat = torch.randn(61).to(dev)
    assert torch.equal(pkg.embed(tok, flat[1:].view(10, 6)), flat[1:].view(10, 6)[tok])  # (any element)


def test_embed_graph_streams_and_workspace():
    """Captured and replayed with other tokens, on another stream, with a workspace of any content."""
    say("embed graph")
    dev = device()
    V = 500
    tok, w, dy = (t.to(dev) for t in make("f16", (6000, 48, V, "skew"), 5))

    def work(ws=None):
        return pkg.embed(tok, w, scale=2.0), pkg.embed_bwd(tok, dy, V, scale=2.0, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = work(torch.full((32 << 20,), 255, dtype=torch.uint8, device=dev))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(first, work()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    gen = torch.Generator().manual_seed(1)
    for i in range(4):
        tok.copy_(torch.randint(0, 5 if i == 2 else V, tok.shape, generator=gen).to(dev))
        dy.copy_(torch.randn(dy.shape, generator=gen).to(dev))
        graph.replay()
        want = work()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)), i


def test_embed_refusals():
    dev = device()
    w, tok = torch.randn(10, 6).to(dev), torch.zeros(4, dtype=torch.int64, device=dev)
    for bad in (dict(tokens=tok.int()), dict(w=w.t()), dict(w=w.double()), dict(tokens=tok.cpu()), dict(out=w)):
        with pytest.raises(ValueError):
            pkg.embed(**{**dict(tokens=tok, w=w), **bad})
    with pytest.raises(ValueError):
        pkg.embed_bwd(tok, w, 10)                            # rows of dy that are not the tokens'
    with pytest.raises(ValueError):
        pkg.embed_bwd(tok, w[:4].contiguous(), -1)
    with pytest.raises(pkg.H3ConvError):
        pkg.embed(tok, w[:, :6], out=w[:4])                  # output over input
