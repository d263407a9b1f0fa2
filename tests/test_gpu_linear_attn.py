"""Linear attention with decay (h3conv_linear_attn, _bwd, _step) against its 64-bit definition."""
import pytest
import torch

import fft_long_convolution_flashconv_amd as pkg
import layer_reference as lref
import lm_reference as ref
from parity_util import device, say

pytestmark = pytest.mark.gpu
DT = ref.DT
IOS = ["f32", "f16", "bf16"]

# (B, N, H, G, dk, dv, a decay per token, a state, lengths)
CASES = [
    (1, 1, 1, 1, 1, 1, False, False, None),                  # one token, one number
    (2, 3, 2, 1, 5, 7, True, True, [0, 2]),                  # an empty row and a short one
    (3, 1, 4, 2, 24, 41, True, True, [1, 0, 5]),             # one token; a length past N is N
    (1, 16, 1, 1, 16, 16, False, True, None),
    (2, 32, 2, 2, 32, 32, True, False, [32, 31]),
    (1, 64, 1, 1, 64, 64, False, False, None),               # one whole chunk
    (2, 65, 3, 1, 16, 48, True, True, [65, 64]),             # one step past it
    (2, 63, 2, 2, 33, 40, False, True, [63, -4]),            # odd; a negative length is empty
    (1, 129, 2, 1, 64, 64, True, True, None),
    (2, 200, 4, 2, 64, 128, True, True, [200, 129]),
    (1, 97, 1, 1, 128, 64, False, False, None),
    (1, 70, 2, 1, 130, 256, True, True, [67]),               # more than 128 of either
    (1, 70, 1, 1, 256, 9, True, True, None),
    (1, 700, 1, 1, 20, 12, True, True, [699]),               # many chunks of one head
    (2, 333, 6, 2, 64, 32, False, False, None),
    (40, 5, 8, 8, 16, 16, True, True, None),                 # many short rows
]
IDS = ["B%d_N%d_H%d_G%d_%dx%d%s" % (*c[:6], "_token" if c[6] else "") for c in CASES]


def make(io, case, seed, strength=0.2):
    B, N, H, G, dk, dv, token, state, lengths = case
    gen = torch.Generator().manual_seed(seed)

    def n(*s, dtype=DT[io], std=1.0):
        return (torch.randn(*s, generator=gen) * std).to(dtype)

    d = dict(q=n(B, N, G, dk), k=n(B, N, G, dk), v=n(B, N, H, dv),
             g=-strength * n(*((B, N, H) if token else (H,)), dtype=torch.float32).abs(),
             x_in=n(B, H, dk, dv, dtype=torch.float32) if state else None, dy=n(B, N, H, dv),
             dx_out=n(B, H, dk, dv, dtype=torch.float32) if state else None,
             lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32))
    if lengths is not None:  # nothing past a row's end may be read into a result
        for b, m in enumerate(lengths):
            for key in ("q", "k", "v", "dy") + (("g",) if token else ()):
                d[key][b, max(m, 0):] = float("nan")
                d[key][b, max(m, 0) + 1:] = float("inf")
    return d


def gpu(d):
    return {k: v.to(device()) if torch.is_tensor(v) else v for k, v in d.items()}


def clean(d):
    return {k: torch.nan_to_num(v.double(), 0.0, 0.0, 0.0) if torch.is_tensor(v) and v.is_floating_point() else v
            for k, v in d.items()}


def grads(d, scale, lengths):
    """Leaves with their gradients by the definition, y, x_out, and the size of dg's terms."""
    c = clean(d)
    G, H = c["q"].shape[2], c["v"].shape[2]
    leaf = {k: ref.leaf(c[k]) for k in ("q", "k", "v", "g", "x_in")}
    wide = {k: leaf[k].repeat_interleave(H // G, 2) for k in ("q", "k")}
    for t in wide.values():
        t.retain_grad()
    y, xo = lref.linear_attn(wide["q"], wide["k"], leaf["v"], leaf["g"], scale, leaf["x_in"], lengths)
    s = (y * c["dy"]).sum()
    if c["dx_out"] is not None:
        s = s + (xo * c["dx_out"]).sum()
    if s.requires_grad:
        s.backward()
    for t in [*leaf.values(), *wide.values()]:
        if t is not None and t.grad is None:
            t.grad = torch.zeros_like(t)
    terms = ((wide["q"] * wide["q"].grad).sum(-1).square().sum() + (wide["k"] * wide["k"].grad).sum(-1).square().sum()).sqrt()
    return leaf, y.detach(), xo.detach(), terms.item()


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_linear_attn(io, case):
    say("linear_attn", io, case)
    d = make(io, case, 3)
    g = gpu(d)
    y, xo = pkg.linear_attn(g["q"], g["k"], g["v"], g["g"], scale=0.3, x_in=g["x_in"], lengths=g["lengths"],
                            return_state=True)
    torch.cuda.synchronize()
    c = clean(d)
    ry, rx = lref.linear_attn(c["q"], c["k"], c["v"], c["g"], 0.3, c["x_in"], case[8])
    ref.close(y, ry, io, what="y")
    ref.close(xo, rx, what="x_out")
    for b, n in enumerate(case[8] or []):
        assert bool((y[b, max(n, 0):] == 0).all())
    only = pkg.linear_attn(g["q"], g["k"], g["v"], g["g"], scale=0.3, x_in=g["x_in"], lengths=g["lengths"])
    assert torch.equal(only, y)


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_linear_attn_bwd(io, case):
    say("linear_attn_bwd", io, case)
    d = make(io, case, 5)
    g = gpu(d)
    o = pkg.linear_attn_bwd(g["q"], g["k"], g["v"], g["g"], g["dy"], scale=0.3, x_in=g["x_in"], lengths=g["lengths"],
                            dx_out=g["dx_out"])
    torch.cuda.synchronize()
    leaf, _, _, terms = grads(d, 0.3, case[8])
    for name, got in (("q", o.dq), ("k", o.dk), ("v", o.dv)):
        ref.close(got, leaf[name].grad, io, what="d" + name)
    lref.close_dg(o.dg, leaf["g"].grad, terms, case[1])
    if leaf["x_in"] is not None:
        ref.close(o.dx_in, leaf["x_in"].grad, what="dx_in")
    for b, n in enumerate(case[8] or []):
        for t in (o.dq, o.dk, o.dv) + ((o.dg,) if case[6] else ()):
            assert bool((t[b, max(n, 0):] == 0).all())


@pytest.mark.parametrize("token", [False, True])
def test_linear_attn_differences(token):
    """The gradients as directional derivatives of the definition."""
    case = (2, 41, 2, 1, 6, 5, token, True, [41, 30])
    d = make("f32", case, 8)
    g = gpu(d)
    o = pkg.linear_attn_bwd(g["q"], g["k"], g["v"], g["g"], g["dy"], scale=0.7, x_in=g["x_in"], lengths=g["lengths"],
                            dx_out=g["dx_out"])
    c = clean(d)

    def f(a):
        y, xo = lref.linear_attn(a["q"], a["k"], a["v"], a["g"], 0.7, a["x_in"], case[8])
        return (y * c["dy"]).sum() + (xo * c["dx_out"]).sum()

    args = {k: c[k] for k in ("q", "k", "v", "g", "x_in")}
    dot, diff, size = ref.directional(f, args, dict(zip(("q", "k", "v", "g", "x_in"), o)), 5)
    assert abs(dot - diff) <= 2e-5 * size + 1e-7


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("strength", [0.0, 3.0, 30.0])
def test_linear_attn_decays(io, strength):
    """No decay, strong decay, factors that underflow, and steps that start the state anew."""
    case = (2, 150, 3, 3, 24, 40, True, True, None)
    d = make(io, case, 9, strength)
    d["g"][0, 70] = float("-inf")
    d["g"][1, 0] = -1e30
    g = gpu(d)
    y, xo = pkg.linear_attn(g["q"], g["k"], g["v"], g["g"], x_in=g["x_in"], return_state=True)
    o = pkg.linear_attn_bwd(g["q"], g["k"], g["v"], g["g"], g["dy"], x_in=g["x_in"], dx_out=g["dx_out"])
    d["g"] = d["g"].clamp(min=-1e4)  # (its factor is zero in 64 bits too)
    leaf, ry, rx, terms = grads(d, 1.0, None)
    ref.close(y, ry, io, what="y")
    ref.close(xo, rx, what="x_out")
    for name, got in (("q", o.dq), ("k", o.dk), ("v", o.dv)):
        ref.close(got, leaf[name].grad, io, what="d" + name)
    lref.close_dg(o.dg, leaf["g"].grad, terms, case[1])
    ref.close(o.dx_in, leaf["x_in"].grad, what="dx_in")
    assert bool((o.dg[0, 70] == 0).all())


@pytest.mark.parametrize("io", IOS)
def test_linear_attn_growth(io):
    """Factors above one."""
    case = (1, 140, 2, 2, 16, 16, True, True, None)
    d = make(io, case, 10)
    d["g"] = -d["g"] * 0.3
    g = gpu(d)
    y, xo = pkg.linear_attn(g["q"], g["k"], g["v"], g["g"], scale=2.0 ** -12, x_in=g["x_in"], return_state=True)
    c = clean(d)
    ry, rx = lref.linear_attn(c["q"], c["k"], c["v"], c["g"], 2.0 ** -12, c["x_in"], None)
    ref.close(y, ry, io, what="y")
    ref.close(xo, rx, what="x_out")


def test_linear_attn_scales_f16():
    """Products and states beyond fp16's range, next to small ones, whose results are within it."""
    say("linear_attn scales")
    case = (1, 200, 2, 2, 32, 32, True, True, None)
    d = make("f16", case, 11)
    q, k, v = d["q"].float(), d["k"].float(), d["v"].float()
    big = torch.arange(200) % 3 == 0
    d["q"] = torch.where(big[None, :, None, None], q * 300, q * 2.0 ** -6).half()
    d["k"], d["v"] = (k * 3000).half(), (v * 2.0 ** -10).half()
    d["x_in"] = d["x_in"] * 4000
    g = gpu(d)
    scale = 2.0 ** -8
    y, xo = pkg.linear_attn(g["q"], g["k"], g["v"], g["g"], scale=scale, x_in=g["x_in"], return_state=True)
    c = clean(d)
    ry, rx = lref.linear_attn(c["q"], c["k"], c["v"], c["g"], scale, c["x_in"], None)
    ref.close(y[:, big.to(device())], ry[:, big], "f16", what="y, large")
    ref.close(y[:, ~big.to(device())], ry[:, ~big], "f16", what="y, small")
    ref.close(xo, rx, what="x_out")


@pytest.mark.parametrize("io", IOS)
def test_linear_attn_slices(io):
    """q, k and v as slices of one projection, at any element."""
    say("linear_attn slices", io)
    B, N, H, G, dk, dv = 2, 77, 4, 2, 16, 24
    gen = torch.Generator().manual_seed(2)
    for off in (0, 1):
        wide = torch.randn(B, N, off + 2 * G * dk + H * dv + 3, generator=gen).to(DT[io]).to(device())
        q = wide[..., off:off + G * dk].unflatten(-1, (G, dk))
        k = wide[..., off + G * dk:off + 2 * G * dk].unflatten(-1, (G, dk))
        v = wide[..., off + 2 * G * dk:off + 2 * G * dk + H * dv].unflatten(-1, (H, dv))
        g, dy = torch.full((H,), -0.05, device=device()), torch.randn(B, N, H, dv, generator=gen).to(DT[io]).to(device())
        a = pkg.linear_attn(q, k, v, g, return_state=True)
        b = pkg.linear_attn(q.contiguous(), k.contiguous(), v.contiguous(), g, return_state=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        a = pkg.linear_attn_bwd(q, k, v, g, dy)
        b = pkg.linear_attn_bwd(q.contiguous(), k.contiguous(), v.contiguous(), g, dy)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        x1, x2 = (torch.ones(B, H, dk, dv, device=device()) for _ in range(2))
        a = pkg.linear_attn_step(q[:, 5], k[:, 5], v[:, 5], g, x1)
        b = pkg.linear_attn_step(q[:, 5].contiguous(), k[:, 5].contiguous(), v[:, 5].contiguous(), g, x2)
        assert torch.equal(a, b) and torch.equal(x1, x2)


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("B,H,G,P,dk,dv,token", [(1, 1, 1, 1, 1, 1, False), (5, 4, 2, 9, 24, 41, True), (4, 3, 3, 4, 64, 64, False),
                                                 (3, 2, 1, 6, 128, 130, True), (3, 2, 1, 6, 256, 256, True)])
def test_linear_attn_step(io, B, H, G, P, dk, dv, token):
    """Tokens one at a time, in place and into a second pool, with idle rows."""
    say("linear_attn_step", io, B, H, G, P, dk, dv)
    dev = device()
    d = make(io, (B, 4, H, G, dk, dv, token, False, None), 6)
    gen = torch.Generator().manual_seed(1)
    pool = torch.randn(P, H, dk, dv, generator=gen)
    slots = torch.randperm(P, generator=gen)[:B].to(torch.int32)
    if B > 2:
        slots[1] = -1 if io == "f16" else P
    busy = [b for b in range(B) if 0 <= int(slots[b]) < P]
    used = torch.zeros(P, dtype=torch.bool)
    used[slots[busy].long()] = True
    state, ys = pool.to(dev), []
    for t in range(4):
        a = [d[n][:, t].contiguous().to(dev) for n in ("q", "k", "v")] + [(d["g"][:, t].contiguous() if token else d["g"]).to(dev)]
        nxt, before = torch.full_like(state, 7.0), state.clone()
        y2 = pkg.linear_attn_step(*a, state, scale=0.5, slots=slots.to(dev), x_out=nxt)
        y = pkg.linear_attn_step(*a, state, scale=0.5, slots=slots.to(dev))
        assert torch.equal(y, y2) and torch.equal(nxt[used.to(dev)], state[used.to(dev)])
        assert bool((nxt[~used.to(dev)] == 7.0).all()) and torch.equal(before[~used.to(dev)], state[~used.to(dev)])
        ys.append(y)
    c = clean(d)
    ry, rx = lref.linear_attn(c["q"][busy], c["k"][busy], c["v"][busy], c["g"][busy] if token else c["g"], 0.5,
                              pool[slots[busy].long()].double(), None)
    y = torch.stack(ys, 1).cpu()
    ref.close(y[busy], ry, io, what="y")
    ref.close(state.cpu()[slots[busy].long()], rx, what="state")
    if B > 2:
        assert bool((y[1] == 0).all())


@pytest.mark.parametrize("io", IOS)
def test_linear_attn_pieces_and_steps(io):
    """A row in pieces joined by the state, and a prompt that goes on token by token."""
    say("linear_attn pieces", io)
    d = gpu(make(io, (2, 300, 2, 1, 40, 64, True, True, None), 4))
    a = [d[n] for n in ("q", "k", "v", "g")]
    y, end = pkg.linear_attn(*a, x_in=d["x_in"], return_state=True)
    for cut in (1, 63, 64, 200, 299):
        y1, s = pkg.linear_attn(*[t[:, :cut].contiguous() for t in a], x_in=d["x_in"], return_state=True)
        y2, e = pkg.linear_attn(*[t[:, cut:].contiguous() for t in a], x_in=s, return_state=True)
        ref.close(torch.cat([y1, y2], 1), y.double().cpu(), io, roundings=2, what="y")
        ref.close(e, end.double().cpu(), what="state")
    _, s = pkg.linear_attn(*[t[:, :290].contiguous() for t in a], x_in=d["x_in"], return_state=True)
    last = [pkg.linear_attn_step(*[t[:, i].contiguous() for t in a], s) for i in range(290, 300)]
    ref.close(torch.stack(last, 1), y[:, 290:].double().cpu(), io, roundings=2, what="steps")
    ref.close(s, end.double().cpu(), what="state by steps")


def test_linear_attn_empty():
    dev = device()

    def z(*s):
        return torch.zeros(*s, device=dev)

    x, dx = torch.randn(2, 3, 4, 5).to(dev), torch.randn(2, 3, 4, 5).to(dev)
    y, xo = pkg.linear_attn(z(2, 0, 3, 4), z(2, 0, 3, 4), z(2, 0, 3, 5), z(3), x_in=x, return_state=True)
    assert y.shape == (2, 0, 3, 5) and torch.equal(xo, x)
    y, xo = pkg.linear_attn(z(2, 0, 3, 4), z(2, 0, 3, 4), z(2, 0, 3, 5), z(2, 0, 3), return_state=True)
    assert not xo.any()
    o = pkg.linear_attn_bwd(z(2, 0, 3, 4), z(2, 0, 3, 4), z(2, 0, 3, 5), z(3), z(2, 0, 3, 5), x_in=x, dx_out=dx)
    assert torch.equal(o.dx_in, dx) and not o.dg.any()
    o = pkg.linear_attn_bwd(z(0, 6, 3, 4), z(0, 6, 3, 4), z(0, 6, 3, 5), z(3), z(0, 6, 3, 5))
    assert o.dq.shape == (0, 6, 3, 4) and not o.dg.any()
    assert pkg.linear_attn_step(z(0, 3, 4), z(0, 3, 4), z(0, 3, 5), z(3), z(2, 3, 4, 5)).shape == (0, 3, 5)


def test_linear_attn_same_bits_other_stream_and_workspace():
    """Two runs give the same bits, also on a stream and with a workspace of the caller's, whatever it holds."""
    d = gpu(make("bf16", (2, 500, 4, 2, 64, 48, True, True, None), 2))
    a = [d[n] for n in ("q", "k", "v", "g")]
    k = dict(x_in=d["x_in"])
    one, og = pkg.linear_attn(*a, return_state=True, **k), pkg.linear_attn_bwd(*a, d["dy"], dx_out=d["dx_out"], **k)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=device())
        two = pkg.linear_attn(*a, return_state=True, workspace=ws, **k)
        ws.fill_(255)
        tg = pkg.linear_attn_bwd(*a, d["dy"], dx_out=d["dx_out"], workspace=ws, **k)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(one + tuple(og), two + tuple(tg)))


def test_linear_attn_in_a_graph():
    """Forward, backward and a token's step captured once and replayed, against eager calls."""
    say("linear_attn in a graph")
    dev = device()
    d = gpu(make("f16", (2, 400, 3, 3, 32, 64, True, True, None), 3))
    a = [d[n] for n in ("q", "k", "v", "g")]
    pool = torch.zeros(4, 3, 32, 64, device=dev)
    slots = torch.tensor([3, 1], dtype=torch.int32, device=dev)

    def work(pool):
        y, x = pkg.linear_attn(*a, x_in=d["x_in"], return_state=True)
        o = pkg.linear_attn_bwd(*a, d["dy"], x_in=d["x_in"], dx_out=d["dx_out"])
        return (y, x, *o, pkg.linear_attn_step(*[t[:, 7].contiguous() for t in a], pool, slots=slots))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(pool.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work(pool)
    pool.zero_()
    eager = torch.zeros_like(pool)
    gen = torch.Generator().manual_seed(7)
    for i in range(4):
        for t in (*a[:3], d["dy"], d["x_in"], d["dx_out"]):
            t.copy_(torch.randn(t.shape, generator=gen).to(dev))
        graph.replay()
        want = work(eager)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)) and torch.equal(pool, eager), i


def test_linear_attn_refusals():
    dev = device()

    def r(*s):
        return torch.randn(*s).to(dev)

    q, k, v, g = r(2, 6, 2, 8), r(2, 6, 2, 8), r(2, 6, 4, 8), r(4)
    for bad in (dict(q=q.transpose(1, 2)), dict(k=k[:1]), dict(k=k.half()), dict(v=v[..., ::2]), dict(g=r(3)), dict(g=r(2, 6, 2)),
                dict(g=g.double()), dict(q=r(2, 6, 3, 8)), dict(x_in=r(2, 4, 8, 7)), dict(lengths=torch.tensor([1, 2]).to(dev)),
                dict(v=v[:, :, :1].expand(2, 6, 4, 8)), dict(q=r(2, 6, 2, 9)), dict(k=k.cpu())):
        a = dict(q=q, k=k, v=v, g=g)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            pkg.linear_attn(**a)
    with pytest.raises(pkg.H3ConvError):
        pkg.linear_attn(r(1, 2, 1, 257), r(1, 2, 1, 257), r(1, 2, 1, 4), r(1))     # more than MAX_HEAD
    with pytest.raises(pkg.H3ConvError):
        pkg.linear_attn(q, k, v, g, out=v)                                        # output over input
    with pytest.raises(ValueError):
        pkg.linear_attn_bwd(q, k, v, g, v[:, :5].contiguous())
    with pytest.raises(pkg.H3ConvError):
        pkg.linear_attn_step(q[:, 0], k[:, 0], v[:, 0], g, r(1, 4, 8, 8))          # pool below the batch
