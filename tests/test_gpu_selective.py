"""Selective scan (h3conv_selective_scan, _bwd, h3conv_selective_step) against its 64-bit definition."""
import pytest
import torch

import fft_long_convolution_flashconv_amd as pkg
import lm_reference as ref
from parity_util import device, say

pytestmark = pytest.mark.gpu
DT = ref.DT

# (B, H, N, S, G, D, gate, bias, softplus, state, lengths)
CASES = [
    (1, 1, 1, 1, 1, True, True, True, True, False, None),          # one token, one mode
    (2, 3, 5, 16, 1, True, True, True, True, True, [0, 4]),        # an empty row
    (2, 4, 64, 8, 2, True, False, True, True, True, None),
    (1, 6, 255, 5, 3, False, True, False, True, False, [254]),     # one short of a piece of saved states
    (1, 2, 257, 16, 1, True, True, True, True, True, None),        # one past it
    (3, 5, 300, 17, 5, True, True, True, True, True, [300, 1, 256]),  # modes past a block of 16
    (2, 9, 513, 16, 3, True, True, True, False, True, [512, 513]),
    (1, 3, 700, 64, 1, True, True, True, True, False, None),       # the most modes
    (1, 70, 130, 16, 1, True, True, True, True, False, None),      # more channels than one set
    (1, 2, 1100, 3, 2, True, False, True, True, True, [1023]),
]


def _make(io, case, seed):
    B, H, N, S, G, D, gate, bias, softplus, state, lengths = case
    g = torch.Generator().manual_seed(seed)
    t = DT[io]

    def n(*s, std=1.0, dtype=t):
        return (torch.randn(*s, generator=g) * std).to(dtype)

    dt = n(B, H, N, std=0.5)
    if not softplus:
        dt = (dt.float().abs() * 0.1).to(t)
    d = dict(u=n(B, H, N), dt=dt, A=-torch.arange(1, S + 1).float() * torch.exp(0.2 * n(H, S, dtype=torch.float32)),
             Bm=n(B, G, S, N), C=n(B, G, S, N), D=n(H, dtype=torch.float32) if D else None,
             z=n(B, H, N) if gate else None,
             dt_bias=(n(H, dtype=torch.float32) - 2.0 if softplus else n(H, dtype=torch.float32).abs() * 0.05) if bias else None,
             x_in=n(B, H, S, dtype=torch.float32) if state else None, dy=n(B, H, N),
             dx_out=n(B, H, S, dtype=torch.float32),
             lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32))
    if lengths is not None:
        for b, k in enumerate(lengths):
            for key in ("u", "dt", "Bm", "C", "z", "dy"):
                if d[key] is not None:
                    d[key][b, ..., k:] = float("nan")
                    if k + 1 < N:
                        d[key][b, ..., k + 1] = float("inf")
    return d


def _gpu(d):
    dev = device()
    return {k: v.to(dev) if torch.is_tensor(v) else v for k, v in d.items()}


def _args(g):
    return (g["u"], g["dt"], g["A"], g["Bm"], g["C"]), dict(D=g["D"], z=g["z"], dt_bias=g["dt_bias"])


KEYS = ("u", "dt", "A", "Bm", "C", "D", "z", "dt_bias", "x_in")


def _clean(d):
    return {k: (torch.nan_to_num(d[k].double(), 0.0, 0.0, 0.0) if d[k] is not None else None) for k in KEYS + ("dy", "dx_out")}


def _definition(a, case):
    return ref.selective_scan(a["u"], a["dt"], a["A"], a["Bm"], a["C"], a["D"], a["z"], a["dt_bias"], case[8], a["x_in"],
                              case[10])


ids = lambda c: "B%d_H%d_N%d_S%d_G%d" % c[:5]


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=ids)
def test_selective_scan(io, case):
    say("selective_scan", io, case)
    d = _make(io, case, 7)
    g = _gpu(d)
    a, k = _args(g)
    y, xo = pkg.selective_scan(*a, softplus=case[8], x_in=g["x_in"], lengths=g["lengths"], return_state=True, **k)
    torch.cuda.synchronize()
    ry, ro = _definition(_clean(d), case)
    ref.close(y, ry, io, what="y")
    ref.close(xo, ro, what="x_out")


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=ids)
def test_selective_scan_bwd(io, case):
    say("selective_scan_bwd", io, case)
    d = _make(io, case, 11)
    g = _gpu(d)
    a, k = _args(g)
    y, saved = pkg.selective_scan(*a, softplus=case[8], x_in=g["x_in"], lengths=g["lengths"], return_saved=True, **k)
    o = pkg.selective_scan_bwd(*a, g["dy"], saved, softplus=case[8], lengths=g["lengths"], dx_out=g["dx_out"], **k)
    torch.cuda.synchronize()
    c = _clean(d)
    leaves = {key: ref.leaf(c[key]) for key in KEYS}
    ry, ro = _definition(leaves, case)
    ((ry * c["dy"]).sum() + (ro * c["dx_out"]).sum()).backward()
    for name, got, key, kind in (("du", o.du, "u", io), ("ddt", o.ddt, "dt", io), ("dA", o.dA, "A", "f32"),
                                 ("dB", o.dB, "Bm", io), ("dC", o.dC, "C", io), ("dD", o.dD, "D", "f32"),
                                 ("dz", o.dz, "z", io), ("ddt_bias", o.ddt_bias, "dt_bias", "f32"),
                                 ("dx_in", o.dx_in, "x_in", "f32")):
        if leaves[key] is None:
            assert got is None or key == "x_in"
        else:
            ref.close(got, leaves[key].grad, kind, what=name)


def test_selective_scan_bwd_differences():
    """The gradients as directional derivatives of the definition."""
    case = (2, 4, 37, 6, 2, True, True, True, True, True, [37, 20])
    d = _make("f32", case, 3)
    g = _gpu(d)
    a, k = _args(g)
    _, saved = pkg.selective_scan(*a, x_in=g["x_in"], lengths=g["lengths"], return_saved=True, **k)
    o = pkg.selective_scan_bwd(*a, g["dy"], saved, lengths=g["lengths"], dx_out=g["dx_out"], **k)
    c = _clean(d)

    def f(v):
        y, xo = _definition(v, case)
        return (y * c["dy"]).sum() + (xo * c["dx_out"]).sum()

    grads = dict(u=o.du, dt=o.ddt, A=o.dA, Bm=o.dB, C=o.dC, D=o.dD, z=o.dz, dt_bias=o.ddt_bias, x_in=o.dx_in)
    dot, diff, size = ref.directional(f, {key: c[key] for key in KEYS}, grads, 5)
    assert abs(dot - diff) <= 1e-5 * size + 1e-6


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,H,P,S,G", [(1, 1, 1, 1, 1), (5, 34, 9, 16, 2), (3, 12, 4, 5, 1), (4, 300, 4, 64, 4), (3, 7, 3, 20, 7)])
def test_selective_step(io, B, H, P, S, G):
    """Tokens one at a time, in place and into a second pool, with idle rows."""
    say("selective_step", io, B, H, P, S, G)
    dev = device()
    K = 4
    case = (B, H, K, S, G, True, True, True, True, False, None)
    d = _make(io, case, 13)
    gen = torch.Generator().manual_seed(1)
    pool = torch.randn(P, H, S, generator=gen)
    slots = torch.randperm(P, generator=gen)[:B].to(torch.int32)
    idle = B > 2
    if idle:
        slots[1] = -1 if io == "f16" else P
    busy = [b for b in range(B) if 0 <= int(slots[b]) < P]
    used = torch.zeros(P, dtype=torch.bool)
    used[slots[busy].long()] = True
    used = used.to(dev)
    x, sl = pool.to(dev), slots.to(dev)
    g = _gpu(d)
    ys = []
    for t in range(K):
        a = [g[k][..., t].contiguous() for k in ("u", "dt")] + [g["A"]] + [g[k][..., t].contiguous() for k in ("Bm", "C")]
        k = dict(D=g["D"], z=g["z"][..., t].contiguous(), dt_bias=g["dt_bias"], slots=sl)
        nxt = torch.full_like(x, 7.0)
        y0 = pkg.selective_step(*a, x, x_out=nxt, **k)
        before = x.clone()
        y1 = pkg.selective_step(*a, x, **k)
        assert torch.equal(y0, y1) and torch.equal(nxt[used], x[used])
        assert bool((nxt[~used] == 7.0).all()) and torch.equal(before[~used], x[~used])
        ys.append(y1)
    y = torch.stack(ys, -1).cpu()
    c = {key: (v[busy] if key not in ("A", "D", "dt_bias") and v is not None else v) for key, v in _clean(d).items()}
    c["x_in"] = pool[slots[busy].long()].double()
    ry, ro = _definition(c, case)
    ref.close(y[busy], ry, io, what="y")
    ref.close(x.cpu()[slots[busy].long()], ro, what="state")
    if idle:
        assert bool((y[1] == 0).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prompt_then_tokens(io):
    """A ragged prompt's final states continue token by token."""
    dev = device()
    case = (3, 10, 70, 16, 1, True, True, True, True, False, None)
    d = _make(io, case, 17)
    g = _gpu(d)
    n = [64, 1, 33]
    a, k = _args(g)
    _, x = pkg.selective_scan(*a, lengths=torch.tensor(n, dtype=torch.int32, device=dev), return_state=True, **k)
    ys = []
    for t in range(3):  # the next tokens of each row are at its own length
        pick = lambda m: torch.stack([m[b, ..., n[b] + t] for b in range(3)]).contiguous()
        ys.append(pkg.selective_step(pick(g["u"]), pick(g["dt"]), g["A"], pick(g["Bm"]), pick(g["C"]), x, D=g["D"],
                                     z=pick(g["z"]), dt_bias=g["dt_bias"]))
    ry, _ = _definition(_clean(d), case)
    for t in range(3):
        ref.close(ys[t], torch.stack([ry[b, :, n[b] + t] for b in range(3)]), io, what="token %d" % t)


def test_selective_pieces_join():
    """A row in two pieces joined by the state is the row in one (bit for bit where the cut is on a piece)."""
    d = _gpu(_make("f32", (2, 5, 1300, 16, 1, True, True, True, True, True, None), 19))
    a, k = _args(d)
    y, x = pkg.selective_scan(*a, x_in=d["x_in"], return_state=True, **k)
    for cut in (1, 511, 700, 1299):
        def part(s):
            p = [t[..., s].contiguous() if t.dim() > 2 else t for t in a]
            return p, dict(k, z=k["z"][..., s].contiguous())
        p, q = part(slice(0, cut))
        y0, m = pkg.selective_scan(*p, x_in=d["x_in"], return_state=True, **q)
        p, q = part(slice(cut, None))
        y1, e = pkg.selective_scan(*p, x_in=m, return_state=True, **q)
        ref.close(torch.cat([y0, y1], -1), y.double().cpu(), what="y")
        ref.close(e, x.double().cpu(), what="x")


def test_selective_long_memory_and_stiff_modes():
    """Steps from 1e-6 to 60, rates from 1e-4 to 1e3: states that hardly decay and states that vanish at once."""
    case = (1, 6, 900, 4, 1, True, False, False, False, True, None)
    d = _make("f32", case, 23)
    d["dt"] = torch.logspace(-6, 1.7, 900).repeat(1, 6, 1).contiguous()
    d["A"] = -torch.tensor([1e-4, 1e-1, 3.0, 1e3]).repeat(6, 1).contiguous()
    g = _gpu(d)
    a, k = _args(g)
    y, xo = pkg.selective_scan(*a, softplus=False, x_in=g["x_in"], return_state=True, **k)
    ry, ro = _definition(_clean(d), case)
    ref.close(y, ry, what="y")
    ref.close(xo, ro, what="x")


def test_softplus_range():
    """d from -80 to 80: the smallest steps keep their relative precision."""
    dev = device()
    N = 401
    dt = torch.linspace(-80, 80, N).view(1, 1, N)
    one = torch.ones(1, 1, N)
    # A = 0, B = C = u = 1: y_t is the running sum of the steps
    y = pkg.selective_scan(one.to(dev), dt.to(dev), torch.zeros(1, 1, device=dev), one.view(1, 1, 1, N).to(dev),
                           one.view(1, 1, 1, N).to(dev))
    want = torch.nn.functional.softplus(dt.double(), threshold=1e9).cumsum(-1)
    rel = ((y.double().cpu() - want).abs() / want).max().item()
    assert rel <= 1e-5, rel


def test_selective_empty():
    dev = device()
    A, x = -torch.ones(4, 3, device=dev), torch.randn(2, 4, 3).to(dev)
    e, bc = torch.empty(2, 4, 0, device=dev), torch.empty(2, 1, 3, 0, device=dev)
    y, xo, saved = pkg.selective_scan(e, e, A, bc, bc, x_in=x, return_state=True, return_saved=True)
    assert y.shape == (2, 4, 0) and torch.equal(xo, x)
    g = torch.randn(2, 4, 3).to(dev)
    o = pkg.selective_scan_bwd(e, e, A, bc, bc, e, saved, D=A[:, 0].contiguous(), dx_out=g)
    assert bool((o.dA == 0).all()) and bool((o.dD == 0).all()) and torch.equal(o.dx_in, g)
    e, bc = torch.empty(0, 4, 5, device=dev), torch.empty(0, 1, 3, 5, device=dev)
    y, saved = pkg.selective_scan(e, e, A, bc, bc, return_saved=True)
    o = pkg.selective_scan_bwd(e, e, A, bc, bc, e, saved)
    assert bool((o.dA == 0).all()) and y.shape == (0, 4, 5)


def test_selective_same_bits_and_other_stream():
    d = _gpu(_make("bf16", (2, 96, 600, 16, 2, True, True, True, True, False, None), 29))
    a, k = _args(d)

    def once():
        y, saved = pkg.selective_scan(*a, return_saved=True, **k)
        return (y,) + tuple(t for t in pkg.selective_scan_bwd(*a, d["dy"], saved, **k) if t is not None)

    one = once()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        two = once()
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(one, two))


def test_selective_refusals():
    d = _gpu(_make("f32", (2, 4, 8, 3, 2, True, True, True, True, False, None), 1))
    a, k = _args(d)
    u, dt, A, Bm, C = a
    _, saved = pkg.selective_scan(*a, return_saved=True, **k)
    with pytest.raises(ValueError):
        pkg.selective_scan(u, dt.half(), A, Bm, C)
    with pytest.raises(ValueError):
        pkg.selective_scan(u, dt, A, Bm[:, :1].expand(2, 3, 3, 8).contiguous(), C)   # 3 groups over 4 channels
    with pytest.raises(ValueError):
        pkg.selective_scan(u, dt, A, Bm.transpose(2, 3), C)
    with pytest.raises(ValueError):
        pkg.selective_scan(u, dt, A, Bm, C, z=d["z"][..., :4].contiguous())
    with pytest.raises(ValueError):
        pkg.selective_scan_bwd(u, dt, A, Bm, C, d["dy"], saved[:-1].contiguous())
    with pytest.raises(TypeError):
        pkg.selective_scan_bwd(u, dt, A, Bm, C, d["dy"], None)
    with pytest.raises(pkg.H3ConvError):
        pkg.selective_scan(u, dt, A, Bm, C, out=u)
    wide = torch.zeros(4, 65, device=u.device)
    with pytest.raises(pkg.H3ConvError):
        pkg.selective_scan(u, dt, wide, torch.zeros(2, 2, 65, 8, device=u.device), torch.zeros(2, 2, 65, 8, device=u.device))
    with pytest.raises(pkg.H3ConvError):  # pool below the batch
        pkg.selective_step(u[..., 0].contiguous(), dt[..., 0].contiguous(), A, Bm[..., 0].contiguous(),
                           C[..., 0].contiguous(), torch.zeros(1, 4, 3, device=u.device))


# Many rows and long rows: the waves of a block have rows of their own, share a
# row's steps, or share its modes; pieces end inside, before and after a lane.
WIDE = [
    (3, 700, 9, 5, 1, True, True, True, True, True, [0, 9, 4]),        # fewer steps than a lane takes
    (4, 520, 201, 4, 2, True, True, True, True, True, [201, 1, 17, 200]),
    (2, 300, 301, 3, 3, True, True, True, True, True, None),
    (2, 300, 1040, 6, 1, True, False, True, True, True, [1024, 1033]),
    (2, 3, 3090, 5, 1, True, True, True, True, True, [3090, 3079]),
    (1, 2, 7171, 4, 1, True, True, True, True, True, [4097]),
]


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", WIDE, ids=ids)
def test_selective_scan_wide(io, case):
    test_selective_scan(io, case)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("case", WIDE[1:5], ids=ids)
def test_selective_scan_bwd_wide(io, case):
    test_selective_scan_bwd(io, case)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("S", [2, 4, 7, 9, 15, 19, 33, 48])
def test_selective_scan_bwd_modes(io, S):
    """Blocks of modes of every size, an odd number of steps."""
    test_selective_scan_bwd(io, (2, 10, 131, S, 2, True, True, True, True, True, [131, 40]))
