"""Short causal convolution (h3conv_short_conv, _bwd, _step) against its 64-bit definition."""
import pytest
import torch

import fft_long_convolution_flashconv_amd as pkg
import lm_reference as ref
from parity_util import device, say

pytestmark = pytest.mark.gpu
DT = ref.DT

# (B, H, N, W, bias, silu, state, lengths)
CASES = [
    (1, 1, 1, 4, True, True, False, None),           # one token
    (2, 3, 2, 4, True, True, True, [0, 2]),          # rows shorter than the taps, one empty
    (3, 5, 7, 3, False, True, True, [1, 7, 9]),      # a length past N is N
    (2, 4, 8, 2, True, False, False, None),          # one vector per row
    (2, 3, 9, 4, True, True, False, [8, -3]),        # one past a vector; a negative length is empty
    (3, 7, 33, 1, True, True, False, [3, 32, 33]),   # one tap: no state
    (2, 6, 257, 4, False, False, True, [255, 256]),
    (2, 2, 2049, 4, True, True, True, None),         # more than one block's vectors per row
    (1, 3, 5001, 3, True, True, False, [4999]),
    (300, 2, 16, 4, True, True, False, None),        # many short rows per channel
]


def _make(io, case, seed):
    B, H, N, W, bias, silu, state, lengths = case
    g = torch.Generator().manual_seed(seed)
    t = DT[io]

    def n(*s, dtype=t):
        return torch.randn(*s, generator=g).to(dtype)

    x = n(B, H, N)
    if lengths is not None:  # nothing past a row's end may be read into a result
        for b, k in enumerate(lengths):
            x[b, :, max(k, 0):] = float("nan")
            if max(k, 0) + 1 < N:
                x[b, :, max(k, 0) + 1] = float("inf")
    return dict(x=x, w=n(H, W, dtype=torch.float32), bias=n(H, dtype=torch.float32) if bias else None,
                x_in=n(B, H, W - 1) if state else None, dy=n(B, H, N), dx_out=n(B, H, W - 1),
                lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32))


def _gpu(d):
    dev = device()
    return {k: v.to(dev) if torch.is_tensor(v) else v for k, v in d.items()}


def _f64(t):
    return None if t is None else t.double()


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "B%d_H%d_N%d_W%d" % c[:4])
def test_short_conv(io, case):
    say("short_conv", io, case)
    d = _make(io, case, 7)
    g = _gpu(d)
    y, xo = pkg.short_conv(g["x"], g["w"], bias=g["bias"], silu=case[5], x_in=g["x_in"], lengths=g["lengths"],
                           return_state=True)
    torch.cuda.synchronize()
    ry, ro = ref.short_conv(_f64(d["x"]), _f64(d["w"]), _f64(d["bias"]), case[5], _f64(d["x_in"]), case[7])
    ref.close(y, ry, io, what="y")
    assert torch.equal(xo.cpu(), ro.to(DT[io])), "saved inputs are copies"


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "B%d_H%d_N%d_W%d" % c[:4])
def test_short_conv_bwd(io, case):
    say("short_conv_bwd", io, case)
    d = _make(io, case, 11)
    if case[7] is not None:
        for b, k in enumerate(case[7]):
            d["dy"][b, :, max(k, 0):] = float("nan")
    g = _gpu(d)
    dx, dw, db, di = pkg.short_conv_bwd(g["x"], g["w"], g["dy"], bias=g["bias"], silu=case[5], x_in=g["x_in"],
                                        lengths=g["lengths"], dx_out=g["dx_out"])
    torch.cuda.synchronize()
    clean = {k: torch.nan_to_num(d[k].double(), 0.0, 0.0, 0.0) for k in ("x", "dy")}
    x, w, b, xi = ref.leaf(clean["x"]), ref.leaf(d["w"]), ref.leaf(d["bias"]), ref.leaf(d["x_in"])
    y, xo = ref.short_conv(x, w, b, case[5], xi, case[7])
    ((y * clean["dy"]).sum() + (xo * d["dx_out"].double()).sum()).backward()
    ref.close(dx, x.grad if x.grad is not None else torch.zeros_like(x), io, what="dx")
    ref.close(dw, w.grad, what="dw")
    if b is not None:
        ref.close(db, b.grad, what="dbias")
    else:
        assert db is None
    if xi is not None:
        ref.close(di, xi.grad, io, what="dx_in")
    else:
        assert di is None


def test_short_conv_bwd_differences():
    """The gradients as directional derivatives of the definition."""
    case = (2, 3, 21, 4, True, True, True, [21, 13])
    d = _make("f32", case, 3)
    d["x"] = torch.nan_to_num(d["x"], 0.0, 0.0, 0.0)
    g = _gpu(d)
    out = pkg.short_conv_bwd(g["x"], g["w"], g["dy"], bias=g["bias"], x_in=g["x_in"], lengths=g["lengths"],
                             dx_out=g["dx_out"])

    def f(a):
        y, xo = ref.short_conv(a["x"], a["w"], a["bias"], True, a["x_in"], case[7])
        return (y * d["dy"].double()).sum() + (xo * d["dx_out"].double()).sum()

    args = {k: d[k].double() for k in ("x", "w", "bias", "x_in")}
    dot, diff, size = ref.directional(f, args, dict(zip(("x", "w", "bias", "x_in"), out)), 5)
    assert abs(dot - diff) <= 1e-5 * size + 1e-7


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,H,P,W", [(1, 1, 1, 4), (5, 33, 9, 4), (4, 300, 4, 2), (3, 17, 6, 3), (2, 5, 2, 1)])
def test_short_conv_step(io, B, H, P, W):
    """Tokens one at a time, in place and into a second pool, with idle rows; a prompt continues."""
    say("short_conv_step", io, B, H, P, W)
    dev = device()
    gen = torch.Generator().manual_seed(1)
    w, bias = torch.randn(H, W, generator=gen), torch.randn(H, generator=gen)
    pool = torch.randn(P, H, W - 1, generator=gen).to(DT[io])
    x = torch.randn(B, H, 5, generator=gen).to(DT[io])
    slots = torch.randperm(P, generator=gen)[:B].to(torch.int32)
    idle = B > 2
    if idle:
        slots[1] = -1 if io == "f16" else P
    busy = [b for b in range(B) if 0 <= int(slots[b]) < P]
    state = pool.to(dev)
    ys = []
    for t in range(5):
        nxt = torch.full_like(state, 7.0)
        a = pkg.short_conv_step(x[:, :, t].contiguous().to(dev), w.to(dev), state, bias=bias.to(dev),
                                slots=slots.to(dev), state_out=nxt)
        before = state.clone()
        b = pkg.short_conv_step(x[:, :, t].contiguous().to(dev), w.to(dev), state, bias=bias.to(dev), slots=slots.to(dev))
        assert torch.equal(a, b)
        used = torch.zeros(P, dtype=torch.bool)
        used[slots[busy].long()] = True
        assert torch.equal(nxt[used.to(dev)], state[used.to(dev)])
        assert bool((nxt[~used.to(dev)] == 7.0).all()) and torch.equal(before[~used.to(dev)], state[~used.to(dev)])
        ys.append(b)
    y = torch.stack(ys, -1).cpu()
    ry, ro = ref.short_conv(x[busy].double(), w.double(), bias.double(), True, pool[slots[busy].long()].double(), None)
    ref.close(y[busy], ry, io, what="y")
    assert torch.equal(state.cpu()[slots[busy].long()], ro.to(DT[io]))
    if idle:
        assert bool((y[1] == 0).all())


def test_short_conv_pieces_join():
    """A row in two pieces joined by the saved inputs is the row in one."""
    dev = device()
    x, w = torch.randn(2, 5, 300).to(dev), torch.randn(5, 4).to(dev)
    y, last = pkg.short_conv(x, w, return_state=True)
    for cut in (1, 2, 3, 128, 299):
        a, s = pkg.short_conv(x[..., :cut].contiguous(), w, return_state=True)
        b, e = pkg.short_conv(x[..., cut:].contiguous(), w, x_in=s, return_state=True)
        assert torch.equal(torch.cat([a, b], -1), y) and torch.equal(e, last)


def test_short_conv_empty():
    dev = device()
    w, s = torch.randn(3, 4).to(dev), torch.randn(2, 3, 3).to(dev)
    y, last = pkg.short_conv(torch.empty(2, 3, 0, device=dev), w, x_in=s, return_state=True)
    assert y.shape == (2, 3, 0) and torch.equal(last, s)
    g = torch.randn(2, 3, 3).to(dev)
    dx, dw, db, di = pkg.short_conv_bwd(torch.empty(2, 3, 0, device=dev), w, torch.empty(2, 3, 0, device=dev), x_in=s,
                                        dx_out=g)
    assert bool((dw == 0).all()) and db is None and torch.equal(di, g)
    dx, dw, db, di = pkg.short_conv_bwd(torch.empty(0, 3, 5, device=dev), w, torch.empty(0, 3, 5, device=dev),
                                        bias=w[:, 0].contiguous())
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_short_conv_same_bits_and_other_stream():
    """Two runs give the same bits, also on a stream of the caller's."""
    dev = device()
    d = _gpu(_make("bf16", (4, 40, 700, 4, True, True, False, None), 2))
    one = pkg.short_conv_bwd(d["x"], d["w"], d["dy"], bias=d["bias"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        two = pkg.short_conv_bwd(d["x"], d["w"], d["dy"], bias=d["bias"])
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(one[:3], two[:3]))


def test_short_conv_refusals():
    dev = device()
    x, w = torch.randn(2, 3, 8).to(dev), torch.randn(3, 4).to(dev)
    with pytest.raises(ValueError):
        pkg.short_conv(x.transpose(1, 2), w)                        # not contiguous
    with pytest.raises(ValueError):
        pkg.short_conv(x, w.half())
    with pytest.raises(ValueError):
        pkg.short_conv(x, torch.randn(4, 4).to(dev))
    with pytest.raises(ValueError):
        pkg.short_conv(x, w, lengths=torch.tensor([1, 2]).to(dev))  # int64
    with pytest.raises(ValueError):
        pkg.short_conv(x, w, x_in=torch.zeros(2, 3, 4).to(dev))
    with pytest.raises(pkg.H3ConvError):
        pkg.short_conv(x, torch.randn(3, 5).to(dev))                # more than MAX_TAPS
    with pytest.raises(pkg.H3ConvError):
        pkg.short_conv(x, w, out=x)                                 # output over input
    with pytest.raises(pkg.H3ConvError):
        pkg.short_conv_step(x[:, :, 0].contiguous(), w, torch.zeros(1, 3, 3).to(dev))  # pool below the batch


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
def test_short_conv_bwd_many_steps(io):
    """Enough steps for two vectors per thread; rows that end inside one, between the two, and before their taps."""
    B, H, N = 4, 160, 2501
    say("short_conv_bwd many steps", io)
    g = torch.Generator().manual_seed(5)
    t, dev = ref.DT[io], device()
    x, dy = torch.randn(B, H, N, generator=g).to(t), torch.randn(B, H, N, generator=g).to(t)
    w, bias = torch.randn(H, 4, generator=g) * 0.5, torch.randn(H, generator=g)
    x_in, dx_out = torch.randn(B, H, 3, generator=g).to(t), torch.randn(B, H, 3, generator=g).to(t)
    lengths = [2501, 2488, 2, 1000]
    got = pkg.short_conv_bwd(x.to(dev), w.to(dev), dy.to(dev), bias.to(dev), x_in=x_in.to(dev),
                             lengths=torch.tensor(lengths, dtype=torch.int32, device=dev), dx_out=dx_out.to(dev))
    torch.cuda.synchronize()
    leaves = [ref.leaf(v) for v in (x, w, bias, x_in)]
    y, xo = ref.short_conv(leaves[0], leaves[1], leaves[2], True, leaves[3], lengths)
    ((y * dy.double()).sum() + (xo * dx_out.double()).sum()).backward()
    for name, a, b, kind in zip(("dx", "dw", "dbias", "dx_in"), got, leaves, (io, "f32", "f32", io)):
        ref.close(a, b.grad, kind, what=name)
