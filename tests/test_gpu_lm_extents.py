"""Sizes inside the documented ranges whose kernels need 2^32 threads and more (what one dispatch takes along x is less).

Every result is compared where it is cheap to: with closed forms on the GPU (one step per row), or with the 64-bit
definitions on the first and the last rows.
"""
import pytest
import torch

import fft_long_convolution_flashconv_amd as pkg
import lm_reference as ref
from parity_util import device, say

pytestmark = pytest.mark.gpu


@pytest.fixture
def room():
    """Skips where the card has less free memory than the case needs, and frees what it used."""
    def need(gib):
        torch.cuda.empty_cache()
        if torch.cuda.mem_get_info()[0] < gib * 2 ** 30:
            pytest.skip("needs %d GiB of free GPU memory" % gib)
    yield need
    torch.cuda.empty_cache()


def _close(got, want, io, what):
    """As lm_reference.close, on the GPU, in slices."""
    half = ref.HALF_ULP[io]
    err = norm = 0.0
    for g, w in zip(got.reshape(-1).split(1 << 26), want.reshape(-1).split(1 << 26)):
        assert bool(torch.isfinite(g).all()), what
        err += float((g.double() - w.double()).square().sum())
        norm += float(w.double().square().sum())
    slack = (2.0 ** -25 if io == "f16" else 1e-30) * got.numel() ** 0.5
    assert err ** 0.5 <= (1e-5 + half) * norm ** 0.5 + slack, (what, err ** 0.5, norm ** 0.5)


def test_short_conv_rows(room):
    """2^24 + 3 rows of 1025 steps: a block each."""
    room(80)
    H, N = (1 << 24) + 3, 1025
    say("short_conv", H, N)
    g = torch.Generator(device=device()).manual_seed(1)
    x = torch.empty(1, H, N, device=device(), dtype=torch.float16)
    for part in x[0].split(1 << 21):
        part.copy_(torch.randn(part.shape, generator=g, device=device(), dtype=torch.float16))
    w = torch.randn(H, 4, generator=g, device=device())
    y, last = pkg.short_conv(x, w, return_state=True)
    assert torch.equal(last, x[..., N - 3:])
    for at in (slice(0, 2), slice((1 << 24) - 2, (1 << 24) + 3)):
        want, _ = ref.short_conv(x[:, at].double().cpu(), w[at].double().cpu(), None, True, None, None)
        ref.close(y[:, at], want, "f16", what=str(at))


def test_short_conv_bwd_channels(room):
    """2^24 + 3 channels of one step."""
    room(4)
    H = (1 << 24) + 3
    say("short_conv_bwd", H)
    dev = device()
    g = torch.Generator(device=dev).manual_seed(2)
    x, dy = (torch.randn(1, H, 1, generator=g, device=dev) for _ in range(2))
    w, b = torch.randn(H, 2, generator=g, device=dev), torch.randn(H, generator=g, device=dev)
    dx, dw, db, _ = pkg.short_conv_bwd(x, w, dy, bias=b)
    p = w[:, 0].double() * x[0, :, 0].double() + b.double()
    s = torch.sigmoid(p)
    dp = dy[0, :, 0].double() * (s + p * s * (1 - s))
    _close(dx[0, :, 0], dp * w[:, 0], "f32", "dx")
    _close(dw[:, 0], dp * x[0, :, 0], "f32", "dw")
    _close(db, dp, "f32", "dbias")
    assert not dw[:, 1].any()


def test_selective_scan_rows(room):
    """2^28 + 5 rows of one step."""
    room(30)
    H = (1 << 28) + 5
    say("selective_scan", H)
    dev = device()
    g = torch.Generator(device=dev).manual_seed(3)
    u, dt = (torch.randn(1, H, 1, generator=g, device=dev, dtype=torch.float16) for _ in range(2))
    A = torch.full((H, 1), -1.0, device=dev)
    Bm, C = (torch.full((1, 1, 1, 1), v, device=dev, dtype=torch.float16) for v in (0.5, 2.0))
    y = pkg.selective_scan(u, dt, A, Bm, C)
    del A
    want = torch.nn.functional.softplus(dt.float()) * u.float()
    _close(y, want, "f16", "y")


def test_selective_scan_bwd_groups(room):
    """2^23 + 9 channels, each a group of its own, of one step."""
    room(8)
    H = (1 << 23) + 9
    say("selective_scan_bwd", H)
    dev = device()
    g = torch.Generator(device=dev).manual_seed(4)

    def r(*s):
        return torch.randn(*s, generator=g, device=dev)

    u, dt, z, dy = r(1, H, 1), r(1, H, 1), r(1, H, 1), r(1, H, 1)
    A, Bm, C, D, x_in = -r(H, 1).abs(), r(1, H, 1, 1), r(1, H, 1, 1), r(H), r(1, H, 1)
    y, saved = pkg.selective_scan(u, dt, A, Bm, C, D, z, x_in=x_in, return_saved=True)
    o = pkg.selective_scan_bwd(u, dt, A, Bm, C, dy, saved, D, z)
    leaves = [t.double().reshape(H).requires_grad_(True) for t in (u, dt, A, Bm, C, D, z, x_in)]
    lu, ld, lA, lB, lC, lD, lz, lx = leaves
    d = torch.nn.functional.softplus(ld, threshold=1e9)
    raw = lC * (torch.exp(d * lA) * lx + d * lu * lB) + lD * lu
    want = raw * lz * torch.sigmoid(lz)
    want.backward(dy.double().reshape(H))
    _close(y, want.detach(), "f32", "y")
    for name, got, leaf in zip(("du", "ddt", "dA", "dB", "dC", "dD", "dz", "dx_in"),
                               (o.du, o.ddt, o.dA, o.dB, o.dC, o.dD, o.dz, o.dx_in), leaves):
        _close(got, leaf.grad, "f32", name)


def test_selective_scan_bwd_joins(room):
    """B and C of 2^32 + 2^17 values."""
    room(110)
    B, N, S = (1 << 16) + 2, 1024, 64
    say("selective_scan_bwd", B, N, S)
    dev = device()
    g = torch.Generator(device=dev).manual_seed(5)

    def r(*s):
        t = torch.empty(*s, device=dev, dtype=torch.float16)
        for part in t.split(1 << 12):
            part.copy_(torch.randn(part.shape, generator=g, device=dev, dtype=torch.float16))
        return t

    u, dt, dy, Bm, C = r(B, 1, N), r(B, 1, N), r(B, 1, N), r(B, 1, S, N), r(B, 1, S, N)
    A = -torch.arange(1, S + 1, device=dev).float()[None].contiguous()
    bias = torch.tensor([-3.0], device=dev)
    y, saved = pkg.selective_scan(u, dt, A, Bm, C, dt_bias=bias, return_saved=True)
    o = pkg.selective_scan_bwd(u, dt, A, Bm, C, dy, saved, dt_bias=bias)
    for b in (0, B - 1):
        at = slice(b, b + 1)
        leaves = [ref.leaf(t) for t in (u[at], dt[at], Bm[at], C[at])]
        want, _ = ref.selective_scan(leaves[0], leaves[1], A.double().cpu(), leaves[2], leaves[3], None, None,
                                     bias.double().cpu(), True, None, None)
        (want * dy[at].double().cpu()).sum().backward()
        ref.close(y[at], want, "f16", what="y %d" % b)
        for name, got, leaf in zip(("du", "ddt", "dB", "dC"), (o.du, o.ddt, o.dB, o.dC), leaves):
            ref.close(got[at], leaf.grad, "f16", what="%s %d" % (name, b))


def _lse(x, w, t):
    return torch.logsumexp(w.double() @ x[t].double(), 0)


def test_xent_tiles(room):
    """fp32, 513 x 32769 tiles of logits."""
    room(24)
    T, D, V = (1 << 15) + 1, 4, (1 << 21) + 1
    say("linear_xent tiles", T, D, V)
    dev = device()
    g = torch.Generator(device=dev).manual_seed(6)
    x, w = torch.randn(T, D, generator=g, device=dev), torch.randn(V, D, generator=g, device=dev)
    labels = torch.randint(0, V, (T,), generator=g, device=dev)
    labels[-1] = V - 1
    loss, lse = pkg.linear_xent(x, w, labels, return_lse=True)
    for t in (0, 1, T // 2, T - 2, T - 1):
        want = float(_lse(x, w, t))
        hit = float(w[labels[t]].double() @ x[t].double())
        # fp32 logits of four products, up to about 25 in magnitude
        assert abs(float(lse[t]) - want) <= 1e-4 and abs(float(loss[t]) - (want - hit)) <= 2e-4, t


def test_xent_tokens(room):
    """2^28 + 7 tokens of a vocabulary of two."""
    room(30)
    T = (1 << 28) + 7
    say("linear_xent tokens", T)
    dev = device()
    g = torch.Generator(device=dev).manual_seed(7)
    x = torch.randn(T, 1, generator=g, device=dev)
    w = torch.tensor([[1.0], [-0.5]], device=dev)
    loss = pkg.linear_xent(x, w, torch.ones(T, device=dev, dtype=torch.int64))
    _close(loss, torch.nn.functional.softplus(1.5 * x[:, 0]), "f32", "loss")


def test_xent_no_tokens(room):
    """dw of no tokens, 2^32 values."""
    room(40)
    V, D = 1 << 22, 1024
    say("linear_xent_bwd no tokens", V, D)
    dev = device()
    none = torch.empty(0, device=dev)
    torch.full((V, D), 7.0, device=dev, dtype=torch.bfloat16)  # (the memory that dw may get)
    _, dw = pkg.linear_xent_bwd(torch.empty(0, D, device=dev, dtype=torch.bfloat16),
                                torch.zeros(V, D, device=dev, dtype=torch.bfloat16),
                                torch.empty(0, device=dev, dtype=torch.int64), none, none)
    assert not any(bool(part.any()) for part in dw.split(1 << 18))


def test_selective_step_channels(room):
    """2^28 + 3 channels of 33 modes, sixteen threads each."""
    room(90)
    H, S = (1 << 28) + 3, 33
    say("selective_step", H, S)
    dev = device()
    g = torch.Generator(device=dev).manual_seed(8)
    u, dt = (torch.randn(1, H, generator=g, device=dev, dtype=torch.float16) for _ in range(2))
    A, x = torch.full((H, S), -1.0, device=dev), torch.ones(1, H, S, device=dev)
    Bm, C = (torch.full((1, 1, S), v, device=dev, dtype=torch.float16) for v in (0.5, 0.25))
    y = pkg.selective_step(u, dt, A, Bm, C, x)
    del A
    d = torch.nn.functional.softplus(dt.float())
    state = torch.exp(-d) + 0.5 * d * u.float()
    _close(y, S * 0.25 * state, "f16", "y")
    for j in (0, S - 1):
        _close(x[0, :, j].contiguous(), state[0], "f32", "state %d" % j)


def test_xent_padding(room):
    """A padded copy of w of 2^36 bytes: 2^22 rows of 8129 elements."""
    room(160)
    V, D = 1 << 22, 8129
    say("linear_xent padding", V, D)
    dev = device()
    x = torch.ones(1, D, device=dev, dtype=torch.bfloat16)
    w = torch.zeros(V, D, device=dev, dtype=torch.bfloat16)
    w[0, 0], w[V // 2, D - 1], w[V - 1, D - 1] = 10.0, 11.0, 12.0  # logits 10, 11, 12 and zeros
    for label, logit in ((V - 1, 12.0), (V // 2, 11.0), (0, 10.0), (5, 0.0)):
        loss, lse = pkg.linear_xent(x, w, torch.tensor([label], device=dev), return_lse=True)
        want = float(torch.tensor([V - 3.0]).double().add(torch.tensor([10.0, 11.0, 12.0]).double().exp().sum()).log())
        # fp32 sums of 2^22 equal terms in pairs, a logarithm of about 15
        assert abs(float(lse) - want) <= 1e-4 and abs(float(loss) - (want - logit)) <= 1e-4, label
