"""Tensors of more than 2^32 elements or bytes through linear attention, the norms and the embedding: their ends are
compared with what the same rows give in tensors of their own."""
import pytest
import torch

import fft_long_convolution_flashconv_amd as pkg
import layer_reference as lref
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


def _normal(*shape):
    """bf16, filled in slices (the generator's own temporaries stay small)."""
    t = torch.empty(*shape, dtype=torch.bfloat16, device=device())
    for part in t.view(-1).split(1 << 28):
        part.normal_()
    return t


@pytest.mark.parametrize("H,d", [(8, 16), (9, 15)])
def test_attention_over_a_long_row(room, H, d):
    """2^25 + 37 steps, 2^32 elements and more: the decays leave nothing of a step after 300 others."""
    say("attention over a long row", H, d)
    room(90)
    N, tail = (1 << 25) + 37, 1000
    q, k, v, dy = (_normal(1, N, H, d) for _ in range(4))
    g = torch.full((H,), -0.5, device=device())
    y, x = pkg.linear_attn(q, k, v, g, 0.3, return_state=True)
    last = [t[:, -tail:].contiguous() for t in (q, k, v, dy)]
    y1, x1 = pkg.linear_attn(*last[:3], g, 0.3, return_state=True)
    ref.close(y[:, -tail + 300:], y1[:, 300:].double().cpu(), "bf16", roundings=2, what="y")
    ref.close(x, x1.double().cpu(), what="x")
    first = [t[:, :tail].contiguous() for t in (q, k, v, dy)]
    ref.close(y[:, :tail], pkg.linear_attn(*first[:3], g, 0.3).double().cpu(), "bf16", roundings=2, what="first y")
    del y, x
    o, o1, o0 = (pkg.linear_attn_bwd(*t[:3], g, t[3], 0.3) for t in ((q, k, v, dy), last, first))
    for name in ("dq", "dk", "dv"):
        ref.close(getattr(o, name)[:, -tail + 300:], getattr(o1, name)[:, 300:].double().cpu(), "bf16", roundings=2, what=name)
        ref.close(getattr(o, name)[:, :tail - 300], getattr(o0, name)[:, :tail - 300].double().cpu(), "bf16", roundings=2,
                  what="first " + name)


def test_steps_in_a_large_pool(room):
    """A pool of 2^32 elements and more: its last slots."""
    say("steps in a large pool")
    room(40)
    P, H, d, B = (1 << 16) + 3, 1, 256, 4
    pool = torch.zeros(P, H, d, d, device=device())
    slots = torch.tensor([P - 1, 0, 1 << 15, P - 2], dtype=torch.int32, device=device())
    q, k, v = (_normal(B, H, d) for _ in range(3))
    g = torch.full((H,), -0.1, device=device())
    small = pool[:B].clone()
    for _ in range(2):
        y, y1 = pkg.linear_attn_step(q, k, v, g, pool, 0.1, slots=slots), pkg.linear_attn_step(q, k, v, g, small, 0.1)
        assert torch.equal(y, y1)
    assert torch.equal(pool[slots.long()], small) and not pool[P - 3].any() and not pool[1].any()


@pytest.mark.parametrize("D", [2560, 1031])
def test_norm_over_many_rows(room, D):
    say("norm over many rows", D)
    room(90)
    T = (1 << 32) // D + 3
    f, dy = _normal(T, D), _normal(T, D)
    w = torch.randn(D, device=device())
    r, y = pkg.block_norm(f, w_in=w)
    o = pkg.block_norm_bwd(f, None, dy, w_in=w)
    for at in (slice(0, 3), slice(T - 3, T)):
        r1, y1 = pkg.block_norm(f[at], w_in=w)
        o1 = pkg.block_norm_bwd(f[at], None, dy[at], w_in=w)
        assert torch.equal(r[at], r1) and torch.equal(y[at], y1) and torch.equal(o.df[at], o1.df)
    # dw_in = sum over T of dy rh, in slices and 64 bits
    want = torch.zeros(D, dtype=torch.float64, device=device())
    for a, b in zip(f.split(1 << 16), dy.split(1 << 16)):
        x = a.double()
        want += (b.double() * x / (x.square().mean(1, keepdim=True) + 1e-5).sqrt()).sum(0)
    # sums of up to 2^22 terms of size 1, in 2^10 parts of 2^12: a part is 2^6 large, its roundings of 2^-19 (on average)
    # come to 2^-13, all parts' to 2^-8, and joining them adds as much: 2^-7 of a sum of 2^11, 4e-6
    assert (o.dw_in.double() - want).norm() <= 1e-5 * want.norm()


def test_embedding_of_many_tokens(room):
    """2^26 + 5 tokens of 64 channels: 2^32 elements and more each way."""
    say("embedding of many tokens")
    room(60)
    T, D, V = (1 << 26) + 5, 64, 1000
    tok = torch.randint(0, V, (T,), device=device())
    w = _normal(V, D)
    y = pkg.embed(tok, w, 2.0)
    for at in (slice(0, 100), slice(T - 100, T)):
        assert torch.equal(y[at], (w[tok[at]].float() * 2.0).to(torch.bfloat16))
    y.view(-1)[:].zero_()
    y[-7:] = 1.0  # (only the last rows count, so that the sums are whole numbers)
    y[:5] = 3.0
    dw = pkg.embed_bwd(tok, y, V, 2.0)
    want = torch.zeros(V, device=device())
    want.index_add_(0, tok[-7:], torch.full((7,), 2.0, device=device())).index_add_(0, tok[:5], torch.full((5,), 6.0, device=device()))
    assert torch.equal(dw, want[:, None].expand(V, D).to(torch.bfloat16))
