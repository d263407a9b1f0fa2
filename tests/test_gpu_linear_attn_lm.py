"""The embedding, the norms around a block, linear attention and the loss together, as examples/linear_attn_lm.py uses
them: gradients against plain operators, steps against the prompt, a captured token."""
import importlib.util
import os

import pytest
import torch

import layer_reference as lref
import lm_reference as ref
from parity_util import device, say

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "linear_attn_lm.py")
    spec = importlib.util.spec_from_file_location("linear_attn_lm", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
def test_training_runs(io):
    """Steps of training in every type: finite losses, and parameters that all have gradients."""
    say("linear_attn_lm train", io)
    ex = _example()
    model = ex.LinearAttnLM(dtype=ref.DT[io]).to(device())
    losses = ex.train(model, 5, B=4)
    assert all(l == l and abs(l) < 100 for l in losses)
    for name, p in model.named_parameters():
        assert p.grad is not None and bool(torch.isfinite(p.grad).all()) and bool(p.grad.any()), name


def _plain_loss(p, tokens):
    """The model with its operators replaced by their 64-bit definitions."""
    B, N = tokens.shape
    D, H = p.width, p.heads
    f, res = lref.embed(tokens, p.embedding, D ** 0.5).view(-1, D), None
    for i in range(len(p.w_out)):
        res, y = lref.block_norm(f, res=res, w_in=p.before[i])
        q, k, v, g, gate = p._parts_plain(i, y, (B, N))
        a = lref.linear_attn(q, k, v, g, (D // H) ** -0.5)[0]
        f = lref.block_norm(a.reshape(-1, D), gate=gate, w_out=p.inside[i], groups=H)[0] @ p.w_out[i].t()
    x = lref.block_norm(f, res=res, w_in=p.before[-1])[1].view(B, N, D)
    return torch.nn.functional.cross_entropy((x[:, :-1] @ p.head.t()).reshape(-1, p.vocab), tokens[:, 1:].reshape(-1))


def test_gradients_against_plain_operators():
    say("linear_attn_lm gradients")
    ex = _example()
    model = ex.LinearAttnLM(vocab=11, width=16, heads=2, layers=2).to(device())
    tokens = ex.batch(11, 2, 70, torch.Generator().manual_seed(3), device())
    loss = model.loss(tokens)
    loss.backward()

    class Plain(ex.LinearAttnLM):
        def _parts_plain(self, i, y, lead):
            D, H = self.width, self.heads
            z = y @ self.w_in[i].t()
            q, k, v = (t.reshape(*lead, H, D // H) for t in z[:, :3 * D].split(D, 1))
            g = -torch.nn.functional.softplus(z[:, 4 * D:] + self.rate[i]).view(*lead, H)
            return q, k, v, g, z[:, 3 * D:4 * D]

    plain = Plain(vocab=11, width=16, heads=2, layers=2, dtype=torch.float64).double()
    want = _plain_loss(plain, tokens.cpu())
    want.backward()
    assert abs(loss.item() - want.item()) <= 1e-5 * abs(want.item())
    for (name, a), (_, b) in zip(model.named_parameters(), plain.named_parameters()):
        # fp32 throughout, a few hundred operations deep
        err, norm = (a.grad.double().cpu() - b.grad).norm(), b.grad.norm()
        assert err <= 1e-4 * norm + 1e-7, (name, float(err), float(norm))


def test_steps_follow_the_prompt():
    """Logits of a row's last tokens: by steps after a prompt, and by longer prompts."""
    say("linear_attn_lm steps")
    ex = _example()
    dev = device()
    model = ex.LinearAttnLM().to(dev)
    tokens = ex.batch(model.vocab, 3, 76, torch.Generator().manual_seed(2), dev)
    pool = model.pool(5)
    slots = torch.tensor([4, 0, 2], device=dev, dtype=torch.int32)
    got = [model.prompt(tokens[:, :70].contiguous(), pool, slots)]
    for t in range(70, 76):
        got.append(model.step(tokens[:, t].contiguous(), pool, slots))
    for n, g in zip(range(70, 77), got):
        want = model.prompt(tokens[:, :n].contiguous(), model.pool(5), slots)
        # fp32 states and sums over at most 260 terms on both sides, two layers deep
        assert (g - want).abs().max() <= 1e-4 * (1.0 + want.abs().max()), n
    assert all(not p[1].any() and not p[3].any() for p in pool)


def test_a_token_in_a_graph():
    """The library's calls of one token captured once and replayed, against eager calls."""
    say("a token in a graph")
    ex = _example()
    h3, dev = ex.h3, device()
    gen = torch.Generator().manual_seed(4)

    def r(*s):
        return torch.randn(*s, generator=gen).to(dev)

    B, H, d, P, V = 6, 4, 16, 9, 40
    D = H * d
    tokens = torch.randint(0, V, (B,), generator=gen).to(dev)
    table, w, res, gate, g = r(V, D), r(D), r(B, D), r(B, D), -r(B, H).abs()
    slots = torch.tensor([8, 2, -1, 0, 5, 3], dtype=torch.int32, device=dev)
    pools = [torch.zeros(P, H, d, d, device=dev) for _ in range(2)]

    def token(pool):
        e = h3.embed(tokens, table, 2.0)
        x, y = h3.block_norm(e, res=res, w_in=w)
        q = y.view(B, H, d)
        a = h3.linear_attn_step(q, q, x.view(B, H, d), g, pool, slots=slots)
        return h3.block_norm(a.view(B, D), gate=gate, w_out=w, groups=H)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        token(pools[0].clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token(pools[0])
    pools[0].zero_()
    for i in range(5):
        for t in (res, gate):
            t.copy_(r(*t.shape))
        tokens.copy_(torch.randint(0, V, (B,), generator=gen).to(dev))
        graph.replay()
        want = token(pools[1])
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(pools[0], pools[1]), i
