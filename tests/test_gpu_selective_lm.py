"""examples/selective_lm.py: training lowers the loss, and tokens one by one give what the whole row gives."""
import importlib.util
import os

import pytest
import torch

import lm_reference as ref
from parity_util import device, say

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "selective_lm.py")
    spec = importlib.util.spec_from_file_location("selective_lm", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
def test_training_lowers_the_loss(io):
    say("selective_lm train", io)
    ex = _example()
    model = ex.SelectiveLM(dtype=ref.DT[io]).to(device())
    losses = ex.train(model, 60)
    assert all(l == l for l in losses)
    assert sum(losses[-5:]) / 5 < 0.6 * sum(losses[:5]) / 5, losses


def test_steps_follow_the_prompt():
    """Logits of a row's last tokens: by steps after a prompt, and by longer prompts."""
    say("selective_lm steps")
    ex = _example()
    dev = device()
    model = ex.SelectiveLM().to(dev)
    tokens = ex.batch(model.vocab, 3, 40, torch.Generator().manual_seed(2), dev)
    pool = model.pool(5)
    slots = torch.tensor([4, 0, 2], device=dev, dtype=torch.int32)
    got = [model.prompt(tokens[:, :33].contiguous(), pool, slots)]
    for t in range(33, 40):
        got.append(model.step(tokens[:, t].contiguous(), pool, slots))
    for n, g in zip(range(33, 41), got):
        want = model.prompt(tokens[:, :n].contiguous(), model.pool(5), slots)
        # fp32 states and sums over at most 96 terms on both sides
        assert (g - want).abs().max() <= 1e-4 * (1.0 + want.abs().max()), n
    assert not pool["scan"][1].any() and not pool["scan"][3].any()


def test_gradients_against_plain_operators():
    """The model's gradients, its three operators replaced by their 64-bit definitions."""
    say("selective_lm gradients")
    ex = _example()
    model = ex.SelectiveLM(vocab=11, width=6, channels=8).to(device())
    tokens = ex.batch(11, 2, 20, torch.Generator().manual_seed(3), device())
    model.loss(tokens).backward()
    plain = ex.SelectiveLM(vocab=11, width=6, channels=8, dtype=torch.float64).double()
    p, t = plain, tokens.cpu()
    e = p.embed[t].permute(0, 2, 1)
    x, z = ex.rows(p.w_in, e).chunk(2, dim=1)
    u = ref.short_conv(x, p.taps, p.tap_bias, True, None, None)[0]
    dt, Bm, C = p._scan_inputs(u)
    y = ref.selective_scan(u, dt, -torch.exp(p.log_A), Bm, C, p.D, z, p.dt_bias, True, None, None)[0]
    h = (e + ex.rows(p.w_out, y)).permute(0, 2, 1)
    logits = h[:, :-1] @ p.head.t()
    torch.nn.functional.cross_entropy(logits.reshape(-1, 11), t[:, 1:].reshape(-1)).backward()
    for (name, a), (_, b) in zip(model.named_parameters(), plain.named_parameters()):
        # fp32 throughout, a few hundred operations deep
        err, norm = (a.grad.double().cpu() - b.grad).norm(), b.grad.norm()
        assert err <= 1e-4 * norm + 1e-7, (name, float(err), float(norm))


def test_token_steps_in_a_graph():
    """short_conv_step and selective_step captured once and replayed token by token, against eager calls."""
    say("token steps in a graph")
    ex = _example()
    h3, dev = ex.h3, device()
    g = torch.Generator().manual_seed(4)

    def r(*s):
        return torch.randn(*s, generator=g).to(dev)

    B, H, S, P = 6, 40, 16, 9
    w, bias, A, D = r(H, 4), r(H), -r(H, S).abs(), r(H)
    x, z, dt, Bm, C = r(B, H), r(B, H), r(B, H), r(B, 1, S), r(B, 1, S)
    slots = torch.tensor([8, 2, -1, 0, 5, 3], dtype=torch.int32, device=dev)
    pools = [(torch.zeros(P, H, 3, device=dev), torch.zeros(P, H, S, device=dev)) for _ in range(2)]

    def token(pool):
        u = h3.short_conv_step(x, w, pool[0], bias, slots=slots)
        return h3.selective_step(u, dt, A, Bm, C, pool[1], D, z, slots=slots)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        token(tuple(t.clone() for t in pools[0]))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = token(pools[0])
    for t in pools[0]:
        t.zero_()
    for i in range(5):
        for t in (x, z, dt, Bm, C):
            t.copy_(r(*t.shape))
        graph.replay()
        want = token(pools[1])
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
        assert torch.equal(pools[0][0], pools[1][0]) and torch.equal(pools[0][1], pools[1][1]), i
