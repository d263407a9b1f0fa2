"""A small language model of linear attention, trained and then run token by token.

    embed -> [block_norm -> q, k, v, decay, gate -> linear_attn -> block_norm (heads, gate) -> projection] x layers
          -> block_norm -> linear_xent

Between two layers one block_norm does the residual sum of the last one and the norm before the next; inside a layer
another does the norm of every head's output and its gate.  Generation runs the prompt once, keeps the states that
linear_attn returns in a pool with one slot per sequence, and goes on with linear_attn_step.  The projections are plain
matrix products; q, k and v are slices of one, which linear_attn takes as they are.

The data are synthetic: every sequence counts up by its own stride modulo the vocabulary.

    python examples/linear_attn_lm.py [--steps 300] [--dtype f32|bf16|f16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fft_long_convolution_flashconv_amd as h3  # noqa: E402


class Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, w, scale):
        ctx.save_for_backward(tokens)
        ctx.rows, ctx.scale = w.shape[0], scale
        return h3.embed(tokens, w, scale)

    @staticmethod
    def backward(ctx, dy):
        return None, h3.embed_bwd(ctx.saved_tensors[0], dy.contiguous(), ctx.rows, ctx.scale), None


class AddNorm(torch.autograd.Function):
    """(r, norm(r) w) of r = f + res; without a res r is f."""

    @staticmethod
    def forward(ctx, f, res, w):
        ctx.save_for_backward(f, res, w)
        return h3.block_norm(f, res=res, w_in=w)

    @staticmethod
    def backward(ctx, dr, dy):
        f, res, w = ctx.saved_tensors
        g = h3.block_norm_bwd(f, dr.contiguous(), dy.contiguous(), res=res, w_in=w)
        return g.df, g.dres, g.dw_in


class GatedNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, f, gate, w, heads):
        ctx.save_for_backward(f, gate, w)
        ctx.heads = heads
        return h3.block_norm(f, gate=gate, w_out=w, groups=heads)

    @staticmethod
    def backward(ctx, dr):
        f, gate, w = ctx.saved_tensors
        g = h3.block_norm_bwd(f, dr.contiguous(), gate=gate, w_out=w, groups=ctx.heads)
        return g.df, g.dgate, g.dw_out, None


class LinearAttn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, scale):
        ctx.save_for_backward(q, k, v, g)
        ctx.scale = scale
        return h3.linear_attn(q, k, v, g, scale)

    @staticmethod
    def backward(ctx, dy):
        q, k, v, g = ctx.saved_tensors
        d = h3.linear_attn_bwd(q, k, v, g, dy.contiguous(), ctx.scale)
        return d.dq, d.dk, d.dv, d.dg, None


class LinearXent(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, labels):
        loss, lse = h3.linear_xent(x, w, labels, return_lse=True)
        ctx.save_for_backward(x, w, labels, lse)
        return loss

    @staticmethod
    def backward(ctx, dloss):
        x, w, labels, lse = ctx.saved_tensors
        return (*h3.linear_xent_bwd(x, w, labels, lse, dloss.contiguous()), None)


class LinearAttnLM(torch.nn.Module):
    """Parameters in fp32; ``dtype`` is that of the activations and of the projections."""

    def __init__(self, vocab=48, width=64, heads=4, layers=2, dtype=torch.float32, seed=0):
        super().__init__()
        gen = torch.Generator().manual_seed(seed)

        def p(*shape, std=1.0):
            return torch.nn.Parameter(torch.randn(*shape, generator=gen) * std)

        self.vocab, self.width, self.heads, self.dtype = vocab, width, heads, dtype
        self.embedding = p(vocab, width, std=0.3)
        self.before = torch.nn.ParameterList(torch.nn.Parameter(torch.ones(width)) for _ in range(layers + 1))
        self.inside = torch.nn.ParameterList(torch.nn.Parameter(torch.ones(width)) for _ in range(layers))
        self.w_in = torch.nn.ParameterList(p(4 * width + heads, width, std=width ** -0.5) for _ in range(layers))
        self.rate = torch.nn.ParameterList(torch.nn.Parameter(torch.linspace(-4.0, 0.0, heads)) for _ in range(layers))
        self.w_out = torch.nn.ParameterList(p(width, width, std=0.5 * width ** -0.5) for _ in range(layers))
        self.head = p(vocab, width, std=width ** -0.5)

    def _c(self, w):
        return w.to(self.dtype)

    def _parts(self, i, y, lead):
        """q, k, v [*lead,H,d] (slices of one projection), the logs of the decays [*lead,H] and the gate, of y [T,width]."""
        D, H = self.width, self.heads
        z = y @ self._c(self.w_in[i]).t()
        q, k, v = (t.view(*lead, H, D // H) for t in z[:, :3 * D].view(*lead, 3 * D).split(D, -1))
        g = -torch.nn.functional.softplus(z[:, 4 * D:].float() + self.rate[i]).view(*lead, H)
        return q, k, v, g.contiguous(), z[:, 3 * D:4 * D].contiguous()

    def _layers(self, tokens, attend):
        """What the head sees, [T,width]; attend(layer, q, k, v, g) is the layers' recurrence."""
        lead, scale = tokens.shape, (self.width // self.heads) ** -0.5
        f, res = Embed.apply(tokens, self._c(self.embedding), self.width ** 0.5).view(-1, self.width), None
        for i in range(len(self.w_out)):
            res, y = AddNorm.apply(f, res, self.before[i])
            q, k, v, g, gate = self._parts(i, y, lead)
            a = attend(i, q, k, v, g, scale)
            f = GatedNorm.apply(a.reshape(-1, self.width), gate, self.inside[i], self.heads) @ self._c(self.w_out[i]).t()
        return AddNorm.apply(f, res, self.before[-1])[1]

    def loss(self, tokens):
        """Mean next-token loss; the last token of a row has no next one."""
        labels = torch.full_like(tokens, -100)
        labels[:, :-1] = tokens[:, 1:]
        x = self._layers(tokens, lambda i, *a: LinearAttn.apply(*a))
        return LinearXent.apply(x, self._c(self.head), labels.reshape(-1)).sum() / (tokens.shape[0] * (tokens.shape[1] - 1))

    @torch.no_grad()
    def prompt(self, tokens, pool, slots):
        """Runs tokens [B,N] and leaves their states in ``slots`` of the pool; the logits [B,vocab] of what follows."""
        def attend(i, q, k, v, g, scale):
            y, state = h3.linear_attn(q, k, v, g, scale, return_state=True)
            pool[i][slots.long()] = state
            return y

        x = self._layers(tokens, attend).view(*tokens.shape, -1)[:, -1]
        return x @ self._c(self.head).t()

    @torch.no_grad()
    def step(self, tokens, pool, slots):
        """One token [B] of each sequence: the logits of the next."""
        x = self._layers(tokens, lambda i, q, k, v, g, scale: h3.linear_attn_step(q, k, v, g, pool[i], scale, slots=slots))
        return x @ self._c(self.head).t()

    def pool(self, size):
        """States of ``size`` sequences."""
        d = self.width // self.heads
        return [torch.zeros(size, self.heads, d, d, device=self.head.device) for _ in self.w_out]


def batch(vocab, B, N, gen, device):
    start, stride = torch.randint(0, vocab, (B, 1), generator=gen), torch.randint(1, 6, (B, 1), generator=gen)
    return ((start + stride * torch.arange(N)) % vocab).to(device)


def train(model, steps, B=32, N=64, lr=3e-3, seed=1, report=None):
    """The loss of every step."""
    gen, dev = torch.Generator().manual_seed(seed), model.head.device
    opt = torch.optim.Adam(model.parameters(), lr=lr)
    losses = []
    for i in range(steps):
        loss = model.loss(batch(model.vocab, B, N, gen, dev))
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
        if report and i % report == 0:
            print("step %4d  loss %.4f" % (i, losses[-1]), flush=True)
    return losses


def generate(model, prompt, count):
    """``count`` tokens after prompt [B,N], the likeliest each time: [B,count]."""
    B, dev = prompt.shape[0], prompt.device
    pool = model.pool(B + 2)
    slots = torch.arange(B, 0, -1, device=dev, dtype=torch.int32)  # (any slots, in any order)
    token = model.prompt(prompt, pool, slots).argmax(1)
    out = [token]
    for _ in range(count - 1):
        token = model.step(token, pool, slots).argmax(1)
        out.append(token)
    return torch.stack(out, 1)


def main():
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--steps", type=int, default=300)
    a.add_argument("--dtype", default="f32", choices=["f32", "f16", "bf16"])
    a = a.parse_args()
    dev = torch.device("cuda:0")
    model = LinearAttnLM(dtype={"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[a.dtype]).to(dev)
    losses = train(model, a.steps, report=50)
    print("last loss %.4f (uniform: %.4f)" % (losses[-1], torch.log(torch.tensor(float(model.vocab)))))
    whole = batch(model.vocab, 8, 40, torch.Generator().manual_seed(9), dev)
    got = generate(model, whole[:, :16].contiguous(), 24)
    print("generated after a prompt of 16, right: %.1f %%" % (100.0 * (got == whole[:, 16:]).float().mean()))
    print("  prompt end", whole[0, 10:16].tolist(), "->", got[0, :8].tolist())


if __name__ == "__main__":
    main()
