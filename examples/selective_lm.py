"""A small language model of one selective state-space layer, trained and then run token by token.

    embedding -> in-projection -> short_conv (SiLU) -> selective_scan (gated) -> out-projection -> linear_xent

Training uses short_conv, selective_scan and linear_xent with their backward passes; generation runs the prompt
once, keeps the states that short_conv and selective_scan return in a pool with one slot per sequence, and goes on
with short_conv_step and selective_step.  The projections are plain matrix products.

The data are synthetic: every sequence counts up by its own stride modulo the vocabulary, so that the next token
follows from the two before it.

    python examples/selective_lm.py [--steps 300] [--dtype f32|bf16|f16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fft_long_convolution_flashconv_amd as h3  # noqa: E402

TAPS, MODES, RANK = 4, 16, 8


class ShortConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias):
        ctx.save_for_backward(x, w, bias)
        return h3.short_conv(x, w, bias)

    @staticmethod
    def backward(ctx, dy):
        x, w, bias = ctx.saved_tensors
        return h3.short_conv_bwd(x, w, dy.contiguous(), bias)[:3]


class SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, dt, A, Bm, C, D, z, dt_bias):
        y, saved = h3.selective_scan(u, dt, A, Bm, C, D, z, dt_bias, return_saved=True)
        ctx.save_for_backward(u, dt, A, Bm, C, D, z, dt_bias, saved)
        return y

    @staticmethod
    def backward(ctx, dy):
        u, dt, A, Bm, C, D, z, dt_bias, saved = ctx.saved_tensors
        g = h3.selective_scan_bwd(u, dt, A, Bm, C, dy.contiguous(), saved, D, z, dt_bias)
        return g.du, g.ddt, g.dA, g.dB, g.dC, g.dD, g.dz, g.ddt_bias


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


def rows(w, x):
    """w [M,K] on the channels of x [B,K,N]: [B,M,N]."""
    B, K, N = x.shape
    return (w @ x.permute(1, 0, 2).reshape(K, B * N)).view(w.shape[0], B, N).permute(1, 0, 2).contiguous()


class SelectiveLM(torch.nn.Module):
    """Parameters in fp32; ``dtype`` is that of the activations and of the projections."""

    def __init__(self, vocab=48, width=48, channels=96, dtype=torch.float32, seed=0):
        super().__init__()
        g = torch.Generator().manual_seed(seed)

        def p(*shape, std=1.0):
            return torch.nn.Parameter(torch.randn(*shape, generator=g) * std)

        self.vocab, self.dtype = vocab, dtype
        self.embed = p(vocab, width)
        self.w_in = p(2 * channels, width, std=width ** -0.5)
        self.taps, self.tap_bias = p(channels, TAPS, std=TAPS ** -0.5), p(channels, std=0.0)
        self.w_dbc = p(RANK + 2 * MODES, channels, std=channels ** -0.5)
        self.w_dt = p(channels, RANK, std=RANK ** -0.5)
        self.dt_bias = torch.nn.Parameter(torch.linspace(-4.0, -1.0, channels))
        self.log_A = torch.nn.Parameter(torch.log(torch.arange(1, MODES + 1).float()).repeat(channels, 1))
        self.D = torch.nn.Parameter(torch.ones(channels))
        self.w_out = p(width, channels, std=channels ** -0.5)
        self.head = p(vocab, width, std=width ** -0.5)

    def _c(self, w):
        return w.to(self.dtype)

    def _scan_inputs(self, u):
        """dt [B,H,N], B and C [B,1,S,N] from the scan's input."""
        dbc = rows(self._c(self.w_dbc), u)
        dt = rows(self._c(self.w_dt), dbc[:, :RANK].contiguous())
        Bm, C = dbc[:, None, RANK:RANK + MODES].contiguous(), dbc[:, None, RANK + MODES:].contiguous()
        return dt, Bm, C

    def hidden(self, tokens):
        """What the head sees, [B*N, width], of tokens [B,N]."""
        e = self._c(self.embed[tokens]).permute(0, 2, 1).contiguous()
        x, z = (t.contiguous() for t in rows(self._c(self.w_in), e).chunk(2, dim=1))
        u = ShortConv.apply(x, self.taps, self.tap_bias)
        dt, Bm, C = self._scan_inputs(u)
        y = SelectiveScan.apply(u, dt, -torch.exp(self.log_A), Bm, C, self.D, z, self.dt_bias)
        h = e + rows(self._c(self.w_out), y)
        return h.permute(0, 2, 1).reshape(-1, e.shape[1]).contiguous()

    def loss(self, tokens):
        """Mean next-token loss; the last token of a row has no next one."""
        labels = torch.full_like(tokens, -100)
        labels[:, :-1] = tokens[:, 1:]
        per_token = LinearXent.apply(self.hidden(tokens), self._c(self.head), labels.reshape(-1))
        return per_token.sum() / (tokens.shape[0] * (tokens.shape[1] - 1))

    @torch.no_grad()
    def prompt(self, tokens, pool, slots):
        """Runs tokens [B,N] and leaves their states in ``slots`` of the pool; the logits [B,vocab] of what follows."""
        e = self._c(self.embed[tokens]).permute(0, 2, 1).contiguous()
        x, z = (t.contiguous() for t in rows(self._c(self.w_in), e).chunk(2, dim=1))
        u, last = h3.short_conv(x, self.taps, self.tap_bias, return_state=True)
        dt, Bm, C = self._scan_inputs(u)
        y, state = h3.selective_scan(u, dt, -torch.exp(self.log_A), Bm, C, self.D, z, self.dt_bias, return_state=True)
        pool["conv"][slots.long()], pool["scan"][slots.long()] = last, state
        h = (e + rows(self._c(self.w_out), y))[:, :, -1]
        return h @ self._c(self.head).t()

    @torch.no_grad()
    def step(self, tokens, pool, slots):
        """One token [B] of each sequence: the logits of the next."""
        e = self._c(self.embed[tokens])
        x, z = (t.contiguous() for t in (e @ self._c(self.w_in).t()).chunk(2, dim=1))
        u = h3.short_conv_step(x, self.taps, pool["conv"], self.tap_bias, slots=slots)
        dbc = u @ self._c(self.w_dbc).t()
        dt = dbc[:, :RANK].contiguous() @ self._c(self.w_dt).t()
        Bm, C = dbc[:, None, RANK:RANK + MODES].contiguous(), dbc[:, None, RANK + MODES:].contiguous()
        y = h3.selective_step(u, dt, -torch.exp(self.log_A), Bm, C, pool["scan"], self.D, z, self.dt_bias, slots=slots)
        return (e + y @ self._c(self.w_out).t()) @ self._c(self.head).t()

    def pool(self, size):
        """States of ``size`` sequences."""
        channels, dev = self.taps.shape[0], self.taps.device
        return {"conv": torch.zeros(size, channels, TAPS - 1, device=dev, dtype=self.dtype),
                "scan": torch.zeros(size, channels, MODES, device=dev)}


def batch(vocab, B, N, gen, device):
    start, stride = torch.randint(0, vocab, (B, 1), generator=gen), torch.randint(1, 6, (B, 1), generator=gen)
    return ((start + stride * torch.arange(N)) % vocab).to(device)


def train(model, steps, B=32, N=64, lr=3e-3, seed=1, report=None):
    """The loss of every step."""
    gen, dev = torch.Generator().manual_seed(seed), model.taps.device
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
    model = SelectiveLM(dtype={"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[a.dtype]).to(dev)
    losses = train(model, a.steps, report=50)
    print("last loss %.4f (uniform: %.4f)" % (losses[-1], torch.log(torch.tensor(float(model.vocab)))))
    whole = batch(model.vocab, 8, 40, torch.Generator().manual_seed(9), dev)
    got = generate(model, whole[:, :16].contiguous(), 24)
    print("generated after a prompt of 16, right: %.1f %%" % (100.0 * (got == whole[:, 16:]).float().mean()))
    print("  prompt end", whole[0, 10:16].tolist(), "->", got[0, :8].tolist())


if __name__ == "__main__":
    main()
