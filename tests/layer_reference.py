"""Plain 64-bit definitions of linear attention, the norms around a block and the
embedding (torch float64 on the CPU), which the GPU tests compare against;
gradients come from automatic differentiation of these definitions.

Tolerances are those of lm_reference: a result held in fp32 is within 1e-5 (sums
of at most a few thousand terms), one held in 16 bits is rounded once on top.
Weights and states that multiply a 16-bit input once more are kept to 22 bits or
more, an error of 2^-22 that 1e-5 holds many times over.

dg, the gradient of the decays, is the one result that is a difference: a sum over
time of terms of either sign, each the sum of at most 256 products that lose
sqrt(256) 2^-24 = 2^-20 of the term's size; N of them, independent, lose sqrt(N)
2^-20 of it.  What terms there are is part of what the definition returns.
"""
import torch


def _lens(lengths, B, N):
    return [N] * B if lengths is None else [min(max(int(n), 0), N) for n in lengths]


def linear_attn(q, k, v, g, scale=1.0, x_in=None, lengths=None):
    """(y, x_out) by the recurrence, one step at a time."""
    B, N, H, dv = v.shape
    G, dk = q.shape[2:]
    of = torch.arange(H) // (H // G)
    ys, ends = [], []
    for b, n in enumerate(_lens(lengths, B, N)):
        S = torch.zeros(H, dk, dv, dtype=torch.float64) if x_in is None else x_in[b]
        row = []
        for t in range(n):
            a = torch.exp(g[b, t] if g.dim() == 3 else g)
            S = a[:, None, None] * S + k[b, t, of][:, :, None] * v[b, t][:, None, :]
            row.append(scale * (q[b, t, of][:, :, None] * S).sum(1))
        row += [torch.zeros(H, dv, dtype=torch.float64)] * (N - n)
        ys.append(torch.stack(row) if N else torch.zeros(0, H, dv, dtype=torch.float64))
        ends.append(S)
    return torch.stack(ys), torch.stack(ends)


def dg_terms(q, dq_heads, N):
    """How large the terms are that dg is a sum of: the norm of q_t . dq_t (per head, shared heads apart)."""
    return (q * dq_heads).sum(-1).norm().item()


def close_dg(got, ref, terms, N, what="dg"):
    g, r = got.detach().double().cpu(), ref.detach().double()
    assert g.shape == r.shape and torch.isfinite(g).all(), what
    err, bound = (g - r).norm().item(), 1e-5 * r.norm().item() + N ** 0.5 * 2.0 ** -20 * terms
    if ref.dim() == 1:  # a decay per head: the N gradients of its steps are summed, errors that are themselves sums
        bound = 1e-5 * r.norm().item() + N ** 1.5 * 2.0 ** -20 * terms
    assert err <= bound + 1e-30, "%s: error %.3e of %.3e, bound %.3e" % (what, err, r.norm().item(), bound)


def block_norm(f, res=None, gate=None, w_out=None, scale=None, w_in=None, groups=1, eps=1e-5):
    """(r, y); y is None without a w_in."""
    m = f
    if w_out is not None:
        p = f.reshape(f.shape[0], groups, -1)
        m = (p / torch.sqrt((p * p).mean(-1, keepdim=True) + eps)).reshape(f.shape) * w_out
    if gate is not None:
        m = m * gate * torch.sigmoid(gate)
    r = m if scale is None else m * scale
    r = r if res is None else r + res
    y = None if w_in is None else r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps) * w_in
    return r, y


def embed(tokens, w, scale=1.0):
    on = (tokens >= 0) & (tokens < w.shape[0])
    rows = w[torch.where(on, tokens, torch.zeros_like(tokens))] * scale
    return torch.where(on[..., None], rows, torch.zeros_like(rows))
