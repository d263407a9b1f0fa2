"""Plain 64-bit definitions of the short convolution, the selective scan and
the linear cross entropy (torch float64 on the CPU, step by step), which the
GPU tests compare against; gradients come from automatic differentiation of
these definitions.

Tolerances, relative L2 against the definition on the same (rounded) inputs:
a result held in fp32 is computed in fp32, with sums over at most a few
thousand terms and exponentials good to an ulp or two: 1e-5.  A result held in
16 bits is computed in fp32 and rounded once: half an ulp of its type, 2^-8
(bf16 has 8 significant bits) or 2^-11, over that.  The loss's gradients round
one factor of their products (G) to 16 bits as well: two roundings; and e^l
carries the rounding of the logits themselves, a few 2^-24 of the largest one.
An fp16 result below 2^-14 rounds to a multiple of 2^-24: half of that per
element on top.
"""
import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def close(got, ref, io="f32", roundings=1, what="", extra=0.0):
    """Relative L2 within the bound derived above."""
    g, r = got.detach().double().cpu(), ref.detach().double()
    assert g.shape == r.shape, (what, g.shape, r.shape)
    assert torch.isfinite(g).all(), what
    tol = 1e-5 + roundings * HALF_ULP[io] + extra
    slack = (2.0 ** -25 if io == "f16" else 1e-30) * r.numel() ** 0.5
    err, norm = (g - r).norm().item(), r.norm().item()
    assert err <= tol * norm + slack, "%s: error %.3e of %.3e (rel %.3e, bound %.3e)" % (
        what, err, norm, err / max(norm, 1e-300), tol)


def _lens(lengths, B, N):
    return [N] * B if lengths is None else [min(max(int(n), 0), N) for n in lengths]


def short_conv(x, w, bias, silu, x_in, lengths):
    """(y, x_out): y_t = act(bias + sum_i w_i x_{t-i}), rows cut at their lengths."""
    B, H, N = x.shape
    W = w.shape[1]
    head = torch.zeros(B, H, W - 1, dtype=torch.float64) if x_in is None else x_in
    ys, last = [], []
    for b, n in enumerate(_lens(lengths, B, N)):
        ext = torch.cat([head[b], x[b, :, :n]], -1)
        p = torch.zeros(H, n, dtype=torch.float64) if bias is None else bias[:, None].expand(H, n)
        for i in range(W):
            p = p + w[:, i, None] * ext[:, W - 1 - i: W - 1 - i + n]
        y = p * torch.sigmoid(p) if silu else p
        ys.append(torch.cat([y, torch.zeros(H, N - n, dtype=torch.float64)], -1))
        last.append(ext[:, ext.shape[1] - (W - 1):])
    return torch.stack(ys) if B else x.new_zeros(0, H, N), torch.stack(last) if B else x.new_zeros(0, H, W - 1)


def selective_scan(u, dt, A, Bm, C, D, z, dt_bias, softplus, x_in, lengths):
    """(y, x_out) by the recurrence, one step at a time."""
    B, H, N = u.shape
    S, G = A.shape[1], Bm.shape[1]
    of = torch.arange(H) // (H // G)
    ys, ends = [], []
    for b, n in enumerate(_lens(lengths, B, N)):
        x = torch.zeros(H, S, dtype=torch.float64) if x_in is None else x_in[b]
        row = []
        for t in range(n):
            d = dt[b, :, t] + (0 if dt_bias is None else dt_bias)
            d = torch.nn.functional.softplus(d, threshold=1e9) if softplus else d
            x = torch.exp(d[:, None] * A) * x + (d * u[b, :, t])[:, None] * Bm[b, of, :, t]
            r = (C[b, of, :, t] * x).sum(-1)
            if D is not None:
                r = r + D * u[b, :, t]
            if z is not None:
                r = r * z[b, :, t] * torch.sigmoid(z[b, :, t])
            row.append(r)
        row += [torch.zeros(H, dtype=torch.float64)] * (N - n)
        ys.append(torch.stack(row, -1) if N else torch.zeros(H, 0, dtype=torch.float64))
        ends.append(x)
    return torch.stack(ys), torch.stack(ends)


def linear_xent(x, w, labels, ignore=-100):
    """(loss, lse)."""
    z = x @ w.t()
    lse = torch.logsumexp(z, 1)
    on = (labels != ignore) & (labels >= 0) & (labels < w.shape[0])
    hit = z[torch.arange(len(labels)), torch.where(on, labels, torch.zeros_like(labels))]
    return torch.where(on, lse - hit, torch.zeros_like(lse)), lse


def leaf(t):
    """A 64-bit copy that gradients are taken of."""
    return None if t is None else t.detach().double().cpu().requires_grad_(True)


def directional(f, args, grads, seed, eps=1e-5):
    """(<grads, v>, central difference of f along v) for a random direction v over the given leaves."""
    g = torch.Generator().manual_seed(seed)
    keys = [k for k in args if grads.get(k) is not None]
    v = {k: torch.randn(args[k].shape, generator=g, dtype=torch.float64) for k in keys}

    def at(s):
        with torch.no_grad():
            return float(f({k: (a + s * v[k] if k in v else a) for k, a in args.items()}))

    dot = sum(float((grads[k].detach().double().cpu() * v[k]).sum()) for k in keys)
    size = sum(float((grads[k].detach().double().cpu() * v[k]).square().sum()) for k in keys) ** 0.5
    return dot, (at(eps) - at(-eps)) / (2 * eps), size
