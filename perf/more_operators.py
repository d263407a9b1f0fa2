"""Timed cases of linear attention with decay, of the norms around a block, and of the embedding.

Three operators of a recurrent language model built from this library's layers, each in the directions it is used in:

  linear_attn  a matrix state per head that decays by a factor per step, S_t = e^{g_t} S_{t-1} + k_t v_t^T and
               y_t = scale S_t^T q_t: prompts ("prompt"), a training pass ("train"), one token per sequence ("step")
  block_norm   what stands between two blocks: the norm of a block's output, its gate, the scaled residual sum and
               the norm before the next block: forward ("eval") and with gradients ("train")
  embed        rows of a table by token, scaled: lookup ("eval") and with the table's gradient ("train")

``own`` selects what ``run`` computes with: elementary torch operations in 32 bits, or this
package's entry points.  ``exact`` is the same definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5


def _attn(name, do, io, B, N, H, dk, dv, G=0, token=False, state=False, ragged=False, slots=0):
    """G: groups of heads that share q and k (0: none do); token: a decay for each token, not for each head alone."""
    return dict(name=name, op="linear_attn", do=do, io=io, B=B, N=N, H=H, G=G or H, dk=dk, dv=dv, token=token,
                state=state, ragged=ragged, slots=slots)


def _norm(name, do, io, T, D, res=True, gate=True, after=True, scale=True, before=True, groups=1):
    return dict(name=name, op="block_norm", do=do, io=io, T=T, D=D, res=res, gate=gate, after=after, scale=scale,
                before=before, groups=groups)


def _embed(name, do, io, T, D, V, zipf=1.0, pad=0.0):
    """zipf: the exponent of the tokens' frequencies; pad: the share of the most frequent token on top."""
    return dict(name=name, op="embed", do=do, io=io, T=T, D=D, V=V, zipf=zipf, pad=pad)


def listed():
    return [
        # a batch of 1K prompts at width 768, 12 heads of 64: one decay per head, the state kept for generation
        _attn("attn_prompt_1k", "prompt", "f16", 8, 1024, 12, 64, 64, state=True),
        # one very long document, width 1024 in 8 heads: the sequence is all there is to share out
        _attn("attn_prompt_64k", "prompt", "bf16", 1, 65536, 8, 128, 128, token=True, state=True),
        # prompts of unlike lengths (one empty, one of one token), odd sizes, shared keys, 32-bit activations
        _attn("attn_ragged_odd", "prompt", "f32", 5, 777, 6, 24, 41, G=2, token=True, state=True, ragged=True),
        # a training pass at width 2560 and length 2048, 20 heads of 128, a decay for each token
        _attn("attn_train_2k", "train", "bf16", 4, 2048, 20, 128, 128, token=True),
        # a small training pass whose queries and keys are shared by groups of 3 heads, odd length
        _attn("attn_train_groups", "train", "f16", 3, 301, 6, 64, 32, G=2),
        # generation at batch 64, width 768: one token each, states in a pool of 96 slots
        _attn("attn_step_b64", "step", "f16", 64, 1, 12, 64, 64, slots=96),
        # between two blocks of generation at batch 64, width 768
        _norm("norm_token_b64", "eval", "f16", 64, 768),
        # a training pass over 8 x 1024 tokens at width 768, the norm after the block in 12 heads
        _norm("norm_train_768", "train", "f16", 8192, 768, groups=12),
        # a training pass over 4 x 2048 tokens at width 2560
        _norm("norm_train_2560", "train", "bf16", 8192, 2560),
        # small and odd, in 32 bits: the norm before a block alone, with its residual sum
        _norm("norm_train_odd", "train", "f32", 517, 201, gate=False, after=False, scale=False),
        # training over 8 x 1024 tokens at width 768 and a vocabulary of 50K, frequencies as in text
        _embed("embed_train_50k", "train", "bf16", 8192, 768, 50021),
        # long rows with padding: 32 x 2048 tokens at width 1024, a third of them one token
        _embed("embed_train_pad", "train", "f16", 65536, 1024, 32768, pad=0.33),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["linear_attn", "linear_attn", "block_norm", "embed"])
    io = rng.choice(["f16", "bf16", "f16", "bf16", "f32"])
    if op == "embed":
        D, V = _log(rng, 48, 2560), _log(rng, 100, 50021)
        T = _log(rng, 1, max(1, min(65536, 65536 * 1024 // D)))
        c = _embed("", rng.choice(["eval", "train"]), io, T, D, V, zipf=rng.choice([0.0, 1.0]), pad=rng.choice([0.0, 0.0, 0.3]))
    elif op == "block_norm":
        groups = rng.choice([1, 1, 1, 4, 12])
        D = _log(rng, max(8, 48 // groups), 2560 // groups) * groups
        T = _log(rng, 1, max(1, min(65536, 8192 * 2560 // D // (2 if io == "f32" else 1))))
        after = rng.random() < 0.7
        c = _norm("", rng.choice(["eval", "train"]), io, T, D, res=rng.random() < 0.8, gate=rng.random() < 0.6, after=after,
                  scale=rng.random() < 0.5, before=not after or rng.random() < 0.7, groups=groups if after else 1)
    else:
        do = rng.choice(["prompt", "train", "step"])
        dk = rng.choice([16, 32, 64, 64, 128, rng.randrange(8, 129)])
        dv = rng.choice([dk, dk, 64, 128, rng.randrange(8, 129)])
        G = rng.choice([0, 0, 1, 2])
        H = _log(rng, 1, max(2, 2560 // max(dk, dv)))
        H = -(-H // G) * G if G else H
        token, state = rng.random() < 0.5, rng.random() < 0.5
        if do == "step":
            B = _log(rng, 1, 256)
            c = _attn("", do, io, B, 1, H, dk, dv, G, token, slots=B + rng.randrange(0, 33))
        else:
            B = _log(rng, 1, 8)
            most = 4 * 2560 * 2048 // (B * H * max(dk, dv)) // (4 if io == "f32" else 1)
            N = _log(rng, 1, max(1, min(65536 if do == "prompt" else 8192, most)))
            c = _attn("", do, io, B, N, H, dk, dv, G, token, state=do == "prompt" and state,
                      ragged=do == "prompt" and rng.random() < 0.4)
    return {k: v for k, v in c.items() if k != "name"}


# ------------------------------------------------------------------ inputs


def _lengths(B, N, g, dev):
    """Valid lengths in 0 .. N; the first rows are the ends of the range."""
    n = torch.randint(0, N + 1, (B,), generator=g, device=dev)
    ends = torch.tensor([N, 0, min(1, N)], device=dev)[:B]
    n[: len(ends)] = ends
    return n.to(torch.int32)


def _uniform(g, dev, lo, hi, *shape):
    return lo + (hi - lo) * torch.rand(*shape, generator=g, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    t, c = TYPES[case["io"]], case

    def normal(*shape, std=1.0, dtype=t):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    s = {"case": case}
    train = c["do"] == "train"
    if c["op"] == "embed":
        T, D, V = c["T"], c["D"], c["V"]
        s["w"] = normal(V, D, std=1.0)
        s["scale"] = math.sqrt(D)
        # frequencies that fall as rank^-zipf, ranks spread over the vocabulary
        odds = torch.arange(1, V + 1, device=dev, dtype=torch.float64) ** -c["zipf"]
        edge = torch.cumsum(odds / odds.sum(), 0)
        rank = torch.searchsorted(edge, torch.rand(T, generator=g, device=dev, dtype=torch.float64)).clamp(max=V - 1)
        rank[torch.rand(T, generator=g, device=dev) < c["pad"]] = 0
        s["tokens"] = torch.randperm(V, generator=g, device=dev)[rank]
        if train:
            s["dy"] = normal(T, D, std=0.01)
        return s
    if c["op"] == "block_norm":
        T, D = c["T"], c["D"]
        s["f"] = normal(T, D, std=0.5)
        s["res"] = normal(T, D, std=2.0) if c["res"] else None
        s["gate"] = normal(T, D) if c["gate"] else None
        s["w_out"] = 1.0 + normal(D, std=0.1, dtype=torch.float32) if c["after"] else None
        s["scale"] = 0.5 + normal(D, std=0.1, dtype=torch.float32) if c["scale"] else None
        s["w_in"] = 1.0 + normal(D, std=0.1, dtype=torch.float32) if c["before"] else None
        if train:
            s["dr"], s["dy"] = normal(T, D), normal(T, D) if c["before"] else None
        return s
    B, N, H, G, dk, dv = (c[k] for k in ("B", "N", "H", "G", "dk", "dv"))
    step = c["do"] == "step"
    lead = (B,) if step else (B, N)
    s["q"], s["k"], s["v"] = normal(*lead, G, dk), normal(*lead, G, dk), normal(*lead, H, dv)
    s["scale"] = dk ** -0.5
    if c["token"]:  # a step size, log-uniform on [1e-3, 1e-1] and spread per token, times a rate of 1 .. 16 per head
        size = torch.exp(_uniform(g, dev, math.log(1e-3), math.log(1e-1), H) + 0.5 * normal(*lead, H, dtype=torch.float32))
        s["g"] = (-size * _uniform(g, dev, 1.0, 16.0, H)).contiguous()
    else:  # factors 1 - 2^-5 .. 1 - 2^-12, spread over the heads
        s["g"] = torch.log1p(-torch.exp2(-_uniform(g, dev, 5.0, 12.0, H)))
    s["lengths"] = _lengths(B, N, g, dev) if c["ragged"] else None
    if step:  # every sequence has a slot of its own in the pool of states
        s["slots"] = torch.randperm(c["slots"], generator=g, device=dev)[:B].to(torch.int32)
        s["x_in"] = normal(c["slots"], H, dk, dv, std=3.0, dtype=torch.float32)
        s["x_out"] = torch.zeros_like(s["x_in"])
    else:
        s["x_in"] = normal(B, H, dk, dv, std=3.0, dtype=torch.float32) if c["state"] else None
    if train:
        s["dy"] = normal(B, N, H, dv)
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    c = s["case"]
    return (_run_own if own else _run_plain)(s, c["op"], c["do"], c)


def _run_own(s, op, do, c):
    import fft_long_convolution_flashconv_amd as h3

    if op == "embed":
        y = h3.embed(s["tokens"], s["w"], scale=s["scale"])
        return y if do == "eval" else (y, h3.embed_bwd(s["tokens"], s["dy"], c["V"], scale=s["scale"]))
    if op == "block_norm":
        k = dict(res=s["res"], gate=s["gate"], w_out=s["w_out"], scale=s["scale"], w_in=s["w_in"], groups=c["groups"], eps=EPS)
        out = h3.block_norm(s["f"], **k)
        if do == "eval":
            return out
        return out, tuple(h3.block_norm_bwd(s["f"], s["dr"], s["dy"], **k))
    a = (s["q"], s["k"], s["v"], s["g"])
    if do == "step":
        return h3.linear_attn_step(*a, s["x_in"], scale=s["scale"], slots=s["slots"], x_out=s["x_out"]), s["x_out"]
    if do == "prompt":
        return h3.linear_attn(*a, scale=s["scale"], x_in=s["x_in"], lengths=s["lengths"], return_state=True)
    y = h3.linear_attn(*a, scale=s["scale"])
    d = h3.linear_attn_bwd(*a, s["dy"], scale=s["scale"])
    return y, d.dq, d.dk, d.dv, d.dg


def _run_plain(s, op, do, c):
    if op == "embed":
        return _plain_embed(s, do, c)
    if op == "block_norm":
        return _plain_norm(s, do, c)
    return _plain_step(s, c) if do == "step" else _plain_attn(s, do, c)


# ------------------------------------------------------------------ plain forms, 32 bits


CHUNK = 64


def _cut(t, H):
    """[B,N,G,...] -> [B,H,n,CHUNK,...] in fp32 (or its own 64 bits), zeros behind the last step."""
    B, N = t.shape[:2]
    t = t if t.dtype == torch.float64 else t.float()
    t = t.repeat_interleave(H // t.shape[2], 2).transpose(1, 2)
    pad = -N % CHUNK
    if pad:
        t = torch.cat([t, t.new_zeros(B, H, pad, *t.shape[3:])], 2)
    return t.reshape(B, H, (N + pad) // CHUNK, CHUNK, *t.shape[3:]).contiguous()


def _sew(t, N):
    """[B,H,n,CHUNK,d] -> [B,N,H,d]."""
    B, H = t.shape[:2]
    return t.reshape(B, H, -1, *t.shape[4:])[:, :, :N].transpose(1, 2).contiguous()


def _carry(a, b):
    """The states after each chunk, h_n = a_n h_{n-1} + b_n, by doubling."""
    k = 1
    while k < b.shape[2]:
        b[:, :, k:] += a[:, :, k:] * b[:, :, :-k].clone()
        a[:, :, k:] = a[:, :, k:] * a[:, :, :-k].clone()
        k *= 2
    return b


def _t(x):
    return x.transpose(-1, -2).contiguous()


def _plain_attn(s, do, c):
    B, N, H, G, scale, t = c["B"], c["N"], c["H"], c["G"], s["scale"], s["v"].dtype
    dev = s["v"].device
    g = s["g"].double().expand(B, N, H)
    q, k, v = s["q"], s["k"], s["v"]
    valid = None
    if s["lengths"] is not None:
        valid = (torch.arange(N, device=dev) < s["lengths"][:, None])[:, :, None]
        g = torch.where(valid, g, torch.zeros_like(g))
        k, v = (torch.where(valid[..., None], m, torch.zeros_like(m)) for m in (k, v))
    g = _cut(g, H)
    q, k, v = _cut(q, H), _cut(k, H), _cut(v, H)
    Gc = torch.cumsum(g, -1)                                   # 64 bits: differences of these are exponents
    diff = Gc[..., :, None] - Gc[..., None, :]
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    w = torch.where(low, torch.exp(diff.clamp(max=80.0)), torch.zeros_like(diff)).float()
    del diff
    into = torch.exp(Gc).float()[..., None]                    # from the chunk's start to a step
    out = torch.exp(Gc[..., -1:] - Gc).float()[..., None]      # from a step to the chunk's end
    whole = torch.exp(Gc[..., -1]).float()[..., None, None]
    first = s["x_in"] if s["x_in"] is not None else q.new_zeros(B, H, c["dk"], c["dv"])
    local = torch.matmul(_t(k * out), v)
    local[:, :, 0] += whole[:, :, 0] * first
    ends = _carry(whole.clone(), local)
    S = torch.cat([first[:, :, None], ends[:, :, :-1]], 2)
    qk = torch.matmul(q, _t(k)) * w
    y = scale * (torch.matmul(q * into, S) + torch.matmul(qk, v))
    y = _sew(y, N)
    if valid is not None:
        y = torch.where(valid[..., None], y, torch.zeros_like(y))
    y = y.to(t)
    if do == "prompt":
        return y, ends[:, :, -1].contiguous()
    d = _cut(s["dy"], H)
    back = scale * torch.matmul(_t(q * into), d)
    # adjoint states at the chunks' ends, from the last one on; nothing comes from behind the sequence
    D = torch.cat([_carry(whole.flip(2).clone(), back.flip(2)).flip(2)[:, :, 1:], torch.zeros_like(back[:, :, :1])], 2)
    dvw = torch.matmul(d, _t(v)) * w
    qS, kD = scale * into * torch.matmul(d, _t(S)), out * torch.matmul(v, _t(D))
    dq = scale * torch.matmul(dvw, k) + qS
    dk = scale * torch.matmul(_t(dvw), q) + kD
    dv = scale * torch.matmul(_t(qk), d) + out * torch.matmul(k, D)
    # dg_t: every product that reaches over the border before step t, without the steps' own
    pairs = (scale * qk * torch.matmul(d, _t(v))).tril(-1).double()
    over = pairs.sum(-1) + (q * qS).double().sum(-1) - pairs.sum(-2) - (k * kD).double().sum(-1)
    dg = over.flip(-1).cumsum(-1).flip(-1) + (ends.double() * D).sum((-1, -2))[..., None]
    dg = _sew(dg, N)
    dg = dg.float() if c["token"] else dg.sum((0, 1)).float()

    def shared(m):
        return _sew(m, N).view(B, N, G, H // G, c["dk"]).sum(3).to(t)

    return y, shared(dq), shared(dk), _sew(dv, N).to(t), dg


def _plain_step(s, c):
    at, t, H = s["slots"].long(), s["v"].dtype, c["H"]
    q, k = (m.float().repeat_interleave(H // c["G"], 1) for m in (s["q"], s["k"]))
    a = torch.exp(s["g"]).expand(c["B"], H)
    x = a[..., None, None] * s["x_in"][at] + k[..., :, None] * s["v"].float()[..., None, :]
    y = s["scale"] * (q[..., :, None] * x).sum(2)
    s["x_out"][at] = x
    return y.to(t), s["x_out"]


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _plain_norm(s, do, c):
    T, D, n, t = c["T"], c["D"], c["groups"], s["f"].dtype
    f = s["f"].float()
    m = f
    if s["w_out"] is not None:
        parts = f.view(T, n, D // n)
        ra = torch.rsqrt(parts.square().mean(-1, keepdim=True) + EPS)
        fh = (parts * ra).view(T, D)
        m = nrm = fh * s["w_out"]
    if s["gate"] is not None:
        z = s["gate"].float()
        sg = _sigmoid(z)
        m = m * z * sg
    r = m * s["scale"] if s["scale"] is not None else m
    if s["res"] is not None:
        r = r + s["res"].float()
    y = None
    if s["w_in"] is not None:
        rb = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)
        rh = r * rb
        y = rh * s["w_in"]
    out = (r.to(t), y.to(t)) if y is not None else r.to(t)
    if do == "eval":
        return out
    dr = s["dr"].float()
    dw_in = dw_out = dscale = dgate = None
    if y is not None:
        dy = s["dy"].float()
        dw_in = (dy * rh).sum(0)
        e = dy * s["w_in"]
        dr = dr + rb * (e - rh * (e * rh).mean(-1, keepdim=True))
    dres = dr.to(t) if s["res"] is not None else None
    dm = dr
    if s["scale"] is not None:
        dscale = (dr * m).sum(0)
        dm = dr * s["scale"]
    if s["gate"] is not None:
        dgate = (dm * (nrm if s["w_out"] is not None else f) * sg * (1.0 + z * (1.0 - sg))).to(t)
        dm = dm * z * sg
    if s["w_out"] is not None:
        dw_out = (dm * fh).sum(0)
        e, h = (dm * s["w_out"]).view(T, n, D // n), fh.view(T, n, D // n)
        dm = (ra * (e - h * (e * h).mean(-1, keepdim=True))).view(T, D)
    return out, (dm.to(t), dres, dgate, dw_out, dscale, dw_in)


def _plain_embed(s, do, c):
    y = (s["w"][s["tokens"]].float() * s["scale"]).to(s["w"].dtype)
    if do == "eval":
        return y
    dw = torch.zeros(c["V"], c["D"], device=y.device)
    dw.index_add_(0, s["tokens"], s["dy"].float())
    return y, (dw * s["scale"]).to(y.dtype)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    c, e = case, SIZE[case["io"]]
    train = c["do"] == "train"
    if c["op"] == "embed":
        T, D, V = c["T"], c["D"], c["V"]
        n = T * D
        return {"bytes": 2 * n * e + T * 8 + ((n + V * D) * e + T * 8 if train else 0), "flops": float(n * (2 if train else 1))}
    if c["op"] == "block_norm":
        n = c["T"] * c["D"]
        rows = 1 + c["res"] + c["gate"]                        # read
        wide = 1 + c["before"]                                 # r and y
        par = c["D"] * 4 * (c["after"] + c["scale"] + c["before"])
        moved = (rows + wide) * n * e + par
        if train:  # the inputs and the upstream gradients again, and the gradients
            moved += (rows + wide + rows) * n * e + 2 * par
        return {"bytes": moved, "flops": n * (12.0 if not train else 40.0)}
    B, N, H, G, dk, dv = (c[k] for k in ("B", "N", "H", "G", "dk", "dv"))
    state, steps = B * H * dk * dv * 4, B * N
    decay = (steps * H if c["token"] else H) * 4
    rows = steps * (2 * G * dk + H * dv) * e                   # q, k and v, or their gradients
    y = steps * H * dv * e
    if c["do"] == "step":
        return {"bytes": rows + y + decay + 2 * state, "flops": 4.0 * B * H * dk * dv}
    # the state is updated and read at every step, a product of dk x dv each
    flops = 4.0 * steps * H * dk * dv
    if train:  # then dq from the state, dk and dv from its adjoint, which is updated in turn
        return {"bytes": rows + y + decay + rows + y + decay + rows + decay, "flops": flops + 10.0 * steps * H * dk * dv}
    return {"bytes": rows + y + decay + state * (2 if c["state"] else 1), "flops": flops}


# ------------------------------------------------------------------ the definitions, 64 bits


def exact(case, seed):
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in prepare(case, seed).items()}
    return {"embed": _exact_embed, "block_norm": _exact_norm, "linear_attn": _exact_attn}[case["op"]](s, case)


def _exact_embed(s, c):
    y = torch.index_select(s["w"], 0, s["tokens"]) * s["scale"]
    if c["do"] == "eval":
        return y
    dw = torch.zeros_like(s["w"]).index_put_((s["tokens"],), s["dy"] * s["scale"], accumulate=True)
    return y, dw


def _exact_norm(s, c):
    names = ("f", "res", "gate", "w_out", "scale", "w_in")
    leaf = {k: s[k].requires_grad_(True) for k in names if s[k] is not None}
    r = leaf["f"]
    if "w_out" in leaf:
        p = r.unflatten(1, (c["groups"], -1))
        r = (p / torch.sqrt((p * p).mean(2, keepdim=True) + EPS)).flatten(1) * leaf["w_out"]
    if "gate" in leaf:
        r = r * leaf["gate"] * torch.sigmoid(leaf["gate"])
    if "scale" in leaf:
        r = r * leaf["scale"]
    if "res" in leaf:
        r = leaf["res"] + r
    out, up = [r], [s.get("dr")]
    if "w_in" in leaf:
        out.append(r / torch.sqrt((r * r).mean(1, keepdim=True) + EPS) * leaf["w_in"])
        up.append(s.get("dy"))
    values = tuple(v.detach() for v in out) if len(out) > 1 else r.detach()
    if c["do"] == "eval":
        return values
    grads = dict(zip(leaf, torch.autograd.grad(out, list(leaf.values()), up)))
    return values, tuple(grads.get(k) for k in names)


def _exact_attn(s, c):
    B, N, H, G, scale = c["B"], c["N"], c["H"], c["G"], s["scale"]
    of = torch.arange(H, device=s["v"].device) // (H // G)    # the group of each head
    if c["do"] == "step":
        at = s["slots"].long()
        for b in range(B):
            a = torch.exp(s["g"][b] if c["token"] else s["g"])[:, None, None]
            s["x_out"][at[b]] = a * s["x_in"][at[b]] + torch.einsum("hi,hj->hij", s["k"][b, of], s["v"][b])
        return scale * torch.einsum("bhi,bhij->bhj", s["q"][:, of], s["x_out"][at]), s["x_out"]
    train = c["do"] == "train"

    def by_time(m):
        return m.transpose(0, 1).contiguous()

    q, k, v = by_time(s["q"][:, :, of])[..., None, :], by_time(s["k"][:, :, of])[..., None], by_time(s["v"])[..., None, :]
    a = torch.exp(by_time(s["g"].expand(B, N, H)))[..., None, None]
    n = None if s["lengths"] is None else s["lengths"].to(q.device)
    x = torch.zeros(B, H, c["dk"], c["dv"], dtype=torch.float64, device=v.device) if s["x_in"] is None else s["x_in"].clone()
    hs = torch.empty(N + 1, *x.shape, dtype=torch.float64, device=v.device) if train else None
    y = torch.zeros(N, B, H, c["dv"], dtype=torch.float64, device=v.device)
    if train:
        hs[0] = x
    for i in range(N):
        new = torch.addcmul(a[i] * x, k[i], v[i])
        row = torch.matmul(q[i], new)[..., 0, :]
        if n is not None:
            on = (i < n)[:, None, None]
            new, row = torch.where(on[..., None], new, x), torch.where(on, row, torch.zeros_like(row))
        x = new
        y[i] = row
        if train:
            hs[i + 1] = x
    y = by_time(y * scale)
    if not train:
        return y, x
    d = by_time(s["dy"])[..., None, :]
    D = torch.zeros_like(x)
    dq, dk, dv = torch.empty_like(q[..., 0, :]), torch.empty_like(k[..., 0]), torch.empty_like(v[..., 0, :])
    dg = torch.empty(N, B, H, dtype=torch.float64, device=x.device)
    for i in range(N - 1, -1, -1):
        D = torch.addcmul(D, scale * q[i].transpose(-1, -2), d[i])        # d loss / d S_i
        dq[i] = scale * (hs[i + 1] * d[i]).sum(-1)
        dk[i] = (D * v[i]).sum(-1)
        dv[i] = (D * k[i]).sum(-2)
        D = a[i] * D
        dg[i] = (hs[i] * D).sum((-1, -2))

    def shared(m):
        return by_time(m).view(B, N, G, H // G, c["dk"]).sum(3)

    return y, shared(dq), shared(dk), by_time(dv), by_time(dg) if c["token"] else dg.sum((0, 1))
