"""Timed cases of the selective state-space operators and of the language-model loss.

Three operators of a model built from this library's layers, each in the directions it is used in:

  short_conv      causal depthwise convolution over the last W steps, with bias and SiLU:
                  prompts ("prompt"), a training pass ("train"), one token per sequence ("step")
  selective_scan  diagonal state-space scan with input-dependent step, B and C, gated output:
                  prompts, a training pass, one token per sequence
  linear_xent     cross entropy of a linear output layer over a large vocabulary, without the
                  logits of the whole vocabulary at once: "eval" (loss), "train" (loss and gradients)

``own`` selects what ``run`` computes with: elementary torch operations in 32 bits, or this
package's entry points.  ``exact`` is the same definition in 64 bits, step by step.
"""
from __future__ import annotations

import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
IGNORE = -100


def _conv(name, do, io, B, H, N, W=4, bias=True, silu=True, state=False, ragged=False, slots=0):
    return dict(name=name, op="short_conv", do=do, io=io, B=B, H=H, N=N, W=W, bias=bias, silu=silu, state=state,
                ragged=ragged, slots=slots)


def _scan(name, do, io, B, H, N, S=16, G=1, gate=True, state=False, ragged=False, slots=0):
    return dict(name=name, op="selective_scan", do=do, io=io, B=B, H=H, N=N, S=S, G=G, gate=gate, state=state,
                ragged=ragged, slots=slots)


def _xent(name, do, io, T, D, V):
    return dict(name=name, op="linear_xent", do=do, io=io, T=T, D=D, V=V)


def listed():
    return [
        # a batch of 1K prompts at width 768: the mixing layer's convolution, its last inputs kept for generation
        _conv("conv_prompt_1k", "prompt", "f16", 8, 768, 1024, state=True),
        # a training pass at width 2560 and length 2048
        _conv("conv_train_2k", "train", "bf16", 4, 2560, 2048),
        # generation at batch 64, width 768: one token each, states in a pool of 96 slots
        _conv("conv_step_b64", "step", "f16", 64, 768, 1, slots=96),
        # the scan of the same 1K prompts
        _scan("scan_prompt_1k", "prompt", "f16", 8, 768, 1024, state=True),
        # one very long document, few channels: the sequence is all there is to share out
        _scan("scan_prompt_64k", "prompt", "bf16", 1, 1024, 65536),
        # prompts of unlike lengths (one empty, one of one token), odd sizes, 32-bit activations
        _scan("scan_ragged_odd", "prompt", "f32", 5, 193, 777, S=7, gate=False, state=True, ragged=True),
        # a training pass at width 2560 and length 2048
        _scan("scan_train_2k", "train", "bf16", 4, 2560, 2048),
        # a training pass whose B and C are shared by groups of 32 channels, 24 modes, odd length
        _scan("scan_train_groups", "train", "f16", 3, 96, 301, S=24, G=3),
        # generation at batch 64, width 768
        _scan("scan_step_b64", "step", "f16", 64, 768, 1, slots=96),
        # scoring 4K tokens: the loss alone, width 2560
        _xent("xent_eval_32k", "eval", "f16", 4096, 2560, 32768),
        # a training pass over 8 x 1024 tokens at width 768, a vocabulary that no tile divides
        _xent("xent_train_50k", "train", "bf16", 8192, 768, 50021),
        # a small head in 32 bits, nothing a multiple of anything
        _xent("xent_train_odd", "train", "f32", 517, 201, 1009),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["short_conv", "selective_scan", "selective_scan", "linear_xent"])
    io = rng.choice(["f16", "bf16", "f16", "bf16", "f32"])
    if op == "linear_xent":
        do = rng.choice(["eval", "train"])
        D = _log(rng, 64, 2560)
        V = _log(rng, 500, 50021)
        top = 8192 * 768 * 50021 // (1 if io != "f32" else 16) // (D * V)
        return {k: v for k, v in _xent("", do, io, _log(rng, 16, max(16, min(8192, top))), D, V).items() if k != "name"}
    do = rng.choice(["prompt", "train", "step"])
    H = _log(rng, 48, 2560)
    if do == "step":
        B = _log(rng, 1, 256)
        N, slots = 1, B + rng.randrange(0, 33)
    else:
        B = _log(rng, 1, 8)
        N, slots = _log(rng, 1, max(1, min(65536, 4 * 2560 * 2048 // (B * H)))), 0
    ragged, state = do == "prompt" and rng.random() < 0.4, do == "prompt" and rng.random() < 0.5
    if op == "short_conv":
        c = _conv("", do, io, B, H, N, W=rng.choice([2, 3, 4]), bias=rng.random() < 0.7, silu=rng.random() < 0.7,
                  state=state, ragged=ragged, slots=slots)
    else:
        S = rng.choice([8, 16, 16, 16, 5, 24, 32])
        G = rng.choice([1, 1, 1, 2, 4])
        N = max(1, N // 2) if S > 16 and do != "step" else N
        H = -(-H // G) * G
        c = _scan("", do, io, B, H, N, S=S, G=G, gate=rng.random() < 0.6, state=state, ragged=ragged, slots=slots)
    return {k: v for k, v in c.items() if k != "name"}


# ------------------------------------------------------------------ inputs


def _lengths(B, N, g, dev):
    """Valid lengths in 0 .. N; the first rows are the ends of the range."""
    n = torch.randint(0, N + 1, (B,), generator=g, device=dev)
    ends = torch.tensor([N, 0, min(1, N)], device=dev)[:B]
    n[: len(ends)] = ends
    return n.to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    t = TYPES[case["io"]]

    def normal(*shape, std=1.0, dtype=t):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    s = {"case": case}
    if case["op"] == "linear_xent":
        T, D, V = case["T"], case["D"], case["V"]
        s["x"] = normal(T, D)                                 # a normalised hidden state
        s["w"] = normal(V, D, std=2.0 / math.sqrt(D))         # logits of a trained head: a few units wide
        s["labels"] = torch.randint(0, V, (T,), generator=g, device=dev)
        s["labels"][:: 7] = IGNORE                            # padding and prompt tokens carry no loss
        # the gradient of a mean over the tokens that count, times the loss scale of a 16-bit float's training
        s["dloss"] = (s["labels"] != IGNORE).float() * ((1024.0 if case["io"] == "f16" else 1.0) / max(1, T - (T + 6) // 7))
        return s
    B, H, N = case["B"], case["H"], case["N"]
    step, train = case["do"] == "step", case["do"] == "train"
    row = (B, H) if step else (B, H, N)
    s["lengths"] = _lengths(B, N, g, dev) if case["ragged"] else None
    if step:  # every sequence has a slot of its own in the pool of states
        s["slots"] = torch.randperm(case["slots"], generator=g, device=dev)[:B].to(torch.int32)
    P = case["slots"] if step else B
    if case["op"] == "short_conv":
        W = case["W"]
        s["x"] = normal(*row)
        s["w"] = normal(H, W, std=1.0 / math.sqrt(W), dtype=torch.float32)
        s["bias"] = normal(H, std=0.1, dtype=torch.float32) if case["bias"] else None
        s["x_in"] = normal(P, H, W - 1) if step or case["state"] else None
        if step:
            s["x_out"] = torch.zeros_like(s["x_in"])
        if train:
            s["dy"] = normal(*row)
        return s
    S, G = case["S"], case["G"]
    s["u"] = normal(*row)
    s["dt"] = normal(*row, std=0.5)
    # softplus(dt_bias) log-uniform on [1e-3, 1e-1]; A the negated mode numbers, a little spread per channel
    step0 = torch.exp(torch.rand(H, generator=g, device=dev) * math.log(100.0) + math.log(1e-3))
    s["dt_bias"] = torch.log(torch.expm1(step0))
    s["A"] = -(torch.arange(1, S + 1, device=dev, dtype=torch.float32) * torch.exp(0.1 * normal(H, 1, dtype=torch.float32))).contiguous()
    s["Bm"] = normal(B, G, S) if step else normal(B, G, S, N)
    s["C"] = normal(B, G, S) if step else normal(B, G, S, N)
    s["D"] = normal(H, std=0.1, dtype=torch.float32) + 1.0
    s["z"] = normal(*row) if case["gate"] else None
    s["x_in"] = normal(P, H, S, dtype=torch.float32) if step or case["state"] else None
    if step:
        s["x_out"] = torch.zeros_like(s["x_in"])
    if train:
        s["dy"] = normal(*row)
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    c = s["case"]
    return (_run_own if own else _run_plain)(s, c["op"], c["do"], c)


def _run_own(s, op, do, c):
    import fft_long_convolution_flashconv_amd as h3

    if op == "linear_xent":
        loss, lse = h3.linear_xent(s["x"], s["w"], s["labels"], ignore_index=IGNORE, return_lse=True)
        if do == "eval":
            return loss, lse
        dx, dw = h3.linear_xent_bwd(s["x"], s["w"], s["labels"], lse, s["dloss"], ignore_index=IGNORE)
        return loss, lse, dx, dw
    if op == "short_conv":
        w, bias, silu = s["w"], s["bias"], c["silu"]
        if do == "step":
            y = h3.short_conv_step(s["x"], w, s["x_in"], bias=bias, silu=silu, slots=s["slots"], state_out=s["x_out"])
            return y, s["x_out"]
        if do == "prompt":
            return h3.short_conv(s["x"], w, bias=bias, silu=silu, x_in=s["x_in"], lengths=s["lengths"], return_state=True)
        y = h3.short_conv(s["x"], w, bias=bias, silu=silu)
        dx, dw, dbias, _ = h3.short_conv_bwd(s["x"], w, s["dy"], bias=bias, silu=silu)
        return y, dx, dw, dbias
    a = (s["u"], s["dt"], s["A"], s["Bm"], s["C"])
    k = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"], softplus=True)
    if do == "step":
        y = h3.selective_step(*a, s["x_in"], slots=s["slots"], x_out=s["x_out"], **k)
        return y, s["x_out"]
    if do == "prompt":
        return h3.selective_scan(*a, x_in=s["x_in"], lengths=s["lengths"], return_state=True, **k)
    y, saved = h3.selective_scan(*a, return_saved=True, **k)
    d = h3.selective_scan_bwd(*a, s["dy"], saved, **k)
    return y, d.du, d.ddt, d.dA, d.dB, d.dC, d.dD, d.dz, d.ddt_bias


def _run_plain(s, op, do, c):
    if op == "linear_xent":
        return _plain_xent(s, do)
    if op == "short_conv":
        return _plain_conv_step(s, c) if do == "step" else _plain_conv(s, do, c)
    return _plain_scan_step(s, c) if do == "step" else _plain_scan(s, do, c)


# ------------------------------------------------------------------ plain forms, 32 bits


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _softplus(x):
    return torch.where(x > 20.0, x, torch.log1p(torch.exp(torch.minimum(x, torch.full_like(x, 20.0)))))


def _plain_conv(s, do, c):
    """y_t = silu(bias + sum_i w_i x_{t-i}), x before the row's start from x_in (or zero)."""
    x, w, W, N, t = s["x"].float(), s["w"], c["W"], c["N"], s["x"].dtype
    B, H = x.shape[:2]
    head = x.new_zeros(B, H, W - 1) if s["x_in"] is None else s["x_in"].float()
    valid = None
    if s["lengths"] is not None:
        valid = (torch.arange(N, device=x.device) < s["lengths"][:, None])[:, None]
        x = torch.where(valid, x, torch.zeros_like(x))
    ext = torch.cat([head, x], -1)
    pre = s["bias"][:, None].expand(B, H, N) if s["bias"] is not None else x.new_zeros(B, H, N)
    for i in range(W):
        pre = pre + w[:, i, None] * ext[..., W - 1 - i: W - 1 - i + N]
    sg = _sigmoid(pre)
    y = pre * sg if c["silu"] else pre
    if valid is not None:
        y = torch.where(valid, y, torch.zeros_like(y))
    if do == "prompt":
        n = torch.full((B,), N, device=x.device) if s["lengths"] is None else s["lengths"].long()
        at = n[:, None] + torch.arange(W - 1, device=x.device)
        return y.to(t), torch.gather(ext, 2, at[:, None].expand(B, H, W - 1)).to(t)
    dpre = s["dy"].float()
    if c["silu"]:
        dpre = dpre * sg * (1.0 + pre * (1.0 - sg))
    dext = torch.zeros_like(ext)
    dw = []
    for i in range(W):
        part = slice(W - 1 - i, W - 1 - i + N)
        dext[..., part] += w[:, i, None] * dpre
        dw.append((dpre * ext[..., part]).sum((0, 2)))
    dbias = dpre.sum((0, 2)) if s["bias"] is not None else None
    return y.to(t), dext[..., W - 1:].to(t), torch.stack(dw, 1), dbias


def _plain_conv_step(s, c):
    x, w, W, t, at = s["x"].float(), s["w"], c["W"], s["x"].dtype, s["slots"].long()
    ext = torch.cat([s["x_in"][at].float(), x[..., None]], -1)
    pre = (ext * w.flip(1)).sum(-1)
    if s["bias"] is not None:
        pre = pre + s["bias"]
    y = pre * _sigmoid(pre) if c["silu"] else pre
    s["x_out"][at] = ext[..., 1:].to(t)
    return y.to(t), s["x_out"]


def _prefix(a, b):
    """The states of h_n = a_n h_{n-1} + b_n along the last axis, by doubling."""
    k = 1
    while k < b.shape[-1]:
        b[..., k:] += a[..., k:] * b[..., :-k]
        a[..., k:] = a[..., k:] * a[..., :-k]
        k *= 2
    return b


def _per_channel(m, H):
    """[B,G,S,N] shared by groups of channels -> [B,H,S,N]."""
    return m.float().repeat_interleave(H // m.shape[1], 1)


def _plain_scan(s, do, c):
    u, t, N, G, S = s["u"].float(), s["u"].dtype, c["N"], c["G"], c["S"]
    B, H = u.shape[:2]
    pre = s["dt"].float() + s["dt_bias"][:, None]
    dt = _softplus(pre)
    Bm, C = _per_channel(s["Bm"], H), _per_channel(s["C"], H)
    valid = None
    if s["lengths"] is not None:
        valid = (torch.arange(N, device=u.device) < s["lengths"][:, None])[:, None]
        dt = torch.where(valid, dt, torch.zeros_like(dt))
    A = s["A"][:, :, None]
    a = torch.exp(dt[:, :, None] * A)                          # [B,H,S,N]
    b = (dt * u)[:, :, None] * Bm
    if s["x_in"] is not None:
        b[..., 0] += a[..., 0] * s["x_in"]
    h = _prefix(a.clone() if do == "train" else a, b)
    raw = (h * C).sum(2) + s["D"][:, None] * u
    y = raw
    if s["z"] is not None:
        z = s["z"].float()
        sz = _sigmoid(z)
        y = raw * z * sz
    if valid is not None:
        y = torch.where(valid, y, torch.zeros_like(y))
    if do == "prompt":
        return y.to(t), h[..., -1].contiguous()
    dy = s["dy"].float()
    dz = None
    if s["z"] is not None:
        dz = (dy * raw * sz * (1.0 + z * (1.0 - sz))).to(t)
        dy = dy * z * sz
    dC = (dy[:, :, None] * h).view(B, G, H // G, S, N).sum(2)
    # the adjoint recurrence runs from the end: g_n = C_n dy_n + a_{n+1} g_{n+1}
    back = torch.cat([torch.zeros_like(a[..., :1]), a[..., 1:].flip(-1)], -1)
    g = _prefix(back, (dy[:, :, None] * C).flip(-1)).flip(-1)
    dB = (g * (dt * u)[:, :, None]).view(B, G, H // G, S, N).sum(2)
    gB = (g * Bm).sum(2)
    keep = g * (h - (dt * u)[:, :, None] * Bm)                 # g_n a_n h_{n-1}
    dA = (keep * dt[:, :, None]).sum((0, 3))
    ddt = ((keep * A).sum(2) + gB * u) * _sigmoid(pre)
    du = s["D"][:, None] * dy + gB * dt
    return (y.to(t), du.to(t), ddt.to(t), dA, dB.to(t), dC.to(t), (dy * u).sum((0, 2)), dz, ddt.sum((0, 2)))


def _plain_scan_step(s, c):
    u, t, H, at = s["u"].float(), s["u"].dtype, c["H"], s["slots"].long()
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    Bm, C = (m.float().repeat_interleave(H // c["G"], 1) for m in (s["Bm"], s["C"]))
    x = torch.exp(dt[..., None] * s["A"]) * s["x_in"][at] + (dt * u)[..., None] * Bm
    y = (x * C).sum(-1) + s["D"] * u
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * _sigmoid(z)
    s["x_out"][at] = x
    return y.to(t), s["x_out"]


def _plain_xent(s, do):
    x, w, labels, t = s["x"].float(), s["w"].float(), s["labels"], s["x"].dtype
    logits = x @ w.t()
    m = logits.amax(1, keepdim=True)
    e = torch.exp(logits - m)
    total = e.sum(1, keepdim=True)
    lse = (m + torch.log(total))[:, 0]
    on = labels != IGNORE
    at = torch.where(on, labels, torch.zeros_like(labels))[:, None]
    loss = torch.where(on, lse - torch.gather(logits, 1, at)[:, 0], torch.zeros_like(lse))
    if do == "eval":
        return loss, lse
    del logits
    scale = torch.where(on, s["dloss"], torch.zeros_like(lse))[:, None]
    e *= scale / total
    e.scatter_add_(1, at, -scale)
    return loss, lse, (e @ w).to(t), (e.t() @ x).to(t)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    c, e = case, SIZE[case["io"]]
    if c["op"] == "linear_xent":
        T, D, V = c["T"], c["D"], c["V"]
        io = (T * D + V * D) * e + T * 16
        # the products of the logits (twice where they are not kept), and of each gradient
        return {"bytes": io if c["do"] == "eval" else 2 * io, "flops": 2.0 * T * D * V * (1 if c["do"] == "eval" else 4)}
    B, H, N = c["B"], c["H"], c["N"]
    n = B * H * N
    if c["op"] == "short_conv":
        W = c["W"]
        state = B * H * (W - 1) * e
        par = H * (W + 1) * 4
        moved = {"prompt": 2 * n * e + state * (2 if c["state"] else 1) + par, "step": 2 * n * e + 2 * state + par,
                 "train": 4 * n * e + 2 * par}[c["do"]]
        return {"bytes": moved, "flops": n * (2.0 * W + 5) * (1 if c["do"] != "train" else 4)}
    S, G = c["S"], c["G"]
    rows = 4 if c["gate"] else 3                               # u, dt, y and the gate
    bc = 2 * B * G * S * N * e
    par = H * (S + 2) * 4
    state = B * H * S * 4
    if c["do"] == "train":  # the forward, then the inputs and dy again, and the gradients
        return {"bytes": (rows + rows + rows - 1) * n * e + 3 * bc + 2 * par, "flops": 22.0 * n * S}
    return {"bytes": rows * n * e + bc + par + state * (2 if c["do"] == "step" or c["state"] else 1), "flops": 7.0 * n * S}


# ------------------------------------------------------------------ the definitions, 64 bits


def exact(case, seed):
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in prepare(case, seed).items()}
    with torch.no_grad():
        if case["op"] == "linear_xent":
            return _exact_xent(s, case)
        return (_exact_conv if case["op"] == "short_conv" else _exact_scan)(s, case)


def _exact_xent(s, c):
    x, w, labels = s["x"], s["w"], s["labels"]
    out = []
    dw = torch.zeros_like(w)
    for i in range(0, x.shape[0], 1024):  # tokens are independent but for dw
        xi, li, gi = x[i:i + 1024], labels[i:i + 1024], s["dloss"][i:i + 1024]
        z = torch.mm(xi, w.t().contiguous())
        lse = torch.logsumexp(z, 1)
        hot = torch.zeros_like(z)
        on = li != IGNORE
        hot[on, li[on]] = 1.0
        loss = (lse - (z * hot).sum(1)) * on
        dz = (torch.exp(z - lse[:, None]) - hot) * (gi * on)[:, None]
        if c["do"] == "train":
            dw += torch.mm(dz.t().contiguous(), xi)
        out.append((loss, lse, torch.mm(dz, w) if c["do"] == "train" else None))
    loss, lse = torch.cat([o[0] for o in out]), torch.cat([o[1] for o in out])
    return (loss, lse) if c["do"] == "eval" else (loss, lse, torch.cat([o[2] for o in out]), dw)


def _exact_conv(s, c):
    W, H = c["W"], c["H"]
    bias = s["bias"] if s["bias"] is not None else torch.zeros(H, dtype=torch.float64, device=s["x"].device)

    def act(p):
        return p * torch.sigmoid(p) if c["silu"] else p

    if c["do"] == "step":
        for b, slot in enumerate(s["slots"].tolist()):
            s["x_out"][slot, :, : W - 2] = s["x_in"][slot, :, 1:]
            if W > 1:
                s["x_out"][slot, :, W - 2] = s["x"][b]
        old = s["x_in"][s["slots"].long()]
        p = bias + s["w"][:, 0] * s["x"]
        for i in range(1, W):
            p = p + s["w"][:, i] * old[:, :, W - 1 - i]
        return act(p), s["x_out"]
    B, N = c["B"], c["N"]
    n = [N] * B if s["lengths"] is None else s["lengths"].tolist()
    x = torch.zeros(B, H, W - 1 + N, dtype=torch.float64, device=s["x"].device)
    if s["x_in"] is not None:
        x[:, :, : W - 1] = s["x_in"]
    for b in range(B):
        x[b, :, W - 1: W - 1 + n[b]] = s["x"][b, :, : n[b]]
    kernel = s["w"].flip(1)
    windows = x.unfold(2, W, 1)                               # [B,H,N,W]
    p = (windows * kernel[:, None]).sum(-1) + bias[:, None]
    y = act(p)
    if c["do"] == "prompt":
        last = torch.stack([x[b, :, n[b]: n[b] + W - 1] for b in range(B)])
        for b in range(B):
            y[b, :, n[b]:] = 0
        return y, last
    sg = torch.sigmoid(p)
    d = s["dy"] * (sg + p * sg * (1 - sg)) if c["silu"] else s["dy"]
    ahead = torch.cat([d, torch.zeros(B, H, W - 1, dtype=torch.float64, device=d.device)], 2).unfold(2, W, 1)
    dx = (ahead * s["w"][:, None]).sum(-1)
    dw = (windows * d[..., None]).sum((0, 2)).flip(1)
    return y, dx, dw, d.sum((0, 2)) if c["bias"] else None


def _exact_scan(s, c):
    H, G, S = c["H"], c["G"], c["S"]
    of = torch.arange(H, device=s["u"].device) // (H // G)    # the group of each channel
    A, D = s["A"], s["D"]

    def gate(v, z):
        return v if z is None else v * z * torch.sigmoid(z)

    if c["do"] == "step":
        at = s["slots"].long()
        dt = torch.log1p(torch.exp(s["dt"] + s["dt_bias"]))
        x = torch.exp(dt[..., None] * A) * s["x_in"][at] + (dt * s["u"])[..., None] * s["Bm"][:, of]
        s["x_out"][at] = x
        return gate((x * s["C"][:, of]).sum(-1) + D * s["u"], s["z"]), s["x_out"]
    B, N = c["B"], c["N"]

    def by_time(m):
        return m.movedim(-1, 0).contiguous()

    u, pre = by_time(s["u"]), by_time(s["dt"]) + s["dt_bias"]
    dt = torch.log1p(torch.exp(pre))
    Bm, C = by_time(s["Bm"]), by_time(s["C"])                 # [N,B,G,S]
    z = None if s["z"] is None else by_time(s["z"])
    inside = torch.ones(N, B, dtype=torch.bool, device=u.device)
    if s["lengths"] is not None:
        inside = torch.arange(N, device=u.device)[:, None] < s["lengths"][None]
    x = torch.zeros(B, H, S, dtype=torch.float64, device=u.device) if s["x_in"] is None else s["x_in"].clone()
    train = c["do"] == "train"
    hs = [x] if train else None
    raw = torch.empty_like(u)
    for k in range(0, N, 64):                                 # 64 steps' coefficients at once
        m = min(N, k + 64)
        a = torch.exp(dt[k:m, ..., None] * A)
        b = (dt[k:m] * u[k:m])[..., None] * Bm[k:m][:, :, of]
        part = []
        for j in range(m - k):
            new = torch.addcmul(b[j], a[j], x)
            x = new if s["lengths"] is None else torch.where(inside[k + j][:, None, None], new, x)
            part.append(x)
        raw[k:m] = (torch.stack(part) * C[k:m][:, :, of]).sum(-1)
        if train:
            hs += part
    raw += D * u
    y = gate(raw, z) * inside[..., None]
    if not train:
        return y.movedim(0, -1), x
    dy, dz = by_time(s["dy"]), None
    if z is not None:
        sg = torch.sigmoid(z)
        dz = (dy * raw * (sg + z * sg * (1 - sg))).movedim(0, -1)
        dy = dy * z * sg
    g = torch.zeros_like(x)
    dA = torch.zeros_like(A)
    du, ddt = D * dy, torch.empty_like(u)
    dB, dC = torch.zeros_like(Bm), torch.zeros_like(C)
    for k in range(N - 1, -1, -1):                            # the adjoint of one step at a time
        Bk, Ck = Bm[k][:, of], C[k][:, of]
        g = g + dy[k][..., None] * Ck                         # d loss / d h_k
        dC[k] = (dy[k][..., None] * hs[k + 1]).view(B, G, H // G, S).sum(2)
        dB[k] = (g * (dt[k] * u[k])[..., None]).view(B, G, H // G, S).sum(2)
        a = torch.exp(dt[k][..., None] * A)
        da = g * hs[k] * a                                    # d loss / d (dt A)
        gb = (g * Bk).sum(-1)
        dA += (da * dt[k][..., None]).sum(0)
        ddt[k] = (da * A).sum(-1) + gb * u[k]
        du[k] += gb * dt[k]
        g = g * a
    ddt = ddt * torch.sigmoid(pre)

    def rows(m):
        return m.movedim(0, -1)

    return (rows(y), rows(du), rows(ddt), dA, rows(dB), rows(dC), (dy * u).sum((0, 1)), dz, ddt.sum((0, 1)))
