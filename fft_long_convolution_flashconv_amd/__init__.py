"""Python binding of the gfx950 causal SSM long-convolution library (libh3conv.so).

Thin ctypes marshalling over the C ABI declared in ``include/h3conv.h``: the
functions here check dtype, device and contiguity of torch tensors, pass raw
device pointers and the current HIP stream, and turn status codes into
exceptions.  Every step of the computation runs in the HIP kernels; there is no
host or PyTorch fallback, and importing the binding fails loudly if the
library has not been built.

Operations (after "Hungry Hungry Hippos: Towards Language Modeling with State
Space Models"):
  fft_conv    y = (f * u)[:N] + D u, fused FFT convolution per channel
  ssm_filter  f_k = 2 Re(sum_j C_j exp(dt A_j k) dt B_j)
  state_pass  chunked convolution with the diagonal-SSM state carried
              between chunks (exactly the full-length SSM; 16-bit activations
              pass the state every 64 samples, fp32 convolve chunks of T by FFT)
  h3_mix      out = q * (f * (shift(k) * v) + D * shift(k) * v)

and the layers and loss of a language model with input-dependent state spaces:
  short_conv      y = silu(bias + sum_i w_i x_{t-i}), with short_conv_bwd and,
                  for one token per sequence, short_conv_step
  selective_scan  x_t = exp(d_t A) x_{t-1} + d_t B_t u_t, y = (C_t x_t + D u) silu(z),
                  with selective_scan_bwd and selective_step
  linear_xent     cross entropy of x w^T without the logits in memory, with
                  linear_xent_bwd
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# H3CONV_LIB selects another build of the library (e.g. libh3conv_san.so,
# host code under AddressSanitizer, for host-only checks)
LIB_PATH = os.environ.get("H3CONV_LIB") or os.path.join(HERE, "libh3conv.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_NO_DEVICE, ERR_HIP, ERR_WORKSPACE = range(6)
F32, F16, BF16 = 0, 1, 2
OP_FFT_CONV, OP_STATE_PASS, OP_H3_MIX, OP_H3_MIX_MH = 0, 1, 2, 3
MAX_FUSED_N = 8192
MAX_FUSED_N_16BIT = 16384
MAX_STATE = 64
MAX_TAPS = 4

_IO = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
_lib = None

EXPORTS = ("h3conv_fft_conv", "h3conv_fft_conv_bidir", "h3conv_fft_conv_bwd", "h3conv_ssm_filter", "h3conv_state_pass", "h3conv_state_pass_noalloc",
           "h3conv_ssm_step", "h3conv_h3_mix", "h3conv_h3_mix_mh", "h3conv_workspace_size", "h3conv_status_string", "h3conv_version",
           "h3conv_short_conv", "h3conv_short_conv_bwd", "h3conv_short_conv_bwd_workspace_size", "h3conv_short_conv_step",
           "h3conv_selective_scan", "h3conv_selective_saved_size", "h3conv_selective_scan_bwd",
           "h3conv_selective_scan_bwd_workspace_size", "h3conv_selective_step",
           "h3conv_linear_xent", "h3conv_linear_xent_bwd", "h3conv_linear_xent_workspace_size")
NOALLOC_WORKSPACE_BYTES = 128 * 1024 * 1024


class H3ConvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, status_string(status), status))


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libh3conv.so (built by ``build.py``); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("libh3conv.so not built: run `python fft_long_convolution_flashconv_amd/build.py` "
                           "(looked for %s)" % path)
    lib = ctypes.CDLL(path)
    P, I64, I, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    lib.h3conv_fft_conv.argtypes = [P, P, P, P, I64, I64, I64, I, P]
    lib.h3conv_fft_conv_bidir.argtypes = [P, P, P, P, P, I64, I64, I64, I, P]
    lib.h3conv_fft_conv_bwd.argtypes = [P, P, P, P, P, P, P, I64, I64, I64, I, P]
    lib.h3conv_ssm_filter.argtypes = [P, P, P, P, P, I64, I64, I64, P]
    lib.h3conv_state_pass.argtypes = [P, P, P, P, P, P, P, P, P, I64, I64, I64, I64, I64, I, P, SZ, P]
    lib.h3conv_state_pass_noalloc.argtypes = [P, P, P, P, P, P, P, P, P, I64, I64, I64, I64, I64, I, P]
    lib.h3conv_ssm_step.argtypes = [P, P, P, P, P, P, P, P, I64, I64, I64, I64, I, P]
    lib.h3conv_h3_mix.argtypes = [P, P, P, P, P, P, P, I64, I64, I64, I64, I, P, ctypes.c_size_t, P]
    lib.h3conv_h3_mix_mh.argtypes = [P, P, P, P, P, P, P, I64, I64, I64, I64, I64, I, P, SZ, P]
    lib.h3conv_workspace_size.argtypes = [I, I64, I64, I64, I64, I64]
    lib.h3conv_workspace_size.restype = SZ
    lib.h3conv_status_string.argtypes = [I]
    lib.h3conv_status_string.restype = ctypes.c_char_p
    lib.h3conv_version.restype = I
    for name in ("h3conv_fft_conv", "h3conv_fft_conv_bidir", "h3conv_fft_conv_bwd", "h3conv_ssm_filter", "h3conv_state_pass", "h3conv_state_pass_noalloc",
                 "h3conv_ssm_step", "h3conv_h3_mix", "h3conv_h3_mix_mh"):
        getattr(lib, name).restype = I
    lib.h3conv_short_conv.argtypes = [P] * 7 + [I64] * 4 + [I, I, P]
    lib.h3conv_short_conv_bwd.argtypes = [P] * 11 + [I64] * 4 + [I, I, P, SZ, P]
    lib.h3conv_short_conv_step.argtypes = [P] * 7 + [I64] * 4 + [I, I, P]
    lib.h3conv_selective_scan.argtypes = [P] * 13 + [I64] * 5 + [I, I, P]
    lib.h3conv_selective_scan_bwd.argtypes = [P] * 21 + [I64] * 5 + [I, I, P, SZ, P]
    lib.h3conv_selective_step.argtypes = [P] * 12 + [I64] * 5 + [I, I, P]
    lib.h3conv_linear_xent.argtypes = [P, P, P, I64, P, P, I64, I64, I64, I, P, SZ, P]
    lib.h3conv_linear_xent_bwd.argtypes = [P, P, P, I64, P, P, P, P, I64, I64, I64, I, P, SZ, P]
    for name in ("h3conv_short_conv", "h3conv_short_conv_bwd", "h3conv_short_conv_step", "h3conv_selective_scan",
                 "h3conv_selective_scan_bwd", "h3conv_selective_step", "h3conv_linear_xent", "h3conv_linear_xent_bwd"):
        getattr(lib, name).restype = I
    lib.h3conv_short_conv_bwd_workspace_size.argtypes = [I64] * 4
    lib.h3conv_selective_saved_size.argtypes = [I64] * 4
    lib.h3conv_selective_scan_bwd_workspace_size.argtypes = [I64] * 5
    lib.h3conv_linear_xent_workspace_size.argtypes = [I64, I64, I64, I, I]
    for name in ("h3conv_short_conv_bwd_workspace_size", "h3conv_selective_saved_size",
                 "h3conv_selective_scan_bwd_workspace_size", "h3conv_linear_xent_workspace_size"):
        getattr(lib, name).restype = SZ
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().h3conv_status_string(int(status)).decode()


def workspace_size(op: int, B: int = 0, H: int = 0, N: int = 0, S: int = 0, T: int = 0) -> int:
    n = load().h3conv_workspace_size(int(op), int(B), int(H), int(N), int(S), int(T))
    if n == ctypes.c_size_t(-1).value:
        raise H3ConvError(ERR_UNSUPPORTED, "workspace_size")
    return int(n)


def _check(status: int, where: str) -> None:
    if status != OK:
        raise H3ConvError(status, where)


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t: torch.Tensor, name: str, dtype=None, shape=None):
    """Type, dtype, exact shape and contiguity of one tensor argument (the
    device is checked for all arguments of a call together, by _same_device)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(int(x) for x in shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _same_device(**ts):
    """Every tensor on one HIP device, which is the current one (the library
    launches on the current device and its current stream)."""
    devs = {n: t.device for n, t in ts.items() if t is not None}
    for n, d in devs.items():
        if d.type != "cuda":
            raise ValueError("%s must be on a HIP device, got %s" % (n, d))
    if len(set(devs.values())) > 1:
        raise ValueError("all tensors must be on one device, got %s" % devs)
    d = next(iter(devs.values()))
    cur = torch.cuda.current_device()
    if d.index is not None and d.index != cur:
        raise ValueError("tensors are on %s but the current device is cuda:%d" % (d, cur))


def _cplx_param(t: torch.Tensor, name: str, shape=None) -> torch.Tensor:
    """Complex parameters are accepted as complex64 [...] or float32 [..., 2]."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.is_complex():
        if t.dtype != torch.complex64:
            raise ValueError("%s must be complex64 or float32 [..., 2], got %s" % (name, t.dtype))
        t = torch.view_as_real(t)
    _need(t, name, torch.float32, None if shape is None else tuple(shape) + (2,))
    if t.dim() < 1 or t.shape[-1] != 2:
        raise ValueError("%s must be complex or have a trailing dimension of 2" % name)
    return t


def _io(t: torch.Tensor, name: str) -> int:
    if t.dtype not in _IO:
        raise ValueError("%s must be float32, float16 or bfloat16, got %s" % (name, t.dtype))
    return _IO[t.dtype]


def fft_conv(u: torch.Tensor, f: torch.Tensor, D: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """y[b,h,:] = causal (f[h] * u[b,h])[:N] + D[h] u[b,h]; u [B,H,N] f32/f16/bf16, f [H,N] f32, D [H] f32."""
    _need(u, "u")
    io = _io(u, "u")
    if u.dim() != 3:
        raise ValueError("u must be [B,H,N], got %s" % (tuple(u.shape),))
    B, H, N = u.shape
    _need(f, "f", torch.float32, (H, N)); _need(D, "D", torch.float32, (H,))
    if out is not None:
        _need(out, "out", u.dtype, (B, H, N))
    _same_device(u=u, f=f, D=D, out=out)
    y = torch.empty_like(u) if out is None else out
    _check(load().h3conv_fft_conv(_ptr(u), _ptr(f), _ptr(D), _ptr(y), B, H, N, io, _stream()),
           "h3conv_fft_conv")
    return y


def fft_conv_bidir(u: torch.Tensor, f: torch.Tensor, g: torch.Tensor, D: torch.Tensor,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """Bidirectional copies: y = causal (f * u) + anti-causal (g * u) + D u;
    u [B,H,N] f32/f16/bf16, f, g [H,N] f32, D [H] f32."""
    _need(u, "u")
    io = _io(u, "u")
    if u.dim() != 3:
        raise ValueError("u must be [B,H,N], got %s" % (tuple(u.shape),))
    B, H, N = u.shape
    _need(f, "f", torch.float32, (H, N)); _need(g, "g", torch.float32, (H, N)); _need(D, "D", torch.float32, (H,))
    if out is not None:
        _need(out, "out", u.dtype, (B, H, N))
    _same_device(u=u, f=f, g=g, D=D, out=out)
    y = torch.empty_like(u) if out is None else out
    _check(load().h3conv_fft_conv_bidir(_ptr(u), _ptr(f), _ptr(g), _ptr(D), _ptr(y), B, H, N, io, _stream()),
           "h3conv_fft_conv_bidir")
    return y


def fft_conv_bwd(u: torch.Tensor, f: torch.Tensor, D: torch.Tensor, dy: torch.Tensor, du=None, df=None, dD=None):
    """Gradients of y = fft_conv(u, f, D) for an upstream gradient dy.

    Returns (du [B,H,N] like u, df [H,N] f32, dD [H] f32); df and dD are
    summed over the batch."""
    _need(u, "u")
    io = _io(u, "u")
    if u.dim() != 3:
        raise ValueError("u must be [B,H,N], got %s" % (tuple(u.shape),))
    B, H, N = u.shape
    _need(f, "f", torch.float32, (H, N)); _need(D, "D", torch.float32, (H,))
    _need(dy, "dy", u.dtype, (B, H, N))
    if du is not None:
        _need(du, "du", u.dtype, (B, H, N))
    if df is not None:
        _need(df, "df", torch.float32, (H, N))
    if dD is not None:
        _need(dD, "dD", torch.float32, (H,))
    _same_device(u=u, f=f, D=D, dy=dy, du=du, df=df, dD=dD)
    du = torch.empty_like(u) if du is None else du
    df = torch.empty(H, N, device=u.device, dtype=torch.float32) if df is None else df
    dD = torch.empty(H, device=u.device, dtype=torch.float32) if dD is None else dD
    _check(load().h3conv_fft_conv_bwd(_ptr(u), _ptr(f), _ptr(D), _ptr(dy), _ptr(du), _ptr(df), _ptr(dD),
                                       B, H, N, io, _stream()),
           "h3conv_fft_conv_bwd")
    return du, df, dD


def ssm_filter(A: torch.Tensor, Bm: torch.Tensor, C: torch.Tensor, dt: torch.Tensor, N: int,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """f[h,k] = 2 Re(sum_j C exp(dt A k) dt B), k < N; A, Bm, C [H,S] complex, dt [H] f32."""
    A = _cplx_param(A, "A")
    if A.dim() != 3:
        raise ValueError("A must be [H,S] complex")
    H, S = A.shape[0], A.shape[1]
    Bm = _cplx_param(Bm, "Bm", (H, S)); C = _cplx_param(C, "C", (H, S))
    _need(dt, "dt", torch.float32, (H,))
    if out is not None:
        _need(out, "out", torch.float32, (H, int(N)))
    _same_device(A=A, Bm=Bm, C=C, dt=dt, out=out)
    f = torch.empty(H, int(N), device=A.device, dtype=torch.float32) if out is None else out
    _check(load().h3conv_ssm_filter(_ptr(A), _ptr(Bm), _ptr(C), _ptr(dt), _ptr(f), H, S, int(N), _stream()),
           "h3conv_ssm_filter")
    return f


def _sp_args(u, A, Bm, C, dt, D, x_in, out, workspace):
    _need(u, "u")
    io = _io(u, "u")
    if u.dim() != 3:
        raise ValueError("u must be [B,H,N], got %s" % (tuple(u.shape),))
    B, H, N = u.shape
    A = _cplx_param(A, "A")
    if A.dim() != 3 or A.shape[0] != H:
        raise ValueError("A must be [H,S] complex with H = %d, got %s" % (H, tuple(A.shape)))
    S = A.shape[1]
    Bm = _cplx_param(Bm, "Bm", (H, S)); C = _cplx_param(C, "C", (H, S))
    _need(dt, "dt", torch.float32, (H,)); _need(D, "D", torch.float32, (H,))
    if x_in is not None:
        x_in = _cplx_param(x_in, "x_in", (B, H, S))
    if out is not None:
        _need(out, "out", u.dtype, (B, H, N))
    if workspace is not None:
        _need(workspace, "workspace")
    _same_device(u=u, A=A, Bm=Bm, C=C, dt=dt, D=D, x_in=x_in, out=out, workspace=workspace)
    return io, B, H, N, S, A, Bm, C, x_in


def state_pass(u, A, Bm, C, dt, D, T: int, x_in=None, return_state: bool = False,
               out=None, workspace=None):
    """Full-length diagonal SSM over u [B,H,N] by chunks of T (state carried between chunks).

    Returns y, or (y, x_out) with x_out [B,H,S] complex64 if ``return_state``.
    """
    io, B, H, N, S, A, Bm, C, x_in = _sp_args(u, A, Bm, C, dt, D, x_in, out, workspace)
    y = torch.empty_like(u) if out is None else out
    x_out = torch.empty(B, H, S, 2, device=u.device, dtype=torch.float32) if return_state else None
    need = workspace_size(OP_STATE_PASS, B, H, N, S, T) if N > 0 else 0
    ws = workspace
    if ws is None or ws.numel() * ws.element_size() < need:
        ws = torch.empty(max(need, 1), device=u.device, dtype=torch.uint8)
    _check(load().h3conv_state_pass(_ptr(u), _ptr(A), _ptr(Bm), _ptr(C), _ptr(dt), _ptr(D), _ptr(x_in),
                                     _ptr(x_out), _ptr(y), B, H, N, S, int(T), io, _ptr(ws),
                                     ws.numel() * ws.element_size(), _stream()),
           "h3conv_state_pass")
    if return_state:
        return y, torch.view_as_complex(x_out)
    return y


def state_pass_noalloc(u, A, Bm, C, dt, D, T: int, out, x_in=None, x_out=None):
    """state_pass through h3conv_state_pass_noalloc: no workspace, no device
    allocation in the library or here (``out``, and ``x_out`` [B,H,S,2]
    float32 if the final state is wanted, are the caller's).  The library's
    static scratch array of NOALLOC_WORKSPACE_BYTES per device is shared by
    all such calls on a device: calls that overlap in time race."""
    io, B, H, N, S, A, Bm, C, x_in = _sp_args(u, A, Bm, C, dt, D, x_in, out, None)
    if out is None:
        raise ValueError("out is required (this entry point allocates nothing)")
    if x_out is not None:
        x_out = _cplx_param(x_out, "x_out", (B, H, S))
        _same_device(u=u, x_out=x_out)
    _check(load().h3conv_state_pass_noalloc(_ptr(u), _ptr(A), _ptr(Bm), _ptr(C), _ptr(dt), _ptr(D),
                                             _ptr(x_in), _ptr(x_out), _ptr(out), B, H, N, S, int(T), io,
                                             _stream()),
           "h3conv_state_pass_noalloc")
    return out


def ssm_step(u, A, Bm, C, dt, D, x, out=None):
    """K recurrent steps per row: x <- exp(dt A) x + dt B u_t, y_t = 2 Re(C.x) + D u_t.

    u [B,H,K] f32/f16/bf16; A, Bm, C [H,S] complex; dt, D [H]; x [B,H,S]
    complex64 (or float32 [B,H,S,2]), updated in place.  Returns y [B,H,K]."""
    _need(u, "u")
    io = _io(u, "u")
    if u.dim() != 3:
        raise ValueError("u must be [B,H,K], got %s" % (tuple(u.shape),))
    B, H, K = u.shape
    A = _cplx_param(A, "A")
    if A.dim() != 3 or A.shape[0] != H:
        raise ValueError("A must be [H,S] complex with H = %d, got %s" % (H, tuple(A.shape)))
    S = A.shape[1]
    Bm = _cplx_param(Bm, "Bm", (H, S)); C = _cplx_param(C, "C", (H, S))
    _need(dt, "dt", torch.float32, (H,)); _need(D, "D", torch.float32, (H,))
    xv = _cplx_param(x, "x", (B, H, S))
    if out is not None:
        _need(out, "out", u.dtype, (B, H, K))
    _same_device(u=u, A=A, Bm=Bm, C=C, dt=dt, D=D, x=xv, out=out)
    y = torch.empty_like(u) if out is None else out
    _check(load().h3conv_ssm_step(_ptr(u), _ptr(A), _ptr(Bm), _ptr(C), _ptr(dt), _ptr(D), _ptr(xv), _ptr(y),
                                   B, H, K, S, io, _stream()),
           "h3conv_ssm_step")
    return y


def h3_mix(q, k, v, w, f, D, out=None, workspace=None):
    """out = q * ((f * m)[:N] + D m), m = shift(k) * v; q,k,v [B,N,Dm], w [Dm,L], f [Dm,N], D [Dm].

    16-bit activations stage m and z channel-major in a workspace
    (allocated here when not given)."""
    _need(q, "q")
    io = _io(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be [B,N,Dm], got %s" % (tuple(q.shape),))
    B, N, Dm = q.shape
    _need(k, "k", q.dtype, (B, N, Dm)); _need(v, "v", q.dtype, (B, N, Dm))
    _need(w, "w", torch.float32)
    if w.dim() != 2 or w.shape[0] != Dm:
        raise ValueError("w must be [Dm,L] with Dm = %d, got %s" % (Dm, tuple(w.shape)))
    L = w.shape[1]
    _need(f, "f", torch.float32, (Dm, N)); _need(D, "D", torch.float32, (Dm,))
    if out is not None:
        _need(out, "out", q.dtype, (B, N, Dm))
    if workspace is not None:
        _need(workspace, "workspace")
    _same_device(q=q, k=k, v=v, w=w, f=f, D=D, out=out, workspace=workspace)
    o = torch.empty_like(q) if out is None else out
    ws, nws = None, 0
    if q.dtype != torch.float32:
        ws = workspace if workspace is not None else torch.empty(
            max(workspace_size(OP_H3_MIX, B, Dm, N), 1), dtype=torch.uint8, device=q.device)
        nws = ws.numel() * ws.element_size()
    _check(load().h3conv_h3_mix(_ptr(q), _ptr(k), _ptr(v), _ptr(w), _ptr(f), _ptr(D), _ptr(o), B, N, Dm, L,
                                io, _ptr(ws) if ws is not None else None, nws, _stream()),
           "h3conv_h3_mix")
    return o


def h3_mix_mh(q, k, v, w, f, D, dh: int, out=None, workspace=None):
    """Multi-head H3 mixing, head dimension dh: per head, m = shift(k)^T v
    (outer product), z = (f * m)[:N] + D m per state entry, out_j = sum_i q_i z_ij.
    q, k, v [B,N,Dm]; w [Dm,L]; f [Dm*dh, N]; D [Dm*dh].  The workspace (two
    channel-major stagings of the B x Dm*dh state rows) is allocated here
    when not given."""
    _need(q, "q")
    io = _io(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be [B,N,Dm], got %s" % (tuple(q.shape),))
    B, N, Dm = q.shape
    dh = int(dh)
    if dh < 1 or Dm % dh != 0:
        raise ValueError("dh must divide Dm = %d" % Dm)
    _need(k, "k", q.dtype, (B, N, Dm)); _need(v, "v", q.dtype, (B, N, Dm))
    _need(w, "w", torch.float32)
    if w.dim() != 2 or w.shape[0] != Dm:
        raise ValueError("w must be [Dm,L] with Dm = %d, got %s" % (Dm, tuple(w.shape)))
    L = w.shape[1]
    _need(f, "f", torch.float32, (Dm * dh, N)); _need(D, "D", torch.float32, (Dm * dh,))
    if out is not None:
        _need(out, "out", q.dtype, (B, N, Dm))
    if workspace is not None:
        _need(workspace, "workspace")
    _same_device(q=q, k=k, v=v, w=w, f=f, D=D, out=out, workspace=workspace)
    o = torch.empty_like(q) if out is None else out
    need = workspace_size(OP_H3_MIX_MH, B, Dm, N, dh) * (2 if io == F32 else 1)
    ws = workspace if workspace is not None else torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _check(load().h3conv_h3_mix_mh(_ptr(q), _ptr(k), _ptr(v), _ptr(w), _ptr(f), _ptr(D), _ptr(o), B, N, Dm, dh, L,
                                   io, _ptr(ws), ws.numel() * ws.element_size(), _stream()),
           "h3conv_h3_mix_mh")
    return o


# ---------------------------------------------------------------------------
# Layers and loss of a language model with input-dependent state spaces.

def _size(name: str, *args) -> int:
    n = getattr(load(), name)(*args)
    if n == ctypes.c_size_t(-1).value:
        raise H3ConvError(ERR_UNSUPPORTED, name)
    return int(n)


def _scratch(workspace, need: int, device) -> torch.Tensor:
    """The caller's workspace where it is large enough, else a new one."""
    if workspace is not None and workspace.numel() * workspace.element_size() >= need:
        return workspace
    return torch.empty(max(need, 1), device=device, dtype=torch.uint8)


def _arg(t, name: str, dtype, shape, optional: bool = True):
    """One tensor argument; None passes where it is optional."""
    if t is None:
        if not optional:
            raise TypeError("%s is required" % name)
        return
    _need(t, name, dtype, shape)


def _conv_args(x, w, bias, dims: int):
    _need(x, "x")
    io = _io(x, "x")
    if x.dim() != dims:
        raise ValueError("x must be %s, got %s" % ("[B,H,N]" if dims == 3 else "[B,H]", tuple(x.shape)))
    H = x.shape[1]
    _need(w, "w", torch.float32)
    if w.dim() != 2 or w.shape[0] != H or w.shape[1] < 1:
        raise ValueError("w must be [H,W] with H = %d, got %s" % (H, tuple(w.shape)))
    _arg(bias, "bias", torch.float32, (H,))
    return io, H, w.shape[1]


def short_conv(x, w, bias=None, silu: bool = True, x_in=None, lengths=None, return_state: bool = False, out=None):
    """y[b,h,t] = silu(bias[h] + sum_i w[h,i] x[b,h,t-i]) (without ``silu`` the sum itself).

    x [B,H,N] f32/f16/bf16; w [H,W] f32, W <= MAX_TAPS; bias [H] f32; x_in
    [B,H,W-1] like x, the inputs before the row, oldest first (zeros if None);
    lengths [B] int32, valid steps of every row.  Returns y, or (y, x_out) with
    the last W-1 inputs of every row if ``return_state``."""
    io, H, W = _conv_args(x, w, bias, 3)
    B, N = x.shape[0], x.shape[2]
    _arg(x_in, "x_in", x.dtype, (B, H, W - 1))
    _arg(lengths, "lengths", torch.int32, (B,))
    _arg(out, "out", x.dtype, (B, H, N))
    _same_device(x=x, w=w, bias=bias, x_in=x_in, lengths=lengths, out=out)
    y = torch.empty_like(x) if out is None else out
    x_out = torch.empty(B, H, W - 1, device=x.device, dtype=x.dtype) if return_state else None
    _check(load().h3conv_short_conv(_ptr(x), _ptr(w), _ptr(bias), _ptr(x_in), _ptr(lengths), _ptr(y), _ptr(x_out),
                                    B, H, N, W, int(bool(silu)), io, _stream()),
           "h3conv_short_conv")
    return (y, x_out) if return_state else y


def short_conv_bwd(x, w, dy, bias=None, silu: bool = True, x_in=None, lengths=None, dx_out=None, workspace=None):
    """Gradients of y (and x_out) = short_conv(x, w, bias, ...) for dy [B,H,N] and dx_out [B,H,W-1] (or None).

    Returns (dx [B,H,N], dw [H,W] f32, dbias [H] f32, dx_in [B,H,W-1]); dbias
    is None without a bias, dx_in without an x_in."""
    io, H, W = _conv_args(x, w, bias, 3)
    B, N = x.shape[0], x.shape[2]
    _arg(dy, "dy", x.dtype, (B, H, N), optional=False)
    _arg(x_in, "x_in", x.dtype, (B, H, W - 1))
    _arg(lengths, "lengths", torch.int32, (B,))
    _arg(dx_out, "dx_out", x.dtype, (B, H, W - 1))
    if workspace is not None:
        _need(workspace, "workspace")
    _same_device(x=x, w=w, dy=dy, bias=bias, x_in=x_in, lengths=lengths, dx_out=dx_out, workspace=workspace)
    dx = torch.empty_like(x)
    dw = torch.empty_like(w)
    dbias = torch.empty_like(bias) if bias is not None else None
    dx_in = torch.empty_like(x_in) if x_in is not None else None
    ws = _scratch(workspace, _size("h3conv_short_conv_bwd_workspace_size", B, H, N, W), x.device)
    _check(load().h3conv_short_conv_bwd(_ptr(x), _ptr(w), _ptr(bias), _ptr(x_in), _ptr(lengths), _ptr(dy),
                                        _ptr(dx_out), _ptr(dx), _ptr(dw), _ptr(dbias), _ptr(dx_in), B, H, N, W,
                                        int(bool(silu)), io, _ptr(ws), ws.numel() * ws.element_size(), _stream()),
           "h3conv_short_conv_bwd")
    return dx, dw, dbias, dx_in


def short_conv_step(x, w, state, bias=None, silu: bool = True, slots=None, state_out=None, out=None):
    """short_conv for one token of each sequence.

    x [B,H]; state [P,H,W-1] like x, a pool of saved inputs, updated in place
    (or into ``state_out``, of which only the slots in use are written); slots
    [B] int32, the slot of each sequence (sequence b in slot b if None).  A
    slot outside the pool marks an idle row: its output is zero.  Returns y [B,H]."""
    io, H, W = _conv_args(x, w, bias, 2)
    B = x.shape[0]
    P = state.shape[0] if isinstance(state, torch.Tensor) and state.dim() == 3 else 0
    _arg(state, "state", x.dtype, (P, H, W - 1), optional=False)
    _arg(state_out, "state_out", x.dtype, (P, H, W - 1))
    _arg(slots, "slots", torch.int32, (B,))
    _arg(out, "out", x.dtype, (B, H))
    _same_device(x=x, w=w, bias=bias, slots=slots, state=state, state_out=state_out, out=out)
    y = torch.empty_like(x) if out is None else out
    to = state if state_out is None else state_out
    _check(load().h3conv_short_conv_step(_ptr(x), _ptr(w), _ptr(bias), _ptr(slots), _ptr(state), _ptr(to), _ptr(y),
                                         B, H, P, W, int(bool(silu)), io, _stream()),
           "h3conv_short_conv_step")
    return y


def _scan_args(u, dt, A, Bm, C, D, z, dt_bias, dims: int):
    _need(u, "u")
    io = _io(u, "u")
    if u.dim() != dims:
        raise ValueError("u must be %s, got %s" % ("[B,H,N]" if dims == 3 else "[B,H]", tuple(u.shape)))
    B, H = u.shape[:2]
    _arg(dt, "dt", u.dtype, u.shape, optional=False)
    _need(A, "A", torch.float32)
    if A.dim() != 2 or A.shape[0] != H or A.shape[1] < 1:
        raise ValueError("A must be [H,S] with H = %d, got %s" % (H, tuple(A.shape)))
    S = A.shape[1]
    _need(Bm, "Bm", u.dtype)
    if Bm.dim() != dims + 1 or Bm.shape[1] < 1 or H % Bm.shape[1] != 0:
        raise ValueError("Bm must be %s with G dividing H = %d, got %s"
                         % ("[B,G,S,N]" if dims == 3 else "[B,G,S]", H, tuple(Bm.shape)))
    G = Bm.shape[1]
    bc = (B, G, S) + tuple(u.shape[2:])
    _need(Bm, "Bm", u.dtype, bc)
    _arg(C, "C", u.dtype, bc, optional=False)
    _arg(D, "D", torch.float32, (H,))
    _arg(z, "z", u.dtype, u.shape)
    _arg(dt_bias, "dt_bias", torch.float32, (H,))
    return io, B, H, S, G


def selective_scan(u, dt, A, Bm, C, D=None, z=None, dt_bias=None, softplus: bool = True, x_in=None, lengths=None,
                   return_state: bool = False, return_saved: bool = False, out=None):
    """Selective state-space scan: d_t = softplus(dt_t + dt_bias), x_t = exp(d_t A) x_{t-1} + d_t B_t u_t,
    y_t = (C_t . x_t + D u_t) silu(z_t).

    u, dt, z [B,H,N] f32/f16/bf16; A [H,S] f32; Bm, C [B,G,S,N] like u, shared
    by the H/G channels of a group; D, dt_bias [H] f32; x_in [B,H,S] f32;
    lengths [B] int32, valid steps of every row.  Returns y, followed by the
    final state [B,H,S] f32 if ``return_state`` and by the saved states that
    selective_scan_bwd needs if ``return_saved``."""
    io, B, H, S, G = _scan_args(u, dt, A, Bm, C, D, z, dt_bias, 3)
    N = u.shape[2]
    _arg(x_in, "x_in", torch.float32, (B, H, S))
    _arg(lengths, "lengths", torch.int32, (B,))
    _arg(out, "out", u.dtype, (B, H, N))
    _same_device(u=u, dt=dt, A=A, Bm=Bm, C=C, D=D, z=z, dt_bias=dt_bias, x_in=x_in, lengths=lengths, out=out)
    y = torch.empty_like(u) if out is None else out
    x_out = torch.empty(B, H, S, device=u.device, dtype=torch.float32) if return_state else None
    saved = None
    if return_saved:
        saved = torch.empty(_size("h3conv_selective_saved_size", B, H, N, S) // 4, device=u.device, dtype=torch.float32)
    _check(load().h3conv_selective_scan(_ptr(u), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(C), _ptr(D), _ptr(z), _ptr(dt_bias),
                                        _ptr(x_in), _ptr(lengths), _ptr(y), _ptr(x_out), _ptr(saved), B, H, N, S, G,
                                        int(bool(softplus)), io, _stream()),
           "h3conv_selective_scan")
    if not (return_state or return_saved):
        return y
    return (y,) + ((x_out,) if return_state else ()) + ((saved,) if return_saved else ())


class SelectiveScanGrads(NamedTuple):
    """Gradients of selective_scan; None for an input that was not given."""
    du: torch.Tensor
    ddt: torch.Tensor
    dA: torch.Tensor
    dB: torch.Tensor
    dC: torch.Tensor
    dD: Optional[torch.Tensor]
    dz: Optional[torch.Tensor]
    ddt_bias: Optional[torch.Tensor]
    dx_in: torch.Tensor


def selective_scan_bwd(u, dt, A, Bm, C, dy, saved, D=None, z=None, dt_bias=None, softplus: bool = True, lengths=None,
                       dx_out=None, workspace=None) -> SelectiveScanGrads:
    """Gradients of selective_scan (same arguments, ``saved`` as it returned it) for dy [B,H,N] and
    dx_out [B,H,S] f32 (upstream of the final state, or None)."""
    io, B, H, S, G = _scan_args(u, dt, A, Bm, C, D, z, dt_bias, 3)
    N = u.shape[2]
    _arg(dy, "dy", u.dtype, (B, H, N), optional=False)
    _arg(saved, "saved", torch.float32, (_size("h3conv_selective_saved_size", B, H, N, S) // 4,), optional=False)
    _arg(lengths, "lengths", torch.int32, (B,))
    _arg(dx_out, "dx_out", torch.float32, (B, H, S))
    if workspace is not None:
        _need(workspace, "workspace")
    _same_device(u=u, dt=dt, A=A, Bm=Bm, C=C, D=D, z=z, dt_bias=dt_bias, dy=dy, saved=saved, lengths=lengths,
                 dx_out=dx_out, workspace=workspace)
    g = SelectiveScanGrads(
        torch.empty_like(u), torch.empty_like(dt), torch.empty_like(A), torch.empty_like(Bm), torch.empty_like(C),
        None if D is None else torch.empty_like(D), None if z is None else torch.empty_like(z),
        None if dt_bias is None else torch.empty_like(dt_bias),
        torch.empty(B, H, S, device=u.device, dtype=torch.float32))
    ws = _scratch(workspace, _size("h3conv_selective_scan_bwd_workspace_size", B, H, N, S, G), u.device)
    _check(load().h3conv_selective_scan_bwd(
        _ptr(u), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(C), _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(lengths), _ptr(saved),
        _ptr(dy), _ptr(dx_out), _ptr(g.du), _ptr(g.ddt), _ptr(g.dA), _ptr(g.dB), _ptr(g.dC), _ptr(g.dD), _ptr(g.dz),
        _ptr(g.ddt_bias), _ptr(g.dx_in), B, H, N, S, G, int(bool(softplus)), io, _ptr(ws),
        ws.numel() * ws.element_size(), _stream()),
        "h3conv_selective_scan_bwd")
    return g


def selective_step(u, dt, A, Bm, C, x, D=None, z=None, dt_bias=None, softplus: bool = True, slots=None, x_out=None,
                   out=None):
    """selective_scan for one token of each sequence.

    u, dt, z [B,H]; Bm, C [B,G,S]; x [P,H,S] f32, a pool of states, updated in
    place (or into ``x_out``, of which only the slots in use are written);
    slots [B] int32, the slot of each sequence (sequence b in slot b if None).
    A slot outside the pool marks an idle row: its output is zero.  Returns y [B,H]."""
    io, B, H, S, G = _scan_args(u, dt, A, Bm, C, D, z, dt_bias, 2)
    P = x.shape[0] if isinstance(x, torch.Tensor) and x.dim() == 3 else 0
    _arg(x, "x", torch.float32, (P, H, S), optional=False)
    _arg(x_out, "x_out", torch.float32, (P, H, S))
    _arg(slots, "slots", torch.int32, (B,))
    _arg(out, "out", u.dtype, (B, H))
    _same_device(u=u, dt=dt, A=A, Bm=Bm, C=C, D=D, z=z, dt_bias=dt_bias, slots=slots, x=x, x_out=x_out, out=out)
    y = torch.empty_like(u) if out is None else out
    to = x if x_out is None else x_out
    _check(load().h3conv_selective_step(_ptr(u), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(C), _ptr(D), _ptr(z), _ptr(dt_bias),
                                        _ptr(slots), _ptr(x), _ptr(to), _ptr(y), B, H, P, S, G, int(bool(softplus)),
                                        io, _stream()),
           "h3conv_selective_step")
    return y


def _xent_args(x, w, labels):
    _need(x, "x")
    io = _io(x, "x")
    if x.dim() != 2 or x.shape[1] < 1:
        raise ValueError("x must be [T,D], got %s" % (tuple(x.shape),))
    T, D = x.shape
    _need(w, "w", x.dtype)
    if w.dim() != 2 or w.shape[1] != D or w.shape[0] < 1:
        raise ValueError("w must be [V,D] with D = %d, got %s" % (D, tuple(w.shape)))
    _arg(labels, "labels", torch.int64, (T,), optional=False)
    return io, T, D, w.shape[0]


def linear_xent(x, w, labels, ignore_index: int = -100, return_lse: bool = False, workspace=None):
    """Cross entropy of the logits x w^T per token, without the logits in memory.

    x [T,D], w [V,D] f32/f16/bf16; labels [T] int64.  Returns loss [T] f32 (0
    where the label is ignore_index or outside 0 .. V-1), or (loss, lse)."""
    io, T, D, V = _xent_args(x, w, labels)
    if workspace is not None:
        _need(workspace, "workspace")
    _same_device(x=x, w=w, labels=labels, workspace=workspace)
    loss = torch.empty(T, device=x.device, dtype=torch.float32)
    lse = torch.empty(T, device=x.device, dtype=torch.float32)
    ws = _scratch(workspace, _size("h3conv_linear_xent_workspace_size", T, D, V, io, 0), x.device)
    _check(load().h3conv_linear_xent(_ptr(x), _ptr(w), _ptr(labels), int(ignore_index), _ptr(loss), _ptr(lse), T, D, V,
                                     io, _ptr(ws), ws.numel() * ws.element_size(), _stream()),
           "h3conv_linear_xent")
    return (loss, lse) if return_lse else loss


def linear_xent_bwd(x, w, labels, lse, dloss, ignore_index: int = -100, workspace=None):
    """Gradients (dx [T,D], dw [V,D], like x) of linear_xent for dloss [T] f32; lse [T] as it returned it."""
    io, T, D, V = _xent_args(x, w, labels)
    _arg(lse, "lse", torch.float32, (T,), optional=False)
    _arg(dloss, "dloss", torch.float32, (T,), optional=False)
    if workspace is not None:
        _need(workspace, "workspace")
    _same_device(x=x, w=w, labels=labels, lse=lse, dloss=dloss, workspace=workspace)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = _scratch(workspace, _size("h3conv_linear_xent_workspace_size", T, D, V, io, 1), x.device)
    _check(load().h3conv_linear_xent_bwd(_ptr(x), _ptr(w), _ptr(labels), int(ignore_index), _ptr(lse), _ptr(dloss),
                                         _ptr(dx), _ptr(dw), T, D, V, io, _ptr(ws), ws.numel() * ws.element_size(),
                                         _stream()),
           "h3conv_linear_xent_bwd")
    return dx, dw
