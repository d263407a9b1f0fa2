"""Host-side checks of the C ABI of linear attention, the norms around a block and the
embedding (no GPU needed, no compute calls).  Pointers handed to the rejecting
calls are never dereferenced."""
import pytest

import fft_long_convolution_flashconv_amd as pkg

A = [0x100000000 * (i + 1) for i in range(24)]  # fake aligned "device" addresses, far apart
BIG = 1 << 45


@pytest.fixture(scope="module")
def lib():
    return pkg.load()


def _attn(lib, q=A[0], k=A[1], v=A[2], g=A[3], x_in=A[4], lengths=A[5], y=A[6], x_out=A[7], B=2, N=5, H=4, G=2, dk=8, dv=6,
          ldq=16, ldk=16, ldv=24, token=1, io=1, ws=A[8], n=BIG):
    return lib.h3conv_linear_attn(q, k, v, g, x_in, lengths, y, x_out, B, N, H, G, dk, dv, ldq, ldk, ldv, 1.0, token, io, ws,
                                  n, None)


def test_linear_attn_validation(lib):
    for bad in (dict(B=-1), dict(N=-1), dict(G=0), dict(G=3), dict(dk=0), dict(dv=0), dict(io=3), dict(q=None), dict(k=None),
                dict(v=None), dict(g=None), dict(y=None), dict(q=A[0] + 1), dict(g=A[3] + 2), dict(y=A[2]), dict(y=A[0] + 64),
                dict(x_out=A[4]), dict(x_out=A[6]), dict(ldq=15), dict(ldk=0), dict(ldv=23), dict(x_in=A[4] + 2)):
        assert _attn(lib, **bad) == pkg.ERR_INVALID_ARG, bad
    for bad in (dict(dk=257), dict(dv=257), dict(B=1 << 20, H=1 << 10), dict(N=1 << 40), dict(ldv=1 << 40)):
        assert _attn(lib, **bad) == pkg.ERR_UNSUPPORTED, bad
    assert _attn(lib, B=0, q=None) == pkg.OK
    assert _attn(lib, N=0, x_out=None, q=None) == pkg.OK


def test_linear_attn_extents(lib):
    """A slice of a projection reaches from its first token to the end of its last: y may stand behind that."""
    end = A[0] + ((2 * 5 - 1) * 40 + 16) * 2
    assert _attn(lib, ldq=40, y=end - 2) == pkg.ERR_INVALID_ARG


def _attn_bwd(lib, dy=A[6], dx_out=A[7], dq=A[8], dk_=A[9], dv_=A[10], dg=A[11], dx_in=A[12], ws=A[13], n=BIG, G=2, dk=8,
              ldv=24, H=4, B=2):
    return lib.h3conv_linear_attn_bwd(A[0], A[1], A[2], A[3], A[4], A[5], dy, dx_out, dq, dk_, dv_, dg, dx_in, B, 5, H, G, dk,
                                      6, 16, 16, ldv, 1.0, 1, 1, ws, n, None)


def test_linear_attn_bwd_validation(lib):
    assert _attn_bwd(lib, ws=None) == pkg.ERR_WORKSPACE
    assert _attn_bwd(lib, n=pkg._size("h3conv_linear_attn_bwd_workspace_size", 2, 5, 4, 2, 8, 6) - 1) == pkg.ERR_WORKSPACE
    assert _attn_bwd(lib, dk=300) == pkg.ERR_UNSUPPORTED
    assert _attn_bwd(lib, H=1 << 40, B=0, G=1) == pkg.ERR_UNSUPPORTED
    for bad in (dict(dy=None), dict(dq=None), dict(dk_=A[8]), dict(dv_=A[2]), dict(dg=A[3]), dict(dx_in=A[7]), dict(ws=A[10]),
                dict(ws=A[13] + 4), dict(G=3), dict(ldv=20), dict(dq=A[8] + 1)):
        assert _attn_bwd(lib, **bad) == pkg.ERR_INVALID_ARG, bad
    assert _attn_bwd(lib, H=0) == pkg.OK


def _attn_step(lib, slots=A[4], xi=A[5], xo=A[5], y=A[6], B=2, P=4, dk=8, ldq=16, v=A[2]):
    return lib.h3conv_linear_attn_step(A[0], A[1], v, A[3], slots, xi, xo, y, B, 4, 2, P, dk, 6, ldq, 16, 24, 1.0, 0, 1, None)


def test_linear_attn_step_validation(lib):
    for bad in (dict(xi=None), dict(xo=A[5] + 16), dict(y=A[5]), dict(slots=None, P=1), dict(P=-1), dict(y=None), dict(ldq=8),
                dict(v=None), dict(xo=A[2])):
        assert _attn_step(lib, **bad) == pkg.ERR_INVALID_ARG, bad
    assert _attn_step(lib, B=65536, P=65536) == pkg.ERR_UNSUPPORTED
    assert _attn_step(lib, dk=257, ldq=1000) in (pkg.ERR_UNSUPPORTED, pkg.ERR_INVALID_ARG)
    assert _attn_step(lib, B=0) == pkg.OK


def _norm(lib, f=A[0], res=A[1], gate=A[2], w_out=A[3], scale=A[4], w_in=A[5], r=A[6], y=A[7], T=3, D=12, groups=2, eps=1e-5,
          io=1):
    return lib.h3conv_block_norm(f, res, gate, w_out, scale, w_in, r, y, T, D, groups, eps, io, None)


def test_block_norm_validation(lib):
    for bad in (dict(f=None), dict(r=None), dict(y=None), dict(w_in=None), dict(T=-1), dict(D=0), dict(groups=0), dict(groups=5),
                dict(eps=-1.0), dict(eps=float("nan")), dict(io=3), dict(r=A[1]), dict(y=A[6] + 16), dict(r=A[3] + 4),
                dict(f=A[0] + 1), dict(scale=A[4] + 2)):
        assert _norm(lib, **bad) == pkg.ERR_INVALID_ARG, bad
    for bad in (dict(D=16385, groups=1), dict(D=16384, groups=2), dict(T=1 << 31)):
        assert _norm(lib, **bad) == pkg.ERR_UNSUPPORTED, bad
    assert _norm(lib, T=0, f=None) == pkg.OK


def _norm_bwd(lib, res=A[1], gate=A[2], w_in=A[5], dr=A[6], dy=A[7], df=A[8], dres=A[9], dgate=A[10], dw_out=A[11], dscale=A[12],
              dw_in=A[13], ws=A[14], n=BIG, D=12):
    return lib.h3conv_block_norm_bwd(A[0], res, gate, A[3], A[4], w_in, dr, dy, df, dres, dgate, dw_out, dscale, dw_in, 3, D, 2,
                                     1e-5, 1, ws, n, None)


def test_block_norm_bwd_validation(lib):
    assert _norm_bwd(lib, ws=None) == pkg.ERR_WORKSPACE
    assert _norm_bwd(lib, n=pkg._size("h3conv_block_norm_bwd_workspace_size", 3, 12) - 1) == pkg.ERR_WORKSPACE
    assert _norm_bwd(lib, D=16386) == pkg.ERR_UNSUPPORTED
    for bad in (dict(gate=None), dict(dgate=None), dict(dw_out=None), dict(dscale=None), dict(w_in=None, dw_in=None), dict(dw_in=None),
                dict(df=None), dict(res=None), dict(df=A[6]), dict(dres=A[9] + 1), dict(dw_out=A[12]), dict(ws=A[8])):
        assert _norm_bwd(lib, **bad) == pkg.ERR_INVALID_ARG, bad
    with pytest.raises(pkg.H3ConvError):
        pkg._size("h3conv_block_norm_bwd_workspace_size", 3, 16385)


def test_embed_validation(lib):
    def f(tok=A[0], w=A[1], y=A[2], T=5, D=8, V=10, io=1):
        return lib.h3conv_embed(tok, w, y, T, D, V, 1.0, io, None)

    for bad in (dict(tok=None), dict(w=None), dict(y=None), dict(T=-1), dict(D=0), dict(V=-1), dict(io=9), dict(tok=A[0] + 4),
                dict(y=A[1]), dict(y=A[2] + 1)):
        assert f(**bad) == pkg.ERR_INVALID_ARG, bad
    for bad in (dict(D=(1 << 20) + 1), dict(V=(1 << 30) + 1), dict(T=(1 << 30) + 1), dict(T=1 << 25, D=1 << 20)):
        assert f(**bad) == pkg.ERR_UNSUPPORTED, bad
    assert f(T=0, tok=None) == pkg.OK


def test_embed_bwd_validation(lib):
    def f(tok=A[0], dy=A[1], dw=A[2], T=5, D=8, V=10, ws=A[3], n=BIG):
        return lib.h3conv_embed_bwd(tok, dy, dw, T, D, V, 1.0, 1, ws, n, None)

    for bad in (dict(tok=None), dict(dy=None), dict(dw=None), dict(T=-1), dict(D=0), dict(dw=A[0]), dict(dw=A[1] + 2), dict(ws=A[2])):
        assert f(**bad) == pkg.ERR_INVALID_ARG, bad
    assert f(ws=None) == pkg.ERR_WORKSPACE
    assert f(n=pkg._size("h3conv_embed_bwd_workspace_size", 5, 8, 10) - 1) == pkg.ERR_WORKSPACE
    assert f(V=(1 << 30) + 1) == pkg.ERR_UNSUPPORTED
    assert f(V=0) == pkg.OK
