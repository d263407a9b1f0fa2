"""Host-side checks of the C ABI of the short convolution, the selective scan
and the linear cross entropy (no GPU needed, no compute calls).  Pointers
handed to the rejecting calls are never dereferenced."""
import pytest

import fft_long_convolution_flashconv_amd as pkg

A = [0x100000000 * (i + 1) for i in range(24)]  # fake aligned "device" addresses, far apart


@pytest.fixture(scope="module")
def lib():
    return pkg.load()


def _conv(lib, x=A[0], w=A[1], bias=A[2], x_in=A[3], lengths=A[4], y=A[5], x_out=A[6], B=2, H=3, N=8, W=4, io=1):
    return lib.h3conv_short_conv(x, w, bias, x_in, lengths, y, x_out, B, H, N, W, 1, io, None)


def test_short_conv_validation(lib):
    for bad in (dict(B=-1), dict(W=0), dict(io=3), dict(x=None), dict(w=None), dict(y=None), dict(x=A[0] + 1),
                dict(w=A[1] + 2), dict(x_in=A[3] + 1), dict(y=A[0] + 16), dict(y=A[3]), dict(x_out=A[5] + 32), dict(x_out=A[2])):
        assert _conv(lib, **bad) == pkg.ERR_INVALID_ARG, bad
    for bad in (dict(W=5), dict(B=1 << 31, H=1), dict(N=1 << 40, B=1, H=2)):
        assert _conv(lib, **bad) == pkg.ERR_UNSUPPORTED, bad
    assert _conv(lib, B=0, x=None, y=None, x_out=None) == pkg.OK
    assert _conv(lib, N=0, x=None, y=None, x_out=None) == pkg.OK


def _conv_bwd(lib, ws=A[11], n=1 << 20, dx=A[7], dw=A[8], dy=A[5], **k):
    return lib.h3conv_short_conv_bwd(A[0], A[1], A[2], A[3], A[4], dy, A[6], dx, dw, A[9], A[10], k.get("B", 2), 3, 8,
                                     k.get("W", 4), 1, 1, ws, n, None)


def test_short_conv_bwd_validation(lib):
    assert _conv_bwd(lib, ws=None) == pkg.ERR_WORKSPACE
    assert _conv_bwd(lib, n=pkg._size("h3conv_short_conv_bwd_workspace_size", 2, 3, 8, 4) - 1) == pkg.ERR_WORKSPACE
    assert _conv_bwd(lib, W=5) == pkg.ERR_UNSUPPORTED
    for bad in (dict(dx=None), dict(dy=None), dict(dw=A[0]), dict(dx=A[5]), dict(ws=A[7]), dict(B=-1), dict(ws=A[11] + 4)):
        assert _conv_bwd(lib, **bad) == pkg.ERR_INVALID_ARG, bad


def _conv_step(lib, slots=A[3], si=A[4], so=A[4], y=A[6], B=2, P=4, W=4):
    return lib.h3conv_short_conv_step(A[0], A[1], A[2], slots, si, so, y, B, 3, P, W, 1, 1, None)


def test_short_conv_step_validation(lib):
    for bad in (dict(si=None), dict(so=A[4] + 16), dict(y=A[4]), dict(y=None), dict(slots=None, P=1), dict(P=-1),
                dict(so=A[0])):
        assert _conv_step(lib, **bad) == pkg.ERR_INVALID_ARG, bad
    assert _conv_step(lib, B=65536, P=65536) == pkg.ERR_UNSUPPORTED
    assert _conv_step(lib, W=5) == pkg.ERR_UNSUPPORTED
    assert _conv_step(lib, B=0) == pkg.OK


def _scan(lib, u=A[0], y=A[10], x_out=A[11], saved=A[12], x_in=A[8], B=2, H=4, N=8, S=3, G=2, io=1):
    return lib.h3conv_selective_scan(u, A[1], A[2], A[3], A[4], A[5], A[6], A[7], x_in, A[9], y, x_out, saved, B, H, N,
                                     S, G, 1, io, None)


def test_selective_scan_validation(lib):
    for bad in (dict(u=None), dict(y=A[0]), dict(x_out=A[8]), dict(saved=A[10]), dict(G=3), dict(G=0), dict(S=0),
                dict(io=-1), dict(N=-1), dict(x_in=A[8] + 2), dict(saved=A[11]),
                dict(saved=A[12] + 8), dict(u=A[0] + 1)):
        assert _scan(lib, **bad) == pkg.ERR_INVALID_ARG, bad
    for bad in (dict(S=65), dict(B=1 << 20, H=1 << 12), dict(N=1 << 39)):
        assert _scan(lib, **bad) == pkg.ERR_UNSUPPORTED, bad
    assert _scan(lib, B=0) == pkg.OK
    with pytest.raises(pkg.H3ConvError):
        pkg._size("h3conv_selective_scan_bwd_workspace_size", 2, 4, 8, 3, 3)
    with pytest.raises(pkg.H3ConvError):
        pkg._size("h3conv_selective_saved_size", 2, 4, 8, 65)


def _scan_bwd(lib, z=A[6], dz=A[17], dy=A[10], du=A[12], ws=A[20], n=1 << 40, S=3, dA=A[14]):
    return lib.h3conv_selective_scan_bwd(A[0], A[1], A[2], A[3], A[4], A[5], z, A[7], A[8], A[9], dy, A[11], du, A[13],
                                         dA, A[15], A[16], A[18], dz, A[19], A[21], 2, 4, 8, S, 2, 1, 1, ws, n, None)


def test_selective_scan_bwd_validation(lib):
    assert _scan_bwd(lib, ws=None) == pkg.ERR_WORKSPACE
    assert _scan_bwd(lib, n=16) == pkg.ERR_WORKSPACE
    assert _scan_bwd(lib, S=65) == pkg.ERR_UNSUPPORTED
    for bad in (dict(z=None), dict(dz=None), dict(dy=None), dict(du=A[10]), dict(dA=A[2]), dict(dA=None), dict(du=A[13])):
        assert _scan_bwd(lib, **bad) == pkg.ERR_INVALID_ARG, bad


def _step(lib, slots=A[8], xi=A[9], xo=A[9], y=A[11], B=2, P=4, S=3, G=2):
    return lib.h3conv_selective_step(A[0], A[1], A[2], A[3], A[4], A[5], A[6], A[7], slots, xi, xo, y, B, 4, P, S, G, 1, 1,
                                     None)


def test_selective_step_validation(lib):
    for bad in (dict(xi=None), dict(xo=A[9] + 16), dict(y=A[9]), dict(slots=None, P=1), dict(G=3), dict(y=None)):
        assert _step(lib, **bad) == pkg.ERR_INVALID_ARG, bad
    assert _step(lib, S=65) == pkg.ERR_UNSUPPORTED
    assert _step(lib, B=70000, P=70000) == pkg.ERR_UNSUPPORTED
    assert _step(lib, B=0) == pkg.OK


def _xent(lib, x=A[0], w=A[1], labels=A[2], loss=A[3], lse=A[4], ws=A[5], n=1 << 40, T=5, D=8, V=10, io=1):
    return lib.h3conv_linear_xent(x, w, labels, -100, loss, lse, T, D, V, io, ws, n, None)


def test_linear_xent_validation(lib):
    assert _xent(lib, ws=None) == pkg.ERR_WORKSPACE
    assert _xent(lib, n=8) == pkg.ERR_WORKSPACE
    for bad in (dict(x=None), dict(labels=None), dict(loss=A[4]), dict(lse=A[2]), dict(D=0), dict(V=0), dict(T=-1),
                dict(io=9), dict(w=A[1] + 2), dict(ws=A[0])):
        assert _xent(lib, **bad) == pkg.ERR_INVALID_ARG, bad
    for bad in (dict(V=(1 << 22) + 1), dict(D=(1 << 20) + 1), dict(T=(1 << 30) + 1)):
        assert _xent(lib, **bad) == pkg.ERR_UNSUPPORTED, bad
    assert _xent(lib, T=0, x=None, labels=None, loss=None, lse=None, ws=None) == pkg.OK


def test_linear_xent_bwd_validation(lib):
    def f(dx=A[5], dw=A[6], lse=A[3], ws=A[7], n=1 << 40, V=10):
        return lib.h3conv_linear_xent_bwd(A[0], A[1], A[2], -100, lse, A[4], dx, dw, 5, 8, V, 1, ws, n, None)

    assert f(ws=None) == pkg.ERR_WORKSPACE and f(n=8) == pkg.ERR_WORKSPACE
    for bad in (dict(dx=None), dict(dw=A[1]), dict(lse=None), dict(dx=A[6]), dict(ws=A[6])):
        assert f(**bad) == pkg.ERR_INVALID_ARG, bad
    assert f(V=(1 << 22) + 1) == pkg.ERR_UNSUPPORTED
