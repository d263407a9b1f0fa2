// lm_api.hip -- C ABI of the short convolution, the selective scan, linear
// attention, the norms around a block, the embedding and the linear cross
// entropy: argument validation (host only, before any HIP call) and dispatch to
// the kernel launchers.  See include/h3conv.h for the
// contract of every entry point.
#include <initializer_list>

#include "../api_checks.h"
#include "lm_internal.h"

namespace {

using namespace h3c;  // the host-side checks

int64_t esize(int io) { return io == H3CONV_F32 ? 4 : 2; }

// One buffer argument of a call.
struct Buf {
    const void *p;
    int64_t bytes;
    bool needed;
    uintptr_t align = 16;
};

bool overlap(const Buf &a, const Buf &b) {
    return a.bytes > 0 && b.bytes > 0 && h3c::overlap(a.p, (size_t)a.bytes, b.p, (size_t)b.bytes);
}

// Pointers present and aligned; no output overlaps an input or another output.
bool bufs_ok(std::initializer_list<Buf> ins, std::initializer_list<Buf> outs) {
    for (const auto *l : {&ins, &outs})
        for (const Buf &b : *l) {
            if (b.needed && b.bytes > 0 && !b.p) return false;
            if (reinterpret_cast<uintptr_t>(b.p) & (b.align - 1)) return false;
        }
    for (const Buf *o = outs.begin(); o != outs.end(); ++o) {
        for (const Buf &i : ins)
            if (overlap(*o, i)) return false;
        for (const Buf *q = o + 1; q != outs.end(); ++q)
            if (overlap(*o, *q)) return false;
    }
    return true;
}

// The product of the sizes is at most `most` (each factor non-negative).
bool product_ok(std::initializer_list<int64_t> f, int64_t most) {
    int64_t n = 1;
    for (int64_t v : f) {
        if (v < 0) return false;
        if (v == 0) return true;
        if (n > most / v) return false;
        n *= v;
    }
    return true;
}

constexpr int64_t kElems = (int64_t)1 << 40;  // elements of one tensor
constexpr int64_t kRows = (int64_t)1 << 30;   // rows (b, h): one dispatch's grid

bool conv_sizes_ok(int64_t B, int64_t H, int64_t N, int64_t W) {
    return W <= H3CONV_MAX_TAPS && product_ok({B, H}, kRows) && product_ok({B, H, N}, kElems);
}
bool scan_sizes_ok(int64_t B, int64_t H, int64_t N, int64_t S, int64_t G) {
    return S <= H3CONV_MAX_STATE && product_ok({B, H}, kRows) && product_ok({B, H, N}, kElems) &&
           product_ok({B, G, S, N}, kElems) && product_ok({B, G, S, N}, (int64_t)1 << 38);
}
bool xent_sizes_ok(int64_t T, int64_t D, int64_t V) {
    return T <= ((int64_t)1 << 30) && D <= ((int64_t)1 << 20) && V <= ((int64_t)1 << 22) &&
           product_ok({T, D}, kElems) && product_ok({V, D}, kElems) &&
           product_ok({T / 64 + 1, V / 64 + 1}, (int64_t)1 << 31) &&                       // tiles of one dispatch
           product_ok({(T > V ? T : V) / 64 + 2, D / 64 + 1}, (int64_t)1 << 27);
}

bool attn_sizes_ok(int64_t B, int64_t N, int64_t H, int64_t dk, int64_t dv) {
    return N <= ((int64_t)1 << 30) && dk <= H3CONV_MAX_HEAD && dv <= H3CONV_MAX_HEAD && H <= H3CONV_MAX_LD / (dk > dv ? dk : dv) &&
           product_ok({B, H}, (int64_t)1 << 28) && product_ok({B, N, H * (dk > dv ? dk : dv)}, kElems) && product_ok({B, H, dk, dv}, kElems);
}
// Elements from the first to the last of n tokens' rows, ld apart.
int64_t extent(int64_t n, int64_t ld, int64_t row) { return n == 0 ? 0 : (n - 1) * ld + row; }
// Rows ld apart stay within the largest tensor, and 64 of them within 32 bits.
bool ld_small(int64_t n, int64_t ld) { return ld <= H3CONV_MAX_LD && product_ok({n, ld}, kElems); }

bool norm_sizes_ok(int64_t T, int64_t D, int64_t groups) {
    return D <= H3CONV_MAX_NORM && (groups == 1 || D + groups <= H3CONV_MAX_NORM) && T <= ((int64_t)1 << 30);
}
bool embed_sizes_ok(int64_t T, int64_t D, int64_t V) {
    return T <= ((int64_t)1 << 30) && V <= ((int64_t)1 << 30) && D <= ((int64_t)1 << 20) && product_ok({T, D}, kElems) &&
           product_ok({V, D}, kElems);
}

}  // namespace

extern "C" {

h3conv_status h3conv_short_conv(const void *x, const float *w, const float *bias, const void *x_in,
                                const int32_t *lengths, void *y, void *x_out, int64_t B, int64_t H, int64_t N,
                                int64_t W, int silu, int io, void *stream) {
    if (B < 0 || H < 0 || N < 0 || W < 1 || !valid_io(io)) return H3CONV_ERR_INVALID_ARG;
    if (B == 0 || H == 0 || (N == 0 && !x_out)) return H3CONV_OK;
    if (!conv_sizes_ok(B, H, N, W)) return H3CONV_ERR_UNSUPPORTED;
    const int64_t e = esize(io), n = B * H * N * e, st = B * H * (W - 1) * e;
    const uintptr_t ea = (uintptr_t)e;
    if (!bufs_ok({{x, n, true, ea}, {w, H * W * 4, true, 4}, {bias, H * 4, false, 4}, {x_in, st, false, ea}, {lengths, B * 4, false, 4}},
                 {{y, n, true, ea}, {x_out, st, false, ea}}))
        return H3CONV_ERR_INVALID_ARG;
    const h3conv_status s = device_check();
    if (s != H3CONV_OK) return s;
    const h3c::ShortConvArgs a = {x, x_in, w, bias, lengths, B, H, N, (int)W, silu};
    return from_hip(h3c::launch_short_conv(a, y, x_out, io, (hipStream_t)stream));
}

size_t h3conv_short_conv_bwd_workspace_size(int64_t B, int64_t H, int64_t N, int64_t W) {
    if (B < 0 || H < 0 || N < 0 || W < 1 || !conv_sizes_ok(B, H, N, W)) return (size_t)-1;
    if (H == 0) return 0;
    return h3c::short_conv_bwd_workspace(B, H, N, (int)W);
}

h3conv_status h3conv_short_conv_bwd(const void *x, const float *w, const float *bias, const void *x_in,
                                    const int32_t *lengths, const void *dy, const void *dx_out, void *dx, float *dw,
                                    float *dbias, void *dx_in, int64_t B, int64_t H, int64_t N, int64_t W, int silu,
                                    int io, void *ws, size_t ws_bytes, void *stream) {
    if (B < 0 || H < 0 || N < 0 || W < 1 || !valid_io(io)) return H3CONV_ERR_INVALID_ARG;
    if (H == 0) return H3CONV_OK;
    if (!conv_sizes_ok(B, H, N, W)) return H3CONV_ERR_UNSUPPORTED;
    const int64_t e = esize(io), n = B * H * N * e, st = B * H * (W - 1) * e;
    const uintptr_t ea = (uintptr_t)e;
    const size_t need = h3c::short_conv_bwd_workspace(B, H, N, (int)W);
    if (!ws || ws_bytes < need) return H3CONV_ERR_WORKSPACE;
    if (!bufs_ok({{x, n, true, ea}, {w, H * W * 4, true, 4}, {bias, H * 4, false, 4}, {x_in, st, false, ea},
                  {lengths, B * 4, false, 4}, {dy, n, true, ea}, {dx_out, st, false, ea}},
                 {{dx, n, true, ea}, {dw, H * W * 4, true, 4}, {dbias, H * 4, false, 4}, {dx_in, st, false, ea},
                  {ws, (int64_t)need, true}}))
        return H3CONV_ERR_INVALID_ARG;
    const h3conv_status s = device_check();
    if (s != H3CONV_OK) return s;
    const h3c::ShortConvArgs a = {x, x_in, w, bias, lengths, B, H, N, (int)W, silu};
    return from_hip(h3c::launch_short_conv_bwd(a, dy, dx_out, dx, dw, dbias, dx_in, io, ws, (hipStream_t)stream));
}

h3conv_status h3conv_short_conv_step(const void *x, const float *w, const float *bias, const int32_t *slots,
                                     const void *state_in, void *state_out, void *y, int64_t B, int64_t H, int64_t P,
                                     int64_t W, int silu, int io, void *stream) {
    if (B < 0 || H < 0 || P < 0 || W < 1 || !valid_io(io) || (!slots && P < B)) return H3CONV_ERR_INVALID_ARG;
    if (B == 0 || H == 0) return H3CONV_OK;
    if (B > 65535 || !conv_sizes_ok(B, H, 1, W) || !product_ok({P, H, W}, kElems)) return H3CONV_ERR_UNSUPPORTED;
    const int64_t e = esize(io), n = B * H * e, st = P * H * (W - 1) * e;
    const uintptr_t ea = (uintptr_t)e;
    // state_out is state_in itself, or apart from it
    const Buf from = {state_in, st, true, ea}, to = {state_out, st, true, ea};
    if (!bufs_ok({{x, n, true, ea}, {w, H * W * 4, true, 4}, {bias, H * 4, false, 4}, {slots, B * 4, false, 4},
                  state_in == state_out ? Buf{nullptr, 0, false, 4} : from},
                 {{y, n, true, ea}, to}))
        return H3CONV_ERR_INVALID_ARG;
    const h3conv_status s = device_check();
    if (s != H3CONV_OK) return s;
    return from_hip(h3c::launch_short_conv_step(x, w, bias, slots, state_in, state_out, y, B, H, P, (int)W, silu, io,
                                                (hipStream_t)stream));
}

h3conv_status h3conv_selective_scan(const void *u, const void *dt, const float *A, const void *Bm, const void *C,
                                    const float *D, const void *z, const float *dt_bias, const float *x_in,
                                    const int32_t *lengths, void *y, float *x_out, float *saved, int64_t B, int64_t H,
                                    int64_t N, int64_t S, int64_t G, int softplus, int io, void *stream) {
    if (B < 0 || H < 0 || N < 0 || S < 1 || G < 1 || H % G != 0 || !valid_io(io)) return H3CONV_ERR_INVALID_ARG;
    if (B == 0 || H == 0 || (N == 0 && !x_out)) return H3CONV_OK;
    if (!scan_sizes_ok(B, H, N, S, G)) return H3CONV_ERR_UNSUPPORTED;
    const int64_t e = esize(io), n = B * H * N * e, bc = B * G * S * N * e, st = B * H * S * 4;
    const uintptr_t ea = (uintptr_t)e;
    const int64_t sv = (int64_t)h3c::selective_saved_floats(B, H, N, S) * 4;
    if (!bufs_ok({{u, n, true, ea}, {dt, n, true, ea}, {A, H * S * 4, true, 4}, {Bm, bc, true, ea}, {C, bc, true, ea}, {D, H * 4, false, 4},
                  {z, n, false, ea}, {dt_bias, H * 4, false, 4}, {x_in, st, false, 4}, {lengths, B * 4, false, 4}},
                 {{y, n, true, ea}, {x_out, st, false, 4}, {saved, sv, false}}))
        return H3CONV_ERR_INVALID_ARG;
    const h3conv_status s = device_check();
    if (s != H3CONV_OK) return s;
    const h3c::SelArgs a = {u, dt, Bm, C, z, A, D, dt_bias, x_in, lengths, B, H, N, (int)S, (int)G, softplus};
    return from_hip(h3c::launch_selective_scan(a, y, x_out, saved, io, (hipStream_t)stream));
}

size_t h3conv_selective_saved_size(int64_t B, int64_t H, int64_t N, int64_t S) {
    if (B < 0 || H < 0 || N < 0 || S < 1 || !scan_sizes_ok(B, H, N, S, 1)) return (size_t)-1;
    return h3c::selective_saved_floats(B, H, N, S) * 4;
}

size_t h3conv_selective_scan_bwd_workspace_size(int64_t B, int64_t H, int64_t N, int64_t S, int64_t G) {
    if (B < 0 || H < 0 || N < 0 || S < 1 || G < 1 || H % G != 0 || !scan_sizes_ok(B, H, N, S, G)) return (size_t)-1;
    if (H == 0) return 0;
    return h3c::selective_bwd_workspace(B, H, N, S, G);
}

h3conv_status h3conv_selective_scan_bwd(const void *u, const void *dt, const float *A, const void *Bm, const void *C,
                                        const float *D, const void *z, const float *dt_bias, const int32_t *lengths,
                                        const float *saved, const void *dy, const float *dx_out, void *du, void *ddt,
                                        float *dA, void *dB, void *dC, float *dD, void *dz, float *ddt_bias,
                                        float *dx_in, int64_t B, int64_t H, int64_t N, int64_t S, int64_t G,
                                        int softplus, int io, void *ws, size_t ws_bytes, void *stream) {
    if (B < 0 || H < 0 || N < 0 || S < 1 || G < 1 || H % G != 0 || !valid_io(io)) return H3CONV_ERR_INVALID_ARG;
    if (H == 0) return H3CONV_OK;
    if (!scan_sizes_ok(B, H, N, S, G)) return H3CONV_ERR_UNSUPPORTED;
    if ((z == nullptr) != (dz == nullptr)) return H3CONV_ERR_INVALID_ARG;
    const int64_t e = esize(io), n = B * H * N * e, bc = B * G * S * N * e, st = B * H * S * 4, hs = H * S * 4;
    const uintptr_t ea = (uintptr_t)e;
    const int64_t sv = (int64_t)h3c::selective_saved_floats(B, H, N, S) * 4;
    const size_t need = h3c::selective_bwd_workspace(B, H, N, S, G);
    if (!ws || ws_bytes < need) return H3CONV_ERR_WORKSPACE;
    if (!bufs_ok({{u, n, true, ea}, {dt, n, true, ea}, {A, hs, true, 4}, {Bm, bc, true, ea}, {C, bc, true, ea}, {D, H * 4, false, 4},
                  {z, n, false, ea}, {dt_bias, H * 4, false, 4}, {lengths, B * 4, false, 4}, {saved, sv, true}, {dy, n, true, ea},
                  {dx_out, st, false, 4}},
                 {{du, n, true, ea}, {ddt, n, true, ea}, {dA, hs, true, 4}, {dB, bc, true, ea}, {dC, bc, true, ea}, {dD, H * 4, false, 4},
                  {dz, n, false, ea}, {ddt_bias, H * 4, false, 4}, {dx_in, st, false, 4}, {ws, (int64_t)need, true}}))
        return H3CONV_ERR_INVALID_ARG;
    const h3conv_status s = device_check();
    if (s != H3CONV_OK) return s;
    const h3c::SelArgs a = {u, dt, Bm, C, z, A, D, dt_bias, nullptr, lengths, B, H, N, (int)S, (int)G, softplus};
    const h3c::SelGrads g = {du, ddt, dB, dC, dz, dA, dD, ddt_bias, dx_in};
    return from_hip(h3c::launch_selective_scan_bwd(a, saved, dy, dx_out, g, io, ws, (hipStream_t)stream));
}

h3conv_status h3conv_selective_step(const void *u, const void *dt, const float *A, const void *Bm, const void *C,
                                    const float *D, const void *z, const float *dt_bias, const int32_t *slots,
                                    const float *x_in, float *x_out, void *y, int64_t B, int64_t H, int64_t P,
                                    int64_t S, int64_t G, int softplus, int io, void *stream) {
    if (B < 0 || H < 0 || P < 0 || S < 1 || G < 1 || H % G != 0 || !valid_io(io) || (!slots && P < B))
        return H3CONV_ERR_INVALID_ARG;
    if (B == 0 || H == 0) return H3CONV_OK;
    if (B > 65535 || !scan_sizes_ok(B, H, 1, S, G) || !product_ok({P, H, S}, kElems)) return H3CONV_ERR_UNSUPPORTED;
    const int64_t e = esize(io), n = B * H * e, bc = B * G * S * e, st = P * H * S * 4;
    const uintptr_t ea = (uintptr_t)e;
    const Buf from = {x_in, st, true, 4}, to = {x_out, st, true, 4};
    if (!bufs_ok({{u, n, true, ea}, {dt, n, true, ea}, {A, H * S * 4, true, 4}, {Bm, bc, true, ea}, {C, bc, true, ea}, {D, H * 4, false, 4},
                  {z, n, false, ea}, {dt_bias, H * 4, false, 4}, {slots, B * 4, false, 4},
                  x_in == x_out ? Buf{nullptr, 0, false, 4} : from},
                 {{y, n, true, ea}, to}))
        return H3CONV_ERR_INVALID_ARG;
    const h3conv_status s = device_check();
    if (s != H3CONV_OK) return s;
    return from_hip(h3c::launch_selective_step(u, dt, A, Bm, C, D, z, dt_bias, slots, x_in, x_out, y, B, H, P, (int)S,
                                               (int)G, softplus, io, (hipStream_t)stream));
}

size_t h3conv_linear_xent_workspace_size(int64_t T, int64_t D, int64_t V, int io, int bwd) {
    if (T < 0 || D < 1 || V < 1 || !valid_io(io) || !xent_sizes_ok(T, D, V)) return (size_t)-1;
    return T == 0 ? 0 : h3c::linear_xent_workspace(T, D, V, io, bwd != 0);
}

h3conv_status h3conv_linear_xent(const void *x, const void *w, const int64_t *labels, int64_t ignore_index,
                                 float *loss, float *lse, int64_t T, int64_t D, int64_t V, int io, void *ws,
                                 size_t ws_bytes, void *stream) {
    if (T < 0 || D < 1 || V < 1 || !valid_io(io)) return H3CONV_ERR_INVALID_ARG;
    if (T == 0) return H3CONV_OK;
    if (!xent_sizes_ok(T, D, V)) return H3CONV_ERR_UNSUPPORTED;
    const int64_t e = esize(io);
    const size_t need = h3c::linear_xent_workspace(T, D, V, io, false);
    if (!ws || ws_bytes < need) return H3CONV_ERR_WORKSPACE;
    if (!bufs_ok({{x, T * D * e, true}, {w, V * D * e, true}, {labels, T * 8, true}},
                 {{loss, T * 4, true}, {lse, T * 4, true}, {ws, (int64_t)need, true}}))
        return H3CONV_ERR_INVALID_ARG;
    const h3conv_status s = device_check();
    if (s != H3CONV_OK) return s;
    return from_hip(h3c::launch_linear_xent(x, w, labels, ignore_index, loss, lse, T, D, V, io, ws,
                                            (hipStream_t)stream));
}

h3conv_status h3conv_linear_xent_bwd(const void *x, const void *w, const int64_t *labels, int64_t ignore_index,
                                     const float *lse, const float *dloss, void *dx, void *dw, int64_t T, int64_t D,
                                     int64_t V, int io, void *ws, size_t ws_bytes, void *stream) {
    if (T < 0 || D < 1 || V < 1 || !valid_io(io)) return H3CONV_ERR_INVALID_ARG;
    if (!xent_sizes_ok(T, D, V)) return H3CONV_ERR_UNSUPPORTED;
    const int64_t e = esize(io);
    const size_t need = T > 0 ? h3c::linear_xent_workspace(T, D, V, io, true) : 0;
    if (T > 0 && (!ws || ws_bytes < need)) return H3CONV_ERR_WORKSPACE;
    if (!bufs_ok({{x, T * D * e, true}, {w, V * D * e, true}, {labels, T * 8, true}, {lse, T * 4, true},
                  {dloss, T * 4, true}},
                 {{dx, T * D * e, true}, {dw, V * D * e, true}, {ws, (int64_t)need, true}}))
        return H3CONV_ERR_INVALID_ARG;
    const h3conv_status s = device_check();
    if (s != H3CONV_OK) return s;
    return from_hip(h3c::launch_linear_xent_bwd(x, w, labels, ignore_index, lse, dloss, dx, dw, T, D, V, io, ws,
                                                (hipStream_t)stream));
}

size_t h3conv_linear_attn_workspace_size(int64_t B, int64_t N, int64_t H, int64_t dk, int64_t dv) {
    if (B < 0 || N < 0 || H < 0 || dk < 1 || dv < 1 || !attn_sizes_ok(B, N, H, dk, dv)) return (size_t)-1;
    return h3c::linear_attn_workspace(B, N, H, dk, dv);
}

h3conv_status h3conv_linear_attn(const void *q, const void *k, const void *v, const float *g, const float *x_in,
                                 const int32_t *lengths, void *y, float *x_out, int64_t B, int64_t N, int64_t H,
                                 int64_t G, int64_t dk, int64_t dv, int64_t ldq, int64_t ldk, int64_t ldv, float scale,
                                 int per_token, int io, void *ws, size_t ws_bytes, void *stream) {
    if (B < 0 || N < 0 || H < 0 || G < 1 || H % G != 0 || dk < 1 || dv < 1 || !valid_io(io)) return H3CONV_ERR_INVALID_ARG;
    if (B == 0 || H == 0 || (N == 0 && !x_out)) return H3CONV_OK;
    if (!attn_sizes_ok(B, N, H, dk, dv)) return H3CONV_ERR_UNSUPPORTED;
    const int64_t n = B * N;
    if (ldq < G * dk || ldk < G * dk || ldv < H * dv) return H3CONV_ERR_INVALID_ARG;
    if (!ld_small(n, ldq) || !ld_small(n, ldk) || !ld_small(n, ldv)) return H3CONV_ERR_UNSUPPORTED;
    const size_t need = h3c::linear_attn_workspace(B, N, H, dk, dv);
    if (need > 0 && (!ws || ws_bytes < need)) return H3CONV_ERR_WORKSPACE;
    const int64_t e = esize(io), st = B * H * dk * dv * 4;
    const uintptr_t ea = (uintptr_t)e;
    if (!bufs_ok({{q, extent(n, ldq, G * dk) * e, true, ea}, {k, extent(n, ldk, G * dk) * e, true, ea},
                  {v, extent(n, ldv, H * dv) * e, true, ea}, {g, (per_token ? n * H : H) * 4, true, 4}, {x_in, st, false, 4},
                  {lengths, B * 4, false, 4}},
                 {{y, n * H * dv * e, true, ea}, {x_out, st, false, 4}, {ws, (int64_t)need, need > 0}}))
        return H3CONV_ERR_INVALID_ARG;
    const h3conv_status s = device_check();
    if (s != H3CONV_OK) return s;
    const h3c::LinAttnArgs a = {q, k, v, g, x_in, lengths, B, N, H, G, (int)dk, (int)dv, ldq, ldk, ldv, scale, per_token};
    return from_hip(h3c::launch_linear_attn(a, y, x_out, io, ws, (hipStream_t)stream));
}

size_t h3conv_linear_attn_bwd_workspace_size(int64_t B, int64_t N, int64_t H, int64_t G, int64_t dk, int64_t dv) {
    if (B < 0 || N < 0 || H < 0 || G < 1 || H % G != 0 || dk < 1 || dv < 1 || !attn_sizes_ok(B, N, H, dk, dv))
        return (size_t)-1;
    return h3c::linear_attn_bwd_workspace(B, N, H, G, dk, dv);
}

h3conv_status h3conv_linear_attn_bwd(const void *q, const void *k, const void *v, const float *g, const float *x_in,
                                     const int32_t *lengths, const void *dy, const float *dx_out, void *dq, void *dk_,
                                     void *dv_, float *dg, float *dx_in, int64_t B, int64_t N, int64_t H, int64_t G,
                                     int64_t dk, int64_t dv, int64_t ldq, int64_t ldk, int64_t ldv, float scale,
                                     int per_token, int io, void *ws, size_t ws_bytes, void *stream) {
    if (B < 0 || N < 0 || H < 0 || G < 1 || H % G != 0 || dk < 1 || dv < 1 || !valid_io(io)) return H3CONV_ERR_INVALID_ARG;
    if (H == 0) return H3CONV_OK;
    if (!attn_sizes_ok(B, N, H, dk, dv)) return H3CONV_ERR_UNSUPPORTED;
    const int64_t n = B * N;
    if (ldq < G * dk || ldk < G * dk || ldv < H * dv) return H3CONV_ERR_INVALID_ARG;
    if (!ld_small(n, ldq) || !ld_small(n, ldk) || !ld_small(n, ldv)) return H3CONV_ERR_UNSUPPORTED;
    const size_t need = h3c::linear_attn_bwd_workspace(B, N, H, G, dk, dv);
    if (need > 0 && (!ws || ws_bytes < need)) return H3CONV_ERR_WORKSPACE;
    const int64_t e = esize(io), st = B * H * dk * dv * 4, gs = (per_token ? n * H : H) * 4;
    const uintptr_t ea = (uintptr_t)e;
    if (!bufs_ok({{q, extent(n, ldq, G * dk) * e, true, ea}, {k, extent(n, ldk, G * dk) * e, true, ea},
                  {v, extent(n, ldv, H * dv) * e, true, ea}, {g, gs, true, 4}, {x_in, st, false, 4},
                  {lengths, B * 4, false, 4}, {dy, n * H * dv * e, true, ea}, {dx_out, st, false, 4}},
                 {{dq, n * G * dk * e, true, ea}, {dk_, n * G * dk * e, true, ea}, {dv_, n * H * dv * e, true, ea},
                  {dg, gs, false, 4}, {dx_in, st, false, 4}, {ws, (int64_t)need, need > 0}}))
        return H3CONV_ERR_INVALID_ARG;
    const h3conv_status s = device_check();
    if (s != H3CONV_OK) return s;
    const h3c::LinAttnArgs a = {q, k, v, g, x_in, lengths, B, N, H, G, (int)dk, (int)dv, ldq, ldk, ldv, scale, per_token};
    const h3c::LinAttnGrads o = {dq, dk_, dv_, dg, dx_in};
    return from_hip(h3c::launch_linear_attn_bwd(a, dy, dx_out, o, io, ws, (hipStream_t)stream));
}

h3conv_status h3conv_linear_attn_step(const void *q, const void *k, const void *v, const float *g, const int32_t *slots,
                                      const float *x_in, float *x_out, void *y, int64_t B, int64_t H, int64_t G,
                                      int64_t P, int64_t dk, int64_t dv, int64_t ldq, int64_t ldk, int64_t ldv,
                                      float scale, int per_token, int io, void *stream) {
    if (B < 0 || H < 0 || P < 0 || G < 1 || H % G != 0 || dk < 1 || dv < 1 || !valid_io(io) || (!slots && P < B))
        return H3CONV_ERR_INVALID_ARG;
    if (B == 0 || H == 0) return H3CONV_OK;
    if (B > 65535 || !attn_sizes_ok(B, 1, H, dk, dv) || !product_ok({P, H, dk, dv}, kElems)) return H3CONV_ERR_UNSUPPORTED;
    if (ldq < G * dk || ldk < G * dk || ldv < H * dv) return H3CONV_ERR_INVALID_ARG;
    if (!ld_small(B, ldq) || !ld_small(B, ldk) || !ld_small(B, ldv)) return H3CONV_ERR_UNSUPPORTED;
    const int64_t e = esize(io), st = P * H * dk * dv * 4;
    const uintptr_t ea = (uintptr_t)e;
    const Buf from = {x_in, st, true, 4}, to = {x_out, st, true, 4};
    if (!bufs_ok({{q, extent(B, ldq, G * dk) * e, true, ea}, {k, extent(B, ldk, G * dk) * e, true, ea},
                  {v, extent(B, ldv, H * dv) * e, true, ea}, {g, (per_token ? B * H : H) * 4, true, 4},
                  {slots, B * 4, false, 4}, x_in == x_out ? Buf{nullptr, 0, false, 4} : from},
                 {{y, B * H * dv * e, true, ea}, to}))
        return H3CONV_ERR_INVALID_ARG;
    const h3conv_status s = device_check();
    if (s != H3CONV_OK) return s;
    const h3c::LinStepArgs a = {q, k, v, g, x_in, slots, x_out, y, B, H, G, P, (int)dk, (int)dv, ldq, ldk, ldv, scale, per_token};
    return from_hip(h3c::launch_linear_attn_step(a, io, (hipStream_t)stream));
}

h3conv_status h3conv_block_norm(const void *f, const void *res, const void *gate, const float *w_out, const float *scale,
                                const float *w_in, void *r, void *y, int64_t T, int64_t D, int64_t groups, float eps,
                                int io, void *stream) {
    if (T < 0 || D < 1 || groups < 1 || D % groups != 0 || !(eps >= 0.f) || !valid_io(io)) return H3CONV_ERR_INVALID_ARG;
    if (T == 0) return H3CONV_OK;
    if ((w_in == nullptr) != (y == nullptr)) return H3CONV_ERR_INVALID_ARG;
    if (!norm_sizes_ok(T, D, groups)) return H3CONV_ERR_UNSUPPORTED;
    const int64_t e = esize(io), n = T * D * e;
    const uintptr_t ea = (uintptr_t)e;
    if (!bufs_ok({{f, n, true, ea}, {res, n, false, ea}, {gate, n, false, ea}, {w_out, D * 4, false, 4},
                  {scale, D * 4, false, 4}, {w_in, D * 4, false, 4}},
                 {{r, n, true, ea}, {y, n, false, ea}}))
        return H3CONV_ERR_INVALID_ARG;
    const h3conv_status s = device_check();
    if (s != H3CONV_OK) return s;
    const h3c::BlockNormArgs a = {f, res, gate, w_out, scale, w_in, T, D, groups, eps};
    return from_hip(h3c::launch_block_norm(a, r, y, io, (hipStream_t)stream));
}

size_t h3conv_block_norm_bwd_workspace_size(int64_t T, int64_t D) {
    if (T < 0 || D < 1 || !norm_sizes_ok(T, D, 1)) return (size_t)-1;
    return h3c::block_norm_bwd_workspace(T, D);
}

h3conv_status h3conv_block_norm_bwd(const void *f, const void *res, const void *gate, const float *w_out,
                                    const float *scale, const float *w_in, const void *dr, const void *dy, void *df,
                                    void *dres, void *dgate, float *dw_out, float *dscale, float *dw_in, int64_t T,
                                    int64_t D, int64_t groups, float eps, int io, void *ws, size_t ws_bytes, void *stream) {
    if (T < 0 || D < 1 || groups < 1 || D % groups != 0 || !(eps >= 0.f) || !valid_io(io)) return H3CONV_ERR_INVALID_ARG;
    if ((T > 0 && (gate == nullptr) != (dgate == nullptr)) || (w_out == nullptr) != (dw_out == nullptr) ||
        (scale == nullptr) != (dscale == nullptr) || (w_in == nullptr) != (dw_in == nullptr) ||
        (dres && !res && T > 0) || (dy && !w_in))
        return H3CONV_ERR_INVALID_ARG;
    if (!norm_sizes_ok(T, D, groups)) return H3CONV_ERR_UNSUPPORTED;
    const size_t need = h3c::block_norm_bwd_workspace(T, D);
    if (need > 0 && (!ws || ws_bytes < need)) return H3CONV_ERR_WORKSPACE;
    const int64_t e = esize(io), n = T * D * e;
    const uintptr_t ea = (uintptr_t)e;
    if (!bufs_ok({{f, n, true, ea}, {res, n, false, ea}, {gate, n, false, ea}, {w_out, D * 4, false, 4},
                  {scale, D * 4, false, 4}, {w_in, D * 4, false, 4}, {dr, n, false, ea}, {dy, n, false, ea}},
                 {{df, n, true, ea}, {dres, n, false, ea}, {dgate, n, false, ea}, {dw_out, D * 4, false, 4},
                  {dscale, D * 4, false, 4}, {dw_in, D * 4, false, 4}, {ws, (int64_t)need, need > 0}}))
        return H3CONV_ERR_INVALID_ARG;
    const h3conv_status s = device_check();
    if (s != H3CONV_OK) return s;
    const h3c::BlockNormArgs a = {f, res, gate, w_out, scale, w_in, T, D, groups, eps};
    const h3c::BlockNormGrads o = {df, dres, dgate, dw_out, dscale, dw_in};
    return from_hip(h3c::launch_block_norm_bwd(a, dr, dy, o, io, ws, (hipStream_t)stream));
}

h3conv_status h3conv_embed(const int64_t *tokens, const void *w, void *y, int64_t T, int64_t D, int64_t V, float scale,
                           int io, void *stream) {
    if (T < 0 || D < 1 || V < 0 || !valid_io(io)) return H3CONV_ERR_INVALID_ARG;
    if (T == 0) return H3CONV_OK;
    if (!embed_sizes_ok(T, D, V)) return H3CONV_ERR_UNSUPPORTED;
    const int64_t e = esize(io);
    const uintptr_t ea = (uintptr_t)e;
    if (!bufs_ok({{tokens, T * 8, true, 8}, {w, V * D * e, true, ea}}, {{y, T * D * e, true, ea}})) return H3CONV_ERR_INVALID_ARG;
    const h3conv_status s = device_check();
    if (s != H3CONV_OK) return s;
    return from_hip(h3c::launch_embed(tokens, w, y, T, D, V, scale, io, (hipStream_t)stream));
}

size_t h3conv_embed_bwd_workspace_size(int64_t T, int64_t D, int64_t V) {
    if (T < 0 || D < 1 || V < 0 || !embed_sizes_ok(T, D, V)) return (size_t)-1;
    return h3c::embed_bwd_workspace(T, D, V);
}

h3conv_status h3conv_embed_bwd(const int64_t *tokens, const void *dy, void *dw, int64_t T, int64_t D, int64_t V,
                               float scale, int io, void *ws, size_t ws_bytes, void *stream) {
    if (T < 0 || D < 1 || V < 0 || !valid_io(io)) return H3CONV_ERR_INVALID_ARG;
    if (V == 0) return H3CONV_OK;
    if (!embed_sizes_ok(T, D, V)) return H3CONV_ERR_UNSUPPORTED;
    const size_t need = h3c::embed_bwd_workspace(T, D, V);
    if (need > 0 && (!ws || ws_bytes < need)) return H3CONV_ERR_WORKSPACE;
    const int64_t e = esize(io);
    const uintptr_t ea = (uintptr_t)e;
    if (!bufs_ok({{tokens, T * 8, true, 8}, {dy, T * D * e, true, ea}}, {{dw, V * D * e, true, ea}, {ws, (int64_t)need, need > 0}}))
        return H3CONV_ERR_INVALID_ARG;
    const h3conv_status s = device_check();
    if (s != H3CONV_OK) return s;
    return from_hip(h3c::launch_embed_bwd(tokens, dy, dw, T, D, V, scale, io, ws, (hipStream_t)stream));
}

}  // extern "C"
