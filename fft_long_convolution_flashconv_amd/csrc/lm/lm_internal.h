// lm_internal.h -- launchers of the selective state-space and language-model
// loss kernels, shared between their C-ABI shim and the kernel translation
// units.  As in h3conv_internal.h: arguments were validated by the shim, a
// launcher only enqueues work on `s` and returns the launch status.
#pragma once

#include "../h3conv_internal.h"

namespace h3c {

// A dispatch takes fewer than 2^32 threads along x.  A grid of n blocks (of up
// to 1024 threads): along x, and past kGridX of them along z.  The last of
// several z may hold blocks numbered n and up, which have nothing to do.
constexpr int64_t kGridX = (int64_t)1 << 21;
inline dim3 grid_of(int64_t n, unsigned y = 1) {
    return n <= kGridX ? dim3((unsigned)n, y, 1) : dim3((unsigned)kGridX, y, (unsigned)((n + kGridX - 1) / kGridX));
}

// ------------------------------------------------------------ short_conv
struct ShortConvArgs {
    const void *x, *x_in;        // [B,H,N], [B,H,W-1] or null
    const float *w, *bias;       // [H,W], [H] or null
    const int32_t *lengths;      // [B] or null
    int64_t B, H, N;
    int W, silu;
};
hipError_t launch_short_conv(const ShortConvArgs &a, void *y, void *x_out, int io, hipStream_t s);
hipError_t launch_short_conv_bwd(const ShortConvArgs &a, const void *dy, const void *dx_out, void *dx, float *dw,
                                 float *dbias, void *dx_in, int io, void *ws, hipStream_t s);
size_t short_conv_bwd_workspace(int64_t B, int64_t H, int64_t N, int W);
hipError_t launch_short_conv_step(const void *x, const float *w, const float *bias, const int32_t *slots,
                                  const void *st_in, void *st_out, void *y, int64_t B, int64_t H, int64_t P, int W,
                                  int silu, int io, hipStream_t s);

// -------------------------------------------------------- selective_scan
// Samples between two saved states of a training pass.
constexpr int kSelChunk = 128;

struct SelArgs {
    const void *u, *dt, *Bm, *C, *z;                 // [B,H,N] (z may be null), [B,G,S,N]
    const float *A, *D, *dt_bias, *x_in;             // [H,S], [H] or null, [H] or null, [B,H,S] or null
    const int32_t *lengths;                          // [B] or null
    int64_t B, H, N;
    int S, G, softplus;
};
hipError_t launch_selective_scan(const SelArgs &a, void *y, float *x_out, float *saved, int io, hipStream_t s);

struct SelGrads {
    void *du, *ddt, *dB, *dC, *dz;                   // dz null without a gate
    float *dA, *dD, *ddt_bias, *dx_in;               // dD, ddt_bias, dx_in may be null
};
hipError_t launch_selective_scan_bwd(const SelArgs &a, const float *saved, const void *dy, const float *dx_out,
                                     const SelGrads &g, int io, void *ws, hipStream_t s);
size_t selective_saved_floats(int64_t B, int64_t H, int64_t N, int64_t S);
size_t selective_bwd_workspace(int64_t B, int64_t H, int64_t N, int64_t S, int64_t G);
hipError_t launch_selective_step(const void *u, const void *dt, const float *A, const void *Bm, const void *C,
                                 const float *D, const void *z, const float *dt_bias, const int32_t *slots,
                                 const float *x_in, float *x_out, void *y, int64_t B, int64_t H, int64_t P, int S,
                                 int G, int softplus, int io, hipStream_t s);

// ----------------------------------------------------------- linear_xent
size_t linear_xent_workspace(int64_t T, int64_t D, int64_t V, int io, bool bwd);
hipError_t launch_linear_xent(const void *x, const void *w, const int64_t *labels, int64_t ignore, float *loss,
                              float *lse, int64_t T, int64_t D, int64_t V, int io, void *ws, hipStream_t s);
hipError_t launch_linear_xent_bwd(const void *x, const void *w, const int64_t *labels, int64_t ignore,
                                  const float *lse, const float *dloss, void *dx, void *dw, int64_t T, int64_t D,
                                  int64_t V, int io, void *ws, hipStream_t s);

// ----------------------------------------------------------- linear_attn
struct LinAttnArgs {
    const void *q, *k, *v;                           // [B,N,G,dk] twice, [B,N,H,dv]; ld elements between tokens
    const float *g, *x_in;                           // [H] or [B,N,H], [B,H,dk,dv] or null
    const int32_t *lengths;                          // [B] or null
    int64_t B, N, H, G;
    int dk, dv;
    int64_t ldq, ldk, ldv;
    float scale;
    int per_token;
};
struct LinAttnGrads {
    void *dq, *dk, *dv;
    float *dg, *dx_in;                               // may be null
};
struct LinStepArgs {
    const void *q, *k, *v;                           // [B,G,dk] twice, [B,H,dv]; ld elements between sequences
    const float *g, *x_in;                           // [H] or [B,H], [P,H,dk,dv]
    const int32_t *slots;
    float *x_out;
    void *y;
    int64_t B, H, G, P;
    int dk, dv;
    int64_t ldq, ldk, ldv;
    float scale;
    int per_token;
};
size_t linear_attn_workspace(int64_t B, int64_t N, int64_t H, int64_t dk, int64_t dv);
size_t linear_attn_bwd_workspace(int64_t B, int64_t N, int64_t H, int64_t G, int64_t dk, int64_t dv);
hipError_t launch_linear_attn(const LinAttnArgs &a, void *y, float *x_out, int io, void *ws, hipStream_t s);
hipError_t launch_linear_attn_bwd(const LinAttnArgs &a, const void *dy, const float *dx_out, const LinAttnGrads &o, int io,
                                  void *ws, hipStream_t s);
hipError_t launch_linear_attn_step(const LinStepArgs &a, int io, hipStream_t s);

// ------------------------------------------------------------ block_norm
struct BlockNormArgs {
    const void *f, *res, *gate;                      // [T,D]; res, gate may be null
    const float *w_out, *scale, *w_in;               // [D] or null
    int64_t T, D, groups;
    float eps;
};
struct BlockNormGrads {
    void *df, *dres, *dgate;                         // dres, dgate null without a res, a gate
    float *dw_out, *dscale, *dw_in;                  // null without their parameters
};
hipError_t launch_block_norm(const BlockNormArgs &a, void *r, void *y, int io, hipStream_t s);
size_t block_norm_bwd_workspace(int64_t T, int64_t D);
hipError_t launch_block_norm_bwd(const BlockNormArgs &a, const void *dr, const void *dy, const BlockNormGrads &o, int io,
                                 void *ws, hipStream_t s);

// ----------------------------------------------------------------- embed
hipError_t launch_embed(const int64_t *tok, const void *w, void *y, int64_t T, int64_t D, int64_t vocab, float scale, int io,
                        hipStream_t s);
size_t embed_bwd_workspace(int64_t T, int64_t D, int64_t vocab);
hipError_t launch_embed_bwd(const int64_t *tok, const void *dy, void *dw, int64_t T, int64_t D, int64_t vocab, float scale,
                            int io, void *ws, hipStream_t s);

}  // namespace h3c
