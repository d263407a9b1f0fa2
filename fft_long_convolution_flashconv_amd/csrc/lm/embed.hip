// embed.hip -- rows of a table by token, scaled, and the table's gradient.
//
//   y[t] = scale w[tok[t]],   dw[v] = scale sum_{t: tok[t] = v} dy[t]
// A token outside the table gives a zero row and no gradient.  Both are copies
// with a little arithmetic: HBM bound.  A row's sum runs over its tokens in
// order, in fp32, and is rounded once: equal calls give equal bits.
#include <hip/hip_runtime.h>

#include "lm_device.h"
#include "lm_internal.h"

namespace h3c {
namespace {

constexpr int V = 8;

// One wave per token.
template <int IO>
__global__ __launch_bounds__(256) void k_embed(const int64_t *__restrict__ tok, const typename io_elem<IO>::T *__restrict__ w,
                                               typename io_elem<IO>::T *__restrict__ y, int64_t T, int64_t D, int64_t vocab,
                                               float scale) {
    const int64_t t = block_id() * 4 + (threadIdx.x >> 6);
    if (t >= T) return;
    const int64_t id = tok[t];
    const bool in = id >= 0 && id < vocab;
    for (int64_t c = (threadIdx.x & 63) * V; c < D; c += 64 * V) {
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.f;
        if (in) ld_row<IO, V>(w + id * D + c, v, D - c);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= scale;
        st_row<IO, V>(y + t * D + c, v, D - c);
    }
}

// One wave per row of the table; it looks through all tokens.
template <int IO>
__global__ __launch_bounds__(256) void k_embed_bwd(const int64_t *__restrict__ tok,
                                                   const typename io_elem<IO>::T *__restrict__ dy,
                                                   typename io_elem<IO>::T *__restrict__ dw, int64_t T, int64_t D,
                                                   int64_t vocab, float scale) {
    const int64_t id = block_id() * 4 + (threadIdx.x >> 6);
    if (id >= vocab) return;
    const int lane = threadIdx.x & 63;
    for (int64_t c0 = 0; c0 < D; c0 += 64 * V) {
        const int64_t c = c0 + lane * V;
        float s[V];
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = 0.f;
        for (int64_t t0 = 0; t0 < T; t0 += 64) {
            uint64_t hit = __ballot(t0 + lane < T && tok[t0 + lane < T ? t0 + lane : 0] == id);
            while (hit) {
                const int64_t t = t0 + __builtin_ctzll(hit);
                hit &= hit - 1;
                float v[V];
                ld_row<IO, V>(dy + t * D + c, v, D - c);
#pragma unroll
                for (int i = 0; i < V; ++i) s[i] += v[i];
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] *= scale;
        st_row<IO, V>(dw + id * D + c, s, D - c);
    }
}

template <int IO>
hipError_t fwd_io(const int64_t *tok, const void *w, void *y, int64_t T, int64_t D, int64_t vocab, float scale, hipStream_t s) {
    using E = typename io_elem<IO>::T;
    return launch(k_embed<IO>, grid_of((T + 3) / 4), dim3(256), 0, s, tok, (const E *)w, (E *)y, T, D, vocab, scale);
}
template <int IO>
hipError_t bwd_io(const int64_t *tok, const void *dy, void *dw, int64_t T, int64_t D, int64_t vocab, float scale, hipStream_t s) {
    using E = typename io_elem<IO>::T;
    return launch(k_embed_bwd<IO>, grid_of((vocab + 3) / 4), dim3(256), 0, s, tok, (const E *)dy, (E *)dw, T, D, vocab, scale);
}

}  // namespace

size_t embed_bwd_workspace(int64_t T, int64_t D, int64_t vocab) { return 0; }

hipError_t launch_embed(const int64_t *tok, const void *w, void *y, int64_t T, int64_t D, int64_t vocab, float scale, int io,
                        hipStream_t s) {
    switch (io) {
        case IO_F32: return fwd_io<IO_F32>(tok, w, y, T, D, vocab, scale, s);
        case IO_F16: return fwd_io<IO_F16>(tok, w, y, T, D, vocab, scale, s);
        default: return fwd_io<IO_BF16>(tok, w, y, T, D, vocab, scale, s);
    }
}

hipError_t launch_embed_bwd(const int64_t *tok, const void *dy, void *dw, int64_t T, int64_t D, int64_t vocab, float scale,
                            int io, void *ws, hipStream_t s) {
    switch (io) {
        case IO_F32: return bwd_io<IO_F32>(tok, dy, dw, T, D, vocab, scale, s);
        case IO_F16: return bwd_io<IO_F16>(tok, dy, dw, T, D, vocab, scale, s);
        default: return bwd_io<IO_BF16>(tok, dy, dw, T, D, vocab, scale, s);
    }
}

}  // namespace h3c
