// linear_attn.hip -- linear attention with a decay for each head.
//
// Per sequence and head, with a state S of dk x dv:
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   y_t = scale S_t^T q_t
// and backwards, D_t the gradient of S_t:
//   D_t = scale q_t dy_t^T + e^{g_{t+1}} D_{t+1},
//   dq_t = scale S_t dy_t,  dk_t = D_t v_t,  dv_t = D_t^T k_t,  dg_t = e^{g_t} <S_{t-1}, D_t>
// All four sequences y, dq, dk and dv are one recurrence over other tensors:
//   X_t = e^{..} X + upd b_t c_t^T,  o_t = out X_t^T a_t
//   y:  (a, b, c) = (q, k, v),        dq: (dy, v, k), the state transposed,
//   dv: (k, q, dy) from the end on,   dk: (v, dy, q) from the end on, transposed.
// From <S_t, D_t> = dg_t + k_t.dk_t = q_t.dq_t + dg_{t+1} the decays' gradients are
// sums over time, dg_t = dg_{t+1} + q_t.dq_t - k_t.dk_t, where the step's own
// products are in both and are left out of both.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "lm_device.h"
#include "lm_internal.h"

namespace h3c {
namespace {

// A factor e^g of g below this is zero in fp32, and so is what follows from it.
constexpr float kLeast = -200.f, kZeroBelow = -104.f;

// One tensor of tokens and heads, [B,N,heads,dim] with `ld` elements between tokens.
struct Seq {
    const void *p;
    int64_t ld;
    int share, dim;  // heads that share one of the tensor's
};

struct Role {
    Seq a, b, c, e;      // read by the state; rows; columns; what the outputs' dot products are taken with
    void *o;             // [B,N,H,M] in the io type, or fp32 if wide
    float *dot;          // [column tiles][B,H,N]: e_t . (o_t without the step's own product), or null
    const float *s0;     // the state before the first step, or null
    float *s1;           // and behind the last, or null
    int rs, cs;          // of the states: between rows, between columns
    float out, upd;
    int reverse, wide;
};
struct Roles {
    Role r[3];
};

struct Shape {
    int64_t B, N, H;
    const float *g;
    const int32_t *lengths;
    int per_token;
};

constexpr int kCols = 64, kStep = 16;

// Step by step: 64 columns of a state per block, its rows over four threads each.
template <int IO, int KP>
__global__ __launch_bounds__(256) void k_lin_rec(Roles roles, Shape s) {
    using T = typename io_elem<IO>::T;
    const Role &r = roles.r[blockIdx.y];
    const int K = r.a.dim, M = r.c.dim, tiles = (M + kCols - 1) / kCols;
    constexpr int R = KP / 4;
    __shared__ float la[kStep][KP], lb[kStep][KP], part[2][kStep][4][kCols], dec[kStep];
    const int64_t id = block_id();
    const int tile = (int)(id % 4), col = tile * kCols + (int)(threadIdx.x & 63), rg = threadIdx.x >> 6;
    const int64_t bh = id / 4;
    if (bh >= s.B * s.H || tile >= tiles) return;
    const int64_t b = bh / s.H, h = bh - b * s.H, n = row_len(s.lengths, b, s.N);
    const auto row = [&](const Seq &q, int64_t t) {
        return (const T *)q.p + (b * s.N + t) * q.ld + h / q.share * q.dim;
    };
    const bool on = col < M;
    float x[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int k = rg + 4 * i;
        x[i] = r.s0 && on && k < K ? r.s0[bh * K * M + (int64_t)k * r.rs + (int64_t)col * r.cs] : 0.f;
    }
    for (int64_t i0 = 0; i0 < n; i0 += kStep) {
        const int m = (int)std::min<int64_t>(kStep, n - i0);
        const auto time = [&](int j) { return r.reverse ? n - 1 - (i0 + j) : i0 + j; };
        __syncthreads();
        for (int q = threadIdx.x; q < kStep * KP; q += 256) {
            const int j = q / KP, k = q % KP;
            const bool ok = j < m && k < K;
            la[j][k] = ok ? to_f<IO>(row(r.a, time(j))[k]) : 0.f;
            lb[j][k] = ok ? to_f<IO>(row(r.b, time(j))[k]) * r.upd : 0.f;
        }
        if (threadIdx.x < kStep) {
            float g = 0.f;
            if ((int)threadIdx.x < m) g = s.per_token ? s.g[(b * s.N + time(threadIdx.x)) * s.H + h] : s.g[h];
            dec[threadIdx.x] = __builtin_amdgcn_exp2f(g * kLog2e);
        }
        __syncthreads();
        for (int j = 0; j < m; ++j) {
            const float c = on ? to_f<IO>(row(r.c, time(j))[col]) : 0.f, e = dec[j];
            float before = 0.f, after = 0.f;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float a = la[j][rg + 4 * i];
                if (!r.reverse) x[i] *= e;
                before = fmaf(a, x[i], before);
                x[i] = fmaf(lb[j][rg + 4 * i], c, x[i]);
                after = fmaf(a, x[i], after);
                if (r.reverse) x[i] *= e;
            }
            part[0][j][rg][threadIdx.x & 63] = before;
            part[1][j][rg][threadIdx.x & 63] = after;
        }
        __syncthreads();
        for (int j = rg; j < m; j += 4) {
            const int l = threadIdx.x & 63;
            const auto sum = [&](int w) { return ((part[w][j][0][l] + part[w][j][1][l]) + part[w][j][2][l]) + part[w][j][3][l]; };
            const int64_t t = time(j), at = ((b * s.N + t) * s.H + h) * M + col;
            const float o = sum(1) * r.out;
            if (on) {
                if (r.wide) ((float *)r.o)[at] = o;
                else ((T *)r.o)[at] = from_f<IO>(o);
            }
            if (r.dot) {
                float d = on ? sum(0) * r.out * to_f<IO>(row(r.e, t)[col]) : 0.f;
#pragma unroll
                for (int k = 1; k < 64; k <<= 1) d += __shfl_xor(d, k);
                if (l == 0) r.dot[(tile * s.B * s.H + bh) * s.N + t] = d;
            }
        }
    }
    for (int64_t t = n + rg; t < s.N; t += 4)
        if (on) {
            const int64_t at = ((b * s.N + t) * s.H + h) * M + col;
            if (r.wide) ((float *)r.o)[at] = 0.f;
            else ((T *)r.o)[at] = T(0);
        }
    if (r.s1 && on) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int k = rg + 4 * i;
            if (k < K) r.s1[bh * K * M + (int64_t)k * r.rs + (int64_t)col * r.cs] = x[i];
        }
    }
}

// dg of one sequence and head from the dot products, from the end on, in 64 bits.
__global__ __launch_bounds__(256) void k_lin_dg(const float *__restrict__ dq, const float *__restrict__ dk, int tiles_q,
                                                int tiles_k, const float *__restrict__ s_end,
                                                const float *__restrict__ ds_end, int64_t kv, Shape s, float *dg,
                                                double *sums) {
    __shared__ double lds[256];
    const int64_t bh = block_id();
    if (bh >= s.B * s.H) return;
    const int64_t b = bh / s.H, h = bh - b * s.H, n = row_len(s.lengths, b, s.N), plane = s.B * s.H * s.N;
    const int tid = threadIdx.x;
    double carry = 0.0, total = 0.0;
    if (ds_end) {
        double v = 0.0;
        for (int64_t i = tid; i < kv; i += 256) v += (double)s_end[bh * kv + i] * ds_end[bh * kv + i];
        lds[tid] = v;
        __syncthreads();
        for (int d = 128; d > 0; d >>= 1) {
            if (tid < d) lds[tid] += lds[tid + d];
            __syncthreads();
        }
        carry = lds[0];
        __syncthreads();
    }
    for (int64_t i0 = 0; i0 < n; i0 += 256) {  // from the end
        const int64_t t = n - 1 - i0 - tid;
        double v = 0.0;
        if (t >= 0) {
            for (int i = 0; i < tiles_q; ++i) v += dq[i * plane + bh * s.N + t];
            for (int i = 0; i < tiles_k; ++i) v -= dk[i * plane + bh * s.N + t];
        }
        lds[tid] = v;
        __syncthreads();
        for (int d = 1; d < 256; d <<= 1) {
            const double u = tid >= d ? lds[tid - d] : 0.0;
            __syncthreads();
            lds[tid] += u;
            __syncthreads();
        }
        if (t >= 0) {
            const float g = s.per_token ? s.g[(b * s.N + t) * s.H + h] : s.g[h];
            const double d = g < kZeroBelow ? 0.0 : carry + lds[tid];
            if (s.per_token) dg[(b * s.N + t) * s.H + h] = (float)d;
            else total += d;
        }
        carry += lds[255];
        __syncthreads();
    }
    if (s.per_token) {
        for (int64_t t = n + tid; t < s.N; t += 256) dg[(b * s.N + t) * s.H + h] = 0.f;
    } else {
        lds[tid] = total;
        __syncthreads();
        for (int d = 128; d > 0; d >>= 1) {
            if (tid < d) lds[tid] += lds[tid + d];
            __syncthreads();
        }
        if (tid == 0) sums[bh] = lds[0];
    }
}

// dg of a decay per head: the sequences' sums, in order.
__global__ void k_lin_dg_heads(const double *__restrict__ sums, float *dg, int64_t B, int64_t H) {
    const int64_t h = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (h >= H) return;
    double v = 0.0;
    for (int64_t b = 0; b < B; ++b) v += sums[b * H + h];
    dg[h] = (float)v;
}

// Gradients of shared heads: the sum over a group's heads, in order.
template <int IO>
__global__ __launch_bounds__(256) void k_lin_share(const float *__restrict__ wide, typename io_elem<IO>::T *__restrict__ o,
                                                   int64_t n, int dim, int share) {
    const int64_t i = block_id() * 256 + threadIdx.x;
    if (i >= n) return;
    const int64_t g = i / dim, c = i - g * dim;
    float s = 0.f;
    for (int j = 0; j < share; ++j) s += wide[(g * share + j) * dim + c];
    o[i] = from_f<IO>(s);
}

// One token of each sequence: a block per sequence and head.
template <int IO>
__global__ __launch_bounds__(256) void k_lin_step(LinStepArgs s) {
    using T = typename io_elem<IO>::T;
    __shared__ float lds[256];
    const int64_t bh = block_id();
    if (bh >= s.B * s.H) return;
    const int64_t b = bh / s.H, h = bh - b * s.H, grp = h / (s.H / s.G);
    const int64_t slot = s.slots ? s.slots[b] : b;
    T *y = (T *)s.y + bh * s.dv;
    if (slot < 0 || slot >= s.P) {
        for (int c = threadIdx.x; c < s.dv; c += 256) y[c] = T(0);
        return;
    }
    const T *q = (const T *)s.q + b * s.ldq + grp * s.dk, *k = (const T *)s.k + b * s.ldk + grp * s.dk;
    const T *v = (const T *)s.v + b * s.ldv + h * s.dv;
    const float e = __builtin_amdgcn_exp2f((s.per_token ? s.g[b * s.H + h] : s.g[h]) * kLog2e);
    const float *from = s.x_in + (slot * s.H + h) * s.dk * s.dv;
    float *to = s.x_out + (slot * s.H + h) * s.dk * s.dv;
    const int rg = threadIdx.x >> 6;
    for (int c0 = 0; c0 < s.dv; c0 += 64) {
        const int c = c0 + (threadIdx.x & 63);
        float sum = 0.f;
        if (c < s.dv) {
            const float vc = to_f<IO>(v[c]);
            for (int i = rg; i < s.dk; i += 4) {
                const float x = fmaf(to_f<IO>(k[i]), vc, e * from[(int64_t)i * s.dv + c]);
                to[(int64_t)i * s.dv + c] = x;
                sum = fmaf(to_f<IO>(q[i]), x, sum);
            }
        }
        __syncthreads();
        lds[threadIdx.x] = sum;
        __syncthreads();
        if (rg == 0 && c < s.dv) {
            const float o = ((lds[threadIdx.x] + lds[threadIdx.x + 64]) + lds[threadIdx.x + 128]) + lds[threadIdx.x + 192];
            y[c] = from_f<IO>(o * s.scale);
        }
    }
}

int tiles_of(int64_t dim) { return (int)((dim + kCols - 1) / kCols); }

template <int IO>
hipError_t run_roles(const Roles &r, int n, const Shape &s, int K, hipStream_t st) {
    dim3 grid = grid_of(s.B * s.H * 4, (unsigned)n);
    if (K <= 64) return launch(k_lin_rec<IO, 64>, grid, dim3(256), 0, st, r, s);
    if (K <= 128) return launch(k_lin_rec<IO, 128>, grid, dim3(256), 0, st, r, s);
    return launch(k_lin_rec<IO, 256>, grid, dim3(256), 0, st, r, s);
}

// The parts of the backward pass's workspace, in bytes from its start.
struct BwdSpace {
    int64_t row, col, s_end, sums, dq, dk, all;
};
int64_t up(int64_t n) { return (n + 255) & ~(int64_t)255; }
BwdSpace space_of(int64_t B, int64_t N, int64_t H, int64_t G, int64_t dk, int64_t dv) {
    BwdSpace w;
    const int64_t dots = up(tiles_of(dk) * B * H * N * 4), wide = G < H ? up(B * N * H * dk * 4) : 0;
    int64_t at = 0;
    const auto take = [&](int64_t n) { const int64_t p = at; at += n; return p; };
    w.row = take(dots);
    w.col = take(dots);
    w.s_end = take(up(B * H * dk * dv * 4));
    w.sums = take(up(B * H * 8));
    w.dq = take(wide);
    w.dk = take(wide);
    w.all = at;
    return w;
}

Shape shape_of(const LinAttnArgs &a) { return {a.B, a.N, a.H, a.g, a.lengths, a.per_token}; }

template <int IO>
hipError_t fwd_io(const LinAttnArgs &a, void *y, float *x_out, hipStream_t s) {
    const int share = (int)(a.H / a.G);
    const Seq q = {a.q, a.ldq, share, a.dk}, k = {a.k, a.ldk, share, a.dk}, v = {a.v, a.ldv, 1, a.dv};
    Roles r = {};
    r.r[0] = {q, k, v, v, y, nullptr, a.x_in, x_out, a.dv, 1, a.scale, 1.f, 0, 0};
    return run_roles<IO>(r, 1, shape_of(a), a.dk, s);
}

template <int IO>
hipError_t bwd_io(const LinAttnArgs &a, const void *dy_, const float *dx_out, const LinAttnGrads &o, void *ws, hipStream_t st) {
    using T = typename io_elem<IO>::T;
    const int share = (int)(a.H / a.G), wide = share > 1;
    const BwdSpace w = space_of(a.B, a.N, a.H, a.G, a.dk, a.dv);
    char *base = (char *)ws;
    const Shape s = shape_of(a);
    const Seq q = {a.q, a.ldq, share, a.dk}, k = {a.k, a.ldk, share, a.dk}, v = {a.v, a.ldv, 1, a.dv};
    const Seq dy = {dy_, a.H * a.dv, 1, a.dv};
    float *row = (float *)(base + w.row), *col = (float *)(base + w.col), *s_end = (float *)(base + w.s_end);
    void *dq = wide ? base + w.dq : o.dq, *dk = wide ? base + w.dk : o.dk;
    Roles r = {};
    r.r[0] = {dy, v, k, q, dq, o.dg ? row : nullptr, a.x_in, dx_out ? s_end : nullptr, 1, a.dv, a.scale, 1.f, 0, wide};
    r.r[1] = {v, dy, q, k, dk, o.dg ? col : nullptr, dx_out, nullptr, 1, a.dv, 1.f, a.scale, 1, wide};
    r.r[2] = {k, q, dy, dy, o.dv, nullptr, dx_out, o.dx_in, a.dv, 1, 1.f, a.scale, 1, 0};
    hipError_t e = a.B > 0 ? run_roles<IO>(r, 3, s, std::max(a.dk, a.dv), st) : hipSuccess;
    if (e != hipSuccess) return e;
    const int64_t n = a.B * a.N * a.G * a.dk;
    if (wide && n > 0) {
        for (int i = 0; i < 2; ++i) {
            e = launch(k_lin_share<IO>, grid_of((n + 255) / 256), dim3(256), 0, st, (const float *)(i ? dk : dq),
                       (T *)(i ? o.dk : o.dq), n, a.dk, share);
            if (e != hipSuccess) return e;
        }
    }
    if (!o.dg) return hipSuccess;
    double *sums = (double *)(base + w.sums);
    if (a.B > 0)
        e = launch(k_lin_dg, grid_of(a.B * a.H), dim3(256), 0, st, row, col, tiles_of(a.dk), tiles_of(a.dk), s_end, dx_out,
                   (int64_t)a.dk * a.dv, s, o.dg, sums);
    if (e != hipSuccess || a.per_token) return e;
    return launch(k_lin_dg_heads, dim3((unsigned)((a.H + 255) / 256)), dim3(256), 0, st, sums, o.dg, a.B, a.H);
}

}  // namespace

size_t linear_attn_workspace(int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

size_t linear_attn_bwd_workspace(int64_t B, int64_t N, int64_t H, int64_t G, int64_t dk, int64_t dv) {
    return (size_t)space_of(B, N, H, G, dk, dv).all;
}

hipError_t launch_linear_attn(const LinAttnArgs &a, void *y, float *x_out, int io, void *ws, hipStream_t s) {
    switch (io) {
        case IO_F32: return fwd_io<IO_F32>(a, y, x_out, s);
        case IO_F16: return fwd_io<IO_F16>(a, y, x_out, s);
        default: return fwd_io<IO_BF16>(a, y, x_out, s);
    }
}

hipError_t launch_linear_attn_bwd(const LinAttnArgs &a, const void *dy, const float *dx_out, const LinAttnGrads &o, int io,
                                  void *ws, hipStream_t s) {
    switch (io) {
        case IO_F32: return bwd_io<IO_F32>(a, dy, dx_out, o, ws, s);
        case IO_F16: return bwd_io<IO_F16>(a, dy, dx_out, o, ws, s);
        default: return bwd_io<IO_BF16>(a, dy, dx_out, o, ws, s);
    }
}

hipError_t launch_linear_attn_step(const LinStepArgs &a, int io, hipStream_t s) {
    switch (io) {
        case IO_F32: return launch(k_lin_step<IO_F32>, grid_of(a.B * a.H), dim3(256), 0, s, a);
        case IO_F16: return launch(k_lin_step<IO_F16>, grid_of(a.B * a.H), dim3(256), 0, s, a);
        default: return launch(k_lin_step<IO_BF16>, grid_of(a.B * a.H), dim3(256), 0, s, a);
    }
}

}  // namespace h3c
