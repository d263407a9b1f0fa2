// short_conv.hip -- short causal depthwise convolution with bias and SiLU.
//
// Per channel h and step t, with W <= 4 taps:
//   p_t = bias[h] + sum_{i<W} w[h,i] x_{t-i},   y_t = silu(p_t) or p_t,
// the tap order of the shift SSM in the H3 mix (w[h,0] on the current input).
// Inputs before the row's start come from x_in (the last W-1 inputs of the
// previous piece, oldest first) or are zero.  About 2W + 5 operations per
// element against 4 to 8 bytes: HBM bound in both directions.
#include <hip/hip_runtime.h>

#include "lm_device.h"
#include "lm_internal.h"

namespace h3c {
namespace {

constexpr int kThreads = 256;
constexpr int kTaps = 4;  // taps and halo are held for the largest W; missing taps are zero

// Threads of a block along one row (a power of two), the others take rows.
__host__ __device__ inline int threads_per_row(int64_t nvec) {
    int t = 1;
    while (t < kThreads && t < nvec) t <<= 1;
    return t;
}

__device__ __forceinline__ int64_t row_len(const int32_t *lengths, int64_t b, int64_t N) {
    if (!lengths) return N;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : (n > N ? N : n);
}

// x at position p of a row that starts at p = -(W-1), the first W-1 from the
// saved inputs
template <int IO>
__device__ __forceinline__ float at_ext(const typename io_elem<IO>::T *x, const typename io_elem<IO>::T *xin,
                                        int64_t p, int W) {
    if (p >= 0) return to_f<IO>(x[p]);
    return (xin && p >= -(int64_t)(W - 1)) ? to_f<IO>(xin[p + W - 1]) : 0.f;
}

__device__ __forceinline__ void load_taps(const float *w, int64_t h, int W, float (&tap)[kTaps]) {
#pragma unroll
    for (int i = 0; i < kTaps; ++i) tap[i] = i < W ? w[h * W + i] : 0.f;
}

template <int IO>
__global__ __launch_bounds__(kThreads) void k_short_conv(const typename io_elem<IO>::T *__restrict__ x,
                                                         const typename io_elem<IO>::T *__restrict__ x_in,
                                                         const float *__restrict__ w, const float *__restrict__ bias,
                                                         const int32_t *__restrict__ lengths,
                                                         typename io_elem<IO>::T *__restrict__ y,
                                                         typename io_elem<IO>::T *__restrict__ x_out, int64_t B,
                                                         int64_t H, int64_t N, int W, int silu, int tpr) {
    using T = typename io_elem<IO>::T;
    constexpr int V = 16 / (int)sizeof(T);
    const int64_t r = (int64_t)blockIdx.x * (kThreads / tpr) + threadIdx.x / tpr;
    if (r >= B * H) return;
    const int64_t b = r / H, h = r - b * H;
    const int64_t len = row_len(lengths, b, N);
    const T *xr = x + r * N, *xi = x_in ? x_in + r * (W - 1) : nullptr;
    const int tl = (int)threadIdx.x % tpr;
    float tap[kTaps];
    load_taps(w, h, W, tap);
    const float bs = bias ? bias[h] : 0.f;
    if (x_out && blockIdx.y == 0)
        for (int j = tl; j < W - 1; j += tpr) x_out[r * (W - 1) + j] = from_f<IO>(at_ext<IO>(xr, xi, len - (W - 1) + j, W));
    for (int64_t t0 = ((int64_t)blockIdx.y * tpr + tl) * V; t0 < N; t0 += (int64_t)gridDim.y * tpr * V) {
        float v[V + kTaps - 1], o[V];
        {
            float cur[V];
            ld_row<IO, V>(xr + t0, cur, len - t0);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i + kTaps - 1] = cur[i];
        }
        if (t0 >= V && t0 < len) {
            float pre[V];
            ld_row<IO, V>(xr + t0 - V, pre);
#pragma unroll
            for (int i = 0; i < kTaps - 1; ++i) v[i] = pre[V - (kTaps - 1) + i];
        } else {
#pragma unroll
            for (int i = 0; i < kTaps - 1; ++i) v[i] = t0 < len ? at_ext<IO>(xr, xi, t0 - (kTaps - 1) + i, W) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float p = bs;
#pragma unroll
            for (int k = 0; k < kTaps; ++k)
                if (k < W) p = fmaf(tap[k], v[i + kTaps - 1 - k], p);
            if (silu) p *= sigmoid(p);
            o[i] = t0 + i < len ? p : 0.f;
        }
        st_row<IO, V>(y + r * N + t0, o, N - t0);
    }
}

// d p_t = dy_t silu'(p_t) at one step
__device__ __forceinline__ float act_bwd(float p, float dy, int silu) {
    if (!silu) return dy;
    const float s = sigmoid(p);
    return dy * s * (1.f + p * (1.f - s));
}

// Backward pass of one channel: block (h, k) takes the tasks k, k + K, ... of
// the channel's B rows cut into pieces, so the sums over batch and time stay
// in one block's registers and are joined in a fixed order:
//   dx_s = sum_i w_i dp_{s+i},  dw_i = sum_{b,t} dp_t x_{t-i},  dbias = sum dp.
template <int IO>
__global__ __launch_bounds__(kThreads) void k_short_conv_bwd(
    const typename io_elem<IO>::T *__restrict__ x, const typename io_elem<IO>::T *__restrict__ x_in,
    const float *__restrict__ w, const float *__restrict__ bias, const int32_t *__restrict__ lengths,
    const typename io_elem<IO>::T *__restrict__ dy, const typename io_elem<IO>::T *__restrict__ dx_out,
    typename io_elem<IO>::T *__restrict__ dx, typename io_elem<IO>::T *__restrict__ dx_in, float *__restrict__ part,
    int64_t B, int64_t H, int64_t N, int W, int silu, int tpr, int64_t pieces) {
    using T = typename io_elem<IO>::T;
    constexpr int V = 16 / (int)sizeof(T), E = V + kTaps - 1;
    const int64_t h = blockIdx.x;
    const int rpb = kThreads / tpr, tl = (int)threadIdx.x % tpr;
    float tap[kTaps];
    load_taps(w, h, W, tap);
    const float bs = bias ? bias[h] : 0.f;
    float sw[kTaps] = {0.f, 0.f, 0.f, 0.f}, sb = 0.f;
    const int64_t tasks = (B + rpb - 1) / rpb * pieces;
    for (int64_t task = blockIdx.y; task < tasks; task += gridDim.y) {
        const int64_t b = task / pieces * rpb + threadIdx.x / tpr, t0 = (task % pieces * tpr + tl) * V;
        if (b >= B || (t0 >= N && t0 > 0)) continue;  // (step 0 of an empty row: dx_in alone)
        const int64_t r = b * H + h, len = row_len(lengths, b, N);
        const T *xr = x + r * N, *xi = x_in ? x_in + r * (W - 1) : nullptr, *gr = dy + r * N;
        // v[j]: x at t0 - (kTaps-1) + j, for the steps t0 .. t0 + V + kTaps - 2
        float v[E + kTaps - 1], g[E], dp[E], o[V];
#pragma unroll
        for (int j = 0; j < E + kTaps - 1; ++j) {
            const int64_t p = t0 - (kTaps - 1) + j;
            v[j] = p < len ? at_ext<IO>(xr, xi, p, W) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < E; ++j) g[j] = t0 + j < len ? to_f<IO>(gr[t0 + j]) : 0.f;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            float p = bs;
#pragma unroll
            for (int k = 0; k < kTaps; ++k)
                if (k < W) p = fmaf(tap[k], v[j + kTaps - 1 - k], p);
            dp[j] = t0 + j < len ? act_bwd(p, g[j], silu) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float a = 0.f;
#pragma unroll
            for (int k = 0; k < kTaps; ++k)
                if (k < W) a = fmaf(tap[k], dp[j + k], a);
            // the saved last inputs are inputs len-(W-1) .. len-1
            const int64_t q = t0 + j - (len - (W - 1));
            if (dx_out && q >= 0 && q < W - 1) a += to_f<IO>(dx_out[r * (W - 1) + q]);
            o[j] = t0 + j < len ? a : 0.f;
            sb += dp[j];
#pragma unroll
            for (int k = 0; k < kTaps; ++k) sw[k] = fmaf(dp[j], v[j + kTaps - 1 - k], sw[k]);
        }
        st_row<IO, V>(dx + r * N + t0, o, N - t0);
        if (dx_in && t0 == 0) {
            // saved input j stands at position j - (W-1): it meets the steps
            // 0 .. j through the taps W-1-j .. W-1; with len < W-1 it is also
            // kept as the saved input j - len of the next piece
            for (int j = 0; j < W - 1; ++j) {
                float a = 0.f;
#pragma unroll
                for (int k = 0; k < kTaps - 1; ++k)
                    if (k <= j && W - 1 - j + k < W) a = fmaf(w[h * W + W - 1 - j + k], dp[k], a);
                if (dx_out && j >= len) a += to_f<IO>(dx_out[r * (W - 1) + j - len]);
                dx_in[r * (W - 1) + j] = from_f<IO>(a);
            }
        }
    }
    // joined over the block in a fixed order
    __shared__ float red[kTaps + 1][kThreads / 64];
#pragma unroll
    for (int k = 0; k <= kTaps; ++k) {
        float s = k < kTaps ? sw[k] : sb;
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) s += __shfl_xor(s, m);
        if ((threadIdx.x & 63) == 0) red[k][threadIdx.x >> 6] = s;
    }
    __syncthreads();
    if (threadIdx.x <= kTaps) {
        float s = 0.f;
        for (int i = 0; i < kThreads / 64; ++i) s += red[threadIdx.x][i];
        part[((int64_t)blockIdx.y * H + h) * (kTaps + 1) + threadIdx.x] = s;
    }
}

__global__ void k_short_conv_sums(const float *__restrict__ part, float *__restrict__ dw, float *__restrict__ dbias,
                                  int64_t H, int W, int K) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t h = i / (kTaps + 1);
    const int k = (int)(i - h * (kTaps + 1));
    if (h >= H) return;
    float s = 0.f;
    for (int j = 0; j < K; ++j) s += part[((int64_t)j * H + h) * (kTaps + 1) + k];
    if (k < W) dw[h * W + k] = s;
    else if (k == kTaps && dbias) dbias[h] = s;
}

// One token per sequence: the saved inputs of slot slots[b] move on by one.
// A slot outside the pool leaves its row's output zero and no state changed.
template <int IO>
__global__ __launch_bounds__(kThreads) void k_short_conv_step(
    const typename io_elem<IO>::T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ bias,
    const int32_t *__restrict__ slots, const typename io_elem<IO>::T *st_in, typename io_elem<IO>::T *st_out,
    typename io_elem<IO>::T *__restrict__ y, int64_t B, int64_t H, int64_t P, int W, int silu) {
    using T = typename io_elem<IO>::T;
    const int64_t h = (int64_t)blockIdx.x * kThreads + threadIdx.x, b = blockIdx.y;
    if (h >= H) return;
    const int64_t slot = slots ? (int64_t)slots[b] : b;
    if (slot < 0 || slot >= P) {
        y[b * H + h] = from_f<IO>(0.f);
        return;
    }
    const T cur = x[b * H + h];
    const int64_t o = (slot * H + h) * (W - 1);
    float p = (bias ? bias[h] : 0.f);
    p = fmaf(w[h * W], to_f<IO>(cur), p);
    T old[kTaps];
#pragma unroll
    for (int j = 0; j < kTaps - 1; ++j)
        if (j < W - 1) {
            old[j] = st_in[o + j];
            p = fmaf(w[h * W + W - 1 - j], to_f<IO>(old[j]), p);
        }
#pragma unroll
    for (int j = 0; j < kTaps - 1; ++j)
        if (j < W - 1) st_out[o + j] = j + 1 < W - 1 ? old[j + 1] : cur;
    if (silu) p *= sigmoid(p);
    y[b * H + h] = from_f<IO>(p);
}

int bwd_splits(int64_t B, int64_t H, int64_t N, int64_t *pieces, int *tpr, int V) {
    const int64_t nvec = (N + V - 1) / V;
    *tpr = threads_per_row(nvec);
    *pieces = nvec > 0 ? (nvec + *tpr - 1) / *tpr : 1;
    const int rpb = kThreads / *tpr;
    const int64_t tasks = (B + rpb - 1) / rpb * *pieces;
    // about 2048 blocks fill the chip; each join costs one more partial sum
    int64_t k = (2048 + H - 1) / H;
    if (k > tasks) k = tasks;
    if (k > 256) k = 256;
    return (int)(k < 1 ? 1 : k);
}

}  // namespace

size_t short_conv_bwd_workspace(int64_t B, int64_t H, int64_t N, int W) {
    int64_t pieces;
    int tpr;
    const int k16 = bwd_splits(B, H, N, &pieces, &tpr, 8), k32 = bwd_splits(B, H, N, &pieces, &tpr, 4);
    return (size_t)(k16 > k32 ? k16 : k32) * (size_t)H * (kTaps + 1) * 4;
}

template <int IO>
static hipError_t short_conv_io(const ShortConvArgs &a, void *y, void *x_out, hipStream_t s) {
    using T = typename io_elem<IO>::T;
    constexpr int V = 16 / (int)sizeof(T);
    const int64_t nvec = (a.N + V - 1) / V, R = a.B * a.H;
    const int tpr = threads_per_row(nvec);
    const int64_t rows = (R + kThreads / tpr - 1) / (kThreads / tpr);
    int64_t gy = (nvec + tpr - 1) / tpr;
    gy = gy < 1 ? 1 : (gy > 4096 ? 4096 : gy);
    return launch(k_short_conv<IO>, dim3((unsigned)rows, (unsigned)gy), dim3(kThreads), 0, s, (const T *)a.x,
                  (const T *)a.x_in, a.w, a.bias, a.lengths, (T *)y, (T *)x_out, a.B, a.H, a.N, a.W, a.silu, tpr);
}

hipError_t launch_short_conv(const ShortConvArgs &a, void *y, void *x_out, int io, hipStream_t s) {
    switch (io) {
        case IO_F32: return short_conv_io<IO_F32>(a, y, x_out, s);
        case IO_F16: return short_conv_io<IO_F16>(a, y, x_out, s);
        case IO_BF16: return short_conv_io<IO_BF16>(a, y, x_out, s);
        default: return hipErrorInvalidValue;
    }
}

template <int IO>
static hipError_t short_conv_bwd_io(const ShortConvArgs &a, const void *dy, const void *dx_out, void *dx, float *dw,
                                    float *dbias, void *dx_in, float *part, hipStream_t s) {
    using T = typename io_elem<IO>::T;
    int64_t pieces;
    int tpr;
    const int K = bwd_splits(a.B, a.H, a.N, &pieces, &tpr, 16 / (int)sizeof(T));
    hipError_t e = launch(k_short_conv_bwd<IO>, dim3((unsigned)a.H, (unsigned)K), dim3(kThreads), 0, s,
                          (const T *)a.x, (const T *)a.x_in, a.w, a.bias, a.lengths, (const T *)dy, (const T *)dx_out,
                          (T *)dx, (T *)dx_in, part, a.B, a.H, a.N, a.W, a.silu, tpr, pieces);
    if (e != hipSuccess) return e;
    return launch(k_short_conv_sums, dim3((unsigned)((a.H * (kTaps + 1) + 255) / 256)), dim3(256), 0, s, part, dw,
                  dbias, a.H, a.W, K);
}

hipError_t launch_short_conv_bwd(const ShortConvArgs &a, const void *dy, const void *dx_out, void *dx, float *dw,
                                 float *dbias, void *dx_in, int io, void *ws, hipStream_t s) {
    float *p = (float *)ws;
    switch (io) {
        case IO_F32: return short_conv_bwd_io<IO_F32>(a, dy, dx_out, dx, dw, dbias, dx_in, p, s);
        case IO_F16: return short_conv_bwd_io<IO_F16>(a, dy, dx_out, dx, dw, dbias, dx_in, p, s);
        case IO_BF16: return short_conv_bwd_io<IO_BF16>(a, dy, dx_out, dx, dw, dbias, dx_in, p, s);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_short_conv_step(const void *x, const float *w, const float *bias, const int32_t *slots,
                                  const void *st_in, void *st_out, void *y, int64_t B, int64_t H, int64_t P, int W,
                                  int silu, int io, hipStream_t s) {
    const dim3 grid((unsigned)((H + kThreads - 1) / kThreads), (unsigned)B);
    switch (io) {
        case IO_F32:
            return launch(k_short_conv_step<IO_F32>, grid, dim3(kThreads), 0, s, (const float *)x, w, bias, slots,
                          (const float *)st_in, (float *)st_out, (float *)y, B, H, P, W, silu);
        case IO_F16:
            return launch(k_short_conv_step<IO_F16>, grid, dim3(kThreads), 0, s, (const _Float16 *)x, w, bias, slots,
                          (const _Float16 *)st_in, (_Float16 *)st_out, (_Float16 *)y, B, H, P, W, silu);
        case IO_BF16:
            return launch(k_short_conv_step<IO_BF16>, grid, dim3(kThreads), 0, s, (const uint16_t *)x, w, bias, slots,
                          (const uint16_t *)st_in, (uint16_t *)st_out, (uint16_t *)y, B, H, P, W, silu);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace h3c
