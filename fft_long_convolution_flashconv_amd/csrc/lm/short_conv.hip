// short_conv.hip -- short causal depthwise convolution with bias and SiLU.
//
// Per channel h and step t, with W <= 4 taps:
//   p_t = bias[h] + sum_{i<W} w[h,i] x_{t-i},   y_t = silu(p_t) or p_t,
// the tap order of the shift SSM in the H3 mix (w[h,0] on the current input).
// Inputs before the row's start come from x_in (the last W-1 inputs of the
// previous piece, oldest first) or are zero.  About 2W + 10 operations per
// element against 4 to 8 bytes forward, 5W + 20 against 6 to 12 backward: HBM
// bound, with the vector ALUs close behind in 16 bits.  Sums are fp32; y and dx
// are rounded once.
#include <hip/hip_runtime.h>

#include "lm_device.h"
#include "lm_internal.h"

namespace h3c {
namespace {

constexpr int kThreads = 256;
constexpr int kTaps = 4;  // the largest W

// Threads of a block along one row (a power of two that covers it, up to the
// block), the others take rows: short rows leave few threads idle.
__host__ __device__ inline int threads_per_row_log2(int64_t nvec) {
    int t = 0;
    while (1 << t < kThreads && 1 << t < nvec) ++t;
    return t;
}

// This thread's row among the block's.  WAVE: a wave has threads of one row, whose
// addresses, length and taps are then the wave's own (scalar).
template <bool WAVE>
__device__ __forceinline__ int row_of(int tpr_log2) {
    const int sub = (int)threadIdx.x >> tpr_log2;
    return WAVE ? __builtin_amdgcn_readfirstlane(sub) : sub;
}

// x at position p of a row that starts at p = -(W-1), the first W-1 from the
// saved inputs
template <int IO, int W>
__device__ __forceinline__ float at_ext(const typename io_elem<IO>::T *x, const typename io_elem<IO>::T *xin,
                                        int64_t p) {
    if (p >= 0) return to_f<IO>(x[p]);
    return (xin && p >= -(W - 1)) ? to_f<IO>(xin[p + W - 1]) : 0.f;
}

// The W - 1 elements of x before step t0, oldest first; what lies at or past
// `len` is zero.
template <int IO, int W>
__device__ __forceinline__ void before(const typename io_elem<IO>::T *x, const typename io_elem<IO>::T *xin, int64_t t0,
                                       int64_t len, float *v) {
    if constexpr (W > 1) {
        if (t0 > 0) {  // (t0 is a multiple of the vector: at least four elements come before it)
            float near[4];
            ld_row<IO, 4>(x + t0 - 4, near, len - t0 + 4);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) v[j] = near[j + 5 - W];
        } else {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) v[j] = at_ext<IO, W>(x, xin, j - (W - 1));
        }
    }
}

// As before(), of a row of four steps at least without saved inputs whose steps
// up to t0 are valid: one load, whatever t0.
template <int IO, int W>
__device__ __forceinline__ void before_plain(const typename io_elem<IO>::T *x, int64_t t0, float *v) {
    if constexpr (W > 1) {
        float near[4];
        ld_row<IO, 4>(x + (t0 > 0 ? t0 - 4 : 0), near);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) v[j] = t0 > 0 ? near[j + 5 - W] : 0.f;
    }
}

// A count of steps as a small int: at most V matter.
__device__ __forceinline__ int few(int64_t n) { return (int)(n < 0 ? 0 : (n > 64 ? 64 : n)); }

// A thread takes one 16-byte vector of a row, and the W - 1 elements before it
// from the caches (one more load; two vectors per thread were a sixth slower).
// 4 x 2560 x 2048, 4 taps: bf16 16.7 us, 5.0 TB/s (a copy reaches 5.1), fp32 25.4
// (168 MB, which the caches hold in part); with a wave's addresses and masks on
// the vector ALUs, 29 instructions per element, these bounded it: 21.6 us in bf16.
// 8 x 768 x 1024 fp16: 8.5 us.
template <int IO, int W, bool WAVE>
__global__ __launch_bounds__(kThreads) void k_short_conv(const typename io_elem<IO>::T *__restrict__ x,
                                                         const typename io_elem<IO>::T *__restrict__ x_in,
                                                         const float *__restrict__ w, const float *__restrict__ bias,
                                                         const int32_t *__restrict__ lengths,
                                                         typename io_elem<IO>::T *__restrict__ y,
                                                         typename io_elem<IO>::T *__restrict__ x_out, int64_t B,
                                                         int64_t H, int64_t N, int silu, int tpr_log2) {
    using T = typename io_elem<IO>::T;
    constexpr int V = 16 / (int)sizeof(T);
    const int tpr = 1 << tpr_log2, tl = (int)threadIdx.x & (tpr - 1);
    const uint32_t row = (uint32_t)block_id() * (uint32_t)(kThreads >> tpr_log2) + row_of<WAVE>(tpr_log2);
    if (row >= (uint32_t)(B * H)) return;
    const uint32_t b = row / (uint32_t)H, h = row - b * (uint32_t)H;
    const int64_t r = row, len = row_len(lengths, b, N);
    const T *xr = x + r * N, *xi = x_in ? x_in + r * (W - 1) : nullptr;
    float tap[W];
#pragma unroll
    for (int k = 0; k < W; ++k) tap[k] = w[(int64_t)h * W + k];
    const float bs = bias ? bias[h] : 0.f;
    if (x_out && blockIdx.y == 0)
        for (int j = tl; j < W - 1; j += tpr) x_out[r * (W - 1) + j] = from_f<IO>(at_ext<IO, W>(xr, xi, len - (W - 1) + j));
    for (int64_t t0 = ((int64_t)blockIdx.y * tpr + tl) * V; t0 < N; t0 += (int64_t)gridDim.y * tpr * V) {
        float v[V + W - 1], cur[V], o[V];
        const auto sums = [&] {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i + W - 1] = cur[i];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float p = bs;
#pragma unroll
                for (int k = 0; k < W; ++k) p = fmaf(tap[k], v[i + W - 1 - k], p);
                o[i] = silu ? p * sigmoid(p) : p;
            }
        };
        if (__all(t0 + V <= len && (t0 > 0 || !xi))) {  // (of the wave: its loads and stores need no choice)
            ld_row<IO, V>(xr + t0, cur);
            before_plain<IO, W>(xr, t0, v);
            sums();
            st_row<IO, V>(y + r * N + t0, o, V);
        } else {
            ld_row<IO, V>(xr + t0, cur, len - t0);
            before<IO, W>(xr, xi, t0, len, v);
            sums();
            const int valid = few(len - t0);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i >= valid) o[i] = 0.f;
            st_row<IO, V>(y + r * N + t0, o, N - t0);
        }
    }
}

// d p_t = dy_t silu'(p_t) at one step
__device__ __forceinline__ float act_bwd(float p, float dy, int silu) {
    if (!silu) return dy;
    const float s = sigmoid(p);
    return dy * fmaf(p * s, 1.f - s, s);
}

// Backward pass of one channel: block (h, k) takes the tasks k, k + K, ... of
// the channel's B rows cut into pieces, so the sums over batch and time stay
// in one block's registers and are joined in a fixed order:
//   dx_s = sum_i w_i dp_{s+i},  dw_i = sum_{b,t} dp_t x_{t-i},  dbias = sum dp.
// A thread forms dp of its own V steps and of the W - 1 after them, which costs
// 3 of 11 (V = 8) or of 19 (16) activations at 4 taps and saves an exchange
// between threads.  4 x 2560 x 2048, 4 taps: bf16 24.8 us, 5.1 TB/s, fp32 41.1 us
// (252 MB), from inputs that the caches hold in part; 27.3 in bf16 after a forward
// pass.
template <int IO, int W, bool WAVE, int V>
__global__ __launch_bounds__(kThreads) void k_short_conv_bwd(
    const typename io_elem<IO>::T *__restrict__ x, const typename io_elem<IO>::T *__restrict__ x_in,
    const float *__restrict__ w, const float *__restrict__ bias, const int32_t *__restrict__ lengths,
    const typename io_elem<IO>::T *__restrict__ dy, const typename io_elem<IO>::T *__restrict__ dx_out,
    typename io_elem<IO>::T *__restrict__ dx, typename io_elem<IO>::T *__restrict__ dx_in, float *__restrict__ part,
    float *__restrict__ dw, float *__restrict__ dbias, int64_t B, int64_t H, int64_t N, int silu, int tpr_log2,
    int64_t pieces) {
    using T = typename io_elem<IO>::T;
    constexpr int E = V + W - 1;
    const int64_t h = block_id();
    if (h >= H) return;
    const int tpr = 1 << tpr_log2, rpb = kThreads >> tpr_log2, tl = (int)threadIdx.x & (tpr - 1);
    const int sub = row_of<WAVE>(tpr_log2);
    float tap[W], sw[W], sb = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
        tap[k] = w[h * W + k];
        sw[k] = 0.f;
    }
    const float bs = bias ? bias[h] : 0.f;
    int64_t bg = 0, piece = blockIdx.y;  // task: rows bg .. bg + rpb - 1, a piece of them
    for (;; piece += gridDim.y) {
        for (; piece >= pieces; piece -= pieces) bg += rpb;
        if (bg >= B) break;
        const int64_t b = bg + sub, t0 = (piece * tpr + tl) * V;
        if (b >= B || (t0 >= N && t0 > 0)) continue;  // (step 0 of an empty row: dx_in alone)
        const int64_t r = b * H + h, len = row_len(lengths, b, N);
        const T *xr = x + r * N, *xi = x_in ? x_in + r * (W - 1) : nullptr, *gr = dy + r * N;
        // v[j]: x at t0 - (W-1) + j, g[j]: dy at t0 + j; the neighbours'
        // elements come from the caches
        float v[E + W - 1], g[E], dp[E], o[V], cur[V], gc[V], near[4], gn[4];
        const int64_t end = t0 + V;
        const auto grads = [&](auto mask) {  // mask(j): whether step t0 + j counts
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[j + W - 1] = cur[j];
                g[j] = gc[j];
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                v[j + V + W - 1] = near[j];
                g[j + V] = gn[j];
            }
#pragma unroll
            for (int j = 0; j < E; ++j) {
                float p = bs;
#pragma unroll
                for (int k = 0; k < W; ++k) p = fmaf(tap[k], v[j + W - 1 - k], p);
                dp[j] = mask(j) ? act_bwd(p, g[j], silu) : 0.f;
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float a = 0.f;
#pragma unroll
                for (int k = 0; k < W; ++k) a = fmaf(tap[k], dp[j + k], a);
                o[j] = a;
                sb += dp[j];
#pragma unroll
                for (int k = 0; k < W; ++k) sw[k] = fmaf(dp[j], v[j + W - 1 - k], sw[k]);
            }
        };
        // the saved last inputs are inputs len-(W-1) .. len-1
        const auto last_inputs = [&](int valid) {
            if (dx_out && valid < V + W) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int q = j - (valid - (W - 1));
                    if (q >= 0 && q < W - 1) o[j] += to_f<IO>(dx_out[r * (W - 1) + q]);
                }
            }
        };
        if (__all((end + 4 <= len || (end == len && len == N)) && (t0 > 0 || !xi))) {
            // (of the wave: its loads and stores need no choice; past the row's end
            // the thread's own first steps stand in, which do not count)
            ld_row<IO, V>(xr + t0, cur);
            ld_row<IO, V>(gr + t0, gc);
            if constexpr (W > 1) {
                ld_row<IO, 4>(xr + (end < len ? end : t0), near);
                ld_row<IO, 4>(gr + (end < len ? end : t0), gn);
            }
            before_plain<IO, W>(xr, t0, v);
            grads([&](int j) { return j < V || end < len; });
            last_inputs(few(len - t0));
            st_row<IO, V>(dx + r * N + t0, o, V);
        } else {
            ld_row<IO, V>(xr + t0, cur, len - t0);
            ld_row<IO, V>(gr + t0, gc, len - t0);
            if constexpr (W > 1) {
                ld_row<IO, 4>(xr + end, near, len - end);
                ld_row<IO, 4>(gr + end, gn, len - end);
            }
            before<IO, W>(xr, xi, t0, len, v);
            const int valid = few(len - t0);
            grads([&](int j) { return j < valid; });
            last_inputs(valid);
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j >= valid) o[j] = 0.f;
            st_row<IO, V>(dx + r * N + t0, o, N - t0);
        }
        if (dx_in && t0 == 0) {
            // saved input j stands at position j - (W-1): it meets the steps
            // 0 .. j through the taps W-1-j .. W-1; with len < W-1 it is also
            // kept as the saved input j - len of the next piece
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                float a = 0.f;
#pragma unroll
                for (int k = 0; k <= j; ++k) a = fmaf(tap[W - 1 - j + k], dp[k], a);
                if (dx_out && j >= len) a += to_f<IO>(dx_out[r * (W - 1) + j - len]);
                dx_in[r * (W - 1) + j] = from_f<IO>(a);
            }
        }
    }
    // joined over the block in a fixed order
    __shared__ float red[kTaps + 1][kThreads / 64];
#pragma unroll
    for (int k = 0; k <= W; ++k) {
        float s = k < W ? sw[k < W ? k : 0] : sb;
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) s += __shfl_xor(s, m);
        if ((threadIdx.x & 63) == 0) red[k][threadIdx.x >> 6] = s;
    }
    __syncthreads();
    if (threadIdx.x <= W) {
        float s = 0.f;
        for (int i = 0; i < kThreads / 64; ++i) s += red[threadIdx.x][i];
        const int k = threadIdx.x;
        if (gridDim.y > 1) part[((int64_t)blockIdx.y * H + h) * (kTaps + 1) + k] = s;
        else if (k < W) dw[h * W + k] = s;
        else if (dbias) dbias[h] = s;
    }
}

__global__ void k_short_conv_sums(const float *__restrict__ part, float *__restrict__ dw, float *__restrict__ dbias,
                                  int64_t H, int W, int K) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t h = i / (kTaps + 1);
    const int k = (int)(i - h * (kTaps + 1));
    if (h >= H || k > W) return;
    float s = 0.f;
#pragma unroll 8
    for (int j = 0; j < K; ++j) s += part[((int64_t)j * H + h) * (kTaps + 1) + k];
    if (k < W) dw[h * W + k] = s;
    else if (dbias) dbias[h] = s;
}

// One token per sequence: the saved inputs of slot slots[b] move on by one.
// Bound by the launch and one chain of loads (slot, saved inputs): 3.3 us for
// 64 x 768 in fp16.
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

int bwd_splits(int64_t B, int64_t H, int64_t N, int64_t *pieces, int *tpr_log2, int V) {
    const int64_t nvec = (N + V - 1) / V;
    *tpr_log2 = threads_per_row_log2(nvec);
    const int tpr = 1 << *tpr_log2, rpb = kThreads / tpr;
    *pieces = nvec > 0 ? (nvec + tpr - 1) / tpr : 1;
    const int64_t tasks = (B + rpb - 1) / rpb * *pieces;
    // about 2048 blocks fill the chip; each join costs one more partial sum, and
    // one more launch (4 x 2560 x 2048, before the scalar addresses: one block per
    // channel 38.0 us, two 39.5 and 4.6 for the sums, four 43.7 and 4.6)
    int64_t k = (2048 + H - 1) / H;
    if (k > tasks) k = tasks;
    if (k > 256) k = 256;
    return (int)(k < 1 ? 1 : k);
}

}  // namespace

size_t short_conv_bwd_workspace(int64_t B, int64_t H, int64_t N, int W) {
    int64_t pieces;
    int tpr_log2, most = 0;
    for (int V = 4; V <= 16; V *= 2) {  // whatever the type
        const int k = bwd_splits(B, H, N, &pieces, &tpr_log2, V);
        if (k > most) most = k;
    }
    return (size_t)most * (size_t)H * (kTaps + 1) * 4;
}

template <int IO, int W>
static hipError_t short_conv_taps(const ShortConvArgs &a, void *y, void *x_out, hipStream_t s) {
    using T = typename io_elem<IO>::T;
    constexpr int V = 16 / (int)sizeof(T);
    const int64_t nvec = (a.N + V - 1) / V, R = a.B * a.H;
    const int lg = threads_per_row_log2(nvec), tpr = 1 << lg;
    const int64_t rows = (R + kThreads / tpr - 1) / (kThreads / tpr);
    int64_t gy = (nvec + tpr - 1) / tpr;
    gy = gy < 1 ? 1 : (gy > 4096 ? 4096 : gy);
    return launch(tpr >= 64 ? k_short_conv<IO, W, true> : k_short_conv<IO, W, false>, grid_of(rows, (unsigned)gy), dim3(kThreads), 0, s, (const T *)a.x,
                  (const T *)a.x_in, a.w, a.bias, a.lengths, (T *)y, (T *)x_out, a.B, a.H, a.N, a.silu, lg);
}

template <int IO>
static hipError_t short_conv_io(const ShortConvArgs &a, void *y, void *x_out, hipStream_t s) {
    switch (a.W) {
        case 1: return short_conv_taps<IO, 1>(a, y, x_out, s);
        case 2: return short_conv_taps<IO, 2>(a, y, x_out, s);
        case 3: return short_conv_taps<IO, 3>(a, y, x_out, s);
        case 4: return short_conv_taps<IO, 4>(a, y, x_out, s);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_short_conv(const ShortConvArgs &a, void *y, void *x_out, int io, hipStream_t s) {
    switch (io) {
        case IO_F32: return short_conv_io<IO_F32>(a, y, x_out, s);
        case IO_F16: return short_conv_io<IO_F16>(a, y, x_out, s);
        case IO_BF16: return short_conv_io<IO_BF16>(a, y, x_out, s);
        default: return hipErrorInvalidValue;
    }
}

// Steps per thread of the backward pass: one vector of 16 bytes, or two where
// there are enough steps for every compute unit (bf16, us, one and two: 4 x 2560
// x 2048 28.2 25.9, 8 x 768 x 1024 15.2 14.1, 3 x 96 x 5000 7.9 11.2, 2 x 768 x
// 100 6.3 7.5).
static int bwd_steps(int64_t B, int64_t H, int64_t N, int bytes) {
    return (B * H * N >= (int64_t)3 << 19 ? 32 : 16) / bytes;
}

template <int IO, int W, int V>
static hipError_t short_conv_bwd_taps(const ShortConvArgs &a, const void *dy, const void *dx_out, void *dx, float *dw,
                                      float *dbias, void *dx_in, float *part, hipStream_t s) {
    using T = typename io_elem<IO>::T;
    int64_t pieces;
    int tpr_log2;
    const int K = bwd_splits(a.B, a.H, a.N, &pieces, &tpr_log2, V);
    const hipError_t e = launch(tpr_log2 >= 6 ? k_short_conv_bwd<IO, W, true, V> : k_short_conv_bwd<IO, W, false, V>, grid_of(a.H, (unsigned)K), dim3(kThreads), 0, s,
                                (const T *)a.x, (const T *)a.x_in, a.w, a.bias, a.lengths, (const T *)dy,
                                (const T *)dx_out, (T *)dx, (T *)dx_in, part, dw, dbias, a.B, a.H, a.N, a.silu, tpr_log2,
                                pieces);
    if (e != hipSuccess || K == 1) return e;
    return launch(k_short_conv_sums, dim3((unsigned)((a.H * (kTaps + 1) + 255) / 256)), dim3(256), 0, s, part, dw,
                  dbias, a.H, W, K);
}

template <int IO, int W>
static hipError_t short_conv_bwd_vec(const ShortConvArgs &a, const void *dy, const void *dx_out, void *dx, float *dw,
                                     float *dbias, void *dx_in, float *part, hipStream_t s) {
    constexpr int bytes = (int)sizeof(typename io_elem<IO>::T), V = 16 / bytes;
    return bwd_steps(a.B, a.H, a.N, bytes) == V
               ? short_conv_bwd_taps<IO, W, V>(a, dy, dx_out, dx, dw, dbias, dx_in, part, s)
               : short_conv_bwd_taps<IO, W, 2 * V>(a, dy, dx_out, dx, dw, dbias, dx_in, part, s);
}

template <int IO>
static hipError_t short_conv_bwd_io(const ShortConvArgs &a, const void *dy, const void *dx_out, void *dx, float *dw,
                                    float *dbias, void *dx_in, float *part, hipStream_t s) {
    switch (a.W) {
        case 1: return short_conv_bwd_vec<IO, 1>(a, dy, dx_out, dx, dw, dbias, dx_in, part, s);
        case 2: return short_conv_bwd_vec<IO, 2>(a, dy, dx_out, dx, dw, dbias, dx_in, part, s);
        case 3: return short_conv_bwd_vec<IO, 3>(a, dy, dx_out, dx, dw, dbias, dx_in, part, s);
        case 4: return short_conv_bwd_vec<IO, 4>(a, dy, dx_out, dx, dw, dbias, dx_in, part, s);
        default: return hipErrorInvalidValue;
    }
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
