// xent.hip -- softmax cross entropy of a linear output layer over a large
// vocabulary, without the logits of the whole vocabulary at once.
//
//   l[t,v] = x[t] . w[v],  lse[t] = log sum_v e^{l[t,v]},  loss[t] = lse[t] - l[t,label[t]]
//   G[t,v] = (e^{l[t,v] - lse[t]} - [v = label[t]]) dloss[t]
//   dx = G w,  dw = G^T x
// Forward: the tiles of x w^T are reduced in registers to one (maximum, sum)
// pair per row and tile; no logit reaches memory.  Backward: piece by piece of
// the vocabulary, the tiles of x w^T are formed again, G of the piece goes to
// the workspace, and two products give dw of the piece and the piece's part
// of dx.  Four products of 2 T D V operations each in all: matrix-core bound.
#include <hip/hip_runtime.h>

#include "lm_device.h"
#include "lm_internal.h"

namespace h3c {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

// One 16-byte fragment per operand and lane: 16x16x32 for 16-bit elements;
// for fp32 four 16x16x4 products whose k indexes are the same permutation on
// both sides.  Lane l: row (column) l & 15, k chunk l >> 4; result rows
// 4 (l >> 4) + i of A, column l & 15 of B.
template <int IO>
__device__ __forceinline__ f4 mfma16(u4 a, u4 b, f4 c) {
    if constexpr (IO == IO_F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
    else if constexpr (IO == IO_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else {
        const f4 x = __builtin_bit_cast(f4, a), y = __builtin_bit_cast(f4, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], y[i], c, 0, 0, 0);
        return c;
    }
}

constexpr int kSlab = 128;  // bytes of k per step and row: operands are padded to whole slabs
constexpr int BM = 128, BN = 128;

// acc[i][j] of this wave's 64 x 64 part of the tile (m0, n0) of A B^T; A has
// M rows of lda bytes, B has N rows of ldb bytes, k bytes each (k a multiple
// of kSlab).  Rows past the end read the last row; their results are dropped
// by the epilogue.
template <int IO>
__device__ __forceinline__ void tile_product(const char *A, int64_t lda, int64_t M, const char *Bt, int64_t ldb,
                                             int64_t N, int64_t k, int64_t m0, int64_t n0, u4 (&sA)[BM * 8],
                                             u4 (&sB)[BN * 8], f4 (&acc)[4][4]) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
    const char *pa[4], *pb[4];
    int at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int id = tid + i * 256, row = id >> 3, c = id & 7;
        int64_t ra = m0 + row, rb = n0 + row;
        ra = ra < M ? ra : M - 1;
        rb = rb < N ? rb : N - 1;
        pa[i] = A + ra * lda + c * 16;
        pb[i] = Bt + rb * ldb + c * 16;
        at[i] = row * 8 + (c ^ (row & 7));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};
    u4 ga[4], gb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        ga[i] = *(const u4 *)pa[i];
        gb[i] = *(const u4 *)pb[i];
    }
    for (int64_t kk = 0; kk < k; kk += kSlab) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sA[at[i]] = ga[i];
            sB[at[i]] = gb[i];
        }
        __syncthreads();
        if (kk + kSlab < k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ga[i] = *(const u4 *)(pa[i] + kk + kSlab);
                gb[i] = *(const u4 *)(pb[i] + kk + kSlab);
            }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            u4 fa[4], fb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int ra = wm + i * 16 + (lane & 15), rb = wn + i * 16 + (lane & 15), c = s * 4 + (lane >> 4);
                fa[i] = sA[ra * 8 + (c ^ (ra & 7))];
                fb[i] = sB[rb * 8 + (c ^ (rb & 7))];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = mfma16<IO>(fa[i], fb[j], acc[i][j]);
        }
    }
}

struct Labels {
    const int64_t *label;
    int64_t ignore, V;
    // the label of token t, or -1 where it carries no loss
    __device__ __forceinline__ int64_t of(int64_t t) const {
        const int64_t l = label[t];
        return (l == ignore || l < 0 || l >= V) ? -1 : l;
    }
};

// Per row of the tile: (maximum, sum of e^{l - maximum}) over the tile's
// columns to part[tile][t], and the label's logit where it is one of them.
template <int IO>
__global__ __launch_bounds__(256) void k_xent_stats(const char *x, int64_t ldx, const char *w, int64_t ldw,
                                                    const Labels lab, float2 *__restrict__ part,
                                                    float *__restrict__ hit, int64_t T, int64_t V, int64_t k) {
    __shared__ u4 sA[BM * 8], sB[BN * 8];
    __shared__ float2 half[BM];
    f4 acc[4][4];
    const int64_t m0 = (int64_t)blockIdx.x * BM, n0 = (int64_t)blockIdx.y * BN;
    tile_product<IO>(x, ldx, T, w, ldw, V, k, m0, n0, sA, sB, acc);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
    float2 st[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t t = m0 + wm + i * 16 + (lane >> 4) * 4 + e;
            const int64_t l = t < T ? lab.of(t) : -1;
            float m = -INFINITY, s = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t v = n0 + wn + j * 16 + (lane & 15);
                if (v < V) m = fmaxf(m, acc[i][j][e]);
                if (v < V && v == l) hit[t] = acc[i][j][e];
            }
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
            const float mm = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t v = n0 + wn + j * 16 + (lane & 15);
                if (v < V) s += __builtin_amdgcn_exp2f((acc[i][j][e] - mm) * kLog2e);
            }
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) s += __shfl_xor(s, d);
            st[i][e] = make_float2(m, s);
        }
    if ((wave & 1) && (lane & 15) == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) half[wm + i * 16 + (lane >> 4) * 4 + e] = st[i][e];
    }
    __syncthreads();
    if (!(wave & 1) && (lane & 15) == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = wm + i * 16 + (lane >> 4) * 4 + e;
                const float2 o = half[row], q = st[i][e];
                const float m = fmaxf(o.x, q.x), mm = m == -INFINITY ? 0.f : m;
                const float s = o.y * __builtin_amdgcn_exp2f((o.x - mm) * kLog2e) +
                                q.y * __builtin_amdgcn_exp2f((q.x - mm) * kLog2e);
                if (m0 + row < T) part[(int64_t)blockIdx.y * T + m0 + row] = make_float2(m, s);
            }
    }
}

// One thread per token joins the tiles' pairs in order.
__global__ __launch_bounds__(256) void k_xent_join(const float2 *__restrict__ part, const float *__restrict__ hit,
                                                   const Labels lab, float *__restrict__ loss,
                                                   float *__restrict__ lse, int64_t T, int64_t tiles) {
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (t >= T) return;
    float m = -INFINITY, s = 0.f;
    for (int64_t i = 0; i < tiles; ++i) {
        const float2 p = part[i * T + t];
        const float n = fmaxf(m, p.x), nn = n == -INFINITY ? 0.f : n;
        s = s * __builtin_amdgcn_exp2f((m - nn) * kLog2e) + p.y * __builtin_amdgcn_exp2f((p.x - nn) * kLog2e);
        m = n;
    }
    const float l = m + logf(s);
    lse[t] = l;
    loss[t] = lab.of(t) >= 0 ? l - hit[t] : 0.f;
}

// fp16 holds G as a share of the largest |dloss|, times 2^15: probabilities
// down to 2^-29 stay normal numbers.  scale[0] is the power of two that G is
// multiplied by, scale[1] its inverse.
__global__ __launch_bounds__(1024) void k_xent_scale(const float *__restrict__ dloss, const Labels lab,
                                                     float *__restrict__ scale, int64_t T) {
    __shared__ float red[16];
    float m = 0.f;
    for (int64_t t = threadIdx.x; t < T; t += 1024)
        if (lab.of(t) >= 0) m = fmaxf(m, fabsf(dloss[t]));
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 16; ++i) m = fmaxf(m, red[i]);
        int e = 0;
        if (m > 0.f && m < INFINITY) frexpf(m, &e);   // m = f 2^e, f < 1
        e = e > 100 ? 100 : (e < -100 ? -100 : e);
        scale[0] = ldexpf(1.f, 15 - e);
        scale[1] = ldexpf(1.f, e - 15);
    }
}

// G of the vocabulary piece [v0, v0 + nv): g[t][v - v0] (row stride ldg
// elements) and its transpose gt[v - v0][t] (row stride ldt >= T, the columns
// past T zero); columns past the piece's end are zero up to ldg.
template <int IO>
__global__ __launch_bounds__(256) void k_xent_grad(const char *x, int64_t ldx, const char *w, int64_t ldw,
                                                   const Labels lab, const float *__restrict__ lse,
                                                   const float *__restrict__ dloss, const float *__restrict__ scale,
                                                   typename io_elem<IO>::T *__restrict__ g, int64_t ldg,
                                                   typename io_elem<IO>::T *__restrict__ gt, int64_t ldt, int64_t T,
                                                   int64_t v0, int64_t nv, int64_t k) {
    using E = typename io_elem<IO>::T;
    __shared__ u4 sA[BM * 8], sB[BN * 8];
    f4 acc[4][4];
    const int64_t m0 = (int64_t)blockIdx.x * BM, n0 = (int64_t)blockIdx.y * BN;
    tile_product<IO>(x, ldx, T, w + v0 * ldw, ldw, nv, k, m0, n0, sA, sB, acc);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
    const float up = IO == IO_F16 ? scale[0] : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t t = m0 + wm + i * 16 + (lane >> 4) * 4;
        float ls[4], dl[4];
        int64_t lb[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            lb[e] = t + e < T ? lab.of(t + e) : -1;
            ls[e] = t + e < T ? lse[t + e] : 0.f;
            dl[e] = lb[e] >= 0 ? dloss[t + e] * up : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t c = n0 + wn + j * 16 + (lane & 15);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float q = __builtin_amdgcn_exp2f((acc[i][j][e] - ls[e]) * kLog2e);
                if (v0 + c == lb[e]) q -= 1.f;
                q = (c < nv && lb[e] >= 0) ? q * dl[e] : 0.f;
                const E o = from_f<IO>(q);
                if (t + e < T && c < ldg) g[(t + e) * ldg + c] = o;
                if (t + e < ldt && c < ldg) gt[c * ldt + t + e] = o;
            }
        }
    }
}

// out = A B^T times scale, added to acc (fp32, row stride D) where there is
// an earlier piece; to acc where a later one follows, else rounded to out.
template <int IO>
__global__ __launch_bounds__(256) void k_xent_product(const char *a, int64_t lda, int64_t M, const char *bt,
                                                      int64_t ldb, int64_t N, int64_t k,
                                                      typename io_elem<IO>::T *__restrict__ out,
                                                      float *__restrict__ accum, int first, int last,
                                                      const float *__restrict__ scale) {
    __shared__ u4 sA[BM * 8], sB[BN * 8];
    f4 acc[4][4];
    const int64_t m0 = (int64_t)blockIdx.x * BM, n0 = (int64_t)blockIdx.y * BN;
    tile_product<IO>(a, lda, M, bt, ldb, N, k, m0, n0, sA, sB, acc);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
    const float down = IO == IO_F16 ? scale[1] : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t m = m0 + wm + i * 16 + (lane >> 4) * 4 + e, n = n0 + wn + j * 16 + (lane & 15);
                if (m >= M || n >= N) continue;
                float v = acc[i][j][e];
                if (!first) v += accum[m * N + n];
                if (last) out[m * N + n] = from_f<IO>(v * down);
                else accum[m * N + n] = v;
            }
}

// dst[r][c] = src[r][c] for c < C, zero up to ldd.
template <class E>
__global__ __launch_bounds__(256) void k_xent_pad(const E *__restrict__ src, E *__restrict__ dst, int64_t R,
                                                  int64_t C, int64_t ldd) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, r = i / ldd, c = i - r * ldd;
    if (r < R) dst[i] = c < C ? src[r * C + c] : (E)0;
}

// dst[c][r] = src[r][c], zero for R <= r < ldd.
template <class E>
__global__ __launch_bounds__(256) void k_xent_transpose(const E *__restrict__ src, E *__restrict__ dst, int64_t R,
                                                        int64_t C, int64_t ldd) {
    __shared__ E tile[64][65];
    const int64_t r0 = (int64_t)blockIdx.x * 64, c0 = (int64_t)blockIdx.y * 64;
    const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
    for (int i = y; i < 64; i += 4)
        tile[i][x] = (r0 + i < R && c0 + x < C) ? src[(r0 + i) * C + c0 + x] : (E)0;
    __syncthreads();
    for (int i = y; i < 64; i += 4)
        if (c0 + i < C && r0 + x < ldd) dst[(c0 + i) * ldd + r0 + x] = tile[x][i];
}

template <class E>
__global__ __launch_bounds__(256) void k_xent_zero(E *__restrict__ p, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = (E)0;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }
int64_t ceil_to(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

struct Plan {
    int64_t kD;            // elements of a padded row of x and w
    int64_t Tp;            // elements of a padded row of x^T and G^T
    int64_t piece, pieces; // vocabulary rows per piece (a multiple of BN)
    char *xp, *wp, *xt, *wt, *g, *gt;
    float *accum, *scale, *hit;
    float2 *part;
    size_t bytes;
};

Plan plan(int64_t T, int64_t D, int64_t V, int io, bool bwd, char *base) {
    Plan p = {};
    const int64_t e = io == IO_F32 ? 4 : 2, slab = kSlab / e;
    p.kD = ceil_to(D, slab);
    p.Tp = ceil_to(T, slab);
    size_t at = 0;
    const auto take = [&](int64_t bytes) {
        char *q = base && bytes ? base + at : nullptr;
        at += align256((size_t)bytes);
        return q;
    };
    p.xp = take(p.kD != D ? T * p.kD * e : 0);
    p.wp = take(p.kD != D ? V * p.kD * e : 0);
    if (!bwd) {
        p.part = (float2 *)take((V + BN - 1) / BN * T * 8);
        p.hit = (float *)take(T * 4);
    } else {
        // G and G^T of a piece: up to 256 MiB each
        int64_t most = ((int64_t)256 << 20) / (p.Tp * e) / BN * BN;
        if (most < BN) most = BN;
        const int64_t n = (V + most - 1) / most;
        p.piece = ceil_to((V + n - 1) / n, BN);
        p.pieces = (V + p.piece - 1) / p.piece;
        p.xt = take(D * p.Tp * e);
        p.wt = take(D * p.piece * e);
        p.g = take(T * p.piece * e);
        p.gt = take(p.piece * p.Tp * e);
        p.accum = (float *)take(p.pieces > 1 ? T * D * 4 : 0);
        p.scale = (float *)take(8);
    }
    p.bytes = at;
    return p;
}

unsigned blocks(int64_t n, int64_t per) { return (unsigned)((n + per - 1) / per); }

// x and w with rows of whole slabs: as they are, or copied.
template <int IO>
hipError_t padded(const void *src, char *dst, int64_t R, int64_t D, int64_t kD, const char **out, hipStream_t s) {
    using E = typename io_elem<IO>::T;
    *out = (const char *)src;
    if (kD == D) return hipSuccess;
    *out = dst;
    return launch(k_xent_pad<E>, dim3(blocks(R * kD, 256)), dim3(256), 0, s, (const E *)src, (E *)dst, R, D, kD);
}

template <int IO>
hipError_t fwd_io(const void *x, const void *w, const Labels &lab, float *loss, float *lse, int64_t T, int64_t D,
                  int64_t V, char *ws, hipStream_t s) {
    const Plan p = plan(T, D, V, IO, false, ws);
    const int64_t ld = p.kD * (int64_t)sizeof(typename io_elem<IO>::T);
    const char *xr, *wr;
    hipError_t e = padded<IO>(x, p.xp, T, D, p.kD, &xr, s);
    if (e == hipSuccess) e = padded<IO>(w, p.wp, V, D, p.kD, &wr, s);
    if (e == hipSuccess)
        e = launch(k_xent_stats<IO>, dim3(blocks(T, BM), blocks(V, BN)), dim3(256), 0, s, xr, ld, wr, ld, lab, p.part,
                   p.hit, T, V, ld);
    if (e != hipSuccess) return e;
    return launch(k_xent_join, dim3(blocks(T, 256)), dim3(256), 0, s, p.part, p.hit, lab, loss, lse, T,
                  (int64_t)blocks(V, BN));
}

template <int IO>
hipError_t bwd_io(const void *x, const void *w, const Labels &lab, const float *lse, const float *dloss, void *dx,
                  void *dw, int64_t T, int64_t D, int64_t V, char *ws, hipStream_t s) {
    using E = typename io_elem<IO>::T;
    const int64_t es = sizeof(E);
    if (T == 0) return launch(k_xent_zero<E>, dim3(blocks(V * D, 256)), dim3(256), 0, s, (E *)dw, V * D);
    const Plan p = plan(T, D, V, IO, true, ws);
    const int64_t ld = p.kD * es;
    const char *xr, *wr;
    hipError_t e = padded<IO>(x, p.xp, T, D, p.kD, &xr, s);
    if (e == hipSuccess) e = padded<IO>(w, p.wp, V, D, p.kD, &wr, s);
    if (e == hipSuccess && IO == IO_F16) e = launch(k_xent_scale, dim3(1), dim3(1024), 0, s, dloss, lab, p.scale, T);
    if (e == hipSuccess)
        e = launch(k_xent_transpose<E>, dim3(blocks(p.Tp, 64), blocks(D, 64)), dim3(256), 0, s, (const E *)x,
                   (E *)p.xt, T, D, p.Tp);
    for (int64_t i = 0; i < p.pieces && e == hipSuccess; ++i) {
        const int64_t v0 = i * p.piece, nv = V - v0 < p.piece ? V - v0 : p.piece, kv = ceil_to(nv, BN);
        const int first = i == 0, last = i + 1 == p.pieces;
        e = launch(k_xent_transpose<E>, dim3(blocks(kv, 64), blocks(D, 64)), dim3(256), 0, s,
                   (const E *)w + v0 * D, (E *)p.wt, nv, D, kv);
        if (e != hipSuccess) break;
        e = launch(k_xent_grad<IO>, dim3(blocks(T, BM), blocks(nv, BN)), dim3(256), 0, s, xr, ld, wr, ld, lab, lse,
                   dloss, p.scale, (E *)p.g, kv, (E *)p.gt, p.Tp, T, v0, nv, ld);
        if (e != hipSuccess) break;
        e = launch(k_xent_product<IO>, dim3(blocks(nv, BM), blocks(D, BN)), dim3(256), 0, s, p.gt, p.Tp * es, nv,
                   p.xt, p.Tp * es, D, p.Tp * es, (E *)dw + v0 * D, (float *)nullptr, 1, 1, p.scale);
        if (e != hipSuccess) break;
        e = launch(k_xent_product<IO>, dim3(blocks(T, BM), blocks(D, BN)), dim3(256), 0, s, p.g, kv * es, T, p.wt,
                   kv * es, D, kv * es, (E *)dx, p.accum, first, last, p.scale);
    }
    return e;
}

}  // namespace

size_t linear_xent_workspace(int64_t T, int64_t D, int64_t V, int io, bool bwd) {
    return plan(T, D, V, io, bwd, nullptr).bytes;
}

hipError_t launch_linear_xent(const void *x, const void *w, const int64_t *labels, int64_t ignore, float *loss,
                              float *lse, int64_t T, int64_t D, int64_t V, int io, void *ws, hipStream_t s) {
    const Labels lab = {labels, ignore, V};
    switch (io) {
        case IO_F32: return fwd_io<IO_F32>(x, w, lab, loss, lse, T, D, V, (char *)ws, s);
        case IO_F16: return fwd_io<IO_F16>(x, w, lab, loss, lse, T, D, V, (char *)ws, s);
        case IO_BF16: return fwd_io<IO_BF16>(x, w, lab, loss, lse, T, D, V, (char *)ws, s);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_linear_xent_bwd(const void *x, const void *w, const int64_t *labels, int64_t ignore,
                                  const float *lse, const float *dloss, void *dx, void *dw, int64_t T, int64_t D,
                                  int64_t V, int io, void *ws, hipStream_t s) {
    const Labels lab = {labels, ignore, V};
    switch (io) {
        case IO_F32: return bwd_io<IO_F32>(x, w, lab, lse, dloss, dx, dw, T, D, V, (char *)ws, s);
        case IO_F16: return bwd_io<IO_F16>(x, w, lab, lse, dloss, dx, dw, T, D, V, (char *)ws, s);
        case IO_BF16: return bwd_io<IO_BF16>(x, w, lab, lse, dloss, dx, dw, T, D, V, (char *)ws, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace h3c
