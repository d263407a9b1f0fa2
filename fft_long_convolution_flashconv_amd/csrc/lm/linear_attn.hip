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

// ---------------------------------------------------------------- chunks on the matrix cores

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef int i2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) s4 lds_s4;

// What a type's products need.  An operand fragment is 8 values of k per lane,
// k = 8 (lane >> 4) + j of 32, of the row (column) lane & 15.
template <int IO>
struct Mx {  // 16-bit elements
    static constexpr int C = 64;                       // steps of a chunk
    static constexpr int UPD = IO == IO_BF16 ? 3 : 2;  // pieces of a weighted value: 24 or 22 bits
    static constexpr bool SCALE = IO == IO_F16;        // pieces are of values brought near 2^14
    struct Frag {
        u4 v;
    };
    __device__ __forceinline__ static f4 mul(const Frag &a, const Frag &b, f4 c) {
        if constexpr (IO == IO_F16)
            return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a.v), __builtin_bit_cast(half8, b.v), c, 0, 0, 0);
        else
            return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.v), __builtin_bit_cast(bf16x8, b.v), c, 0, 0, 0);
    }
    __device__ __forceinline__ static float get(const Frag &f, int j) {
        const uint32_t w = f.v[j >> 1];
        if constexpr (IO == IO_F16) return (float)__builtin_bit_cast(half2v, w)[j & 1];
        else return __uint_as_float((j & 1) ? w & 0xffff0000u : w << 16);
    }
    // The next piece of x: x rounded to the type, which x is left without.
    __device__ __forceinline__ static Frag piece(float (&x)[8], bool last) {
        Frag f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f2 p = {x[2 * j], x[2 * j + 1]};
            if constexpr (IO == IO_F16) f.v[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, half2v));
            else f.v[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
        }
        if (!last) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] -= get(f, j);
        }
        return f;
    }
};
template <>
struct Mx<IO_F32> {
    static constexpr int C = 32, UPD = 1;
    static constexpr bool SCALE = false;
    struct Frag {
        float v[8];
    };
    __device__ __forceinline__ static f4 mul(const Frag &a, const Frag &b, f4 c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[j], b.v[j], c, 0, 0, 0);
        return c;
    }
    __device__ __forceinline__ static float get(const Frag &f, int j) { return f.v[j]; }
    __device__ __forceinline__ static Frag piece(float (&x)[8], bool) {
        Frag f;
#pragma unroll
        for (int j = 0; j < 8; ++j) f.v[j] = x[j];
        return f;
    }
};

// A tile of steps in LDS: rows of COLS elements in units of 16 bytes, which a row's
// number permutes so that neither kind of fragment meets a bank more often than it must.
template <int IO, int COLS>
struct Lds {
    using T = typename io_elem<IO>::T;
    static constexpr int E = 16 / (int)sizeof(T), CH = COLS / E, ROWS = Mx<IO>::C, kBytes = ROWS * COLS * (int)sizeof(T);
    using Frag = typename Mx<IO>::Frag;
    __device__ __forceinline__ static int at(int row, int chunk) {
        const int turn = CH >= 16 ? row & 15 : (row / (16 / CH)) & (CH - 1);
        return (row * CH + (chunk ^ turn)) * 16;
    }
    // the row `row` + lane & 15, its 32 elements from k on, 8 of them per lane
    __device__ __forceinline__ static Frag along(const char *p, int row, int k) {
        const int i = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
        Frag f;
        if constexpr (IO != IO_F32) {
            f.v = *(const u4 *)(p + at(row + i, k / E + g));
        } else {
            const f4 a = *(const f4 *)(p + at(row + i, k / E + 2 * g)), b = *(const f4 *)(p + at(row + i, k / E + 2 * g + 1));
#pragma unroll
            for (int j = 0; j < 4; ++j) f.v[j] = a[j], f.v[4 + j] = b[j];
        }
        return f;
    }
    // one column per lane, the steps 4 g + j and 16 + 4 g + j from `row` on.  spread: columns
    // col + 8 (i >> 2) + (i & 3), the order in which the state's rows lie; else col + i.
    template <bool SPREAD>
    __device__ __forceinline__ static Frag across(const char *p, int row, int col) {
        const int i = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
        Frag f;
        if constexpr (IO != IO_F32) {
            const int c = SPREAD ? col + 8 * (i & 3) : col + 4 * (i & 3);
            i2 h[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int r = row + 16 * q + 4 * g + (i >> 2);
                h[q] = __builtin_bit_cast(i2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(p + at(r, c / E) + (c & 4) * 2)));
            }
            f.v = u4{(uint32_t)h[0].x, (uint32_t)h[0].y, (uint32_t)h[1].x, (uint32_t)h[1].y};
        } else {
            const int c = SPREAD ? col + 8 * (i >> 2) + (i & 3) : col + i;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f.v[j] = *(const float *)(p + at(row + 16 * (j >> 2) + 4 * g + (j & 3), c / E) + (c & 3) * 4);
        }
        return f;
    }
};

__device__ __forceinline__ float lanes_max(float v, int from) {
    for (int d = from; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}
// The power of two that brings a largest magnitude m to 2^13 .. 2^14, as an exponent.
__device__ __forceinline__ int near_2_14(float m) {
    const int e = 14 - __builtin_amdgcn_frexp_expf(m);
    return e < -100 ? -100 : (e > 100 ? 100 : e);
}
__device__ __forceinline__ float pow2(int e) { return __builtin_amdgcn_ldexpf(1.f, e); }
// 2^x of a 64-bit exponent, to 32 bits
__device__ __forceinline__ float exp2_of(double x) {
    const float d = (float)x;
    return __builtin_amdgcn_exp2f(d) * fmaf((float)(x - (double)d), kLn2, 1.f);
}

// Where the segments of the rows meet.
struct Segs {
    int64_t len, n;      // steps of one, number
    float *state;        // [role][seg][B*H][K*M]: what a segment adds, then the state that enters it
    float *factor;       // [role][seg][B*H][2]: the decay over it, in two parts
    int64_t plane;       // K*M
};

template <int IO, int KP, int NV, bool OUT>
__global__ __launch_bounds__(256) void k_lin_chunk(Roles roles, Shape s, Segs sg, int tiles) {
    using T = typename io_elem<IO>::T;
    using X = Mx<IO>;
    using Frag = typename X::Frag;
    constexpr int C = X::C, MB = 4 * NV * 16, KS = KP / 32, NT = C / 16, NU = C / 32;
    using LK = Lds<IO, KP>;
    using LM = Lds<IO, MB>;
    constexpr int E = LK::E;
    constexpr int NA = C * LK::CH / 256, NC = C * LM::CH / 256;  // units of 16 bytes per thread
    static_assert(C * LK::CH % 256 == 0 && C * LM::CH % 256 == 0, "whole units");
    __shared__ __attribute__((aligned(16))) char la[OUT ? LK::kBytes : 16], lb[LK::kBytes], lc[LM::kBytes];
    __shared__ __attribute__((aligned(16))) float dec[4 * C + 4];  // [hi, lo, into, upd][C], then the chunk's factor in two parts
    __shared__ float dots[OUT ? 4 * C : 4];                        // [wave][C]
    const Role &r = roles.r[blockIdx.y];
    const int K = r.a.dim, M = r.c.dim;
    int64_t id = block_id();
    const int tile = (int)(id % tiles);
    id /= tiles;
    const int64_t BH = s.B * s.H, bh = id % BH, seg = id / BH;
    if (seg >= (OUT ? sg.n : sg.n - 1) || tile * MB >= M) return;
    const int64_t b = bh / s.H, h = bh - b * s.H, n = row_len(s.lengths, b, s.N);
    const int64_t i_lo = seg * sg.len, i_hi = std::min(n, i_lo + sg.len);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), li = lane & 15, lg = lane >> 4;
    const int col0 = tile * MB + wave * NV * 16;  // the wave's columns
    const bool dot = OUT && r.dot;
    const int np = IO == IO_F32 ? 1 : IO == IO_F16 ? 2 : dot ? 3 : 2;  // pieces of weights and states in the output's products
    const auto time = [&](int64_t i) { return r.reverse ? n - 1 - i : i; };
    const auto base = [&](const Seq &q) { return (const T *)q.p + b * s.N * q.ld + h / q.share * q.dim; };
    const T *pa = OUT ? base(r.a) : nullptr, *pb = base(r.b), *pc = base(r.c);

    f4 st[2 * KS][NV];  // the state: rows 32 p + 8 g + 4 (m & 1) + j of tile m = 2 p, 2 p + 1, column lane & 15
    const int64_t slot = ((int64_t)blockIdx.y * sg.n + seg) * BH + bh;
    const float *enter = OUT ? (seg == 0 && sg.n == 1 ? (r.s0 ? r.s0 + bh * K * M : nullptr) : sg.state + slot * sg.plane) : nullptr;
#pragma unroll
    for (int m = 0; m < 2 * KS; ++m)
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = 16 * (m & ~1) + 8 * lg + 4 * (m & 1) + j, c = col0 + 16 * v + li;
                st[m][v][j] = enter && k < K && c < M ? enter[(int64_t)k * r.rs + (int64_t)c * r.cs] : 0.f;
            }

    // the next chunk's units, on their way
    Pack<T, E> ga[OUT ? NA : 1], gb[NA], gc[NC];
    float gg = 0.f;
    const auto fetch = [&](const T *p, int64_t ld, int64_t i, int c, int dim) {
        Pack<T, E> u;
        const int left = i < i_hi ? dim - c : 0;
        const T *q = p + time(i) * ld + c;
        if (left >= E) {
            u = *(const Pack<T, E> *)q;
        } else {
#pragma unroll
            for (int j = 0; j < E; ++j) u.v[j] = j < left ? q[j] : T(0);
        }
        return u;
    };
    const auto load = [&](int64_t i0) {
#pragma unroll
        for (int q = 0; q < NA; ++q) {
            const int u = q * 256 + tid, row = u / LK::CH, c = u % LK::CH * E;
            if constexpr (OUT) ga[q] = fetch(pa, r.a.ld, i0 + row, c, K);
            gb[q] = fetch(pb, r.b.ld, i0 + row, c, K);
        }
#pragma unroll
        for (int q = 0; q < NC; ++q) {
            const int u = q * 256 + tid, row = u / LM::CH, c = tile * MB + u % LM::CH * E;
            gc[q] = fetch(pc, r.c.ld, i0 + row, c, M);
        }
        if (wave == 0) {
            gg = 0.f;
            if (i0 + lane < i_hi && lane < C) gg = s.per_token ? s.g[(b * s.N + time(i0 + lane)) * s.H + h] : s.g[h];
        }
    };
    double all = 0.0;  // (of wave 0) the segment's decay, as an exponent of two
    const auto keep = [&] {
#pragma unroll
        for (int q = 0; q < NA; ++q) {
            const int u = q * 256 + tid;
            if constexpr (OUT) *(Pack<T, E> *)(la + LK::at(u / LK::CH, u % LK::CH)) = ga[q];
            *(Pack<T, E> *)(lb + LK::at(u / LK::CH, u % LK::CH)) = gb[q];
        }
#pragma unroll
        for (int q = 0; q < NC; ++q) {
            const int u = q * 256 + tid;
            *(Pack<T, E> *)(lc + LM::at(u / LM::CH, u % LM::CH)) = gc[q];
        }
        if (wave == 0) {
            // exponents of two from the chunk's start on, in 64 bits: with the step's own decay where time runs
            // on, without it where it runs back
            const double own = (double)fmaxf(gg, kLeast) * 1.4426950408889634;
            double sum = own;
#pragma unroll
            for (int d = 1; d < C; d <<= 1) {
                const double u = __shfl_up(sum, d);
                if (lane >= d) sum += u;
            }
            const double total = __shfl(sum, C - 1), e = r.reverse ? sum - own : sum;
            all += total;
            if (lane < C) {
                const float hi = (float)e;
                dec[lane] = hi;
                dec[C + lane] = (float)(e - (double)hi);
                dec[2 * C + lane] = exp2_of(e);
                dec[3 * C + lane] = exp2_of(total - e) * r.upd;
            }
            if (lane == 0) {
                const double f = exp2(total);
                dec[4 * C] = (float)f;
                dec[4 * C + 1] = (float)(f - (double)(float)f);
            }
        }
    };

    if (i_lo < i_hi) load(i_lo);
    for (int64_t i0 = i_lo; i0 < i_hi; i0 += C) {
        __syncthreads();  // (the last chunk has been read)
        keep();
        __syncthreads();
        if (i0 + C < i_hi) load(i0 + C);
        Frag cf[NV][NU];
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int u = 0; u < NU; ++u) cf[v][u] = LM::template across<false>(lc, 32 * u, wave * NV * 16 + 16 * v);
        if constexpr (OUT) {
            f4 acc[NT][NV];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int v = 0; v < NV; ++v) acc[t][v] = f4{0.f, 0.f, 0.f, 0.f};
            // the state's part: o^T = X^T a^T, the pieces of X straight from the accumulators
            int se = 0;
            if constexpr (X::SCALE) {
                float m = 0.f;
#pragma unroll
                for (int p = 0; p < 2 * KS; ++p)
#pragma unroll
                    for (int v = 0; v < NV; ++v)
#pragma unroll
                        for (int j = 0; j < 4; ++j) m = fmaxf(m, fabsf(st[p][v][j]));
                se = near_2_14(lanes_max(m, 1));
            }
            const float up_s = pow2(se);
#pragma unroll
            for (int p = 0; p < KS; ++p) {
                Frag x[NV][3];
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    float w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] = X::SCALE ? st[2 * p + (j >> 2)][v][j & 3] * up_s : st[2 * p + (j >> 2)][v][j & 3];
                    x[v][0] = X::piece(w, IO == IO_F32);
                    if constexpr (IO != IO_F32) x[v][1] = X::piece(w, IO == IO_F16);
                    if constexpr (IO == IO_BF16)
                        if (np == 3) x[v][2] = X::piece(w, true);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const Frag a = LK::along(la, 16 * t, 32 * p);
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        acc[t][v] = X::mul(x[v][0], a, acc[t][v]);
                        if constexpr (IO != IO_F32) acc[t][v] = X::mul(x[v][1], a, acc[t][v]);
                        if constexpr (IO == IO_BF16)
                            if (np == 3) acc[t][v] = X::mul(x[v][2], a, acc[t][v]);
                    }
                }
            }
            // the chunk's own part, 16 steps at a time
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                Frag a[KS];
#pragma unroll
                for (int p = 0; p < KS; ++p) a[p] = LK::along(la, 16 * t, 32 * p);
                const float hi = dec[16 * t + li], lo = dec[C + 16 * t + li], into = dec[2 * C + 16 * t + li];
                float w[NT][4], own[4];  // weights of steps 16 q + 4 g + j, and of the step itself
                float m = 0.f;
#pragma unroll
                for (int q = 0; q < NT; ++q) {
                    if (q > t) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) w[q][j] = 0.f;
                        continue;
                    }
                    f4 d = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int p = 0; p < KS; ++p) d = X::mul(LK::along(lb, 16 * q, 32 * p), a[p], d);
                    const f4 h2 = *(const f4 *)(dec + 16 * q + 4 * lg), l2 = *(const f4 *)(dec + C + 16 * q + 4 * lg);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x = d[j] * (r.out * r.upd) * __builtin_amdgcn_exp2f((hi - h2[j]) + (lo - l2[j]));
                        w[q][j] = q < t || 4 * lg + j <= li ? x : 0.f;
                        if constexpr (X::SCALE) m = fmaxf(m, fabsf(w[q][j]));
                        if (q == t) {
                            own[j] = 4 * lg + j == li ? w[q][j] : 0.f;
                            if (dot) w[q][j] -= own[j];
                        }
                    }
                }
                int we = 0;
                if constexpr (X::SCALE) we = near_2_14(lanes_max(m, 16));
                const float up_w = pow2(we), down = pow2(-we), mid = into * r.out * (X::SCALE ? pow2(-se) : 1.f);
                f4 in[NV];
#pragma unroll
                for (int v = 0; v < NV; ++v) in[v] = f4{0.f, 0.f, 0.f, 0.f};
                const auto value = [&](int v, int j) { return fmaf(in[v][j], X::SCALE ? down : 1.f, acc[t][v][j] * mid); };
                const auto add = [&](float (&x)[8], int u) {
                    if constexpr (X::SCALE) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] *= up_w;
                    }
                    Frag f = X::piece(x, IO == IO_F32);
#pragma unroll
                    for (int v = 0; v < NV; ++v) in[v] = X::mul(cf[v][u], f, in[v]);
                    if constexpr (IO != IO_F32) {
                        f = X::piece(x, IO == IO_F16);
#pragma unroll
                        for (int v = 0; v < NV; ++v) in[v] = X::mul(cf[v][u], f, in[v]);
                    }
                    if constexpr (IO == IO_BF16)
                        if (np == 3) {
                            f = X::piece(x, true);
#pragma unroll
                            for (int v = 0; v < NV; ++v) in[v] = X::mul(cf[v][u], f, in[v]);
                        }
                };
#pragma unroll
                for (int u = 0; u <= t / 2; ++u) {
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = w[2 * u + (j >> 2)][j & 3];
                    add(x, u);
                }
                const int64_t i = i0 + 16 * t + li;
                const bool on = i < i_hi;
                const int64_t step = b * s.N + time(on ? i : i_hi - 1);
                if (dot) {
                    float e = 0.f;
                    const T *pe = (const T *)r.e.p + step * r.e.ld + h / r.e.share * r.e.dim;
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        const int c = col0 + 16 * v + 4 * lg;
                        float y[4];
                        ld_row<IO, 4>(pe + c, y, M - c);
#pragma unroll
                        for (int j = 0; j < 4; ++j) e = fmaf(y[j], value(v, j), e);
                    }
                    e += __shfl_xor(e, 16);
                    e += __shfl_xor(e, 32);
                    if (lg == 0) dots[wave * C + 16 * t + li] = e;
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = (j >> 2) == (t & 1) ? own[j & 3] : 0.f;
                    add(x, t / 2);
                }
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int c = col0 + 16 * v + 4 * lg, left = on ? M - c : 0;
                    float y[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] = value(v, j);
                    const int64_t at = (step * s.H + h) * M + c;
                    if (r.wide) st_row<IO_F32, 4>((float *)r.o + at, y, left);
                    else st_row<IO, 4>((T *)r.o + at, y, left);
                }
            }
        }
        // the state: decayed, and the chunk's products added
        const float f1 = dec[4 * C], f2 = dec[4 * C + 1];
        Frag x[NV][NU][X::UPD];
        float down[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float w[NU][8], m = 0.f;
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const f4 d = *(const f4 *)(dec + 3 * C + 32 * u + 16 * q + 4 * lg);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        w[u][4 * q + j] = X::get(cf[v][u], 4 * q + j) * d[j];
                        if constexpr (X::SCALE) m = fmaxf(m, fabsf(w[u][4 * q + j]));
                    }
                }
            down[v] = 1.f;
            if constexpr (X::SCALE) {
                const int e = near_2_14(lanes_max(m, 16));
                down[v] = pow2(-e);
                const float up_v = pow2(e);
#pragma unroll
                for (int u = 0; u < NU; ++u)
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[u][j] *= up_v;
            }
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int q = 0; q < X::UPD; ++q) x[v][u][q] = X::piece(w[u], q == X::UPD - 1);
        }
#pragma unroll
        for (int m = 0; m < 2 * KS; ++m) {
            Frag k[NU];
#pragma unroll
            for (int u = 0; u < NU; ++u) k[u] = LK::template across<true>(lb, 32 * u, 16 * (m & ~1) + 4 * (m & 1));
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                f4 add = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int u = 0; u < NU; ++u)
#pragma unroll
                    for (int q = 0; q < X::UPD; ++q) add = X::mul(k[u], x[v][u][q], add);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float old = st[m][v][j];
                    st[m][v][j] = fmaf(old, f1, fmaf(old, f2, X::SCALE ? add[j] * down[v] : add[j]));
                }
            }
        }
        if (dot) {
            __syncthreads();
            if (tid < C && i0 + tid < i_hi)
                r.dot[(tile * BH + bh) * s.N + time(i0 + tid)] = ((dots[tid] + dots[C + tid]) + dots[2 * C + tid]) + dots[3 * C + tid];
        }
    }
    const auto put = [&](float *to) {
#pragma unroll
        for (int m = 0; m < 2 * KS; ++m)
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = 16 * (m & ~1) + 8 * lg + 4 * (m & 1) + j, c = col0 + 16 * v + li;
                    if (k < K && c < M) to[(int64_t)k * r.rs + (int64_t)c * r.cs] = st[m][v][j];
                }
    };
    if constexpr (OUT) {
        if (r.s1 && seg == sg.n - 1) put(r.s1 + bh * K * M);
        for (int64_t t = std::max(n, i_lo) + wave; t < std::min(s.N, i_lo + sg.len); t += 4)  // past the row's end
            for (int c = tile * MB + lane; c < std::min(M, (tile + 1) * MB); c += 64) {
                const int64_t at = ((b * s.N + t) * s.H + h) * M + c;
                if (r.wide) ((float *)r.o)[at] = 0.f;
                else ((T *)r.o)[at] = T(0);
            }
    } else {
        put(sg.state + slot * sg.plane);
        if (tile == 0 && tid == 0) {
            const double f = exp2(all);
            sg.factor[slot * 2] = (float)f;
            sg.factor[slot * 2 + 1] = (float)(f - (double)(float)f);
        }
    }
}

// The states that enter the segments, from what each segment adds.
__global__ __launch_bounds__(256) void k_lin_enter(Roles roles, Segs sg, int64_t BH) {
    const int64_t i = block_id() * 256 + threadIdx.x;
    if (i >= BH * sg.plane) return;
    const Role &r = roles.r[blockIdx.y];
    const int64_t bh = i / sg.plane, e = i - bh * sg.plane;
    float x = r.s0 ? r.s0[i] : 0.f;
    for (int64_t j = 0; j < sg.n; ++j) {
        const int64_t slot = ((int64_t)blockIdx.y * sg.n + j) * BH + bh;
        float *p = sg.state + slot * sg.plane + e;
        const float add = j + 1 < sg.n ? *p : 0.f;
        *p = x;
        if (j + 1 < sg.n) x = fmaf(x, sg.factor[slot * 2], fmaf(x, sg.factor[slot * 2 + 1], add));
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

int64_t up(int64_t n) { return (n + 255) & ~(int64_t)255; }

// Columns of a block, from the most that a launch's states have and their rows.
int cols_of(int K, int M) { return M > 64 && K <= 128 ? 128 : 64; }
int tiles_of(int M, int cols) { return (M + cols - 1) / cols; }

// Segments of a row of N steps where `blocks` work on each.
constexpr int kChunk = 64;
Segs segs_of(int64_t N, int64_t blocks) {
    const int64_t chunks = std::max<int64_t>(1, (N + kChunk - 1) / kChunk);
    int64_t n = std::min(chunks, std::max<int64_t>(1, 1024 / std::max<int64_t>(1, blocks)));
    const int64_t per = (chunks + n - 1) / n;
    Segs g = {};
    g.len = per * kChunk;
    g.n = (chunks + per - 1) / per;
    return g;
}
int64_t seg_bytes(const Segs &g, int64_t BH, int roles, int64_t plane) {
    return g.n == 1 ? 0 : up(roles * g.n * BH * plane * 4) + up(roles * g.n * BH * 8);
}

template <int IO, int KP, int NV>
hipError_t run_chunks(const Roles &r, int n, const Shape &s, const Segs &g, int tiles, hipStream_t st) {
    const int64_t BH = s.B * s.H;
    if (g.n > 1) {
        hipError_t e = launch(k_lin_chunk<IO, KP, NV, false>, grid_of((g.n - 1) * BH * tiles, (unsigned)n), dim3(256), 0, st, r,
                              s, g, tiles);
        if (e != hipSuccess) return e;
        e = launch(k_lin_enter, grid_of((BH * g.plane + 255) / 256, (unsigned)n), dim3(256), 0, st, r, g, BH);
        if (e != hipSuccess) return e;
    }
    return launch(k_lin_chunk<IO, KP, NV, true>, grid_of(g.n * BH * tiles, (unsigned)n), dim3(256), 0, st, r, s, g, tiles);
}

// K, M: the most rows and columns of the roles' states; ws: seg_bytes.
template <int IO>
hipError_t run_roles(const Roles &r, int n, const Shape &s, int K, int M, Segs g, int64_t plane, void *ws, hipStream_t st) {
    const int cols = cols_of(K, M), tiles = tiles_of(M, cols);
    g.plane = plane;
    g.state = (float *)ws;
    g.factor = (float *)((char *)ws + up(n * g.n * s.B * s.H * plane * 4));
    if (cols == 64) {
        if (K <= 32) return run_chunks<IO, 32, 1>(r, n, s, g, tiles, st);
        if (K <= 64) return run_chunks<IO, 64, 1>(r, n, s, g, tiles, st);
        if (K <= 128) return run_chunks<IO, 128, 1>(r, n, s, g, tiles, st);
        return run_chunks<IO, 256, 1>(r, n, s, g, tiles, st);
    }
    if (K <= 64) return run_chunks<IO, 64, 2>(r, n, s, g, tiles, st);
    return run_chunks<IO, 128, 2>(r, n, s, g, tiles, st);
}
Segs fwd_segs(int64_t B, int64_t N, int64_t H, int64_t dk, int64_t dv) {
    return segs_of(N, B * H * tiles_of((int)dv, cols_of((int)dk, (int)dv)));
}
Segs bwd_segs(int64_t B, int64_t N, int64_t H, int64_t dk, int64_t dv) {
    const int m = (int)std::max(dk, dv);
    return segs_of(N, 3 * B * H * tiles_of(m, cols_of(m, m)));
}

// The parts of the backward pass's workspace, in bytes from its start.
struct BwdSpace {
    int64_t row, col, s_end, sums, dq, dk, segs, all;
};
int dot_tiles(int64_t dk, int64_t dv) {
    const int m = (int)std::max(dk, dv);
    return tiles_of((int)dk, cols_of(m, m));
}
BwdSpace space_of(int64_t B, int64_t N, int64_t H, int64_t G, int64_t dk, int64_t dv) {
    BwdSpace w;
    const int64_t dots = up(dot_tiles(dk, dv) * B * H * N * 4), wide = G < H ? up(B * N * H * dk * 4) : 0;
    int64_t at = 0;
    const auto take = [&](int64_t n) { const int64_t p = at; at += n; return p; };
    w.row = take(dots);
    w.col = take(dots);
    w.s_end = take(up(B * H * dk * dv * 4));
    w.sums = take(up(B * H * 8));
    w.dq = take(wide);
    w.dk = take(wide);
    w.segs = take(seg_bytes(bwd_segs(B, N, H, dk, dv), B * H, 3, dk * dv));
    w.all = at;
    return w;
}

Shape shape_of(const LinAttnArgs &a) { return {a.B, a.N, a.H, a.g, a.lengths, a.per_token}; }

template <int IO>
hipError_t fwd_io(const LinAttnArgs &a, void *y, float *x_out, void *ws, hipStream_t s) {
    const int share = (int)(a.H / a.G);
    const Seq q = {a.q, a.ldq, share, a.dk}, k = {a.k, a.ldk, share, a.dk}, v = {a.v, a.ldv, 1, a.dv};
    Roles r = {};
    r.r[0] = {q, k, v, v, y, nullptr, a.x_in, x_out, a.dv, 1, a.scale, 1.f, 0, 0};
    return run_roles<IO>(r, 1, shape_of(a), a.dk, a.dv, fwd_segs(a.B, a.N, a.H, a.dk, a.dv), (int64_t)a.dk * a.dv, ws, s);
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
    const int m = std::max(a.dk, a.dv);
    hipError_t e = a.B > 0 ? run_roles<IO>(r, 3, s, m, m, bwd_segs(a.B, a.N, a.H, a.dk, a.dv), (int64_t)a.dk * a.dv,
                                           base + w.segs, st)
                           : hipSuccess;
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
        e = launch(k_lin_dg, grid_of(a.B * a.H), dim3(256), 0, st, row, col, dot_tiles(a.dk, a.dv),
                   dot_tiles(a.dk, a.dv), s_end, dx_out,
                   (int64_t)a.dk * a.dv, s, o.dg, sums);
    if (e != hipSuccess || a.per_token) return e;
    return launch(k_lin_dg_heads, dim3((unsigned)((a.H + 255) / 256)), dim3(256), 0, st, sums, o.dg, a.B, a.H);
}

}  // namespace

size_t linear_attn_workspace(int64_t B, int64_t N, int64_t H, int64_t dk, int64_t dv) {
    return (size_t)seg_bytes(fwd_segs(B, N, H, dk, dv), B * H, 1, dk * dv);
}

size_t linear_attn_bwd_workspace(int64_t B, int64_t N, int64_t H, int64_t G, int64_t dk, int64_t dv) {
    return (size_t)space_of(B, N, H, G, dk, dv).all;
}

hipError_t launch_linear_attn(const LinAttnArgs &a, void *y, float *x_out, int io, void *ws, hipStream_t s) {
    switch (io) {
        case IO_F32: return fwd_io<IO_F32>(a, y, x_out, ws, s);
        case IO_F16: return fwd_io<IO_F16>(a, y, x_out, ws, s);
        default: return fwd_io<IO_BF16>(a, y, x_out, ws, s);
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
