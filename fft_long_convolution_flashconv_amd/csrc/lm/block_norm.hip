// block_norm.hip -- what stands between two blocks of a network: the norm of a
// block's output f, its gate, the scaled residual sum, and the norm before the
// next block.  Per row of D channels, every part optional but one of the norms
// or the gate:
//   fh = f ra,  ra = (mean over each of `groups` equal parts of f^2 + eps)^-1/2
//   m  = fh w_out silu(z),   r = res + scale m
//   y  = r rb w_in,  rb = (mean r^2 + eps)^-1/2
// Backward, from dr and dy, with e = dy w_in and rh = r rb:
//   t = dr + rb (e - rh mean(e rh)) = dres,   dscale = sum t m,   dm = t scale
//   dz = dm fh w_out silu'(z),  dn = dm silu(z),  dw_out = sum dn fh,
//   df = ra (dn w_out - fh mean(dn w_out fh)),  dw_in = sum dy rh
// Five or eight tensors are touched once for some twenty to sixty operations per
// element: HBM bound.  A row stays in the registers of one to eight waves from the
// loads to the stores, so each tensor is read once; the backward pass forms r
// again from f, z and res instead of reading what the forward pass rounded.
// Squares, sums and all values between are fp32; y is the norm of r before r is
// rounded.
// Forward and backward, bf16: 8192 rows of 2560 take 45 and 126 us (4.7 and 2.7
// TB/s; 545 MB, 106 us together at a copy's rate), of 768 15 and 36 us.  The
// backward kernel waits for the row's sums, four rounds of them one behind
// another (f^2, r^2, e r, dn fh; the second and third could be one), with 20 waves
// a CU at most to cover that.  Rows of few channels leave lanes idle (a wave at
// least per row: 65536 rows of 64 take 32 and 97 us for 8 and 13 at a copy's rate).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "lm_device.h"
#include "lm_internal.h"

namespace h3c {
namespace {

constexpr int V = 8;  // channels of one vector
constexpr int block_rows(int W) { return W == 1 ? 4 : W <= 3 ? 2 : 1; }

typedef uint32_t u4 __attribute__((ext_vector_type(4)));

// A row of n elements at p.  Where rows are whole dwords at whole dwords they are read and written through a buffer
// resource that ends with the row: a lane has one offset for all tensors, and of a vector that passes the row's end the
// dwords past it load zeros and store nothing.  (With an address per tensor and lane the backward kernel waits for
// spilled addresses before every load: 215 us and 99 for 8192 x 2560 in bf16.)  SINGLE, every element is loaded by
// itself (8192 x 1031 in bf16 takes 49 and 166 us, more than 2560 channels read whole).
template <int IO, bool SINGLE>
struct Line {
    using T = typename io_elem<IO>::T;
    T *p;
    __amdgpu_buffer_rsrc_t b;
    int n;
    __device__ __forceinline__ Line(const T *q, int64_t at, int n_) : p(const_cast<T *>(q) + at), n(n_) {
        if constexpr (!SINGLE) b = __builtin_amdgcn_make_buffer_rsrc(p, (short)0, n * (int)sizeof(T), 0x00020000);
    }
};

// A vector as loaded, in whole words: elements one by one would take a register each.
template <int IO, bool SINGLE>
struct Vec {
    using T = typename io_elem<IO>::T;
    static constexpr int WORDS = V * (int)sizeof(T) / 4;
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const Line<IO, SINGLE> &l, uint32_t c) {
        if constexpr (!SINGLE) {
#pragma unroll
            for (int q = 0; q < WORDS / 4; ++q) {
                const u4 r = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(l.b, (int)(c * sizeof(T)) + 16 * q, 0, 0));
#pragma unroll
                for (int i = 0; i < 4; ++i) w[4 * q + i] = r[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) w[i] = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if ((int)c + i >= l.n) continue;
                if constexpr (IO == IO_F32) w[i] = __float_as_uint(l.p[c + i]);
                else w[i >> 1] |= (uint32_t)__builtin_bit_cast(uint16_t, l.p[c + i]) << (16 * (i & 1));
            }
        }
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (IO == IO_F32) return __uint_as_float(w[i]);
        else if constexpr (IO == IO_BF16) return __uint_as_float((i & 1) ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
        else return (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i >> 1] >> (16 * (i & 1))));
    }
    // From here on the words are not known to be the same: what was made of them is made again, not kept.
    __device__ __forceinline__ void forget() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) asm volatile("" : "+v"(w[i]));
    }
};

__device__ __forceinline__ void ld_par(const float *p, uint32_t c, int D, float (&o)[V]) {
    Vec<IO_F32, false> v;
    v.load(Line<IO_F32, false>(p, 0, D), c);
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = v[i];
}
template <int IO, bool SINGLE>
__device__ __forceinline__ void st_vec(const Line<IO, SINGLE> &l, uint32_t c, const float (&o)[V]) {
    if constexpr (!SINGLE) {
        using T = typename io_elem<IO>::T;
        T e[V];
#pragma unroll
        for (int i = 0; i < V; ++i) e[i] = from_f<IO>(o[i]);
#pragma unroll
        for (int q = 0; q < V * (int)sizeof(T) / 16; ++q) {
            u4 r;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (IO == IO_F32) r[i] = __float_as_uint(e[4 * q + i]);
                else r[i] = __builtin_bit_cast(uint16_t, e[2 * i]) | (uint32_t)__builtin_bit_cast(uint16_t, e[2 * i + 1]) << 16;
            }
            __builtin_amdgcn_raw_buffer_store_b128(r, l.b, (int)(c * sizeof(T)) + 16 * q, 0, 0);
        }
    } else {
        st_row<IO, V>(l.p + c, o, l.n - (int)c);
    }
}

template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
// Sum over segments of `n` consecutive lanes, n a power of two up to 64; every lane gets its segment's.  Within 16
// lanes by DPP (neighbours, pairs, halves, halves of eight), which waits for no LDS.
__device__ __forceinline__ float seg_sum(float v, int n) {
    if (n >= 2) v = add_dpp<0xb1>(v);
    if (n >= 4) v = add_dpp<0x4e>(v);
    if (n >= 8) v = add_dpp<0x141>(v);
    if (n >= 16) v = add_dpp<0x140>(v);
    if (n == 32) v += __shfl_xor(v, 16);
    if (n == 64) {
        const int i = __float_as_int(v);
        v = (__int_as_float(__builtin_amdgcn_readlane(i, 0)) + __int_as_float(__builtin_amdgcn_readlane(i, 16))) +
            (__int_as_float(__builtin_amdgcn_readlane(i, 32)) + __int_as_float(__builtin_amdgcn_readlane(i, 48)));
    }
    return v;
}

// x^-1/2; the instruction alone takes numbers below fp32's least normal one, which eps = 0 leaves of small rows, for zeros.
__device__ __forceinline__ float inv_root(float x) {
    float r = __builtin_amdgcn_rsqf(x);
    if (__ballot(x < 0x1p-100f)) r = x < 0x1p-100f ? __builtin_amdgcn_rsqf(x * 0x1p+80f) * 0x1p+40f : r;  // (a choice of the wave)
    return r;
}

// The threads of a row: W waves of a block of one, two or four rows.
template <int W>
struct Row {
    static constexpr int kRows = block_rows(W), kLanes = 64 * W, kThreads = kRows * kLanes;
    int sub, lane;  // the row among the block's, the thread among the row's
    // (the same in a wave: its rows' addresses are scalar)
    __device__ __forceinline__ Row() : sub(__builtin_amdgcn_readfirstlane((int)threadIdx.x / kLanes)), lane((int)threadIdx.x % kLanes) {}
    // The sum of v over the row's threads.  lds: a float per wave, free since the last barrier but one.
    __device__ __forceinline__ float sum(float v, float *lds) const {
        v = seg_sum(v, 64);
        if constexpr (W > 1) {
            if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
            __syncthreads();
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) s += lds[sub * W + i];
            v = s;
        }
        return v;
    }
};

// How the channels fall into groups.
struct Groups {
    int n, size;      // groups, channels of one
    int vecs, lanes;  // vectors of one if it is whole ones, at most 64 (else 0); the same if they are a power of two
    float inv;        // 1 / size
};

// Per vector the sums of its elements' values over their group.  A group of a
// power of two of vectors lies in the lanes of one wave; one of other whole
// vectors, up to 64, goes through LDS, a sum per vector (8192 x 2560 in 32 heads,
// bf16: 41 us and 149, by elements 97 and 470); any other (ODD) element by element
// (4 heads of 640: 92 and 449; 128 of 20: 140 and 569).
template <int W, int NV, bool ODD, class F>
__device__ __forceinline__ void group_sums(const Row<W> &row, const Groups &g, int D, F value, float (&out)[NV][ODD ? V : 1],
                                           float *small, float *wide) {
    if (!ODD || g.n == 1) {
        float v[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            v[j] = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) v[j] += value(j, i);
        }
        if (g.n == 1) {
            float all = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j) all += v[j];
            all = row.sum(all, small);
#pragma unroll
            for (int j = 0; j < NV; ++j) v[j] = all;
        } else if (g.lanes) {
#pragma unroll
            for (int j = 0; j < NV; ++j) v[j] = seg_sum(v[j], g.lanes);
        } else {
            float *mine = wide + row.sub * (D / V);
            __syncthreads();  // (what the last sums read of it has been read)
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int i = j * Row<W>::kLanes + row.lane;
                if (i * V < D) mine[i] = v[j];
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int i = j * Row<W>::kLanes + row.lane, first = i / g.vecs * g.vecs;
                v[j] = 0.f;
                if (i * V < D)
#pragma unroll 1  // (rows that do not come here pay for its code: 8192 x 2560 both ways 171 us without, 174, unrolled 176)
                    for (int k = 0; k < g.vecs; ++k) v[j] += mine[first + k];
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < (ODD ? V : 1); ++i) out[j][i] = v[j];
    } else if constexpr (ODD) {
        float *mine = wide + (int64_t)row.sub * (D + g.n), *tot = mine + D;
        __syncthreads();  // (what the last sums read of it has been read)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * Row<W>::kLanes + row.lane) * V;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (c + i < D) mine[c + i] = value(j, i);
        }
        __syncthreads();
        for (int q = row.lane >> 6; q < g.n; q += W) {
            float s = 0.f;
            for (int c = (int)threadIdx.x & 63; c < g.size; c += 64) s += mine[q * g.size + c];
            s = seg_sum(s, 64);
            if ((threadIdx.x & 63) == 0) tot[q] = s;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * Row<W>::kLanes + row.lane) * V;
#pragma unroll
            for (int i = 0; i < V; ++i) out[j][i] = c + i < D ? tot[(c + i) / g.size] : 0.f;
        }
    }
}

template <int IO>
struct Ptr {
    using T = typename io_elem<IO>::T;
    const T *f, *res, *z, *dr, *dy;
    const float *w_out, *scale, *w_in;
    T *r, *y, *df, *dres, *dz;
    float *part;  // [blocks][3][D]: sums of dw_out, dscale, dw_in
};

template <int IO, int W, int NV, bool ODD, bool SINGLE, bool BWD>
__global__ __launch_bounds__(Row<W>::kThreads, ODD || W * NV >= 16 ? 2 : BWD && IO == IO_F32 ? 3 : 4) void k_block_norm(Ptr<IO> p, int64_t T_, int D, Groups g, float eps) {
    using R = Row<W>;
    extern __shared__ float wide[];
    __shared__ float small[4][R::kRows * W];
    const R row;
    const float invD = 1.f / (float)D;
    const bool out_norm = p.w_out != nullptr, in_norm = p.w_in != nullptr;
    float aw[BWD ? NV : 1][V], as[BWD ? NV : 1][V], ai[BWD ? NV : 1][V];
    if constexpr (BWD) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) aw[j][i] = as[j][i] = ai[j][i] = 0.f;
    }
    for (int64_t t0 = block_id() * R::kRows; t0 < T_; t0 += (int64_t)gridDim.x * gridDim.z * R::kRows) {
        // (the parameters are loaded again for every row, from the caches: kept, they would take the registers of a
        // second wave)
        if constexpr (BWD) asm volatile("" ::: "memory");
        const bool on = t0 + row.sub < T_;
        const int64_t at = (on ? t0 + row.sub : T_ - 1) * D;
        const int n = on ? D : 0;
        Vec<IO, SINGLE> f[NV], res[NV], z[NV], dr[BWD ? NV : 1], dy[BWD ? NV : 1];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t c = (j * R::kLanes + row.lane) * V;
            f[j].load(Line<IO, SINGLE>(p.f, at, n), c);
            if (p.res) res[j].load(Line<IO, SINGLE>(p.res, at, n), c);
            if (p.z) z[j].load(Line<IO, SINGLE>(p.z, at, n), c);
            if constexpr (BWD) {
                if (p.dr) dr[j].load(Line<IO, SINGLE>(p.dr, at, n), c);
                if (p.dy) dy[j].load(Line<IO, SINGLE>(p.dy, at, n), c);
            }
        }
        float ra[NV][ODD ? V : 1];
        const auto ra_of = [&](int j, int i) { return ra[j][ODD ? i : 0]; };
        if (out_norm) {
            group_sums<W, NV, ODD>(row, g, D, [&](int j, int i) { return f[j][i] * f[j][i]; }, ra, small[0], wide);
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < (ODD ? V : 1); ++i) ra[j][i] = inv_root(fmaf(ra[j][i], g.inv, eps));
        }
        // m and r of one vector
        const auto middle = [&](int j, float (&m)[V], float (&r)[V], float (&nf)[V], float (&sg)[V]) {
            const uint32_t c = (j * R::kLanes + row.lane) * V;
#pragma unroll
            for (int i = 0; i < V; ++i) nf[i] = f[j][i];
            if (out_norm) {
                float w[V];
                ld_par(p.w_out, c, D, w);
#pragma unroll
                for (int i = 0; i < V; ++i) nf[i] *= ra_of(j, i) * w[i];
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sg[i] = p.z ? sigmoid(z[j][i]) : 1.f;
                m[i] = p.z ? nf[i] * z[j][i] * sg[i] : nf[i];
                r[i] = m[i];
            }
            if (p.scale) {
                float s[V];
                ld_par(p.scale, c, D, s);
#pragma unroll
                for (int i = 0; i < V; ++i) r[i] *= s[i];
            }
            if (p.res) {
#pragma unroll
                for (int i = 0; i < V; ++i) r[i] += res[j][i];
            }
        };
        float m[V], r[NV][V], nf[V], sg[V], rb = 0.f, c1 = 0.f;
        float ss = 0.f, er = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            middle(j, m, r[j], nf, sg);
            if (in_norm) {
                float w[V];
                if constexpr (BWD)
                    if (p.dy) ld_par(p.w_in, (j * R::kLanes + row.lane) * V, D, w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    ss = fmaf(r[j][i], r[j][i], ss);
                    if constexpr (BWD)
                        if (p.dy) er = fmaf(dy[j][i] * w[i], r[j][i], er);
                }
            }
        }
        if (in_norm) {
            rb = inv_root(fmaf(row.sum(ss, small[1]), invD, eps));
            if constexpr (BWD)
                if (p.dy) c1 = row.sum(er, small[2]) * rb * invD;
        }
        if constexpr (!BWD) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const uint32_t c = (j * R::kLanes + row.lane) * V;
                st_vec<IO, SINGLE>(Line<IO, SINGLE>(p.r, at, n), c, r[j]);
                if (in_norm) {
                    float w[V], o[V];
                    ld_par(p.w_in, c, D, w);
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] = r[j][i] * rb * w[i];
                    st_vec<IO, SINGLE>(Line<IO, SINGLE>(p.y, at, n), c, o);
                }
            }
        } else {
            float dn[NV][V];
            asm volatile("" ::: "memory");
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                f[j].forget();
                if (p.res) res[j].forget();
                if (p.z) z[j].forget();
                if (p.dy) dy[j].forget();
                const uint32_t c = (j * R::kLanes + row.lane) * V;
                float t[V];
                middle(j, m, r[j], nf, sg);
#pragma unroll
                for (int i = 0; i < V; ++i) t[i] = p.dr ? dr[j][i] : 0.f;
                if (in_norm && p.dy) {
                    float w[V];
                    ld_par(p.w_in, c, D, w);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float rh = r[j][i] * rb;
                        t[i] = fmaf(rb, fmaf(-rh, c1, dy[j][i] * w[i]), t[i]);
                        if (on) ai[j][i] = fmaf(dy[j][i], rh, ai[j][i]);
                    }
                }
                if (p.dres) st_vec<IO, SINGLE>(Line<IO, SINGLE>(p.dres, at, n), c, t);
                if (p.scale) {
                    float s[V];
                    ld_par(p.scale, c, D, s);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        if (on) as[j][i] = fmaf(t[i], m[i], as[j][i]);
                        t[i] *= s[i];
                    }
                }
                if (p.z) {
                    float dz[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float zz = z[j][i];
                        dz[i] = t[i] * nf[i] * sg[i] * fmaf(zz, 1.f - sg[i], 1.f);
                        t[i] *= zz * sg[i];
                    }
                    st_vec<IO, SINGLE>(Line<IO, SINGLE>(p.dz, at, n), c, dz);
                }
                if (out_norm) {
                    float w[V];
                    ld_par(p.w_out, c, D, w);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        if (on) aw[j][i] = fmaf(t[i], f[j][i] * ra_of(j, i), aw[j][i]);
                        dn[j][i] = t[i] * w[i];
                    }
                } else {
                    st_vec<IO, SINGLE>(Line<IO, SINGLE>(p.df, at, n), c, t);
                }
            }
            if (out_norm) {
                float c2[NV][ODD ? V : 1];
                group_sums<W, NV, ODD>(row, g, D, [&](int j, int i) { return dn[j][i] * f[j][i] * ra_of(j, i); }, c2, small[3], wide);
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const uint32_t c = (j * R::kLanes + row.lane) * V;
                    float o[V];
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        o[i] = ra_of(j, i) * fmaf(-f[j][i] * ra_of(j, i), c2[j][ODD ? i : 0] * g.inv, dn[j][i]);
                    st_vec<IO, SINGLE>(Line<IO, SINGLE>(p.df, at, n), c, o);
                }
            }
        }
        if constexpr (W > 1) __syncthreads();  // (the small sums are free again)
    }
    if constexpr (BWD) {
        // the block's rows joined in LDS, one of the three sums at a time
        float *out = p.part + block_id() * 3 * D;
        const auto join = [&](float (&a)[NV][V], bool wanted, float *to) {
            if (!wanted) return;
            for (int s = 0; s < R::kRows; ++s) {
                __syncthreads();
                if (row.sub == s) {
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        const int c = (j * R::kLanes + row.lane) * V;
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            if (c + i < D) wide[c + i] = s == 0 ? a[j][i] : wide[c + i] + a[j][i];
                    }
                }
            }
            __syncthreads();
            for (int c = threadIdx.x; c < D; c += R::kThreads) to[c] = wide[c];
        };
        join(aw, out_norm, out);
        join(as, p.scale != nullptr, out + D);
        join(ai, in_norm, out + 2 * (int64_t)D);
    }
}

// Column sums of the blocks' parts, in order: 64 columns per block, its sixteen
// waves a share of the parts each, eight loads on their way (6 to 8 us for 768 parts of 3 x 2560).
constexpr int kJoin = 1024;
__global__ __launch_bounds__(kJoin) void k_join_parts(const float *__restrict__ part, int parts, int D, float *dw_out,
                                                      float *dscale, float *dw_in) {
    __shared__ float lds[kJoin / 64][64];
    const int lane = threadIdx.x & 63, q = threadIdx.x >> 6, c = (int)blockIdx.x * 64 + lane, which = blockIdx.y;
    float *to = which == 0 ? dw_out : which == 1 ? dscale : dw_in;
    if (!to) return;
    const int per = (parts + kJoin / 64 - 1) / (kJoin / 64), lo = q * per, hi = min(parts, lo + per);
    float s = 0.f;
    if (c < D) {
#pragma unroll 8
        for (int i = lo; i < hi; ++i) s += part[((int64_t)i * 3 + which) * D + c];
    }
    lds[q][lane] = s;
    __syncthreads();
    if (q == 0 && c < D) {
        for (int w = 1; w < kJoin / 64; ++w) s += lds[w][lane];
        to[c] = s;
    }
}

// Blocks whose sums of weights' gradients are joined by k_join_parts: as many as run at once, 16 waves per CU (rows of
// 2560: 122 us with 768 blocks, 144 with 1024).
constexpr int64_t kParts = 1024;
int64_t parts_of(int W) { return 256 * (16 / (block_rows(W) * W)); }

// Waves of a row and vectors per thread.  Forward: as few waves as hold the row in three vectors per thread (eight of
// them four).  Backward a vector's sums, gradients and inputs take some 120 registers, so one vector per thread and as
// many waves as that takes, up to eight (rows of 2560: five waves 122 us, two of three vectors each 140, eight 179).
// Odd groups and rows read by elements have four shapes only.
struct Shape {
    int W, NV;
};
Shape shape_of(int64_t D, bool odd, bool bwd) {
    const int64_t vecs = (D + V - 1) / V;
    if (bwd && !odd) return vecs <= 512 ? Shape{(int)((vecs + 63) / 64), 1} : Shape{8, vecs <= 1024 ? 2 : 4};
    int W = 1;
    while (W < 8 && vecs > 64 * W * 3) W *= odd && W == 1 ? 4 : 2;
    const int nv = (int)((vecs + 64 * W - 1) / (64 * W));
    return {W, W == 8 ? 4 : odd && nv > 1 ? 3 : nv};
}

Groups groups_of(int64_t D, int64_t n) {
    Groups g;
    g.n = (int)n;
    g.size = (int)(D / n);
    g.inv = 1.f / (float)g.size;
    g.vecs = g.size % V == 0 && g.size <= 64 * V ? g.size / V : 0;
    g.lanes = (g.vecs & (g.vecs - 1)) == 0 ? g.vecs : 0;
    return g;
}

// Whether elements are read one by one: rows that are not whole dwords, or a tensor that does not begin at one.
bool is_single(int64_t row_bytes, std::initializer_list<const void *> tensors) {
    if (row_bytes % 4 != 0) return true;
    for (const void *p : tensors)
        if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return true;
    return false;
}

int64_t blocks_of(int64_t T, int W, bool bwd) {
    const int64_t n = (T + block_rows(W) - 1) / block_rows(W);
    return bwd ? std::min(n, parts_of(W)) : n;
}

template <int IO, bool BWD>
hipError_t run(const Ptr<IO> &p, const BlockNormArgs &a, hipStream_t s, int &blocks) {
    const Groups g = groups_of(a.D, a.groups);
    const bool single = is_single(a.D * (int64_t)sizeof(*p.f), {p.f, p.res, p.z, p.dr, p.dy, p.r, p.y, p.df, p.dres, p.dz});
    const bool odd = single || (a.w_out && g.n > 1 && !g.vecs);
    const Shape sh = shape_of(a.D, odd, BWD);
    const int rows = block_rows(sh.W);
    const int64_t n = blocks_of(a.T, sh.W, BWD);
    // (the root of nothing at all is infinite: lanes past a row's end, whose group is empty, would put 0 times that into
    // the row's sums)
    const float eps = std::max(a.eps, 0x1p-149f);
    blocks = (int)std::min<int64_t>(n, kParts);
    const size_t lds = std::max(g.n == 1 ? 0 : odd ? (size_t)rows * (a.D + g.n) * 4 : g.lanes ? 0 : (size_t)rows * (a.D / V) * 4,
                                BWD ? (size_t)a.D * 4 : 0);
    using std::integral_constant;
    const auto go = [&](auto w, auto nv, auto odds, auto singles) {
        constexpr int W = decltype(w)::value, NV = decltype(nv)::value;
        return launch(k_block_norm<IO, W, NV, decltype(odds)::value, decltype(singles)::value, BWD>, grid_of(n), dim3(Row<W>::kThreads), lds, s, p, a.T,
                      (int)a.D, g, eps);
    };
    const auto whole = [&](auto w, auto nv) { return go(w, nv, std::false_type{}, std::false_type{}); };
    constexpr integral_constant<int, 1> one{};
    constexpr integral_constant<int, 2> two{};
    constexpr integral_constant<int, 3> three{};
    constexpr integral_constant<int, 4> four{};
    constexpr integral_constant<int, 8> eight{};
    if (odd) {
        const auto shape = [&](auto singles) {
            constexpr std::true_type yes{};
            if (sh.W == 1 && sh.NV == 1) return go(one, one, yes, singles);
            return sh.W == 1 ? go(one, three, yes, singles) : sh.W == 4 ? go(four, three, yes, singles) : go(eight, four, yes, singles);
        };
        return single ? shape(std::true_type{}) : shape(std::false_type{});
    }
    if constexpr (BWD) {
        switch (sh.W) {
            case 1: return whole(one, one);
            case 2: return whole(two, one);
            case 3: return whole(three, one);
            case 4: return whole(four, one);
            case 5: return whole(integral_constant<int, 5>{}, one);
            case 6: return whole(integral_constant<int, 6>{}, one);
            case 7: return whole(integral_constant<int, 7>{}, one);
            default: return sh.NV == 1 ? whole(eight, one) : sh.NV == 2 ? whole(eight, two) : whole(eight, four);
        }
    } else {
        switch (sh.W) {
            case 1: return sh.NV == 1 ? whole(one, one) : sh.NV == 2 ? whole(one, two) : whole(one, three);
            case 2: return sh.NV == 2 ? whole(two, two) : whole(two, three);
            case 4: return sh.NV == 2 ? whole(four, two) : whole(four, three);
            default: return whole(eight, four);
        }
    }
}

template <int IO>
Ptr<IO> ptr_of(const BlockNormArgs &a) {
    using T = typename io_elem<IO>::T;
    Ptr<IO> p = {};
    p.f = (const T *)a.f, p.res = (const T *)a.res, p.z = (const T *)a.gate;
    p.w_out = a.w_out, p.scale = a.scale, p.w_in = a.w_in;
    return p;
}

template <int IO>
hipError_t fwd_io(const BlockNormArgs &a, void *r, void *y, hipStream_t s) {
    Ptr<IO> p = ptr_of<IO>(a);
    p.r = (typename io_elem<IO>::T *)r, p.y = (typename io_elem<IO>::T *)y;
    int none;
    return run<IO, false>(p, a, s, none);
}

template <int IO>
hipError_t bwd_io(const BlockNormArgs &a, const void *dr, const void *dy, const BlockNormGrads &o, void *ws, hipStream_t s,
                  int &parts) {
    using T = typename io_elem<IO>::T;
    Ptr<IO> p = ptr_of<IO>(a);
    p.dr = (const T *)dr, p.dy = (const T *)dy;
    p.df = (T *)o.df, p.dres = (T *)o.dres, p.dz = (T *)o.dgate;
    p.part = (float *)ws;
    return run<IO, true>(p, a, s, parts);
}

}  // namespace

size_t block_norm_bwd_workspace(int64_t T, int64_t D) { return (size_t)(std::min(T, kParts) * 3 * D * 4); }

hipError_t launch_block_norm(const BlockNormArgs &a, void *r, void *y, int io, hipStream_t s) {
    switch (io) {
        case IO_F32: return fwd_io<IO_F32>(a, r, y, s);
        case IO_F16: return fwd_io<IO_F16>(a, r, y, s);
        default: return fwd_io<IO_BF16>(a, r, y, s);
    }
}

hipError_t launch_block_norm_bwd(const BlockNormArgs &a, const void *dr, const void *dy, const BlockNormGrads &o, int io,
                                 void *ws, hipStream_t s) {
    int parts = 0;
    if (a.T > 0) {
        hipError_t e = io == IO_F32 ? bwd_io<IO_F32>(a, dr, dy, o, ws, s, parts)
                     : io == IO_F16 ? bwd_io<IO_F16>(a, dr, dy, o, ws, s, parts) : bwd_io<IO_BF16>(a, dr, dy, o, ws, s, parts);
        if (e != hipSuccess) return e;
    }
    if (!o.dw_out && !o.dscale && !o.dw_in) return hipSuccess;
    return launch(k_join_parts, dim3((unsigned)((a.D + 63) / 64), 3), dim3(kJoin), 0, s, (const float *)ws, parts, (int)a.D,
                  o.dw_out, o.dscale, o.dw_in);
}

}  // namespace h3c
