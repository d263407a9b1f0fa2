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
// element: HBM bound.  A row stays in the registers of one to four waves from the
// loads to the stores, so each tensor is read once; the backward pass forms r
// again from f, z and res instead of reading what the forward pass rounded.
// Squares, sums and all values between are fp32; y is the norm of r before r is
// rounded.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "lm_device.h"
#include "lm_internal.h"

namespace h3c {
namespace {

constexpr int V = 8;  // channels of one vector
constexpr int block_waves(int W) { return W < 4 ? 4 : W; }

// A vector as loaded (packed, so that a row of several tensors fits the registers).
template <int IO>
struct Vec {
    using T = typename io_elem<IO>::T;
    Pack<T, V> r;
    __device__ __forceinline__ void load(const T *p, int valid) {
        if (valid >= V) {
            r = *reinterpret_cast<const Pack<T, V> *>(p);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) r.v[i] = i < valid ? p[i] : T(0);
        }
    }
    __device__ __forceinline__ float operator[](int i) const { return to_f<IO>(r.v[i]); }
};

__device__ __forceinline__ void ld_par(const float *p, float (&o)[V], int valid) { ld_row<IO_F32, V>(p, o, valid); }

// Sum over segments of `n` consecutive lanes, n a power of two up to 64; every lane gets its segment's.
__device__ __forceinline__ float seg_sum(float v, int n) {
    for (int d = 1; d < n; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

// The threads of a row: W waves of a block of four, or of W if they are more.
template <int W>
struct Row {
    static constexpr int kRows = block_waves(W) / W, kLanes = 64 * W, kThreads = block_waves(W) * 64;
    int sub, lane;  // the row among the block's, the thread among the row's
    __device__ __forceinline__ Row() : sub((int)threadIdx.x / kLanes), lane((int)threadIdx.x % kLanes) {}
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
    int n, size, lanes;  // groups, channels of one, vectors of one if they are a power of two (else 0)
    float inv;           // 1 / size
};

// Per vector the sums of its elements' products a b over their group.  A group of
// a power of two of vectors lies in the lanes of one wave; any other goes through
// LDS, element by element.  GEN: the latter.
template <int W, int NV, bool GEN, class F>
__device__ __forceinline__ void group_sums(const Row<W> &row, const Groups &g, int D, F value, float (&out)[NV][GEN ? V : 1],
                                           float *small, float *wide) {
    if constexpr (!GEN) {
        float s[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            s[j] = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) s[j] += value(j, i);
        }
        if (g.n == 1) {
            float all = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j) all += s[j];
            all = row.sum(all, small);
#pragma unroll
            for (int j = 0; j < NV; ++j) out[j][0] = all;
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j) out[j][0] = seg_sum(s[j], g.lanes);
        }
    } else {
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

template <int IO, int W, int NV, bool GEN, bool BWD>
__global__ __launch_bounds__(Row<W>::kThreads) void k_block_norm(Ptr<IO> p, int64_t T_, int D, Groups g, float eps) {
    using R = Row<W>;
    using E = typename io_elem<IO>::T;
    extern __shared__ float wide[];
    __shared__ float small[4][block_waves(W)];
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
        const bool on = t0 + row.sub < T_;
        const int64_t at = (on ? t0 + row.sub : T_ - 1) * D;
        Vec<IO> f[NV], res[NV], z[NV], dr[BWD ? NV : 1], dy[BWD ? NV : 1];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * R::kLanes + row.lane) * V, n = D - c;
            f[j].load(p.f + at + c, n);
            if (p.res) res[j].load(p.res + at + c, n);
            if (p.z) z[j].load(p.z + at + c, n);
            if constexpr (BWD) {
                if (p.dr) dr[j].load(p.dr + at + c, n);
                if (p.dy) dy[j].load(p.dy + at + c, n);
            }
        }
        float ra[NV][GEN ? V : 1];
        const auto ra_of = [&](int j, int i) { return ra[j][GEN ? i : 0]; };
        if (out_norm) {
            group_sums<W, NV, GEN>(row, g, D, [&](int j, int i) { return f[j][i] * f[j][i]; }, ra, small[0], wide);
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < (GEN ? V : 1); ++i) ra[j][i] = __builtin_amdgcn_rsqf(fmaf(ra[j][i], g.inv, eps));
        }
        // m and r of one vector
        const auto middle = [&](int j, float (&m)[V], float (&r)[V], float (&n)[V], float (&sg)[V]) {
            const int c = (j * R::kLanes + row.lane) * V, left = D - c;
#pragma unroll
            for (int i = 0; i < V; ++i) n[i] = f[j][i];
            if (out_norm) {
                float w[V];
                ld_par(p.w_out + c, w, left);
#pragma unroll
                for (int i = 0; i < V; ++i) n[i] *= ra_of(j, i) * w[i];
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sg[i] = p.z ? sigmoid(z[j][i]) : 1.f;
                m[i] = p.z ? n[i] * z[j][i] * sg[i] : n[i];
                r[i] = m[i];
            }
            if (p.scale) {
                float s[V];
                ld_par(p.scale + c, s, left);
#pragma unroll
                for (int i = 0; i < V; ++i) r[i] *= s[i];
            }
            if (p.res) {
#pragma unroll
                for (int i = 0; i < V; ++i) r[i] += res[j][i];
            }
        };
        float m[V], r[NV][V], n[V], sg[V], rb = 0.f, c1 = 0.f;
        float ss = 0.f, er = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            middle(j, m, r[j], n, sg);
            if (in_norm) {
                float w[V];
                if constexpr (BWD)
                    if (p.dy) ld_par(p.w_in + (j * R::kLanes + row.lane) * V, w, D - (j * R::kLanes + row.lane) * V);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    ss = fmaf(r[j][i], r[j][i], ss);
                    if constexpr (BWD)
                        if (p.dy) er = fmaf(dy[j][i] * w[i], r[j][i], er);
                }
            }
        }
        if (in_norm) {
            rb = __builtin_amdgcn_rsqf(fmaf(row.sum(ss, small[1]), invD, eps));
            if constexpr (BWD)
                if (p.dy) c1 = row.sum(er, small[2]) * rb * invD;
        }
        if constexpr (!BWD) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * R::kLanes + row.lane) * V, left = on ? D - c : 0;
                st_row<IO, V>(p.r + at + c, r[j], left);
                if (in_norm) {
                    float w[V], o[V];
                    ld_par(p.w_in + c, w, D - c);
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] = r[j][i] * rb * w[i];
                    st_row<IO, V>(p.y + at + c, o, left);
                }
            }
        } else {
            float dn[NV][V];
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * R::kLanes + row.lane) * V, left = on ? D - c : 0;
                float t[V];
                middle(j, m, r[j], n, sg);
#pragma unroll
                for (int i = 0; i < V; ++i) t[i] = p.dr ? dr[j][i] : 0.f;
                if (in_norm && p.dy) {
                    float w[V];
                    ld_par(p.w_in + c, w, D - c);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float rh = r[j][i] * rb;
                        t[i] = fmaf(rb, fmaf(-rh, c1, dy[j][i] * w[i]), t[i]);
                        if (on) ai[j][i] = fmaf(dy[j][i], rh, ai[j][i]);
                    }
                }
                if (p.dres) st_row<IO, V>(p.dres + at + c, t, left);
                if (p.scale) {
                    float s[V];
                    ld_par(p.scale + c, s, D - c);
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
                        dz[i] = t[i] * n[i] * sg[i] * fmaf(zz, 1.f - sg[i], 1.f);
                        t[i] *= zz * sg[i];
                    }
                    st_row<IO, V>(p.dz + at + c, dz, left);
                }
                if (out_norm) {
                    float w[V];
                    ld_par(p.w_out + c, w, D - c);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        if (on) aw[j][i] = fmaf(t[i], f[j][i] * ra_of(j, i), aw[j][i]);
                        dn[j][i] = t[i] * w[i];
                    }
                } else {
                    st_row<IO, V>(p.df + at + c, t, left);
                }
            }
            if (out_norm) {
                float c2[NV][GEN ? V : 1];
                group_sums<W, NV, GEN>(row, g, D, [&](int j, int i) { return dn[j][i] * f[j][i] * ra_of(j, i); }, c2, small[3], wide);
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int c = (j * R::kLanes + row.lane) * V, left = on ? D - c : 0;
                    float o[V];
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        o[i] = ra_of(j, i) * fmaf(-f[j][i] * ra_of(j, i), c2[j][GEN ? i : 0] * g.inv, dn[j][i]);
                    st_row<IO, V>(p.df + at + c, o, left);
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

// Column sums of the blocks' parts, in order: 64 columns per block, its four
// waves a quarter of the parts each.
__global__ __launch_bounds__(256) void k_join_parts(const float *__restrict__ part, int parts, int D, float *dw_out,
                                                    float *dscale, float *dw_in) {
    __shared__ float lds[4][64];
    const int lane = threadIdx.x & 63, q = threadIdx.x >> 6, c = (int)blockIdx.x * 64 + lane, which = blockIdx.y;
    float *to = which == 0 ? dw_out : which == 1 ? dscale : dw_in;
    if (!to) return;
    const int per = (parts + 3) / 4, lo = q * per, hi = min(parts, lo + per);
    float s = 0.f;
    if (c < D)
        for (int i = lo; i < hi; ++i) s += part[((int64_t)i * 3 + which) * D + c];
    lds[q][lane] = s;
    __syncthreads();
    if (q == 0 && c < D) to[c] = ((lds[0][lane] + lds[1][lane]) + lds[2][lane]) + lds[3][lane];
}


// Blocks whose sums of weights' gradients are joined by k_join_parts.
constexpr int64_t kParts = 512;

// Waves of a row and vectors per thread: as few waves as hold the row in three
// vectors per thread (eight of them four).  Groups that go through LDS are for odd
// sizes: they have three shapes only.
struct Shape {
    int W, NV;
};
Shape shape_of(int64_t D, bool gen) {
    const int64_t vecs = (D + V - 1) / V;
    int W = 1;
    while (W < 8 && vecs > 64 * W * 3) W *= gen && W == 1 ? 4 : 2;
    const int nv = (int)((vecs + 64 * W - 1) / (64 * W));
    return {W, W == 8 ? 4 : gen ? 3 : nv};
}

Groups groups_of(int64_t D, int64_t n) {
    Groups g;
    g.n = (int)n;
    g.size = (int)(D / n);
    g.inv = 1.f / (float)g.size;
    const int lanes = g.size / V;
    g.lanes = (g.size % V == 0 && (lanes & (lanes - 1)) == 0 && lanes <= 64) ? lanes : 0;
    return g;
}

int64_t blocks_of(int64_t T, int rows, bool bwd) {
    const int64_t n = (T + rows - 1) / rows;
    return bwd ? std::min(n, kParts) : n;
}

template <int IO, bool BWD>
hipError_t run(const Ptr<IO> &p, const BlockNormArgs &a, hipStream_t s) {
    const Groups g = groups_of(a.D, a.groups);
    const bool gen = a.w_out && g.n > 1 && !g.lanes;
    const Shape sh = shape_of(a.D, gen);
    const int rows = block_waves(sh.W) / sh.W;
    const int64_t n = blocks_of(a.T, rows, BWD);
    const size_t lds = std::max(gen ? (size_t)rows * (a.D + g.n) * 4 : 0, BWD ? (size_t)a.D * 4 : 0);
    const auto go = [&](auto w, auto nv, auto ge) {
        constexpr int W = decltype(w)::value, NV = decltype(nv)::value;
        return launch(k_block_norm<IO, W, NV, decltype(ge)::value, BWD>, grid_of(n), dim3(Row<W>::kThreads), lds, s, p, a.T,
                      (int)a.D, g, a.eps);
    };
    using std::integral_constant;
    constexpr integral_constant<int, 1> one{};
    constexpr integral_constant<int, 2> two{};
    constexpr integral_constant<int, 3> three{};
    constexpr integral_constant<int, 4> four{};
    constexpr integral_constant<int, 8> eight{};
    constexpr std::true_type wide{};
    constexpr std::false_type lanes{};
    if (gen) return sh.W == 1 ? go(one, three, wide) : sh.W == 4 ? go(four, three, wide) : go(eight, four, wide);
    switch (sh.W) {
        case 1: return sh.NV == 1 ? go(one, one, lanes) : sh.NV == 2 ? go(one, two, lanes) : go(one, three, lanes);
        case 2: return sh.NV == 2 ? go(two, two, lanes) : go(two, three, lanes);
        case 4: return sh.NV == 2 ? go(four, two, lanes) : go(four, three, lanes);
        default: return go(eight, four, lanes);
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
    return run<IO, false>(p, a, s);
}

template <int IO>
hipError_t bwd_io(const BlockNormArgs &a, const void *dr, const void *dy, const BlockNormGrads &o, void *ws, hipStream_t s) {
    using T = typename io_elem<IO>::T;
    Ptr<IO> p = ptr_of<IO>(a);
    p.dr = (const T *)dr, p.dy = (const T *)dy;
    p.df = (T *)o.df, p.dres = (T *)o.dres, p.dz = (T *)o.dgate;
    p.part = (float *)ws;
    return run<IO, true>(p, a, s);
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
    if (a.T > 0) {
        hipError_t e = io == IO_F32 ? bwd_io<IO_F32>(a, dr, dy, o, ws, s)
                     : io == IO_F16 ? bwd_io<IO_F16>(a, dr, dy, o, ws, s) : bwd_io<IO_BF16>(a, dr, dy, o, ws, s);
        if (e != hipSuccess) return e;
    }
    if (!o.dw_out && !o.dscale && !o.dw_in) return hipSuccess;
    const Groups g = groups_of(a.D, a.groups);
    const int W = shape_of(a.D, a.w_out && g.n > 1 && !g.lanes).W;
    const int parts = (int)blocks_of(a.T, block_waves(W) / W, true);
    return launch(k_join_parts, dim3((unsigned)((a.D + 63) / 64), 3), dim3(256), 0, s, (const float *)ws, parts, (int)a.D,
                  o.dw_out, o.dscale, o.dw_in);
}

}  // namespace h3c
