// selective.hip -- selective state-space scan: prompts, backward pass, tokens.
//
// Per channel h with S real modes and step t (B_t, C_t shared by the channels
// of a group):
//   d_t = softplus(dt_t + dt_bias)  (or dt_t + dt_bias)
//   x_t[j] = exp(d_t A[j]) x_{t-1}[j] + d_t u_t B_t[j]
//   r_t = sum_j C_t[j] x_t[j] + D u_t,   y_t = r_t silu(z_t)  (or r_t)
// All arithmetic is fp32.  Steps at and past a row's length have d_t = 0: the
// state passes them unchanged.
#include <hip/hip_runtime.h>

#include "lm_device.h"
#include "lm_internal.h"

namespace h3c {
namespace {

__device__ __forceinline__ int64_t row_len(const int32_t *lengths, int64_t b, int64_t N) {
    if (!lengths) return N;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : (n > N ? N : n);
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ float lane_of(float v, int l) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}

// DPP moves: lanes without a source read zero; and, for row broadcasts, lanes
// of the rows outside RMASK read `old`.
template <int CTRL>
__device__ __forceinline__ float dpp0(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
template <int CTRL, int RMASK>
__device__ __forceinline__ float dpp_rows(float old, float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, old), __builtin_bit_cast(int, v),
                                                                 CTRL, RMASK, 0xf, false));
}

// The maps x -> P x + Q of consecutive lanes, composed: on return (P, Q) is
// the composition of all lanes before this one (the identity for lane 0).
__device__ __forceinline__ void prefix_maps(float &P, float &Q, int lane) {
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
        const float p = __shfl_up(P, k), q = __shfl_up(Q, k);
        if (lane >= k) {
            Q = fmaf(P, q, Q);
            P *= p;
        }
    }
    P = __shfl_up(P, 1);
    Q = __shfl_up(Q, 1);
    if (lane == 0) { P = 1.f; Q = 0.f; }
}

// The same from the last lane down: the composition of all lanes after this
// one.
__device__ __forceinline__ void suffix_maps(float &P, float &Q, int lane) {
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
        const float p = __shfl_down(P, k), q = __shfl_down(Q, k);
        if (lane + k < 64) {
            Q = fmaf(P, q, Q);
            P *= p;
        }
    }
    P = __shfl_down(P, 1);
    Q = __shfl_down(Q, 1);
    if (lane == 63) { P = 1.f; Q = 0.f; }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

// ------------------------------------------------------------------ prompts

template <class T>
struct SelK {
    const T *u, *dt, *Bm, *C, *z;
    const float *A, *D, *dt_bias, *x_in;
    const int32_t *lengths;
    int64_t B, H, N;
    int S, G, softplus;
};

// Modes whose B and C are in flight.
constexpr int kAhead = 2;
// Steps per lane and piece; modes per channel at most.
constexpr int kIT = 16, kMaxModes = 64;

// n consecutive elements as loaded (words of one or two elements; the words
// keep partly valid pieces from being held element by element).
template <int IO, int n>
struct Raw {
    static constexpr int kWords = n * (int)sizeof(typename io_elem<IO>::T) / 4;
    uint32_t w[kWords];
};

// FULL: all n are valid; else elements from `valid` on are zero.
template <int IO, int n, bool FULL>
__device__ __forceinline__ Raw<IO, n> ld_raw(const typename io_elem<IO>::T *p, int64_t valid) {
    using T = typename io_elem<IO>::T;
    Raw<IO, n> r;
    if (FULL || valid >= n) {
        const Pack<T, n> q = *reinterpret_cast<const Pack<T, n> *>(p);
        __builtin_memcpy(&r, &q, sizeof(r));
    } else {
#pragma unroll
        for (int i = 0; i < Raw<IO, n>::kWords; ++i) {
            if constexpr (sizeof(T) == 4) {
                r.w[i] = i < valid ? __builtin_bit_cast(uint32_t, p[i]) : 0u;
            } else {
                const uint32_t lo = 2 * i < valid ? __builtin_bit_cast(uint16_t, p[2 * i]) : 0u;
                const uint32_t hi = 2 * i + 1 < valid ? __builtin_bit_cast(uint16_t, p[2 * i + 1]) : 0u;
                r.w[i] = lo | hi << 16;
            }
        }
    }
    return r;
}
template <int IO, int n>
__device__ __forceinline__ void unpack(const Raw<IO, n> &r, float (&o)[n]) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
        if constexpr (IO == IO_F32) o[i] = __uint_as_float(r.w[i]);
        else if constexpr (IO == IO_BF16) o[i] = __uint_as_float((i & 1) ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
        else o[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(r.w[i / 2] >> (16 * (i & 1))));
    }
}

// Keeps the values' computation here: the compiler otherwise moves it past
// later work, and its operands stay in registers for all that time.
template <int n>
__device__ __forceinline__ void hold(float (&v)[n]) {
#pragma unroll
    for (int i = 0; i < n; ++i) asm volatile("" : "+v"(v[i]));
}

// P times the P of the lane CTRL names.  In a group of one DPP row (16 lanes)
// the lanes without such a source have reached the group's start, whose
// entering state is folded into Q: their P is not needed any more, and reading
// zero is as good as one (and is one instruction).  Otherwise it reads one.
template <int LPR, int CTRL>
__device__ __forceinline__ float shorten(float P) {
    return P * (LPR == 16 ? dpp0<CTRL>(P) : dpp_rows<CTRL, 0xf>(1.f, P));
}

// Inclusive composition over groups of LPR lanes of maps x -> P x + Q, whose
// first lane has its entering state folded into Q: on return Q is the state
// that leaves each lane.
template <int LPR>
__device__ __forceinline__ void scan_states(float P, float &Q) {
    Q = fmaf(P, dpp0<0x111>(Q), Q);  // row_shr:1
    P = shorten<LPR, 0x111>(P);
    Q = fmaf(P, dpp0<0x112>(Q), Q);
    P = shorten<LPR, 0x112>(P);
    Q = fmaf(P, dpp0<0x114>(Q), Q);
    P = shorten<LPR, 0x114>(P);
    Q = fmaf(P, dpp0<0x118>(Q), Q);
    if constexpr (LPR == 64) {
        P = shorten<LPR, 0x118>(P);
        // the rows of 16 lanes: row 1 after row 0 and row 3 after row 2, then
        // rows 2 and 3 after row 1
        const float q = dpp_rows<0x142, 0xa>(0.f, Q), p = dpp_rows<0x142, 0xa>(1.f, P);  // row_bcast:15
        Q = fmaf(P, q, Q);
        P *= p;
        Q = fmaf(P, dpp_rows<0x143, 0xc>(0.f, Q), Q);  // row_bcast:31
    }
}

// Sums of d over one lane's steps, over the lanes before it in its wave, and
// over the wave.
struct Sums {
    float lane, before, wave;
};

// One mode of one piece: o += C x.  WPR == 1: the state `in` enters the first
// lane, and the state that leaves the row's last lane is kept in *st.
// WPR == 4: the block's four waves hold four pieces in a row of one row; they
// exchange the maps of their pieces through `maps` (one barrier), and every
// wave keeps in its own *st the state before the first and then after the
// last.  B and C arrive as
// loaded; nextB() and nextC() load a later mode's into the same registers once
// they are unpacked.
template <int IO, int LPR, int WPR, class NextB, class NextC>
__device__ __forceinline__ void scan_mode(Raw<IO, kIT> &rB, Raw<IO, kIT> &rC, float A2, float in,
                                          const float (&d)[kIT], const float (&u)[kIT], const Sums &sum,
                                          float (&o)[kIT], float *st, int l, float2 (*maps)[4], float *saved,
                                          const NextB &nextB, const NextC &nextC) {
    constexpr int IT = kIT;
    float a[IT], w[IT], c[IT], P = exp2_(sum.lane * A2), Q = WPR == 1 ? in : 0.f;
    unpack<IO, IT>(rB, w);
    hold(w);
    nextB();
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        a[i] = exp2_(d[i] * A2);
        w[i] *= u[i];
        Q = fmaf(a[i], Q, w[i]);
    }
    scan_states<LPR>(P, Q);
    float x0 = dpp0<LPR == 64 ? 0x138 : 0x111>(Q);  // from the lane before
    if constexpr (WPR == 1) {
        x0 += in;
    } else {
        const int wave = threadIdx.x >> 6;
        if (l == LPR - 1) (*maps)[wave] = make_float2(exp2_(sum.wave * A2), Q);
        __syncthreads();
        float x = *st, enter = x;
#pragma unroll
        for (int i = 0; i < WPR; ++i) {
            const float2 m = (*maps)[i];
            x = fmaf(m.x, x, m.y);
            if (i + 1 == wave) enter = x;
        }
        Q = x;
        x0 = fmaf(exp2_(sum.before * A2), enter, x0);
    }
    float x = x0;
    unpack<IO, IT>(rC, c);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        x = fmaf(a[i], x, w[i]);
        o[i] = fmaf(c[i], x, o[i]);
    }
    hold(o);
    nextC();
    if (l == LPR - 1) *st = Q;
    if (saved) *saved = x0;
}

// The steps of one lane in one piece: the first, how many are valid, and the
// offsets of the first in u, dt, z, y and in mode 0 of B and C.
struct Lane {
    int64_t t0, valid, row, bc;
};

// One piece of LPR*IT steps of each of the wave's rows, from its u and dt as
// loaded; reload() loads the next piece's into the same registers.  FULL:
// every lane's steps are valid.
template <int IO, int LPR, int WPR, bool FULL, class Reload>
__device__ __forceinline__ void scan_piece(const SelK<typename io_elem<IO>::T> &k, const Lane &p, Raw<IO, kIT> &ru,
                                           Raw<IO, kIT> &rd, const float *Ap, float Dh, float bias, float *st, int l,
                                           bool live, float2 (*maps)[4], typename io_elem<IO>::T *y, float *saved,
                                           const Reload &reload) {
    constexpr int IT = kIT, AH = kAhead;
    const int last = k.S - 1;
    Raw<IO, IT> rB[AH], rC[AH];
    const auto loadB = [&](int n) { return ld_raw<IO, IT, FULL>(k.Bm + p.bc + (n < last ? n : last) * k.N, p.valid); };
    const auto loadC = [&](int n) { return ld_raw<IO, IT, FULL>(k.C + p.bc + (n < last ? n : last) * k.N, p.valid); };
#pragma unroll
    for (int j = 0; j < AH; ++j) {
        rB[j] = loadB(j);
        rC[j] = loadC(j);
    }
    float u[IT], d[IT], o[IT];
    Sums sum = {0.f, 0.f, 0.f};
    unpack<IO, IT>(ru, u);
    unpack<IO, IT>(rd, d);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        d[i] += bias;
        if (k.softplus) d[i] = softplus(d[i]);
        if (!FULL && i >= p.valid) d[i] = 0.f;
        o[i] = Dh * u[i];
        u[i] *= d[i];
        sum.lane += d[i];
    }
    if (WPR > 1) {
            float s = sum.lane;
        scan_states<64>(1.f, s);
        sum.before = dpp0<0x138>(s);
        sum.wave = lane_of(s, 63);
    }
    reload();
    // a lane's first step is where a state is saved
    float *sv = saved && live && p.t0 < k.N && p.t0 % kSelChunk == 0 ? saved + p.t0 / kSelChunk * k.S : nullptr;
    float A = Ap[0], in = st[0];
    for (int n0 = 0; n0 < k.S; n0 += AH) {
#pragma unroll
        for (int j = 0; j < AH; ++j) {
            const int n = n0 + j;
            if (AH > 1 && n >= k.S) break;
            const float A2 = A * kLog2e, in0 = l == 0 ? in : 0.f;
            A = Ap[n < last ? n + 1 : last];
            in = st[n < last ? n + 1 : last];
            scan_mode<IO, LPR, WPR>(rB[j], rC[j], A2, in0, d, u, sum, o, st + n, l, maps + (n & 1), sv ? sv + n : nullptr,
                               [&] { rB[j] = loadB(n + AH); }, [&] { rC[j] = loadC(n + AH); });
        }
    }
    if (k.z) {
        float z[IT];
        unpack<IO, IT>(ld_raw<IO, IT, FULL>(k.z + p.row, p.valid), z);
#pragma unroll
        for (int i = 0; i < IT; ++i) o[i] *= z[i] * sigmoid(z[i]);
    }
#pragma unroll
    for (int i = 0; i < IT; ++i)
        if (!FULL && i >= p.valid) o[i] = 0.f;
    if (live) st_row<IO, IT>(y + p.row, o, FULL ? IT : k.N - p.t0);
}

// LPR lanes per row (b, h), 64 / LPR rows per wave; lane l of a row holds
// steps l*IT .. l*IT + IT - 1 of each piece of LPR*IT steps.  Per mode, each
// lane runs its steps from a zero state, the lanes' maps x -> P x + Q are
// composed by a scan over the row's lanes, and each lane runs its steps again
// from the state that enters it: two multiply-adds per (step, mode) instead
// of one, and no state leaves the chip between pieces.
template <int IO, int LPR, int WPR>
__global__ __launch_bounds__(256, 2) void k_sel_scan(const SelK<typename io_elem<IO>::T> k,
                                                     typename io_elem<IO>::T *__restrict__ y,
                                                     float *__restrict__ x_out, float *__restrict__ saved,
                                                     int64_t nchunk) {
    constexpr int IT = kIT, RPW = 64 / LPR, PIECE = WPR * LPR * IT;
    static_assert(WPR == 1 || (WPR == 4 && LPR == 64), "");
    static_assert(kSelChunk % IT == 0, "saved states fall on a lane's first step");
    __shared__ float state[4][RPW][kMaxModes];
    __shared__ float2 maps[2][4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane / LPR, l = lane % LPR;
    const uint32_t R = (uint32_t)(k.B * k.H), H = (uint32_t)k.H;
    const uint32_t r = WPR == 1 ? (blockIdx.x * 4 + wave) * RPW + sub : blockIdx.x;
    if (r - sub >= R) return;  // (the whole wave)
    const bool live = r < R;
    const uint32_t rr = live ? r : R - 1, b = rr / H, h = rr - b * H, g = h / (H / (uint32_t)k.G);
    const int64_t N = k.N, len = row_len(k.lengths, b, N);
    const float Dh = k.D ? k.D[h] : 0.f, bias = k.dt_bias ? k.dt_bias[h] : 0.f;
    const float *Ap = k.A + (int64_t)h * k.S;
    float *st = state[wave][sub];
    for (int n = l; n < k.S; n += LPR) st[n] = k.x_in ? k.x_in[(int64_t)rr * k.S + n] : 0.f;
    __builtin_amdgcn_wave_barrier();
    float *sv = saved ? saved + (int64_t)rr * nchunk * k.S : nullptr;
    const auto piece = [&](int64_t base) {
        const int64_t t0 = base + (WPR == 1 ? 0 : wave * 64 * IT) + l * IT;
        return Lane{t0, len - t0, rr * N + t0, (int64_t)(b * (uint32_t)k.G + g) * k.S * N + t0};
    };
    Raw<IO, IT> ru, rd;
    int64_t base = 0;
    if (__all(len >= PIECE)) {  // the pieces that are full in every row of the wave
        Lane p = piece(0);
        ru = ld_raw<IO, IT, true>(k.u + p.row, 0);
        rd = ld_raw<IO, IT, true>(k.dt + p.row, 0);
        bool more;
        do {
            more = __all(len >= base + 2 * PIECE);
            scan_piece<IO, LPR, WPR, true>(k, p, ru, rd, Ap, Dh, bias, st, l, live, maps, y, sv, [&] {
                const int64_t o = more ? p.row + PIECE : p.row;
                ru = ld_raw<IO, IT, true>(k.u + o, 0);
                rd = ld_raw<IO, IT, true>(k.dt + o, 0);
            });
            __builtin_amdgcn_wave_barrier();
            base += PIECE;
            p = piece(base);
        } while (more);
    }
    for (; base < N; base += PIECE) {
        const Lane p = piece(base);
        ru = ld_raw<IO, IT, false>(k.u + p.row, p.valid);
        rd = ld_raw<IO, IT, false>(k.dt + p.row, p.valid);
        scan_piece<IO, LPR, WPR, false>(k, p, ru, rd, Ap, Dh, bias, st, l, live, maps, y, sv, [] {});
        __builtin_amdgcn_wave_barrier();
    }
    if (x_out && live && (WPR == 1 || wave == 0))
        for (int n = l; n < k.S; n += LPR) x_out[(int64_t)rr * k.S + n] = st[n];
}

// ------------------------------------------------------------------ backward

// With dr = dy silu(z), x the states and e_t = a_t g_t (a_t = exp(d_t A)):
//   g_t = C_t dr_t + e_{t+1}                  gradient of x_t
//   dC_t = sum_h dr_t x_t                     dB_t = sum_h g_t d_t u_t
//   du_t = D dr_t + d_t sum_j g_t B_t         dd_t = sum_j g_t (a_t x_{t-1}) A + u_t sum_j g_t B_t
//   dA = sum_t g_t (a_t x_{t-1}) d_t          dD = sum dr u,  dz = dy r silu'(z)
// One block takes one batch row and a set of channels of one group, and walks
// the row's pieces of kSelChunk steps from the end, with the states at each
// piece's start as the forward pass saved them.  Wave w owns the modes 4w ..
// 4w+3 of a block of 16: their dB and dC over the block's channels stay in
// its registers, so no sum needs an atomic.  Channels go through in fours:
// wave w prepares channel w (softplus, gate) for all waves in LDS, and joins
// the waves' sums over modes for it.
constexpr int kModes = 16, kSetMax = 64, kJT = kSelChunk / 64;

struct SelBwdWs {
    float *dB, *dC;        // [sets][B][G][S][N]
    float *dA;             // [B][H][S]
    float *dDb;            // [B][H][2]
    float *acc;            // [3][B*H*N], more than kModes modes only
    int sets, per;         // sets per group, channels per set
};

template <int IO>
__global__ __launch_bounds__(256) void k_sel_bwd(const SelK<typename io_elem<IO>::T> k,
                                                 const float *__restrict__ saved,
                                                 const typename io_elem<IO>::T *__restrict__ dy,
                                                 const float *__restrict__ dx_out,
                                                 typename io_elem<IO>::T *__restrict__ du,
                                                 typename io_elem<IO>::T *__restrict__ ddt,
                                                 typename io_elem<IO>::T *__restrict__ dz, float *__restrict__ dx_in,
                                                 const SelBwdWs ws, int64_t nchunk, int n0, int last_block) {
    __shared__ float pre[4][3][kSelChunk];
    __shared__ float part[4][4][3][kSelChunk];
    __shared__ float carry[kSetMax][kModes], sumA[kSetMax][kModes], sumDb[kSetMax][2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t N = k.N, Hg = k.H / k.G;
    const int set = (int)(blockIdx.x % ws.sets);
    const int64_t bg = blockIdx.x / ws.sets, g = bg % k.G, b = bg / k.G;
    const int64_t len = row_len(k.lengths, b, N);
    const int64_t h0 = g * Hg + (int64_t)set * ws.per;
    const int64_t left = Hg - (int64_t)set * ws.per;
    const int nch = (int)(left < ws.per ? left : ws.per);
    for (int i = threadIdx.x; i < nch * kModes; i += 256) {
        const int c = i / kModes, n = n0 + i % kModes;
        sumA[c][i % kModes] = 0.f;
        carry[c][i % kModes] = (dx_out && n < k.S) ? dx_out[(b * k.H + h0 + c) * k.S + n] : 0.f;
    }
    for (int i = threadIdx.x; i < nch * 2; i += 256) sumDb[i / 2][i & 1] = 0.f;
    __syncthreads();
    for (int64_t ch = nchunk - 1; ch >= 0; --ch) {
        const int64_t t0 = ch * kSelChunk + lane * kJT, valid = len - t0;
        float Bv[4][kJT], Cv[4][kJT], aB[4][kJT], aC[4][kJT];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int n = n0 + wave * 4 + q;
            const int64_t bc = ((b * k.G + g) * k.S + (n < k.S ? n : 0)) * N + t0;
            ld_row<IO, kJT>(k.Bm + bc, Bv[q], valid);
            ld_row<IO, kJT>(k.C + bc, Cv[q], valid);
#pragma unroll
            for (int i = 0; i < kJT; ++i) aB[q][i] = aC[q][i] = 0.f;
        }
        for (int c0 = 0; c0 < nch; c0 += 4) {
            const int mine = c0 + wave;
            const int64_t h = h0 + mine, r = b * k.H + h;
            float u[kJT], p[kJT], z[kJT], gy[kJT], d[kJT], dr[kJT];
            if (mine < nch) {
                const float bias = k.dt_bias ? k.dt_bias[h] : 0.f;
                ld_row<IO, kJT>(k.u + r * N + t0, u, valid);
                ld_row<IO, kJT>(k.dt + r * N + t0, p, valid);
                ld_row<IO, kJT>(dy + r * N + t0, gy, valid);
                if (k.z) ld_row<IO, kJT>(k.z + r * N + t0, z, valid);
#pragma unroll
                for (int i = 0; i < kJT; ++i) {
                    p[i] += bias;
                    d[i] = k.softplus ? softplus(p[i]) : p[i];
                    if (i >= valid) d[i] = 0.f;
                    dr[i] = k.z ? gy[i] * z[i] * sigmoid(z[i]) : gy[i];
                    pre[wave][0][lane * kJT + i] = d[i];
                    pre[wave][1][lane * kJT + i] = d[i] * u[i];
                    pre[wave][2][lane * kJT + i] = dr[i];
                }
            }
            __syncthreads();
            for (int j = 0; j < 4 && c0 + j < nch; ++j) {
                const int c = c0 + j;
                const int64_t rc = b * k.H + h0 + c;
                float dd[kJT], bu[kJT], rr[kJT], sr[kJT], sb[kJT], sk[kJT];
#pragma unroll
                for (int i = 0; i < kJT; ++i) {
                    dd[i] = pre[j][0][lane * kJT + i];
                    bu[i] = pre[j][1][lane * kJT + i];
                    rr[i] = pre[j][2][lane * kJT + i];
                    sr[i] = sb[i] = sk[i] = 0.f;
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int m = wave * 4 + q, n = n0 + m;
                    if (n >= k.S) break;
                    const float A = k.A[(h0 + c) * k.S + n], A2 = A * kLog2e;
                    float a[kJT], ax[kJT], P = 1.f, Q = 0.f;
#pragma unroll
                    for (int i = 0; i < kJT; ++i) {
                        a[i] = exp2_(dd[i] * A2);
                        P *= a[i];
                        Q = fmaf(a[i], Q, bu[i] * Bv[q][i]);
                    }
                    const float Pl = P;
                    prefix_maps(P, Q, lane);
                    float x = fmaf(P, saved[(rc * nchunk + ch) * k.S + n], Q);
#pragma unroll
                    for (int i = 0; i < kJT; ++i) {
                        ax[i] = a[i] * x;
                        x = fmaf(bu[i], Bv[q][i], ax[i]);
                        sr[i] = fmaf(Cv[q][i], x, sr[i]);
                        aC[q][i] = fmaf(rr[i], x, aC[q][i]);
                    }
                    P = Pl;
                    Q = 0.f;
#pragma unroll
                    for (int i = kJT - 1; i >= 0; --i) Q = a[i] * fmaf(Cv[q][i], rr[i], Q);
                    suffix_maps(P, Q, lane);
                    float e = fmaf(P, carry[c][m], Q), sA = 0.f;
#pragma unroll
                    for (int i = kJT - 1; i >= 0; --i) {
                        const float gx = fmaf(Cv[q][i], rr[i], e), w = gx * ax[i];
                        aB[q][i] = fmaf(gx, bu[i], aB[q][i]);
                        sb[i] = fmaf(gx, Bv[q][i], sb[i]);
                        sk[i] = fmaf(w, A, sk[i]);
                        sA = fmaf(w, dd[i], sA);
                        e = a[i] * gx;
                    }
                    sA = wave_sum(sA);
                    if (lane == 0) {
                        carry[c][m] = e;
                        sumA[c][m] += sA;
                    }
                }
#pragma unroll
                for (int i = 0; i < kJT; ++i) {
                    part[j][wave][0][lane * kJT + i] = sr[i];
                    part[j][wave][1][lane * kJT + i] = sb[i];
                    part[j][wave][2][lane * kJT + i] = sk[i];
                }
            }
            __syncthreads();
            if (mine < nch) {
                const float Dh = k.D ? k.D[h] : 0.f;
                const int64_t plane = k.B * k.H * N, keep = N - t0;
                float o0[kJT], o1[kJT], o2[kJT], sD = 0.f, sp = 0.f;
#pragma unroll
                for (int i = 0; i < kJT; ++i) {
                    float s[3];
#pragma unroll
                    for (int f = 0; f < 3; ++f) {
                        s[f] = 0.f;
#pragma unroll
                        for (int w = 0; w < 4; ++w) s[f] += part[wave][w][f][lane * kJT + i];
                        if (ws.acc && i < keep) {
                            float *q = ws.acc + f * plane + r * N + t0 + i;
                            if (n0 > 0) s[f] += *q;
                            if (!last_block) *q = s[f];
                        }
                    }
                    const float raw = fmaf(Dh, u[i], s[0]);
                    o0[i] = fmaf(d[i], s[1], Dh * dr[i]);
                    o1[i] = fmaf(u[i], s[1], s[2]);
                    if (k.softplus) o1[i] *= sigmoid(p[i]);
                    if (k.z) {
                        const float sg = sigmoid(z[i]);
                        o2[i] = gy[i] * raw * sg * (1.f + z[i] * (1.f - sg));
                    }
                    if (i >= valid) o0[i] = o1[i] = o2[i] = 0.f;
                    sD = fmaf(dr[i], u[i], sD);
                    sp += o1[i];
                }
                if (last_block) {
                    st_row<IO, kJT>(du + r * N + t0, o0, keep);
                    st_row<IO, kJT>(ddt + r * N + t0, o1, keep);
                    if (dz) st_row<IO, kJT>(dz + r * N + t0, o2, keep);
                    sD = wave_sum(sD);
                    sp = wave_sum(sp);
                    if (lane == 0) {
                        sumDb[mine][0] += sD;
                        sumDb[mine][1] += sp;
                    }
                }
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int n = n0 + wave * 4 + q;
            if (n >= k.S) break;
            const int64_t o = ((((int64_t)set * k.B + b) * k.G + g) * k.S + n) * N + t0;
#pragma unroll
            for (int i = 0; i < kJT; ++i)
                if (t0 + i < N) {
                    ws.dB[o + i] = aB[q][i];
                    ws.dC[o + i] = aC[q][i];
                }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nch * kModes; i += 256) {
        const int c = i / kModes, m = i % kModes, n = n0 + m;
        if (n >= k.S) continue;
        const int64_t o = (b * k.H + h0 + c) * k.S + n;
        ws.dA[o] = sumA[c][m];
        if (dx_in) dx_in[o] = carry[c][m];
    }
    if (last_block)
        for (int i = threadIdx.x; i < nch * 2; i += 256) ws.dDb[(b * k.H + h0) * 2 + i] = sumDb[i / 2][i & 1];
}

// dB, dC: the sets' sums, in order; M = B*G*S*N values each.
template <int IO>
__global__ __launch_bounds__(256) void k_sel_join(const float *__restrict__ pB, const float *__restrict__ pC,
                                                  typename io_elem<IO>::T *__restrict__ dB,
                                                  typename io_elem<IO>::T *__restrict__ dC, int64_t M, int sets) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= M) return;
    float sB = 0.f, sC = 0.f;
    for (int s = 0; s < sets; ++s) {
        sB += pB[s * M + i];
        sC += pC[s * M + i];
    }
    dB[i] = from_f<IO>(sB);
    dC[i] = from_f<IO>(sC);
}

// dA, dD, ddt_bias: sums over the batch, in order.
__global__ __launch_bounds__(256) void k_sel_params(const float *__restrict__ pA, const float *__restrict__ pDb,
                                                    float *__restrict__ dA, float *__restrict__ dD,
                                                    float *__restrict__ ddt_bias, int64_t B, int64_t H, int S) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, HS = H * S;
    if (i < HS) {
        float s = 0.f;
        for (int64_t b = 0; b < B; ++b) s += pA[b * HS + i];
        dA[i] = s;
    } else if (i < HS + H) {
        const int64_t h = i - HS;
        float s = 0.f, t = 0.f;
        for (int64_t b = 0; b < B; ++b) {
            s += pDb[(b * H + h) * 2];
            t += pDb[(b * H + h) * 2 + 1];
        }
        if (dD) dD[h] = s;
        if (ddt_bias) ddt_bias[h] = t;
    }
}

// -------------------------------------------------------------- single token

// LPC lanes per channel, four modes each (a channel's states are read as
// whole lines).  A slot outside the pool leaves its row's output zero and no
// state changed.
template <int IO>
__global__ __launch_bounds__(256) void k_sel_step(const typename io_elem<IO>::T *__restrict__ u,
                                                  const typename io_elem<IO>::T *__restrict__ dt,
                                                  const float *__restrict__ A,
                                                  const typename io_elem<IO>::T *__restrict__ Bm,
                                                  const typename io_elem<IO>::T *__restrict__ C,
                                                  const float *__restrict__ D,
                                                  const typename io_elem<IO>::T *__restrict__ z,
                                                  const float *__restrict__ dt_bias,
                                                  const int32_t *__restrict__ slots, const float *x_in, float *x_out,
                                                  typename io_elem<IO>::T *__restrict__ y, int64_t H, int64_t P,
                                                  int S, int G, int softplus_, int lpc) {
    const int sub = (int)threadIdx.x % lpc;
    const int64_t h = (int64_t)blockIdx.x * (256 / lpc) + threadIdx.x / lpc, b = blockIdx.y;
    const int64_t slot = slots ? (int64_t)slots[b] : b;
    const bool in = h < H, ok = in && slot >= 0 && slot < P;
    float s = 0.f, uv = 0.f;
    if (ok) {
        uv = to_f<IO>(u[b * H + h]);
        float d = to_f<IO>(dt[b * H + h]) + (dt_bias ? dt_bias[h] : 0.f);
        if (softplus_) d = softplus(d);
        const float du = d * uv;
        const int64_t g = h / (H / G), o = (slot * H + h) * S, bc = (b * G + g) * S;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = sub * 4 + i;
            if (n < S) {
                const float a = exp2_(d * (A[h * S + n] * kLog2e));
                const float x = fmaf(a, x_in[o + n], du * to_f<IO>(Bm[bc + n]));
                x_out[o + n] = x;
                s = fmaf(to_f<IO>(C[bc + n]), x, s);
            }
        }
    }
    for (int m = lpc >> 1; m >= 1; m >>= 1) s += __shfl_xor(s, m);
    if (in && sub == 0) {
        float v = 0.f;
        if (ok) {
            v = fmaf(D ? D[h] : 0.f, uv, s);
            if (z) {
                const float zz = to_f<IO>(z[b * H + h]);
                v *= zz * sigmoid(zz);
            }
        }
        y[b * H + h] = from_f<IO>(v);
    }
}

template <int IO>
SelK<typename io_elem<IO>::T> pack_args(const SelArgs &a) {
    using T = typename io_elem<IO>::T;
    return SelK<T>{(const T *)a.u, (const T *)a.dt, (const T *)a.Bm, (const T *)a.C, (const T *)a.z, a.A, a.D,
                   a.dt_bias, a.x_in, a.lengths, a.B, a.H, a.N, a.S, a.G, a.softplus};
}

// Sets of channels per group: enough blocks to fill the chip twice, sets of
// at most kSetMax channels.
void bwd_sets(int64_t B, int64_t H, int64_t G, int *sets, int *per) {
    const int64_t Hg = H / G;
    const int64_t want = B > 0 ? (512 + B * G - 1) / (B * G) : 1;
    int64_t p = (Hg + want - 1) / want;
    p = (p + 3) / 4 * 4;
    if (p > kSetMax) p = kSetMax;
    *per = (int)p;
    *sets = (int)((Hg + p - 1) / p);
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace layout; base may be null (sizes only).
size_t bwd_layout(int64_t B, int64_t H, int64_t N, int64_t S, int64_t G, char *base, SelBwdWs *w) {
    bwd_sets(B, H, G, &w->sets, &w->per);
    const size_t m = align256((size_t)w->sets * (size_t)(B * G * S * N) * 4);
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        float *p = base && bytes ? (float *)(base + at) : nullptr;
        at += align256(bytes);
        return p;
    };
    w->dB = take(m);
    w->dC = take(m);
    w->dA = take((size_t)(B * H * S) * 4);
    w->dDb = take((size_t)(B * H) * 8);
    w->acc = take(S > kModes ? (size_t)(B * H * N) * 12 : 0);
    return at;
}

int64_t chunks(int64_t N) { return (N + kSelChunk - 1) / kSelChunk; }

template <int IO, int LPR, int WPR>
hipError_t scan_lanes(const SelArgs &a, void *y, float *x_out, float *saved, hipStream_t s) {
    using T = typename io_elem<IO>::T;
    constexpr int rows = 4 / WPR * 64 / LPR;
    return launch(k_sel_scan<IO, LPR, WPR>, dim3((unsigned)((a.B * a.H + rows - 1) / rows)), dim3(256), 0, s,
                  pack_args<IO>(a), (T *)y, x_out, saved, chunks(a.N));
}

template <int IO>
hipError_t scan_io(const SelArgs &a, void *y, float *x_out, float *saved, hipStream_t s) {
    if (a.N <= 16 * kIT) return scan_lanes<IO, 16, 1>(a, y, x_out, saved, s);
    if (a.N > 64 * kIT && a.B * a.H < 4096) return scan_lanes<IO, 64, 4>(a, y, x_out, saved, s);
    return scan_lanes<IO, 64, 1>(a, y, x_out, saved, s);
}

template <int IO>
hipError_t bwd_io(const SelArgs &a, const float *saved, const void *dy, const float *dx_out, const SelGrads &g,
                  char *ws, hipStream_t s) {
    using T = typename io_elem<IO>::T;
    SelBwdWs w;
    bwd_layout(a.B, a.H, a.N, a.S, a.G, ws, &w);
    const dim3 grid((unsigned)(a.B * a.G * w.sets));
    for (int n0 = 0; n0 < a.S && a.B > 0; n0 += kModes) {
        const hipError_t e =
            launch(k_sel_bwd<IO>, grid, dim3(256), 0, s, pack_args<IO>(a), saved, (const T *)dy, dx_out, (T *)g.du,
                   (T *)g.ddt, (T *)g.dz, g.dx_in, w, chunks(a.N), n0, n0 + kModes >= a.S ? 1 : 0);
        if (e != hipSuccess) return e;
    }
    const int64_t M = a.B * a.G * a.S * a.N;
    if (M > 0) {
        const hipError_t e = launch(k_sel_join<IO>, dim3((unsigned)((M + 255) / 256)), dim3(256), 0, s, w.dB, w.dC,
                                    (T *)g.dB, (T *)g.dC, M, w.sets);
        if (e != hipSuccess) return e;
    }
    return launch(k_sel_params, dim3((unsigned)((a.H * (a.S + 1) + 255) / 256)), dim3(256), 0, s, w.dA, w.dDb, g.dA,
                  g.dD, g.ddt_bias, a.B, a.H, a.S);
}

}  // namespace

size_t selective_saved_floats(int64_t B, int64_t H, int64_t N, int64_t S) {
    return (size_t)(B * H * S) * (size_t)chunks(N);
}

size_t selective_bwd_workspace(int64_t B, int64_t H, int64_t N, int64_t S, int64_t G) {
    SelBwdWs w;
    return bwd_layout(B, H, N, S, G, nullptr, &w);
}

hipError_t launch_selective_scan(const SelArgs &a, void *y, float *x_out, float *saved, int io, hipStream_t s) {
    switch (io) {
        case IO_F32: return scan_io<IO_F32>(a, y, x_out, saved, s);
        case IO_F16: return scan_io<IO_F16>(a, y, x_out, saved, s);
        case IO_BF16: return scan_io<IO_BF16>(a, y, x_out, saved, s);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_selective_scan_bwd(const SelArgs &a, const float *saved, const void *dy, const float *dx_out,
                                     const SelGrads &g, int io, void *ws, hipStream_t s) {
    switch (io) {
        case IO_F32: return bwd_io<IO_F32>(a, saved, dy, dx_out, g, (char *)ws, s);
        case IO_F16: return bwd_io<IO_F16>(a, saved, dy, dx_out, g, (char *)ws, s);
        case IO_BF16: return bwd_io<IO_BF16>(a, saved, dy, dx_out, g, (char *)ws, s);
        default: return hipErrorInvalidValue;
    }
}

template <int IO>
static hipError_t step_io(const void *u, const void *dt, const float *A, const void *Bm, const void *C,
                          const float *D, const void *z, const float *dt_bias, const int32_t *slots,
                          const float *x_in, float *x_out, void *y, int64_t B, int64_t H, int64_t P, int S, int G,
                          int softplus, hipStream_t s) {
    using T = typename io_elem<IO>::T;
    int lpc = 1;
    while (lpc * 4 < S) lpc <<= 1;
    return launch(k_sel_step<IO>, dim3((unsigned)((H * lpc + 255) / 256), (unsigned)B), dim3(256), 0, s, (const T *)u,
                  (const T *)dt, A, (const T *)Bm, (const T *)C, D, (const T *)z, dt_bias, slots, x_in, x_out, (T *)y,
                  H, P, S, G, softplus, lpc);
}

hipError_t launch_selective_step(const void *u, const void *dt, const float *A, const void *Bm, const void *C,
                                 const float *D, const void *z, const float *dt_bias, const int32_t *slots,
                                 const float *x_in, float *x_out, void *y, int64_t B, int64_t H, int64_t P, int S,
                                 int G, int softplus, int io, hipStream_t s) {
    switch (io) {
        case IO_F32: return step_io<IO_F32>(u, dt, A, Bm, C, D, z, dt_bias, slots, x_in, x_out, y, B, H, P, S, G, softplus, s);
        case IO_F16: return step_io<IO_F16>(u, dt, A, Bm, C, D, z, dt_bias, slots, x_in, x_out, y, B, H, P, S, G, softplus, s);
        case IO_BF16: return step_io<IO_BF16>(u, dt, A, Bm, C, D, z, dt_bias, slots, x_in, x_out, y, B, H, P, S, G, softplus, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace h3c
