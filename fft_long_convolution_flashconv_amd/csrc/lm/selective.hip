// selective.hip -- selective state-space scan: prompts, backward pass, tokens.
//
// Per channel h with S real modes and step t (B_t, C_t shared by the channels
// of a group):
//   d_t = softplus(dt_t + dt_bias)  (or dt_t + dt_bias)
//   x_t[j] = exp(d_t A[j]) x_{t-1}[j] + d_t u_t B_t[j]
//   r_t = sum_j C_t[j] x_t[j] + D u_t,   y_t = r_t silu(z_t)  (or r_t)
// All arithmetic is fp32, and so are states and saved states; y and the gradients
// of 16-bit inputs are rounded once.  Steps at and past a row's length have
// d_t = 0: the state passes them unchanged.
// An exponential (two issue slots) and six multiply-adds or conversions per mode
// and step forward, against 8 to 16 bytes per step of all modes: the vector ALUs
// bound it, at 16 modes about three times above the memory traffic.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "lm_device.h"
#include "lm_internal.h"

namespace h3c {
namespace {

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

// Sum over the 16 lanes of a DPP row, in every lane of it.
__device__ __forceinline__ float row_sum(float v) {
    v += dpp0<0xb1>(v);   // quad_perm [1,0,3,2]
    v += dpp0<0x4e>(v);   // quad_perm [2,3,0,1]
    v += dpp0<0x141>(v);  // row_half_mirror
    v += dpp0<0x140>(v);  // row_mirror
    return v;
}
// Sum over the wave, in its last lane.
__device__ __forceinline__ float wave_sum_last(float v) {
    v = row_sum(v);
    v += dpp_rows<0x142, 0xa>(0.f, v);  // row_bcast:15
    v += dpp_rows<0x143, 0xc>(0.f, v);  // row_bcast:31
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

// Elements off .. off + n - 1 of p.  FULL: all n are valid; else elements from
// `valid` on are zero: a lane with some of them loads the n elements that end
// at its last valid one (still in the tensor unless at its very start) and
// shifts them down.
template <int IO, int n, bool FULL>
__device__ __forceinline__ Raw<IO, n> ld_raw(const typename io_elem<IO>::T *p, int64_t off, int64_t valid) {
    using T = typename io_elem<IO>::T;
    constexpr int W = Raw<IO, n>::kWords, E = 4 / (int)sizeof(T);
    Raw<IO, n> r;
    if (FULL || valid >= n) {
        const Pack<T, n> q = *reinterpret_cast<const Pack<T, n> *>(p + off);
        __builtin_memcpy(&r, &q, sizeof(r));
        return r;
    }
#pragma unroll
    for (int i = 0; i < W; ++i) r.w[i] = 0;
    if (valid <= 0) return r;
    if (off + valid >= n) {
        const Pack<T, n> q = *reinterpret_cast<const Pack<T, n> *>(p + off + valid - n);
        __builtin_memcpy(&r, &q, sizeof(r));
        const int s = n - (int)valid;  // elements to drop, 1 .. n - 1
        if (E == 2) {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const uint32_t hi = i + 1 < W ? r.w[i + 1] : 0u;
                r.w[i] = (s & 1) ? (r.w[i] >> 16 | hi << 16) : r.w[i];
            }
        }
#pragma unroll
        for (int k = 1; k < W; k *= 2)
#pragma unroll
            for (int i = 0; i < W; ++i) r.w[i] = (s & (E * k)) ? (i + k < W ? r.w[i + k] : 0u) : r.w[i];
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (E == 1) {
                if (i < valid) r.w[i] = __builtin_bit_cast(uint32_t, p[off + i]);
            } else {
                if (2 * i < valid) r.w[i] = __builtin_bit_cast(uint16_t, p[off + 2 * i]);
                if (2 * i + 1 < valid) r.w[i] |= (uint32_t)__builtin_bit_cast(uint16_t, p[off + 2 * i + 1]) << 16;
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

// o = r times u, element by element.  fp16: one instruction converts and
// multiplies (the compiler converts first).
template <int IO, int n>
__device__ __forceinline__ void times(const Raw<IO, n> &r, const float (&u)[n], float (&o)[n]) {
    if constexpr (IO == IO_F16) {
#pragma unroll
        for (int i = 0; i < n; i += 2) {
            asm("v_fma_mix_f32 %0, %1, %2, 0 op_sel_hi:[1,0,0]" : "=v"(o[i]) : "v"(r.w[i / 2]), "v"(u[i]));
            asm("v_fma_mix_f32 %0, %1, %2, 0 op_sel:[1,0,0] op_sel_hi:[1,0,0]"
                : "=v"(o[i + 1])
                : "v"(r.w[i / 2]), "v"(u[i + 1]));
        }
    } else {
        unpack<IO, n>(r, o);
#pragma unroll
        for (int i = 0; i < n; ++i) o[i] *= u[i];
    }
}

// Keeps the values' computation here: the compiler otherwise moves it past
// later work, and its operands stay in registers for all that time.
template <int n>
__device__ __forceinline__ void hold(float (&v)[n]) {
#pragma unroll
    for (int i = 0; i < n; ++i) asm volatile("" : "+v"(v[i]));
}

// A map x -> 2^E x + Q by its factor.  Where no mode has A > 0 and no step is
// negative, E <= 0, and the factor is 2^E itself.  Else (GROWS) the factor of
// many steps may pass the largest float where the state, zero or small, does
// not: it is held as 2^(E/2), at most 2^127, and applied twice.  (At that bound
// a state that is not zero passes the largest float itself.)
constexpr float kMostGrowth = 0x1p127f;
template <bool GROWS>
__device__ __forceinline__ float factor(float E) {
    return GROWS ? fminf(exp2_(0.5f * E), kMostGrowth) : exp2_(E);
}
template <bool GROWS>
__device__ __forceinline__ float apply(float P, float x, float Q) {
    return GROWS ? fmaf(P * x, P, Q) : fmaf(P, x, Q);
}
template <bool GROWS>
__device__ __forceinline__ float compose(float P, float R) {
    return GROWS ? fminf(P * R, kMostGrowth) : P * R;
}

// P composed with the P of the lane CTRL names.  In a group of one DPP row (16
// lanes) the lanes without such a source have reached the group's start, whose
// entering state is folded into Q: their P is not needed any more, and reading
// zero is as good as one (and is one instruction; P is finite).  Otherwise it
// reads one.
template <int LPR, bool GROWS, int CTRL>
__device__ __forceinline__ float shorten(float P) {
    return compose<GROWS>(P, LPR == 16 ? dpp0<CTRL>(P) : dpp_rows<CTRL, 0xf>(1.f, P));
}

// Inclusive composition over groups of LPR lanes of maps with factors P, whose
// first lane has its entering state folded into Q: on return Q is the state
// that leaves each lane.
template <int LPR, bool GROWS>
__device__ __forceinline__ void scan_states(float P, float &Q) {
    Q = apply<GROWS>(P, dpp0<0x111>(Q), Q);  // row_shr:1
    P = shorten<LPR, GROWS, 0x111>(P);
    Q = apply<GROWS>(P, dpp0<0x112>(Q), Q);
    P = shorten<LPR, GROWS, 0x112>(P);
    Q = apply<GROWS>(P, dpp0<0x114>(Q), Q);
    P = shorten<LPR, GROWS, 0x114>(P);
    Q = apply<GROWS>(P, dpp0<0x118>(Q), Q);
    if constexpr (LPR == 64) {
        P = shorten<LPR, GROWS, 0x118>(P);
        // the rows of 16 lanes: row 1 after row 0 and row 3 after row 2, then
        // rows 2 and 3 after row 1
        const float q = dpp_rows<0x142, 0xa>(0.f, Q), p = dpp_rows<0x142, 0xa>(1.f, P);  // row_bcast:15
        Q = apply<GROWS>(P, q, Q);
        P = compose<GROWS>(P, p);
        Q = apply<GROWS>(P, dpp_rows<0x143, 0xc>(0.f, Q), Q);  // row_bcast:31
    }
}

// Sums of d over one lane's steps, over the lanes before it in its wave, and
// over the wave.
struct Sums {
    float lane, before, wave;
};

// How a piece lies in its rows.
enum Fit {
    kFull,  // every lane has kIT valid steps
    kTail,  // some lane has fewer: a lane that would read past its row's end reads
            // the row's last kIT steps instead and passes over those of others (so
            // every load is one in-row vector, whatever the length)
    kShort  // as kTail, of rows with fewer than kIT steps: element loads
};

// Steps at .. at + n - 1 of the kIT at p + off.
template <int IO, int n, Fit F>
__device__ __forceinline__ Raw<IO, n> ld_steps(const typename io_elem<IO>::T *p, int64_t off, int at, int64_t N) {
    if constexpr (F != kShort) return ld_raw<IO, n, true>(p, off + at, 0);
    typename io_elem<IO>::T v[n];
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = p[off + (at + i < N ? at + i : N - 1)];
    Raw<IO, n> r;
    __builtin_memcpy(&r, v, sizeof(r));
    return r;
}

// How the four waves of a block share their rows.
enum Share {
    kOwnRows,  // each wave has rows of its own
    kTime,     // four pieces in a row of one row
    kModeMod4  // the same pieces of the same rows; wave w has modes w, w + 4, ...
};

// One mode of one piece: o += C x.  The state `in` enters the first lane, and
// the state that leaves the row's last lane is kept in *st.  kTime: the waves
// exchange the maps of their pieces through `maps` (one barrier), and every
// wave keeps in its own *st the state before the first and then after the
// last.  B and C arrive as loaded; nextB() and nextC() load a later mode's
// into the same registers once they are unpacked.
template <int IO, int LPR, Share SH, Fit F, bool GROWS, class NextB, class NextC>
__device__ __forceinline__ void scan_mode(Raw<IO, kIT> &rB, Raw<IO, kIT> &rC, float A2, float in,
                                          const float (&d)[kIT], const float (&u)[kIT], const Sums &sum,
                                          float (&o)[kIT], float *st, int l, float2 (*maps)[4], float *saved,
                                          const Raw<IO, kIT> &own, const NextB &nextB, const NextC &nextC) {
    constexpr int IT = kIT;
    float a[IT], w[IT], c[IT], P = factor<GROWS>(sum.lane * A2), Q = SH != kTime ? in : 0.f;
    if (F != kFull) {
#pragma unroll
        for (int i = 0; i < Raw<IO, IT>::kWords; ++i) rB.w[i] &= own.w[i];  // (what is passed over may be NaN)
    }
    times<IO, IT>(rB, u, w);
    hold(w);
    nextB();
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        a[i] = exp2_(d[i] * A2);
        Q = fmaf(a[i], Q, w[i]);
    }
    scan_states<LPR, GROWS>(P, Q);
    float x0 = dpp0<LPR == 64 ? 0x138 : 0x111>(Q);  // from the lane before
    if constexpr (SH != kTime) {
        x0 += in;
    } else {
        const int wave = threadIdx.x >> 6;
        if (l == LPR - 1) (*maps)[wave] = make_float2(factor<GROWS>(sum.wave * A2), Q);
        __syncthreads();
        float x = *st, enter = x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 m = (*maps)[i];
            x = apply<GROWS>(m.x, x, m.y);
            if (i + 1 == wave) enter = x;
        }
        Q = x;
        x0 = apply<GROWS>(factor<GROWS>(sum.before * A2), enter, x0);
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

// The steps of one lane in one piece: its first is t0; it loads kIT of them at
// offset `row` of u and dt and `bc` of mode 0 of B and C, and has loaded steps
// lo .. hi - 1 for its own.
struct Lane {
    int64_t t0, row, bc;
    int lo, hi;
};

// One piece of LPR*IT steps of each of the wave's rows, from its u and dt as
// loaded; reload() loads the next piece's into the same registers.  turn: which
// of the two buffers of maps mode 0 takes.  The modes take them in turn, across
// pieces too: with one barrier per mode, a wave may write a mode's map while
// another still reads those of the mode before, never of the one before that.
template <int IO, int LPR, Share SH, Fit F, bool GROWS, class Reload>
__device__ __forceinline__ void scan_piece(const SelK<typename io_elem<IO>::T> &k, const Lane &p, Raw<IO, kIT> &ru,
                                           Raw<IO, kIT> &rd, const float *Ap, float Dh, float bias, float *st, int l,
                                           bool live, int turn, float2 (*maps)[4], float (*part)[kIT][64],
                                           typename io_elem<IO>::T *y, float *saved, const Reload &reload) {
    constexpr int IT = kIT, AH = kAhead, MS = SH == kModeMod4 ? 4 : 1;
    const int last = k.S - 1, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), first = MS > 1 ? wave : 0;
    Raw<IO, IT> rB[AH], rC[AH];
    const auto loadB = [&](int n) { return ld_steps<IO, IT, F>(k.Bm, p.bc + (n < last ? n : last) * k.N, 0, k.N); };
    const auto loadC = [&](int n) { return ld_steps<IO, IT, F>(k.C, p.bc + (n < last ? n : last) * k.N, 0, k.N); };
#pragma unroll
    for (int j = 0; j < AH; ++j) {
        rB[j] = loadB(first + MS * j);
        rC[j] = loadC(first + MS * j);
    }
    float u[IT], d[IT], o[IT];
    Sums sum = {0.f, 0.f, 0.f};
    Raw<IO, IT> own;
    if (F != kFull) {
        constexpr int E = 4 / (int)sizeof(typename io_elem<IO>::T);
#pragma unroll
        for (int i = 0; i < Raw<IO, IT>::kWords; ++i) {
            const auto in = [&](int t) { return t >= p.lo && t < p.hi; };
            if (E == 1) own.w[i] = in(i) ? ~0u : 0u;
            else own.w[i] = (in(2 * i) ? 0xffffu : 0u) | (in(2 * i + 1) ? 0xffff0000u : 0u);
            ru.w[i] &= own.w[i];
        }
    }
    unpack<IO, IT>(ru, u);
    unpack<IO, IT>(rd, d);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        d[i] += bias;
        if (k.softplus) d[i] = softplus(d[i]);
        if (F != kFull && (i < p.lo || i >= p.hi)) d[i] = 0.f;
        o[i] = first == 0 ? Dh * u[i] : 0.f;
        u[i] *= d[i];
        sum.lane += d[i];
    }
    if (SH == kTime) {
        float s = sum.lane;
        scan_states<64, false>(1.f, s);
        sum.before = dpp0<0x138>(s);
        sum.wave = lane_of(s, 63);
    }
    reload();
    // a lane's first step is where a state is saved
    float *sv = saved && live && p.t0 < k.N && p.t0 % kSelChunk == 0 ? saved + p.t0 / kSelChunk * k.S : nullptr;
    float A = Ap[first < last ? first : last], in = st[first];
    for (int n0 = first; n0 < k.S; n0 += MS * AH) {
#pragma unroll
        for (int j = 0; j < AH; ++j) {
            const int n = n0 + MS * j, next = n + MS < last ? n + MS : last;
            if (AH > 1 && n >= k.S) break;
            const float A2 = A * kLog2e, in0 = l == 0 ? in : 0.f;
            A = Ap[next];
            in = st[next];
            scan_mode<IO, LPR, SH, F, GROWS>(rB[j], rC[j], A2, in0, d, u, sum, o, st + n, l, maps + ((n + turn) & 1), sv ? sv + n : nullptr,
                               own, [&] { rB[j] = loadB(n + MS * AH); }, [&] { rC[j] = loadC(n + MS * AH); });
        }
    }
    // y of the lane: all of its steps, or with the modes' waves a quarter each
    constexpr int OT = IT / MS;
    const int at = OT * first;
    float out[OT];
    if constexpr (MS > 1) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < IT; ++i) part[wave][i][lane] = o[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < OT; ++i)
            out[i] = (part[0][at + i][lane] + part[1][at + i][lane]) + (part[2][at + i][lane] + part[3][at + i][lane]);
        __syncthreads();
    } else {
#pragma unroll
        for (int i = 0; i < OT; ++i) out[i] = o[i];
    }
    if (k.z) {
        float z[OT];
        unpack<IO, OT>(ld_steps<IO, OT, F>(k.z, p.row, at, k.N), z);
#pragma unroll
        for (int i = 0; i < OT; ++i) out[i] *= z[i] * sigmoid(z[i]);
    }
    if (!live) return;
    if (F == kFull || (p.lo <= at && p.hi >= at + OT)) {
        st_row<IO, OT>(y + p.row + at, out, OT);
    } else {
#pragma unroll
        for (int i = 0; i < OT; ++i)
            if (at + i >= p.lo && (F != kShort || at + i < k.N))
                y[p.row + at + i] = from_f<IO>(at + i < p.hi ? out[i] : 0.f);
    }
}

// LPR lanes per row (b, h), 64 / LPR rows per wave; lane l of a row holds
// steps l*IT .. l*IT + IT - 1 of each piece of LPR*IT steps.  Per mode, each
// lane runs its steps from a zero state, the lanes' maps x -> P x + Q are
// composed by a scan over the row's lanes, and each lane runs its steps again
// from the state that enters it: two multiply-adds per (step, mode) instead
// of one, and no state leaves the chip between pieces.  Sixteen steps per lane
// make the scan over lanes (14 instructions) a tenth of a mode's work.  The next
// mode's B and C are in flight while one is worked on; three and more modes ahead
// spilled registers, and B and C staged in LDS for the block's rows gained
// nothing.
// Measured, 16 modes with a gate: 8 x 768 x 1024 fp16 36.9 us, 1 x 1024 x 65536
// bf16 483 us, 4 x 2560 x 2048 bf16 with saved states 124 us (146 in a
// training pass): 2.2 to 2.7 million million mode-steps a second, the vector ALUs
// busy 90 to 95 % of the compute units' time.  (In bf16, rows of their own spill 11
// registers at three waves per SIMD.)
template <int IO, int LPR, Share SH>
__global__ __launch_bounds__(256, IO == IO_F32 || LPR == 16 ? 2 : 3) void k_sel_scan(const SelK<typename io_elem<IO>::T> k,
                                                     typename io_elem<IO>::T *__restrict__ y,
                                                     float *__restrict__ x_out, float *__restrict__ saved,
                                                     int64_t nchunk) {
    constexpr int IT = kIT, RPW = 64 / LPR, PIECE = (SH == kTime ? 4 : 1) * LPR * IT;
    static_assert(SH != kTime || LPR == 64, "");
    static_assert(kSelChunk % IT == 0, "saved states fall on a lane's first step");
    __shared__ float state[4][RPW][kMaxModes];
    __shared__ float2 maps[2][4];
    __shared__ float part[SH == kModeMod4 ? 4 : 1][kIT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane / LPR, l = lane % LPR;
    const uint32_t R = (uint32_t)(k.B * k.H), H = (uint32_t)k.H;
    const uint32_t block = (uint32_t)block_id(), r = (SH == kOwnRows ? block * 4 + wave : block) * RPW + sub;
    if (r - sub >= R) return;  // (the whole wave)
    const bool live = r < R;
    const uint32_t rr = live ? r : R - 1, b = rr / H, h = rr - b * H, g = h / (H / (uint32_t)k.G);
    const int64_t N = k.N, len = row_len(k.lengths, b, N);
    const float Dh = k.D ? k.D[h] : 0.f, bias = k.dt_bias ? k.dt_bias[h] : 0.f;
    const float *Ap = k.A + (int64_t)h * k.S;
    float *st = state[wave][sub];
    bool grows = !k.softplus;  // (or might: the same for the waves of a shared row)
    for (int n = l; n < k.S; n += LPR) {
        st[n] = k.x_in ? k.x_in[(int64_t)rr * k.S + n] : 0.f;
        grows |= Ap[n] > 0.f;
    }
    __builtin_amdgcn_wave_barrier();
    float *sv = saved ? saved + (int64_t)rr * nchunk * k.S : nullptr;
    const auto piece = [&](int64_t base) {
        const int64_t t0 = base + (SH == kTime ? wave * 64 * IT : 0) + l * IT;
        const int64_t w0 = t0 <= N - IT ? t0 : (N > IT ? N - IT : 0);  // the first step loaded
        const int lo = (int)(t0 - w0 < IT ? t0 - w0 : IT), hi = (int)(len - w0 < IT ? (len > w0 ? len - w0 : 0) : IT);
        return Lane{t0, rr * N + w0, (int64_t)(b * (uint32_t)k.G + g) * k.S * N + w0, lo, hi > lo ? hi : lo};
    };
    const auto scan = [&](auto growing) {
        constexpr bool GROWS = decltype(growing)::value;
        Raw<IO, IT> ru, rd;
        int64_t base = 0;
        int turn = 0;
        if (__all(len >= PIECE)) {  // the pieces that are full in every row of the wave
            Lane p = piece(0);
            ru = ld_steps<IO, IT, kFull>(k.u, p.row, 0, N);
            rd = ld_steps<IO, IT, kFull>(k.dt, p.row, 0, N);
            bool more;
            do {
                more = __all(len >= base + 2 * PIECE);
                scan_piece<IO, LPR, SH, kFull, GROWS>(k, p, ru, rd, Ap, Dh, bias, st, l, live, turn, maps, part, y, sv, [&] {
                    const int64_t o = more ? p.row + PIECE : p.row;
                    ru = ld_steps<IO, IT, kFull>(k.u, o, 0, N);
                    rd = ld_steps<IO, IT, kFull>(k.dt, o, 0, N);
                });
                __builtin_amdgcn_wave_barrier();
                base += PIECE;
                turn ^= k.S & 1;
                p = piece(base);
            } while (more);
        }
        const auto rest = [&](auto fit) {
            constexpr Fit F = decltype(fit)::value;
            for (; base < N; base += PIECE) {
                const Lane p = piece(base);
                ru = ld_steps<IO, IT, F>(k.u, p.row, 0, N);
                rd = ld_steps<IO, IT, F>(k.dt, p.row, 0, N);
                scan_piece<IO, LPR, SH, F, GROWS>(k, p, ru, rd, Ap, Dh, bias, st, l, live, turn, maps, part, y, sv, [] {});
                __builtin_amdgcn_wave_barrier();
                turn ^= k.S & 1;
            }
        };
        if (LPR == 16 && N < IT) rest(std::integral_constant<Fit, kShort>{});
        else rest(std::integral_constant<Fit, kTail>{});
    };
    // The form that bears growth has a body of its own: without softplus, where
    // it is always taken, 1 x 1024 x 65536 bf16 takes 460 us with it and 439
    // without, 8 x 768 x 1024 fp16 36.5 and 35.8.  (The marks keep the compiler
    // from merging the two, with the registers of both.)
    if (__any(grows)) {
        asm volatile("; growing" ::: "memory");
        scan(std::true_type{});
        asm volatile("; growing" ::: "memory");
    } else {
        asm volatile("; steady" ::: "memory");
        scan(std::false_type{});
        asm volatile("; steady" ::: "memory");
    }
    if (x_out && live)
        for (int n = l; n < k.S; n += LPR)
            if (SH == kOwnRows || wave == (SH == kTime ? 0 : n % 4)) x_out[(int64_t)rr * k.S + n] = st[n];
}

// ------------------------------------------------------------------ backward

// With dr = dy silu(z), x the states and a_t = exp(d_t A):
//   g_t = C_t dr_t + a_{t+1} g_{t+1}          gradient of x_t
//   dC_t = sum_h dr_t x_t                     dB_t = sum_h g_t d_t u_t
//   du_t = D dr_t + d_t sum_j g_t B_t         dd_t = sum_j g_t (a_t x_{t-1}) A + u_t sum_j g_t B_t
//   dA = sum_t g_t (a_t x_{t-1}) d_t          dD = sum dr u,  dz = dy r silu'(z)
// One block takes one batch row and a set of channels of one group, and walks
// the row's pieces of kSelChunk steps from the end, with the states at each
// piece's start as the forward pass saved them.  A wave takes the set's
// channels w, w + 8, ... alone: its four DPP rows of 16 lanes hold four modes
// at a time (row r: modes 4r .. 4r+3 of a block of 16, in four rounds; of fewer
// modes, fewer rounds), lane l
// of a row kJT steps.  So dB and dC of every mode and step stay in one lane's
// registers over all the wave's channels (no atomics), the scans over time
// stay within a DPP row, and the sums over modes are two exchanges between
// rows.  A lane prepares and finishes a quarter of its steps (softplus, gate)
// and the rows share them through LDS.  Factors always take their GROWS form,
// which costs 2 % (4 x 2560 x 2048 bf16, both passes, 506 to 517 us; a second
// body, as the forward pass has, cost 3 to 10: the registers of both).
// Measured: 4 x 2560 x 2048 bf16 with 16 modes 400 us, 0.84 million million
// mode-steps a second; vector ALUs busy 75 % of the time at two waves per SIMD
// (about 250 registers, which dB and dC of 4 modes x 8 steps need; numbers of
// modes other than 16 spill 8 to 17).  Two launches of 16 and 8 modes take 210
// and 174 us at 4 x 2560 x 1024, 8 modes alone 149.
constexpr int kModes = 16, kJT = kSelChunk / 16, kQ = kJT / 4, kWaves = 8, kPerWave = 16;
static_assert(kJT == 8 && kQ == 2 && 2 * kModes * kSelChunk == kWaves * 64 * 8, "one 8-step load of B or C per thread and piece");

struct SelBwdWs {
    float *dB, *dC;        // [sets][B][G][S][N]
    float *dA;             // [B][H][S]
    float *dDb;            // [B][H][2]
    float *acc;            // [B*H][N, in pairs][3][kQ], more than kModes modes only
    int sets, per;         // sets per group, channels per set
};

// As scan_states<16, true>, from the last lane of a DPP row down.
__device__ __forceinline__ void scan_back(float P, float &Q) {
    Q = apply<true>(P, dpp0<0x101>(Q), Q);  // row_shl:1
    P = compose<true>(P, dpp0<0x101>(P));
    Q = apply<true>(P, dpp0<0x102>(Q), Q);
    P = compose<true>(P, dpp0<0x102>(P));
    Q = apply<true>(P, dpp0<0x104>(Q), Q);
    P = compose<true>(P, dpp0<0x104>(P));
    Q = apply<true>(P, dpp0<0x108>(Q), Q);
}

// Sums over the wave's four DPP rows of v[0 .. 7]; row r gets those of
// v[2r], v[2r+1].
__device__ __forceinline__ void sum_rows(const float (&v)[kJT], float (&o)[kQ]) {
    float h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // rows 0, 1 keep i, rows 2, 3 keep i + 4
        const auto x = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, v[i]),
                                                        __builtin_bit_cast(unsigned, v[i + 4]), false, false);
        h[i] = __uint_as_float(x[0]) + __uint_as_float(x[1]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const auto x = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, h[i]),
                                                        __builtin_bit_cast(unsigned, h[i + 2]), false, false);
        o[i] = __uint_as_float(x[0]) + __uint_as_float(x[1]);
    }
}

__device__ __forceinline__ void get8(const float4 *p, int step, float (&v)[8]) {
    const float4 x = p[0], y = p[step];
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
}

// What a lane loads of one channel and piece ahead of its use.
template <int IO>
struct BwdIn {
    Raw<IO, kQ> u, p, z, gy;
    float A[4], x[4];
};

// WHOLE: exactly kModes modes, the common case: no mode is missing, and one
// launch has all of them (else: a launch per kModes modes, whose sums over modes
// pass through ws.acc).
template <int IO, bool WHOLE>
__global__ __launch_bounds__(kWaves * 64, 2) void k_sel_bwd(
    const SelK<typename io_elem<IO>::T> k, const float *__restrict__ saved,
    const typename io_elem<IO>::T *__restrict__ dy, const float *__restrict__ dx_out,
    typename io_elem<IO>::T *__restrict__ du, typename io_elem<IO>::T *__restrict__ ddt,
    typename io_elem<IO>::T *__restrict__ dz, float *__restrict__ dx_in, const SelBwdWs ws, int64_t nchunk, int n0,
    int last_block) {
    constexpr int F4 = kSelChunk / 4;  // float4 per row of steps
    // B and C of the piece, then the rows' exchange; both over again as the
    // buffer that joins the waves' dB and dC
    __shared__ float4 lds[2048];
    __shared__ float4 carry[kWaves][kPerWave][4], sumA[kWaves][kPerWave][4];
    __shared__ float sumDb[kWaves][kPerWave][2];
    float4(*const BC)[kModes][F4] = (float4(*)[kModes][F4])lds;
    const int tid = threadIdx.x, lane = tid & 63, row = lane >> 4, l = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // (scalar: so are the rows' base addresses)
    float4(*const mine)[F4] = (float4(*)[F4])(lds + 2 * kModes * F4) + 3 * wave;
    const int64_t N = k.N, Hg = k.H / k.G;
    const uint32_t block = (uint32_t)block_id();
    const int set = (int)(block % (uint32_t)ws.sets);
    const int64_t bg = block / (uint32_t)ws.sets, g = bg % k.G, b = bg / k.G;
    if (b >= k.B) return;
    const int64_t len = row_len(k.lengths, b, N);
    const int64_t left = Hg - (int64_t)set * ws.per, h0 = g * Hg + (int64_t)set * ws.per;
    const int nset = (int)(left < ws.per ? left : ws.per);
    const int nch = nset > wave ? (nset - wave + kWaves - 1) / kWaves : 0;  // this wave's channels
    const int S = WHOLE ? kModes : k.S;
    const int rounds = WHOLE || S - n0 >= kModes ? 4 : (S - n0 + 3) / 4, m0 = n0 + rounds * row;  // this row's modes
    // channel c of this wave: row r0 + kWaves c of the batch, channel hw + kWaves c
    const int64_t hw = h0 + wave, r0 = b * k.H + hw;
    for (int c = 0; c < nch; ++c)
        if (l < 4) {
            (&carry[wave][c][row].x)[l] = (dx_out && l < rounds && m0 + l < S) ? dx_out[(r0 + kWaves * c) * S + m0 + l] : 0.f;
            (&sumA[wave][c][row].x)[l] = 0.f;
            if (row == 0 && l < 2) sumDb[wave][c][l] = 0.f;
        }
    // this thread's eight steps of B or C in LDS: matrix, mode, steps
    const int cm = tid >> 8, cn = (tid >> 4) & 15, ct = tid & 15;
    const typename io_elem<IO>::T *const bc = cm ? k.C : k.Bm;
    const int n = WHOLE ? cn : n0 + rounds * (cn >> 2) + (cn & 3);
    const bool mode = WHOLE || ((cn & 3) < rounds && n < S);
    const int64_t bc0 = (bg * S + (mode ? n : 0)) * N + ct * 8;
    // valid steps of a piece, and those from step `from` of it on
    const auto steps = [&](int64_t ch, int64_t end) {
        const int64_t n = end - ch * kSelChunk;
        return (int)(n < 0 ? 0 : (n < kSelChunk ? n : kSelChunk));
    };
    const auto load_bc = [&](int64_t ch) {
        return ld_raw<IO, 8, false>(bc, bc0 + ch * kSelChunk, mode ? steps(ch, len) - ct * 8 : 0);
    };
    const int tq = l * kJT + row * kQ;  // this lane's own steps within a piece
    BwdIn<IO> f;
    // the next channel and piece to load: offsets of its row's steps, states
    // and decay rates
    int64_t on = 0, xn = 0;
    const float *An = nullptr;
    const auto start = [&](int64_t ch) {
        on = r0 * N + ch * kSelChunk;
        xn = (r0 * nchunk + ch) * S;
        An = k.A + hw * S;
    };
    const auto load_in = [&](int valid) {
        f.u = ld_raw<IO, kQ, false>(k.u, on + tq, valid);
        f.p = ld_raw<IO, kQ, false>(k.dt, on + tq, valid);
        f.gy = ld_raw<IO, kQ, false>(dy, on + tq, valid);
        if (k.z) f.z = ld_raw<IO, kQ, false>(k.z, on + tq, valid);
        const float *const xh = saved + xn;
        if constexpr (WHOLE) {
            const float4 a = *(const float4 *)(An + m0), x = *(const float4 *)(xh + m0);
            f.A[0] = a.x, f.A[1] = a.y, f.A[2] = a.z, f.A[3] = a.w;
            f.x[0] = x.x, f.x[1] = x.y, f.x[2] = x.z, f.x[3] = x.w;
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const bool in = q < rounds && m0 + q < S;
                f.A[q] = in ? An[m0 + q] : 0.f;
                f.x[q] = in ? xh[m0 + q] : 0.f;
            }
        }
    };
    Raw<IO, 8> rbc;
    if (nchunk > 0) {
        rbc = load_bc(nchunk - 1);
        if (nch > 0) {
            start(nchunk - 1);
            load_in(steps(nchunk - 1, len) - tq);
        }
    }
    for (int64_t ch = nchunk - 1; ch >= 0; --ch) {
        const int valid = steps(ch, len) - tq, keep = steps(ch, N) - tq;  // this lane's steps: valid, and in the row
        {
            // steps 4j .. 4j+3 at (j % 2) * 16 + j / 2: a lane's two reads are
            // consecutive over the lanes of a row
            float v[8];
            unpack<IO, 8>(rbc, v);
            BC[cm][cn][ct] = make_float4(v[0], v[1], v[2], v[3]);
            BC[cm][cn][16 + ct] = make_float4(v[4], v[5], v[6], v[7]);
        }
        __syncthreads();
        if (ch > 0) rbc = load_bc(ch - 1);
        float aB[4][kJT], aC[4][kJT];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < kJT; ++i) aB[q][i] = aC[q][i] = 0.f;
        for (int c = 0; c < nch; ++c) {
            const int64_t h = hw + kWaves * c, o0 = on;
            const float bias = k.dt_bias ? k.dt_bias[h] : 0.f, Dh = k.D ? k.D[h] : 0.f;
            float u[kQ], p[kQ], z[kQ], gy[kQ], d[kQ], dr[kQ], A[4], xs[4];
            unpack<IO, kQ>(f.u, u);
            unpack<IO, kQ>(f.p, p);
            unpack<IO, kQ>(f.gy, gy);
            if (k.z) unpack<IO, kQ>(f.z, z);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                A[q] = f.A[q];
                xs[q] = f.x[q];
            }
            if (c + 1 < nch) {
                on += kWaves * N;
                xn += kWaves * nchunk * S;
                An += kWaves * S;
                load_in(valid);
            } else if (ch > 0) {
                start(ch - 1);
                load_in(steps(ch - 1, len) - tq);
            }
#pragma unroll
            for (int i = 0; i < kQ; ++i) {
                p[i] += bias;
                d[i] = k.softplus ? softplus(p[i]) : p[i];
                if (i >= valid) d[i] = 0.f;
                dr[i] = k.z ? gy[i] * z[i] * sigmoid(z[i]) : gy[i];
            }
            {
                const int at = 4 * ((row >> 1) * 16 + l) + 2 * (row & 1);
                float *const to0 = &mine[0][0].x + at, *const to1 = &mine[1][0].x + at, *const to2 = &mine[2][0].x + at;
#pragma unroll
                for (int i = 0; i < kQ; ++i) {
                    to0[i] = d[i];
                    to1[i] = d[i] * u[i];
                    to2[i] = dr[i];
                }
            }
            __builtin_amdgcn_wave_barrier();
            float dd[kJT], bu[kJT], rr[kJT], sr[kJT], sb[kJT], sk[kJT], sum = 0.f;
            get8(mine[0] + l, 16, dd);
            get8(mine[1] + l, 16, bu);
            get8(mine[2] + l, 16, rr);
#pragma unroll
            for (int i = 0; i < kJT; ++i) {
                sum += dd[i];
                sr[i] = sb[i] = sk[i] = 0.f;
            }
            const float4 cy4 = carry[wave][c][row];
            const float cy[4] = {cy4.x, cy4.y, cy4.z, cy4.w};
            float out[4] = {0.f, 0.f, 0.f, 0.f}, sA[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (!WHOLE && q >= rounds) break;
                const float A2 = A[q] * kLog2e, P = factor<true>(sum * A2);
                float Bv[kJT], Cv[kJT], a[kJT], ax[kJT];
                get8(BC[0][4 * row + q] + l, 16, Bv);
                const float in = l == 0 ? xs[q] : 0.f;
                float Q = in;
#pragma unroll
                for (int i = 0; i < kJT; ++i) {
                    a[i] = exp2_(dd[i] * A2);
                    ax[i] = bu[i] * Bv[i];
                    Q = fmaf(a[i], Q, ax[i]);
                }
                scan_states<16, true>(P, Q);
                float x = dpp0<0x111>(Q) + in;
                get8(BC[1][4 * row + q] + l, 16, Cv);
#pragma unroll
                for (int i = 0; i < kJT; ++i) {
                    const float w = ax[i];
                    ax[i] = a[i] * x;
                    x = ax[i] + w;
                    sr[i] = fmaf(Cv[i], x, sr[i]);
                    aC[q][i] = fmaf(rr[i], x, aC[q][i]);
                    Cv[i] *= rr[i];
                }
                // g_t = C_t dr_t + a_{t+1} g_{t+1}, and a g of a lane's first
                // step goes to the lane before
                const float back = l == 15 ? cy[q] : 0.f;
                float gx = Cv[kJT - 1] + back;
#pragma unroll
                for (int i = kJT - 2; i >= 0; --i) gx = fmaf(a[i + 1], gx, Cv[i]);
                Q = a[0] * gx;
                scan_back(P, Q);
                out[q] = Q;  // what lane 0 hands to the piece before
                gx = Cv[kJT - 1] + (dpp0<0x101>(Q) + back);
#pragma unroll
                for (int i = kJT - 1; i >= 0; --i) {
                    const float w = gx * ax[i];
                    aB[q][i] = fmaf(gx, bu[i], aB[q][i]);
                    sb[i] = fmaf(gx, Bv[i], sb[i]);
                    sk[i] = fmaf(w, A[q], sk[i]);
                    sA[q] = fmaf(w, dd[i], sA[q]);
                    if (i > 0) gx = fmaf(a[i], gx, Cv[i - 1]);
                }
                // one round's registers at a time
                hold(aC[q]);
                hold(aB[q]);
                hold(sr);
                hold(sb);
                hold(sk);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) sA[q] = row_sum(sA[q]);
            if (l == 0) {
                carry[wave][c][row] = make_float4(out[0], out[1], out[2], out[3]);
                float4 t = sumA[wave][c][row];
                t.x += sA[0], t.y += sA[1], t.z += sA[2], t.w += sA[3];
                sumA[wave][c][row] = t;
            }
            float s3[3][kQ], o[3][kQ], sD = 0.f, sp = 0.f;
            sum_rows(sr, s3[0]);
            sum_rows(sb, s3[1]);
            sum_rows(sk, s3[2]);
            if constexpr (!WHOLE) {
                if (ws.acc && keep > 0) {
                    auto *const acc = (Pack<float, 3 * kQ> *)ws.acc + ((b * k.H + h) * ((N + 1) / kQ) + (ch * kSelChunk + tq) / kQ);
                    Pack<float, 3 * kQ> t{};
                    if (n0 > 0) t = *acc;
#pragma unroll
                    for (int i = 0; i < 3 * kQ; ++i) t.v[i] = s3[i / kQ][i % kQ] += t.v[i];
                    if (!last_block) *acc = t;
                }
            }
            if (WHOLE || last_block) {
#pragma unroll
                for (int i = 0; i < kQ; ++i) {
                    const float raw = fmaf(Dh, u[i], s3[0][i]);
                    o[0][i] = fmaf(d[i], s3[1][i], Dh * dr[i]);
                    o[1][i] = fmaf(u[i], s3[1][i], s3[2][i]);
                    if (k.softplus) o[1][i] *= sigmoid(p[i]);
                    if (k.z) {
                        const float sg = sigmoid(z[i]);
                        o[2][i] = gy[i] * raw * sg * (1.f + z[i] * (1.f - sg));
                    }
                    if (i >= valid) o[0][i] = o[1][i] = o[2][i] = 0.f;
                    sD = fmaf(dr[i], u[i], sD);
                    sp += o[1][i];
                }
                st_row<IO, kQ>(du + o0 + tq, o[0], keep);
                st_row<IO, kQ>(ddt + o0 + tq, o[1], keep);
                if (dz) st_row<IO, kQ>(dz + o0 + tq, o[2], keep);
                sD = wave_sum_last(sD);
                sp = wave_sum_last(sp);
                if (lane == 63) {
                    sumDb[wave][c][0] += sD;
                    sumDb[wave][c][1] += sp;
                }
            }
        }
        // dB, dC of the piece: the waves' sums, in order, two rounds at a time;
        // thread t joins steps 8 (t % 16) .. of matrix t / 256, DPP row
        // (t / 16) % 4 of round (t / 128) % 2 ... as values v of a lane
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (!WHOLE && q >= rounds) break;
            float4(*const buf)[4][64] = (float4(*)[4][64])lds;  // [wave][quarter of the 16 values][lane]
            buf[wave][0][lane] = make_float4(aB[q][0], aB[q][1], aB[q][2], aB[q][3]);
            buf[wave][1][lane] = make_float4(aB[q][4], aB[q][5], aB[q][6], aB[q][7]);
            buf[wave][2][lane] = make_float4(aC[q][0], aC[q][1], aC[q][2], aC[q][3]);
            buf[wave][3][lane] = make_float4(aC[q][4], aC[q][5], aC[q][6], aC[q][7]);
            __syncthreads();
            // thread: quarter v, lane ll of the waves' values
            const int half = tid & 1, ll = (tid >> 1) & 63, v = tid >> 7;
            float2 s = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float *x = &buf[w][v][ll].x + 2 * half;
                s.x += x[0];
                s.y += x[1];
            }
            const int n = (WHOLE ? 0 : n0) + (WHOLE ? 4 : rounds) * (ll >> 4) + q;
            const int t = (ll & 15) * kJT + (v & 1) * 4 + half * 2;
            if (WHOLE || n < S) {
                float *o = (v < 2 ? ws.dB : ws.dC) + ((((int64_t)set * k.B + b) * k.G + g) * S + n) * N + ch * kSelChunk + t;
                if (t < steps(ch, N)) o[0] = s.x;
                if (t + 1 < steps(ch, N)) o[1] = s.y;
            }
            __syncthreads();
        }
    }
    for (int c = 0; c < nch; ++c) {
        const int64_t r = r0 + kWaves * c, o = r * S + m0;
        if (l < rounds && (WHOLE || m0 + l < S)) {
            ws.dA[o + l] = (&sumA[wave][c][row].x)[l];
            if (dx_in) dx_in[o + l] = (&carry[wave][c][row].x)[l];
        }
        if ((WHOLE || last_block) && lane < 2) ws.dDb[r * 2 + lane] = sumDb[wave][c][lane];
    }
}

// What the blocks of k_sel_bwd left apart, joined in order.  Blocks y = 0 and 1:
// dB and dC, the sets' sums, M = B*G*S*N values each; bound by reading the
// partial sums, eight loads of a thread at a time (11.5 us for 67 MB at 4 x 2560
// x 2048 with 16 modes and 64 sets; one load at a time took 33).  y = 2: dA, dD,
// ddt_bias, sums over the batch.
template <int IO>
__global__ __launch_bounds__(256) void k_sel_join(const SelBwdWs ws, typename io_elem<IO>::T *__restrict__ dB,
                                                  typename io_elem<IO>::T *__restrict__ dC, float *__restrict__ dA,
                                                  float *__restrict__ dD, float *__restrict__ ddt_bias, int64_t M,
                                                  int64_t B, int64_t H, int S) {
    const int64_t i = block_id() * 256 + threadIdx.x, HS = H * S;
    if (blockIdx.y < 2) {
        if (i >= M) return;
        const float *const p = (blockIdx.y ? ws.dC : ws.dB) + i;
        float sum = 0.f;
#pragma unroll 8
        for (int s = 0; s < ws.sets; ++s) sum += p[s * M];
        (blockIdx.y ? dC : dB)[i] = from_f<IO>(sum);
    } else if (i < HS) {
        float s = 0.f;
#pragma unroll 4
        for (int64_t b = 0; b < B; ++b) s += ws.dA[b * HS + i];
        dA[i] = s;
    } else if (i < HS + H) {
        const int64_t h = i - HS;
        float s = 0.f, t = 0.f;
#pragma unroll 4
        for (int64_t b = 0; b < B; ++b) {
            s += ws.dDb[(b * H + h) * 2];
            t += ws.dDb[(b * H + h) * 2 + 1];
        }
        if (dD) dD[h] = s;
        if (ddt_bias) ddt_bias[h] = t;
    }
}

// -------------------------------------------------------------- single token

// LPC lanes per channel, four modes each (a channel's states are read as whole
// lines).  Bound by the launch and a chain of about eight trips to memory: the
// slot; u, dt and bias; a lane's four modes one after another (the pools may be
// one, so the load of a state stands behind the store of the one before it); D;
// z.  6.5 us for 64 x 768 with 16 modes (6.7 MB, 1.3 us at a copy's rate).  A
// slot outside the pool leaves its row's output zero and no state changed.
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
    const int64_t h = block_id() * (256 / lpc) + threadIdx.x / lpc, b = blockIdx.y;
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

// Sets of channels per group.  A compute unit holds one block of eight waves:
// 256 blocks fill the chip, more channels per block mean fewer partial sums of
// dB and dC (written and read once per set).
void bwd_sets(int64_t B, int64_t H, int64_t G, int *sets, int *per) {
    const int64_t Hg = H / G, want = B > 0 ? (256 + B * G - 1) / (B * G) : 1;
    int64_t p = (Hg + want - 1) / want;
    p = (p + kWaves - 1) / kWaves * kWaves;
    if (p > kWaves * kPerWave) p = kWaves * kPerWave;
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
    w->acc = take(S > kModes ? (size_t)(B * H * ((N + 1) / kQ)) * (12 * kQ) : 0);
    return at;
}

int64_t chunks(int64_t N) { return (N + kSelChunk - 1) / kSelChunk; }

// Which lanes and waves take a row (scan_io says when).
template <int IO, int LPR, Share SH>
hipError_t scan_lanes(const SelArgs &a, void *y, float *x_out, float *saved, hipStream_t s) {
    using T = typename io_elem<IO>::T;
    constexpr int rows = (SH == kOwnRows ? 4 : 1) * 64 / LPR;
    return launch(k_sel_scan<IO, LPR, SH>, grid_of((a.B * a.H + rows - 1) / rows), dim3(256), 0, s,
                  pack_args<IO>(a), (T *)y, x_out, saved, chunks(a.N));
}

template <int IO>
hipError_t scan_io(const SelArgs &a, void *y, float *x_out, float *saved, hipStream_t s) {
    // Measured in fp16 with 16 modes and a gate, us, at (rows x steps):
    //                    288x301  288x4096  1024x2048  1024x4096  2048x250  4096x250  4096x4096
    //   own rows            12.1      35.4       19.3       36.7      11.3      11.5       95.4
    //   time                           17.7       31.3       30.3                          102.1
    //   modes                8.4      21.1       19.8       37.8       8.2      14.2      128.5
    // A quarter of the time is won where four pieces at once leave no wave idle
    // and the rows alone are too few to fill the chip; a quarter of the modes
    // where there is but one wave or two per compute unit.
    const int64_t rows = a.B * a.H, pieces = (a.N + 64 * kIT - 1) / (64 * kIT);
    const bool rows16 = a.N <= 16 * kIT;  // lanes per row: 16, else 64
    if (rows <= 2048 && pieces > 3 * ((pieces + 3) / 4)) return scan_lanes<IO, 64, kTime>(a, y, x_out, saved, s);
    if (rows <= (rows16 ? 2048 : 512) && a.S >= 4)
        return rows16 ? scan_lanes<IO, 16, kModeMod4>(a, y, x_out, saved, s)
                      : scan_lanes<IO, 64, kModeMod4>(a, y, x_out, saved, s);
    return rows16 ? scan_lanes<IO, 16, kOwnRows>(a, y, x_out, saved, s)
                  : scan_lanes<IO, 64, kOwnRows>(a, y, x_out, saved, s);
}

template <int IO>
hipError_t bwd_io(const SelArgs &a, const float *saved, const void *dy, const float *dx_out, const SelGrads &g,
                  char *ws, hipStream_t s) {
    using T = typename io_elem<IO>::T;
    SelBwdWs w;
    bwd_layout(a.B, a.H, a.N, a.S, a.G, ws, &w);
    const dim3 grid = grid_of(a.B * a.G * w.sets);
    // (float4 loads of decay rates: A may start at any element)
    const bool whole = a.S == kModes && ((uintptr_t)a.A & 15) == 0;
    for (int n0 = 0; n0 < a.S && a.B > 0; n0 += kModes) {
        const hipError_t e =
            launch(whole ? k_sel_bwd<IO, true> : k_sel_bwd<IO, false>, grid, dim3(kWaves * 64), 0, s, pack_args<IO>(a),
                   saved, (const T *)dy, dx_out, (T *)g.du, (T *)g.ddt, (T *)g.dz, g.dx_in, w, chunks(a.N), n0,
                   n0 + kModes >= a.S ? 1 : 0);
        if (e != hipSuccess) return e;
    }
    const int64_t M = a.B * a.G * a.S * a.N, P = a.H * (a.S + 1);
    return launch(k_sel_join<IO>, grid_of(((M > P ? M : P) + 255) / 256, 3), dim3(256), 0, s, w, (T *)g.dB,
                  (T *)g.dC, g.dA, g.dD, g.ddt_bias, M, a.B, a.H, a.S);
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
    return launch(k_sel_step<IO>, grid_of((H * lpc + 255) / 256, (unsigned)B), dim3(256), 0, s, (const T *)u,
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
