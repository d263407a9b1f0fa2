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
//
// Steps are taken in chunks of 64 (fp32: 32), with L the decays' exponents summed
// from the chunk's first step on:
//   o_t = out (e^{L_t} X_in^T a_t + sum_{j<=t} e^{L_t - L_j} (a_t.b_j) upd c_j)
//   X_out = e^{L_end} X_in + sum_j (e^{L_end - L_j} upd b_j) c_j^T
// which are four matrix products.  What is multiplied is either as it was given
// or held in pieces that come to 22 bits or more (the matrix cores' 16-bit types
// would round weights and states to 8 or 11), sums and states are fp32, exponents
// 64 bits.  A wave has 16 of the state's columns, in its accumulators from the
// first chunk to the last; a block's waves share the tiles of a and b and the
// chunk's weights in LDS.  A row is cut into segments where sequences times heads
// do not fill the chip: STATES finds what each segment adds to a state, the
// segments are joined, and the last launch goes through each from the state that
// enters it.
//
// What bounds it: neither memory (64K steps of 8 heads of 128 in bf16 read and
// write 539 MB, 105 us at a copy's rate, and take 255 to 280) nor the matrix cores
// (a quarter busy), but the chain of a chunk: scan, weights, products, update, with a
// barrier or two between.  One block of eight waves per CU is all that 220
// registers a lane allow (two at 128 registers spill 30 to 77 and are no faster:
// 76 us against 75 forward, with two pieces, and 314 against 286 backward; two of
// four waves and half the columns have not been measured); a sixth to a quarter of
// the time goes by without loads, a tenth without the exponents, none without the
// stores or with the weights formed elsewhere.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "lm_device.h"
#include "lm_internal.h"

namespace h3c {
namespace {

// A factor e^g of g below this is zero in fp32, and so is what follows from it.  (A g that is NaN is below neither.)
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
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef int i2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) s4 lds_s4;

// What a type's products need.  An operand fragment is 8 values of k per lane,
// of the row (column) lane & 15; which of 32 they are is up to both operands alike.
template <int IO>
struct Mx {  // 16-bit elements
    static constexpr int C = 64;                       // steps of a chunk: more need more weights, fewer more updates
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

// A tile of steps in LDS, rows of COLS elements and PAD bytes.  With 32 bytes of padding the reads across 8 rows, of 8
// bytes per lane, meet every bank once.  A tile that is only read along its rows (TURNED, 16-bit) has the halves of its
// units where a fragment wants them side by side, so that this is a read of 16 bytes, for which 16 bytes of padding do
// the same.  Every address is one of the lane plus a constant.
template <int IO, int COLS, int PAD, bool TURNED>
struct Lds {
    using T = typename io_elem<IO>::T;
    static constexpr int E = 16 / (int)sizeof(T), CH = COLS / E, ROWS = Mx<IO>::C, STRIDE = CH * 16 + PAD, kBytes = ROWS * STRIDE;
    using Frag = typename Mx<IO>::Frag;
    __device__ __forceinline__ static int at(int row, int chunk) { return row * STRIDE + chunk * 16; }
    // the unit `chunk` of a row to its place
    __device__ __forceinline__ static void keep(char *p, int row, int chunk, u4 v) {
        if constexpr (TURNED) {  // elements 8 q + 4 h of 32: group 2 q + h (mod 4), its first half below 16
            char *to = p + at(row, (chunk & ~3) + 2 * (chunk & 1)) + 8 * ((chunk >> 1) & 1);
            *(u2 *)to = u2{v.x, v.y};
            *(u2 *)(to + 16) = u2{v.z, v.w};
        } else {
            *(u4 *)(p + at(row, chunk)) = v;
        }
    }
    // 32 elements of k of a row per lane & 15: k + 4 g + j and k + 16 + 4 g + j, the order in which accumulators hold rows
    __device__ __forceinline__ static Frag along(const char *p, int row, int k) {
        constexpr int B = (int)sizeof(T);
        const int i = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
        const char *mine = p + at(i, 0) + 4 * g * B + at(row, 0) + k * B;
        Frag f;
        if constexpr (TURNED) {
            f.v = *(const u4 *)(mine + 4 * g * B);
        } else if constexpr (IO != IO_F32) {
            const u2 a = *(const u2 *)mine, b = *(const u2 *)(mine + 16 * B);
            f.v = u4{a.x, a.y, b.x, b.y};
        } else {
            const f4 a = *(const f4 *)mine, b = *(const f4 *)(mine + 16 * B);
#pragma unroll
            for (int j = 0; j < 4; ++j) f.v[j] = a[j], f.v[4 + j] = b[j];
        }
        return f;
    }
    // the column col + lane & 15, the steps 4 g + j and 16 + 4 g + j from `row` on
    __device__ __forceinline__ static Frag across(const char *p, int row, int col) {
        const int i = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
        Frag f;
        if constexpr (IO != IO_F32) {
            const char *mine = p + at(4 * g + (i >> 2), 0) + 8 * (i & 3);
            i2 h[2];
#pragma unroll
            for (int q = 0; q < 2; ++q)
                h[q] = __builtin_bit_cast(i2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(mine + at(row + 16 * q, 0) + col * 2)));
            f.v = u4{(uint32_t)h[0].x, (uint32_t)h[0].y, (uint32_t)h[1].x, (uint32_t)h[1].y};
        } else {
            const char *mine = p + at(4 * g, 0) + i * 4;
#pragma unroll
            for (int j = 0; j < 8; ++j) f.v[j] = *(const float *)(mine + at(row + 16 * (j >> 2) + (j & 3), 0) + col * 4);
        }
        return f;
    }
};

__device__ __forceinline__ float lanes_max(float v, int from) {
    for (int d = from; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}
// The power of two that brings a largest magnitude m to 2^13 .. 2^14 (two pieces then hold a number to 22 bits, or to
// 2^-25, which is 2^-39 of the largest), as an exponent (fp32's largest takes 2^-114; from
// 2^-86 down less than 2^14 is reached, and what the pieces lose is below 2^-125).
__device__ __forceinline__ int near_2_14(float m) {
    const int e = 14 - __builtin_amdgcn_frexp_expf(m);
    return e > 100 ? 100 : e;
}
__device__ __forceinline__ float pow2(int e) { return __builtin_amdgcn_ldexpf(1.f, e); }
// Sum over the lanes up to this one, in 64 bits: within 16 lanes and then across them by DPP.
template <int CTRL, int ROWS>
__device__ __forceinline__ double add_from(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
    return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double sum_up_to(double v) {
    v = add_from<0x111, 0xf>(v);  // one lane before, two, four, eight
    v = add_from<0x112, 0xf>(v);
    v = add_from<0x114, 0xf>(v);
    v = add_from<0x118, 0xf>(v);
    v = add_from<0x142, 0xa>(v);  // the sixteenth's of rows 0 and 2 to rows 1 and 3
    return add_from<0x143, 0xc>(v);  // the thirty-second's to rows 2 and 3
}
__device__ __forceinline__ double lane_of(double v, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane), hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// 2^x of a 64-bit exponent, to 32 bits
__device__ __forceinline__ float exp2_of(double x) {
    const float d = (float)x;
    return __builtin_amdgcn_exp2f(d) * fmaf((float)(x - (double)d), kLn2, 1.f);
}

enum { STATES, FORWARD, BACKWARD };  // what a launch of chunks is for

// Segments whose states each block joins for itself: that reads a state per segment before it, and saves a launch (eight
// prompts of 1024 steps: 31.5 us, with the launch 35.7).
constexpr int64_t kFew = 8;

// The decay over a segment, 2^up (hi + lo).  A segment is longer than the 64 steps whose factor has to be within fp32, so
// its own may be far outside (e^96 over 128 steps of +0.75) while the states at both its ends are not.  Past 2^96 either
// way hi is 1 to 2, so that a state times 2^up is within fp32 where what it comes to is.
struct Factor {
    float hi, lo;
    int up, unused;
};
__device__ __forceinline__ Factor factor_of(double e) {  // 2^e
    double up = 0.0;
    if (!(fabs(e) <= 96.0)) up = fmin(fmax(floor(e), -512.0), 512.0);  // (2^512 of any state but zero is infinite, 2^-512 zero)
    const double f = exp2(e - up);
    const float hi = (float)f;
    return {hi, (float)(f - (double)hi), (int)up, 0};
}
// (without a choice: one for each number keeps the loads apart, 51 us instead of 33 for eight prompts of 1024 steps)
__device__ __forceinline__ float carried(float x, const Factor &f, float add) {
    x = __builtin_amdgcn_ldexpf(x, f.up);
    return fmaf(x, f.hi, fmaf(x, f.lo, add));
}

// Where the segments of the rows meet.
struct Segs {
    int64_t len, n;      // steps of one, number
    float *state;        // [role][seg][B*H][K*M]: what a segment adds, then the state that enters it
    Factor *factor;      // [role][seg][B*H]: the decay over it
    int64_t plane;       // K*M
};

// Waves of a SIMD that the registers are to leave room for: as many as the LDS does (heads of more than 128 take what
// they need, and more than there is: 68 to 159 registers are spilled where blocks have eight waves).
constexpr int waves_per_simd(int io, int KP, int WV, int what, bool whole_heads) {
    return KP > 128 && WV == 4                                           ? 1
           : io == IO_F32 || KP > 64 || !whole_heads || WV == 8          ? 2
           : KP == 32 && !(io == IO_BF16 && what != STATES)              ? 4
                                                                         : 3;
}

// (a lambda left as a call would keep all that it captures in memory)
#define INLINE __attribute__((always_inline))

template <int IO, int KP, int WV, int DO, bool WHOLE>
__global__ __launch_bounds__(WV * 64, waves_per_simd(IO, KP, WV, DO, WHOLE)) void k_lin_chunk(Roles roles, Shape s, Segs sg, int tiles) {
    using T = typename io_elem<IO>::T;
    using X = Mx<IO>;
    using Frag = typename X::Frag;
    constexpr bool OUT = DO != STATES;
    constexpr int C = X::C, TH = WV * 64, MB = WV * 16, KS = KP / 32, NT = C / 16, NU = C / 32;
    using LA = Lds<IO, KP, 16, IO != IO_F32>;
    using LK = Lds<IO, KP, 32, false>;
    using LM = Lds<IO, MB, 32, false>;
    constexpr int E = LK::E;
    constexpr int NA = C * LK::CH / TH, NC = C * LM::CH / TH;  // units of 16 bytes per thread
    static_assert(C * LK::CH % TH == 0 && C * LM::CH % TH == 0 && NT <= 4, "whole units, a wave per 16 steps");
    // pieces of weights and states in the output's products: 22 bits in fp16, 24 in bf16 (two pieces, 17 bits, would take 91
    // us forward down to 85 for 4 x 2048 steps of 20 heads of 128); fragments of weights
    constexpr int NP = X::UPD, WF = NT == 4 ? 6 : 2;
    // Two places for tiles where the LDS has room for them without giving up a block: a chunk's are then written while
    // the last one's are still read.
    constexpr int TWO = OUT && WV == 8 && KP <= 128 ? 2 : 1;
    __shared__ __attribute__((aligned(16))) char tile_a[OUT ? TWO * LA::kBytes : 16], tile_b[TWO * LK::kBytes], tile_c[TWO * LM::kBytes];
    __shared__ __attribute__((aligned(16))) float decays[2][4 * C + 4];  // of a chunk [hi, lo, into, upd][C] and its factor
    __shared__ Frag weights[OUT ? WF * NP * 64 : 1];                     // [fragment][piece][lane]
    __shared__ float owns[OUT ? C : 1], downs[OUT ? NU * C : 1];         // a step's weight of itself, what its weights of 32 steps were scaled by
    __shared__ float dots[OUT ? WV * C : 1];                             // [wave][C]
    // (read once: the compiler keeps a struct of a launch's arguments that varies by block in memory)
    const Role *role = &roles.r[blockIdx.y];
    const float out = role->out, upd = role->upd;
    const int rs = role->rs, cs = role->cs, wide = role->wide;
    float *const dot_to = role->dot, *const s1 = role->s1;
    const float *const s0 = role->s0;
    void *const o = role->o;
    const int K = role->a.dim, M = role->c.dim;
    int64_t id = block_id();
    const int tile = (int)(id % tiles);
    id /= tiles;
    const int64_t BH = s.B * s.H, bh = id % BH, seg = id / BH;
    if (seg >= (OUT ? sg.n : sg.n - 1) || tile * MB >= M) return;
    const int64_t b = bh / s.H;
    const int h = (int)(bh - b * s.H), n = (int)row_len(s.lengths, b, s.N);
    const int i_lo = (int)(seg * sg.len), i_hi = (int)std::min<int64_t>(n, seg * sg.len + sg.len);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), li = lane & 15, lg = lane >> 4;
    const int col0 = tile * MB + wave * 16;  // the wave's columns
    constexpr int EW = WV > NT ? WV - 1 : 0;  // the wave of the decays' exponents, one with few weights to form
    const bool dot = DO == BACKWARD && dot_to, back = role->reverse;
    // A chunk takes steps i0 .. i0 + cnt - 1 in the order of the recurrence, which lie in memory from `low` on, in
    // this order or the other: step i0 + j at low + at(j).  What lies past them is taken to be the last.
    const auto low = [&](int i0, int cnt) INLINE { return b * s.N + (back ? n - i0 - cnt : i0); };
    const auto at = [&](int j, int cnt) INLINE { return back ? cnt - 1 - std::min(j, cnt - 1) : std::min(j, cnt - 1); };
    const auto count = [&](int i0) INLINE { return std::min(C, i_hi - i0); };
    const auto base = [&](const Seq &q) INLINE { return (const T *)q.p + h / q.share * q.dim; };
    const T *pa = OUT ? base(role->a) : nullptr, *pb = base(role->b), *pc = base(role->c), *pe = dot ? base(role->e) : nullptr;
    const int lda = (int)role->a.ld, ldb = (int)role->b.ld, ldc = (int)role->c.ld, lde = (int)role->e.ld, ldo = (int)s.H * M;

    f4 st[2 * KS];  // the state: rows 16 m + 4 g + j of tile m, column lane & 15
    const int64_t slot = ((int64_t)blockIdx.y * sg.n + seg) * BH + bh;
    const bool few = sg.n <= kFew;  // (segments: their states are joined here, else by k_lin_enter)
    const float *enter = !OUT ? nullptr : sg.n == 1 || few ? (s0 ? s0 + bh * K * M : nullptr) : sg.state + slot * sg.plane;
    const auto state_at = [&](int m, int j) INLINE { return std::min(16 * m + 4 * lg + j, K - 1) * rs + std::min(col0 + li, M - 1) * cs; };
#pragma unroll
    for (int m = 0; m < 2 * KS; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) st[m][j] = enter ? enter[state_at(m, j)] : 0.f;
    if (OUT && few)
        for (int64_t q = 0; q < seg; ++q) {
            const int64_t at_q = ((int64_t)blockIdx.y * sg.n + q) * BH + bh;
            const Factor f = sg.factor[at_q];
            const float *add = sg.state + at_q * sg.plane;
#pragma unroll
            for (int m = 0; m < 2 * KS; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j) st[m][j] = carried(st[m][j], f, add[state_at(m, j)]);
        }
#pragma unroll
    for (int m = 0; m < 2 * KS; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (16 * m + 4 * lg + j >= K || col0 + li >= M) st[m][j] = 0.f;

    // the next chunk's units, on their way
    u4 ga[OUT ? NA : 1], gb[NA], gc[NC];
    float gg = 0.f;
    // WHOLE: heads are whole units at whole dwords, and tiles go through buffer resources that end with the chunk's
    // last row: what is past the rows (or, by its offset, past the head) loads as zero and is not stored.  Else
    // every element is loaded by itself, from a place in bounds.
    const auto window = [&](const void *p, int ld, int dim, int cnt, int e) INLINE {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, ((cnt - 1) * ld + dim) * e, 0x00020000);
    };
    // a row's offset: a part of the lane, and one of the rows before it
    const auto lane_at = [&](int row, int ld, int c, int dim, int e) INLINE {
        return c < dim ? (back ? -row : row) * ld * e + c * e : (int)0x80000000;
    };
    const auto rows_at = [&](int row, int ld, int cnt, int e) INLINE { return (back ? cnt - 1 - row : row) * ld * e; };
    const auto element = [&](const T *p, int ld, int j, int cnt, int c, int dim) INLINE {
        u4 u = {0, 0, 0, 0};
        const uint32_t row = (uint32_t)at(j, cnt) * (uint32_t)ld;
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const T v = p[row + std::min(c + k, dim - 1)];
            const bool in = j < cnt && c + k < dim;
            if constexpr (E == 4) u[k] = in ? __float_as_uint(v) : 0;
            else u[k >> 1] |= (in ? (uint32_t)__builtin_bit_cast(uint16_t, v) : 0u) << (16 * (k & 1));
        }
        return u;
    };
    constexpr int RA = TH / LK::CH, RC = TH / LM::CH, EB = (int)sizeof(T);
    const int ra = tid / LK::CH, ca = tid % LK::CH * E, rc = tid / LM::CH, cc = tile * MB + tid % LM::CH * E;
    const int va = lane_at(ra, lda, ca, K, EB), vb = lane_at(ra, ldb, ca, K, EB), vc = lane_at(rc, ldc, cc, M, EB);
    const auto load = [&](int i0) INLINE {
        const int cnt = count(i0);
        const int64_t l = low(i0, cnt);
        const T *qa = OUT ? pa + l * lda : nullptr, *qb = pb + l * ldb, *qc = pc + l * ldc;
        if constexpr (WHOLE) {
            const __amdgpu_buffer_rsrc_t wb = window(qb, ldb, K, cnt, EB), wc = window(qc, ldc, M, cnt, EB);
#pragma unroll
            for (int q = 0; q < NA; ++q)
                gb[q] = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(wb, vb + rows_at(q * RA, ldb, cnt, EB), 0, 0));
#pragma unroll
            for (int q = 0; q < NC; ++q)
                gc[q] = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(wc, vc + rows_at(q * RC, ldc, cnt, EB), 0, 0));
            if constexpr (OUT) {
                const __amdgpu_buffer_rsrc_t wa = window(qa, lda, K, cnt, EB);
#pragma unroll
                for (int q = 0; q < NA; ++q)
                    ga[q] = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(wa, va + rows_at(q * RA, lda, cnt, EB), 0, 0));
            }
        } else {
#pragma unroll
            for (int q = 0; q < NA; ++q) {
                if constexpr (OUT) ga[q] = element(qa, lda, ra + q * RA, cnt, ca, K);
                gb[q] = element(qb, ldb, ra + q * RA, cnt, ca, K);
            }
#pragma unroll
            for (int q = 0; q < NC; ++q) gc[q] = element(qc, ldc, rc + q * RC, cnt, cc, M);
        }
    };
    const auto decay = [&](int i0) INLINE {
        float g = 0.f;
        const int cnt = i0 < i_hi ? count(i0) : 0;
        if (lane < cnt) g = s.per_token ? s.g[(low(i0, cnt) + at(lane, cnt)) * s.H + h] : s.g[h];
        return g;
    };
    double all = 0.0;  // (of wave EW) the segment's decay, as an exponent of two
    const auto keep = [&](char *la, char *lb, char *lc) INLINE {
#pragma unroll
        for (int q = 0; q < NA; ++q) {
            const int u = q * TH + tid;
            if constexpr (OUT) LA::keep(la, u / LK::CH, u % LK::CH, ga[q]);
            LK::keep(lb, u / LK::CH, u % LK::CH, gb[q]);
        }
#pragma unroll
        for (int q = 0; q < NC; ++q) {
            const int u = q * TH + tid;
            LM::keep(lc, u / LM::CH, u % LM::CH, gc[q]);
        }
    };
    // (wave EW) Exponents of two from the chunk's start on, in 64 bits: with the step's own decay where time runs
    // on, without it where it runs back.  The state is multiplied by the chunk's factor in 32 bits, and what that loses
    // is given to the next chunk's: the product of all stays within one rounding of what it should be.
    double lost = 1.0;
    const auto exponents = [&](float *dec, float g) INLINE {
        const double own = (double)(g < kLeast ? kLeast : g) * 1.4426950408889634;
        const double sum = sum_up_to(own), total = lane_of(sum, C - 1), e = back ? sum - own : sum;
        all += total;
        if (lane < C) {
            const float hi = (float)e;
            dec[lane] = hi;
            dec[C + lane] = (float)(e - (double)hi);
            dec[2 * C + lane] = exp2_of(e);
            dec[3 * C + lane] = exp2_of(total - e) * upd;
        }
        const double f = exp2(total) * lost;
        const float f1 = (float)f;
        lost = f1 > 1e-30f ? 1.0 + (double)((float)(f - (double)f1) * __builtin_amdgcn_rcpf(f1)) : 1.0;
        if (lane == 0) dec[4 * C] = f1;
    };

    // the dot products of the chunk of i0
    const auto put_dots = [&](int i0) INLINE {
        const int cnt = count(i0);
        if (tid >= cnt) return;
        float e = dots[tid];
#pragma unroll
        for (int q = 1; q < WV; ++q) e += dots[q * C + tid];
        dot_to[(tile * BH + bh) * s.N + (low(i0, cnt) - b * s.N) + at(tid, cnt)] = e;
    };

    int turn = 0;
    if (i_lo < i_hi) {
        load(i_lo);
        if (wave == EW) {
            exponents(decays[0], decay(i_lo));
            gg = decay(i_lo + C);
        }
    }
    for (int i0 = i_lo; i0 < i_hi; i0 += C, turn ^= 1) {
        const float *dec = decays[turn];
        const int place = TWO == 2 ? turn : 0;
        char *la = tile_a + place * LA::kBytes, *lb = tile_b + place * LK::kBytes, *lc = tile_c + place * LM::kBytes;
        const int cnt = count(i0);
        const int64_t row0 = low(i0, cnt);
        if constexpr (TWO == 1) __syncthreads();  // (the last chunk has been read)
        keep(la, lb, lc);
        __syncthreads();
        if (dot && i0 > i_lo) put_dots(i0 - C);
        // what the outputs are multiplied by for the decays' gradients, on its way before the next chunk's tiles
        u4 ge[DO == BACKWARD ? NT : 1];
        if constexpr (DO == BACKWARD)
            if (dot) {
                const int c = col0 + 4 * lg;
                const T *qe = pe + row0 * lde;
                const __amdgpu_buffer_rsrc_t we = window(qe, lde, M, cnt, EB);
                const int ve = lane_at(li, lde, c, M, EB);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if constexpr (!WHOLE) {
                        float z[4];
                        ld_row<IO, 4>(qe + ((uint32_t)at(16 * t + li, cnt) * (uint32_t)lde + c), z, M - c);
#pragma unroll
                        for (int j = 0; j < 4; ++j) ge[t][j] = __float_as_uint(z[j]);
                    } else if constexpr (IO == IO_F32) {
                        ge[t] = __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(we, ve + rows_at(16 * t, lde, cnt, EB), 0, 0));
                    } else {
                        const u2 v = __builtin_bit_cast(u2, __builtin_amdgcn_raw_buffer_load_b64(we, ve + rows_at(16 * t, lde, cnt, EB), 0, 0));
                        ge[t] = u4{v.x, v.y, 0, 0};
                    }
                }
            }
        if (i0 + C < i_hi) load(i0 + C);
        if constexpr (OUT) {
            // the chunk's weights, once for all columns: of 16 steps t and 32 steps u by a wave (or of all u, where waves are
            // few), transposed, as they are operands
            constexpr int SPLIT = WV == 8 ? NU : 1;
            if (wave < NT * SPLIT && 2 * (wave % SPLIT) <= wave / SPLIT) {
                const int t = wave / SPLIT;
                Frag a[KS];
#pragma unroll
                for (int p = 0; p < KS; ++p) a[p] = LA::along(la, 16 * t, 32 * p);
                const float hi = dec[16 * t + li], lo = dec[C + 16 * t + li];
#pragma unroll
                for (int v = 0; v < NU / SPLIT; ++v) {
                    const int u = SPLIT > 1 ? wave % SPLIT : v;
                    if (2 * u > t) continue;
                    float x[8], m = 0.f, own = 0.f;  // of steps 32 u + 16 q + 4 g + j
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[4 * q + j] = 0.f;
                        if (2 * u + q > t) continue;
                        f4 d = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int p = 0; p < KS; ++p) d = X::mul(LK::along(lb, 32 * u + 16 * q, 32 * p), a[p], d);
                        const float *from = dec + 32 * u + 16 * q + 4 * lg;
                        const f4 h2 = *(const f4 *)from, l2 = *(const f4 *)(from + C);
                        const bool edge = 2 * u + q == t;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float w = d[j] * (out * upd) * __builtin_amdgcn_exp2f((hi - h2[j]) + (lo - l2[j]));
                            const bool self = edge && 4 * lg + j == li;
                            x[4 * q + j] = (edge && 4 * lg + j > li) || (dot && self) ? 0.f : w;
                            if (dot && self) own = w;
                            if constexpr (X::SCALE) m = fmaxf(m, fabsf(x[4 * q + j]));
                        }
                    }
                    if (dot && 2 * u <= t && t <= 2 * u + 1 && (li >> 2) == lg) owns[16 * t + li] = own;
                    if constexpr (X::SCALE) {
                        const int e = near_2_14(lanes_max(m, 16));
                        const float up_w = pow2(e);
                        if (lg == 0) downs[u * C + 16 * t + li] = pow2(-e);
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] *= up_w;
                    }
                    Frag *to = weights + (t < 2 ? t : 2 * t - 2 + u) * NP * 64 + lane;
#pragma unroll
                    for (int q = 0; q < NP; ++q) to[q * 64] = X::piece(x, q == NP - 1);
                }
            }
        }
        if (wave == EW && i0 + C < i_hi) {
            exponents(decays[turn ^ 1], gg);
            gg = decay(i0 + 2 * C);
        }
        Frag cf[NU];
#pragma unroll
        for (int u = 0; u < NU; ++u) cf[u] = LM::across(lc, 32 * u, wave * 16);
        f4 acc[OUT ? NT : 1];
        int se = 0;
        if constexpr (OUT) {
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] = f4{0.f, 0.f, 0.f, 0.f};
            // the state's part: o^T = X^T a^T, the pieces of X straight from the accumulators
            if constexpr (X::SCALE) {
                float m = 0.f;
#pragma unroll
                for (int p = 0; p < 2 * KS; ++p)
#pragma unroll
                    for (int j = 0; j < 4; ++j) m = fmaxf(m, fabsf(st[p][j]));
                se = near_2_14(lanes_max(m, 1));
            }
            const float up_s = pow2(se);
#pragma unroll
            for (int p = 0; p < KS; ++p) {
                Frag x[NP];
                float w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = X::SCALE ? st[2 * p + (j >> 2)][j & 3] * up_s : st[2 * p + (j >> 2)][j & 3];
#pragma unroll
                for (int q = 0; q < NP; ++q)
                    x[q] = X::piece(w, q == NP - 1);
                Frag a[NT];  // (products in chains side by side: one waits for the last of its own chain)
#pragma unroll
                for (int t = 0; t < NT; ++t) a[t] = LA::along(la, 16 * t, 32 * p);
#pragma unroll
                for (int q = 0; q < NP; ++q)
#pragma unroll
                    for (int t = 0; t < NT; ++t) acc[t] = X::mul(x[q], a[t], acc[t]);
            }
        }
        // the state: decayed, and the chunk's products added
        const float factor = dec[4 * C];
        Frag x[NU][X::UPD];
        float vw[NU][8], vm = 0.f, vdown = 1.f;
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const f4 d = *(const f4 *)(dec + 3 * C + 32 * u + 16 * q + 4 * lg);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    vw[u][4 * q + j] = X::get(cf[u], 4 * q + j) * d[j];
                    if constexpr (X::SCALE) vm = fmaxf(vm, fabsf(vw[u][4 * q + j]));
                }
            }
        if constexpr (X::SCALE) {
            const int e = near_2_14(lanes_max(vm, 16));
            const float up_v = pow2(e);
            vdown = pow2(-e);
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int j = 0; j < 8; ++j) vw[u][j] *= up_v;
        }
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int q = 0; q < X::UPD; ++q) x[u][q] = X::piece(vw[u], q == X::UPD - 1);
#pragma unroll
        for (int p = 0; p < KS; ++p) {
            f4 add[2] = {f4{0.f, 0.f, 0.f, 0.f}, f4{0.f, 0.f, 0.f, 0.f}};
            Frag k[2][NU];
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i) k[i][u] = LK::across(lb, 32 * u, 32 * p + 16 * i);
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int q = 0; q < X::UPD; ++q)
#pragma unroll
                    for (int i = 0; i < 2; ++i) add[i] = X::mul(k[i][u], x[u][q], add[i]);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    st[2 * p + i][j] = fmaf(st[2 * p + i][j], factor, X::SCALE ? add[i][j] * vdown : add[i][j]);
        }
        if constexpr (OUT) {
            __syncthreads();  // (the weights are there)
            // the chunk's own part, 16 steps at a time
            const int eo = wide ? 4 : EB;
            const __amdgpu_buffer_rsrc_t wo = window((char *)o + (row0 * ldo + h * M) * eo, ldo, M, cnt, eo);
            const int vo = lane_at(li, ldo, col0 + 4 * lg, M, eo);
            f4 in[NT][X::SCALE ? NU : 1];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int u = 0; u < (X::SCALE ? NU : 1); ++u) in[t][u] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int q = 0; q < NP; ++q)
#pragma unroll
                    for (int t = 2 * u; t < NT; ++t)
                        in[t][X::SCALE ? u : 0] = X::mul(cf[u], weights[((t < 2 ? t : 2 * t - 2 + u) * NP + q) * 64 + lane],
                                                         in[t][X::SCALE ? u : 0]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float mid = dec[2 * C + 16 * t + li] * out * (X::SCALE ? pow2(-se) : 1.f);
                float y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = acc[t][j] * mid;
#pragma unroll
                for (int u = 0; u < (X::SCALE ? NU : 1); ++u) {
                    if (2 * u > t) continue;
                    const float down = X::SCALE ? downs[u * C + 16 * t + li] : 1.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] = fmaf(in[t][u][j], down, y[j]);
                }
                const int j0 = 16 * t + li, c = col0 + 4 * lg;
                const uint32_t row = (uint32_t)at(j0, cnt);
                if (dot) {  // and then the step's own product
                    float z[4], e = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const u4 w = ge[DO == BACKWARD ? t : 0];
                        if constexpr (IO == IO_F32 || !WHOLE) z[j] = __uint_as_float(w[j]);
                        else z[j] = to_f<IO>(__builtin_bit_cast(T, (uint16_t)(w[j >> 1] >> (16 * (j & 1)))));
                        e = fmaf(z[j], y[j], e);
                    }
                    e += __shfl_xor(e, 16);
                    e += __shfl_xor(e, 32);
                    if (lg == 0) dots[wave * C + 16 * t + li] = e;
                    const int cl = wave * 16 + 4 * lg;
                    const float own = owns[16 * t + li];
                    ld_row<IO, 4>((const T *)(lc + LM::at(16 * t + li, cl / E)) + cl % E, z);
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] = fmaf(own, z[j], y[j]);
                }
                if constexpr (WHOLE) {
                    if (IO == IO_F32 || wide) {
                        const f4 v = {y[0], y[1], y[2], y[3]};
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, v), wo, vo + rows_at(16 * t, ldo, cnt, 4), 0, 0);
                    } else {
                        uint16_t v[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[j] = __builtin_bit_cast(uint16_t, from_f<IO == IO_F32 ? IO_F16 : IO>(y[j]));
                        __builtin_amdgcn_raw_buffer_store_b64(u2{v[0] | (uint32_t)v[1] << 16, v[2] | (uint32_t)v[3] << 16}, wo,
                                                              vo + rows_at(16 * t, ldo, cnt, 2), 0, 0);
                    }
                } else {
                    const int64_t first = row0 * ldo + h * M;
                    const uint32_t to = row * (uint32_t)ldo + c;
                    if (wide) st_row<IO_F32, 4>((float *)o + first + to, y, j0 < cnt ? M - c : 0);
                    else st_row<IO, 4>((T *)o + first + to, y, j0 < cnt ? M - c : 0);
                }
            }
        }
    }
    if (dot && i_lo < i_hi) {
        __syncthreads();
        put_dots(i_lo + (i_hi - i_lo - 1) / C * C);
    }
    int rows = K;
    asm volatile("" : "+s"(rows));  // (else the choices made for the state that entered are kept for this one)
    const auto put = [&](float *to) INLINE {
#pragma unroll
        for (int m = 0; m < 2 * KS; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = 16 * m + 4 * lg + j, c = col0 + li;
                if (k < rows && c < M) to[k * rs + c * cs] = st[m][j];
            }
    };
    if constexpr (OUT) {
        if (s1 && seg == sg.n - 1) put(s1 + bh * K * M);
        for (int64_t t = std::max<int64_t>(n, seg * sg.len) + wave; t < std::min<int64_t>(s.N, seg * sg.len + sg.len); t += WV)  // past the row's end
            for (int c = tile * MB + lane; c < std::min(M, (tile + 1) * MB); c += 64) {
                const int64_t to = (b * s.N + t) * ldo + h * M + c;
                if (wide) ((float *)o)[to] = 0.f;
                else ((T *)o)[to] = T(0);
            }
    } else {
        put(sg.state + slot * sg.plane);
        if (tile == 0 && wave == EW && lane == 0) sg.factor[slot] = factor_of(all);
    }
}

// The states that enter the segments, from what each segment adds.  One pass over the segments' states: 14 us for 32
// segments of each of 8 heads of 128 x 128, in order, so that equal calls give equal bits.
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
        if (j + 1 < sg.n) x = carried(x, sg.factor[slot], add);
    }
}

// dg of one sequence and head from the dot products, from the end on, in 64 bits.  The dot products are fp32, and what
// they are off by adds up along the sequence; but before the first step it has to come to <x_in, dx_in>, so what it
// misses that by is taken back evenly over the steps (a third of the squared error on average is left).  Before a step
// whose factor is 0 it has to come to 0: the sum begins anew there and is corrected for itself, so that nothing of a
// document reaches the one before it (a document before one of 1e4 times its gradients: 1e-3 of dg without).  Two or
// three passes over N numbers and two over a state by one block: 7 us beside 310 for four sequences of 2048 steps and
// 20 heads.
constexpr int kDg = 1024;
__device__ __forceinline__ double block_sum(double v, double *lds) {
    v = lane_of(sum_up_to(v), 63);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
    for (int w = 0; w < kDg / 64; ++w) v += lds[w];
    return v;
}
// The sum over the lanes from the last one in `starts` up to this one (or from the wave's first, where there is none).
__device__ __forceinline__ double sum_from_start(double v, uint64_t starts) {
    if (starts == 0) return sum_up_to(v);
    const int lane = threadIdx.x & 63;
    int from = 63 - __builtin_clzll((starts & (~0ull >> (63 - lane))) | 1);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double u = __shfl_up(v, d);
        if (lane - d >= from) v += u;
    }
    return v;
}
__global__ __launch_bounds__(kDg) void k_lin_dg(float *dq, float *dk, int tiles, const float *__restrict__ s_end,
                                                const float *__restrict__ ds_end, const float *__restrict__ x_in,
                                                const float *__restrict__ dx_in, int64_t kv, Shape s, float *dg, double *sums) {
    constexpr int W = kDg / 64;
    __shared__ double lds[W];
    __shared__ int edge[W];
    const int64_t bh = block_id();
    if (bh >= s.B * s.H) return;
    const int64_t b = bh / s.H, h = bh - b * s.H, plane = s.B * s.H * s.N;
    const int n = (int)row_len(s.lengths, b, s.N), tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    dq += bh * s.N, dk += bh * s.N;
    double carry = 0.0, front = 0.0;  // <S, D> behind the last step, and before the first
    if (ds_end) {
        for (int64_t i = tid; i < kv; i += kDg) carry += (double)s_end[bh * kv + i] * ds_end[bh * kv + i];
        carry = block_sum(carry, lds);
    }
    if (x_in && dx_in) {
        for (int64_t i = tid; i < kv; i += kDg) front += (double)x_in[bh * kv + i] * dx_in[bh * kv + i];
        front = block_sum(front, lds);
    }
    const bool known = !x_in || dx_in;  // (front)
    const auto step = [&](int t) {
        double v = 0.0;
        for (int i = 0; i < tiles; ++i) v += (double)dq[i * plane + t] - (double)dk[i * plane + t];
        return v;
    };
    dg += s.per_token ? b * s.N * s.H + h : 0;
    const auto clears = [&](int t) { return (s.per_token ? s.g[(b * s.N + t) * s.H + h] : s.g[h]) < kZeroBelow; };
    double all = 0.0, weighted = 0.0;  // sums of all steps, and of all of their sums
    bool any = false;
    for (int t = tid; t < n; t += kDg) {
        const double v = step(t);
        all += v;
        weighted += v * (double)(t + 1);
        any |= clears(t);
    }
    const double missed = known && n > 0 ? (block_sum(all, lds) + carry - front) / (double)n : 0.0;
    if (!s.per_token) {
        weighted = block_sum(weighted, lds) + carry * (double)n - missed * 0.5 * (double)n * (double)(n + 1);
        if (tid == 0) sums[bh] = any || n == 0 ? 0.0 : weighted;
        return;
    }
    for (int t = n + tid; t < s.N; t += kDg) dg[t * s.H] = 0.f;
    if (!__syncthreads_or(any)) {  // one part: 9 us for rows of 2048, as below 16
        for (int i0 = 0; i0 < n; i0 += kDg) {
            const int t = n - 1 - i0 - tid;
            const double sum = sum_up_to(t >= 0 ? step(t) : 0.0);
            __syncthreads();
            if (lane == 63) lds[wave] = sum;
            __syncthreads();
            double before = carry;
            for (int w = 0; w < W; ++w) {
                before += w < wave ? lds[w] : 0.0;
                carry += lds[w];
            }
            if (t >= 0) dg[t * s.H] = (float)(before + sum - missed * (double)(n - t));
        }
        return;
    }
    // From the end: the sums, in two parts in the place of the dot products, and where each began, in that of dg.
    int last = n;
    for (int i0 = 0; i0 < n; i0 += kDg) {
        const int t = n - 1 - i0 - tid;
        const bool start = t >= 0 && t + 1 < n && clears(t + 1);
        const uint64_t starts = __ballot(start), mine = starts & (~0ull >> (63 - lane));
        double sum = sum_from_start(t >= 0 ? step(t) : 0.0, starts);
        int end = mine ? t + 1 + lane - (63 - __builtin_clzll(mine)) : -1;
        __syncthreads();
        if (lane == 63) lds[wave] = sum, edge[wave] = end;
        __syncthreads();
        for (int w = 0; w < W; ++w) {
            if (w == wave && end < 0) sum += carry, end = last;
            carry = edge[w] < 0 ? carry + lds[w] : lds[w];
            last = edge[w] < 0 ? last : edge[w];
        }
        if (t >= 0) {
            const float hi = (float)sum;
            dq[t] = hi, dk[t] = (float)(sum - (double)hi);
            dg[t * s.H] = __int_as_float(end);
        }
    }
    __syncthreads();
    // From the front: what each sum misses at its first step (one that clears, or the row's first) is spread over its steps.
    int first = -1;
    for (int t0 = 0; t0 < n; t0 += kDg) {
        const int t = t0 + tid;
        double sum = 0.0;
        int end = 0, from = -1;
        bool clear = false;
        if (t < n) {
            clear = clears(t);
            sum = (double)dq[t] + (double)dk[t];
            end = __float_as_int(dg[t * s.H]);
        }
        const uint64_t mine = __ballot(clear) & (~0ull >> (63 - lane));
        if (mine) from = t - lane + (63 - __builtin_clzll(mine));
        __syncthreads();
        if (lane == 63) edge[wave] = from;
        __syncthreads();
        for (int w = 0; w < W; ++w) {
            if (w == wave && from < 0) from = first;
            first = edge[w] < 0 ? first : edge[w];
        }
        if (t < n) {
            const int at = from < 0 ? 0 : from;
            const double there = (double)dq[at] + (double)dk[at], off = from >= 0 ? there : known ? there - front : 0.0;
            dg[t * s.H] = clear ? 0.f : (float)(sum - off * ((double)(end - t) / (double)(end - at)));
        }
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

// One token of each sequence: a block per sequence and head, which reads and writes every state once: HBM bound, and by
// the launch where the states are few.  A thread has VEC columns side by side and every 256 / (64 / VEC)-th row.
// 25.5 MB of states and tokens (64 sequences of 12 heads of 64 x 64, fp16): 6.2 us, 7.4 with a column per thread.
template <int IO, int VEC>
__global__ __launch_bounds__(256) void k_lin_step(LinStepArgs s) {
    using T = typename io_elem<IO>::T;
    typedef float fv __attribute__((ext_vector_type(VEC)));
    constexpr int CG = 64 / VEC, RG = 256 / CG;  // threads across 64 columns, and down the rows
    __shared__ float lds[RG][64];
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
    const int rg = threadIdx.x / CG, cl = threadIdx.x % CG * VEC;
    for (int c0 = 0; c0 < s.dv; c0 += 64) {
        const int c = c0 + cl;
        fv sum = {};
        if (c < s.dv) {  // (and so are all VEC)
            fv vc;
#pragma unroll
            for (int j = 0; j < VEC; ++j) vc[j] = to_f<IO>(v[c + j]);
#pragma unroll 4
            for (int i = rg; i < s.dk; i += RG) {
                const float ki = to_f<IO>(k[i]), qi = to_f<IO>(q[i]);
                fv x = *(const fv *)(from + i * s.dv + c);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    x[j] = fmaf(ki, vc[j], e * x[j]);
                    sum[j] = fmaf(qi, x[j], sum[j]);
                }
                *(fv *)(to + i * s.dv + c) = x;
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < VEC; ++j) lds[rg][cl + j] = sum[j];
        __syncthreads();
        if (threadIdx.x < 64 && c0 + (int)threadIdx.x < s.dv) {
            float o = lds[0][threadIdx.x];
#pragma unroll
            for (int r = 1; r < RG; ++r) o += lds[r][threadIdx.x];
            y[c0 + threadIdx.x] = from_f<IO>(o * s.scale);
        }
    }
}

int64_t up(int64_t n) { return (n + 255) & ~(int64_t)255; }

// Columns of a block: 16 for each of its waves.
int cols_of(int M) { return M > 64 ? 128 : 64; }
int tiles_of(int M) { return (M + cols_of(M) - 1) / cols_of(M); }

// Blocks that the chip holds at once.  A row has segments for that many: with half as many blocks the chip is half
// empty, with twice as many every segment's state is found twice over (eight waves: 377 us with 256, 469 with 512; four
// waves and small states: 35.9 with 768, 38 with 512).
int64_t at_once(int K, int M) { return cols_of(M) == 64 && K <= 64 ? 768 : cols_of(M) == 64 && K <= 128 ? 512 : 256; }

// Segments of a row of N steps where `blocks` work on each.
constexpr int kChunk = 64;
Segs segs_of(int64_t N, int64_t blocks, int64_t at_once) {
    const int64_t chunks = std::max<int64_t>(1, (N + kChunk - 1) / kChunk);
    int64_t n = std::min(chunks, std::max<int64_t>(1, at_once / std::max<int64_t>(1, blocks)));
    const int64_t per = (chunks + n - 1) / n;
    Segs g = {};
    g.len = per * kChunk;
    g.n = (chunks + per - 1) / per;
    return g;
}
int64_t seg_bytes(const Segs &g, int64_t BH, int roles, int64_t plane) {
    return g.n == 1 ? 0 : up(roles * g.n * BH * plane * 4) + up(roles * g.n * BH * (int64_t)sizeof(Factor));
}

template <int IO, int KP, int WV, int DO, bool WHOLE>
hipError_t run_chunks(const Roles &r, int n, const Shape &s, const Segs &g, int tiles, hipStream_t st) {
    const int64_t BH = s.B * s.H;
    if (g.n > 1) {
        hipError_t e = launch(k_lin_chunk<IO, KP, WV, STATES, WHOLE>, grid_of((g.n - 1) * BH * tiles, (unsigned)n), dim3(WV * 64), 0, st, r,
                              s, g, tiles);
        if (e != hipSuccess) return e;
        if (g.n > kFew) e = launch(k_lin_enter, grid_of((BH * g.plane + 255) / 256, (unsigned)n), dim3(256), 0, st, r, g, BH);
        if (e != hipSuccess) return e;
    }
    return launch(k_lin_chunk<IO, KP, WV, DO, WHOLE>, grid_of(g.n * BH * tiles, (unsigned)n), dim3(WV * 64), 0, st, r, s, g, tiles);
}

// Whether every head is whole units of 16 bytes, and every token begins at a dword.
template <int IO>
bool whole(const Roles &r, int n) {
    constexpr int e = IO == IO_F32 ? 4 : 2;
    for (int i = 0; i < n; ++i) {
        for (const Seq *q : {&r.r[i].a, &r.r[i].b, &r.r[i].c, &r.r[i].e})
            if (q->dim * e % 16 != 0 || q->ld * e % 4 != 0 || reinterpret_cast<uintptr_t>(q->p) % 4 != 0) return false;
        if (reinterpret_cast<uintptr_t>(r.r[i].o) % 4 != 0) return false;
    }
    return true;
}

// K, M: the most rows and columns of the roles' states; ws: seg_bytes.
template <int IO, int DO>
hipError_t run_roles(const Roles &r, int n, const Shape &s, int K, int M, Segs g, int64_t plane, void *ws, hipStream_t st) {
    const int tiles = tiles_of(M);
    g.plane = plane;
    g.state = (float *)ws;
    g.factor = (Factor *)((char *)ws + up(n * g.n * s.B * s.H * plane * 4));
    if (!whole<IO>(r, n)) {
        const bool few = cols_of(M) == 64;
        if (K <= 64) return few ? run_chunks<IO, 64, 4, DO, false>(r, n, s, g, tiles, st) : run_chunks<IO, 64, 8, DO, false>(r, n, s, g, tiles, st);
        if (K <= 128) return few ? run_chunks<IO, 128, 4, DO, false>(r, n, s, g, tiles, st) : run_chunks<IO, 128, 8, DO, false>(r, n, s, g, tiles, st);
        return few ? run_chunks<IO, 256, 4, DO, false>(r, n, s, g, tiles, st) : run_chunks<IO, 256, 8, DO, false>(r, n, s, g, tiles, st);
    }
    if (cols_of(M) == 64) {
        if (K <= 32) return run_chunks<IO, 32, 4, DO, true>(r, n, s, g, tiles, st);
        if (K <= 64) return run_chunks<IO, 64, 4, DO, true>(r, n, s, g, tiles, st);
        if (K <= 128) return run_chunks<IO, 128, 4, DO, true>(r, n, s, g, tiles, st);
        return run_chunks<IO, 256, 4, DO, true>(r, n, s, g, tiles, st);
    }
    if (K <= 64) return run_chunks<IO, 64, 8, DO, true>(r, n, s, g, tiles, st);
    if (K <= 128) return run_chunks<IO, 128, 8, DO, true>(r, n, s, g, tiles, st);
    return run_chunks<IO, 256, 8, DO, true>(r, n, s, g, tiles, st);
}
Segs fwd_segs(int64_t B, int64_t N, int64_t H, int64_t dk, int64_t dv) {
    return segs_of(N, B * H * tiles_of((int)dv), at_once((int)dk, (int)dv));
}
Segs bwd_segs(int64_t B, int64_t N, int64_t H, int64_t dk, int64_t dv) {
    const int m = (int)std::max(dk, dv);
    return segs_of(N, 3 * B * H * tiles_of(m), at_once(m, m));
}

// The parts of the backward pass's workspace, in bytes from its start.
struct BwdSpace {
    int64_t row, col, s_end, sums, dq, dk, segs, all;
};
int dot_tiles(int64_t dk, int64_t dv) {
    const int cols = cols_of((int)std::max(dk, dv));
    return (int)((dk + cols - 1) / cols);
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
    return run_roles<IO, FORWARD>(r, 1, shape_of(a), a.dk, a.dv, fwd_segs(a.B, a.N, a.H, a.dk, a.dv), (int64_t)a.dk * a.dv, ws, s);
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
    hipError_t e = a.B > 0 ? run_roles<IO, BACKWARD>(r, 3, s, m, m, bwd_segs(a.B, a.N, a.H, a.dk, a.dv), (int64_t)a.dk * a.dv,
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
        e = launch(k_lin_dg, grid_of(a.B * a.H), dim3(kDg), 0, st, row, col, dot_tiles(a.dk, a.dv), s_end, dx_out, a.x_in, o.dx_in,
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

template <int IO>
static hipError_t step_io(const LinStepArgs &a, hipStream_t s) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.x_in) | reinterpret_cast<uintptr_t>(a.x_out);
    if (a.dv % 4 == 0 && at % 16 == 0) return launch(k_lin_step<IO, 4>, grid_of(a.B * a.H), dim3(256), 0, s, a);
    return launch(k_lin_step<IO, 1>, grid_of(a.B * a.H), dim3(256), 0, s, a);
}

hipError_t launch_linear_attn_step(const LinStepArgs &a, int io, hipStream_t s) {
    switch (io) {
        case IO_F32: return step_io<IO_F32>(a, s);
        case IO_F16: return step_io<IO_F16>(a, s);
        default: return step_io<IO_BF16>(a, s);
    }
}

}  // namespace h3c
