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
// Logits, maxima, sums and the products' sums are fp32.  With 16-bit inputs G is
// rounded to them, as the operand of two 16-bit products (in 32 bits they would
// run at a sixteenth of the rate).  Its error averages out over the sums: at 8192
// x 768 x 50021 bf16, dx and dw are off by 1.660e-3 and 1.663e-3 of their norms
// with it and by 1.658e-3 and 1.661e-3 with G in 32 bits, which is what rounding
// dx and dw themselves to bf16 makes.
//
// Measured in bf16 at 8192 x 768 x 50021: logits and statistics 640 us (980
// TFLOP/s; a library product of that size 986), G 2 x 400 us, dx and dw 2 x 750 us
// (840 TFLOP/s; the library's 1066 and 1254); fp16 at 4096 x 2560 x 32768 forward
// 580 to 605 us (1140 to 1180 TFLOP/s; 1433); fp32 at 4096 x 768 x 8192 109 TFLOP/s
// forward, 114 backward (154 at 8192^3).  The 256-sided tiles of G and of the
// products spill two and three registers, outside their loops.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "lm_device.h"
#include "lm_internal.h"
#include "xent_plan.h"

namespace h3c {
namespace {

using namespace xent;  // tile sides, pieces, ranges and the workspace

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

// ------------------------------------------------------- 16-bit tile products
//
// One block forms a BM x BN tile of A B^T, its waves WM x WN parts of it.  An
// operand is K-contiguous (row m of A holds its k elements) or K-major (row k
// holds the m elements; read back transposed by ds_read_b64_tr_b16).  Slabs of
// KS elements of k go straight from memory to LDS, NS of them in a ring; the
// fragments of the next k step are read while the matrix cores work on this
// one, so the only wait is for a slab that was requested NS - 1 slabs earlier.
// LDS positions are permuted in units of 16 (32) bytes on the way in, by
// choosing the address each lane loads, so that fragment reads meet no bank
// twice.
typedef short s4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s4 lds_s4;
typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void glb_void;

// ROWS x KS of one operand.  mem: its element (0, 0) of the tile's rows;
// ld: bytes per memory row.  rows: valid rows (K-contiguous) or row bytes
// (K-major), k: valid k; what lies beyond repeats the last valid one.
template <int ROWS, int KS, int NT, bool KMAJOR>
struct Operand {
    static constexpr int kBytes = ROWS * KS * 2, kLoads = kBytes / 16 / NT;
    static constexpr int kRowChunks = KMAJOR ? ROWS / 8 : KS / 8;  // 16-byte chunks per LDS row
    const char *mem;
    int64_t ld, k;
    int32_t off[kLoads];  // (the shim keeps 256 rows within 31 bits)

    __device__ __forceinline__ static int slot(int krow) { return ((krow & 3) | ((krow >> 3) & 1) << 2) & (ROWS / 16 - 1); }
    __device__ __forceinline__ static int turn(int row) { return row & (KS / 8 - 1); }

    __device__ __forceinline__ void init(const char *m, int64_t ld_, int64_t rows, int64_t k_) {
        mem = m;
        ld = ld_;
        k = k_;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int q = i * NT + (int)threadIdx.x, row = q / kRowChunks, pos = q % kRowChunks;
            if constexpr (KMAJOR) {
                const int c = ((pos >> 1) ^ slot(row)) * 2 + (pos & 1);
                const int64_t last = rows / 16 - 1;
                off[i] = (int32_t)((c < last ? c : last) * 16);
            } else {
                const int64_t r = row < rows ? row : rows - 1;
                off[i] = (int32_t)(r * ld + (pos ^ turn(row)) * 16);
            }
        }
    }
    // slab s into the LDS bytes at `to`
    __device__ __forceinline__ void load(int64_t s, char *to) const {
        const char *base = mem + s * (KMAJOR ? KS * ld : (int64_t)KS * 2);
        const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            int32_t o = off[i];
            if constexpr (KMAJOR) {
                // rows past the end read the last valid one, which lies behind
                // `base` where the whole slab is past it
                const int row = (i * NT + (int)threadIdx.x) / kRowChunks;
                const int64_t last = k - 1 - s * KS;
                o += (row < last ? row : (int)last) * (int32_t)ld;
            }
            __builtin_amdgcn_global_load_lds((glb_void *)(base + o), (lds_void *)(to + (i * NT + wave * 64) * 16), 16, 0, 0);
        }
    }
    // fragment of the 16 rows from `m`, k step s of the slab
    __device__ __forceinline__ static u4 frag(const char *from, int m, int s) {
        const int l = threadIdx.x & 63, g = l >> 4, i = l & 15;
        if constexpr (KMAJOR) {
            typedef int i2 __attribute__((ext_vector_type(2)));
            i2 h[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int kr = s * 32 + g * 8 + q * 4 + (i >> 2);
                const char *p = from + kr * (ROWS * 2) + (((m >> 4) ^ slot(kr)) * 32) + (i & 3) * 8;
                h[q] = __builtin_bit_cast(i2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)p));
            }
            return u4{(uint32_t)h[0].x, (uint32_t)h[0].y, (uint32_t)h[1].x, (uint32_t)h[1].y};
        } else {
            const int row = m + i, c = s * 4 + g;
            return *(const u4 *)(from + row * (KS * 2) + ((c ^ turn(row)) * 16));
        }
    }
};

template <int IO, int BM_, int BN_, int WM, int WN, int KS_, int NS, bool AK, bool BK>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, KS = KS_, NT = WM * WN * 64, TM = BM / WM / 16, TN = BN / WN / 16;
    using OA = Operand<BM, KS, NT, AK>;
    using OB = Operand<BN, KS, NT, BK>;
    static constexpr int kStage = OA::kBytes + OB::kBytes, kLds = NS * kStage;
    static constexpr int kLoads = OA::kLoads + OB::kLoads;
    static_assert(KS == 64 && KS == kSlab16, "two k steps per slab; what rows are padded to");
    f4 acc[TM][TN];

    __device__ __forceinline__ static int wave() { return __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6); }
    __device__ __forceinline__ static int row0() { return wave() / WN * (BM / WM); }
    __device__ __forceinline__ static int col0() { return wave() % WN * (BN / WN); }

    __device__ __forceinline__ static void read(const char *stage, int s, u4 (&a)[TM], u4 (&b)[TN]) {
#pragma unroll
        for (int i = 0; i < TM; ++i) a[i] = OA::frag(stage, row0() + i * 16, s);
#pragma unroll
        for (int j = 0; j < TN; ++j) b[j] = OB::frag(stage + OA::kBytes, col0() + j * 16, s);
    }
    __device__ __forceinline__ void mul(const u4 (&a)[TM], const u4 (&b)[TN]) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = mfma16<IO>(a[i], b[j], acc[i][j]);
    }
    // Slab s + 1 has landed for every wave, and every wave has read its last
    // fragment of slab s: its place takes slab s + NS.
    __device__ __forceinline__ static void turn(const OA &a, const OB &b, char *lds, int64_t s, int64_t slabs) {
        // this thread's loads of slabs s + 2 .. s + NS - 1 may still be out
        if (s + NS - 1 < slabs) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NS - 2) * kLoads) : "memory");
        else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (s + NS < slabs) {
            char *to = lds + (s % NS) * kStage;
            a.load(s + NS, to);
            b.load(s + NS, to + OA::kBytes);
        }
    }
    // acc = A B^T over `slabs` slabs
    __device__ __forceinline__ void run(const OA &a, const OB &b, int64_t slabs, char *lds) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < NS; ++s)
            if (s < slabs) {
                a.load(s, lds + s * kStage);
                b.load(s, lds + s * kStage + OA::kBytes);
            }
        // slab 0 has landed: all loads but those of the slabs after it
        if (slabs >= NS) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NS - 1) * kLoads) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        u4 fa[2][TM], fb[2][TN];
        read(lds, 0, fa[0], fb[0]);
        int64_t s = 0;
        int st = 0;  // s % NS
        for (; s + 1 < slabs; ++s) {
            const int nx = st + 1 == NS ? 0 : st + 1;
            read(lds + st * kStage, 1, fa[1], fb[1]);
            __builtin_amdgcn_sched_barrier(0);
            mul(fa[0], fb[0]);
            turn(a, b, lds, s, slabs);
            read(lds + nx * kStage, 0, fa[0], fb[0]);
            __builtin_amdgcn_sched_barrier(0);
            mul(fa[1], fb[1]);
            st = nx;
        }
        read(lds + st * kStage, 1, fa[1], fb[1]);
        mul(fa[0], fb[0]);
        mul(fa[1], fb[1]);
    }
};

// ------------------------------------------------------------ fp32 tile products
//
// BT x BT tiles on the fp32 matrix cores (a sixteenth of the 16-bit rate, so
// LDS and caches keep up with small tiles, and small problems fill the chip).
// Rows may start at any element and have any length: operands are loaded
// through registers, some slabs of KS32 elements ahead, what lies past the end
// is zero.
constexpr int KS32 = 32;

// An operand of a tile: K-contiguous (rows of the tile are memory rows) or
// K-major (memory rows are k).
template <bool KMAJOR, int BT>
struct Operand32 {
    const float *mem;
    int64_t ld, total;  // elements per memory row, and in all from mem on (its memory has four at least, some before mem)
    int64_t rows, k;    // of the operand, from the tile's first row on

    // chunk `id` of the slab from k0, four k of a row or four rows at one k: its
    // memory row and first element there
    __device__ __forceinline__ static int64_t row(int64_t k0, int id) { return KMAJOR ? k0 + id / (BT / 4) : id >> 3; }
    __device__ __forceinline__ static int64_t col(int64_t k0, int id) { return KMAJOR ? id % (BT / 4) * 4 : k0 + (id & 7) * 4; }
    __device__ __forceinline__ int64_t last() const { return total - 4; }
    __device__ __forceinline__ int64_t offset(int64_t k0, int id) const { return row(k0, id) * ld + col(k0, id); }
    __device__ __forceinline__ int64_t step() const { return KMAJOR ? KS32 * ld : KS32; }
    // As loaded: always one vector, the operand's last where the chunk passes its
    // end, so that no load waits for a choice.
    __device__ __forceinline__ f4 load(int64_t o) const {
        float v[4];
        ld_row<IO_F32, 4>(mem + (o < last() ? o : last()), v);
        return f4{v[0], v[1], v[2], v[3]};
    }
    // The chunk from what load() gave: zeros past the k.  (Of slabs that end four
    // k before the last it is what load() gave: all k are valid, and only vectors
    // of rows past the last, whose products no one stores, pass the end.)
    __device__ __forceinline__ f4 chunk(f4 v, int64_t k0, int id) const {
        const int64_t r = row(k0, id), c = col(k0, id), o = offset(k0, id) - last(), n = KMAJOR ? rows : k;
        const int down = o > 0 ? (int)(o < 4 ? o : 0) : 0;  // (of 4 and more all are past the end)
        const int valid = r < (KMAJOR ? k : rows) ? (int)(n - c < 4 ? (n > c ? n - c : 0) : 4) : 0;
        float a = v[0], b = v[1], d = v[2], e = v[3];
        a = (down & 1) ? b : a, b = (down & 1) ? d : b, d = (down & 1) ? e : d;
        a = (down & 2) ? d : a, b = (down & 2) ? e : b;
        return f4{valid > 0 ? a : 0.f, valid > 1 ? b : 0.f, valid > 2 ? d : 0.f, valid > 3 ? e : 0.f};
    }
    // where element (row, k) of the slab is kept: fragment reads (16 rows, one
    // chunk of four k) and transposed writes both spread over the banks
    __device__ __forceinline__ static int at(int row, int chunk) { return row * 8 + (chunk ^ ((row ^ row >> 2) & 7)); }
    __device__ __forceinline__ static void keep(f4 *s, int id, f4 v) {
        if constexpr (KMAJOR) {
            const int kr = id / (BT / 4), m = id % (BT / 4) * 4;
#pragma unroll
            for (int j = 0; j < 4; ++j) ((float *)&s[at(m + j, kr >> 2)])[kr & 3] = v[j];
        } else {
            s[at(id >> 3, id & 7)] = v;
        }
    }
};

// A tile of A B^T; four waves have a quarter each.
template <int BT>
struct Tile32 {
    static constexpr int WT = BT / 2, TM = WT / 16, CH = BT * 8 / 256, AHEAD = 128 / BT;  // (slabs in flight)
    f4 acc[TM][TM];

    __device__ __forceinline__ static int row0() { return (threadIdx.x >> 7) * WT; }
    __device__ __forceinline__ static int col0() { return ((threadIdx.x >> 6) & 1) * WT; }

    // lds: two slabs of A and of B
    template <bool AK, bool BK>
    __device__ __forceinline__ void run(const Operand32<AK, BT> &a, const Operand32<BK, BT> &b, int64_t k,
                                        f4 (&lds)[2][2][BT * 8]) {
        const int tid = threadIdx.x, lane = tid & 63;
        f4 ga[AHEAD][CH], gb[AHEAD][CH];
        int64_t oa[CH], ob[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            oa[i] = a.offset(0, tid + i * 256);
            ob[i] = b.offset(0, tid + i * 256);
        }
        const auto load = [&](int p) {  // the next slab
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                ga[p][i] = a.load(oa[i]);
                gb[p][i] = b.load(ob[i]);
                oa[i] += a.step();
                ob[i] += b.step();
            }
        };
        // one slab; one barrier: the buffer written here was read two slabs ago
        const auto slab = [&](int64_t k0, int p) {
            if (k0 + KS32 + 3 >= k) {
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    ga[p][i] = a.chunk(ga[p][i], k0, tid + i * 256);
                    gb[p][i] = b.chunk(gb[p][i], k0, tid + i * 256);
                }
            }
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                a.keep(lds[p & 1][0], tid + i * 256, ga[p][i]);
                b.keep(lds[p & 1][1], tid + i * 256, gb[p][i]);
            }
            load(p);
            __syncthreads();
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                u4 fa[TM], fb[TM];
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const int c = s * 4 + (lane >> 4);
                    fa[i] = __builtin_bit_cast(u4, lds[p & 1][0][Operand32<AK, BT>::at(row0() + i * 16 + (lane & 15), c)]);
                    fb[i] = __builtin_bit_cast(u4, lds[p & 1][1][Operand32<BK, BT>::at(col0() + i * 16 + (lane & 15), c)]);
                }
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TM; ++j) acc[i][j] = mfma16<IO_F32>(fa[i], fb[j], acc[i][j]);
            }
        };
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TM; ++j) acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int p = 0; p < AHEAD; ++p) load(p);
        for (int64_t k0 = 0; k0 < k; k0 += AHEAD * KS32) {
#pragma unroll
            for (int p = 0; p < AHEAD; ++p)
                if (p == 0 || k0 + p * KS32 < k) slab(k0 + p * KS32, p);
        }
    }
};

struct Labels {
    const int64_t *label;
    int64_t ignore, V;
    // the label of token t, or -1 where it carries no loss
    __device__ __forceinline__ int64_t of(int64_t t) const {
        const int64_t l = label[t];
        return (l == ignore || l < 0 || l >= V) ? -1 : l;
    }
};

__device__ __forceinline__ float2 join(float2 a, float2 b);

// Per token of the tile (its rows): (maximum, sum of e^{l - maximum}) over the
// tile's columns to part[tile][t], and the label's logit where it is one of them.
template <int BT>
__global__ __launch_bounds__(256, 4) void k_xent_stats32(const float *x, const float *w, int64_t ld, const Labels lab,
                                                      float2 *__restrict__ part, float *__restrict__ hit, int64_t T,
                                                      int64_t D, int64_t V) {
    using P = Tile32<BT>;
    constexpr int TM = P::TM;
    __shared__ f4 lds[2][2][BT * 8];
    __shared__ float2 half[BT];
    const int64_t id = block_id(), tiles = (T + BT - 1) / BT, tile = id / tiles;  // of the vocabulary; tokens run first
    const int64_t m0 = (id - tile * tiles) * BT, n0 = tile * BT;
    if (n0 >= V) return;
    P tile32;
    tile32.run(Operand32<false, BT>{x + m0 * ld, ld, (T - m0) * ld, T - m0, D},
               Operand32<false, BT>{w + n0 * ld, ld, (V - n0) * ld, V - n0, D}, D, lds);
    const auto &acc = tile32.acc;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = P::row0(), wn = P::col0();
    float2 st[TM][4];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t t = m0 + wm + i * 16 + (lane >> 4) * 4 + e;
            const int64_t l = t < T ? lab.of(t) : -1;
            float m = -INFINITY, s = 0.f;
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const int64_t v = n0 + wn + j * 16 + (lane & 15);
                if (v < V) m = fmaxf(m, acc[i][j][e]);
                if (v < V && v == l) hit[t] = acc[i][j][e];
            }
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
            const float mm = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int j = 0; j < TM; ++j)
                if (n0 + wn + j * 16 + (lane & 15) < V) s += __builtin_amdgcn_exp2f((acc[i][j][e] - mm) * kLog2e);
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) s += __shfl_xor(s, d);
            st[i][e] = make_float2(m, s);
            if ((wave & 1) && (lane & 15) == 0) half[wm + i * 16 + (lane >> 4) * 4 + e] = st[i][e];
        }
    __syncthreads();
    if (!(wave & 1) && (lane & 15) == 0) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = wm + i * 16 + (lane >> 4) * 4 + e;
                if (m0 + row < T) part[tile * T + m0 + row] = join(st[i][e], half[row]);
            }
    }
}

// Joins the tiles' pairs of 64 tokens per block: 16 threads per token take
// every 16th tile, then one joins those, both in order.
__device__ __forceinline__ float2 join(float2 a, float2 b) {
    const float m = fmaxf(a.x, b.x), mm = m == -INFINITY ? 0.f : m;
    return make_float2(m, a.y * __builtin_amdgcn_exp2f((a.x - mm) * kLog2e) + b.y * __builtin_amdgcn_exp2f((b.x - mm) * kLog2e));
}
__global__ __launch_bounds__(1024) void k_xent_join(const float2 *__restrict__ part, const float *__restrict__ hit,
                                                    const Labels lab, float *__restrict__ loss,
                                                    float *__restrict__ lse, int64_t T, int64_t tiles) {
    __shared__ float2 red[16][64];
    const int64_t t = block_id() * 64 + (threadIdx.x & 63);
    const int g = threadIdx.x >> 6;
    float2 a = make_float2(-INFINITY, 0.f);
    if (t < T)
        for (int64_t i = g; i < tiles; i += 16) a = join(a, part[i * T + t]);
    red[g][threadIdx.x & 63] = a;
    __syncthreads();
    if (g == 0 && t < T) {
        for (int i = 1; i < 16; ++i) a = join(a, red[i][threadIdx.x]);
        const float l = a.x + logf(a.y);
        lse[t] = l;
        loss[t] = lab.of(t) >= 0 ? l - hit[t] : 0.f;
    }
}

// Vector i (16 bytes) of dst[r][c] = src[r][c] for c < C, zero up to ldd (whole
// vectors) and in rows that keep(r) does not.
template <class E, class Keep>
__device__ __forceinline__ void pad_vector(const E *src, E *dst, int64_t R, int64_t C, int64_t ldd, int64_t i,
                                           const Keep &keep) {
    constexpr int n = 16 / (int)sizeof(E);
    const int64_t v = ldd / n, r = i / v, c = (i - r * v) * n;
    if (r >= R) return;
    Pack<E, n> q{};
    if (keep(r)) {
        if (c + n <= C) {
            q = *reinterpret_cast<const Pack<E, n> *>(src + r * C + c);
        } else {
#pragma unroll
            for (int e = 0; e < n; ++e) q.v[e] = c + e < C ? src[r * C + c + e] : (E)0;
        }
    }
    *reinterpret_cast<Pack<E, n> *>(dst + r * ldd + c) = q;
}

// What the 16-bit gradients need of the tokens, in one launch.  Blocks from 1 on
// copy x to rows of whole slabs, and to zeros where a token carries no loss: dw
// multiplies those by a G of zero, but they may hold anything.  Block 0, which
// takes longer, finds the scale of G: it is held as a share of the largest
// finite |dloss| of a token that counts.  With the usual equal weights the entry of a
// label, -(1 - p), is then held almost exactly, and it dominates its row.  fp16
// multiplies by 2^15 more, so that probabilities down to 2^-29 stay normal
// numbers.  scale[0]: the divisor, scale[1]: what undoes both in the fp32 sums.
template <int IO>
__global__ __launch_bounds__(1024) void k_xent_tokens16(const typename io_elem<IO>::T *__restrict__ x,
                                                        typename io_elem<IO>::T *__restrict__ xc, int64_t D, int64_t kD,
                                                        const float *__restrict__ dloss, const Labels lab,
                                                        float *__restrict__ scale, int64_t T) {
    if (block_id() > 0) {
        pad_vector(x, xc, T, D, kD, (block_id() - 1) * 1024 + threadIdx.x, [&](int64_t t) { return lab.of(t) >= 0; });
        return;
    }
    __shared__ float red[16];
    float m = 0.f;
#pragma unroll 8
    for (int64_t t = threadIdx.x; t < T; t += 1024)
        if (lab.of(t) >= 0 && fabsf(dloss[t]) < INFINITY) m = fmaxf(m, fabsf(dloss[t]));
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 16; ++i) m = fmaxf(m, red[i]);
        if (!(m > 0.f)) m = 1.f;
        scale[0] = m;
        scale[1] = IO == IO_F16 ? m * 0x1p-15f : m;
    }
}
// this token's weight in G
template <int IO>
__device__ __forceinline__ float weight(float dloss, float divisor) {
    return dloss / divisor * (IO == IO_F16 ? 0x1p15f : 1.f);
}

// G of the vocabulary piece [v0, v0 + nv): g[t][v - v0], rows of nv.  xc, unless
// null: x for dw's product, with zero rows as in k_xent_tokens16, each block a
// share of its tokens' (so that small problems need no launch more).
template <int BT>
__global__ __launch_bounds__(256, 4) void k_xent_grad32(const float *x, const float *w, int64_t ld, const Labels lab,
                                                     const float *__restrict__ lse, const float *__restrict__ dloss,
                                                     float *__restrict__ g, float *__restrict__ xc, int64_t T,
                                                     int64_t D, int64_t v0, int64_t nv) {
    using P = Tile32<BT>;
    constexpr int TM = P::TM;
    __shared__ f4 lds[2][2][BT * 8];
    const int64_t id = block_id(), tiles = (T + BT - 1) / BT, tile = id / tiles;  // of the vocabulary; tokens run first
    const int64_t m0 = (id - tile * tiles) * BT, n0 = tile * BT;
    if (n0 >= nv) return;
    P tile32;
    tile32.run(Operand32<false, BT>{x + m0 * ld, ld, (T - m0) * ld, T - m0, D},
               Operand32<false, BT>{w + (v0 + n0) * ld, ld, (nv - n0) * ld, nv - n0, D}, D, lds);
    const auto &acc = tile32.acc;
    const int lane = threadIdx.x & 63, wm = P::row0(), wn = P::col0();
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t t = m0 + wm + i * 16 + (lane >> 4) * 4 + e;
            if (t >= T) continue;
            const int64_t l = lab.of(t);
            const float ls = lse[t], dl = l >= 0 ? dloss[t] : 0.f;
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const int64_t c = n0 + wn + j * 16 + (lane & 15);
                float q = __builtin_amdgcn_exp2f((acc[i][j][e] - ls) * kLog2e);
                if (v0 + c == l) q -= 1.f;
                if (c < nv) g[t * nv + c] = l >= 0 ? q * dl : 0.f;
            }
        }
    if (xc) {
        const int n = (int)((T - m0 < BT ? T - m0 : BT) * ld), shares = (int)((nv + BT - 1) / BT);
        for (int i = (int)tile * 256 + (int)threadIdx.x; i < n; i += shares * 256)
            xc[m0 * ld + i] = lab.of(m0 + i / (int)ld) >= 0 ? x[m0 * ld + i] : 0.f;
    }
}

// dx and dw of a piece in one launch: first the tiles of
// dx[t][d] += sum_v G[t][v] w[v][d], then those of dw[v][d] = sum_t G[t][v] x[t][d].
// As in 16 bits, the v may be cut into `splits` ranges of kx with sums of their
// own in accum.
template <int BT>
__global__ __launch_bounds__(256) void k_xent_products32(const float *x, const float *w, int64_t ld, const float *g,
                                                         float *__restrict__ dx, float *__restrict__ dw,
                                                         float *__restrict__ accum, int64_t T, int64_t D, int64_t nv,
                                                         int64_t kx, int splits, int64_t ndx, int first) {
    using P = Tile32<BT>;
    constexpr int TM = P::TM;
    __shared__ f4 lds[2][2][BT * 8];
    const int64_t cols = (D + BT - 1) / BT, block = block_id();
    const bool is_dx = block < ndx;
    const int64_t tiles = ndx / splits, part = is_dx ? block / tiles : 0, k0 = part * kx;
    const int64_t id = is_dx ? block - part * tiles : block - ndx, m0 = id / cols * BT, n0 = id % cols * BT;
    if (!is_dx && m0 >= nv) return;
    const int64_t kn = nv - k0 < kx ? nv - k0 : kx;
    const int64_t ng = T * nv > 4 ? T * nv : 4;  // (there is room for four)
    P tile32;
    if (is_dx)
        tile32.run(Operand32<false, BT>{g + m0 * nv + k0, nv, ng - m0 * nv - k0, T - m0, kn},
                   Operand32<true, BT>{w + k0 * ld + n0, ld, (nv - k0) * ld - n0, D - n0, kn}, kn, lds);
    else
        tile32.run(Operand32<true, BT>{g + m0, nv, ng - m0, nv - m0, T},
                   Operand32<true, BT>{x + n0, ld, T * ld - n0, D - n0, T}, T, lds);
    const auto &acc = tile32.acc;
    const int lane = threadIdx.x & 63, wm = P::row0(), wn = P::col0();
    const int64_t M = is_dx ? T : nv;
    float *const out = is_dx ? (accum ? accum + part * T * D : dx) : dw;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t m = m0 + wm + i * 16 + (lane >> 4) * 4 + e, n = n0 + wn + j * 16 + (lane & 15);
                if (m >= M || n >= D) continue;
                const float q = acc[i][j][e];
                out[m * D + n] = is_dx && !first ? out[m * D + n] + q : q;
            }
}

// ------------------------------------------------------------ 16-bit kernels

// Blocks go to the eight XCDs in turn; each XCD takes one stretch of the
// tiles, so that neighbours in memory meet in its L2.
__device__ __forceinline__ int64_t xcd_order(int64_t id, int64_t n) {
    const int64_t x = id & 7, per = n >> 3, more = n & 7;
    return x * per + (x < more ? x : more) + (id >> 3);
}
// Tile `id` of rows x cols tiles: groups of four rows go through all columns.
__device__ __forceinline__ void tile_of(int64_t id, int64_t rows, int64_t cols, int64_t &r, int64_t &c) {
    const int64_t g = id / (4 * cols), left = rows - 4 * g, h = left < 4 ? left : 4, k = id - 4 * g * cols;
    c = k / h;
    r = 4 * g + k - c * h;
}

// Tiles of side BT: large ones need the least traffic per product (eight waves
// with 128 x 64 parts each), small ones fill the chip when there are few.
template <int IO, int BT, bool AK, bool BK>
using Side = std::conditional_t<
    BT == 256, Tile<IO, 256, 256, 2, 4, 64, 2, AK, BK>,
    std::conditional_t<BT == 128, Tile<IO, 128, 128, 2, 2, 64, 2, AK, BK>, Tile<IO, 64, 64, 2, 2, 64, 3, AK, BK>>>;
template <int IO, int BT>
using LogitTile = Side<IO, BT, false, false>;
template <int IO, int BT, bool G_KMAJOR>
using GradTile = Side<IO, BT, true, G_KMAJOR>;
template <int BT>
constexpr int kThreads16 = BT == 256 ? 512 : 256;

// As k_xent_stats32, with w's rows as the tile's rows and tokens as its columns:
// a lane holds four consecutive rows of w for a token, so it reduces most of the
// tile's rows by itself and two shuffles finish a wave's.  The reduction (one
// exponential per logit) takes about 150 of 655 us at 8192 x 768 x 50021, which
// one block per compute unit does not hide.
template <int IO, int BT>
__global__ __launch_bounds__(kThreads16<BT>, BT == 256 ? 1 : 2) void k_xent_stats16(const char *x, const char *w, int64_t ld,
                                                                       const Labels lab, float2 *__restrict__ part,
                                                                       float *__restrict__ hit, int64_t T, int64_t V) {
    using L = LogitTile<IO, BT>;
    __shared__ __align__(16) char lds[L::kLds];
    const int64_t rows = (V + L::BM - 1) / L::BM, cols = (T + L::BN - 1) / L::BN;
    int64_t rt, ct;
    if (block_id() >= rows * cols) return;
    tile_of(xcd_order(block_id(), rows * cols), rows, cols, rt, ct);
    const int64_t v0 = rt * L::BM, t0 = ct * L::BN;
    typename L::OA a;
    typename L::OB b;
    a.init(w + v0 * ld, ld, V - v0, 0);
    b.init(x + t0 * ld, ld, T - t0, 0);
    const int lane = threadIdx.x & 63, g = lane >> 4;
    int lr[L::TN];  // the labels' rows in this tile, or -1; loaded ahead of the products
#pragma unroll
    for (int j = 0; j < L::TN; ++j) {
        const int64_t t = t0 + L::col0() + j * 16 + (lane & 15), lb = (t < T ? lab.of(t) : -1) - v0;
        lr[j] = lb >= 0 && lb < L::BM ? (int)lb : -1;
        asm volatile("" : "+v"(lr[j]));
    }
    L tile;
    tile.run(a, b, ld / 2 / L::KS, lds);
    __syncthreads();
    float2(*const red)[L::BN] = (float2(*)[L::BN])lds;  // [wave row][token]
    const bool whole = v0 + L::BM <= V;
#pragma unroll
    for (int j = 0; j < L::TN; ++j) {
        const int col = L::col0() + j * 16 + (lane & 15);
        float m = -INFINITY, s = 0.f;
#pragma unroll
        for (int i = 0; i < L::TM; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = L::row0() + i * 16 + g * 4 + e;
                if (!whole && v0 + row >= V) tile.acc[i][j][e] = -INFINITY;
                m = fmaxf(m, tile.acc[i][j][e]);
            }
        if (__any(lr[j] >= 0)) {
            float found = 0.f;
#pragma unroll
            for (int i = 0; i < L::TM; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (L::row0() + i * 16 + g * 4 + e == lr[j]) found = tile.acc[i][j][e];
            if (lr[j] >= L::row0() && lr[j] < L::row0() + L::TM * 16 && (lr[j] >> 2 & 3) == g) hit[t0 + col] = found;
        }
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        const float mm = m == -INFINITY ? 0.f : m * kLog2e;
#pragma unroll
        for (int i = 0; i < L::TM; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s += __builtin_amdgcn_exp2f(fmaf(tile.acc[i][j][e], kLog2e, -mm));
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if (g == 0) red[L::row0() / (L::TM * 16)][col] = make_float2(m, s);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < L::BN; c += L::NT) {
        float2 q = red[0][c];
#pragma unroll
        for (int r = 1; r < L::BM / (L::TM * 16); ++r) q = join(q, red[r][c]);
        if (t0 + c < T) part[rt * T + t0 + c] = q;
    }
}

// G of the vocabulary piece [v0, v0 + nv): g[t][v - v0], rows of ldg elements;
// zero for nv <= v - v0 < ldg and for T <= t < Tp.  400 us for 8192 x 25088 of
// width 768, about 70 more than the statistics' half: writing 411 MB.
template <int IO, int BT>
__global__ __launch_bounds__(kThreads16<BT>, BT == 256 ? 1 : 2) void k_xent_grad16(const char *x, const char *w, int64_t ld,
                                                                      const Labels lab, const float *__restrict__ lse,
                                                                      const float *__restrict__ dloss,
                                                                      const float *__restrict__ scale,
                                                                      typename io_elem<IO>::T *__restrict__ gout,
                                                                      int64_t ldg, int64_t T, int64_t Tp, int64_t v0,
                                                                      int64_t nv) {
    using L = LogitTile<IO, BT>;
    using E = typename io_elem<IO>::T;
    __shared__ __align__(16) char lds[L::kLds];
    const int64_t rows = (nv + L::BM - 1) / L::BM, cols = (T + L::BN - 1) / L::BN;
    int64_t rt, ct;
    if (block_id() >= rows * cols) return;
    tile_of(xcd_order(block_id(), rows * cols), rows, cols, rt, ct);
    const int64_t r0 = rt * L::BM, t0 = ct * L::BN;
    typename L::OA a;
    typename L::OB b;
    a.init(w + (v0 + r0) * ld, ld, nv - r0, 0);
    b.init(x + t0 * ld, ld, T - t0, 0);
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const float top = scale[0];
    const bool whole = r0 + L::BM <= nv;
    // of this lane's tokens, loaded ahead of the products: the label's row in
    // the tile (or -1), the log-sum, the weight (0 where the token does not count)
    int lr[L::TN];
    float ls[L::TN], dl[L::TN];
    bool on[L::TN];
#pragma unroll
    for (int j = 0; j < L::TN; ++j) {
        const int64_t t = t0 + L::col0() + j * 16 + (lane & 15), label = t < T ? lab.of(t) : -1, lb = label - v0 - r0;
        on[j] = label >= 0;
        lr[j] = lb >= 0 && lb < L::BM ? (int)lb : -1;
        ls[j] = t < T ? lse[t] * kLog2e : 0.f;
        dl[j] = on[j] ? weight<IO>(dloss[t], top) : 0.f;
        asm volatile("" : "+v"(lr[j]), "+v"(ls[j]), "+v"(dl[j]));
    }
    L tile;
    tile.run(a, b, ld / 2 / L::KS, lds);
#pragma unroll
    for (int j = 0; j < L::TN; ++j) {
        const int64_t t = t0 + L::col0() + j * 16 + (lane & 15);
        const bool any = __any(lr[j] >= 0);
#pragma unroll
        for (int i = 0; i < L::TM; ++i) {
            const int row = L::row0() + i * 16 + g * 4;
            float q[4];
            Pack<E, 4> o;
#pragma unroll
            for (int e = 0; e < 4; ++e) q[e] = __builtin_amdgcn_exp2f(fmaf(tile.acc[i][j][e], kLog2e, -ls[j]));
            if (any) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (row + e == lr[j]) q[e] -= 1.f;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                q[e] = on[j] ? q[e] * dl[j] : 0.f;
                if (!whole && r0 + row + e >= nv) q[e] = 0.f;
                o.v[e] = from_f<IO>(q[e]);
            }
            if (t < Tp && r0 + row < ldg) *reinterpret_cast<Pack<E, 4> *>(gout + t * ldg + r0 + row) = o;
        }
    }
}

// dx and dw of a piece in one launch: blocks 0 .. ndx-1 form dx[t][d] +=
// sum_v G[t][v] w[v][d], the others dw[v][d] = sum_t G[t][v] x[t][d].  The
// tile's rows are d (so that a lane stores four consecutive values), its
// columns t or v.  dx has few tiles where D is small: the piece's v are cut
// into `splits` ranges of kx, each with a sum of its own in accum over all
// pieces; without a cut and with one piece dx is stored at once.  dw has few
// tiles where V and D are small: the tokens are cut into `wsplits` ranges of
// kw, each with a sum of its own in waccum.
template <int IO, int BT>
__global__ __launch_bounds__(kThreads16<BT>, BT == 256 ? 1 : 2) void k_xent_products16(
    const char *x, const char *w, int64_t ld, const char *g, int64_t ldg, typename io_elem<IO>::T *__restrict__ dx,
    typename io_elem<IO>::T *__restrict__ dw, float *__restrict__ accum, float *__restrict__ waccum,
    const float *__restrict__ scale, int64_t T, int64_t Tp, int64_t D, int64_t nv, int64_t kv, int64_t kx, int splits,
    int64_t kw, int wsplits, int64_t ndx, int first, int whole) {
    using PX = GradTile<IO, BT, false>;
    using PW = GradTile<IO, BT, true>;
    __shared__ __align__(16) char lds[PX::kLds];
    const int64_t rows = (D + PX::BM - 1) / PX::BM;
    const int lane = threadIdx.x & 63;
    const float down = scale[1];
    int64_t rt, ct;
    const int64_t block = block_id();
    if (block < ndx) {
        const int64_t cols = ndx / rows / splits, id = xcd_order(block, ndx), part = id / (rows * cols);
        tile_of(id - part * rows * cols, rows, cols, rt, ct);
        const int64_t d0 = rt * PX::BM, t0 = ct * PX::BN, k0 = part * kx, kn = kv - k0 < kx ? kv - k0 : kx;
        typename PX::OA a;
        typename PX::OB b;
        a.init(w + k0 * ld + d0 * 2, ld, ld - d0 * 2, nv - k0);
        b.init(g + t0 * ldg * 2 + k0 * 2, ldg * 2, T - t0, 0);
        PX tile;
        tile.run(a, b, kn / PX::KS, lds);
        float *const sum = accum + part * T * D;
#pragma unroll
        for (int i = 0; i < PX::TM; ++i)
#pragma unroll
            for (int j = 0; j < PX::TN; ++j) {
                const int64_t d = d0 + PX::row0() + i * 16 + (lane >> 4) * 4;
                const int64_t t = t0 + PX::col0() + j * 16 + (lane & 15);
                if (t >= T || d >= D) continue;
                float q[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) q[e] = tile.acc[i][j][e];
                if (whole) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) q[e] *= down;
                    st_row<IO, 4>(dx + t * D + d, q, D - d);
                    continue;
                }
                if (!first) {
                    float o[4];
                    ld_row<IO_F32, 4>(sum + t * D + d, o, D - d);
#pragma unroll
                    for (int e = 0; e < 4; ++e) q[e] += o[e];
                }
                st_row<IO_F32, 4>(sum + t * D + d, q, D - d);
            }
    } else {
        const int64_t cols = (nv + PW::BN - 1) / PW::BN, n = rows * cols * wsplits;
        if (block - ndx >= n) return;
        const int64_t id = xcd_order(block - ndx, n), part = id / (rows * cols);
        tile_of(id - part * rows * cols, rows, cols, rt, ct);
        const int64_t d0 = rt * PW::BM, c0 = ct * PW::BN, k0 = part * kw, kn = Tp - k0 < kw ? Tp - k0 : kw;
        typename PW::OA a;
        typename PW::OB b;
        a.init(x + k0 * ld + d0 * 2, ld, ld - d0 * 2, T - k0);
        b.init(g + k0 * ldg * 2 + c0 * 2, ldg * 2, (ldg - c0) * 2, Tp - k0);
        PW tile;
        tile.run(a, b, kn / PW::KS, lds);
        float *const sum = waccum + part * nv * D;
#pragma unroll
        for (int i = 0; i < PW::TM; ++i)
#pragma unroll
            for (int j = 0; j < PW::TN; ++j) {
                const int64_t d = d0 + PW::row0() + i * 16 + (lane >> 4) * 4;
                const int64_t v = c0 + PW::col0() + j * 16 + (lane & 15);
                if (v >= nv || d >= D) continue;
                float q[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) q[e] = wsplits > 1 ? tile.acc[i][j][e] : tile.acc[i][j][e] * down;
                if (wsplits > 1) st_row<IO_F32, 4>(sum + v * D + d, q, D - d);
                else st_row<IO, 4>(dw + v * D + d, q, D - d);
            }
    }
}

// dx (or dw) from the sums of its ranges, in order; n values each.
template <int IO>
__global__ __launch_bounds__(256) void k_xent_dx(const float *__restrict__ accum, const float *__restrict__ scale,
                                                 typename io_elem<IO>::T *__restrict__ dx, int64_t n, int splits) {
    const int64_t i = (block_id() * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    float s[4];
    ld_row<IO_F32, 4>(accum + i, s, n - i);
#pragma unroll 4
    for (int k = 1; k < splits; ++k) {
        float o[4];
        ld_row<IO_F32, 4>(accum + k * n + i, o, n - i);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += o[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (scale) s[e] *= scale[1];
    st_row<IO, 4>(dx + i, s, n - i);
}

template <class E>
__global__ __launch_bounds__(256) void k_xent_pad(const E *__restrict__ src, E *__restrict__ dst, int64_t R,
                                                  int64_t C, int64_t ldd) {
    pad_vector(src, dst, R, C, ldd, block_id() * 256 + threadIdx.x, [](int64_t) { return true; });
}

// dw of no tokens.
template <class E>
__global__ __launch_bounds__(256) void k_xent_zero(E *__restrict__ p, int64_t n) {
    const int64_t i = block_id() * 256 + threadIdx.x;
    if (i < n) p[i] = (E)0;
}

int64_t blocks(int64_t n, int64_t per) { return (n + per - 1) / per; }

// x or w with rows of whole slabs: as it is, or copied.
template <int IO>
hipError_t padded(const void *src, char *dst, int64_t R, int64_t D, int64_t kD, const char **out, hipStream_t s) {
    using E = typename io_elem<IO>::T;
    *out = (const char *)src;
    if (kD == D) return hipSuccess;
    *out = dst;
    return launch(k_xent_pad<E>, grid_of(blocks(R * kD, 256 * 16 / (int64_t)sizeof(E))), dim3(256), 0, s, (const E *)src, (E *)dst, R, D, kD);
}

template <int IO>
hipError_t fwd_io(const void *x, const void *w, const Labels &lab, float *loss, float *lse, int64_t T, int64_t D,
                  int64_t V, char *ws, hipStream_t s) {
    constexpr bool wide = IO == IO_F32;
    const XentPlan p = plan(T, D, V, wide, false, ws);
    const int64_t ld = p.kD * (int64_t)sizeof(typename io_elem<IO>::T);
    const char *xr, *wr;
    hipError_t e = padded<IO>(x, p.xp, T, D, p.kD, &xr, s);
    if (e == hipSuccess) e = padded<IO>(w, p.wp, V, D, p.kD, &wr, s);
    if (e != hipSuccess) return e;
    if constexpr (IO == IO_F32) {
        const int64_t bt = side32(T, V);
        e = launch(bt == 32 ? k_xent_stats32<32> : k_xent_stats32<64>, grid_of(blocks(T, bt) * blocks(V, bt)), dim3(256), 0, s,
                   (const float *)xr, (const float *)wr, p.kD, lab, (float2 *)p.part, p.hit, T, D, V);
    } else {
        const int64_t bt = side16(T, V);
        e = launch(bt == 256 ? k_xent_stats16<IO, 256> : (bt == 128 ? k_xent_stats16<IO, 128> : k_xent_stats16<IO, 64>),
                   grid_of(blocks(V, bt) * blocks(T, bt)), dim3(bt == 256 ? 512 : 256), 0, s, xr, wr, ld, lab, (float2 *)p.part, p.hit, T, V);
    }
    if (e != hipSuccess) return e;
    return launch(k_xent_join, grid_of(blocks(T, 64)), dim3(1024), 0, s, (float2 *)p.part, p.hit, lab, loss, lse, T, p.tiles);
}

template <int IO>
hipError_t bwd_io(const void *x, const void *w, const Labels &lab, const float *lse, const float *dloss, void *dx,
                  void *dw, int64_t T, int64_t D, int64_t V, char *ws, hipStream_t s) {
    using E = typename io_elem<IO>::T;
    const int64_t es = sizeof(E);
    if (T == 0) return launch(k_xent_zero<E>, grid_of(blocks(V * D, 256)), dim3(256), 0, s, (E *)dw, V * D);
    constexpr bool wide = IO == IO_F32;
    const XentPlan p = plan(T, D, V, wide, true, ws);
    const int64_t ld = p.kD * es;
    const char *xr = p.xc, *wr;
    hipError_t e = padded<IO>(w, p.wp, V, D, p.kD, &wr, s);
    if (e == hipSuccess) {
        if constexpr (IO == IO_F32) e = padded<IO>(x, p.xp, T, D, p.kD, &xr, s);
        else
            e = launch(k_xent_tokens16<IO>, grid_of(1 + blocks(T * p.kD, 1024 * 8)), dim3(1024), 0, s, (const E *)x, (E *)p.xc,
                       D, p.kD, dloss, lab, p.scale, T);
    }
    for (int64_t i = 0; i < p.pieces && e == hipSuccess; ++i) {
        const int64_t v0 = i * p.piece, nv = V - v0 < p.piece ? V - v0 : p.piece;
        const int first = i == 0, last = i + 1 == p.pieces;
        if constexpr (IO == IO_F32) {
            const float *const xf = (const float *)xr, *const wf = (const float *)wr;
            int64_t bt = side32(T, nv);
            e = launch(bt == 32 ? k_xent_grad32<32> : k_xent_grad32<64>, grid_of(blocks(T, bt) * blocks(nv, bt)), dim3(256), 0, s,
                       xf, wf, p.kD, lab, lse, dloss, (float *)p.g, first ? (float *)p.xc : nullptr, T, D, v0, nv);
            if (e != hipSuccess) break;
            bt = p.side;
            const int64_t parts = (nv + p.range - 1) / p.range;  // (a shorter last piece has fewer)
            const int64_t ndx = blocks(T, bt) * blocks(D, bt) * parts, ndw = blocks(nv, bt) * blocks(D, bt);
            e = launch(bt == 32 ? k_xent_products32<32> : k_xent_products32<64>, grid_of(ndx + ndw), dim3(256), 0, s,
                       (const float *)p.xc, wf + v0 * p.kD, p.kD, (const float *)p.g, (float *)dx, (float *)dw + v0 * D, p.accum, T, D, nv,
                       p.range, (int)parts, ndx, first);
            if (e == hipSuccess && last && p.accum)
                e = launch(k_xent_dx<IO>, grid_of(blocks(T * D, 1024)), dim3(256), 0, s, p.accum, p.scale, (E *)dx, T * D,
                           (int)p.ranges);
        } else {
            const int64_t kv = ceil_to(nv, 64);
            int64_t bt = side16(T, nv);
            e = launch(bt == 256 ? k_xent_grad16<IO, 256> : (bt == 128 ? k_xent_grad16<IO, 128> : k_xent_grad16<IO, 64>),
                       grid_of(blocks(nv, bt) * blocks(T, bt)), dim3(bt == 256 ? 512 : 256), 0, s, xr, wr,
                       ld, lab, lse, dloss, p.scale, (E *)p.g, kv, T, p.Tp, v0, nv);
            if (e != hipSuccess) break;
            // ranges of whole slabs, as long as the first piece's (a shorter last piece has fewer)
            const int64_t kx = p.range, parts = (kv + kx - 1) / kx;
            bt = p.side;
            const int64_t rows = blocks(D, bt), ndx = rows * blocks(T, bt) * parts, ndw = rows * blocks(nv, bt) * p.wranges;
            e = launch(bt == 256 ? k_xent_products16<IO, 256>
                                 : (bt == 128 ? k_xent_products16<IO, 128> : k_xent_products16<IO, 64>),
                       grid_of(ndx + ndw), dim3(bt == 256 ? 512 : 256), 0, s, xr, wr + v0 * ld, ld, p.g,
                       kv, (E *)dx, (E *)dw + v0 * D, p.accum, p.waccum, p.scale, T, p.Tp, D, nv, kv, kx, (int)parts, p.wrange, (int)p.wranges, ndx,
                       first, p.accum ? 0 : 1);
            if (e == hipSuccess && last && p.accum)
                e = launch(k_xent_dx<IO>, grid_of(blocks(T * D, 1024)), dim3(256), 0, s, p.accum, p.scale, (E *)dx, T * D,
                           (int)p.ranges);
            if (e == hipSuccess && p.waccum)
                e = launch(k_xent_dx<IO>, grid_of(blocks(nv * D, 1024)), dim3(256), 0, s, p.waccum, p.scale, (E *)dw + v0 * D,
                           nv * D, (int)p.wranges);
        }
    }
    return e;
}

}  // namespace

size_t linear_xent_workspace(int64_t T, int64_t D, int64_t V, int io, bool bwd) {
    return xent::plan(T, D, V, io == IO_F32, bwd, nullptr).bytes;
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
