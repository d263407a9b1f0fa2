// embed.hip -- rows of a table by token, scaled, and the table's gradient.
//
//   y[t] = scale w[tok[t]],   dw[v] = scale sum_{t: tok[t] = v} dy[t]
// A token outside the table gives a zero row and no gradient.  Both are copies
// with a little arithmetic: HBM bound.  A row's sum runs over its tokens in a
// fixed order (that of time, or by units of it), in fp32, and is rounded once:
// equal calls give equal bits.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "lm_device.h"
#include "lm_internal.h"

namespace h3c {
namespace {

constexpr int V = 8;

// One wave per token: 8192 x 768 in bf16 7.6 us, 65536 x 1024 in fp16 58 us (268 MB, 4.6 TB/s).
template <int IO>
__global__ __launch_bounds__(256) void k_embed(const int64_t *__restrict__ tok, const typename io_elem<IO>::T *__restrict__ w,
                                               typename io_elem<IO>::T *__restrict__ y, int64_t T, int64_t D, int64_t vocab,
                                               float scale) {
    const int64_t t = block_id() * 4 + (threadIdx.x >> 6);
    if (t >= T) return;
    const int64_t id = tok[t];
    const bool in = id >= 0 && id < vocab;
    for (int64_t c = (threadIdx.x & 63) * V; c < D; c += 64 * V) {
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.f;
        if (in) ld_row<IO, V>(w + id * D + c, v, D - c);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= scale;
        st_row<IO, V>(y + t * D + c, v, D - c);
    }
}

// The gradient goes by the tokens in sorted order:
//   k_embed_cut   pieces of kPiece tokens, each sorted by the upper bits of its ids into
//                 at most 256 ranges of ids
//   k_embed_sort  a range's entries of all pieces, sorted by the other bits; for every id
//                 that occurs, where its entries stand
//   k_embed_hot   ids of more than kUnit entries: sums of the entries in each kUnit places
//   k_embed_rows  the table's rows, from their entries or from such sums
// Every sort is stable, so an id's entries are in the order of time.  The rows of dy are read once, the table is written
// once, 16 bytes per token sorted: HBM bound where there are many columns.  8192 tokens of 768 channels, 50021 ids, bf16:
// cut 5 us, sort 11, hot 6, rows 28 (90 MB, 3.2 TB/s); 65536 of 1024, 32768 ids, a third one id, fp16: 5, 56, 30 and
// 68 us (the sort's length is that of its longest range: an id that fills a third of the entries is in one block's hands).
constexpr int kPiece = 1024, kUnit = 32, kSort = 1024, kCols = 64 * V;

struct Sorted {
    int2 *buf[3];    // (id, time) of every entry: by pieces, then [1] and [2] in turn, by ranges
    int *off;        // [ranges + 1][pieces]: where a range begins in a piece
    int2 *span;      // [vocabulary]: where an id's entries begin and end (0, 0: none)
    int64_t *total;  // entries
    float *part;     // [units][2][D]: sums of a unit's first id, and of its last if it is another
    int64_t pieces, ranges, units;
    int shift, passes;
    __device__ __forceinline__ const int2 *done() const { return buf[1 + (passes & 1)]; }
};

// Lanes of the wave whose 8-bit digit is this one's, among those that are `on`.
__device__ __forceinline__ uint64_t same_digit(int d, bool on) {
    uint64_t m = __ballot(on);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint64_t bit = __ballot((d >> i) & 1);
        m &= (d >> i) & 1 ? bit : ~bit;
    }
    return m;
}
__device__ __forceinline__ int lanes_before(uint64_t m) { return __popcll(m & ((1ull << (threadIdx.x & 63)) - 1)); }

// The counts of every wave and digit become the entries of the digit in earlier waves;
// first[d] is where digit d begins.
template <int NT>
__device__ __forceinline__ void places(int (*cnt)[256], int *first) {
    const int d = threadIdx.x;
    if (d < 256) {
        int total = 0;
        for (int w = 0; w < NT / 64; ++w) {
            const int n = cnt[w][d];
            cnt[w][d] = total;
            total += n;
        }
        first[d] = total;
    }
    __syncthreads();
    if (d < 64) {  // 256 counts, four per lane
        int v[4], sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = sum;
            sum += first[4 * d + i];
        }
        int run = sum;
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) {
            const int u = __shfl_up(run, k);
            if (d >= k) run += u;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) first[4 * d + i] = v[i] + run - sum;
        if (d == 63) first[256] = run;
    }
    __syncthreads();
}

__global__ __launch_bounds__(256) void k_embed_cut(const int64_t *__restrict__ tok, int64_t T, int64_t vocab, Sorted s) {
    __shared__ int cnt[4][256], first[257];
    const int64_t piece = block_id(), blocks = (int64_t)gridDim.x * gridDim.z;
    for (int64_t v = piece * 256 + threadIdx.x; v < vocab; v += blocks * 256) s.span[v] = int2{0, 0};
    if (piece >= s.pieces) return;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    for (int i = threadIdx.x; i < 4 * 256; i += 256) cnt[i >> 8][i & 255] = 0;
    __syncthreads();
    constexpr int R = kPiece / 256;
    const int64_t t0 = piece * kPiece + wave * (kPiece / 4) + lane;
    int id[R], rank[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t t = t0 + i * 64, v = t < T ? tok[t] : -1;
        id[i] = v >= 0 && v < vocab ? (int)v : -1;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const bool on = id[i] >= 0;
        const int d = on ? id[i] >> s.shift : 0;
        const uint64_t same = same_digit(d, on);
        rank[i] = cnt[wave][d] + lanes_before(same);
        __builtin_amdgcn_wave_barrier();
        if (on && lanes_before(same) == 0) cnt[wave][d] += __popcll(same);
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    places<256>(cnt, first);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (id[i] < 0) continue;
        const int d = id[i] >> s.shift;
        s.buf[0][piece * kPiece + first[d] + cnt[wave][d] + rank[i]] = int2{id[i], (int)(t0 + i * 64)};
    }
    for (int64_t r = threadIdx.x; r <= s.ranges; r += 256) s.off[r * s.pieces + piece] = first[r];
}

// One stable pass over n entries by the digit from `bit` on; a wave has consecutive ones, whose loads go out
// kBatch at a time.
constexpr int kBatch = 8;
__device__ __forceinline__ void sort_pass(const int2 *from, int2 *to, int64_t n, int bit, int (*cnt)[256], int *first) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t per = (n + kSort - 1) / kSort * 64, lo = wave * per, hi = lo + per < n ? lo + per : n;
    for (int i = threadIdx.x; i < kSort / 64 * 256; i += kSort) cnt[i >> 8][i & 255] = 0;
    __syncthreads();
    for (int place = 0; place < 2; ++place) {
        for (int64_t i0 = lo; i0 < hi; i0 += 64 * kBatch) {
            int2 e[kBatch];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) e[q] = from[i0 + q * 64 + lane < hi ? i0 + q * 64 + lane : lo];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                if (i0 + q * 64 >= hi) break;
                const bool on = i0 + q * 64 + lane < hi;
                const int d = (e[q].x >> bit) & 255, d0 = __builtin_amdgcn_readfirstlane(d);
                // (one id most often where there are many entries)
                const uint64_t all = __ballot(on);
                const bool one = __ballot(on && d != d0) == 0;
                if (!place) {
                    if (one) {
                        if (lane == 0) cnt[wave][d0] += __popcll(all);
                    } else if (on) {
                        atomicAdd(&cnt[wave][d], 1);
                    }
                    continue;
                }
                const uint64_t same = one ? all : same_digit(d, on);
                const int before = lanes_before(same), have = cnt[wave][d];
                __builtin_amdgcn_wave_barrier();
                if (on) to[first[d] + have + before] = e[q];
                if (on && before == 0) cnt[wave][d] = have + __popcll(same);
                __builtin_amdgcn_wave_barrier();
            }
        }
        __syncthreads();
        if (!place) places<kSort>(cnt, first);
    }
}

__global__ __launch_bounds__(kSort) void k_embed_sort(Sorted s) {
    __shared__ int cnt[kSort / 64][256], first[257];
    __shared__ int64_t sums[kSort / 64], to[kSort];
    __shared__ int from[kSort], many[kSort];
    const int64_t r = blockIdx.x;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    // where the range begins among all entries
    int64_t base = 0, n = 0;
    for (int64_t p = threadIdx.x; p < s.pieces; p += kSort) base += s.off[r * s.pieces + p];
    for (int d = 32; d > 0; d >>= 1) base += __shfl_xor(base, d);
    if (lane == 0) sums[wave] = base;
    __syncthreads();
    base = 0;
    for (int w = 0; w < kSort / 64; ++w) base += sums[w];
    __syncthreads();
    // its entries from the pieces, in order: a thread has a piece's place, the waves copy pieces in turn
    for (int64_t p0 = 0; p0 < s.pieces; p0 += kSort) {
        const int64_t p = p0 + threadIdx.x;
        const int lo = p < s.pieces ? s.off[r * s.pieces + p] : 0, hi = p < s.pieces ? s.off[(r + 1) * s.pieces + p] : 0;
        int64_t run = hi - lo;
        for (int k = 1; k < 64; k <<= 1) {
            const int64_t u = __shfl_up(run, k);
            if (lane >= k) run += u;
        }
        if (lane == 63) sums[wave] = run;
        __syncthreads();
        int64_t at = base + n + run - (hi - lo), all = 0;
        for (int w = 0; w < kSort / 64; ++w) {
            if (w < wave) at += sums[w];
            all += sums[w];
        }
        from[threadIdx.x] = lo;
        many[threadIdx.x] = hi - lo;
        to[threadIdx.x] = at;
        __syncthreads();
        const int last = (int)std::min<int64_t>(kSort, s.pieces - p0);
        for (int q = wave; q < last; q += kSort / 64) {
            const int2 *src = s.buf[0] + (p0 + q) * kPiece + from[q];
            int2 *dst = s.buf[1] + to[q];
            const int m = many[q];
#pragma unroll 4
            for (int j = lane; j < m; j += 64) dst[j] = src[j];
        }
        __syncthreads();
        n += all;
    }
    __syncthreads();
    for (int i = 0; i < s.passes; ++i) sort_pass(s.buf[1 + (i & 1)] + base, s.buf[2 - (i & 1)] + base, n, 8 * i, cnt, first);
    const int2 *e = s.done() + base;
    for (int64_t i0 = threadIdx.x; i0 < n; i0 += kSort * kBatch) {
        int id[kBatch][3];
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const int64_t i = i0 + q * kSort + k - 1;
                id[q][k] = e[i < 0 ? 0 : i < n ? i : n - 1].x;
            }
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const int64_t i = i0 + q * kSort;
            if (i < n && (i == 0 || id[q][0] != id[q][1])) s.span[id[q][1]].x = (int)(base + i);
            if (i < n && (i == n - 1 || id[q][2] != id[q][1])) s.span[id[q][1]].y = (int)(base + i + 1);
        }
    }
    if (r == s.ranges - 1 && threadIdx.x == 0) *s.total = base + n;
}

// The sum of n rows of dy, n at most 64, in order: this lane's columns, c to c + V - 1.  t: the rows, lane by lane from
// `first` on.  DEEP rows are on their way at a time, their loads without branches: a vector that passes the row's end
// is taken to end with it, and where rows are not whole vectors all lanes sum theirs once more, element by element, which
// the lane of that vector takes (the gradient of 8192 tokens of 1031 channels, bf16: 78 us, of 1024 53; 65536 with
// padding, fp16: 216 and 130).
template <int IO, int DEEP>
__device__ __forceinline__ void sum_rows(int t, int first, int n, const typename io_elem<IO>::T *dy, int64_t D, int64_t c,
                                         float (&sum)[V]) {
    using T = typename io_elem<IO>::T;
    if (D >= V) {
        const int64_t cc = c + V <= D ? c : D - V;
        for (int j = 0; j < n; j += DEEP) {
            Pack<T, V> v[DEEP];
#pragma unroll
            for (int k = 0; k < DEEP; ++k)
                v[k] = *reinterpret_cast<const Pack<T, V> *>(dy + (int64_t)__builtin_amdgcn_readlane(t, first + (j + k < n ? j + k : n - 1)) * D + cc);
#pragma unroll
            for (int k = 0; k < DEEP; ++k)
                if (j + k < n) {
#pragma unroll
                    for (int i = 0; i < V; ++i) sum[i] += to_f<IO>(v[k].v[i]);
                }
        }
    }
    if (D % V != 0) {
        float one[V] = {};
        for (int j = 0; j < n; ++j) {
            const T *row = dy + (int64_t)__builtin_amdgcn_readlane(t, first + j) * D;
#pragma unroll
            for (int i = 0; i < V; ++i) one[i] += to_f<IO>(row[c + i < D ? c + i : D - 1]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] = c + V <= D ? sum[i] : one[i];
    }
}

// A wave per unit of places and kCols columns.
template <int IO>
__global__ __launch_bounds__(256) void k_embed_hot(const typename io_elem<IO>::T *__restrict__ dy, int64_t D, Sorted s) {
    const int64_t u = block_id() * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), p0 = u * kUnit;
    const int lane = threadIdx.x & 63;
    const int64_t total = *s.total, c = (int64_t)blockIdx.y * kCols + lane * V;
    if (p0 >= total) return;
    const int many = __builtin_amdgcn_readfirstlane((int)(total - p0 < kUnit ? total - p0 : kUnit));
    const int2 e = s.done()[p0 + (lane < many ? lane : 0)];
    const int ida = __builtin_amdgcn_readfirstlane(e.x), idb = __builtin_amdgcn_readlane(e.x, many - 1);
    const int2 spa = s.span[ida], spb = s.span[idb];
    for (int w = 0; w < (ida == idb ? 1 : 2); ++w) {
        const int2 sp = w ? spb : spa;
        if (sp.y - sp.x <= kUnit) continue;
        const int lo = sp.x > p0 ? (int)(sp.x - p0) : 0, hi = sp.y < p0 + many ? (int)(sp.y - p0) : many;
        float sum[V] = {};
        sum_rows<IO, 16>(e.y, __builtin_amdgcn_readfirstlane(lo), __builtin_amdgcn_readfirstlane(hi - lo), dy, D, c, sum);
        st_row<IO_F32, V>(s.part + (2 * u + w) * D + c, sum, D - c);
    }
}

// A wave has kIds ids and kCols columns.  Their places and the first 64 of their entries are loaded together; rows of
// absent ids are zeros at once.  The block's four waves join the sums of an id of many entries.
constexpr int kIds = 8;
template <int IO>
__global__ __launch_bounds__(256) void k_embed_rows(const typename io_elem<IO>::T *__restrict__ dy,
                                                    typename io_elem<IO>::T *__restrict__ dw, int64_t D, int64_t vocab,
                                                    float scale, Sorted s) {
    __shared__ float lds[4][kCols];
    __shared__ int2 spans[4 * kIds];
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t block0 = block_id() * 4 * kIds, id0 = block0 + wave * kIds, c = (int64_t)blockIdx.y * kCols + lane * V;
    if (block0 >= vocab) return;
    const int ids = (int)(vocab - id0 < kIds ? (vocab > id0 ? vocab - id0 : 0) : kIds);
    const int2 sp = lane < ids ? s.span[id0 + lane] : int2{0, 0};
    const int n = sp.y - sp.x;
    if (lane < kIds) spans[wave * kIds + lane] = sp;
    const auto put = [&](int q, const float (&sum)[V]) {
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = sum[i] * scale;
        st_row<IO, V>(dw + (id0 + q) * D + c, o, D - c);
    };
    const uint64_t some = __ballot(n > 0);
    if (some) {
        // the entries stand one after another: lane l has the l-th from the first id's first
        const int e0 = __builtin_amdgcn_readlane(sp.x, __builtin_ctzll(some));
        const int end = __builtin_amdgcn_readlane(sp.y, 63 - __builtin_clzll(some));
        const int t = s.done()[e0 + lane < end ? e0 + lane : e0].y;
        for (uint64_t left = some; left; left &= left - 1) {
            const int q = __builtin_ctzll(left), nq = __builtin_amdgcn_readlane(n, q), at = __builtin_amdgcn_readlane(sp.x, q) - e0;
            if (nq > kUnit) continue;
            int tq = t, first = at;
            if (at + nq > 64) {
                tq = lane < nq ? s.done()[e0 + at + lane].y : 0;
                first = 0;
            }
            float sum[V] = {};
            sum_rows<IO, 4>(tq, first, nq, dy, D, c, sum);
            put(q, sum);
        }
    }
    const float none[V] = {};
    for (int q = 0; q < ids; ++q)
        if (!((some >> q) & 1)) put(q, none);
    if (!__syncthreads_or(n > kUnit)) return;
    for (int w = 0; w < 4 * kIds; ++w) {
        const int2 x = spans[w];
        if (x.y - x.x <= kUnit) continue;
        // units first .. last; the first is the id's own only where it begins with it
        const int64_t u0 = x.x / kUnit, u1 = (x.y - 1) / kUnit + 1, per = (u1 - u0 + 3) / 4;
        const int64_t lo = u0 + wave * per, hi = lo + per < u1 ? lo + per : u1;
        float sum[V] = {};
#pragma unroll 8
        for (int64_t u = lo; u < hi; ++u) {
            float v[V];
            ld_row<IO_F32, V>(s.part + (2 * u + (u == u0 && x.x % kUnit != 0 ? 1 : 0)) * D + c, v, D - c);
#pragma unroll
            for (int i = 0; i < V; ++i) sum[i] += v[i];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) lds[wave][lane * V + i] = sum[i];
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int k = lane * V + i;
                sum[i] = (((lds[0][k] + lds[1][k]) + lds[2][k]) + lds[3][k]) * scale;
            }
            st_row<IO, V>(dw + (block0 + w) * D + c, sum, D - c);
        }
        __syncthreads();
    }
}

int64_t up(int64_t n) { return (n + 255) & ~(int64_t)255; }

// The workspace's parts from `base` on; its size.
int64_t plan(int64_t T, int64_t D, int64_t vocab, char *base, Sorted &s) {
    s.pieces = (T + kPiece - 1) / kPiece;
    s.units = (T + kUnit - 1) / kUnit;
    int bits = 0;
    while (bits < 31 && ((vocab - 1) >> bits) > 0) ++bits;
    s.shift = bits > 8 ? bits - 8 : 0;
    s.passes = (s.shift + 7) / 8;
    s.ranges = vocab > 0 ? ((vocab - 1) >> s.shift) + 1 : 0;
    int64_t at = 0;
    const auto take = [&](int64_t n) { char *p = base + at; at += up(n); return p; };
    for (int2 *&b : s.buf) b = (int2 *)take(s.pieces * kPiece * 8);
    s.off = (int *)take((s.ranges + 1) * s.pieces * 4);
    s.span = (int2 *)take(vocab * 8);
    s.total = (int64_t *)take(8);
    s.part = (float *)take(s.units * 2 * D * 4);
    return at;
}

template <int IO>
hipError_t fwd_io(const int64_t *tok, const void *w, void *y, int64_t T, int64_t D, int64_t vocab, float scale, hipStream_t s) {
    using E = typename io_elem<IO>::T;
    return launch(k_embed<IO>, grid_of((T + 3) / 4), dim3(256), 0, s, tok, (const E *)w, (E *)y, T, D, vocab, scale);
}
template <int IO>
hipError_t bwd_io(const int64_t *tok, const void *dy_, void *dw, int64_t T, int64_t D, int64_t vocab, float scale, void *ws,
                  hipStream_t st) {
    using E = typename io_elem<IO>::T;
    const E *dy = (const E *)dy_;
    Sorted s;
    plan(T, D, vocab, (char *)ws, s);
    const int64_t clear = std::min<int64_t>(1024, vocab / 2048 + 1);
    hipError_t e = launch(k_embed_cut, grid_of(std::max(s.pieces, clear)), dim3(256), 0, st, tok, T, vocab, s);
    if (e == hipSuccess) e = launch(k_embed_sort, dim3((unsigned)s.ranges), dim3(kSort), 0, st, s);
    if (e == hipSuccess && T > kUnit)
        e = launch(k_embed_hot<IO>, grid_of((s.units + 3) / 4, (unsigned)((D + kCols - 1) / kCols)), dim3(256), 0, st, dy, D, s);
    if (e == hipSuccess) e = launch(k_embed_rows<IO>, grid_of((vocab + 4 * kIds - 1) / (4 * kIds), (unsigned)((D + kCols - 1) / kCols)),
                   dim3(256), 0, st, dy, (E *)dw, D, vocab, scale, s);
    return e;
}

}  // namespace

size_t embed_bwd_workspace(int64_t T, int64_t D, int64_t vocab) {
    Sorted s;
    return (size_t)plan(T, D, vocab, nullptr, s);
}

hipError_t launch_embed(const int64_t *tok, const void *w, void *y, int64_t T, int64_t D, int64_t vocab, float scale, int io,
                        hipStream_t s) {
    switch (io) {
        case IO_F32: return fwd_io<IO_F32>(tok, w, y, T, D, vocab, scale, s);
        case IO_F16: return fwd_io<IO_F16>(tok, w, y, T, D, vocab, scale, s);
        default: return fwd_io<IO_BF16>(tok, w, y, T, D, vocab, scale, s);
    }
}

hipError_t launch_embed_bwd(const int64_t *tok, const void *dy, void *dw, int64_t T, int64_t D, int64_t vocab, float scale,
                            int io, void *ws, hipStream_t s) {
    switch (io) {
        case IO_F32: return bwd_io<IO_F32>(tok, dy, dw, T, D, vocab, scale, ws, s);
        case IO_F16: return bwd_io<IO_F16>(tok, dy, dw, T, D, vocab, scale, ws, s);
        default: return bwd_io<IO_BF16>(tok, dy, dw, T, D, vocab, scale, ws, s);
    }
}

}  // namespace h3c
