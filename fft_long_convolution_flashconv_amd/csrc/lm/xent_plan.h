// xent_plan.h -- how the linear cross entropy is cut: sides of its tiles, pieces
// of the vocabulary, ranges of its sums, and the workspace.  Host code without
// any HIP, so that a plan can be looked at without a GPU.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace h3c {
namespace xent {

constexpr int64_t kSlab16 = 64;  // 16-bit: elements that rows and sums are padded to

// Side of the fp32 tiles of a launch that forms n x m outputs, or of two that
// form n x m and o x m: 64, or 32 where those are too few for the compute
// units.  Tokens x width x vocabulary, us, sides 64 and 32:
//   logits:    517 x 201 x 1009  17.0  14.8 (144 tiles of 64)   1024 x 256 x 2048  23.3  26.9 (512)
//   backward:  517 x 201 x 1009  46.4  30.3 (100)               2048 x 512 x 8192   478   586 (1280)
inline int64_t side32(int64_t n, int64_t m, int64_t o = 0) {
    const auto tiles = [](int64_t r) { return (r + 63) / 64; };
    return (tiles(n) + tiles(o)) * tiles(m) < 256 ? 32 : 64;
}

// Side of the 16-bit tiles of n x m logits.  bf16, tokens x width x vocabulary,
// us of the forward pass, sides 256, 128 and 64:
//   300 x 256 x 1000    22.0  14.0   9.4  (24 tiles of 128)
//   300 x 777 x 8000    44.5  33.9  31.5  (189)
//   1000 x 777 x 8000   46.3  39.4  48.5  (504)
//   300 x 256 x 50021   38.8  36.5  46.8  (1173; 392 of 256)
//   1000 x 256 x 50021  64.8  70.4  94.1  (3128; 784 of 256)
inline int64_t side16(int64_t n, int64_t m) {
    const auto tiles = [&](int64_t bt) { return ((n + bt - 1) / bt) * ((m + bt - 1) / bt); };
    return tiles(256) >= 512 ? 256 : (tiles(128) >= 256 ? 128 : 64);
}

inline size_t align256(size_t n) { return (n + 255) / 256 * 256; }
inline int64_t ceil_to(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

struct XentPlan {
    int64_t kD;            // elements of a padded row of x and w
    int64_t Tp;            // tokens, padded (16-bit): rows of G
    int64_t piece, pieces; // vocabulary rows per piece
    int64_t tiles;         // pairs per token of the forward pass
    int64_t side;          // of the tiles of dx and dw
    int64_t range, ranges; // vocabulary rows whose part of dx is summed apart, such parts of a piece
    int64_t wrange, wranges; // tokens whose part of dw is summed apart, such parts (16-bit)
    char *xp, *wp, *xc, *g;
    float *accum, *waccum, *scale, *hit;
    void *part;            // (maximum, sum) pairs
    size_t bytes;
};

// The time of a first-come schedule on `units` units of n tiles of length a, then
// m of length b.
inline int64_t makespan(int64_t units, int64_t n, int64_t a, int64_t m, int64_t b) {
    const int64_t full = n / units, more = n % units;  // `more` units finish one a later
    int64_t early = full * a, late = more ? early + a : early, ne = units - more, nl = more;
    while (m > 0) {  // whole rows of equal units at a time
        if (ne > 0 && (nl == 0 || early <= late)) {
            if (m < ne) return early + b > late ? early + b : late;
            m -= ne;
            early += b;
        } else {
            if (m < nl) return late + b > early ? late + b : early;
            m -= nl;
            late += b;
        }
    }
    return early > late ? early : late;
}

// wide: fp32, else 16-bit; bwd: the gradients' pass.  base may be null (sizes only).
inline XentPlan plan(int64_t T, int64_t D, int64_t V, bool wide, bool bwd, char *base) {
    XentPlan p = {};
    const int64_t e = wide ? 4 : 2, slab = wide ? 1 : kSlab16,
                  rows = bwd ? (wide ? 64 : 256) : (wide ? side32(T, V) : side16(T, V));
    p.kD = wide ? (D < 4 ? 4 : D) : ceil_to(D, slab);  // (fp32: a row holds one vector at least)
    p.Tp = ceil_to(T, slab);
    size_t at = 0;
    const auto take = [&](int64_t bytes) {
        char *q = base && bytes ? base + at : nullptr;
        at += align256((size_t)bytes);
        return q;
    };
    p.xp = take(p.kD != D && (wide || !bwd) ? T * p.kD * e : 0);
    p.xc = take(bwd ? T * p.kD * e : 0);  // x with zero rows for tokens without a loss
    p.wp = take(p.kD != D ? V * p.kD * e : 0);
    p.tiles = (V + rows - 1) / rows;
    if (!bwd) {
        p.part = take(p.tiles * T * 8);
        p.hit = (float *)take(T * 4);
    } else {
        // G of a piece: up to 512 MiB
        int64_t most = ((int64_t)512 << 20) / (p.Tp * e) / rows * rows;
        if (most > (int64_t)1 << 21) most = (int64_t)1 << 21;  // (256 rows of G within 31 bits)
        if (most < rows) most = rows;
        const int64_t n = (V + most - 1) / most;
        p.piece = ceil_to((V + n - 1) / n, rows);
        p.pieces = (V + p.piece - 1) / p.piece;
        p.g = take(p.Tp * p.piece * e);
        p.side = wide ? side32(T, D, p.piece) : 256;
        int64_t splits = 1, wsplits = 1;
        if (wide) {
            // as below; 512 blocks at once (backward pass at 320 x 972 x 27650: about 950 us
            // without ranges, 559 with)
            const int64_t cols = (D + p.side - 1) / p.side, kv = (p.piece + 31) / 32, kt = (T + 31) / 32;
            const int64_t ndx = (T + p.side - 1) / p.side * cols, ndw = (p.piece + p.side - 1) / p.side * cols;
            int64_t best = makespan(512, ndx, kv, ndw, kt);
            for (int64_t k = 2; k <= 64 && (k <= 8 || k * T * D <= 1 << 22) && k * 8 <= kv; k += k < 8 ? 1 : k / 4) {
                const int64_t m = makespan(512, ndx * k, (kv + k - 1) / k, ndw, kt);
                if (m * 20 < best * 19) best = m, splits = k;
            }
        } else {
            const int64_t kv = ceil_to(p.piece, 64) / 64, kt = p.Tp / 64;  // slabs of dx's and of dw's sums
            const auto tiles = [&](int64_t rows) { return (D + p.side - 1) / p.side * ((rows + p.side - 1) / p.side); };
            const auto work = [&](int64_t side) { return p.side = side, tiles(T) * kv + tiles(p.piece) * kt; };
            // bf16, us of the backward pass, sides 256, 128 and 64 (slabs per unit):
            //   1000 x 2048 x 8000   148  153  213  (32)    300 x 777 x 8000   80  66  60  (9, of 128)
            //   1000 x 256 x 50021   196  166  237  (24)    1000 x 777 x 1000  77  51  38  (3, of 128)
            // and where D leaves half of the larger tile empty, 256 and 128:
            //   3000 x 100 x 50021   381  321
            const int64_t w256 = work(256), w128 = work(128), w64 = work(64);
            p.side = w256 >= 30 * 256 && 10 * w128 >= 33 * w256 ? 256 : (w128 >= 8 * 512 && 2 * w64 >= 5 * w128 ? 128 : 64);
            const int64_t units = p.side == 256 ? 256 : 512;  // blocks on the chip at once
            // the numbers of ranges that fill the chip best (a range more is a sum
            // more to write and to read, so it has to save a twentieth)
            const int64_t ndx = tiles(T), ndw = tiles(p.piece);
            int64_t best = makespan(units, ndx, kv, ndw, kt);
            for (int64_t j = 1; j <= 32 && (j == 1 || (ndw < units && j * p.piece * D <= 1 << 22 && j * 4 <= kt)); j *= 2)
                for (int64_t k = 1; k <= 64 && (k <= 8 || k * T * D <= 1 << 22) && (k == 1 || k * 4 <= kv); k += k < 8 ? 1 : k / 4) {
                    const int64_t m = makespan(units, ndx * k, (kv + k - 1) / k, ndw * j, (kt + j - 1) / j);
                    if (m * 20 < best * 19) best = m, splits = k, wsplits = j;
                }
        }
        const int64_t k0 = ceil_to(V < p.piece ? V : p.piece, 64);  // the longest piece's
        p.range = ceil_to((k0 + splits - 1) / splits, 64);
        p.ranges = (k0 + p.range - 1) / p.range;
        p.wrange = ceil_to((p.Tp + wsplits - 1) / wsplits, 64);
        p.wranges = (p.Tp + p.wrange - 1) / p.wrange;
        p.accum = (float *)take((!wide && p.pieces > 1) || p.ranges > 1 ? p.ranges * T * D * 4 : 0);
        p.waccum = (float *)take(!wide && p.wranges > 1 ? p.wranges * p.piece * D * 4 : 0);
        p.scale = (float *)take(wide ? 0 : 8);
    }
    p.bytes = at;
    return p;
}

}  // namespace xent
}  // namespace h3c
