// fp4q_matmul_plan.h -- how a product with 4-bit weights is cut into workgroups, from its sizes
// and types alone: integer work of the host.
#pragma once

#include "fp4q_matmul_launch.h"

namespace fp4q {

// LDS of x in a workgroup of few rows, beside the 54 KiB (two weights 108) of codes on their way,
// of a compute unit's 160
constexpr size_t few_lds(int weights) { return weights == 2 ? 48 * 1024 : 68 * 1024; }
constexpr int kFewRows = 16;          // rows of x that the kernel for few takes in one tile
constexpr int kFewWaves = 1536;       // waves that it is given at least, where the long axis can be shared

inline size_t whole256(size_t n) { return (n + 255) & ~(size_t)255; }

// Waves of a workgroup of few rows that share the long axis: as few as give the chip kFewWaves
// waves (one token, 4096 x 4096: 2, 4 or 8 of them take 8.7, 6.0 and 4.7 us; 14336 x 4096
// 10.0, 10.1 and 11.5), and as few as let a chunk of x, a step of each of them, fit.
inline int few_waves_k(const MatmulArgs& a, int parts)
{
    const int64_t tiles = (a.n + 15) / 16;
    int kw = tiles * 2 >= kFewWaves ? 2 : (tiles * 4 >= kFewWaves ? 4 : 8);
    while (kw > 2 && (size_t)parts * a.m * (kw * kFewStep * 2 + 16) > few_lds(a.weights))
        kw /= 2;
    return kw;
}

// Whether the kernel for few rows takes them.  Up to 16 always.  Up to 32, in two tiles of 16, where
// x, that every workgroup passes through its LDS, is small and one round of workgroups has
// all weight rows; one part of x.  In us, so and by the kernel for many: NVFP4, 14336 x 4096, 17 and
// 32 rows 13.9 and 17.0, 15.9 and 17.5; 4096 x 4096 9.3 and 13.0, 11.5 and 14.3; two weights of
// 14336 x 4096 21.0 and 26.1, 27.4 and 26.7 (MXFP4 16.6 and 23.5, 23.0 and 24.3).  Outside:
// 4096 x 14336 26.8 and 18.8, 34.4 and 19.4; 65536 x 4096 51.9 and 50.4, 60.9 and 51.0.
inline bool takes_few(const MatmulArgs& a, int parts)
{
    return a.m <= kFewRows || (parts == 1 && a.m <= 2 * kFewRows && a.m * a.k <= 1 << 17 &&
                               a.n <= (int64_t)kCus * 16 * (8 / few_waves_k(a, parts)));
}

inline MatmulPlan plan_of(const MatmulArgs& a)
{
    MatmulPlan p{};
    p.splits = 1;
    // x of bf16, not rotated, enters as it is.  Else the workgroups convert the fewest rows on the
    // way, a launch less, and more are prepared by a launch of their own.  Rotated bf16, so and
    // prepared, in us: NVFP4, 4096 x 4096, 1, 2, 4 rows 6.0 and 7.1, 6.2 and 7.2, 7.9 and 7.6; 14336 x
    // 4096 12.4 and 11.5, 12.1 and 11.4, 13.8 and 11.7; 4096 x 14336 13.2 and 14.5, 16.6 and 15.2,
    // 23.9 and 16.1; MXFP4, 14336 x 4096, 1, 4 rows 11.1 and 13.0, 11.5 and 13.5.
    const bool exact = a.bf16 && !a.rotate;
    p.prepared = !exact && a.m > (a.mx ? 4 : 2);
    if (exact)
        p.parts = 1;
    else if (a.mx || !p.prepared)
        p.parts = a.bf16 ? 2 : 3; // in bf16
    else
        p.parts = a.bf16 ? 1 : 2; // in f16
    p.many = !takes_few(a, p.parts);
    size_t at = p.prepared ? whole256((size_t)p.parts * a.m * a.k * 2) : 0;
    p.exponents = at;
    if (p.prepared && !a.mx)
        at = whole256(at + (size_t)a.m * 4);
    p.partials = at;
    if (!p.many) {
        const int kw = few_waves_k(a, p.parts);
        const size_t row = (size_t)p.parts * a.m;
        p.waves_k = kw;
        p.rows = 16 * (8 / kw);
        p.tokens = a.m > kFewRows ? 32 : 16;
        const int steps = (int)((a.k + kFewStep - 1) / kFewStep);
        p.chunk_steps = (steps + kw - 1) / kw * kw;
        while (p.chunk_steps > kw && row * (p.chunk_steps * kFewStep * 2 + 16) > few_lds(a.weights))
            p.chunk_steps = (p.chunk_steps / 2 + kw - 1) / kw * kw;
        const size_t x = row * (p.chunk_steps * kFewStep * 2 + 16), red = (size_t)8 * a.weights * (p.tokens / 16) * 1024;
        p.lds = x > red ? x : red;
        p.workspace = at;
        p.refused = (a.n + p.rows - 1) / p.rows > 0x7FFFFF;
        return p;
    }
    // Tiles of 32, 64 or 128 rows of x by 256 rows of weights, and splits of the long axis: what
    // is least of a cost in us.  Two parts of x are rows of the same step where a tile of twice
    // the rows holds them (32 binary32 rows, 14336 x 4096, NVFP4, 22 us so and 26 a step for each
    // part; 64 rotated ones, MXFP4, 30 and 32).  A compute unit works through its tiles' steps one
    // after the other whether one or two workgroups are there; a launch costs 6, joining 3
    // and the partial sums' way to memory and back (4 TB/s).  As measured against
    // it: 48 rows, 4096 x 14336, MXFP4, 64-row tiles in 1, 4, 8, 16, 32 splits 114, 37, 25, 21,
    // 30 us; 509 rows, 4096 x 4096, NVFP4 rotated, tiles of 32, 64, 128 rows at their best 41
    // (1 split), 35 (2), 42 (4); 8192 rows, 14336 x 4096, tiles of 64 and 128 rows 1185 and 854.
    p.rows = 256 / a.weights;
    const int64_t steps = (a.k + kStepK - 1) / kStepK, tiles_n = (a.n + p.rows - 1) / p.rows;
    int64_t best_tiles = 0;
    double best = 0.0;
    for (int tokens = 32; tokens <= 128 && (tokens == 32 || tokens / 2 < a.m); tokens *= 2) {
        const int64_t tiles_m = (a.m + tokens - 1) / tokens;
        if (tiles_n > 0x7FFFFF / tiles_m)
            continue;
        const int64_t tiles = tiles_n * tiles_m;
        const bool both = p.parts == 2 && tokens <= 64;
        const int wide = both ? 2 * tokens : tokens; // rows of x, or of its parts, in a step
        const double turn = (both ? 1 : p.parts) * (wide == 32 ? 0.95 : (wide == 64 ? 1.15 : 1.9));
        // more splits than fill the chip four times, or than give each two steps, cost more
        for (int64_t c = 1; c == 1 || (c <= steps / 2 && tiles * c <= 4 * kCus); ++c) {
            const int64_t each = (steps + c - 1) / c, splits = each == 0 ? 1 : (steps + each - 1) / each;
            const double mb = (double)tiles * splits * tokens * 256 * 4e-6;
            const double us = 6.0 + (double)((tiles * splits + kCus - 1) / kCus) * each * turn +
                              (splits > 1 ? 3.0 + mb * 2 / 4 : 0.0);
            if (best_tiles == 0 || us < best) {
                best = us;
                best_tiles = tiles;
                p.tokens = tokens;
                p.both = both;
                p.splits = (int)splits;
                p.split_steps = (int)each;
            }
        }
    }
    p.refused = best_tiles == 0;
    p.workspace = at + (p.splits > 1 ? (size_t)p.splits * best_tiles * p.tokens * 256 * 4 : 0);
    return p;
}

} // namespace fp4q
