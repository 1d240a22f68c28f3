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
// 10.0, 10.1 and 11.5),
inline int few_waves_wanted(const MatmulArgs& a)
{
    const int64_t tiles = (a.n + 15) / 16;
    return tiles * 2 >= kFewWaves ? 2 : (tiles * 4 >= kFewWaves ? 4 : 8);
}

// and as few as let a chunk of x, a step of each of them, fit
inline int few_waves_k(const MatmulArgs& a, int parts)
{
    int kw = few_waves_wanted(a);
    while (kw > 2 && (size_t)parts * a.m * (kw * kFewStep * 2 + 16) > few_lds(a.weights))
        kw /= 2;
    return kw;
}

// steps of the long axis whose x a workgroup of few rows holds at once, its waves taking turns
inline int few_chunk(const MatmulArgs& a, int parts, int kw)
{
    const int steps = (int)((a.k + kFewStep - 1) / kFewStep);
    int chunk = (steps + kw - 1) / kw * kw;
    while (chunk > kw && (size_t)parts * a.m * (chunk * kFewStep * 2 + 16) > few_lds(a.weights))
        chunk = (chunk / 2 + kw - 1) / kw * kw;
    return chunk;
}

// Whether the kernel for few rows takes them.
// One part of x: up to 16 always.  Up to 32, in two tiles of 16, where x, that every workgroup
// passes through its LDS, is small, one round of workgroups has all weight rows, and there are at
// most four chunks (MXFP4, whose products are shorter: eight, by the waves wanted).  In us, so and by
// the kernel for many: NVFP4, 14336 x 4096, 17 and 32 rows 13.5 and 16.5, 15.9 and 17.2; 4096 x 4096 9.3
// and 12.6, 11.6 and 14.0; two weights of 14336 x 4096, 17, 20, 24, 32 rows, 4, 4, 8, 8 chunks, 20.9 and
// 25.8, 21.5 and 25.9, 25.5 and 26.0, 27.3 and 26.5 (MXFP4 16.7 and 23.6, 17.2 and 23.8, 21.0 and 24.1,
// 22.9 and 24.5); of 4096 x 4096, 20 and 24 rows, 4 and 8 chunks, 14.7 and 17.4, 23.8 and 17.9 (MXFP4,
// by fewer waves than wanted, 12.3 and 16.3, 19.5 and 16.8).  Outside: 4096 x 14336 26.8 and 18.8, 34.4
// and 19.4; 65536 x 4096 51.9 and 50.4, 60.9 and 51.0.
// Three parts: up to 16 in less than eight chunks of x (two weights, of which the kernel for many
// makes half-wide tiles: sixteen), each of which is waited for.  NVFP4, so and by the kernel for many: 14336 x
// 4096, 8 and 16 rows, 4 and 8 chunks, 19.3 and 25.3, 27.6 and 25.8; 4096 x 4096, 4, 8 and 12 rows, 2,
// 4 and 8 chunks, 9.8 and 16.2, 14.7 and 16.7, 24.1 and 17.5; 4096 x 14336, 4 and 8 rows, 7 and 14
// chunks, 20.6 and 26.3, 36.4 and 26.6; two weights of 14336 x 4096, 16 rows, 8 chunks, 36.1 and 39.4.
inline bool takes_few(const MatmulArgs& a, int parts)
{
    const int kw = few_waves_k(a, parts);
    const int64_t steps = (a.k + kFewStep - 1) / kFewStep;
    auto within = [&](int64_t chunks) { return steps == 0 || steps <= chunks * few_chunk(a, parts, kw); };
    if (parts == 1)
        return a.m <= kFewRows || (a.m <= 2 * kFewRows && a.m * a.k <= 1 << 17 && a.n <= (int64_t)kCus * 16 * (8 / kw) &&
                                   (within(4) || (a.mx && kw == few_waves_wanted(a) && within(8))));
    return a.m <= 2 || (a.m <= kFewRows && within(8 * a.weights - 1));
}

inline MatmulPlan plan_of(const MatmulArgs& a)
{
    MatmulPlan p{};
    p.splits = 1;
    // x of bf16, not rotated, enters as it is, other x in three parts: the workgroups of few rows
    // convert a small x on the way, a launch less, and a larger one is prepared by a launch of its
    // own; up to two rows never, so that they need no workspace.  So and prepared, in us: NVFP4,
    // 14336 x 4096, 1, 2, 3, 4 rows 13.5 and 15.6, 13.1 and 15.3, 15.2 and 16.1, 15.7 and 16.5; 4096 x
    // 4096, 1 and 4 rows 6.2 and 8.4, 8.4 and 9.8; 4096 x 14336, 1, 2, 3 rows 14.3 and 15.6, 18.2 and
    // 17.4, 24.1 and 19.5; two weights of 14336 x 4096, 3 and 4 rows 22.2 and 23.9, 26.2 and 25.5
    // (MXFP4 19.9 and 20.6, 25.4 and 21.9).
    const bool exact = a.bf16 && !a.rotate;
    p.parts = exact ? 1 : 3;
    p.many = !takes_few(a, p.parts);
    p.prepared = !exact && (p.many || (a.m > 2 && a.m * a.k > (a.weights == 2 ? 12288 : 16384)));
    const size_t at = p.prepared ? whole256((size_t)p.parts * a.m * a.k * 2) : 0;
    p.partials = at;
    if (!p.many) {
        const int kw = few_waves_k(a, p.parts);
        const size_t row = (size_t)p.parts * a.m;
        p.waves_k = kw;
        p.rows = 16 * (8 / kw);
        p.tokens = a.m > kFewRows ? 32 : 16;
        p.chunk_steps = few_chunk(a, p.parts, kw);
        const size_t x = row * (p.chunk_steps * kFewStep * 2 + 16), red = (size_t)8 * a.weights * (p.tokens / 16) * 1024;
        p.lds = x > red ? x : red;
        p.workspace = at;
        p.refused = (a.n + p.rows - 1) / p.rows > 0x7FFFFF;
        return p;
    }
    // Tiles of 32, 64 or 128 rows of x by 256 rows of weights, and splits of the long axis: what
    // is least of a cost in us.  A compute unit works through its tiles' steps one after the other
    // whether one or two workgroups are there (three parts in a tile of 32 take 2.1 us a step alone
    // and 1.4 among several: 1.5 chose best); a launch costs 6, joining 3 and the partial sums'
    // way to memory and back (4 TB/s).  As measured against it: 48 rows, 4096 x 14336, MXFP4,
    // 64-row tiles in 1, 4, 8, 16, 32 splits 114, 37, 25, 21, 30 us; 8192 rows, 14336 x 4096, tiles of
    // 64 and 128 rows 1185 and 854.
    // Three parts of x are rows of one step in a tile of 32, and a step for each in one of 128: NVFP4,
    // 14336 x 4096, 64, 203, 1024, 8192 rows 39 and 59, 82 and 103, 311 and 313, 2397 and 2217.  Tiles of 64, a
    // step for each part, were least nowhere (41, 110, 392).
    p.rows = 256 / a.weights;
    const int64_t steps = (a.k + kStepK - 1) / kStepK, tiles_n = (a.n + p.rows - 1) / p.rows;
    int64_t best_tiles = 0;
    double best = 0.0;
    for (int tokens = 32; tokens <= 128 && (tokens == 32 || tokens / 2 < a.m); tokens *= p.parts == 3 ? 4 : 2) {
        const int64_t tiles_m = (a.m + tokens - 1) / tokens;
        if (tiles_n > 0x7FFFFF / tiles_m)
            continue;
        const int64_t tiles = tiles_n * tiles_m;
        const double turn = tokens == 32 ? (p.parts == 3 ? 1.5 : 0.95) : p.parts * (tokens == 64 ? 1.15 : 1.9);
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
