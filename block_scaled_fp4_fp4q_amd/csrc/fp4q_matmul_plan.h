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

// What the kernel for few rows costs with x in parts that are prepared, in us: a round of workgroups its waves'
// steps, a wait for each chunk of x, and x's way into LDS.  This and as measured: NVFP4, 14336 x 4096, 3, 8, 16
// rows 14.4, 18.8, 26.1 and 16.4, 19.3, 27.6; 4096 x 14336, 3, 6, 16 rows 21.5, 37.9, 78.1 and 19.6, 33.4, 79.8;
// 28672 x 8192, 6, 12 rows 55.6, 81.0 and 55.9, 80.8; two weights of 8192 x 8192, 6, 16 rows 30.2, 59.9 and 30.9, 61.2.
inline double few_us(const MatmulArgs& a, int parts)
{
    const int kw = few_waves_k(a, parts), chunk = few_chunk(a, parts, kw), rows = 16 * (8 / kw);
    const int64_t steps = (a.k + kFewStep - 1) / kFewStep, rounds = ((a.n + rows - 1) / rows + kCus - 1) / kCus;
    const double turn = a.weights == 1 ? 0.8 : (a.mx ? 1.3 : 1.6);
    return 4.8 + (double)rounds * (turn * (double)((steps + kw - 1) / kw) + (steps == 0 ? 0.0 : 0.8 * (double)((steps + chunk - 1) / chunk)) +
                                   2.12e-5 * (double)(parts * a.m * a.k * 2));
}

// Whether the kernel for few rows takes x in one part: up to 16 always.  Up to 32, in two tiles of 16, where x,
// that every workgroup passes through its LDS, is small, one round of workgroups has all weight rows, and
// there are at most four chunks (MXFP4, whose products are shorter: eight, by the waves wanted).  In us, so and
// by the kernel for many: NVFP4, 14336 x 4096, 17 and 32 rows 13.5 and 16.5, 15.9 and 17.2; 4096 x 4096 9.3
// and 12.6, 11.6 and 14.0; two weights of 14336 x 4096, 17, 20, 24, 32 rows, 4, 4, 8, 8 chunks, 20.9 and
// 25.8, 21.5 and 25.9, 25.5 and 26.0, 27.3 and 26.5 (MXFP4 16.7 and 23.6, 17.2 and 23.8, 21.0 and 24.1,
// 22.9 and 24.5); of 4096 x 4096, 20 and 24 rows, 4 and 8 chunks, 14.7 and 17.4, 23.8 and 17.9 (MXFP4,
// by fewer waves than wanted, 12.3 and 16.3, 19.5 and 16.8).  Outside: 4096 x 14336 26.8 and 18.8, 34.4
// and 19.4; 65536 x 4096 51.9 and 50.4, 60.9 and 51.0.
inline bool takes_few(const MatmulArgs& a)
{
    if (a.m <= kFewRows || a.m > 2 * kFewRows || a.m * a.k > 1 << 17)
        return a.m <= kFewRows;
    const int kw = few_waves_k(a, 1);
    const int64_t steps = (a.k + kFewStep - 1) / kFewStep;
    auto within = [&](int64_t chunks) { return steps == 0 || steps <= chunks * few_chunk(a, 1, kw); };
    return a.n <= (int64_t)kCus * 16 * (8 / kw) && (within(4) || (a.mx && kw == few_waves_wanted(a) && within(8)));
}

// The kernel for many rows: tiles of 32, 64 or 128 rows of x by 256 rows of weights, and splits of the
// long axis, what is least of a cost in us, which it returns.  A compute unit works through its tiles' steps
// one after the other whether one or two workgroups are there; a launch costs 6, joining 3 and the
// partial sums' way to memory and back (4 TB/s).  As measured against it: 48 rows, 4096 x 14336, MXFP4,
// 64-row tiles in 1, 4, 8, 16, 32 splits 114, 37, 25, 21, 30 us; 8192 rows, 14336 x 4096, tiles of
// 64 and 128 rows 1185 and 854.
//   Three parts of x are rows of one step in a tile of 32, and a step for each in one of 128.  There a workgroup alone
// on its compute unit does not fill it: a step costs 1.7 and 5.9, and 1.4 and 5.0 where there are several;
// the preparation and the product 9, joining 3 for each weight.  NVFP4, 14336 x 4096, 64, 203, 1024, 2048, 8192 rows
// 39 and 59, 82 and 103, 311 and 313, 600 and 611, 2397 and 2217.  Tiles of 64, a step for each part, were
// least nowhere (41, 110, 392, 714).
//   Against few_us: over 186 calls of 3 to 16 rows (1024 x 4096 to 28672 x 8192, both formats, one and two weights, weights in
// the last-level cache and not) the kernel that is taken needs 0.5% more time than the faster one in the mean, 18% at most.
inline double plan_many(const MatmulArgs& a, MatmulPlan& p)
{
    p.rows = 256 / a.weights;
    p.splits = 1;
    const int64_t steps = (a.k + kStepK - 1) / kStepK, tiles_n = (a.n + p.rows - 1) / p.rows;
    int64_t best_tiles = 0;
    double best = 0.0;
    for (int tokens = 32; tokens <= 128 && (tokens == 32 || tokens / 2 < a.m); tokens *= p.parts == 3 ? 4 : 2) {
        const int64_t tiles_m = (a.m + tokens - 1) / tokens;
        if (tiles_n > 0x7FFFFF / tiles_m)
            continue;
        const int64_t tiles = tiles_n * tiles_m;
        // more splits than fill the chip four times, or than give each two steps, cost more
        for (int64_t c = 1; c == 1 || (c <= steps / 2 && tiles * c <= 4 * kCus); ++c) {
            const int64_t each = (steps + c - 1) / c, splits = each == 0 ? 1 : (steps + each - 1) / each;
            const int64_t rounds = (tiles * splits + kCus - 1) / kCus;
            const double turn = p.parts == 1 ? (tokens == 32 ? 0.95 : (tokens == 64 ? 1.15 : 1.9))
                                             : (tokens == 32 ? (rounds == 1 ? 1.7 : 1.4) : (rounds == 1 ? 5.9 : 5.0));
            const double mb = (double)tiles * splits * tokens * 256 * 4e-6;
            const double us = (p.parts == 1 ? 6.0 : 9.0) + (double)rounds * each * turn + (splits > 1 ? (p.parts == 1 ? 3.0 : 3.0 * a.weights) + mb * 2 / 4 : 0.0);
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
    p.workspace = p.partials + (p.splits > 1 ? (size_t)p.splits * best_tiles * p.tokens * 256 * 4 : 0);
    return best;
}

inline MatmulPlan plan_of(const MatmulArgs& a)
{
    MatmulPlan p{};
    p.splits = 1;
    // x of bf16, not rotated, enters as it is, other x in three parts
    p.parts = a.bf16 && !a.rotate ? 1 : 3;
    const size_t prepared = p.parts == 1 ? 0 : whole256((size_t)p.parts * a.m * a.k * 2);
    if (p.parts == 1) {
        p.many = !takes_few(a);
    } else if (a.m <= 2) {
        p.many = false; // by few rows, and without a workspace
    } else {
        MatmulPlan q = p;
        p.many = a.m > kFewRows || few_us(a, p.parts) > plan_many(a, q);
    }
    // The workgroups of few rows convert a small x on the way, a launch less, and a larger one is
    // prepared by a launch of its own.  So and prepared, in us: NVFP4, 14336 x 4096, 1, 2, 3, 4 rows 13.5 and
    // 15.6, 13.1 and 15.3, 15.2 and 16.1, 15.7 and 16.5; 4096 x 4096, 1 and 4 rows 6.2 and 8.4, 8.4 and 9.8;
    // 4096 x 14336, 1, 2, 3 rows 14.3 and 15.6, 18.2 and 17.4, 24.1 and 19.5; two weights of 14336 x 4096, 3 and
    // 4 rows 22.2 and 23.9, 26.2 and 25.5 (MXFP4 19.9 and 20.6, 25.4 and 21.9).
    p.prepared = p.parts == 3 && (p.many || (a.m > 2 && a.m * a.k > (a.weights == 2 ? 12288 : 16384)));
    p.partials = p.prepared ? prepared : 0;
    if (p.many) {
        plan_many(a, p);
        return p;
    }
    const int kw = few_waves_k(a, p.parts);
    const size_t row = (size_t)p.parts * a.m;
    p.waves_k = kw;
    p.rows = 16 * (8 / kw);
    p.tokens = a.m > kFewRows ? 32 : 16;
    p.chunk_steps = few_chunk(a, p.parts, kw);
    const size_t x = row * (p.chunk_steps * kFewStep * 2 + 16), red = (size_t)8 * a.weights * (p.tokens / 16) * 1024;
    p.lds = x > red ? x : red;
    p.workspace = p.partials;
    p.refused = (a.n + p.rows - 1) / p.rows > 0x7FFFFF;
    return p;
}

} // namespace fp4q
