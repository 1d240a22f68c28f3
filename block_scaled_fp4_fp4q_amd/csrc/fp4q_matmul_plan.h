// fp4q_matmul_plan.h -- how a product with 4-bit weights is cut into workgroups: integer
// work of the host.
#pragma once

#include <stdlib.h>

#include "fp4q_matmul_launch.h"

namespace fp4q {

constexpr size_t kFewLds = 64 * 1024;

inline size_t whole256(size_t n) { return (n + 255) & ~(size_t)255; }

inline MatmulPlan plan_of(const MatmulArgs& a)
{
    MatmulPlan p{};
    p.splits = 1;
    const bool exact = a.bf16 && !a.rotate; // x enters as it is
    p.many = a.m > 16;
    const char* e;
    // few rows are converted by the workgroups that use them, more by a launch of its own
    const int64_t conv_most = (e = getenv("FP4Q_CONV")) ? atoi(e) : 4;
    p.prepared = !exact && (p.many || a.m > conv_most);
    if (exact)
        p.parts = 1;
    else if (a.mx || !p.prepared)
        p.parts = a.bf16 ? 2 : 3;
    else
        p.parts = a.bf16 ? 1 : 2;
    size_t at = p.prepared ? whole256((size_t)p.parts * a.m * a.k * 2) : 0;
    p.exponents = at;
    if (p.prepared && !a.mx)
        at = whole256(at + (size_t)a.m * 4);
    p.partials = at;
    if (!p.many) {
        // waves that share the long axis: as few as give the chip two waves a SIMD
        const int64_t tiles = (a.n + 15) / 16;
        int kw = tiles * 2 >= 2048 ? 2 : (tiles * 4 >= 2048 ? 4 : 8);
        if ((e = getenv("FP4Q_KW")))
            kw = atoi(e);
        const size_t row = (size_t)p.parts * a.m;
        while (kw > 2 && row * (kw * kFewStep * 2 + 16) > kFewLds) // a chunk is a step of each of them
            kw /= 2;
        p.waves_k = kw;
        p.rows = 16 * (8 / kw);
        p.tokens = 16;
        const int steps = (int)((a.k + kFewStep - 1) / kFewStep);
        p.chunk_steps = (steps + kw - 1) / kw * kw;
        while (p.chunk_steps > kw && row * (p.chunk_steps * kFewStep * 2 + 16) > kFewLds)
            p.chunk_steps = (p.chunk_steps / 2 + kw - 1) / kw * kw;
        const size_t x = row * (p.chunk_steps * kFewStep * 2 + 16), red = (size_t)8 * a.weights * 1024;
        p.lds = x > red ? x : red;
        p.workspace = at;
        p.refused = (a.n + p.rows - 1) / p.rows > 0x7FFFFF;
        return p;
    }
    p.rows = 256 / a.weights;
    p.tokens = a.m <= 32 ? 32 : (a.m <= 64 ? 64 : 128);
    if ((e = getenv("FP4Q_BM")))
        p.tokens = atoi(e);
    const int64_t steps = (a.k + kStepK - 1) / kStepK;
    const int64_t tiles = (a.n + p.rows - 1) / p.rows * ((a.m + p.tokens - 1) / p.tokens);
    p.refused = (a.n + p.rows - 1) / p.rows > 0x7FFFFF / ((a.m + p.tokens - 1) / p.tokens);
    int64_t splits = (e = getenv("FP4Q_SPLIT")) ? atoi(e) : 1;
    p.split_steps = (int)((steps + splits - 1) / splits);
    if (p.split_steps < 1)
        p.split_steps = 1;
    p.splits = steps == 0 ? 1 : (int)((steps + p.split_steps - 1) / p.split_steps);
    (void)tiles;
    const size_t wide = (size_t)((a.n + 3) & ~(int64_t)3);
    p.workspace = at + (p.splits > 1 ? (size_t)p.splits * a.weights * a.m * wide * 4 : 0);
    return p;
}

} // namespace fp4q
