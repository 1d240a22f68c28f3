// fp4q_attend_index.h -- which keys a workgroup of the attention kernels
// computes and where they lie: integer work shared by the kernels, the launch
// and the host tests.
#pragma once

#include "fp4q_kv_launch.h"

#define FP4Q_INDEX __host__ __device__ __forceinline__

namespace fp4q {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kTileKeys = 32;                     // keys of one wave's step
constexpr int kStepKeys = kWaves * kTileKeys;     // a chunk is a multiple of this
constexpr int kMaxChunk = 4096;                   // keys of one workgroup of the kernel for few queries at most

// what a row tile of one sequence sees
struct Extent {
    int64_t q0;  // first query row of the sequence
    int qn;      // its queries that are computed (at most max_q)
    int shift;   // query i sees keys below i + shift (causal)
    int kn;      // its keys
    bool bad;    // its length cannot be
};

FP4Q_INDEX Extent extent_of(const AttendArgs& a, int b)
{
    Extent e;
    int64_t n;
    if (a.q_starts) {
        e.q0 = a.q_starts[b];
        const int64_t q1 = a.q_starts[b + 1];
        n = (e.q0 < 0 || q1 < e.q0 || q1 > a.total_q) ? 0 : q1 - e.q0;
    } else {
        e.q0 = (int64_t)b * a.max_q;
        n = a.max_q;
    }
    e.kn = a.kv_lens[b];
    const int64_t holds = a.table ? (int64_t)a.table_len * a.kv.page_size
                                  : (b < a.kv.num_pages ? (int64_t)a.kv.page_size : 0);
    e.bad = e.kn < 0 || e.kn > a.max_kv || e.kn > holds;
    if (e.bad)
        e.kn = 0; // nothing is read for it
    // n is below 2^31: it counts rows between two 32-bit starts
    e.shift = (int)((int64_t)e.kn - n + 1);
    e.qn = (int)(n < a.max_q ? n : a.max_q);
    return e;
}

// keys [lo, hi) that query i of the sequence sees
FP4Q_INDEX void seen_by(const AttendArgs& a, const Extent& e, int i, int& lo, int& hi)
{
    hi = a.causal ? i + e.shift : e.kn;
    hi = hi < 0 ? 0 : (hi > e.kn ? e.kn : hi);
    lo = (a.window && hi > a.window) ? hi - a.window : 0;
}

// keys that the rows [r0, r1) of a tile see, from a 32-key boundary on
FP4Q_INDEX void tile_keys(const AttendArgs& a, const Extent& e, int r0, int r1, int& lo, int& hi)
{
    int t;
    seen_by(a, e, r0 / a.group, lo, t);
    seen_by(a, e, (r1 - 1) / a.group, t, hi);
    lo &= ~(kTileKeys - 1);
}

// the key chunks of a row tile that are computed; the first one always is,
// and says that there is nothing where there is nothing
FP4Q_INDEX int chunks_of(const AttendPlan& p, int lo, int hi)
{
    const int n = (int)(((int64_t)hi - lo + p.chunk - 1) / p.chunk);
    return n < 1 ? 1 : n;
}

// where 16 consecutive keys lie: byte offsets of the first one's row in the
// code and in the scale arrays, or -1 where their page does not exist
struct Granule {
    int64_t codes, scales;
};

// the granule of keys [key, key + 16) of sequence b, key a multiple of 16 and
// below its length (so that the table has an entry for it)
FP4Q_INDEX Granule granule_at(const AttendArgs& a, int b, int head, int key)
{
    int64_t page = b, off = key;
    if (a.table) {
        const int p = key / a.kv.page_size;
        page = a.table[(int64_t)b * a.table_stride + p];
        off = key - p * a.kv.page_size;
    }
    if (page < 0 || page >= a.kv.num_pages)
        return Granule{-1, -1};
    return Granule{page * a.kv.c_page + head * a.kv.c_head + off * a.kv.c_token,
                   page * a.kv.s_page + head * a.kv.s_head + off * a.kv.s_token};
}

// Row tiles and key chunks from the sizes that the host knows.  Chunks are cut
// so that about four workgroups per CU (256 CUs) exist where the keys allow.
inline AttendPlan plan_of(const AttendArgs& a)
{
    AttendPlan p{};
    const int64_t rows = (int64_t)a.max_q * a.group;
    p.many = rows > 64;
    if (p.many)
        p.rows_per_tile = (a.bf16 && a.kv.head_dim < 256) ? 256 : 128; // 32 rows a wave
    else
        p.rows_per_tile = rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
    p.tiles = (int)((rows + p.rows_per_tile - 1) / p.rows_per_tile);
    const int64_t units = (int64_t)a.batch * a.kv.heads * p.tiles;
    const int64_t span = attend_span(a);
    int64_t want = ((p.many ? 512 : 1024) + units - 1) / units;
    int64_t chunk = (span + want - 1) / want;
    const int64_t step = p.many ? 2 * kStepKeys : kStepKeys;
    chunk = (chunk + step - 1) / step * step;
    chunk = chunk < step ? step : chunk;
    if (!p.many && chunk > kMaxChunk)
        chunk = kMaxChunk;
    p.chunk = (int)chunk;
    const int64_t chunks = span <= chunk ? 1 : (span + chunk - 1) / chunk;
    // a launch holds fewer than 2^32 threads
    const int64_t most = (((int64_t)1 << 32) - 1) / 512;
    if (units > most / chunks || (chunks > 1 && (int64_t)a.batch * a.kv.heads > most / rows)) {
        p.chunks = 0;
        return p;
    }
    p.chunks = (int)chunks;
    if (chunks > 1) {
        const size_t all = (size_t)a.batch * a.kv.heads * rows * chunks;
        p.workspace = ((all * 8 + 255) & ~(size_t)255) + all * a.kv.head_dim * 4;
    }
    return p;
}

} // namespace fp4q
