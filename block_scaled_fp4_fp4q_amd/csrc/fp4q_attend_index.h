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
constexpr int kStepKeys = kWaves * kTileKeys;     // keys of a workgroup's step at most
constexpr int kMinPart = 2;                       // steps that are not cut further
constexpr int kCus = 256;
constexpr int kScanBatch = 256;                   // sequences that every workgroup looks through itself
constexpr int kSegment = 4096;                    // keys whose places are looked up at once

inline size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

// Waves per SIMD that the kernel for few queries is built for (rows16: 16-row
// tiles of a wave; parts: 16-bit parts of a query): as many as its registers
// allow without spilling, but for three parts (MXFP4, rotated or binary32) at 128
// values, which spill 9 to 17 of them.  One wave less spills nothing there and
// was faster at most sizes (32 sequences of 8192 keys, 4 heads, binary32: 1 query
// 43 -> 39 us, 4 queries 85 -> 68; 3 of 65521, rotated, 8 queries 81 -> 85), as at
// 64 values, where it is taken.
constexpr int few_waves_of(int dim, int parts, int rows16)
{
    return dim == 64    ? (rows16 == 1 ? 4 : 3) - (parts == 3 ? 1 : 0)
           : dim == 128 ? (rows16 == 1 ? 3 : 2)
                        : (parts == 3 ? 1 : 2);
}

inline int few_waves(const AttendArgs& a)
{
    const int parts = a.bf16 && !a.rotate ? 1 : (a.kv.mx ? 3 : 2);
    return few_waves_of(a.kv.head_dim, parts, (int64_t)a.max_q * a.group > 16 && a.kv.head_dim < 256 ? 2 : 1);
}

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

// the first key that a row of a tile sees, the lowest row being r0: those from
// the 32-key boundary up to it are computed with the tile's keys, but no query
// sees them, and what they hold may be anything
FP4Q_INDEX int first_seen(const AttendArgs& a, const Extent& e, int r0)
{
    int lo, hi;
    seen_by(a, e, r0 / a.group, lo, hi);
    return lo;
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

// ---- few queries: equal shares of the work -----------------------------------------
//
// A pair (a sequence and a KV head) of n steps of kStepKeys keys is computed by
// ceil(n / most) workgroups, in equal parts; `most` follows from the sum of all
// lengths, which lie on the device, so that the parts about fill the
// chip once whatever the lengths are.  A pair in more than one part has
// partial results, each in a slot of its own.  Steps count in 31 bits.

// steps of each KV head of a sequence; a sequence with queries has at least
// one, which says that there is nothing where there is nothing
FP4Q_INDEX int few_steps(const AttendArgs& a, const Extent& e)
{
    if (e.qn == 0)
        return 0;
    int lo, hi;
    tile_keys(a, e, 0, e.qn * a.group, lo, hi);
    const int n = (int)(((int64_t)hi - lo + kStepKeys - 1) / kStepKeys);
    return n < 1 ? 1 : n;
}

// steps of a part at most, where all pairs together have `total`
FP4Q_INDEX uint32_t few_most(const AttendPlan& p, uint32_t total)
{
    const uint32_t n = (total + p.parts - 1) / p.parts;
    return n < kMinPart ? kMinPart : n;
}

FP4Q_INDEX uint32_t few_parts(uint32_t steps, uint32_t most) { return (steps + most - 1) / most; }

// What a kernel of its own writes down before the parts are computed, where
// there are more than kScanBatch sequences (a look through them by every
// workgroup would cost more than the launch): the sequence of each workgroup,
// and the parts and slots before each sequence.
struct FewTable {
    uint32_t* sequence; // [groups], ~0 where a workgroup has no part
    uint32_t* before;   // [batch][3]: parts, slots, steps per head
    uint32_t* most;     // steps of a part at most
};

FP4Q_INDEX size_t few_table_bytes(int64_t groups, int64_t batch)
{
    return batch > kScanBatch ? (((size_t)groups + 3 * (size_t)batch + 1) * 4 + 255) & ~(size_t)255 : 0;
}

FP4Q_INDEX FewTable few_table(void* workspace, int groups, int batch)
{
    FewTable t;
    t.sequence = static_cast<uint32_t*>(workspace);
    t.before = t.sequence + groups;
    t.most = t.before + (size_t)3 * batch;
    return t;
}

// first step of part i of `parts`
FP4Q_INDEX int few_from(uint32_t steps, uint32_t parts, uint32_t i) { return (int)((uint64_t)steps * i / parts); }

// Row tiles, and key chunks or parts, from the sizes that the host knows.
inline AttendPlan plan_of(const AttendArgs& a)
{
    AttendPlan p{};
    const int64_t rows = (int64_t)a.max_q * a.group, pairs = (int64_t)a.batch * a.kv.heads;
    const int64_t span = attend_span(a);
    const int64_t most = (((int64_t)1 << 32) - 1) / 512; // a launch holds fewer than 2^32 threads
    p.chunks = 1;
    p.many = rows > 64;
    if (!p.many) {
        p.rows_per_tile = rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
        p.tiles = 1;
        const int64_t steps = (span + kStepKeys - 1) / kStepKeys;
        // the joining launch has a workgroup for each row; all steps count in 31 bits
        if (pairs > most / rows || (steps != 0 && pairs > 0x7FFFFFFF / steps) || a.total_q > 0x7FFFFFFF)
            return p; // groups == 0: refused
        p.groups = (int)pairs;
        if (steps > kMinPart) {
            // workgroups that are resident at once: 256 CUs, one wave of each
            // on every SIMD
            p.parts = kCus * few_waves(a);
            p.groups += p.parts;
            p.chunks = 2; // partial results
            const size_t places = (size_t)2 * p.parts * p.rows_per_tile;
            p.workspace = few_table_bytes(p.groups, a.batch) + round256((size_t)pairs * 8) + round256(places * 8) +
                          places * a.kv.head_dim * 4;
        }
        return p;
    }
    p.rows_per_tile = (a.bf16 && a.kv.head_dim < 256) ? 256 : 128; // 32 rows a wave
    p.tiles = (int)((rows + p.rows_per_tile - 1) / p.rows_per_tile);
    const int64_t units = pairs * p.tiles;
    // A workgroup is given a CU of its own (of those with four waves and 64 values
    // a head two would fit).  Fewer row tiles than CUs are cut along the keys where
    // that pays: c chunks save steps of 64 keys, and cost the joining launch (5 us)
    // and the partial results' way to memory and back (5 TB/s).  A step is charged
    // 1.9 us at 128 values a head, as measured for unrotated NVFP4 in bf16; forms
    // with more products in a step take up to three times that and are cut no
    // finer.  512 queries of 32 heads alone are not cut (26 us, 33 with two
    // chunks), after 16384 keys they are (180 against 511 us; MXFP4 binary32 416
    // against 799).  Of 70 to 1024 rows over 512 to 65536 keys, NVFP4 bf16 and MXFP4
    // binary32, 64, 128 and 256 values, none was slower than without the cut: 96
    // rows of one head over 1024 keys 21 against 33 us, over 8192 30 against 197.
    const int64_t most_cuts = (kCus + units - 1) / units;
    double best = 0.0;
    int64_t chunk = 0;
    for (int64_t c = 1; c <= most_cuts; ++c) {
        const int64_t keys = ((span + c - 1) / c + 255) / 256 * 256;
        const double us = (double)((keys + 63) / 64) * 1.9 * a.kv.head_dim / 128 +
                          (c > 1 ? 5.0 + 2.0 * (double)pairs * rows * c * (a.kv.head_dim * 4 + 8) / 5e6 : 0.0);
        if (c == 1 || us < best) {
            best = us;
            chunk = keys;
        }
    }
    p.chunk = (int)(chunk < 256 ? 256 : chunk);
    chunk = p.chunk;
    const int64_t chunks = span <= chunk ? 1 : (span + chunk - 1) / chunk;
    if (units > most / chunks || (chunks > 1 && pairs > most / rows))
        return p; // groups == 0: refused
    p.groups = (int)(units * chunks);
    p.chunks = (int)chunks;
    if (chunks > 1) {
        const size_t all = (size_t)pairs * rows * chunks;
        p.workspace = round256(all * 8) + all * a.kv.head_dim * 4;
    }
    return p;
}

} // namespace fp4q
