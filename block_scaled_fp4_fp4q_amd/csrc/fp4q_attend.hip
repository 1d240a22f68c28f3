// fp4q_attend.hip -- attention over the 4-bit KV cache.
//
//   out_i = sum_j p_ij v_j,   p_ij = exp(scale q_i.k_j - lse_i)
//
// in one pass over the keys with a running maximum and sum.  A code times its
// E4M3 scale has at most six significant bits and lies in [2^-10, 2688], so
// NVFP4 rows enter the matrix cores exactly as f16; a code times 2^e is exact
// in bf16, so MXFP4 rows enter as bf16.  The global scales are one binary32
// factor of the logits (K) and of the output (V).  Rows that are stored
// rotated are never rotated back: q.k = (Hq).(Hk) and sum p v = H sum p (Hv),
// with H the orthonormal block Hadamard, so the queries are rotated once and
// so is the output.
//
// Parts.  A 16-bit operand that is not exact is given as the sum of up to
// three 16-bit parts, one matrix product each: q of bf16 needs one (f16 after a
// power of two per row that brings its largest value to [2^14, 2^15): what
// falls below f16's range is under 2^-38 of that value), rotated or binary32 q
// two in f16 (22 bits) or three in bf16 (24 bits).  Probabilities take one f16
// part (11 bits, 8 times finer than the bf16 result), two bf16 parts, and one
// part more for binary32 results.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "fp4q_device.h"
#include "fp4q_attend_index.h"
#include "fp4q_kv_launch.h"

namespace fp4q {

namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 b16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 b16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---- number formats ----------------------------------------------------------

// two 16-bit operands of the matrix cores, and the product of a 16x32 by a
// 32x16 tile of them
template <bool MX>
__device__ __forceinline__ f32x4 mfma16(u32x4 x, u32x4 y, f32x4 c)
{
    if constexpr (MX)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b16x8, x), __builtin_bit_cast(b16x8, y), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
}

// the 16-bit images of two binary32 values (nearest even), and what they leave
template <bool MX>
__device__ __forceinline__ uint32_t take_part(float& x, float& y)
{
    if constexpr (MX) {
        const b16x2 h = {(__bf16)x, (__bf16)y};
        x -= (float)h[0];
        y -= (float)h[1];
        return __builtin_bit_cast(uint32_t, h);
    } else {
        const f16x2 h = {(_Float16)x, (_Float16)y};
        x -= (float)h[0];
        y -= (float)h[1];
        return __builtin_bit_cast(uint32_t, h);
    }
}

// binary32 step of an E8M0 byte for the conversions, which apply its exponent
// alone (255 stands for NaN)
__device__ __forceinline__ float e8m0_step(uint32_t byte) { return __uint_as_float(byte << 23); }

// the f16 values of E4M3 bytes 0 and 1 (SEL 0) or 2 and 3 of a word, exact
template <bool HI>
__device__ __forceinline__ f16x2 e4m3_pair(uint32_t w)
{
    return __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
}

template <int SEL>
__device__ __forceinline__ f16x2 fp4_pair_f16(uint32_t w)
{
    return __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, SEL));
}

template <int SEL>
__device__ __forceinline__ uint32_t fp4_pair_bf16(uint32_t w, float step)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, step, SEL));
}

// eight codes of one row (NVFP4: times their scale s, given twice)
__device__ __forceinline__ u32x4 expand_f16(uint32_t w, f16x2 s)
{
    u32x4 r;
    r.x = __builtin_bit_cast(uint32_t, fp4_pair_f16<0>(w) * s);
    r.y = __builtin_bit_cast(uint32_t, fp4_pair_f16<1>(w) * s);
    r.z = __builtin_bit_cast(uint32_t, fp4_pair_f16<2>(w) * s);
    r.w = __builtin_bit_cast(uint32_t, fp4_pair_f16<3>(w) * s);
    return r;
}

__device__ __forceinline__ u32x4 expand_bf16(uint32_t w, float step)
{
    u32x4 r;
    r.x = fp4_pair_bf16<0>(w, step);
    r.y = fp4_pair_bf16<1>(w, step);
    r.z = fp4_pair_bf16<2>(w, step);
    r.w = fp4_pair_bf16<3>(w, step);
    return r;
}

// ---- lanes -----------------------------------------------------------------

// the maximum (sum) over the four lanes n, n+16, n+32, n+48, in all of them
__device__ __forceinline__ float column_max(float x)
{
    x = __builtin_fmaxf(x, __shfl_xor(x, 16, 64));
    return __builtin_fmaxf(x, __shfl_xor(x, 32, 64));
}

__device__ __forceinline__ float column_sum(float x)
{
    x += __shfl_xor(x, 16, 64);
    return x + __shfl_xor(x, 32, 64);
}

// Orthonormal Hadamard of the blocks of B values of a row of D whose quarter g
// (D/4 values) each of the lanes n + 16 g holds.
template <int B, int D>
__device__ __forceinline__ void rotate_quarter(float* v, int g)
{
    constexpr int N = D / 4;
    constexpr int W = N < B ? N : B; // butterflies within the lane
#pragma unroll
    for (int h = 1; h < W; h *= 2)
#pragma unroll
        for (int i = 0; i < N; i += 2 * h)
#pragma unroll
            for (int j = i; j < i + h; ++j) {
                const float p = v[j], q = v[j + h];
                v[j] = p + q;
                v[j + h] = p - q;
            }
    if constexpr (N < B) { // D = 64 in blocks of 32: lanes g and g ^ 1 share one
        static_assert(2 * N == B, "one exchange");
        const float sign = (g & 1) ? -1.0f : 1.0f;
#pragma unroll
        for (int j = 0; j < N; ++j)
            v[j] = __builtin_fmaf(sign, v[j], __shfl_xor(v[j], 16, 64));
    }
    const float c = (B == 16) ? 0.25f : __uint_as_float(0x3E3504F3u); // fl32(1/sqrt(B))
#pragma unroll
    for (int j = 0; j < N; ++j)
        v[j] *= c;
}

// ---- the cache ----------------------------------------------------------------

// Raw buffer resource over `bytes` bytes from p (uniform): a load past the end
// gives zeros, so rows behind the last key read as zero codes with zero
// scales, whatever the memory holds.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const uint8_t* p, int bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, bytes, 0x00027000);
}

__device__ __forceinline__ int64_t uniform64(int64_t x)
{
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)x >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// The granules of keys [k0, k1) of sequence b (k0 a multiple of 16) into LDS,
// by the whole workgroup.
__device__ __forceinline__ void find_granules(const AttendArgs& a, int b, int head, int k0, int k1, Granule* g)
{
    for (int j = threadIdx.x; j * 16 < k1 - k0; j += kThreads)
        g[j] = granule_at(a, b, head, k0 + j * 16);
}

// ---- few queries: one wave per 16 rows and 32 keys ------------------------------
//
// S^T = K Q^T and O^T = V^T P^T by 16x16x32 products whose accumulators give a
// lane one query (column n = lane % 16), so the running maximum and sum are
// one value per lane and the probabilities never move between lanes: the
// accumulator of S^T is, after rounding, the operand of O^T.  Which key, and
// which value of a row, stands at which place of an operand is free as long as
// both operands agree.  With g = lane / 16:
//   - values of a row: lane g holds the quarter g, D/8 contiguous bytes of
//     codes, so one wide load brings 16 whole rows;
//   - keys of a tile: row 4 j + i of the first product is key 4 i + j, so a
//     lane's four logits are keys g, g+4, g+8, g+12, and each load of V's
//     codes brings four whole consecutive rows;
//   - V's code words of two keys are interleaved by nibbles (two shifts and two
//     bit selects for 16 values), after which the conversion's pair is the
//     two keys of one value, the pair that the product wants.
// Nothing passes through LDS in the loop, and the codes of the next 32 keys
// are loaded while these are computed.

template <bool MX, int D>
struct Tile {
    static constexpr int KW = D / 32;            // code words of a lane's quarter row
    static constexpr int VB = D / 32;            // code bytes of a lane's D/16 values
    static constexpr int VW = VB < 4 ? 1 : VB / 4;
    uint32_t k[2][KW], ks[2];
    uint32_t v[2][4][VW], vs[2][4];
    bool lost[2]; // 16 keys whose page does not exist (uniform)
};

// a lane's fixed byte offsets within 16 rows
struct Lane {
    int k, ks, v[4], vs[4];
};

template <bool MX, int D>
__device__ __forceinline__ Lane lane_offsets(const AttendArgs& a, int n, int g)
{
    constexpr int B = MX ? 32 : 16;
    Lane o;
    const int row = 4 * (n & 3) + (n >> 2);
    o.k = row * (int)a.kv.c_token + g * (D / 8);
    o.ks = row * (int)a.kv.s_token + (g * (D / 4)) / B;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o.v[i] = (4 * i + g) * (int)a.kv.c_token + n * (D / 32);
        o.vs[i] = (4 * i + g) * (int)a.kv.s_token + (n * (D / 16)) / B;
    }
    return o;
}

// the codes and scales of keys [key, key + 32), of which those from `end` on
// are not read
template <bool MX, int D>
__device__ __forceinline__ void load_tile(const AttendArgs& a, const Granule* g, int key, int end,
                                          const Lane& o, Tile<MX, D>& t)
{
    constexpr int B = MX ? 32 : 16;
    constexpr int QS = D / 4 >= B ? D / 4 / B : 1; // scales of a quarter row
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int rows = end - key - 16 * h;
        rows = rows < 0 ? 0 : (rows > 16 ? 16 : rows);
        const Granule at = g[rows > 0 ? h : 0];
        const int64_t co = uniform64(at.codes), so = uniform64(at.scales);
        t.lost[h] = rows > 0 && co < 0;
        if (co < 0)
            rows = 0; // read nothing
        const int cb = rows > 0 ? (rows - 1) * (int)a.kv.c_token + D / 2 : 0;
        const int sb = rows > 0 ? (rows - 1) * (int)a.kv.s_token + D / B : 0;
        const auto kc = buffer_of(a.kv.codes[0] + co, cb), vc = buffer_of(a.kv.codes[1] + co, cb);
        const auto ks = buffer_of(a.kv.scales[0] + so, sb), vs = buffer_of(a.kv.scales[1] + so, sb);
        if constexpr (D == 64) {
            const u32x2 w = __builtin_amdgcn_raw_buffer_load_b64(kc, o.k, 0, 0);
            t.k[h][0] = w.x;
            t.k[h][1] = w.y;
        } else {
#pragma unroll
            for (int j = 0; j < D / 128; ++j) {
                const u32x4 w = __builtin_amdgcn_raw_buffer_load_b128(kc, o.k + 16 * j, 0, 0);
                t.k[h][4 * j + 0] = w.x;
                t.k[h][4 * j + 1] = w.y;
                t.k[h][4 * j + 2] = w.z;
                t.k[h][4 * j + 3] = w.w;
            }
        }
        if constexpr (QS == 1)
            t.ks[h] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(ks, o.ks, 0, 0);
        else if constexpr (QS == 2)
            t.ks[h] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(ks, o.ks, 0, 0);
        else
            t.ks[h] = __builtin_amdgcn_raw_buffer_load_b32(ks, o.ks, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (D == 64) {
                t.v[h][i][0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(vc, o.v[i], 0, 0);
            } else if constexpr (D == 128) {
                t.v[h][i][0] = __builtin_amdgcn_raw_buffer_load_b32(vc, o.v[i], 0, 0);
            } else {
                const u32x2 w = __builtin_amdgcn_raw_buffer_load_b64(vc, o.v[i], 0, 0);
                t.v[h][i][0] = w.x;
                t.v[h][i][Tile<MX, D>::VW - 1] = w.y;
            }
            t.vs[h][i] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(vs, o.vs[i], 0, 0);
        }
    }
}

// the 16-bit operand of K's values 8c .. 8c+7 of the lane's quarter row
template <bool MX, int D>
__device__ __forceinline__ u32x4 k_operand(const Tile<MX, D>& t, int h, int c)
{
    constexpr int B = MX ? 32 : 16;
    const int s = (8 * c) / B; // scale of these eight values among the lane's
    if constexpr (MX) {
        return expand_bf16(t.k[h][c], e8m0_step((t.ks[h] >> (8 * s)) & 0xFFu));
    } else {
        const f16x2 two = s < 2 ? e4m3_pair<false>(t.ks[h]) : e4m3_pair<true>(t.ks[h]);
        const _Float16 one = two[s & 1];
        return expand_f16(t.k[h][c], f16x2{one, one});
    }
}

// V's operands of the lane's value pair (2 m, 2 m + 1): eight keys each
template <bool MX, int D>
__device__ __forceinline__ void v_operands(const Tile<MX, D>& t, int m, u32x4& even, u32x4& odd)
{
    const int w = m / 4, sel = m % 4;
    uint32_t e[4], o[4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const uint32_t x = t.v[h][2 * p][w], y = t.v[h][2 * p + 1][w];
            const int at = 2 * h + p;
            if constexpr (MX) {
                // each key's step goes into its own conversion, and the pairs
                // (value, value + 1) of two keys are then exchanged
                const float sx = e8m0_step(t.vs[h][2 * p]), sy = e8m0_step(t.vs[h][2 * p + 1]);
                uint32_t cx, cy;
                switch (sel) {
                case 0: cx = fp4_pair_bf16<0>(x, sx); cy = fp4_pair_bf16<0>(y, sy); break;
                case 1: cx = fp4_pair_bf16<1>(x, sx); cy = fp4_pair_bf16<1>(y, sy); break;
                case 2: cx = fp4_pair_bf16<2>(x, sx); cy = fp4_pair_bf16<2>(y, sy); break;
                default: cx = fp4_pair_bf16<3>(x, sx); cy = fp4_pair_bf16<3>(y, sy); break;
                }
                e[at] = __builtin_amdgcn_perm(cy, cx, 0x05040100u);
                o[at] = __builtin_amdgcn_perm(cy, cx, 0x07060302u);
            } else {
                const uint32_t lo = (x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u);
                const uint32_t hi = ((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u);
                const f16x2 s = e4m3_pair<false>(t.vs[h][2 * p] | (t.vs[h][2 * p + 1] << 8));
                f16x2 ce, co;
                switch (sel) {
                case 0: ce = fp4_pair_f16<0>(lo); co = fp4_pair_f16<0>(hi); break;
                case 1: ce = fp4_pair_f16<1>(lo); co = fp4_pair_f16<1>(hi); break;
                case 2: ce = fp4_pair_f16<2>(lo); co = fp4_pair_f16<2>(hi); break;
                default: ce = fp4_pair_f16<3>(lo); co = fp4_pair_f16<3>(hi); break;
                }
                e[at] = __builtin_bit_cast(uint32_t, ce * s);
                o[at] = __builtin_bit_cast(uint32_t, co * s);
            }
        }
    even = u32x4{e[0], e[1], e[2], e[3]};
    odd = u32x4{o[0], o[1], o[2], o[3]};
}

// where a workgroup's partial result for one query row goes
struct Partial {
    float* o;     // [rows, chunks, D] sums of p v, in units of V's global scale
    float2* stat; // [rows, chunks] (maximum in log2 units, sum)
};

__device__ __forceinline__ Partial partials_of(const AttendArgs& a, const AttendPlan& p)
{
    const int64_t rows = (int64_t)a.batch * a.kv.heads * a.max_q * a.group;
    Partial r;
    r.stat = static_cast<float2*>(a.workspace);
    const size_t stat = (size_t)rows * p.chunks * sizeof(float2);
    r.o = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + ((stat + 255) & ~(size_t)255));
    return r;
}

// one row's quarter of the result, from its sums, their total and maximum
template <int B, int D>
__device__ __forceinline__ void finish_quarter(const AttendArgs& a, const Extent& e, int head, int r, int g,
                                               float* o, float m, float l, float Sv)
{
    const float inv = l == 0.0f ? 0.0f : Sv / l; // nothing seen: zeros
#pragma unroll
    for (int j = 0; j < D / 4; ++j)
        o[j] *= inv;
    if (a.rotate)
        rotate_quarter<B, D>(o, g);
    const int i = r / a.group, j = r - i * a.group;
    if (i >= e.qn)
        return;
    const int64_t row = e.q0 + i;
    const int qh = head * a.group + j;
    if (a.lse && g == 0)
        a.lse[row * a.q_heads + qh] = l == 0.0f ? -__builtin_huge_valf() : (m + __builtin_log2f(l)) * kLn2;
    if (a.bf16) {
        uint16_t* y = static_cast<uint16_t*>(a.out) + row * a.o_row + qh * a.o_head + g * (D / 4);
#pragma unroll
        for (int t = 0; t < D / 32; ++t) {
            u32x4 w;
            w.x = bf16_pair(o[8 * t + 0], o[8 * t + 1]);
            w.y = bf16_pair(o[8 * t + 2], o[8 * t + 3]);
            w.z = bf16_pair(o[8 * t + 4], o[8 * t + 5]);
            w.w = bf16_pair(o[8 * t + 6], o[8 * t + 7]);
            reinterpret_cast<u32x4*>(y)[t] = w;
        }
    } else {
        float* y = static_cast<float*>(a.out) + row * a.o_row + qh * a.o_head + g * (D / 4);
#pragma unroll
        for (int t = 0; t < D / 16; ++t)
            reinterpret_cast<f32x4*>(y)[t] = f32x4{o[4 * t], o[4 * t + 1], o[4 * t + 2], o[4 * t + 3]};
    }
}

// The running maximum is raised only where a logit passes it by more than
// kLazy, in log2 units; probabilities are kept times 2^kUp, so that they stay
// within f16 (2^(kLazy + kUp) = 2^15) and those down to 2^-33 of the largest
// are still told from zero.
constexpr float kLazy = 6.0f, kUp = 9.0f;

template <bool MX, int D, int NQ, int NP>
__global__ __launch_bounds__(kThreads) void attend_few(const AttendArgs a, const AttendPlan p)
{
    constexpr int B = MX ? 32 : 16;
    constexpr int KW = D / 32;
    constexpr int N = D / 4;
    __shared__ Granule granule[kMaxChunk / 16 + 2];
    __shared__ float merge_o[2][16][D + 4];
    __shared__ float2 merge_s[2][16];

    // blocks: chunk fastest, then row tile, KV head, sequence
    int64_t id = blockIdx.x;
    const int chunk = (int)(id % p.chunks);
    id /= p.chunks;
    const int tile = (int)(id % p.tiles);
    id /= p.tiles;
    const int head = (int)(id % a.kv.heads);
    const int b = (int)(id / a.kv.heads);

    const Extent e = extent_of(a, b);
    const int rows = e.qn * a.group;
    const int r0 = tile * p.rows_per_tile;
    if (r0 >= rows)
        return;
    const int r1 = r0 + p.rows_per_tile < rows ? r0 + p.rows_per_tile : rows;
    int lo, hi;
    tile_keys(a, e, r0, r1, lo, hi);
    if (chunk >= chunks_of(p, lo, hi))
        return; // the joining kernel does not read it
    const int k0 = lo + chunk * p.chunk;
    const int k1 = hi - k0 < p.chunk ? hi : k0 + p.chunk;
    find_granules(a, b, head, k0, k1, granule);

    // this wave's 16 rows and its share of the keys
    const int tiles16 = p.rows_per_tile / 16; // 1, 2 or 4
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int n = lane & 15, g = lane >> 4;
    const int part = wave % tiles16, turn = wave / tiles16, turns = kWaves / tiles16;
    const int r = r0 + part * 16 + n;
    const bool live = r < r1;
    int row_lo = 0, row_hi = 0;

    // the row's quarter, rotated, as parts
    u32x4 q[NQ][KW];
    float factor; // of the row's logits, to log2 units
    {
        float v[N];
#pragma unroll
        for (int j = 0; j < N; ++j)
            v[j] = 0.0f;
        if (live) {
            const int i = r / a.group, j = r - i * a.group;
            seen_by(a, e, i, row_lo, row_hi);
            const int64_t at = (e.q0 + i) * a.q_row + (head * a.group + j) * a.q_head + g * N;
            if (a.bf16) {
                const u32x4* x = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.q) + at);
#pragma unroll
                for (int t = 0; t < N / 8; ++t) {
                    const u32x4 w = x[t];
                    v[8 * t + 0] = bf16_lo(w.x); v[8 * t + 1] = bf16_hi(w.x);
                    v[8 * t + 2] = bf16_lo(w.y); v[8 * t + 3] = bf16_hi(w.y);
                    v[8 * t + 4] = bf16_lo(w.z); v[8 * t + 5] = bf16_hi(w.z);
                    v[8 * t + 6] = bf16_lo(w.w); v[8 * t + 7] = bf16_hi(w.w);
                }
            } else {
                const f32x4* x = reinterpret_cast<const f32x4*>(static_cast<const float*>(a.q) + at);
#pragma unroll
                for (int t = 0; t < N / 4; ++t) {
                    const f32x4 w = x[t];
                    v[4 * t + 0] = w.x; v[4 * t + 1] = w.y; v[4 * t + 2] = w.z; v[4 * t + 3] = w.w;
                }
            }
        }
        if (a.rotate)
            rotate_quarter<B, D>(v, g);
        factor = a.scale * kLog2e;
        if constexpr (!MX) {
            factor *= *a.kv.global[0];
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < N; ++j)
                top = __builtin_fmaxf(top, __builtin_fabsf(v[j]));
            top = column_max(top);
            // a power of two to [2^14, 2^15); zero and non-finite rows stay
            const int up = (top > 0.0f && top < __builtin_huge_valf())
                               ? 141 - (int)(__float_as_uint(top) >> 23) : 0;
#pragma unroll
            for (int j = 0; j < N; ++j)
                v[j] = __builtin_ldexpf(v[j], up);
            factor = __builtin_ldexpf(factor, -up);
        }
#pragma unroll
        for (int s = 0; s < NQ; ++s)
#pragma unroll
            for (int c = 0; c < KW; ++c) {
                q[s][c].x = take_part<MX>(v[8 * c + 0], v[8 * c + 1]);
                q[s][c].y = take_part<MX>(v[8 * c + 2], v[8 * c + 3]);
                q[s][c].z = take_part<MX>(v[8 * c + 4], v[8 * c + 5]);
                q[s][c].w = take_part<MX>(v[8 * c + 6], v[8 * c + 7]);
            }
    }
    __syncthreads(); // granules

    f32x4 o[D / 16];
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
        o[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float m = -__builtin_huge_valf(), l = 0.0f;
    const Lane at = lane_offsets<MX, D>(a, n, g);
    const int step = turns * kTileKeys;
    // keys that every row of the workgroup sees need no mask
    int all_lo, all_hi, unused;
    seen_by(a, e, (r1 - 1) / a.group, all_lo, unused);
    seen_by(a, e, r0 / a.group, unused, all_hi);

    Tile<MX, D> now, next;
    int key = k0 + turn * kTileKeys;
    if (key < k1)
        load_tile<MX, D>(a, granule + (key - k0) / 16, key, k1, at, now);
    for (; key < k1; key += step) {
        if (key + step < k1)
            load_tile<MX, D>(a, granule + (key + step - k0) / 16, key + step, k1, at, next);
        f32x4 s[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            s[h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < KW; ++c) {
                const u32x4 k = k_operand<MX, D>(now, h, c);
#pragma unroll
                for (int t = NQ - 1; t >= 0; --t) // small parts first
                    s[h] = mfma16<MX>(k, q[t][c], s[h]);
            }
        }
        float x[8];
        float top = -__builtin_huge_valf();
        const bool whole = key >= all_lo && key + kTileKeys <= all_hi && key + kTileKeys <= k1 &&
                           !now.lost[0] && !now.lost[1];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float t = s[h][i] * factor;
                if (!whole) {
                    const int k = key + 16 * h + 4 * i + g;
                    t = now.lost[h] ? __builtin_nanf("") : t;
                    t = (k >= row_lo && k < row_hi) ? t : -__builtin_huge_valf();
                }
                x[4 * h + i] = t;
                top = __builtin_fmaxf(top, t);
            }
        top = column_max(top);
        if (__builtin_amdgcn_ballot_w64(top > m + kLazy) != 0) {
            const float raised = __builtin_fmaxf(m, top);
            const float f = m == raised ? 1.0f : __builtin_amdgcn_exp2f(m - raised);
            m = raised;
            l *= f;
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
                o[c] *= f;
        }
        const float base = m == -__builtin_huge_valf() ? 0.0f : m - kUp;
        u32x4 pr[NP];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = __builtin_amdgcn_exp2f(x[j] - base);
            l += x[j];
        }
#pragma unroll
        for (int t = 0; t < NP; ++t) {
            pr[t].x = take_part<MX>(x[0], x[1]);
            pr[t].y = take_part<MX>(x[2], x[3]);
            pr[t].z = take_part<MX>(x[4], x[5]);
            pr[t].w = take_part<MX>(x[6], x[7]);
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            u32x4 even, odd;
            v_operands<MX, D>(now, c, even, odd);
#pragma unroll
            for (int t = NP - 1; t >= 0; --t) {
                o[2 * c] = mfma16<MX>(even, pr[t], o[2 * c]);
                o[2 * c + 1] = mfma16<MX>(odd, pr[t], o[2 * c + 1]);
            }
        }
        now = next;
    }
    l = column_sum(l);
    if (e.bad)
        l = __builtin_nanf("");

    // join the waves that share these rows: half of them hand over, in turn
    // (kUp cancels: l and o carry it alike until the end)
    for (int half = turns / 2; half >= 1; half /= 2) {
        __syncthreads();
        const int slot = part + (turn - half) * tiles16;
        if (turn >= half && turn < 2 * half) {
            if (g == 0)
                merge_s[slot][n] = float2{m, l};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < D / 16; c += 4)
                    *reinterpret_cast<f32x4*>(&merge_o[slot][n][g * N + i * (D / 16) + c]) =
                        f32x4{o[c][i], o[c + 1][i], o[c + 2][i], o[c + 3][i]};
        }
        __syncthreads();
        if (turn < half) {
            const int from = part + turn * tiles16;
            const float2 other = merge_s[from][n];
            const float raised = __builtin_fmaxf(m, other.x);
            const float f0 = m == raised ? 1.0f : __builtin_amdgcn_exp2f(m - raised);
            const float f1 = other.x == raised ? 1.0f : __builtin_amdgcn_exp2f(other.x - raised);
            m = raised;
            l = l * f0 + other.y * f1;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < D / 16; c += 4) {
                    const f32x4 t = *reinterpret_cast<const f32x4*>(&merge_o[from][n][g * N + i * (D / 16) + c]);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        o[c + j][i] = o[c + j][i] * f0 + t[j] * f1;
                }
        }
    }
    if (turn != 0)
        return;
    float y[N];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
            y[i * (D / 16) + c] = o[c][i];
    // back from 2^kUp: as the maximum's unit, exactly
    m = m - kUp;
    if (p.chunks == 1) {
        // (rows past the last one take part in the rotation's exchanges)
        finish_quarter<B, D>(a, e, head, live ? r : 0x7FFFFFFF, g, y, m, l, MX ? 1.0f : *a.kv.global[1]);
    } else if (live) {
        const Partial w = partials_of(a, p);
        const int64_t at_row = (((int64_t)b * a.kv.heads + head) * a.max_q * a.group + r) * p.chunks + chunk;
        if (g == 0)
            w.stat[at_row] = float2{m, l};
        float* to = w.o + at_row * D + g * N;
#pragma unroll
        for (int j = 0; j < N; j += 4)
            *reinterpret_cast<f32x4*>(to + j) = f32x4{y[j], y[j + 1], y[j + 2], y[j + 3]};
    }
}

// ---- joining the chunks of a row ---------------------------------------------------
//
// One workgroup per query row: D/4 lanes hold four values each, and the
// 256 / (D/4) groups of lanes take every so-manieth chunk; reads every partial
// result once.
template <bool MX, int D>
__global__ __launch_bounds__(kThreads) void attend_join(const AttendArgs a, const AttendPlan p)
{
    constexpr int B = MX ? 32 : 16;
    constexpr int L = D / 4, T = kThreads / L;
    __shared__ f32x4 sum[T][L];
    __shared__ float red[kWaves];
    const int rows_seq = a.max_q * a.group;
    const int64_t id = blockIdx.x;
    const int r = (int)(id % rows_seq);
    const int head = (int)(id / rows_seq % a.kv.heads);
    const int b = (int)(id / rows_seq / a.kv.heads);
    const Extent e = extent_of(a, b);
    const int rows = e.qn * a.group;
    if (r >= rows)
        return;
    const int r0 = r - r % p.rows_per_tile;
    int lo, hi;
    tile_keys(a, e, r0, r0 + p.rows_per_tile < rows ? r0 + p.rows_per_tile : rows, lo, hi);
    const int chunks = chunks_of(p, lo, hi);
    const Partial w = partials_of(a, p);
    const float2* stat = w.stat + id * p.chunks;
    const float* part = w.o + id * p.chunks * D;

    // the maximum over the chunks (a NaN is in the sums, never in a maximum)
    float m = -__builtin_huge_valf();
    for (int c = threadIdx.x; c < chunks; c += kThreads)
        m = __builtin_fmaxf(m, stat[c].x);
    m = wave_max(m);
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kWaves; ++t)
        m = __builtin_fmaxf(m, red[t]);

    const int j = threadIdx.x % L, turn = threadIdx.x / L;
    f32x4 o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float l = 0.0f;
    for (int c = turn; c < chunks; c += T) {
        const float2 s = stat[c];
        const float f = s.x == m ? 1.0f : __builtin_amdgcn_exp2f(s.x - m);
        const f32x4 t = *reinterpret_cast<const f32x4*>(part + (int64_t)c * D + 4 * j);
        l += s.y * f;
        o += t * f;
    }
    sum[turn][j] = o;
    __shared__ float total[T];
    if (j == 0)
        total[turn] = l;
    __syncthreads();
    if (threadIdx.x >= 64)
        return;
    // D = 256: a whole wave; else the lanes past L repeat the first ones
    o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    l = 0.0f;
#pragma unroll
    for (int t = 0; t < T; ++t) {
        o += sum[t][j];
        l += total[t];
    }
    const float inv = l == 0.0f ? 0.0f : (MX ? 1.0f : *a.kv.global[1]) / l;
    o *= inv;
    if (a.rotate) {
        const float p0 = o.x + o.y, p1 = o.x - o.y, p2 = o.z + o.w, p3 = o.z - o.w;
        o = f32x4{p0 + p2, p1 + p3, p0 - p2, p1 - p3};
#pragma unroll
        for (int h = 1; h < B / 4; h *= 2) {
            const float sign = (j & h) ? -1.0f : 1.0f;
#pragma unroll
            for (int t = 0; t < 4; ++t)
                o[t] = __builtin_fmaf(sign, o[t], __shfl_xor(o[t], h, 64));
        }
        o *= (B == 16) ? 0.25f : __uint_as_float(0x3E3504F3u);
    }
    if (threadIdx.x >= L)
        return;
    const int i = r / a.group;
    const int qh = head * a.group + (r - i * a.group);
    const int64_t row = e.q0 + i;
    if (a.lse && j == 0)
        a.lse[row * a.q_heads + qh] = l == 0.0f ? -__builtin_huge_valf() : (m + __builtin_log2f(l)) * kLn2;
    if (a.bf16) {
        uint16_t* y = static_cast<uint16_t*>(a.out) + row * a.o_row + qh * a.o_head;
        reinterpret_cast<u32x2*>(y)[j] = u32x2{bf16_pair(o.x, o.y), bf16_pair(o.z, o.w)};
    } else {
        float* y = static_cast<float*>(a.out) + row * a.o_row + qh * a.o_head;
        reinterpret_cast<f32x4*>(y)[j] = o;
    }
}

template <bool MX, int D>
hipError_t launch_few(const AttendArgs& a, const AttendPlan& p)
{
    const int64_t groups = (int64_t)a.batch * a.kv.heads * p.tiles * p.chunks;
    const dim3 grid((uint32_t)groups);
    if (!a.bf16)
        attend_few<MX, D, MX ? 3 : 2, MX ? 3 : 2><<<grid, kThreads, 0, a.stream>>>(a, p);
    else if (a.rotate)
        attend_few<MX, D, MX ? 3 : 2, MX ? 2 : 1><<<grid, kThreads, 0, a.stream>>>(a, p);
    else
        attend_few<MX, D, 1, MX ? 2 : 1><<<grid, kThreads, 0, a.stream>>>(a, p);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || p.chunks == 1)
        return err;
    attend_join<MX, D><<<dim3((uint32_t)((int64_t)a.batch * a.kv.heads * a.max_q * a.group)), kThreads, 0, a.stream>>>(a, p);
    return hipGetLastError();
}

template <bool MX>
hipError_t launch_dim(const AttendArgs& a, const AttendPlan& p)
{
    switch (a.kv.head_dim) {
    case 64: return launch_few<MX, 64>(a, p);
    case 128: return launch_few<MX, 128>(a, p);
    default: return launch_few<MX, 256>(a, p);
    }
}

} // namespace

AttendPlan plan_attend(const AttendArgs& a) { return plan_of(a); }

hipError_t launch_attend(const AttendArgs& a, const AttendPlan& p)
{
    return a.kv.mx ? launch_dim<true>(a, p) : launch_dim<false>(a, p);
}

} // namespace fp4q
