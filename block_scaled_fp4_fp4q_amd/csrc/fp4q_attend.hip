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

constexpr uint32_t kNanScales = 0xFFFFFFFFu; // bytes that are NaN in E4M3 and in E8M0
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

// the last digit of `id` to base `n`, which leaves it
__device__ __forceinline__ uint32_t take_digit(uint32_t& id, int n)
{
    const uint32_t q = id / (uint32_t)n, r = id - q * (uint32_t)n;
    id = q;
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

// What the queries are multiplied by so that the largest product is the largest
// logit: the sign of scale S.  A global scale that is not finite makes them NaN
// (in the factor of the logits it would meet the infinities of masked keys).
__device__ __forceinline__ float query_sign(float scale, float S)
{
    if (!(__builtin_fabsf(S) < __builtin_huge_valf()))
        return __builtin_nanf("");
    return (scale < 0.0f) != (S < 0.0f) ? -1.0f : 1.0f;
}

// The rest of scale S 2^-up, in log2 units: finite and not zero, since it meets
// infinities and zeros.  Exponents are added apart: scale S may be far below
// binary32 where large queries (up < 0) bring the logits back.
__device__ __forceinline__ float logit_factor(float scale, float S, int up)
{
    const float c = __builtin_fabsf(scale) * kLog2e;
    S = __builtin_fabsf(S);
    S = S < __builtin_huge_valf() ? S : 1.0f;
    const float f = __builtin_ldexpf(__builtin_amdgcn_frexp_mantf(c) * __builtin_amdgcn_frexp_mantf(S),
                                     __builtin_amdgcn_frexp_expf(c) + __builtin_amdgcn_frexp_expf(S) - up);
    return __builtin_fminf(__builtin_fmaxf(f, 0x1p-126f), 0x1.fffffep127f);
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
// scales, whatever the memory holds.  (A size that the compiler holds in a
// vector register would turn every load into a loop over the lanes.)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const uint8_t* p, int bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0,
                                             __builtin_amdgcn_readfirstlane(bytes), 0x00027000);
}

__device__ __forceinline__ int64_t uniform64(int64_t x)
{
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)x >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// The granules of keys [k0, k1) of sequence b (k0 a multiple of 16) into LDS,
// by the whole workgroup.  Those wholly below key `first` are not looked up.
template <int THREADS>
__device__ __forceinline__ void find_granules(const AttendArgs& a, int b, int head, int k0, int k1, int first, Granule* g)
{
    for (int j = threadIdx.x; j * 16 < k1 - k0; j += THREADS) {
        const int key = k0 + j * 16;
        g[j] = key + 16 <= first ? Granule{0, 0} : granule_at(a, b, head, key);
    }
}

// A V row below the first key that is seen meets probabilities of zero, but its
// scale may be NaN: its scales are read from past every buffer's end, as zeros.
// Such keys stand only in the first tile of a workgroup (EDGE); K's need no
// care, the mask replaces their logits.
template <bool EDGE>
__device__ __forceinline__ int seen_offset(int offset, int key, int first)
{
    return EDGE && key < first ? 0x7FFFFFFF : offset;
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
//
// Bound by HBM where there are many keys: 64 sequences of 4096 keys and 32 heads
// of 128 values (1.21 GB of codes and scales) take 219 us with the joining's 5,
// 5.65 TB/s over the kernel.  Short of that by the fixed cost of a workgroup
// (about 8 us: lengths, pages, the first loads, the waves' join), which is all
// that 131 keys of 8 heads cost; 32 sequences of up to 8192 keys and 8 heads
// (170 MB, 30 us at that rate) take 45 us with it and with the joining.  With two
// 16-row tiles of a wave and two parts of the probabilities the issue of
// conversions and products joins in: 3 sequences of 4 queries over up to 65521
// keys, MXFP4, 39 us for 95 MB; rotated (three parts of the queries) 51,
// binary32 (three of both) 63.
// Measured and left: codes two tiles ahead (219 -> 245 us), two steps
// unrolled (no change), a pair's workgroups spread by slices of the whole work
// (half the engines idle, 345 us).

template <bool MX, int D>
struct Tile {
    static constexpr int KW = D / 32;            // code words of a lane's quarter row
    static constexpr int VB = D / 32;            // code bytes of a lane's D/16 values
    static constexpr int VW = VB < 4 ? 1 : VB / 4;
    uint32_t k[2][KW], ks[2];
    uint32_t v[2][4][VW], vs[2][4];
    uint32_t lost[2]; // all ones where the 16 keys' page does not exist (uniform)
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

// the codes and scales of keys [key, key + 32), of which those from `end` on,
// and with EDGE V's scales below `first`, are not read; granule 0 is that of key
// k0
template <bool MX, int D, bool EDGE>
__device__ __forceinline__ void load_tile(const AttendArgs& a, const Granule* g, int k0, int key, int first, int end,
                                          int lane16, const Lane& o, Tile<MX, D>& t)
{
    constexpr int B = MX ? 32 : 16;
    constexpr int QS = D / 4 >= B ? D / 4 / B : 1; // scales of a quarter row
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int rows = end - key - 16 * h;
        rows = rows < 0 ? 0 : (rows > 16 ? 16 : rows);
        if (EDGE && key + 16 * h + 16 <= first)
            rows = 0;
        const Granule at = g[rows > 0 ? (key - k0) / 16 + h : 0];
        const int64_t co = uniform64(at.codes), so = uniform64(at.scales);
        const bool lost = rows > 0 && co < 0;
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
        t.lost[h] = lost ? kNanScales : 0u;
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
            t.vs[h][i] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
                vs, seen_offset<EDGE>(o.vs[i], key + 16 * h + 4 * i + lane16, first), 0, 0);
        }
    }
}

// the 16-bit operand of K's values 8c .. 8c+7 of the lane's quarter row
template <bool MX, int D>
__device__ __forceinline__ u32x4 k_operand(const Tile<MX, D>& t, int h, int c)
{
    constexpr int B = MX ? 32 : 16;
    const int s = (8 * c) / B; // scale of these eight values among the lane's
    const uint32_t ks = t.ks[h] | t.lost[h]; // lost: K, and the logits that see it, are NaN
    if constexpr (MX) {
        return expand_bf16(t.k[h][c], e8m0_step((ks >> (8 * s)) & 0xFFu));
    } else {
        const f16x2 two = s < 2 ? e4m3_pair<false>(ks) : e4m3_pair<true>(ks);
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

// Partial results in the workspace, by place: many queries, (row, chunk); few,
// (slot, row of the tile).
struct Partial {
    float* o;     // [places, D] sums of p v, in units of V's global scale
    float2* stat; // [places] (maximum in log2 units, sum)
    int2* pairs;  // few: (first slot, number) of each sequence and KV head
};

__device__ __forceinline__ Partial partials_of(const AttendArgs& a, const AttendPlan& p)
{
    Partial r;
    char* at = static_cast<char*>(a.workspace) + (p.many ? 0 : few_table_bytes(p.groups, a.batch));
    const size_t pairs = (size_t)a.batch * a.kv.heads;
    r.pairs = reinterpret_cast<int2*>(at);
    if (!p.many)
        at += (pairs * sizeof(int2) + 255) & ~(size_t)255;
    const size_t places = p.many ? pairs * a.max_q * a.group * p.chunks : (size_t)2 * p.parts * p.rows_per_tile;
    r.stat = reinterpret_cast<float2*>(at);
    r.o = reinterpret_cast<float*>(at + ((places * sizeof(float2) + 255) & ~(size_t)255));
    return r;
}

// What turns a row's sums into its result: the sums times `by`, times `rest`.
// V's global scale over the sum of probabilities (up to 2^15 for each key) may
// fall below binary32's normal range though the result does not, so a small
// scale is applied times 2^60 and the power of two taken back at the end (exact,
// and 1 for other scales).
struct OutFactor {
    float by, rest;
};

__device__ __forceinline__ OutFactor out_factor(float S, float l)
{
    const bool small = __builtin_fabsf(S) < 0x1p-60f;
    // nothing seen: zeros
    return OutFactor{l == 0.0f ? 0.0f : S * (small ? 0x1p60f : 1.0f) / l, small ? 0x1p-60f : 1.0f};
}

// One query row's result from its sums: eight of the D values (those from
// 8 j on) in each of D/8 lanes, which are lanes of one wave in order.
template <bool MX, int D, bool F32>
__device__ __forceinline__ void finish_row(const AttendArgs& a, const Extent& e, int head, int r, int j,
                                           float* o, float m, float l)
{
    constexpr int B = MX ? 32 : 16;
    const OutFactor f = out_factor(MX ? 1.0f : *a.kv.global[1], l);
#pragma unroll
    for (int k = 0; k < 8; ++k)
        o[k] *= f.by;
    if (a.rotate) {
#pragma unroll
        for (int s = 1; s < 8; s *= 2)
#pragma unroll
            for (int i = 0; i < 8; i += 2 * s)
#pragma unroll
                for (int k = i; k < i + s; ++k) {
                    const float p = o[k], q = o[k + s];
                    o[k] = p + q;
                    o[k + s] = p - q;
                }
#pragma unroll
        for (int s = 1; s < B / 8; s *= 2) {
            const float sign = (j & s) ? -1.0f : 1.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                o[k] = __builtin_fmaf(sign, o[k], __shfl_xor(o[k], s, 64));
        }
        const float c = B == 16 ? 0.25f : __uint_as_float(0x3E3504F3u); // fl32(1/sqrt(B))
#pragma unroll
        for (int k = 0; k < 8; ++k)
            o[k] *= c;
    }
    if constexpr (!MX) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            o[k] *= f.rest;
    }
    const int i = r / a.group;
    const int64_t row = e.q0 + i;
    const int qh = head * a.group + (r - i * a.group);
    if (a.lse && j == 0)
        a.lse[row * a.q_heads + qh] = l == 0.0f ? -__builtin_huge_valf() : (m + __builtin_log2f(l)) * kLn2;
    if constexpr (F32) {
        f32x4* y = reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + row * a.o_row + qh * a.o_head + 8 * j);
        y[0] = f32x4{o[0], o[1], o[2], o[3]};
        y[1] = f32x4{o[4], o[5], o[6], o[7]};
    } else {
        u32x4* y = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + row * a.o_row + qh * a.o_head + 8 * j);
        *y = u32x4{bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3]), bf16_pair(o[4], o[5]), bf16_pair(o[6], o[7])};
    }
}

// The running maximum is raised only where a logit passes it by more than
// kLazy, in log2 units; probabilities are kept times 2^kUp, so that they stay
// within f16 (2^(kLazy + kUp) = 2^15) and those down to 2^-33 of the largest
// are still told from zero.
constexpr float kLazy = 6.0f, kUp = 9.0f;

// the pair of workgroup `blockIdx.x` and its part of it: steps [from, to), the
// number of parts, and the slots of its and of the first part's results
struct FewWhere {
    Extent e;
    int b, head;
    int from, to, parts, slot, first_slot;
};

// inclusive sum over a wave's lanes up to this one, by moves within rows of 16
// and from row to row
__device__ __forceinline__ uint32_t wave_scan(uint32_t v)
{
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, true); // from 1 below, in rows of 16
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, true); // 2
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, true); // 4
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, true); // 8
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, true); // row 0's (2's) sum to row 1 (3)
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, true); // row 1's to rows 2 and 3
    return v;
}

__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// The length of a part, from the sum of all steps and, where one look (64
// sequences, a lane each) shows them all, from the parts that it makes: the
// least length with which all are resident at once, searched from below (a
// second round of a few parts would cost as much as the first); else about that.
__device__ __forceinline__ uint32_t part_length(const AttendArgs& a, const AttendPlan& p, uint32_t total, uint32_t steps)
{
    const uint32_t heads = a.kv.heads, parts = p.parts;
    uint32_t most = few_most(p, total * heads);
    if (a.batch <= 64 && (uint32_t)a.batch * heads <= parts) {
        for (int k = 0; k < 16 && lane_value(wave_scan(few_parts(steps, most)), 63) * heads > parts; ++k)
            most += 1 + most / 16;
    } else {
        const uint32_t pairs = (uint32_t)a.batch * heads;
        most += most * (pairs < parts ? pairs : parts) / (2 * parts);
    }
    return most;
}

// a part from its sequence, the parts and slots before that, and its number
__device__ __forceinline__ void set_part(FewWhere& r, uint32_t steps, uint32_t parts, uint32_t k, uint32_t slot)
{
    const uint32_t head = k / parts, i = k - head * parts;
    r.head = (int)head;
    r.from = few_from(steps, parts, i);
    r.to = few_from(steps, parts, i + 1);
    r.parts = (int)parts;
    r.first_slot = (int)(slot + head * parts);
    r.slot = r.first_slot + (int)i;
}

// By every wave for itself, a lane for each of 64 sequences at a time: the sum
// of all steps, the length of a part, then the parts and slots up to the
// sequence that holds this workgroup's part; or from the table, where there is
// one.  Returns an empty part where there is none.
__device__ __forceinline__ FewWhere find_part(const AttendArgs& a, const AttendPlan& p)
{
    const int lane = threadIdx.x & 63;
    const uint32_t heads = a.kv.heads, id = blockIdx.x;
    FewWhere r{};
    if (a.batch > kScanBatch) {
        const FewTable t = few_table(a.workspace, p.groups, a.batch);
        const uint32_t b = __builtin_amdgcn_readfirstlane(t.sequence[id]);
        if (b >= (uint32_t)a.batch)
            return r;
        const uint32_t* before = t.before + (size_t)3 * b;
        const uint32_t steps = __builtin_amdgcn_readfirstlane(before[2]);
        r.b = (int)b;
        r.e = extent_of(a, (int)b);
        set_part(r, steps, few_parts(steps, __builtin_amdgcn_readfirstlane(*t.most)),
                 id - __builtin_amdgcn_readfirstlane(before[0]), __builtin_amdgcn_readfirstlane(before[1]));
        return r;
    }
    Extent e{};
    auto steps_of = [&](int b0) -> uint32_t {
        const int b = b0 + lane;
        e = extent_of(a, b < a.batch ? b : a.batch - 1);
        return b < a.batch ? (uint32_t)few_steps(a, e) : 0u;
    };
    uint32_t steps = 0, total = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
        steps = steps_of(b0);
        total += lane_value(wave_scan(steps), 63);
    }
    const uint32_t most = part_length(a, p, total, steps);
    uint32_t parts_before = 0, slots_before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
        if (a.batch > 64)
            steps = steps_of(b0);
        const uint32_t parts = few_parts(steps, most);
        const uint32_t mine = parts * heads, taken = parts > 1 ? mine : 0u;
        const uint32_t upto = parts_before + wave_scan(mine), slots = slots_before + wave_scan(taken);
        const uint64_t here = __builtin_amdgcn_ballot_w64(upto > id);
        if (here != 0) { // the first such lane's sequence
            const int at = __builtin_ctzll(here);
            r.e.q0 = (int64_t)lane_value((uint32_t)e.q0, at); // rows count in 31 bits here
            r.e.qn = (int)lane_value((uint32_t)e.qn, at);
            r.e.shift = (int)lane_value((uint32_t)e.shift, at);
            r.e.kn = (int)lane_value((uint32_t)e.kn, at);
            r.e.bad = lane_value(e.bad ? 1u : 0u, at) != 0;
            r.b = b0 + at;
            set_part(r, lane_value(steps, at), lane_value(parts, at), id - (lane_value(upto, at) - lane_value(mine, at)),
                     lane_value(slots, at) - lane_value(taken, at));
            return r;
        }
        parts_before = lane_value(upto, 63);
        slots_before = lane_value(slots, 63);
    }
    return r;
}

// writes the table (one workgroup of one wave: 64 sequences at a time)
__global__ __launch_bounds__(64) void attend_cut(const AttendArgs a, const AttendPlan p)
{
    const FewTable t = few_table(a.workspace, p.groups, a.batch);
    const uint32_t heads = a.kv.heads;
    const int lane = threadIdx.x;
    uint32_t total = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
        const int b = b0 + lane;
        const uint32_t steps = b < a.batch ? (uint32_t)few_steps(a, extent_of(a, b)) : 0u;
        if (b < a.batch)
            t.before[(size_t)3 * b + 2] = steps;
        total += lane_value(wave_scan(steps), 63);
    }
    const uint32_t most = part_length(a, p, total, 0u);
    if (lane == 0)
        *t.most = most;
    uint32_t parts_before = 0, slots_before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
        const int b = b0 + lane;
        const uint32_t steps = b < a.batch ? t.before[(size_t)3 * b + 2] : 0u; // this lane wrote it
        const uint32_t parts = few_parts(steps, most);
        const uint32_t mine = parts * heads, taken = parts > 1 ? mine : 0u;
        const uint32_t upto = parts_before + wave_scan(mine), slots = slots_before + wave_scan(taken);
        if (b < a.batch) {
            t.before[(size_t)3 * b] = upto - mine;
            t.before[(size_t)3 * b + 1] = slots - taken;
        }
        for (uint32_t id = upto - mine; id < upto; ++id)
            t.sequence[id] = (uint32_t)b;
        parts_before = lane_value(upto, 63);
        slots_before = lane_value(slots, 63);
    }
    for (uint32_t id = parts_before + lane; id < (uint32_t)p.groups; id += 64)
        t.sequence[id] = ~0u;
}

// QT: 16-row tiles of one wave, which share the expanded codes.  With QT = 2
// half the expansions are saved; at D = 256 the registers do not hold it.
template <bool MX, int D, int NQ, int NP, int QT>
__global__ __launch_bounds__(kThreads, few_waves_of(D, NQ, QT)) void attend_few(const AttendArgs a, const AttendPlan p)
{
    constexpr int B = MX ? 32 : 16;
    constexpr bool F32 = NP == (MX ? 3 : 2);
    constexpr int KW = D / 32;
    constexpr int N = D / 4;
    constexpr int RW = F32 ? D / 16 : D / 32; // 16-byte words of a row's quarter
    constexpr int R = 16 * QT;
    __shared__ Granule granule[kSegment / 16];
    __shared__ float merge_o[kWaves][R][D + 4]; // by wave
    __shared__ float2 merge_s[kWaves][R];

    FewWhere piece{};
    if (p.chunks == 1) { // one pair per workgroup
        uint32_t id = blockIdx.x;
        piece.head = (int)take_digit(id, a.kv.heads);
        piece.b = (int)id;
        piece.e = extent_of(a, piece.b);
        piece.to = few_steps(a, piece.e);
        piece.parts = 1;
    } else {
        piece = find_part(a, p);
    }
    if (piece.from == piece.to)
        return;
    const int b = piece.b, head = piece.head;
    const Extent e = piece.e;
    const int rows = e.qn * a.group;
    const int steps = few_steps(a, e);
    const int r0 = 0, r1 = rows;
    int lo, hi;
    tile_keys(a, e, r0, r1, lo, hi);
    const int k0 = lo + piece.from * kStepKeys;
    const int k1 = piece.to == steps ? hi : lo + piece.to * kStepKeys;
    // this wave's rows and its share of the keys
    const int parts = p.rows_per_tile / R; // 1, 2 or 4
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int n = lane & 15, g = lane >> 4;
    const int part = wave % parts, turn = wave / parts, turns = kWaves / parts;

    // the rows' quarters are under way while the keys are looked up and the
    // first codes loaded
    u32x4 raw[QT][RW];
    int row_lo[QT], row_hi[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int r = r0 + part * R + 16 * t + n;
        row_lo[t] = row_hi[t] = 0;
#pragma unroll
        for (int c = 0; c < RW; ++c)
            raw[t][c] = u32x4{0u, 0u, 0u, 0u};
        if (r < r1) {
            const int i = r / a.group, j = r - i * a.group;
            seen_by(a, e, i, row_lo[t], row_hi[t]);
            const int64_t at = (e.q0 + i) * a.q_row + (head * a.group + j) * a.q_head + g * N;
            const u32x4* x = reinterpret_cast<const u32x4*>(static_cast<const char*>(a.q) + at * (F32 ? 4 : 2));
#pragma unroll
            for (int c = 0; c < RW; ++c)
                raw[t][c] = x[c];
        }
    }
    const Lane at = lane_offsets<MX, D>(a, n, g);
    const int first = first_seen(a, e, r0);
    const int step = turns * kTileKeys;
    Tile<MX, D> now, next;
    int s0 = k0, s1 = k1 - k0 < kSegment ? k1 : k0 + kSegment;
    find_granules<kThreads>(a, b, head, s0, s1, first, granule);
    __syncthreads();
    int key = s0 + turn * kTileKeys;
    load_tile<MX, D, true>(a, granule, s0, key, first, s1, g, at, now);

    // the quarters, rotated, as parts
    u32x4 q[QT][NQ][KW];
    float factor[QT]; // of the row's logits, to log2 units; positive
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        float v[N];
#pragma unroll
        for (int c = 0; c < RW; ++c) {
            const u32x4 w = raw[t][c];
            if constexpr (F32) {
                v[4 * c + 0] = __uint_as_float(w.x); v[4 * c + 1] = __uint_as_float(w.y);
                v[4 * c + 2] = __uint_as_float(w.z); v[4 * c + 3] = __uint_as_float(w.w);
            } else {
                v[8 * c + 0] = bf16_lo(w.x); v[8 * c + 1] = bf16_hi(w.x);
                v[8 * c + 2] = bf16_lo(w.y); v[8 * c + 3] = bf16_hi(w.y);
                v[8 * c + 4] = bf16_lo(w.z); v[8 * c + 5] = bf16_hi(w.z);
                v[8 * c + 6] = bf16_lo(w.w); v[8 * c + 7] = bf16_hi(w.w);
            }
        }
        if (a.rotate)
            rotate_quarter<B, D>(v, g);
        const float S = MX ? 1.0f : *a.kv.global[0];
        const float sign = query_sign(a.scale, S);
#pragma unroll
        for (int j = 0; j < N; ++j)
            v[j] *= sign;
        int up = 0;
        if constexpr (!MX) {
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < N; ++j)
                top = __builtin_fmaxf(top, __builtin_fabsf(v[j]));
            top = column_max(top);
            // a power of two to [2^14, 2^15); zero and non-finite rows stay
            up = (top > 0.0f && top < __builtin_huge_valf()) ? 141 - (int)(__float_as_uint(top) >> 23) : 0;
#pragma unroll
            for (int j = 0; j < N; ++j)
                v[j] = __builtin_ldexpf(v[j], up);
        }
        factor[t] = logit_factor(a.scale, S, up);
#pragma unroll
        for (int s = 0; s < NQ; ++s)
#pragma unroll
            for (int c = 0; c < KW; ++c) {
                q[t][s][c].x = take_part<MX>(v[8 * c + 0], v[8 * c + 1]);
                q[t][s][c].y = take_part<MX>(v[8 * c + 2], v[8 * c + 3]);
                q[t][s][c].z = take_part<MX>(v[8 * c + 4], v[8 * c + 5]);
                q[t][s][c].w = take_part<MX>(v[8 * c + 6], v[8 * c + 7]);
            }
    }

    f32x4 o[QT][D / 16];
    float m[QT], l[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
            o[t][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        m[t] = -__builtin_huge_valf();
        l[t] = 0.0f;
    }
    // keys that every row of the workgroup sees need no mask
    int all_lo, all_hi, unused;
    seen_by(a, e, (r1 - 1) / a.group, all_lo, unused);
    seen_by(a, e, r0 / a.group, unused, all_hi);
    all_hi = all_hi < k1 ? all_hi : k1;

    for (;;) {
    for (; key < s1; key += step) {
        load_tile<MX, D, false>(a, granule, s0, key + step, 0, s1, g, at, next); // past the end: nothing
        f32x4 s[QT][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int t = 0; t < QT; ++t)
                s[t][h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < KW; ++c) {
                const u32x4 k = k_operand<MX, D>(now, h, c);
#pragma unroll
                for (int t = 0; t < QT; ++t)
#pragma unroll
                    for (int x = NQ - 1; x >= 0; --x) // small parts first
                        s[t][h] = mfma16<MX>(k, q[t][x][c], s[t][h]);
            }
        }
        u32x4 pr[QT][NP];
        const bool whole = key >= all_lo && key + kTileKeys <= all_hi;
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            if (!whole) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = key + 16 * h + 4 * i + g;
                        s[t][h][i] = (k >= row_lo[t] && k < row_hi[t]) ? s[t][h][i] : -__builtin_huge_valf();
                    }
            }
            float top = -__builtin_huge_valf();
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    top = __builtin_fmaxf(top, s[t][h][i]);
            top *= factor[t];
            if (__builtin_amdgcn_ballot_w64(top > m[t] + kLazy) != 0) {
                const float raised = __builtin_fmaxf(m[t], column_max(top));
                const float f = m[t] == raised ? 1.0f : __builtin_amdgcn_exp2f(m[t] - raised);
                m[t] = raised;
                l[t] *= f;
#pragma unroll
                for (int c = 0; c < D / 16; ++c)
                    o[t][c] *= f;
            }
            const float base = m[t] == -__builtin_huge_valf() ? 0.0f : m[t] - kUp;
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][j >> 2][j & 3], factor[t], -base));
                l[t] += x[j];
            }
#pragma unroll
            for (int y = 0; y < NP; ++y) {
                pr[t][y].x = take_part<MX>(x[0], x[1]);
                pr[t][y].y = take_part<MX>(x[2], x[3]);
                pr[t][y].z = take_part<MX>(x[4], x[5]);
                pr[t][y].w = take_part<MX>(x[6], x[7]);
            }
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            u32x4 even, odd;
            v_operands<MX, D>(now, c, even, odd);
#pragma unroll
            for (int t = 0; t < QT; ++t)
#pragma unroll
                for (int y = NP - 1; y >= 0; --y) {
                    o[t][2 * c] = mfma16<MX>(even, pr[t][y], o[t][2 * c]);
                    o[t][2 * c + 1] = mfma16<MX>(odd, pr[t][y], o[t][2 * c + 1]);
                }
        }
        now = next;
    }
    if (s1 >= k1)
        break;
    s0 = s1; // the places of the next keys
    s1 = k1 - s0 < kSegment ? k1 : s0 + kSegment;
    __syncthreads();
    find_granules<kThreads>(a, b, head, s0, s1, 0, granule);
    __syncthreads();
    key = s0 + turn * kTileKeys;
    load_tile<MX, D, false>(a, granule, s0, key, 0, s1, g, at, now);
    }

    // join the waves that share rows, through LDS: D/8 lanes take a row
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const float sum = column_sum(l[t]);
        if (r0 + part * R + 16 * t + n < r1) {
            if (g == 0)
                merge_s[wave][16 * t + n] = float2{m[t], sum};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < D / 16; c += 4)
                    *reinterpret_cast<f32x4*>(&merge_o[wave][16 * t + n][g * N + i * (D / 16) + c]) =
                        f32x4{o[t][c][i], o[t][c + 1][i], o[t][c + 2][i], o[t][c + 3][i]};
        }
    }
    __syncthreads();
    const int j = threadIdx.x % (D / 8);
    for (int x = threadIdx.x / (D / 8); x < r1 - r0; x += kThreads / (D / 8)) {
        const int from = x / R, at_row = x % R; // the row's part, and its place there
        float top = -__builtin_huge_valf(), sum = 0.0f;
        for (int t = 0; t < turns; ++t)
            top = __builtin_fmaxf(top, merge_s[from + t * parts][at_row].x);
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            y[k] = 0.0f;
        for (int t = 0; t < turns; ++t) {
            const float2 st = merge_s[from + t * parts][at_row];
            const float f = st.x == top ? 1.0f : __builtin_amdgcn_exp2f(st.x - top);
            const f32x4* src = reinterpret_cast<const f32x4*>(&merge_o[from + t * parts][at_row][8 * j]);
            const f32x4 u = src[0], w = src[1];
            sum += st.y * f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                y[k] += u[k] * f;
                y[4 + k] += w[k] * f;
            }
        }
        if (e.bad)
            sum = __builtin_nanf("");
        top -= kUp; // the sums' unit
        const int r = r0 + x;
        if (piece.parts == 1) {
            finish_row<MX, D, F32>(a, e, head, r, j, y, top, sum);
        } else {
            const Partial w = partials_of(a, p);
            const int64_t to = (int64_t)piece.slot * p.rows_per_tile + r;
            if (j == 0)
                w.stat[to] = float2{top, sum};
            f32x4* out = reinterpret_cast<f32x4*>(w.o + to * D + 8 * j);
            out[0] = f32x4{y[0], y[1], y[2], y[3]};
            out[1] = f32x4{y[4], y[5], y[6], y[7]};
        }
    }
    if (p.chunks != 1 && piece.from == 0 && threadIdx.x == 0)
        partials_of(a, p).pairs[(int64_t)b * a.kv.heads + head] = int2{piece.first_slot, piece.parts};
}

// ---- many queries: workgroups of 32 rows a wave, keys through LDS ---------------------
//
// S^T = K Q^T and O^T = V^T P^T by 32x32x16 products.  A workgroup's waves
// each own 32 query rows (queries of one sequence and KV head, all heads of
// the group) and share 64 keys at a time, which they expand together from
// 4 bits to the 16-bit operands in LDS: each code is expanded once for all
// rows of the workgroup.  Two buffers: while one is multiplied, the other is
// filled from codes loaded a step earlier; one barrier per step.
// Places of an operand (lane = n + 32 h, n a row or column, h a half):
//   - K: row m of a 32-key tile is key m with bits 2 and 3 exchanged, so that
//     accumulator 8 x + j of half h is key 16 x + 8 h + j: eight consecutive
//     keys, one operand of the second product.  Half h holds values
//     h D/2 + 8 c ... of a row at step c, so a lane's part of a query row is
//     contiguous.
//   - V^T: row 32 t + i is value (D/32) i + t, so that the thread that expands
//     D/32 adjacent values writes rows 32 apart (no bank conflict), and a lane
//     ends with D/8 contiguous values of the result for each a of
//     value = (D/32) (4 h + 8 a) + ...
//   - 16-byte units of a row are exchanged by an XOR with the row, so that 16
//     lanes that read or write one unit of 16 rows meet all 64 banks.
//
// Bound by issue: in a step the products take 37% of the cycles and the vector
// ALU (exponentials, maxima, parts, expansion) 47%, on two waves per SIMD that
// meet at the step's barrier.  8192 queries after themselves, 32 heads of
// 128 over 8 KV heads, NVFP4, 562-600 us: 915-980 TFLOP/s of the pairs seen, where
// a library's large f16 product reaches 1175.  Two times 509 queries after 16384
// keys, MXFP4, 32 heads: 356 us with the joining (MXFP4's probabilities are two
// products each).  Every part of the queries stays in registers, which costs the
// forms of more than one: the same 8192 queries rotated take 702 us (MXFP4 1131,
// 30 registers spilled) and in binary32 1436 (1694), one wave per SIMD; with 256
// values a head there is always one, 1879 us (2185), and more parts spill 28 or
// 94 registers, 2839 (4639).  Measured and left: waves 4-7 half a step behind 0-3 (a third
// buffer of V and the logits kept over the barrier: 594 -> 630 us, and 361 ->
// 413 with spilled registers), wave priorities around the products (no change),
// workgroups of four waves (119 -> 109 us for 96 rows after 8192 keys, but 37 -> 45
// for 128 rows of two short sequences), the causal end's tiles cut along the
// keys (77 -> 107).

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kManyKeys = 64;      // keys of one step
constexpr int kManySegment = 4096; // keys whose places are looked up at once

template <bool MX>
__device__ __forceinline__ f32x16 mfma32(u32x4 x, u32x4 y, f32x16 c)
{
    if constexpr (MX)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b16x8, x), __builtin_bit_cast(b16x8, y), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
}

// the 16-byte unit `u` of K's row m, of V^T's row d
template <int D>
__device__ __forceinline__ int k_unit(int m, int u)
{
    return D == 64 ? m * 8 + (u ^ ((m >> 1) & 7)) : m * (D / 8) + (u ^ (m & 15));
}
__device__ __forceinline__ int v_unit(int d, int u) { return d * 8 + (u ^ ((d >> 1) & 7)); }

// codes and scales of one wave's 16 keys of a step, as loaded
template <int D>
struct StageK {
    uint32_t w[D / 32], s;
    uint32_t lost; // all ones where the keys' page does not exist (uniform)
};
template <int D>
struct StageV {
    uint32_t w[8], s[8]; // by key; D/64 code bytes of D/32 values
};

struct ManyBuffers {
    __amdgpu_buffer_rsrc_t codes, scales;
    bool lost;
};

// resources over the rows of 16 keys from `key` that lie before `end`; none
// where all of them lie below `first`
template <int B, int D, bool EDGE>
__device__ __forceinline__ ManyBuffers many_buffers(const AttendArgs& a, const Granule* g, int side, int key, int first,
                                                    int end)
{
    int rows = end - key;
    if (EDGE && key + 16 <= first)
        rows = 0;
    rows = __builtin_amdgcn_readfirstlane(rows < 0 ? 0 : (rows > 16 ? 16 : rows));
    const int64_t co = rows > 0 ? uniform64(g->codes) : 0, so = rows > 0 ? uniform64(g->scales) : 0;
    const bool lost = co < 0;
    if (lost)
        rows = 0; // read nothing
    const int cb = rows > 0 ? (rows - 1) * (int)a.kv.c_token + D / 2 : 0;
    const int sb = rows > 0 ? (rows - 1) * (int)a.kv.s_token + D / B : 0;
    return ManyBuffers{buffer_of(a.kv.codes[side] + co, cb), buffer_of(a.kv.scales[side] + so, sb), lost};
}

template <bool MX, int D, bool EDGE>
__device__ __forceinline__ void stage_k(const AttendArgs& a, const Granule* g, int key, int first, int end, int lane,
                                        StageK<D>& t)
{
    constexpr int B = MX ? 32 : 16;
    constexpr int QS = D / 4 >= B ? D / 4 / B : 1;
    const ManyBuffers m = many_buffers<B, D, EDGE>(a, g, 0, key, first, end);
    const int row = lane >> 2, quarter = lane & 3;
    const int o = row * (int)a.kv.c_token + quarter * (D / 8);
    const int os = row * (int)a.kv.s_token + (quarter * (D / 4)) / B;
    if constexpr (D == 64) {
        const u32x2 w = __builtin_amdgcn_raw_buffer_load_b64(m.codes, o, 0, 0);
        t.w[0] = w.x;
        t.w[1] = w.y;
    } else {
#pragma unroll
        for (int j = 0; j < D / 128; ++j) {
            const u32x4 w = __builtin_amdgcn_raw_buffer_load_b128(m.codes, o + 16 * j, 0, 0);
            t.w[4 * j + 0] = w.x;
            t.w[4 * j + 1] = w.y;
            t.w[4 * j + 2] = w.z;
            t.w[4 * j + 3] = w.w;
        }
    }
    if constexpr (QS == 1)
        t.s = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(m.scales, os, 0, 0);
    else if constexpr (QS == 2)
        t.s = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(m.scales, os, 0, 0);
    else
        t.s = __builtin_amdgcn_raw_buffer_load_b32(m.scales, os, 0, 0);
    t.lost = m.lost ? kNanScales : 0u;
}

template <bool MX, int D, bool EDGE>
__device__ __forceinline__ void stage_v(const AttendArgs& a, const Granule* g, int key, int first, int end, int lane,
                                        StageV<D>& t)
{
    constexpr int B = MX ? 32 : 16;
    const ManyBuffers m = many_buffers<B, D, EDGE>(a, g, 1, key, first, end);
    const int unit = lane >> 5, i = lane & 31;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int row = 8 * unit + j;
        const int o = row * (int)a.kv.c_token + i * (D / 64);
        if constexpr (D == 64)
            t.w[j] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(m.codes, o, 0, 0);
        else if constexpr (D == 128)
            t.w[j] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(m.codes, o, 0, 0);
        else
            t.w[j] = __builtin_amdgcn_raw_buffer_load_b32(m.codes, o, 0, 0);
        const int os = seen_offset<EDGE>(row * (int)a.kv.s_token + (i * (D / 32)) / B, key + row, first);
        t.s[j] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(m.scales, os, 0, 0);
    }
}

// expand granule `w` (0..3) of a step into K's buffer
template <bool MX, int D>
__device__ __forceinline__ void expand_k(const StageK<D>& t, int w, int lane, u32x4* buf)
{
    constexpr int B = MX ? 32 : 16;
    const int key = 16 * w + (lane >> 2), quarter = lane & 3;
    const int m = (key & ~12) | ((key & 4) << 1) | ((key & 8) >> 1);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        const int s = (8 * c) / B;
        const uint32_t ks = t.s | t.lost; // lost: K, and the logits that see it, are NaN
        u32x4 x;
        if constexpr (MX) {
            x = expand_bf16(t.w[c], e8m0_step((ks >> (8 * s)) & 0xFFu));
        } else {
            const f16x2 two = s < 2 ? e4m3_pair<false>(ks) : e4m3_pair<true>(ks);
            const _Float16 one = two[s & 1];
            x = expand_f16(t.w[c], f16x2{one, one});
        }
        buf[k_unit<D>(m, quarter * (D / 32) + c)] = x;
    }
}

template <bool MX, int D>
__device__ __forceinline__ void expand_v(const StageV<D>& t, int w, int lane, u32x4* buf)
{
    const int unit = 2 * w + (lane >> 5), i = lane & 31;
#pragma unroll
    for (int m = 0; m < D / 64; ++m) { // values 2m and 2m + 1 of the thread's
        uint32_t e[4], o[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const uint32_t x = t.w[2 * p] >> (8 * m), y = t.w[2 * p + 1] >> (8 * m);
            if constexpr (MX) {
                const uint32_t cx = fp4_pair_bf16<0>(x, e8m0_step(t.s[2 * p]));
                const uint32_t cy = fp4_pair_bf16<0>(y, e8m0_step(t.s[2 * p + 1]));
                e[p] = __builtin_amdgcn_perm(cy, cx, 0x05040100u);
                o[p] = __builtin_amdgcn_perm(cy, cx, 0x07060302u);
            } else {
                const f16x2 s = e4m3_pair<false>(t.s[2 * p] | (t.s[2 * p + 1] << 8));
                const uint32_t lo = (x & 0x0Fu) | ((y << 4) & 0xF0u);
                const uint32_t hi = ((x >> 4) & 0x0Fu) | (y & 0xF0u);
                e[p] = __builtin_bit_cast(uint32_t, fp4_pair_f16<0>(lo) * s);
                o[p] = __builtin_bit_cast(uint32_t, fp4_pair_f16<0>(hi) * s);
            }
        }
        buf[v_unit(32 * (2 * m) + i, unit)] = u32x4{e[0], e[1], e[2], e[3]};
        buf[v_unit(32 * (2 * m + 1) + i, unit)] = u32x4{o[0], o[1], o[2], o[3]};
    }
}

// Orthonormal Hadamard of blocks of B among the first N values of a lane, the
// block's other half in lane ^ 32 where N < B
template <int B, int N>
__device__ __forceinline__ void rotate_half(float* v, int h)
{
    constexpr int W = N < B ? N : B;
#pragma unroll
    for (int s = 1; s < W; s *= 2)
#pragma unroll
        for (int i = 0; i < N; i += 2 * s)
#pragma unroll
            for (int j = i; j < i + s; ++j) {
                const float p = v[j], q = v[j + s];
                v[j] = p + q;
                v[j + s] = p - q;
            }
    if constexpr (N < B) {
        const float sign = h ? -1.0f : 1.0f;
#pragma unroll
        for (int j = 0; j < N; ++j)
            v[j] = __builtin_fmaf(sign, v[j], __shfl_xor(v[j], 32, 64));
    }
}

template <bool MX, int D, int NQ, int NP, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void attend_many(const AttendArgs a, const AttendPlan p)
{
    constexpr int B = MX ? 32 : 16;
    constexpr int C = D / 16;  // steps of the first product
    constexpr int T = D / 32;  // row tiles of V^T
    constexpr int KU = kManyKeys * D / 8; // 16-byte units of a buffer
    constexpr bool F32 = NP == (MX ? 3 : 2);
    constexpr int RW = F32 ? D / 8 : D / 16; // 16-byte words of half a row
    __shared__ u32x4 kbuf[2][KU];
    __shared__ u32x4 vbuf[2][KU];
    __shared__ Granule granule[kManySegment / 16];

    // blocks: (sequence, KV head) fastest, so that with a multiple of eight of
    // them the row tiles that read one head's keys share an XCD's L2; then the
    // chunk; the row tiles with the most keys (the last ones) first
    uint32_t id = blockIdx.x;
    const int head = (int)take_digit(id, a.kv.heads);
    const int b = (int)take_digit(id, a.batch);
    const int chunk = (int)take_digit(id, p.chunks);
    const int tile = p.tiles - 1 - (int)id;

    const Extent e = extent_of(a, b);
    const int rows = e.qn * a.group;
    const int r0 = tile * p.rows_per_tile;
    if (r0 >= rows)
        return;
    const int r1 = r0 + p.rows_per_tile < rows ? r0 + p.rows_per_tile : rows;
    int lo, hi;
    tile_keys(a, e, r0, r1, lo, hi);
    if (chunk >= chunks_of(p, lo, hi))
        return;
    const int k0 = lo + chunk * p.chunk;
    const int k1 = hi - k0 < p.chunk ? hi : k0 + p.chunk;

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int n = lane & 31, h = lane >> 5;
    const int w0 = r0 + wave * 32;            // the wave's first row
    const int r = w0 + n;
    const bool live = r < r1;
    int row_lo = 0, row_hi = 0;

    // the row's half is under way while the keys are looked up and the first
    // codes loaded
    u32x4 raw[RW];
#pragma unroll
    for (int c = 0; c < RW; ++c)
        raw[c] = u32x4{0u, 0u, 0u, 0u};
    if (live) {
        const int i = r / a.group, j = r - i * a.group;
        seen_by(a, e, i, row_lo, row_hi);
        const int64_t at = (e.q0 + i) * a.q_row + (head * a.group + j) * a.q_head + h * (D / 2);
        const u32x4* x = reinterpret_cast<const u32x4*>(static_cast<const char*>(a.q) + at * (F32 ? 4 : 2));
#pragma unroll
        for (int c = 0; c < RW; ++c)
            raw[c] = x[c];
    }

    // waves 0-3 expand K and, of eight waves, 4-7 V
    const bool does_k = wave < 4, does_v = WAVES == 4 || wave >= 4;
    const int w = wave & 3;
    StageK<D> sk;
    StageV<D> sv;
    int s0 = k0, s1 = k1 - k0 < kManySegment ? k1 : k0 + kManySegment;
    const int first = first_seen(a, e, r0);
    auto load = [&](int key, auto edge) {
        const int mine = key + 16 * w;
        const Granule* g = granule + (mine < s1 ? (mine - s0) / 16 : 0);
        if (does_k)
            stage_k<MX, D, edge.value>(a, g, mine, first, s1, lane, sk);
        if (does_v)
            stage_v<MX, D, edge.value>(a, g, mine, first, s1, lane, sv);
    };
    constexpr std::true_type at_first{};
    constexpr std::false_type later{};
    auto expand = [&](int to) {
        if (does_k)
            expand_k<MX, D>(sk, w, lane, kbuf[to]);
        if (does_v)
            expand_v<MX, D>(sv, w, lane, vbuf[to]);
    };
    find_granules<64 * WAVES>(a, b, head, s0, s1, first, granule);
    __syncthreads();
    load(s0, at_first);

    u32x4 q[NQ][C];
    float factor; // of the row's logits, to log2 units; positive
    {
        float v[D / 2];
#pragma unroll
        for (int c = 0; c < RW; ++c) {
            const u32x4 x = raw[c];
            if constexpr (F32) {
                v[4 * c + 0] = __uint_as_float(x.x); v[4 * c + 1] = __uint_as_float(x.y);
                v[4 * c + 2] = __uint_as_float(x.z); v[4 * c + 3] = __uint_as_float(x.w);
            } else {
                v[8 * c + 0] = bf16_lo(x.x); v[8 * c + 1] = bf16_hi(x.x);
                v[8 * c + 2] = bf16_lo(x.y); v[8 * c + 3] = bf16_hi(x.y);
                v[8 * c + 4] = bf16_lo(x.z); v[8 * c + 5] = bf16_hi(x.z);
                v[8 * c + 6] = bf16_lo(x.w); v[8 * c + 7] = bf16_hi(x.w);
            }
        }
        const float S = MX ? 1.0f : *a.kv.global[0];
        const float sign = query_sign(a.scale, S);
        const float turn = a.rotate ? (B == 16 ? 0.25f : __uint_as_float(0x3E3504F3u)) * sign : sign;
        if (a.rotate)
            rotate_half<B, D / 2>(v, h);
#pragma unroll
        for (int j = 0; j < D / 2; ++j)
            v[j] *= turn;
        int up = 0;
        if constexpr (!MX) {
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < D / 2; ++j)
                top = __builtin_fmaxf(top, __builtin_fabsf(v[j]));
            top = __builtin_fmaxf(top, __shfl_xor(top, 32, 64));
            up = (top > 0.0f && top < __builtin_huge_valf()) ? 141 - (int)(__float_as_uint(top) >> 23) : 0;
#pragma unroll
            for (int j = 0; j < D / 2; ++j)
                v[j] = __builtin_ldexpf(v[j], up);
        }
        factor = logit_factor(a.scale, S, up);
#pragma unroll
        for (int s = 0; s < NQ; ++s)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                q[s][c].x = take_part<MX>(v[8 * c + 0], v[8 * c + 1]);
                q[s][c].y = take_part<MX>(v[8 * c + 2], v[8 * c + 3]);
                q[s][c].z = take_part<MX>(v[8 * c + 4], v[8 * c + 5]);
                q[s][c].w = take_part<MX>(v[8 * c + 6], v[8 * c + 7]);
            }
    }
    // keys that any row, and that every row, of the wave sees (uniform)
    int wave_lo = 0, wave_hi = 0, all_lo = 0x7FFFFFFF, all_hi = 0;
    if (w0 < r1) {
        const int last = (w0 + 32 < r1 ? w0 + 32 : r1) - 1;
        seen_by(a, e, w0 / a.group, wave_lo, all_hi);
        seen_by(a, e, last / a.group, all_lo, wave_hi);
    }

    f32x16 o[T];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int j = 0; j < 16; ++j)
            o[t][j] = 0.0f;
    float m = -__builtin_huge_valf(), l = 0.0f;

    while (k0 < k1) {
        expand(0);
        if (s0 + kManyKeys < s1)
            load(s0 + kManyKeys, later);
        __syncthreads();
        int at = 0;
        for (int key = s0; key < s1; key += kManyKeys, at ^= 1) {
            if (key + kManyKeys < s1) {
                expand(at ^ 1);
                if (key + 2 * kManyKeys < s1)
                    load(key + 2 * kManyKeys, later);
            }
            if (key < wave_hi && key + kManyKeys > wave_lo) {
                f32x16 s[2];
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        s[x][j] = 0.0f;
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const u32x4 k = kbuf[at][k_unit<D>(32 * x + n, h * C + c)];
#pragma unroll
                        for (int t = NQ - 1; t >= 0; --t)
                            s[x] = mfma32<MX>(k, q[t][c], s[x]);
                    }
                if (!(key >= all_lo && key + kManyKeys <= all_hi)) {
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const int k = key + 32 * x + 16 * (j >> 3) + 8 * h + (j & 7);
                            s[x][j] = (k >= row_lo && k < row_hi) ? s[x][j] : -__builtin_huge_valf();
                        }
                }
                float top = s[0][0];
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        top = __builtin_fmaxf(top, s[x][j]);
                top *= factor;
                if (__builtin_amdgcn_ballot_w64(top > m + kLazy) != 0) {
                    const float raised = __builtin_fmaxf(m, __builtin_fmaxf(top, __shfl_xor(top, 32, 64)));
                    const float f = m == raised ? 1.0f : __builtin_amdgcn_exp2f(m - raised);
                    m = raised;
                    l *= f;
#pragma unroll
                    for (int t = 0; t < T; ++t)
                        o[t] *= f;
                }
                const float base = m == -__builtin_huge_valf() ? 0.0f : m - kUp;
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        s[x][j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x][j], factor, -base));
                        l += s[x][j];
                    }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    u32x4 pr[NP];
                    float y[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        y[j] = s[u >> 1][8 * (u & 1) + j];
#pragma unroll
                    for (int t = 0; t < NP; ++t) {
                        pr[t].x = take_part<MX>(y[0], y[1]);
                        pr[t].y = take_part<MX>(y[2], y[3]);
                        pr[t].z = take_part<MX>(y[4], y[5]);
                        pr[t].w = take_part<MX>(y[6], y[7]);
                    }
#pragma unroll
                    for (int d = 0; d < T; ++d) {
                        const u32x4 v = vbuf[at][v_unit(32 * d + n, 2 * u + h)];
#pragma unroll
                        for (int t = NP - 1; t >= 0; --t)
                            o[d] = mfma32<MX>(v, pr[t], o[d]);
                    }
                }
            }
            __syncthreads();
        }
        if (s1 >= k1)
            break;
        s0 = s1; // the places of the next keys
        s1 = k1 - s0 < kManySegment ? k1 : s0 + kManySegment;
        find_granules<64 * WAVES>(a, b, head, s0, s1, 0, granule);
        __syncthreads();
        load(s0, later);
    }
    l += __shfl_xor(l, 32, 64);
    if (e.bad)
        l = __builtin_nanf("");
    m -= kUp;

    // the lane's values: D/8 contiguous ones for each a, in order
    if (p.chunks == 1) {
        const OutFactor f = out_factor(MX ? 1.0f : *a.kv.global[1], l);
        const float turn = f.by * (a.rotate ? (B == 16 ? 0.25f : __uint_as_float(0x3E3504F3u)) : 1.0f);
        const int i = live ? r / a.group : 0, j = r - i * a.group;
        const int64_t row = e.q0 + i;
        const int qh = head * a.group + j;
        if (live && a.lse && h == 0)
            a.lse[row * a.q_heads + qh] = l == 0.0f ? -__builtin_huge_valf() : (m + __builtin_log2f(l)) * kLn2;
        float y[4][4 * T];
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int t = 0; t < T; ++t)
                    y[x][T * k + t] = o[t][4 * x + k] * turn;
        if (a.rotate) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
                rotate_half<B, 4 * T>(y[x], h);
            if constexpr (8 * T < B) { // D = 64 in blocks of 32: two of them make one
#pragma unroll
                for (int x = 0; x < 4; x += 2)
#pragma unroll
                    for (int k = 0; k < 4 * T; ++k) {
                        const float u = y[x][k], v = y[x + 1][k];
                        y[x][k] = u + v;
                        y[x + 1][k] = u - v;
                    }
            }
        }
        if (!live)
            return;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int at = T * (4 * h + 8 * x);
            if constexpr (!MX) {
#pragma unroll
                for (int k = 0; k < 4 * T; ++k)
                    y[x][k] *= f.rest;
            }
            if (a.bf16) {
                uint16_t* to = static_cast<uint16_t*>(a.out) + row * a.o_row + qh * a.o_head + at;
#pragma unroll
                for (int k = 0; k < T / 2; ++k)
                    reinterpret_cast<u32x4*>(to)[k] =
                        u32x4{bf16_pair(y[x][8 * k], y[x][8 * k + 1]), bf16_pair(y[x][8 * k + 2], y[x][8 * k + 3]),
                              bf16_pair(y[x][8 * k + 4], y[x][8 * k + 5]), bf16_pair(y[x][8 * k + 6], y[x][8 * k + 7])};
            } else {
                float* to = static_cast<float*>(a.out) + row * a.o_row + qh * a.o_head + at;
#pragma unroll
                for (int k = 0; k < T; ++k)
                    reinterpret_cast<f32x4*>(to)[k] = f32x4{y[x][4 * k], y[x][4 * k + 1], y[x][4 * k + 2], y[x][4 * k + 3]};
            }
        }
    } else if (live) {
        const Partial out = partials_of(a, p);
        const int64_t at_row = (((int64_t)b * a.kv.heads + head) * a.max_q * a.group + r) * p.chunks + chunk;
        if (h == 0)
            out.stat[at_row] = float2{m, l};
        float* to = out.o + at_row * D;
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int t = 0; t < T; t += 2)
                    *reinterpret_cast<float2*>(to + T * (4 * h + 8 * x + k) + t) =
                        float2{o[t][4 * x + k], o[t + 1][4 * x + k]};
    }
}

// ---- joining the partial results of a row ------------------------------------------
//
// D/4 lanes hold four values each of a row; T groups of such lanes take every
// T-th of its partial results.  One workgroup has as many rows as fit.  Reads
// every partial result once: bound by that traffic where there are many rows
// (12 us for 32576 rows of 128 values of two partial results: 42 MB, 3.5 TB/s),
// by the latency of a few dependent loads where there are few (5 us).
template <bool MX, int D, int T>
__global__ __launch_bounds__(kThreads) void attend_join(const AttendArgs a, const AttendPlan p, const uint32_t all_rows)
{
    constexpr int B = MX ? 32 : 16;
    constexpr int L = D / 4;
    constexpr int R = kThreads / (L * T); // rows of a workgroup
    __shared__ f32x4 sum[T > 1 ? kThreads : 1];
    __shared__ float2 red[T > 1 ? kThreads / L : 1];
    const int j = threadIdx.x % L, turn = threadIdx.x / L % T, at = threadIdx.x / (L * T);
    const uint32_t id = blockIdx.x * R + at;
    uint32_t rest = id;
    const int r = (int)take_digit(rest, a.max_q * a.group);
    const int head = (int)take_digit(rest, a.kv.heads);
    const int b = (int)rest;
    // a row's lanes leave together; with T > 1 so does the workgroup (R = 1)
    static_assert(T == 1 || R == 1, "rows of one workgroup");
    if (id >= all_rows)
        return;
    const Extent e = extent_of(a, b);
    const int rows = e.qn * a.group;
    if (r >= rows)
        return;
    const Partial w = partials_of(a, p);
    // places of the row's partial results: base + c * stride
    int chunks;
    int64_t base, stride;
    if (p.many) {
        const int r0 = r - r % p.rows_per_tile;
        int lo, hi;
        tile_keys(a, e, r0, r0 + p.rows_per_tile < rows ? r0 + p.rows_per_tile : rows, lo, hi);
        chunks = chunks_of(p, lo, hi);
        base = (int64_t)id * p.chunks;
        stride = 1;
    } else {
        const int2 pair = w.pairs[id / (uint32_t)(a.max_q * a.group)];
        chunks = pair.y;
        if (chunks == 1)
            return; // done by the one workgroup that had it all
        base = (int64_t)pair.x * p.rows_per_tile + r;
        stride = p.rows_per_tile;
    }
    // a running maximum over this lane's share (a NaN is in the sums, never in
    // a maximum)
    f32x4 o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float l = 0.0f, m = -__builtin_huge_valf();
    for (int c = turn; c < chunks; c += T) {
        const float2 s = w.stat[base + c * stride];
        const f32x4 t = *reinterpret_cast<const f32x4*>(w.o + (base + c * stride) * D + 4 * j);
        const float raised = __builtin_fmaxf(m, s.x);
        const float f0 = m == raised ? 1.0f : __builtin_amdgcn_exp2f(m - raised);
        const float f1 = s.x == raised ? 1.0f : __builtin_amdgcn_exp2f(s.x - raised);
        m = raised;
        l = l * f0 + s.y * f1;
        o = o * f0 + t * f1;
    }
    if constexpr (T > 1) {
        sum[threadIdx.x] = o;
        if (j == 0)
            red[turn] = float2{m, l};
        __syncthreads();
        if (threadIdx.x >= L)
            return;
#pragma unroll
        for (int t = 0; t < T; ++t)
            m = __builtin_fmaxf(m, red[t].x);
        o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        l = 0.0f;
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const float2 s = red[t];
            const float f = s.x == m ? 1.0f : __builtin_amdgcn_exp2f(s.x - m);
            l += s.y * f;
            o += sum[t * L + j] * f;
        }
    }
    const OutFactor f = out_factor(MX ? 1.0f : *a.kv.global[1], l);
    o *= f.by;
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
    if constexpr (!MX)
        o *= f.rest;
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

template <bool MX, int D, int QT>
void launch_few(const AttendArgs& a, const AttendPlan& p, dim3 grid)
{
    if (!a.bf16)
        attend_few<MX, D, MX ? 3 : 2, MX ? 3 : 2, QT><<<grid, kThreads, 0, a.stream>>>(a, p);
    else if (a.rotate)
        attend_few<MX, D, MX ? 3 : 2, MX ? 2 : 1, QT><<<grid, kThreads, 0, a.stream>>>(a, p);
    else
        attend_few<MX, D, 1, MX ? 2 : 1, QT><<<grid, kThreads, 0, a.stream>>>(a, p);
}

template <bool MX, int D>
hipError_t launch_parts(const AttendArgs& a, const AttendPlan& p)
{
    const dim3 grid((uint32_t)p.groups);
    if (!p.many && p.chunks > 1 && a.batch > kScanBatch)
        attend_cut<<<1, 64, 0, a.stream>>>(a, p);
    if (p.many) {
        constexpr int WAVES = D == 256 ? 4 : 8;
        if (!a.bf16)
            attend_many<MX, D, MX ? 3 : 2, MX ? 3 : 2, 4><<<grid, 256, 0, a.stream>>>(a, p);
        else if (a.rotate)
            attend_many<MX, D, MX ? 3 : 2, MX ? 2 : 1, WAVES><<<grid, 64 * WAVES, 0, a.stream>>>(a, p);
        else
            attend_many<MX, D, 1, MX ? 2 : 1, WAVES><<<grid, 64 * WAVES, 0, a.stream>>>(a, p);
    } else if (p.rows_per_tile == 16 || D == 256) {
        launch_few<MX, D, 1>(a, p, grid);
    } else {
        launch_few<MX, D, D == 256 ? 1 : 2>(a, p, grid);
    }
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || p.chunks == 1)
        return err;
    // a workgroup per row where there may be many partial results of each
    const uint32_t rows = (uint32_t)((int64_t)a.batch * a.kv.heads * a.max_q * a.group);
    constexpr int per = kThreads / (D / 4);
    if (p.many && p.chunks <= 4 * per)
        attend_join<MX, D, 1><<<dim3((rows + per - 1) / per), kThreads, 0, a.stream>>>(a, p, rows);
    else
        attend_join<MX, D, per><<<dim3(rows), kThreads, 0, a.stream>>>(a, p, rows);
    return hipGetLastError();
}

template <bool MX>
hipError_t launch_dim(const AttendArgs& a, const AttendPlan& p)
{
    switch (a.kv.head_dim) {
    case 64: return launch_parts<MX, 64>(a, p);
    case 128: return launch_parts<MX, 128>(a, p);
    default: return launch_parts<MX, 256>(a, p);
    }
}

} // namespace

AttendPlan plan_attend(const AttendArgs& a) { return plan_of(a); }

hipError_t launch_attend(const AttendArgs& a, const AttendPlan& p)
{
    return a.kv.mx ? launch_dim<true>(a, p) : launch_dim<false>(a, p);
}

} // namespace fp4q
