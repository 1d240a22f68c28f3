// fp4q_append.hip -- new tokens on their way into the 4-bit KV cache: the norm of
// each head of q and k, the rotary positions, and the cache's write, in one launch.
//
//   r   = 1 / sqrt(mean_i x_i^2 + eps)         in binary64, rounded to binary32
//   y_i = fl(fl(x_i r) w_i)
//   (a, b) -> (fl(fl(a c) - fl(b s)), fl(fl(b c) + fl(a s)))    for each turned pair
//
// with c and s of the token's position from a table.  q leaves rounded to its own type;
// k, after this, and v are quantized as fp4q_kv_write quantizes them, from the
// binary32 values.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "fp4q_device.h"
#include "fp4q_kv_device.h"
#include "fp4q_kv_launch.h"

namespace fp4q {

namespace {

constexpr int kThreads = 256;

// 1 / sqrt(d), rounded to binary32, for d > 0 in binary64: one step of third order on
// the hardware's estimate (off by at most 2^-22 or so) leaves 2^-52; infinity gives 0
__device__ __forceinline__ float inverse_root(double d)
{
    const double y = __builtin_amdgcn_rsq(d);
    const double e = __builtin_fma(-(d * y), y, 1.0);
    const double r = __builtin_fma(y * e, __builtin_fma(e, 0.375, 0.5), y);
    return d == __builtin_huge_val() ? 0.0f : (float)r;
}

// the E values from value e0 on of a row, widened
template <int E, bool BF16>
__device__ __forceinline__ void load_part(const char* row, int e0, float* v)
{
    load_block<E, BF16, false>(row + e0 * (BF16 ? 2 : 4), 0, v);
}

// eight floats, 16-byte aligned
__device__ __forceinline__ void load8(const float* p, float* v)
{
    const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
    }
}

// x and the value that the lane of a row of 16 lanes holds which CTRL names
template <int CTRL>
__device__ __forceinline__ double plus_moved(double x)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xF, 0xF, true);
    const uint32_t hi = __builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, true);
    return x + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// the sum over `lanes` neighbouring lanes (a power of two up to 32), in all of them
__device__ __forceinline__ double lanes_sum(double x, int lanes)
{
    if (lanes > 1)
        x = plus_moved<0xB1>(x); // of lane ^ 1
    if (lanes > 2)
        x = plus_moved<0x4E>(x); // lane ^ 2
    if (lanes > 4)
        x = plus_moved<0x141>(x); // the eight lanes backwards: of the other four
    if (lanes > 8)
        x = plus_moved<0x140>(x); // the sixteen backwards: of the other eight
    return lanes > 16 ? x + __shfl_xor(x, 16, 64) : x;
}

// what the values of a row are multiplied by, its `lanes` lanes having E of them each
template <int E>
__device__ __forceinline__ float norm_of(const float* v, int lanes, int dim, float eps)
{
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < E; ++i)
        sum = __builtin_fma((double)v[i], (double)v[i], sum);
    sum = lanes_sum(sum, lanes);
    // head_dim is a power of two: its reciprocal is exact
    return inverse_root(__builtin_fma(sum, dim == 64 ? 0x1p-6 : (dim == 128 ? 0x1p-7 : 0x1p-8), (double)eps));
}

// The E values from e0 on of one row of q or k, normed and turned; `lanes` (a power
// of two) neighbouring lanes hold the row and are here together.  A lane reads the
// partners of its values itself, eight neighbours at a time (half the turned values
// is a multiple of eight).
template <int E, bool BF16>
__device__ __forceinline__ void turned_part(const KvAppendArgs& a, const char* row, int e0, int lanes, const float* weight,
                                            const float* angles, float* v)
{
    load_part<E, BF16>(row, e0, v);
    float r = 1.0f;
    if (weight) {
        r = norm_of<E>(v, lanes, a.kv.head_dim, a.eps);
#pragma unroll
        for (int g = 0; g < E / 8; ++g) {
            float w[8];
            load8(weight + e0 + 8 * g, w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[8 * g + i] = (v[8 * g + i] * r) * w[i];
        }
    }
    const int half = a.turned / 2;
#pragma unroll
    for (int g = 0; g < E / 8; ++g) {
        const int e = e0 + 8 * g;
        if (e >= a.turned)
            break;
        float* y = v + 8 * g;
        if (a.interleaved) {
            const f32x4 c = *reinterpret_cast<const f32x4*>(angles + e / 2);
            const f32x4 s = *reinterpret_cast<const f32x4*>(angles + half + e / 2);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p = y[2 * i], q = y[2 * i + 1];
                y[2 * i] = p * c[i] - q * s[i];
                y[2 * i + 1] = q * c[i] + p * s[i];
            }
            continue;
        }
        const bool first = e < half;
        const int at = first ? e : e - half, other = first ? e + half : e - half;
        float c[8], s[8], z[8];
        load8(angles + at, c);
        load8(angles + half + at, s);
        load_part<8, BF16>(row, other, z);
        if (weight) {
            float w[8];
            load8(weight + other, w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                z[i] = (z[i] * r) * w[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float own = y[i] * c[i], far = z[i] * s[i];
            y[i] = first ? own - far : own + far;
        }
    }
}

// the table's row of a token's position
struct Place {
    const float* angles;
    bool good; // the position has a row, or none is needed
};

__device__ __forceinline__ Place place_of(const KvAppendArgs& a, int64_t token)
{
    if (a.turned == 0)
        return Place{nullptr, true};
    const int64_t p = a.positions[token];
    const bool good = p >= 0 && p < a.rope_rows;
    return Place{good ? a.rope + p * a.rope_row : nullptr, good};
}

// eight values of q
template <bool BF16>
__device__ __forceinline__ void store_q(char* to, const float* y)
{
    if constexpr (BF16) {
        *reinterpret_cast<u32x4*>(to) = u32x4{bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]), bf16_pair(y[4], y[5]), bf16_pair(y[6], y[7])};
    } else {
        reinterpret_cast<f32x4*>(to)[0] = f32x4{y[0], y[1], y[2], y[3]};
        reinterpret_cast<f32x4*>(to)[1] = f32x4{y[4], y[5], y[6], y[7]};
    }
}

// Which rows a workgroup has: the first workgroups K's, then V's, then those of q (the rows
// to be quantized take longer).
struct Share {
    int side;               // 0 K, 1 V, 2 q
    uint32_t group, groups; // its number among that side's, and how many these are
};

__device__ __forceinline__ Share share_of(const AppendPlan& p)
{
    const uint32_t b = blockIdx.x;
    if (b < p.kv_groups)
        return Share{0, b, p.kv_groups};
    if (b < 2 * p.kv_groups)
        return Share{1, b - p.kv_groups, p.kv_groups};
    return Share{2, b - 2 * p.kv_groups, p.q_groups};
}

// The searching rules: a block a lane, whose 16 or 32 values stay in its registers.  Bound by
// the vector ALU where many scales are tried (fp4q_kv.hip has the figures of the pick), by
// latency for a decode step (64 tokens, 32 + 8 + 8 heads of 128 values, NVFP4, 11 scales,
// rotated: 9.6 us).  8192 of those tokens, 92 us (AbsMax 54): q, whose rows are not searched, takes
// a block a lane here too, which the other kernel has shown to be the slower layout.
template <bool MX, int RULE, bool BF16, bool ROT>
__global__ __launch_bounds__(kThreads) void kv_append_search(const KvAppendArgs a, const AppendPlan p)
{
    static_assert(RULE == kRuleSweep || (RULE == kRuleFourSix && !MX), "the searching rules");
    constexpr int B = MX ? 32 : 16;
    __shared__ Pattern tab[RULE == kRuleSweep && !MX ? 128 : 1];
    const Share mine = share_of(p);
    const uint32_t heads = mine.side == 2 ? (uint32_t)a.q_heads : (uint32_t)a.kv.heads;
    const float S = MX || mine.side == 2 ? 1.0f : *a.kv.global[mine.side];
    if constexpr (RULE == kRuleSweep && !MX) {
        if (mine.side != 2) {
            if (threadIdx.x < 128) {
                const float s = e4m3_value(threadIdx.x < 0x7E ? threadIdx.x : 0x7Eu);
                const float D = s * S;
                tab[threadIdx.x] = Pattern{1.0f / D, s * s, D};
            }
            __syncthreads();
        }
    }
    const float S6 = 6.0f * S;
    const int64_t most = a.kv.num_pages * a.kv.page_size;
    const int lanes = 1 << p.lane_shift;
    const uint32_t items = (uint32_t)a.tokens * heads << p.lane_shift;
    for (uint32_t item = mine.group * kThreads + threadIdx.x; item < items; item += mine.groups * kThreads) {
        const uint32_t part = item & (uint32_t)(lanes - 1), row = item >> p.lane_shift;
        const uint32_t token = row / heads, head = row - token * heads;
        const Place at = place_of(a, token);
        float v[B];
        if (mine.side == 2) {
            const char* x = static_cast<const char*>(a.q) + (token * a.q_row + head * a.q_head) * (BF16 ? 2 : 4);
            if (at.good) {
                turned_part<B, BF16>(a, x, (int)part * B, lanes, a.q_weight, at.angles, v);
            } else {
#pragma unroll
                for (int i = 0; i < B; ++i)
                    v[i] = __builtin_nanf("");
            }
            char* to = static_cast<char*>(a.q_out) + (token * a.out_row + head * a.out_head + part * B) * (BF16 ? 2 : 4);
#pragma unroll
            for (int g = 0; g < B / 8; ++g)
                store_q<BF16>(to + 8 * g * (BF16 ? 2 : 4), v + 8 * g);
            continue;
        }
        const int64_t slot = a.slots[token];
        if (!at.good || slot < 0 || slot >= most)
            continue; // with all lanes of its row
        const char* x = static_cast<const char*>(a.x[mine.side]) +
                        (token * a.x_token[mine.side] + head * a.x_head[mine.side]) * (BF16 ? 2 : 4);
        if (mine.side == 0)
            turned_part<B, BF16>(a, x, (int)part * B, lanes, a.k_weight, at.angles, v);
        else
            load_part<B, BF16>(x, (int)part * B, v);
        int64_t page, off;
        slot_place(a.kv, slot, most, page, off);
        uint8_t* codes = a.kv.codes[mine.side] + page * a.kv.c_page + head * a.kv.c_head + off * a.kv.c_token;
        uint8_t* scales = a.kv.scales[mine.side] + page * a.kv.s_page + head * a.kv.s_head + off * a.kv.s_token;
        if constexpr (ROT)
            fwht<B>(v);
        store_block<MX, RULE>(v, block_absmax<B>(v), S, S6, tab, a.lo, a.hi, codes, scales, part);
    }
}

// AbsMax: eight values a lane, the scale's maximum and the transform's wide stages across
// the lanes of a block.  A workgroup has 256 / (head_dim / 8) rows at a time, of one token
// where it has that many heads, else of several; a lane keeps its part of a row, so that the
// cosines and sines of a token and the norm's weights are read once for all of its heads.
//   A block a lane, as the searching rules have it, left each lane's loads 32 bytes apart and
// read partners twice; partners come by shuffles here and sums of squares by moves within 16
// lanes.  Bound by the vector ALU (about 200 instructions for a wave's four rows, the norm's in
// binary64) and by waits: 8192 tokens, 32 heads of q and 8 of k and v, 128 values, bf16,
// NVFP4, normed and turned whole: 52 us, 177 MB, 3.4 TB/s.  A sixth wave a SIMD spills.
template <bool MX, bool BF16, bool ROT>
__global__ __launch_bounds__(kThreads) void kv_append_absmax(const KvAppendArgs a, const AppendPlan p)
{
    constexpr int B = MX ? 32 : 16;
    constexpr int E = 8, SIZE = BF16 ? 2 : 4;
    const Share mine = share_of(p);
    const bool q = mine.side == 2;
    const float S = MX || q ? 1.0f : *a.kv.global[mine.side];
    const float S6 = 6.0f * S;
    const int64_t most = a.kv.num_pages * a.kv.page_size;
    const int lanes = 1 << p.lane_shift, per = kThreads >> p.lane_shift; // rows at a time
    const int heads = q ? a.q_heads : a.kv.heads;
    const int tokens = heads < per ? per / heads : 1; // of these
    const int part = threadIdx.x & (lanes - 1), row = threadIdx.x >> p.lane_shift;
    const int sub = heads < per ? row / heads : 0, head0 = row - sub * heads;
    if (sub >= tokens)
        return;
    const int e0 = part * E, half = a.turned / 2;
    const bool turn = mine.side != 1 && e0 < a.turned;
    const float* weight = q ? a.q_weight : (mine.side == 0 ? a.k_weight : nullptr);
    // the lane that has the partners of this lane's values, and its angles in a row of the table
    const bool first = e0 < half;
    const bool apart = mine.side != 1 && a.turned != 0 && !a.interleaved; // partners in other lanes
    const int partner = (threadIdx.x & 63) + (turn ? (first ? half : -half) / E : 0);
    const int angle = a.interleaved ? e0 / 2 : (first ? e0 : e0 - half);
    float w[E];
    if (weight)
        load8(weight + e0, w);
    const char* from = static_cast<const char*>(q ? a.q : a.x[mine.side]);
    const int64_t x_token = q ? a.q_row : a.x_token[mine.side], x_head = q ? a.q_head : a.x_head[mine.side];
    const int step = heads < per ? heads : per;
    const int64_t stride = (int64_t)mine.groups * tokens;
    // a token's position and slot are read one token ahead, a row's values one row
    struct Token {
        int64_t position, slot;
    };
    auto read_token = [&](int64_t t) {
        Token r{0, 0};
        if (t < a.tokens) {
            r.position = a.turned != 0 ? a.positions[t] : 0;
            r.slot = q ? 0 : a.slots[t];
        }
        return r;
    };
    struct Raw {
        u32x4 w[BF16 ? 1 : 2];
    };
    auto read_row = [&](const char* x) {
        Raw r;
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i)
            r.w[i] = reinterpret_cast<const u32x4*>(x)[i];
        return r;
    };
    auto widen = [](const u32x4* r, float* v) {
        if constexpr (BF16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = bf16_lo(r[0][i]);
                v[2 * i + 1] = bf16_hi(r[0][i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = __uint_as_float(r[i / 4][i % 4]);
        }
    };
    int64_t token = (int64_t)mine.group * tokens + sub;
    Token next = read_token(token);
    for (; token < a.tokens; token += stride) {
        const Token now = next;
        const char* x = from + (token * x_token + head0 * x_head + e0) * SIZE;
        char* to = q ? static_cast<char*>(a.q_out) + (token * a.out_row + head0 * a.out_head + e0) * SIZE : nullptr;
        Raw raw = read_row(x);
        const bool good = a.turned == 0 || (now.position >= 0 && now.position < a.rope_rows);
        int64_t page = 0, off = 0;
        const bool written = q || (good && now.slot >= 0 && now.slot < most);
        float c[E], s[E];
        if (turn && good) {
            const float* angles = a.rope + now.position * a.rope_row;
            if (a.interleaved) { // four pairs
                const f32x4 u = *reinterpret_cast<const f32x4*>(angles + angle);
                const f32x4 v = *reinterpret_cast<const f32x4*>(angles + half + angle);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    c[2 * i] = c[2 * i + 1] = u[i];
                    s[2 * i] = s[2 * i + 1] = v[i];
                }
            } else {
                load8(angles + angle, c);
                load8(angles + half + angle, s);
                // a c - b s of the first of a pair, b c + a s of the second
#pragma unroll
                for (int i = 0; i < E; ++i)
                    s[i] = first ? -s[i] : s[i];
            }
        }
        next = read_token(token + stride);
        if (!written)
            continue; // with all lanes of its rows
        if (!q)
            slot_place(a.kv, now.slot, most, page, off);
        for (int head = head0; head < heads; head += step) {
            float v[E];
            widen(raw.w, v);
            x += step * x_head * SIZE;
            if (head + step < heads)
                raw = read_row(x);
            if (weight) {
                const float r = norm_of<E>(v, lanes, a.kv.head_dim, a.eps);
#pragma unroll
                for (int i = 0; i < E; ++i)
                    v[i] = (v[i] * r) * w[i];
            }
            if (apart) { // a row's lanes are here together
                float z[E];
#pragma unroll
                for (int i = 0; i < E; ++i)
                    z[i] = __shfl(v[i], partner, 64);
                if (turn) {
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        const float own = v[i] * c[i], far = z[i] * s[i];
                        v[i] = own + far;
                    }
                }
            } else if (turn) {
#pragma unroll
                for (int i = 0; i < E; i += 2) {
                    const float u = v[i], y = v[i + 1];
                    v[i] = u * c[i] - y * s[i];
                    v[i + 1] = y * c[i] + u * s[i];
                }
            }
            if (q) {
                if (!good) {
#pragma unroll
                    for (int i = 0; i < E; ++i)
                        v[i] = __builtin_nanf("");
                }
                store_q<BF16>(to, v);
                to += step * a.out_head * SIZE;
                continue;
            }
            uint8_t* codes = a.kv.codes[mine.side] + page * a.kv.c_page + head * a.kv.c_head + off * a.kv.c_token;
            uint8_t* scales = a.kv.scales[mine.side] + page * a.kv.s_page + head * a.kv.s_head + off * a.kv.s_token;
            if constexpr (ROT)
                rotate_lanes<B, E>(v, (uint32_t)part);
            float top = block_absmax<E>(v);
#pragma unroll
            for (int h = 1; h < B / E; h *= 2)
                top = __builtin_fmaxf(top, __shfl_xor(top, h, 64));
            uint32_t sb;
            const float r = absmax_scale<MX>(top, S, S6, sb);
            uint32_t word = fresh_word(v[0]); // every byte of it is written
            word = fp4_pack2<0>(word, v[0] * r, v[1] * r);
            word = fp4_pack2<1>(word, v[2] * r, v[3] * r);
            word = fp4_pack2<2>(word, v[4] * r, v[5] * r);
            word = fp4_pack2<3>(word, v[6] * r, v[7] * r);
            reinterpret_cast<uint32_t*>(codes)[part] = word;
            if (part % (B / E) == 0)
                scales[part / (B / E)] = (uint8_t)sb;
        }
    }
}

template <bool MX, bool BF16>
void launch_rule(const KvAppendArgs& a, const AppendPlan& p)
{
    const dim3 grid(2 * p.kv_groups + p.q_groups);
    if (a.rule == kRuleAbsMax) {
        if (a.rotate)
            kv_append_absmax<MX, BF16, true><<<grid, kThreads, 0, a.stream>>>(a, p);
        else
            kv_append_absmax<MX, BF16, false><<<grid, kThreads, 0, a.stream>>>(a, p);
    } else if (a.rule == kRuleSweep) {
        if (a.rotate)
            kv_append_search<MX, kRuleSweep, BF16, true><<<grid, kThreads, 0, a.stream>>>(a, p);
        else
            kv_append_search<MX, kRuleSweep, BF16, false><<<grid, kThreads, 0, a.stream>>>(a, p);
    } else if constexpr (!MX) {
        if (a.rotate)
            kv_append_search<MX, kRuleFourSix, BF16, true><<<grid, kThreads, 0, a.stream>>>(a, p);
        else
            kv_append_search<MX, kRuleFourSix, BF16, false><<<grid, kThreads, 0, a.stream>>>(a, p);
    }
}

// workgroups of a side, at most: AbsMax's go on to the next tokens with their weights at
// hand, the searching rules' stride over what a grid does not cover
constexpr int64_t kAbsMaxGroups = 2048, kSearchGroups = 1 << 20;

uint32_t groups_for(int64_t tokens, int heads, int lanes, bool search)
{
    if (heads == 0)
        return 0;
    const int per = kThreads / lanes;
    int64_t g;
    if (search) {
        g = (tokens * heads + per - 1) / per;
        return (uint32_t)(g < kSearchGroups ? g : kSearchGroups);
    }
    const int together = heads < per ? per / heads : 1;
    g = (tokens + together - 1) / together;
    return (uint32_t)(g < kAbsMaxGroups ? g : kAbsMaxGroups);
}

} // namespace

hipError_t launch_kv_append(const KvAppendArgs& all)
{
    KvAppendArgs a = all;
    const int block = a.kv.mx ? 32 : 16;
    const int lanes = a.kv.head_dim / (a.rule == kRuleAbsMax ? 8 : block);
    const int heads = a.q_heads > a.kv.heads ? a.q_heads : a.kv.heads;
    AppendPlan p{};
    while ((1 << p.lane_shift) < lanes)
        ++p.lane_shift;
    // item numbers, and a grid's stride past the last of them, stay in 32 bits
    const int64_t most = ((int64_t)1 << 31) / ((int64_t)heads * lanes);
    if (most == 0)
        return hipErrorInvalidValue;
    for (int64_t t0 = 0; t0 < all.tokens; t0 += most) {
        const int size = a.bf16 ? 2 : 4;
        a.tokens = all.tokens - t0 < most ? all.tokens - t0 : most;
        a.slots = all.slots + t0;
        a.positions = all.positions ? all.positions + t0 : nullptr;
        for (int side = 0; side < 2; ++side)
            a.x[side] = static_cast<const char*>(all.x[side]) + t0 * all.x_token[side] * size;
        if (a.q_heads != 0) {
            a.q = static_cast<const char*>(all.q) + t0 * all.q_row * size;
            a.q_out = static_cast<char*>(all.q_out) + t0 * all.out_row * size;
        }
        p.kv_groups = groups_for(a.tokens, a.kv.heads, lanes, a.rule != kRuleAbsMax);
        p.q_groups = groups_for(a.tokens, a.q_heads, lanes, a.rule != kRuleAbsMax);
        if (a.kv.mx)
            a.bf16 ? launch_rule<true, true>(a, p) : launch_rule<true, false>(a, p);
        else
            a.bf16 ? launch_rule<false, true>(a, p) : launch_rule<false, false>(a, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

} // namespace fp4q
