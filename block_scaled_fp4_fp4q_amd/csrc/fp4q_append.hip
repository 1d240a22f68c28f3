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
// the hardware's estimate (off by at most 2^-22 or so) leaves 2^-52
__device__ __forceinline__ float inverse_root(double d)
{
    const double y = __builtin_amdgcn_rsq(d);
    const double e = __builtin_fma(-(d * y), y, 1.0);
    return (float)__builtin_fma(y * e, __builtin_fma(e, 0.375, 0.5), y);
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
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < E; ++i)
            sum = __builtin_fma((double)v[i], (double)v[i], sum);
        for (int h = 1; h < lanes; h *= 2)
            sum += __shfl_xor(sum, h, 64);
        r = inverse_root(sum / (double)a.kv.head_dim + (double)a.eps);
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

// the table's row of a token's position; null where it is out of range
__device__ __forceinline__ const float* angles_of(const KvAppendArgs& a, int64_t token, bool& good)
{
    good = true;
    if (a.turned == 0)
        return nullptr;
    const int64_t p = a.positions[token];
    good = p >= 0 && p < a.rope_rows;
    return good ? a.rope + p * a.rope_row : nullptr;
}

// E values of a row of q from e0 on, to q_out (a bad position: NaN)
template <int E, bool BF16>
__device__ __forceinline__ void store_q(const KvAppendArgs& a, uint32_t token, uint32_t head, int e0, const float* v)
{
    char* to = static_cast<char*>(a.q_out) + (token * a.out_row + head * a.out_head + e0) * (BF16 ? 2 : 4);
#pragma unroll
    for (int g = 0; g < E / 8; ++g) {
        const float* y = v + 8 * g;
        if constexpr (BF16) {
            reinterpret_cast<u32x4*>(to)[g] = u32x4{bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]), bf16_pair(y[4], y[5]), bf16_pair(y[6], y[7])};
        } else {
            reinterpret_cast<f32x4*>(to)[2 * g] = f32x4{y[0], y[1], y[2], y[3]};
            reinterpret_cast<f32x4*>(to)[2 * g + 1] = f32x4{y[4], y[5], y[6], y[7]};
        }
    }
}

// Which rows a workgroup has: the first ones K's, then V's, then those of q (the rows
// to be quantized take longer).  Items are lanes: `last` + 1 of them a row.
struct Share {
    int side;        // 0 K, 1 V, 2 q
    uint32_t first, step, items;
    uint32_t heads;
};

__device__ __forceinline__ Share share_of(const KvAppendArgs& a, const AppendPlan& p)
{
    const uint32_t b = blockIdx.x;
    Share s;
    s.side = b < p.kv_groups ? 0 : (b < 2 * p.kv_groups ? 1 : 2);
    const uint32_t groups = s.side == 2 ? p.q_groups : p.kv_groups;
    s.first = (b - (s.side == 0 ? 0u : (s.side == 1 ? p.kv_groups : 2 * p.kv_groups))) * kThreads + threadIdx.x;
    s.step = groups * kThreads;
    s.items = s.side == 2 ? p.q_items : p.kv_items;
    s.heads = s.side == 2 ? (uint32_t)a.q_heads : (uint32_t)a.kv.heads;
    return s;
}

// RULE AbsMax: eight values a lane, the scale's maximum and the transform's wide stages
// across the lanes of a block; the searching rules: a block a lane.
template <bool MX, int RULE, bool BF16, bool ROT>
__global__ __launch_bounds__(kThreads) void kv_append(const KvAppendArgs a, const AppendPlan p)
{
    constexpr int B = MX ? 32 : 16;
    constexpr int E = RULE == kRuleAbsMax ? 8 : B;
    __shared__ Pattern tab[RULE == kRuleSweep && !MX ? 128 : 1];
    const Share mine = share_of(a, p);
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
    for (uint32_t item = mine.first; item < mine.items; item += mine.step) {
        const uint32_t part = item & (uint32_t)(lanes - 1), row = item >> p.lane_shift;
        const uint32_t token = row / mine.heads, head = row - token * mine.heads;
        bool good;
        const float* angles = angles_of(a, token, good);
        float v[E];
        if (mine.side == 2) {
            if (good) {
                const char* x = static_cast<const char*>(a.q) + (token * a.q_row + head * a.q_head) * (BF16 ? 2 : 4);
                turned_part<E, BF16>(a, x, (int)part * E, lanes, a.q_weight, angles, v);
            } else {
#pragma unroll
                for (int i = 0; i < E; ++i)
                    v[i] = __builtin_nanf("");
            }
            store_q<E, BF16>(a, token, head, (int)part * E, v);
            continue;
        }
        const int64_t slot = a.slots[token];
        if (!good || slot < 0 || slot >= most)
            continue; // with all lanes of its row
        const char* x = static_cast<const char*>(a.x[mine.side]) +
                        (token * a.x_token[mine.side] + head * a.x_head[mine.side]) * (BF16 ? 2 : 4);
        if (mine.side == 0)
            turned_part<E, BF16>(a, x, (int)part * E, lanes, a.k_weight, angles, v);
        else
            load_part<E, BF16>(x, (int)part * E, v);
        int64_t page, off;
        slot_place(a.kv, slot, most, page, off);
        uint8_t* codes = a.kv.codes[mine.side] + page * a.kv.c_page + head * a.kv.c_head + off * a.kv.c_token;
        uint8_t* scales = a.kv.scales[mine.side] + page * a.kv.s_page + head * a.kv.s_head + off * a.kv.s_token;
        if constexpr (RULE == kRuleAbsMax) {
            if constexpr (ROT)
                rotate_lanes<B, E>(v, part);
            float top = block_absmax<E>(v);
#pragma unroll
            for (int h = 1; h < B / E; h *= 2)
                top = __builtin_fmaxf(top, __shfl_xor(top, h, 64));
            uint32_t sb;
            const float r = absmax_scale<MX>(top, S, S6, sb);
            uint32_t w = fresh_word(v[0]); // every byte of it is written
            w = fp4_pack2<0>(w, v[0] * r, v[1] * r);
            w = fp4_pack2<1>(w, v[2] * r, v[3] * r);
            w = fp4_pack2<2>(w, v[4] * r, v[5] * r);
            w = fp4_pack2<3>(w, v[6] * r, v[7] * r);
            reinterpret_cast<uint32_t*>(codes)[part] = w;
            if (part % (B / E) == 0)
                scales[part / (B / E)] = (uint8_t)sb;
        } else {
            if constexpr (ROT)
                fwht<B>(v);
            store_block<MX, RULE>(v, block_absmax<B>(v), S, S6, tab, a.lo, a.hi, codes, scales, part);
        }
    }
}

template <bool MX, int RULE, bool BF16>
void launch_rule(const KvAppendArgs& a, const AppendPlan& p)
{
    const dim3 grid(2 * p.kv_groups + p.q_groups);
    if (a.rotate)
        kv_append<MX, RULE, BF16, true><<<grid, kThreads, 0, a.stream>>>(a, p);
    else
        kv_append<MX, RULE, BF16, false><<<grid, kThreads, 0, a.stream>>>(a, p);
}

template <bool BF16>
void launch_type(const KvAppendArgs& a, const AppendPlan& p)
{
    if (a.kv.mx) {
        if (a.rule == kRuleAbsMax)
            launch_rule<true, kRuleAbsMax, BF16>(a, p);
        else
            launch_rule<true, kRuleSweep, BF16>(a, p);
    } else if (a.rule == kRuleAbsMax) {
        launch_rule<false, kRuleAbsMax, BF16>(a, p);
    } else if (a.rule == kRuleSweep) {
        launch_rule<false, kRuleSweep, BF16>(a, p);
    } else {
        launch_rule<false, kRuleFourSix, BF16>(a, p);
    }
}

constexpr uint32_t kMostGroups = 1u << 20; // of each share; the kernel strides over the rest

uint32_t groups_for(uint32_t items)
{
    const uint32_t g = (items + kThreads - 1) / kThreads;
    return g < kMostGroups ? g : kMostGroups;
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
        p.kv_items = (uint32_t)(a.tokens * a.kv.heads * lanes);
        p.q_items = (uint32_t)(a.tokens * a.q_heads * lanes);
        p.kv_groups = groups_for(p.kv_items);
        p.q_groups = groups_for(p.q_items);
        if (a.bf16)
            launch_type<true>(a, p);
        else
            launch_type<false>(a, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

} // namespace fp4q
