// fp4q_kv_device.h -- device helpers of the kernels that write rows into the
// 4-bit KV cache and read them back (fp4q_kv.hip, fp4q_append.hip).
#pragma once

#include "fp4q_device.h"
#include "fp4q_kv_launch.h"

namespace fp4q {

enum { kRuleAbsMax = 0, kRuleSweep = 1, kRuleFourSix = 2 };
constexpr int kWinLo = -3, kWinHi = 7; // the window that is unrolled

// page and place of a valid slot; 32-bit arithmetic where all slots fit (a
// 64-bit division costs as much as the rest of a block's decode)
__device__ __forceinline__ void slot_place(const KvView& kv, int64_t slot, int64_t slots, int64_t& page, int64_t& off)
{
    if (slots <= (int64_t)0xFFFFFFFF) {
        const uint32_t p = (uint32_t)slot / (uint32_t)kv.page_size;
        page = p;
        off = (uint32_t)slot - p * (uint32_t)kv.page_size;
    } else {
        page = slot / kv.page_size;
        off = slot - page * kv.page_size;
    }
}

// the constants of one E4M3 pattern under the cache's global scale
struct alignas(16) Pattern {
    float r;  // fl32(1/D)
    float s2; // s*s, exact
    float D;  // fl32(s S)
};

__device__ __forceinline__ int pattern_clamp(int c) { return c < 1 ? 1 : (c > 0x7E ? 0x7E : c); }

// 2^k as binary32, exact for k in [-149, 127]
__device__ __forceinline__ float exp2i(int k)
{
    return k >= -126 ? __uint_as_float((uint32_t)(k + 127) << 23) : __uint_as_float(1u << (k + 149));
}

// OCP E8M0 exponent of a block maximum, clamped to [-127, 127]
__device__ __forceinline__ int block_exponent(float a)
{
    if (a == 0.0f)
        return -127;
    const uint32_t u = __float_as_uint(a);
    const int e = (u >= 0x00800000u ? (int)(u >> 23) - 127 : -149 + (31 - __clz((int)u))) - 2;
    return e < -127 ? -127 : (e > 127 ? 127 : e);
}

// binary64 error of the encoding with step D and reciprocal r, summed in
// element order: the quantity that every rule compares
template <int B>
__device__ __forceinline__ double exact_error(const float* v, float D, float r)
{
    double E = 0.0;
#pragma unroll
    for (int i = 0; i < B; ++i) {
        const float a = __builtin_fabsf(v[i]);
        const float xh = e2m1_q(a * r) * D;
        const double d = (double)a - (double)xh;
        E = E + d * d;
    }
    return E;
}

// binary32 estimate of the same error in units of the step squared, the codes
// from the hardware conversion (which are the method's own)
__device__ __forceinline__ float step_error16(const float* v, float r)
{
    float F = 0.0f;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        float y[8], q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] = v[8 * g + j] * r;
        uint32_t c = fresh_word(y[0]);
        // conversions as one group: mixing them with binary32 work costs more
        __builtin_amdgcn_sched_barrier(0);
        c = fp4_pack2<0>(c, y[0], y[1]);
        c = fp4_pack2<1>(c, y[2], y[3]);
        c = fp4_pack2<2>(c, y[4], y[5]);
        c = fp4_pack2<3>(c, y[6], y[7]);
        fp4_unpack2<0>(c, q[0], q[1]);
        fp4_unpack2<1>(c, q[2], q[3]);
        fp4_unpack2<2>(c, q[4], q[5]);
        fp4_unpack2<3>(c, q[6], q[7]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float d = y[j] - q[j];
            F = __builtin_fmaf(d, d, F);
        }
    }
    return F;
}

// ScaleSweep's pick for one block of maximum a > 0: the pattern of least
// binary64 error in the window around the AbsMax pattern sb, the smaller on a
// tie.  For the window [-3, 7] every candidate is first estimated in binary32;
// the estimates lie within a rigorous bound of the binary64 error over S^2
// (a few units of rounding per element, summed by Cauchy-Schwarz: A bounds
// |x| / S and 6 s over the window, 16 elements), so only the candidates whose
// interval reaches below the least upper end can win.  Those, usually one to
// three, are evaluated in binary64 in a loop that the lanes of a wave share.
// Any other window evaluates all of its patterns in binary64.
__device__ __forceinline__ int sweep_pick(const float* v, float a, float S, int sb, const Pattern* tab,
                                          int lo, int hi)
{
    constexpr float u = 0x1p-24f;
    if (lo == kWinLo && hi == kWinHi) {
        constexpr int K = kWinHi - kWinLo + 1;
        float low[K];
        float least = __builtin_huge_valf(); // least upper end
        const float A = __builtin_fmaxf(a / S * (1.0f + 4.0f * u),
                                        6.0f * e4m3_value((uint32_t)pattern_clamp(sb + kWinHi))) *
                        (1.0f + 4.0f * u);
        const float tail = 64.0f * 16.0f * u * u * A * A;
        const bool finite = 6.0f * tab[pattern_clamp(sb + kWinHi)].D < __builtin_huge_valf() &&
                            A < __builtin_huge_valf();
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const Pattern t = tab[pattern_clamp(sb + kWinLo + j)];
            const float E = step_error16(v, t.r) * t.s2;
            const float T = 16.0f * u * A * (4.0f * __builtin_amdgcn_sqrtf(E) * 1.0001f) + 32.0f * u * E + tail;
            low[j] = E - T;
            least = __builtin_fminf(least, E + T);
        }
        uint32_t open = 0;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            // an offset past an end repeats the end pattern, which this window
            // (0 in it, sb a pattern) always holds as itself too
            const int c = sb + kWinLo + j;
            const bool in = finite ? !(low[j] > least) : true;
            open |= (c == pattern_clamp(c) && in) ? 1u << j : 0u;
        }
        if (a == 0.0f) // a zero block has no scale to choose
            open = 1u << -kWinLo;
        if (__builtin_amdgcn_ballot_w64((open & (open - 1u)) != 0u) == 0)
            return sb + kWinLo + __builtin_ctz(open);
        int cb = 0x7F;
        double best = __builtin_huge_val();
        while (__builtin_amdgcn_ballot_w64(open != 0u) != 0) {
            if (open != 0u) {
                const int j = __builtin_ctz(open);
                open &= open - 1u;
                const int c = pattern_clamp(sb + kWinLo + j);
                const double E = exact_error<16>(v, tab[c].D, tab[c].r);
                if (cb == 0x7F || E < best || (E == best && c < cb)) {
                    best = E;
                    cb = c;
                }
            }
        }
        return cb;
    }
    int cb = 0x7F, prev = 0;
    double best = 0.0;
    for (int k = lo; k <= hi; ++k) {
        const int c = pattern_clamp(sb + k);
        if (c == prev)
            continue;
        prev = c;
        const double E = exact_error<16>(v, tab[c].D, tab[c].r);
        if (cb == 0x7F || E < best) {
            best = E;
            cb = c;
        }
    }
    return cb;
}

// A block of maximum `top` by one of the searching rules: its scale chosen, its
// codes and its scale byte stored as the row's block b.  Every active lane of a
// wave takes part.
template <bool MX, int RULE>
__device__ __forceinline__ void store_block(const float* v, float top, float S, float S6, const Pattern* tab, int lo, int hi,
                                            uint8_t* codes, uint8_t* scales, uint32_t b)
{
    constexpr int B = MX ? 32 : 16;
    if constexpr (MX) {
        const int e0 = block_exponent(top);
        int e = e0, prev = 1000;
        double best = 0.0;
        for (int k = lo; k <= hi; ++k) {
            int t = e0 + k;
            t = t < -127 ? -127 : (t > 127 ? 127 : t);
            if (t == prev)
                continue;
            const double E = exact_error<B>(v, exp2i(t), exp2i(-t));
            if (prev == 1000 || E < best) {
                best = E;
                e = t;
            }
            prev = t;
        }
        const float r = exp2i(-e);
        const uint2 c0 = fp4_encode16(v, r), c1 = fp4_encode16(v + 16, r);
        reinterpret_cast<uint4*>(codes)[b] = make_uint4(c0.x, c0.y, c1.x, c1.y);
        scales[b] = (uint8_t)(e + 127);
    } else {
        int sb = 0;
        float r = 1.0f; // an all-zero block keeps only its signs
        if (top != 0.0f) {
            sb = (int)e4m3_round(top / S6);
            sb = sb < 1 ? 1 : sb;
            if constexpr (RULE == kRuleFourSix) {
                int s4 = (int)e4m3_round(top / (4.0f * S));
                s4 = s4 < 1 ? 1 : s4;
                if (s4 != sb) {
                    const float D6 = e4m3_value((uint32_t)sb) * S, D4 = e4m3_value((uint32_t)s4) * S;
                    const double E6 = exact_error<16>(v, D6, 1.0f / D6);
                    const double E4 = exact_error<16>(v, D4, 1.0f / D4);
                    sb = E4 < E6 ? s4 : sb;
                }
            }
        }
        if constexpr (RULE == kRuleSweep) {
            // every active lane takes part, zero blocks too: the pick's
            // loop is shared by the wave
            const int c = sweep_pick(v, top, S, sb < 1 ? 1 : sb, tab, lo, hi);
            sb = top != 0.0f ? c : 0;
        }
        if (sb != 0)
            r = 1.0f / (e4m3_value((uint32_t)sb) * S);
        reinterpret_cast<uint2*>(codes)[b] = fp4_encode16(v, r);
        scales[b] = (uint8_t)sb;
    }
}

// The block transform of rows whose lanes hold E values each: widths below E within the
// lane, the wider ones across the B / E lanes that share a block, in the order and with the
// roundings of the in-register transform.
template <int B, int E>
__device__ __forceinline__ void rotate_lanes(float* v, uint32_t part)
{
#pragma unroll
    for (int h = 1; h < E; h *= 2)
#pragma unroll
        for (int i = 0; i < E; i += 2 * h)
#pragma unroll
            for (int j = i; j < i + h; ++j) {
                const float p = v[j], q = v[j + h];
                v[j] = p + q;
                v[j + h] = p - q;
            }
#pragma unroll
    for (int h = 1; h < B / E; h *= 2) {
        const float sign = (part & h) ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < E; ++i)
            v[i] = __builtin_fmaf(sign, v[i], __shfl_xor(v[i], h, 64));
    }
    const float c = (B == 16) ? 0.25f : __uint_as_float(0x3E3504F3u); // fl32(1/sqrt(B))
#pragma unroll
    for (int i = 0; i < E; ++i)
        v[i] = v[i] * c;
}

// the AbsMax scale byte of a block of maximum `top`; returns what its values are
// multiplied by before they are rounded to codes
template <bool MX>
__device__ __forceinline__ float absmax_scale(float top, float S, float S6, uint32_t& sb)
{
    if constexpr (MX) {
        const int e = block_exponent(top);
        sb = (uint32_t)(e + 127);
        return exp2i(-e);
    } else {
        const int near = (int)e4m3_round(top / S6);
        sb = top == 0.0f ? 0u : (uint32_t)(near < 1 ? 1 : near);
        return sb == 0u ? 1.0f : 1.0f / (e4m3_value(sb) * S); // an all-zero block keeps only its signs
    }
}

} // namespace fp4q
