// fp4q_kv.hip -- writing tokens into the 4-bit KV cache and reading rows back.
//
// A write is fp4q_quantize's method on the blocks of one (token, head) row
// under a given global scale, stored at a slot of the cache; a read is
// fp4q_dequantize's on the row of a slot.  Both move every byte once: they are
// bound by HBM where there are many tokens and by the launch where there are
// few (the sweep's arithmetic, not the traffic, bounds a long swept write).
// Times beside the kernels are of one call on an MI355X.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "fp4q_device.h"
#include "fp4q_kv_launch.h"

namespace fp4q {

namespace {

constexpr int kThreads = 256;
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

// The searching rules, one lane per block: load, rotate, choose the scale,
// encode, store at the slot; a block's 16 or 32 values stay in the lane's
// registers, so that neither the transform nor the candidates move anything
// between lanes.  The NVFP4 sweep is bound by the vector ALU, which every candidate
// asks for 8 conversions each way: at 8 heads of 128 bf16 values, K and V, 8192
// tokens take 36 us, of which about 7 are the latency of a call, 262144 tokens
// 912 us, 590 Gelem/s; a step's 64 tokens take 7 us of dependent loads (slot,
// scale, rows) and launch.  Its registers are held to six waves per SIMD (80,
// one value spilled; with five waves and 94 registers 931 us for 262144 tokens).
template <bool MX, int RULE, bool BF16, bool ROT>
__global__ __launch_bounds__(kThreads, RULE == kRuleSweep && !MX ? 6 : 1) void kv_write(const KvWriteArgs a, const int blocks_shift,
                                                     const uint32_t items)
{
    static_assert(RULE == kRuleSweep || (RULE == kRuleFourSix && !MX), "the searching rules");
    constexpr int B = MX ? 32 : 16;
    __shared__ Pattern tab[RULE == kRuleSweep && !MX ? 128 : 1];
    const int side = blockIdx.y;
    const float S = MX ? 1.0f : *a.kv.global[side];
    if constexpr (RULE == kRuleSweep && !MX) {
        if (threadIdx.x < 128) {
            const float s = e4m3_value(threadIdx.x < 0x7E ? threadIdx.x : 0x7Eu);
            const float D = s * S;
            tab[threadIdx.x] = Pattern{1.0f / D, s * s, D};
        }
        __syncthreads();
    }
    const float S6 = 6.0f * S;
    const uint32_t heads = (uint32_t)a.kv.heads;
    const int64_t most = a.kv.num_pages * a.kv.page_size;
    const uint32_t last = (uint32_t)(1 << blocks_shift) - 1u;
    for (uint32_t item = blockIdx.x * kThreads + threadIdx.x; item < items; item += gridDim.x * kThreads) {
        const uint32_t b = item & last;
        const uint32_t row = item >> blocks_shift;
        const uint32_t token = row / heads, head = row - token * heads;
        const int64_t slot = a.slots[token];
        if (slot < 0 || slot >= most)
            continue;
        float v[B];
        const char* x = static_cast<const char*>(a.x[side]) +
                        (token * a.x_token[side] + head * a.x_head[side]) * (BF16 ? 2 : 4);
        load_block<B, BF16>(x, b, v);
        if constexpr (ROT)
            fwht<B>(v);
        const float top = block_absmax<B>(v);
        int64_t page, off;
        slot_place(a.kv, slot, most, page, off);
        uint8_t* codes = a.kv.codes[side] + page * a.kv.c_page + head * a.kv.c_head + off * a.kv.c_token;
        uint8_t* scales = a.kv.scales[side] + page * a.kv.s_page + head * a.kv.s_head + off * a.kv.s_token;
        if constexpr (MX) {
            const int e0 = block_exponent(top);
            int e = e0, prev = 1000;
            double best = 0.0;
            for (int k = a.lo; k <= a.hi; ++k) {
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
                const int c = sweep_pick(v, top, S, sb < 1 ? 1 : sb, tab, a.lo, a.hi);
                sb = top != 0.0f ? c : 0;
            }
            if (sb != 0)
                r = 1.0f / (e4m3_value((uint32_t)sb) * S);
            reinterpret_cast<uint2*>(codes)[b] = fp4_encode16(v, r);
            scales[b] = (uint8_t)sb;
        }
    }
}

// AbsMax: each lane loads 32 bytes of a row (E = 16 bf16 or 8 binary32 values)
// and writes their codes; the transform's wide stages and the maximum cross the
// 1, 2 or 4 lanes that share a block, the sums in the order and with the
// roundings of the in-register transform.  Bound by HBM: 65536 tokens of 8 heads
// of 128 values, K and V, take 73 us from bf16 and 130 us from binary32 in either
// format, 4.7 TB/s.  With a lane per block a wave's load instruction touches 16
// bytes of each 64 or 128: 161 us for binary32 to NVFP4, 87 and 241 us for bf16
// and binary32 to MXFP4.  With 16 bytes of a row in each lane its share of the
// scale's arithmetic bounds: 97 to 177 us.
template <bool MX, bool BF16, bool ROT>
__global__ __launch_bounds__(kThreads) void kv_write_absmax(const KvWriteArgs a, const int lane_shift,
                                                            const uint32_t items)
{
    constexpr int B = MX ? 32 : 16;
    constexpr int E = BF16 ? 16 : 8;
    const int side = blockIdx.y;
    const float S = MX ? 1.0f : *a.kv.global[side];
    const float S6 = 6.0f * S;
    const uint32_t heads = (uint32_t)a.kv.heads;
    const int64_t most = a.kv.num_pages * a.kv.page_size;
    const uint32_t last = (uint32_t)(1 << lane_shift) - 1u;
    for (uint32_t item = blockIdx.x * kThreads + threadIdx.x; item < items; item += gridDim.x * kThreads) {
        const uint32_t part = item & last;
        const uint32_t row = item >> lane_shift;
        const uint32_t token = row / heads, head = row - token * heads;
        const int64_t slot = a.slots[token];
        if (slot < 0 || slot >= most)
            continue; // with all lanes of its row
        const char* x = static_cast<const char*>(a.x[side]) +
                        (token * a.x_token[side] + head * a.x_head[side]) * (BF16 ? 2 : 4);
        float v[E];
        load_block<E, BF16>(x, part, v);
        if constexpr (ROT) {
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
        float top = block_absmax<E>(v);
#pragma unroll
        for (int h = 1; h < B / E; h *= 2)
            top = __builtin_fmaxf(top, __shfl_xor(top, h, 64));
        int64_t page, off;
        slot_place(a.kv, slot, most, page, off);
        uint8_t* codes = a.kv.codes[side] + page * a.kv.c_page + head * a.kv.c_head + off * a.kv.c_token;
        uint8_t* scales = a.kv.scales[side] + page * a.kv.s_page + head * a.kv.s_head + off * a.kv.s_token;
        float r;
        uint32_t sb;
        if constexpr (MX) {
            const int e = block_exponent(top);
            r = exp2i(-e);
            sb = (uint32_t)(e + 127);
        } else {
            const int near = (int)e4m3_round(top / S6);
            sb = top == 0.0f ? 0u : (uint32_t)(near < 1 ? 1 : near);
            r = sb == 0u ? 1.0f : 1.0f / (e4m3_value(sb) * S); // an all-zero block keeps only its signs
        }
        uint32_t w[E / 8];
#pragma unroll
        for (int g = 0; g < E / 8; ++g) {
            const float* y = v + 8 * g;
            w[g] = fresh_word(y[0]); // every byte of it is written
            w[g] = fp4_pack2<0>(w[g], y[0] * r, y[1] * r);
            w[g] = fp4_pack2<1>(w[g], y[2] * r, y[3] * r);
            w[g] = fp4_pack2<2>(w[g], y[4] * r, y[5] * r);
            w[g] = fp4_pack2<3>(w[g], y[6] * r, y[7] * r);
        }
        if constexpr (BF16)
            reinterpret_cast<uint2*>(codes)[part] = make_uint2(w[0], w[E / 8 - 1]);
        else
            reinterpret_cast<uint32_t*>(codes)[part] = w[0];
        if (part % (B / E) == 0)
            scales[part / (B / E)] = (uint8_t)sb;
    }
}

// Each lane decodes and stores 16 bytes of output (E = 8 bf16 or 4 binary32
// values), so that a wave's stores are contiguous; the un-rotation's wide
// stages cross the 2, 4 or 8 lanes that share a block, in the order and with
// the roundings of the in-register transform.  Bound by HBM: 65536 rows of 8
// heads of 128 values, K and V, rotated, to bf16 move 345 MB in 89 us (3.9 TB/s)
// where every call reads other rows (six caches in turn, 450 MB), in 92 us from
// slots in no order, whose 64 bytes of codes and 8 of scales a row are parts of
// 128-byte lines.  Two or three caches in turn, 150 or 225 MB, stay in part in
// the last-level cache: 68 and 75 us.  (Plain instead of nontemporal stores: 94
// to 96 us whatever is cached.)
template <bool MX, bool BF16, bool ROT>
__global__ __launch_bounds__(kThreads) void kv_read(const KvReadArgs a, const int lane_shift,
                                                    const uint32_t items)
{
    constexpr int B = MX ? 32 : 16;
    constexpr int E = BF16 ? 8 : 4;
    const int side = blockIdx.y;
    const float S = MX ? 1.0f : *a.kv.global[side];
    const uint32_t heads = (uint32_t)a.kv.heads;
    const int64_t most = a.kv.num_pages * a.kv.page_size;
    const uint32_t last = (uint32_t)(1 << lane_shift) - 1u;
    // items is a multiple of the lanes that share a block
    for (uint32_t item = blockIdx.x * kThreads + threadIdx.x; item < items; item += gridDim.x * kThreads) {
        const uint32_t part = item & last;
        const uint32_t row = item >> lane_shift;
        const uint32_t token = row / heads, head = row - token * heads;
        const int64_t slot = a.slots[token];
        float o[E];
        if (slot < 0 || slot >= most) {
#pragma unroll
            for (int i = 0; i < E; ++i)
                o[i] = 0.0f;
        } else {
            int64_t page, off;
            slot_place(a.kv, slot, most, page, off);
            const uint8_t* codes =
                a.kv.codes[side] + page * a.kv.c_page + head * a.kv.c_head + off * a.kv.c_token;
            const uint8_t* scales =
                a.kv.scales[side] + page * a.kv.s_page + head * a.kv.s_head + off * a.kv.s_token;
            const uint32_t w = BF16 ? reinterpret_cast<const uint32_t*>(codes)[part]
                                    : (uint32_t)reinterpret_cast<const uint16_t*>(codes)[part];
            const uint32_t sb = scales[part / (B / E)];
            float D;
            if constexpr (MX) {
                D = (sb == 0xFFu) ? __builtin_nanf("") : exp2i((int)sb - 127);
            } else {
                const uint32_t mag = sb & 0x7Fu;
                float s = (mag == 0x7Fu) ? __builtin_nanf("") : e4m3_value(mag);
                D = (sb & 0x80u ? -s : s) * S;
            }
            fp4_unpack2<0>(w, o[0], o[1]);
            fp4_unpack2<1>(w, o[2], o[3]);
            if constexpr (BF16) {
                fp4_unpack2<2>(w, o[4], o[5]);
                fp4_unpack2<3>(w, o[6], o[7]);
            }
#pragma unroll
            for (int i = 0; i < E; ++i)
                o[i] = o[i] * D;
        }
        if constexpr (ROT) { // a row's lanes share its slot, so they are here together
#pragma unroll
            for (int h = 1; h < E; h *= 2)
#pragma unroll
                for (int i = 0; i < E; i += 2 * h)
#pragma unroll
                    for (int j = i; j < i + h; ++j) {
                        const float p = o[j], q = o[j + h];
                        o[j] = p + q;
                        o[j + h] = p - q;
                    }
#pragma unroll
            for (int h = 1; h < B / E; h *= 2) {
                const float sign = (part & h) ? -1.0f : 1.0f;
#pragma unroll
                for (int i = 0; i < E; ++i)
                    o[i] = __builtin_fmaf(sign, o[i], __shfl_xor(o[i], h, 64));
            }
            const float c = (B == 16) ? 0.25f : __uint_as_float(0x3E3504F3u); // fl32(1/sqrt(B))
#pragma unroll
            for (int i = 0; i < E; ++i)
                o[i] = o[i] * c;
        }
        u32x4 t;
        if constexpr (BF16) {
            t.x = bf16_pair(o[0], o[1]);
            t.y = bf16_pair(o[2], o[3]);
            t.z = bf16_pair(o[4], o[5]);
            t.w = bf16_pair(o[6], o[7]);
        } else {
            t.x = __float_as_uint(o[0]);
            t.y = __float_as_uint(o[1]);
            t.z = __float_as_uint(o[2]);
            t.w = __float_as_uint(o[3]);
        }
        __builtin_nontemporal_store(t, reinterpret_cast<u32x4*>(a.y[side]) + item);
    }
}

int log2_of(int n)
{
    int s = 0;
    while ((1 << s) < n)
        ++s;
    return s;
}

// workgroups for `items` lanes: enough to cover them, at most `most` (the
// kernels stride over the rest).  A write gets one block per lane up to 2^20
// workgroups: 2^20 tokens of 8 heads of 128 values take 1075 us with AbsMax
// and 3519 us swept, with at most 8192 workgroups 1289 and 3562.  A read is
// faster with at most 8192: 65536 such rows to bf16, in order, 89 against 105 us
// from memory and 68 against 76 where much of them is cached.
constexpr uint32_t kWriteGroups = 1u << 20, kReadGroups = 8192u;

int groups_for(uint32_t items, uint32_t most)
{
    const uint32_t g = (items + kThreads - 1) / kThreads;
    return (int)(g < most ? g : most);
}

// Tokens of one launch: item numbers, and a grid's stride past the last of
// them, stay in 32 bits.
int64_t tokens_per_launch(int heads, int lanes_per_row)
{
    const int64_t t = ((int64_t)1 << 31) / ((int64_t)heads * lanes_per_row);
    return t < 1 ? 0 : t;
}

template <bool MX, int RULE, bool BF16>
void launch_write(const KvWriteArgs& a, int shift, uint32_t items)
{
    const dim3 grid(groups_for(items, kWriteGroups), 2);
    if (a.rotate)
        kv_write<MX, RULE, BF16, true><<<grid, kThreads, 0, a.stream>>>(a, shift, items);
    else
        kv_write<MX, RULE, BF16, false><<<grid, kThreads, 0, a.stream>>>(a, shift, items);
}

template <bool MX, bool BF16>
void launch_write_absmax(const KvWriteArgs& a, int shift, uint32_t items)
{
    const dim3 grid(groups_for(items, kWriteGroups), 2);
    if (a.rotate)
        kv_write_absmax<MX, BF16, true><<<grid, kThreads, 0, a.stream>>>(a, shift, items);
    else
        kv_write_absmax<MX, BF16, false><<<grid, kThreads, 0, a.stream>>>(a, shift, items);
}

template <bool BF16>
void launch_write_rule(const KvWriteArgs& a, int shift, uint32_t items)
{
    if (a.rule == kRuleAbsMax) {
        if (a.kv.mx)
            launch_write_absmax<true, BF16>(a, shift, items);
        else
            launch_write_absmax<false, BF16>(a, shift, items);
    } else if (a.kv.mx) {
        launch_write<true, kRuleSweep, BF16>(a, shift, items);
    } else if (a.rule == kRuleSweep) {
        launch_write<false, kRuleSweep, BF16>(a, shift, items);
    } else {
        launch_write<false, kRuleFourSix, BF16>(a, shift, items);
    }
}

} // namespace

hipError_t launch_kv_write(const KvWriteArgs& all)
{
    KvWriteArgs a = all;
    const int lanes = a.kv.head_dim / (a.rule == kRuleAbsMax ? (a.bf16 ? 16 : 8) : (a.kv.mx ? 32 : 16)); // per row
    const int64_t most = tokens_per_launch(a.kv.heads, lanes);
    if (most == 0)
        return hipErrorInvalidValue;
    for (int64_t t0 = 0; t0 < all.tokens; t0 += most) {
        a.tokens = all.tokens - t0 < most ? all.tokens - t0 : most;
        a.slots = all.slots + t0;
        for (int side = 0; side < 2; ++side)
            a.x[side] = static_cast<const char*>(all.x[side]) + t0 * all.x_token[side] * (a.bf16 ? 2 : 4);
        const uint32_t items = (uint32_t)(a.tokens * a.kv.heads * lanes);
        if (a.bf16)
            launch_write_rule<true>(a, log2_of(lanes), items);
        else
            launch_write_rule<false>(a, log2_of(lanes), items);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

hipError_t launch_kv_read(const KvReadArgs& all)
{
    KvReadArgs a = all;
    const int lanes = a.kv.head_dim / (a.bf16 ? 8 : 4); // per row
    const int64_t most = tokens_per_launch(a.kv.heads, lanes);
    if (most == 0)
        return hipErrorInvalidValue;
    const int shift = log2_of(lanes);
    for (int64_t t0 = 0; t0 < all.tokens; t0 += most) {
        a.tokens = all.tokens - t0 < most ? all.tokens - t0 : most;
        a.slots = all.slots + t0;
        for (int side = 0; side < 2; ++side)
            a.y[side] = static_cast<char*>(all.y[side]) + t0 * a.kv.heads * a.kv.head_dim * (a.bf16 ? 2 : 4);
        const uint32_t items = (uint32_t)(a.tokens * a.kv.heads * lanes);
        const dim3 grid(groups_for(items, kReadGroups), 2);
        auto go = [&](auto mx, auto bf16) {
            if (a.rotate)
                kv_read<mx.value, bf16.value, true><<<grid, kThreads, 0, a.stream>>>(a, shift, items);
            else
                kv_read<mx.value, bf16.value, false><<<grid, kThreads, 0, a.stream>>>(a, shift, items);
        };
        if (a.kv.mx)
            a.bf16 ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
        else
            a.bf16 ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

} // namespace fp4q
