// fp4q_matmul_kernels.h -- products of activations with 4-bit weights: the kernels
// and their launch, for one format (fp4q_matmul_nv.hip, fp4q_matmul_mx.hip).
//
//   y_mn = S sum_k x_mk v_nk s_n(k)        (v a code's value, s its block's scale)
//
// and, of two weights, act(x W0^T) * (x W1^T).  A code times its E4M3 scale has
// at most six significant bits and lies in [2^-10, 2688], and a code times 2^e has two:
// dequantized weights enter the matrix cores exactly as bf16, and so does x of bf16; the
// global scale is one binary32 factor of the sum.
// A weight that is stored rotated is never rotated back: x W^T = (x H)(W H)^T with H
// the orthonormal block Hadamard, so x is rotated, in binary32.
//
// Parts.  Where x is not exact in bf16 (binary32, or rotated) it is given as a sum of three
// bf16 parts, one matrix product each, which hold its 24 bits (down to bf16's last bit, 2^-133),
// in every form and for any number of rows.  Fewer lose results: two parts, 16 bits, or f16
// parts under a power of two for each row (one, 11 bits; two, 22, and what lies 2^-39 below the row's
// largest value, which a weight of zero may meet) differ where sums cancel.
#pragma once

#include <hip/hip_runtime.h>

#include "fp4q_device.h"
#include "fp4q_matmul_launch.h"

namespace fp4q {
namespace {

typedef __bf16 b16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

enum Kind { kNv, kMx }; // the weights' format

__device__ __forceinline__ f32x4 mfma16(u32x4 x, u32x4 y, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b16x8, x), __builtin_bit_cast(b16x8, y), c, 0, 0, 0);
}

__device__ __forceinline__ f32x16 mfma32(u32x4 x, u32x4 y, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b16x8, x), __builtin_bit_cast(b16x8, y), c, 0, 0, 0);
}

// ---- weights -------------------------------------------------------------------

// Two codes of a word times their block's scale s.  The product has six bits: cutting it
// from binary32 to bf16 loses nothing.  (Two codes cost about 16 cycles of a SIMD, 7 for a
// power of two.)
template <Kind KIND, int SEL>
__device__ __forceinline__ uint32_t expand_pair(uint32_t w, float s)
{
    if constexpr (KIND == kMx) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, SEL));
    } else {
        float a, b;
        fp4_unpack2<SEL>(w, a, b);
        return __builtin_amdgcn_perm(__float_as_uint(b * s), __float_as_uint(a * s), 0x07060302u);
    }
}

// the eight codes of a word; s from factor_of
template <Kind KIND>
__device__ __forceinline__ u32x4 expand(uint32_t w, float s)
{
    return u32x4{expand_pair<KIND, 0>(w, s), expand_pair<KIND, 1>(w, s), expand_pair<KIND, 2>(w, s), expand_pair<KIND, 3>(w, s)};
}

// 64 values of a row of the weight: codes, and scale bytes as they came: in ONE load, or
// each in one of its own, put together where they are used, so that nothing waits for
// them before.
template <Kind KIND, bool ONE>
struct Wide {
    static constexpr int NS = ONE ? 1 : (KIND == kMx ? 2 : 4);
    u32x4 c[2];
    uint32_t s[NS];
};

template <Kind KIND, bool ONE>
__device__ __forceinline__ uint32_t scale_word(const Wide<KIND, ONE>& w)
{
    if constexpr (ONE)
        return w.s[0];
    else if constexpr (KIND == kMx)
        return w.s[0] | (w.s[1] << 8);
    else
        return w.s[0] | (w.s[1] << 8) | (w.s[2] << 16) | (w.s[3] << 24);
}

// The factor of values 8 j .. 8 j + 7 of 64: the value of their E4M3 byte, or the power of
// two of their E8M0 byte, whose exponent alone the conversions apply (255 stands for NaN).
template <Kind KIND>
__device__ __forceinline__ float factor_of(uint32_t word, int j)
{
    if constexpr (KIND == kMx) {
        return __uint_as_float((j < 4 ? word & 0xFFu : word >> 8) << 23);
    } else {
        const auto t = j < 4 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(word, 1.0f, false)
                             : __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(word, 1.0f, true);
        return t[(j >> 1) & 1];
    }
}

// Raw buffer resource over `bytes` bytes from p (uniform): a load past the end
// gives zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int64_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00027000);
}

typedef __attribute__((address_space(3))) void lds_void;

// The resource as words, and 16 or 4 bytes of every lane from there to LDS, the lanes' in order from
// `place` on (uniform, as lds_place gives it).  The compiler's own form of these loads makes it wait for all of them
// before any read of LDS in a loop; of these it knows nothing, and the caller waits.
__device__ __forceinline__ u32x4 words_of(const void* p, int64_t bytes)
{
    const uint64_t at = reinterpret_cast<uint64_t>(p);
    return u32x4{(uint32_t)at, (uint32_t)(at >> 32) & 0xFFFFu, (uint32_t)bytes, 0x00027000u};
}

template <typename T>
__device__ __forceinline__ uint32_t lds_place(T& array)
{
    return (uint32_t)(uintptr_t)(lds_void*)&array;
}

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm" // m0 is named as written, though nothing is kept there
template <int BYTES>
__device__ __forceinline__ void load_to_lds(u32x4 from, uint32_t place, int at, int uniform = 0)
{
    if constexpr (BYTES == 16)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(place), "v"(at), "s"(from), "s"(uniform) : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(place), "v"(at), "s"(from), "s"(uniform) : "memory", "m0");
}
#pragma clang diagnostic pop

// the loads past the last step have to be over before the workgroup's LDS is another's
__device__ __forceinline__ void all_loads_over()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70); // vmcnt(0)
    asm volatile("" ::: "memory");
}

// OR-ed to an offset, past every buffer's end (a select would become a branch
// around the load)
constexpr int kPast = 0x7FFFFFFF;

// Values 64 of a row from value k on, the row's places within its buffers being c_at and
// s_at (a lane's own) and c_to, s_to (uniform): past the row's end any codes, with scales
// of zero.
template <Kind KIND, bool ONE>
__device__ __forceinline__ Wide<KIND, ONE> load_wide(__amdgpu_buffer_rsrc_t codes, __amdgpu_buffer_rsrc_t scales, int c_at, int s_at,
                                                     int c_to, int s_to, int k, int cols)
{
    constexpr int B = KIND == kMx ? 32 : 16;
    Wide<KIND, ONE> t;
#pragma unroll
    for (int c = 0; c < 2; ++c)
        t.c[c] = __builtin_amdgcn_raw_buffer_load_b128(codes, (c_at + 16 * c) | (k < cols - 32 * c ? 0 : kPast), c_to, 0);
    if constexpr (ONE) {
        const int past = k < cols ? 0 : kPast;
        t.s[0] = KIND == kMx ? (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(scales, s_at | past, s_to, 0)
                                 : __builtin_amdgcn_raw_buffer_load_b32(scales, s_at | past, s_to, 0);
    } else {
#pragma unroll
        for (int q = 0; q < 64 / B; ++q)
            t.s[q] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(scales, (s_at + q) | (k < cols - q * B ? 0 : kPast), s_to, 0);
    }
    return t;
}

// ---- activations ------------------------------------------------------------------

constexpr int kParts = 3; // of x that is not exact in bf16

// x as a sum of three bf16 values, their bits in the upper halves of h: cut, the remainder
// cut again, and the last part rounded to nearest even (exact but for what lies below
// 2^-133).  A value that is not finite is its first part alone.
__device__ __forceinline__ void parts_of(float x, uint32_t* h)
{
    const bool finite = __builtin_fabsf(x) < __builtin_huge_valf();
    h[0] = finite ? __float_as_uint(x) & 0xFFFF0000u : f32_to_bf16(x) << 16;
    float rest = finite ? x - __uint_as_float(h[0]) : 0.0f;
    h[1] = __float_as_uint(rest) & 0xFFFF0000u;
    rest -= __uint_as_float(h[1]);
    h[2] = f32_to_bf16(rest) << 16;
}

// the B values of a block of x, widened and rotated
template <int B>
__device__ __forceinline__ void load_x(const MatmulArgs& a, int64_t row, int64_t k, float* v)
{
    const int64_t at = row * a.x_row + k;
    if (a.bf16)
        load_block<B, true, false>(static_cast<const uint16_t*>(a.x) + at, 0, v);
    else
        load_block<B, false, false>(static_cast<const float*>(a.x) + at, 0, v);
    if (a.rotate)
        fwht<B>(v);
}

// eight values in parts, as they lie in memory
__device__ __forceinline__ void parts_of8(const float* v, u32x4* to)
{
    uint32_t h[8][kParts];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        parts_of(v[j], h[j]);
#pragma unroll
    for (int q = 0; q < kParts; ++q)
        to[q] = u32x4{h[0][q] >> 16 | h[1][q], h[2][q] >> 16 | h[3][q], h[4][q] >> 16 | h[5][q], h[6][q] >> 16 | h[7][q]};
}

// The parts of x: [part][m][k] in the workspace, a block of values a thread.  Moves x once;
// 37 rows of 4064: 5.6 us, a launch's latency; 509 of 4096: 9.
template <Kind KIND>
__global__ __launch_bounds__(256) void matmul_parts(const MatmulArgs a)
{
    constexpr int B = KIND == kMx ? 32 : 16;
    const int64_t blocks = a.k / B, all = a.m * blocks, plane = a.m * a.k;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < all; u += (int64_t)gridDim.x * 256) {
        const int64_t row = u / blocks, b = u - row * blocks;
        float v[B];
        load_x<B>(a, row, b * B, v);
        uint16_t* to = static_cast<uint16_t*>(a.workspace) + u * B;
#pragma unroll
        for (int i = 0; i < B / 8; ++i) {
            u32x4 part[kParts];
            parts_of8(v + 8 * i, part);
#pragma unroll
            for (int q = 0; q < kParts; ++q)
                *reinterpret_cast<u32x4*>(to + q * plane + 8 * i) = part[q];
        }
    }
}

// ---- results --------------------------------------------------------------------------

__device__ __forceinline__ float activation(int act, float g)
{
    if (act == kActSilu)
        return g / (1.0f + expf(-g));
    if (act == kActGelu) // g Phi(g); 1 + erf(g / sqrt 2) would cancel below zero, all digits at -5.5
        return 0.5f * g * erfcf(-g * 0.70710678118654752f);
    // 0.5 g (1 + tanh z) = g / (1 + exp(-2 z))
    const float z = 0.79788456080286536f * (g + 0.044715f * g * g * g);
    return g / (1.0f + expf(-2.0f * z));
}

// four values of row m of y from column n (a multiple of four) on
__device__ __forceinline__ void store4(const MatmulArgs& a, int64_t m, int64_t n, f32x4 v)
{
    const int64_t at = m * a.y_row + n;
    if (a.y_wide && n + 4 <= a.n) {
        if (a.bf16)
            *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.y) + at) = u32x2{bf16_pair(v.x, v.y), bf16_pair(v.z, v.w)};
        else
            *reinterpret_cast<f32x4*>(static_cast<float*>(a.y) + at) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + i < a.n) {
            if (a.bf16)
                static_cast<uint16_t*>(a.y)[at + i] = (uint16_t)(bf16_pair(v[i], v[i]) & 0xFFFFu);
            else
                static_cast<float*>(a.y)[at + i] = v[i];
        }
}

// y's values from the sums of one weight, or of two
template <Kind KIND, int NW>
__device__ __forceinline__ f32x4 finish4(const MatmulArgs& a, f32x4* sum)
{
    if constexpr (KIND != kMx) {
#pragma unroll
        for (int w = 0; w < NW; ++w)
            sum[w] *= *a.global[w];
    }
    f32x4 r = sum[0];
    if constexpr (NW == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = activation(a.act, r[i]) * sum[1][i];
    }
    return r;
}

// eight values of row m of y from column n (a multiple of eight) on
__device__ __forceinline__ void store8(const MatmulArgs& a, int64_t m, int64_t n, f32x4 u, f32x4 v)
{
    if (a.y_wide && a.bf16 && n + 8 <= a.n) {
        const u32x4 w = u32x4{bf16_pair(u.x, u.y), bf16_pair(u.z, u.w), bf16_pair(v.x, v.y), bf16_pair(v.z, v.w)};
        __builtin_memcpy(__builtin_assume_aligned(static_cast<uint16_t*>(a.y) + m * a.y_row + n, 8), &w, 16);
        return;
    }
    store4(a, m, n, u);
    if (n + 4 < a.n)
        store4(a, m, n + 4, v);
}

__device__ __forceinline__ f32x4* partials_of(const MatmulArgs& a, const MatmulPlan& p)
{
    return reinterpret_cast<f32x4*>(static_cast<char*>(a.workspace) + p.partials);
}

// ---- few rows of x ------------------------------------------------------------------
//
// A workgroup of RW x KW waves takes 16 RW rows of the weight (of each of two) and up to 16 XT
// rows of x; RW waves share the rows, KW the long axis, 256 values a step.  W is the
// first operand of 16x16x32 products: lane n + 16 g has the 32 bytes of row n that hold
// values 64 g .. 64 g + 63 of a step and gives them to eight products, eight at a
// time.  In memory neighbouring lanes would so read rows apart, an access of the cache each;
// the codes are therefore loaded into LDS directly, eight neighbouring lanes 128 bytes of a row,
// and read from there (each wave its own: no barrier; 16-byte units are exchanged by an XOR
// with the row, so that 16 rows' meet all banks).  kStages steps are held or on their way.
// x comes from LDS too, where the whole workgroup put it (CONV: rotated and cut into bf16
// parts on the way; else as it is, or as matmul_parts left it).
//   Bound by latency for small weights (one token, 4096 x 4096, NVFP4: 4.5 us in a graph).  14336 x
// 4096, NVFP4, in a graph: one token 10.5 us, 3.1 TB/s of weights (MXFP4 7.9); 16 tokens, whose x of
// 128 KiB each workgroup takes to its LDS, 12.3; with weights that do not stay in the last-level
// cache 11.7 and 12.6.  Of a compute unit's cycles there the vector ALU, which expands, is busy in 43
// and 39 of 100, the matrix cores in 9 and 7, LDS in 14 and 19, and half of the waves' time is
// waiting (52 and 40 of 100): the two waves of a SIMD do not hide the loads behind the expansion.
// Three parts of x: 8 and 16 tokens 19.5 and 28.4, chunk after chunk waited for.  Scale bytes come
// four at a time where every row allows it (two weights of 14336 x 4096, before other steps: 24 us;
// a byte at a time 30).  Waves that begin at different steps, to spread the rows' lines over the
// memory's channels, were slower (10.1 -> 13.4 us).
constexpr int kStages = 3;

template <Kind KIND, int NW, int PARTS, bool CONV, int XT, int RW, int KW, bool ONE>
__global__ __launch_bounds__(64 * RW * KW) void matmul_few(const MatmulArgs a, const MatmulPlan p)
{
    constexpr int B = KIND == kMx ? 32 : 16;
    constexpr int T = 64 * RW * KW;
    constexpr int U = kFewStep / 8; // 16-byte units of x in a step
    constexpr int NS = Wide<KIND, ONE>::NS;
    constexpr bool MX = KIND == kMx;
    extern __shared__ u32x4 lds[];
    __shared__ u32x4 cbuf[RW * KW][kStages][NW][16 * 8]; // by wave
    __shared__ uint32_t sbuf[RW * KW][kStages][NW][ONE ? 64 : 1];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int r = lane & 15, g = lane >> 4;
    const int rw = wave % RW, kw = wave / RW;
    const int64_t n0 = (int64_t)blockIdx.x * p.rows;
    const int mt = (int)a.m;
    const int cols = (int)a.k, steps = (cols + kFewStep - 1) / kFewStep;

    // this wave's rows of each weight, from its first one on
    const int64_t nw = n0 + rw * 16;
    const int64_t left = a.n - nw;
    const int live = left <= 0 ? 0 : (int)(left < 16 ? left : 16);
    const int crow = cols / 2, srow = cols / B;
    const int64_t first = live > 0 ? nw : 0;
    u32x4 codes[NW];
    __amdgpu_buffer_rsrc_t scales[NW];
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        codes[w] = words_of(a.codes[w] + first * crow, live * crow);
        scales[w] = buffer_of(a.scales[w] + first * srow, live * srow);
    }
    // one step's loads, whose number never changes: past the row's end any codes, with scales of
    // zero; past the last step past the buffers' ends
    constexpr int PER = NW * (2 + NS);
    int c_unit[2], c_row[2]; // of this lane's 16 bytes of each load
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = 8 * i + (lane >> 3);
        c_unit[i] = (lane & 7) ^ ((row >> 1) & 7);
        c_row[i] = row * crow;
    }
    const int s_row = MX ? (lane >> 1) & 15 : lane >> 2, s_dword = MX ? lane & 1 : lane & 3;
    uint32_t bytes[kStages][NW][NS];
    const uint32_t c_place = lds_place(cbuf), s_place = lds_place(sbuf), x_place = (uint32_t)(uintptr_t)(lds_void*)lds;
    auto load = [&](int step, int to) {
        asm volatile("" ::: "memory"); // the loads of two steps keep their order
        const int k = step * kFewStep;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                load_to_lds<16>(codes[w], c_place + (((wave * kStages + to) * NW + w) * 128 + 64 * i) * 16, (c_row[i] + k / 2 + c_unit[i] * 16) | (k < cols - c_unit[i] * 32 ? 0 : kPast));
            if constexpr (ONE) {
                load_to_lds<4>(words_of(a.scales[w] + first * srow, live * srow), s_place + ((wave * kStages + to) * NW + w) * 256,
                               (s_row * srow + k / B + 4 * s_dword) | (k < cols - 4 * B * s_dword && !(MX && lane >= 32) ? 0 : kPast));
            } else {
                const int at = r * srow + (k + 64 * g) / B;
#pragma unroll
                for (int q = 0; q < NS; ++q)
                    bytes[to][w][q] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(scales[w], (at + q) | (k < cols - 64 * g - q * B ? 0 : kPast), 0, 0);
            }
        }
        asm volatile("" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
        load(kw + KW * i, i);

    // x of chunk_steps steps from step `from` on: [part][row][value], rows padded
    // by 16 bytes so that 16 rows meet all banks
    const int stride = p.chunk_steps * U + 1;
    auto fill = [&](int from) {
        if constexpr (CONV) {
            const int per = p.chunk_steps * (kFewStep / B); // blocks of a row
            for (int u = threadIdx.x; u < mt * per; u += T) {
                const int row = u / per, b = u - row * per;
                const int k = from * kFewStep + b * B;
                u32x4* to = lds + row * stride + b * (B / 8);
                float v[B];
                if (k < cols) {
                    load_x<B>(a, row, k, v);
                } else {
#pragma unroll
                    for (int i = 0; i < B; ++i)
                        v[i] = 0.0f;
                }
#pragma unroll
                for (int i = 0; i < B / 8; ++i) {
                    u32x4 part[kParts];
                    parts_of8(v + 8 * i, part);
#pragma unroll
                    for (int q = 0; q < kParts; ++q)
                        to[q * mt * stride + i] = part[q];
                }
            }
        } else {
            // 64 units of a row a load, rows of all parts in turn
            const int per = p.chunk_steps * U / 64, row_of = (int)(p.prepared ? a.k : a.x_row) * 2;
            const u32x4 x = words_of(p.prepared ? a.workspace : a.x, (int64_t)(PARTS * mt - 1) * row_of + cols * 2);
            int row = 0, c = wave;
            for (;;) {
                for (; c >= per; c -= per)
                    ++row;
                if (row >= PARTS * mt)
                    break;
                const int k = from * kFewStep + c * 512 + lane * 8;
                load_to_lds<16>(x, x_place + (row * stride + c * 64) * 16, k * 2 | (k < cols ? 0 : kPast), row * row_of);
                c += RW * KW;
            }
            all_loads_over();
        }
    };

    f32x4 acc[NW][XT];
#pragma unroll
    for (int i = 0; i < NW * XT; ++i)
        acc[i / XT][i % XT] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    int x_at[XT]; // this lane's rows of x; lanes past the last repeat it
#pragma unroll
    for (int i = 0; i < XT; ++i)
        x_at[i] = (16 * i + r < mt ? 16 * i + r : mt - 1) * stride + 8 * g;

    const int turns = p.chunk_steps / KW; // of this wave in a chunk
    const int all = (steps + KW - 1) / KW; // the same for every wave of the workgroup
    int in_chunk = turns;
    for (int base = 0; base < all; base += kStages) {
#pragma unroll
        for (int d = 0; d < kStages; ++d) {
            const int i = base + d;
            if (i >= all)
                break;
            if (in_chunk == turns) {
                if (i != 0)
                    __syncthreads();
                fill(i * KW);
                __syncthreads();
                in_chunk = 0;
            }
            const u32x4* x = lds + (in_chunk * KW + kw) * U;
            load(kw + KW * (i + kStages - 1), (d + kStages - 1) % kStages);
            // this step's loads have arrived; those of the later ones may still be on their way
            constexpr int STAY = (kStages - 1) * PER;
            static_assert(STAY < 64, "what the counter of loads holds");
            __builtin_amdgcn_s_waitcnt(0x0F70 | (STAY & 15) | ((STAY >> 4) << 14)); // vmcnt alone
            asm volatile("" ::: "memory");
            Wide<KIND, ONE> t[NW];
            uint32_t word[NW];
#pragma unroll
            for (int w = 0; w < NW; ++w) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    t[w].c[c] = cbuf[wave][d][w][r * 8 + ((2 * g + c) ^ ((r >> 1) & 7))];
                if constexpr (ONE) {
                    word[w] = MX ? (sbuf[wave][d][w][2 * r + (g >> 1)] >> (16 * (g & 1))) & 0xFFFFu : sbuf[wave][d][w][4 * r + g];
                } else {
#pragma unroll
                    for (int q = 0; q < NS; ++q)
                        t[w].s[q] = bytes[d][w][q];
                    word[w] = scale_word(t[w]);
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                u32x4 xv[XT][PARTS];
#pragma unroll
                for (int i = 0; i < XT; ++i)
#pragma unroll
                    for (int q = 0; q < PARTS; ++q)
                        xv[i][q] = x[x_at[i] + q * mt * stride + j];
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const u32x4 wv = expand<KIND>(t[w].c[j >> 2][j & 3], factor_of<KIND>(word[w], j));
#pragma unroll
                    for (int q = PARTS - 1; q >= 0; --q) // small parts first
#pragma unroll
                        for (int i = 0; i < XT; ++i)
                            acc[w][i] = mfma16(wv, xv[i][q], acc[w][i]);
                }
            }
            asm volatile("" ::: "memory"); // the next load into this stage comes after these reads
            ++in_chunk;
        }
    }

    all_loads_over();
    // join the waves that share rows, in order
    __syncthreads();
    f32x4* red = reinterpret_cast<f32x4*>(lds);
#pragma unroll
    for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int i = 0; i < XT; ++i)
            red[((wave * NW + w) * XT + i) * 64 + lane] = acc[w][i];
    __syncthreads();
    for (int u = threadIdx.x; u < RW * XT * 64; u += T) {
        const int l = u & 63, tile = (u >> 6) % XT, part = (u >> 6) / XT;
        const int64_t n = n0 + part * 16 + 4 * (l >> 4), m = 16 * tile + (l & 15);
        if (n >= a.n || m >= a.m)
            continue;
        f32x4 sum[NW];
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            sum[w] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < KW; ++k)
                sum[w] += red[(((k * RW + part) * NW + w) * XT + tile) * 64 + l];
        }
        store4(a, m, n, finish4<KIND, NW>(a, sum));
    }
}

constexpr int kReadAhead = 2; // reads of x from LDS before their products

// ---- many rows of x -------------------------------------------------------------------
//
// A workgroup of WN waves takes 32 TM rows of x and 64 WN of the weight (32 WN of each
// of two), in 32x32x16 products.  The x of a step, 128 values of each row, lies in LDS,
// double buffered, loaded there directly; every wave reads all of it and multiplies it
// by its own 64 rows of the weight, which it loads and expands itself, so that no code
// is expanded twice in a workgroup and no expanded weight passes through LDS.
//   Lane n + 32 h holds, of a row, the values 64 h .. 64 h + 63 of a step, eight for each
// product: W's come as 32 bytes of codes.  16-byte units of a row of x are exchanged in LDS by
// an XOR with the row, so that 16 lanes that read one unit of 16 rows meet all banks; a
// lane loads the unit that belongs at its place.
//   Row 8 q + 4 h + e of a product's 32 rows of W is column 16 h + 4 q + e of y, so that a
// lane ends with 16 neighbouring columns.
//   While the products of eight values run, the weights of the next eight are expanded; the
// last ones' are those of the next step.  Two steps' x and codes are held or on their way, each
// in a buffer and registers of its own.  (Loads three steps ahead changed
// nothing at any size, nor did x read from LDS four products ahead with TM = 1, 2.)
//   The parts of x are rows of one step (PARTS = 3), so that W is read and expanded once for
// them, where a tile has 32 rows; else a part is a step of its own.
//   Bound by several units at once.  8192 rows, 14336 x 4096, NVFP4 bf16, TM = 4: 831 us, 1157
// TFLOP/s; of a SIMD's cycles the matrix cores are busy in 56 of 100 and the vector ALU, which
// expands, in 43, LDS gives x to a CU at 64 bytes a clock and each 16 bytes of a lane feed
// two products, and the clock is at 1.87 GHz under the power that this takes.  MXFP4, whose
// codes take one instruction a pair, 774 to 823 us.  Products of 128 weight rows a wave would
// halve the reads of x and spill registers (1240 us); 16x16x32 products spill too.  A step of a
// workgroup costs its CU 0.95, 1.15, 1.9 us with TM = 1, 2, 4.  Rotated x, in three parts: 2284 us, 1264
// TFLOP/s of its products, the matrix cores busy in 74 of 100.
//   Of few tiles, a wave a SIMD, none of these is near its rate, of 100 cycles: 64 rows, 14336 x 4096,
// NVFP4, and 48 rows, 4096 x 14336, MXFP4 (XM = 2, 14 and 15 us beside the join): matrix cores 23 and
// 23, vector ALU 32 and 15, LDS 8 and 8, waits 27 and 34, memory 3.6 and 3.9 TB/s with the partial
// sums; 32 rows in three parts: 27, 26, 7 and 14.  A wave's products, expansion and waits follow
// each other there.
constexpr int WN = 4; // waves of a workgroup
constexpr int TN = 2; // products of 32 weight rows in a wave

// the tile of number id: eight rows of tiles at a time, the rows fastest
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t tiles_m, uint32_t tiles_n, uint32_t& m, uint32_t& n)
{
    constexpr uint32_t kGroup = 8;
    const uint32_t band = id / (kGroup * tiles_n), first = band * kGroup;
    const uint32_t high = tiles_m - first < kGroup ? tiles_m - first : kGroup;
    const uint32_t in = id - band * kGroup * tiles_n;
    // (division is the vector unit's: the results are brought back to scalar registers)
    m = __builtin_amdgcn_readfirstlane(first + in % high);
    n = __builtin_amdgcn_readfirstlane(in / high);
}

template <Kind KIND, int NW, int XM, int PARTS, bool ONE>
__global__ __launch_bounds__(64 * WN, 2) void matmul_many(const MatmulArgs a, const MatmulPlan p)
{
    constexpr int B = KIND == kMx ? 32 : 16;
    constexpr int TM = XM * PARTS;   // products of 32 rows of x or of its parts in a step
    constexpr int BM = 32 * XM;
    constexpr int D = 2;             // steps held
    constexpr int WC = 32 * TN / NW; // columns of y of a wave
    constexpr int BN = WC * WN;
    constexpr int U = kStepK / 8;    // 16-byte units of a row of x
    constexpr bool MX = KIND == kMx;
    constexpr bool STAGED = TM <= 2;     // codes through LDS
    constexpr int NS = Wide<KIND, ONE>::NS;
    __shared__ u32x4 xbuf[D][32 * TM * U];
    __shared__ u32x4 cbuf[STAGED ? WN : 1][D][STAGED ? 128 * TN : 1];
    __shared__ uint32_t sbuf[STAGED && ONE ? WN : 1][D][STAGED && ONE ? 64 * TN : 1];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int n = lane & 31, h = lane >> 5;

    // workgroups of one XCD (every eighth) take neighbouring tiles
    const uint32_t tiles_m = (uint32_t)((a.m + BM - 1) / BM), tiles_n = (uint32_t)((a.n + BN - 1) / BN);
    const uint32_t all = tiles_m * tiles_n;
    uint32_t id = blockIdx.x;
    {
        const uint32_t xcd = id % 8, per = all / 8, more = all % 8;
        id = xcd * per + (xcd < more ? xcd : more) + id / 8;
    }
    uint32_t tile_m, tile_n;
    tile_of(id, tiles_m, tiles_n, tile_m, tile_n);
    const int64_t m0 = (int64_t)tile_m * BM, n0 = (int64_t)tile_n * BN;

    const int cols = (int)a.k;
    const int steps = (cols + kStepK - 1) / kStepK;
    const int s0 = (int)blockIdx.z * p.split_steps;
    const int s1 = s0 + p.split_steps < steps ? s0 + p.split_steps : steps;
    const int parts = PARTS == 1 ? p.parts : 1;
    const int turns = (s1 - s0) * parts; // a step for each part of x, the small ones first
    // Offsets are a lane's own (in a vector register) and a uniform part that never passes
    // the buffer's end, where the check against it would wrap: rows of a tile that do not
    // exist are replaced by others, whose results are not stored.

    // x, or its parts: plane q, row m
    const int64_t m_left = a.m - m0;
    const int rows = (int)(m_left < BM ? m_left : BM);
    const int x_row = (int)(p.prepared ? a.k : a.x_row) * 2; // bytes
    const char* x = static_cast<const char*>(p.prepared ? a.workspace : a.x) + m0 * x_row;
    const int64_t plane = a.m * a.k * 2;
    constexpr int LOADS = 32 * TM / (4 * WN); // of a wave: four rows each
    const int quad = lane >> 4;          // row of the four
    constexpr int KINDS = LOADS < 4 ? LOADS : 4; // the exchange of units repeats every four loads
    int x_unit[KINDS];
#pragma unroll
    for (int i = 0; i < KINDS; ++i)
        x_unit[i] = (lane & 15) ^ ((4 * (wave * LOADS + i) + quad) & 15);
    const uint32_t x_place = lds_place(xbuf), c_place = lds_place(cbuf), s_place = lds_place(sbuf);
    auto load_x_tile = [&](int step, int turn_part, bool real, int to) {
        const bool whole = (step + 1) * kStepK <= cols;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int place = (wave * LOADS + i) * 4, part = PARTS == 1 ? turn_part : place / BM, row = place - (PARTS == 1 ? 0 : part * BM);
            const u32x4 src = words_of(x + part * plane, (int64_t)(rows - 1) * x_row + cols * 2);
            int at = (quad * x_row + x_unit[i % KINDS] * 16) | (real ? 0 : kPast);
            if (!whole) // values past the row's end are zeros
                at |= step * kStepK + x_unit[i % KINDS] * 8 < cols ? 0 : kPast;
            load_to_lds<16>(src, x_place + (to * 32 * TM * U + (wave * LOADS + i) * 64) * 16, at,
                            (row < rows ? row : 0) * x_row + step * (kStepK * 2));
        }
    };

    // the wave's rows of each weight, 32 for a product
    const int64_t nw = n0 + wave * WC;
    const int64_t left = a.n - nw;
    const int64_t from = left > 0 ? nw : 0;
    const int live = (int)(left <= 0 ? 1 : (left < WC ? left : WC));
    const int crow = cols / 2, srow = cols / B;
    __amdgpu_buffer_rsrc_t codes[NW], scales[NW];
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        codes[w] = buffer_of(a.codes[w] + from * crow, live * crow);
        scales[w] = buffer_of(a.scales[w] + from * srow, live * srow);
    }
    auto row_of = [](int r) { return 16 * ((r >> 2) & 1) + 4 * (r >> 3) + (r & 3); }; // of a product's
    const int w_row = row_of(n);
    const int c_at = w_row * crow + 32 * h, s_at = w_row * srow + 64 * h / B;
    // STAGED: 16 lanes load 16 rows' 64 bytes of codes, four neighbouring ones a row's (an access
    // of the cache for each row, not for each lane), 16-byte units exchanged by an XOR with the
    // row; the scales four bytes a lane
    int c_unit[2], c_row[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = 16 * i + (lane >> 2);
        c_unit[i] = (lane & 3) ^ ((row >> 2) & 3);
        c_row[i] = row_of(row) * crow;
    }
    auto load_w = [&](int step, bool real, int to, Wide<KIND, ONE> (&t)[TN]) {
#pragma unroll
        for (int i = 0; i < TN; ++i) {
            const int w = NW == 2 ? i / (TN / 2) : 0, row = 32 * (NW == 2 ? i % (TN / 2) : i), up = row < live ? row : 0;
            const int c_to = up * crow + step * (kStepK / 2), s_to = up * srow + step * (kStepK / B);
            const int k = real ? step * kStepK : kPast / 2;
            if constexpr (!STAGED) {
                t[i] = load_wide<KIND, ONE>(codes[w], scales[w], c_at, s_at, c_to, s_to, k + 64 * h, cols);
                continue;
            }
            const u32x4 from_c = words_of(a.codes[w] + from * crow, live * crow);
#pragma unroll
            for (int c = 0; c < 2; ++c)
                load_to_lds<16>(from_c, c_place + ((wave * D + to) * 128 * TN + 128 * i + 64 * c) * 16, (c_row[c] + c_unit[c] * 16) | (k < cols - c_unit[c] * 32 ? 0 : kPast),
                                c_to);
            if constexpr (!ONE) {
#pragma unroll
                for (int q = 0; q < NS; ++q)
                    t[i].s[q] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(scales[w], (s_at + q) | (k + 64 * h < cols - q * B ? 0 : kPast), s_to, 0);
            } else if constexpr (MX) { // a dword a row: 32 lanes, the others bring zeros
                load_to_lds<4>(words_of(a.scales[w] + from * srow, live * srow), s_place + ((wave * D + to) * 64 * TN + 64 * i) * 4,
                               (row_of(n) * srow) | (k < cols && lane < 32 ? 0 : kPast), s_to);
            } else {
                const int r = lane >> 1, half = lane & 1;
                load_to_lds<4>(words_of(a.scales[w] + from * srow, live * srow), s_place + ((wave * D + to) * 64 * TN + 64 * i) * 4,
                               (row_of(r) * srow + 4 * half) | (k < cols - 64 * half ? 0 : kPast), s_to);
            }
        }
    };
    // STAGED: half of this lane's codes of a step; with the first half, for which the step's
    // loads must have arrived (but for those of x, which are the last ones), the scales
    auto take_half = [&](int at, int c, Wide<KIND, ONE> (&t)[TN]) {
        if (c == 0) {
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(0x0F70 | LOADS);
            asm volatile("" ::: "memory");
        }
#pragma unroll
        for (int i = 0; i < TN; ++i) {
            t[i].c[c] = cbuf[wave][at][(32 * i + n) * 4 + ((2 * h + c) ^ ((n >> 2) & 3))];
            if (ONE && c == 0)
                t[i].s[0] = MX ? (sbuf[wave][at][64 * i + n] >> (16 * h)) & 0xFFFFu : sbuf[wave][at][2 * (32 * i + n) + h];
        }
    };
    static_assert(LOADS < 16, "what take_half waits for");

    f32x16 acc[XM][TN];
#pragma unroll
    for (int i = 0; i < XM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                acc[i][j][e] = 0.0f;

    Wide<KIND, ONE> ring[D][TN];
    u32x4 wv[2][TN];
    uint32_t word[TN];
    float factor[TN];
    // pairs `at` .. `at` + COUNT - 1 of those of values 8 j .. 8 j + 7, four a tile
    auto expand_pairs = [&](const Wide<KIND, ONE> (&t)[TN], int j, int at, int count) {
#pragma unroll
        for (int q = at; q < at + count; ++q) {
            const int i = q >> 2;
            if ((q & 3) == 0) {
                if (j == 0)
                    word[i] = scale_word(t[i]);
                factor[i] = factor_of<KIND>(word[i], j);
            }
            const uint32_t w = t[i].c[j >> 2][j & 3];
            switch (q & 3) {
            case 0: wv[j & 1][i].x = expand_pair<KIND, 0>(w, factor[i]); break;
            case 1: wv[j & 1][i].y = expand_pair<KIND, 1>(w, factor[i]); break;
            case 2: wv[j & 1][i].z = expand_pair<KIND, 2>(w, factor[i]); break;
            default: wv[j & 1][i].w = expand_pair<KIND, 3>(w, factor[i]); break;
            }
        }
    };
    // Loads of a step, whose number never changes: past the last step they are made past
    // their buffers' ends.
    int next_step = s0, next_part = parts - 1, next_turn = 0;
    auto load_turn = [&](int to) {
        const bool real = next_turn < turns;
        asm volatile("" ::: "memory"); // the loads of two steps keep their order
        load_w(next_step, real, to, ring[to]);
        load_x_tile(next_step, next_part, real, to);
        asm volatile("" ::: "memory");
        ++next_turn;
        if (next_part == 0) {
            next_part = parts;
            next_step += next_turn < turns ? 1 : 0;
        }
        --next_part;
    };
    if (turns > 0) {
        load_turn(0);
        if constexpr (STAGED)
            take_half(0, 0, ring[0]);
        expand_pairs(ring[0], 0, 0, 4 * TN);
    }
    for (int base = 0; base < turns; base += D)
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (base + d >= turns)
                break;
            // this wave's loads have arrived; after the barrier that holds for every wave, and the
            // buffer of the step before this one is free: its reads have all been used by products
            all_loads_over();
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            load_turn((d + 1) % D);
            auto read_x = [&](int i) { // the i-th of the step's reads
                const int row = 32 * (TM - 1 - i % TM) + n; // small parts first
                return xbuf[d][row * U + ((8 * h + i / TM) ^ (n & 15))];
            };
            u32x4 xv[kReadAhead];
#pragma unroll
            for (int i = 0; i < kReadAhead; ++i)
                xv[i] = read_x(i);
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const int x_turn = j * TM + i;
                    if (STAGED && i == 0 && j == 2)
                        take_half(d, 1, ring[d]);
                    if (STAGED && i == 0 && j == 6)
                        take_half((d + 1) % D, 0, ring[(d + 1) % D]);
                    const u32x4 mine = xv[x_turn % kReadAhead];
                    if (x_turn + kReadAhead < 8 * TM)
                        xv[x_turn % kReadAhead] = read_x(x_turn + kReadAhead);
#pragma unroll
                    for (int t = 0; t < TN; ++t) {
                        // the order of these is kept: a product, and what is expanded while it runs
                        __builtin_amdgcn_sched_barrier(0);
                        f32x16& sum = acc[(TM - 1 - i) % XM][t];
                        sum = mfma32(wv[j & 1][t], mine, sum);
                        const int at = (TN * i + t) * 4 / TM, end = (TN * i + t + 1) * 4 / TM;
                        expand_pairs(ring[j < 7 ? d : (d + 1) % D], (j + 1) & 7, at, end - at);
                    }
                }
        }
    all_loads_over();

    // a lane's results: of row m of y 16 neighbouring columns for each tile
    constexpr int TC = TN / NW; // tiles of a weight
    if (p.splits > 1) { // partial sums as they lie in the registers: four a lane, the lanes' in order
        f32x4* to = partials_of(a, p) + ((size_t)blockIdx.z * all + id) * (WN * XM * TN * 4 * 64) + (size_t)wave * (XM * TN * 4 * 64) + lane;
#pragma unroll
        for (int i = 0; i < XM; ++i) {
            if (32 * i + n >= rows)
                break;
#pragma unroll
            for (int t = 0; t < TN; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x16& v = acc[i][t];
                    to[((i * TN + t) * 4 + q) * 64] = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
                }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < XM; ++i) {
        const int64_t m = m0 + 32 * i + n;
        if (m >= a.m)
            continue;
#pragma unroll
        for (int t = 0; t < TC; ++t)
#pragma unroll
            for (int q = 0; q < 4; q += 2) {
                const int64_t col = nw + 32 * t + 16 * h + 4 * q;
                if (col >= a.n)
                    continue;
                f32x4 y[2];
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    f32x4 sum[NW];
#pragma unroll
                    for (int w = 0; w < NW; ++w)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            sum[w][e] = acc[i][w * TC + t][4 * (q + o) + e];
                    y[o] = finish4<KIND, NW>(a, sum);
                }
                store8(a, m, col, y[0], y[1]);
            }
    }
}

// The sums of all splits, in order, and the results: a workgroup for the partial sums of 32 rows
// of x and 32 of each weight, a wave for a quarter of the columns, whose lanes have what
// the lanes that left them had: all reads are of whole lines, in the order they were written.
// 2 to 16 splits of up to 64 x 14336 results: 4 to 7 us.
template <Kind KIND, int NW, int XM>
__global__ __launch_bounds__(256) void matmul_join(const MatmulArgs a, const MatmulPlan p)
{
    constexpr int TC = TN / NW, WC = 32 * TC, BM = 32 * XM, BN = WC * WN;
    const uint32_t tiles_m = (uint32_t)((a.m + BM - 1) / BM), tiles_n = (uint32_t)((a.n + BN - 1) / BN), all = tiles_m * tiles_n;
    const int lane = threadIdx.x & 63, q = threadIdx.x >> 6, n = lane & 31, h = lane >> 5;
    uint32_t rest = blockIdx.x;
    const uint32_t t = rest % TC;
    rest /= TC;
    const uint32_t i = rest % XM;
    rest /= XM;
    const uint32_t wave = rest % WN, id = rest / WN;
    uint32_t row, col;
    tile_of(id, tiles_m, tiles_n, row, col);
    const int64_t m = (int64_t)row * BM + 32 * i + n, c = (int64_t)col * BN + wave * WC + 32 * t + 16 * h + 4 * q;
    if (m >= a.m || c >= a.n)
        return;
    f32x4 sum[NW];
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const f32x4* from = partials_of(a, p) + (size_t)id * (WN * XM * TN * 256) + wave * (XM * TN * 256) + ((i * TN + w * TC + t) * 4 + q) * 64 + lane;
        sum[w] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int s = 0; s < p.splits; ++s)
            sum[w] += from[(size_t)s * all * (WN * XM * TN * 256)];
    }
    store4(a, m, c, finish4<KIND, NW>(a, sum));
}

// ---- launch -------------------------------------------------------------------------------

// whether the scale bytes of every row can be loaded four at a time
inline bool scales_together(const MatmulArgs& a)
{
    uintptr_t places = (uintptr_t)(a.k / (a.mx ? 32 : 16));
    for (int w = 0; w < a.weights; ++w)
        places |= reinterpret_cast<uintptr_t>(a.scales[w]);
    return places % 4 == 0;
}

template <Kind KIND, int NW, int PARTS, bool CONV, int XT = 1>
void few_form(const MatmulArgs& a, const MatmulPlan& p)
{
    const dim3 grid((uint32_t)((a.n + p.rows - 1) / p.rows));
    const bool one = scales_together(a);
    switch (p.waves_k) {
#define FP4Q_FEW(RW, KW)                                                                             \
    if (one)                                                                                         \
        matmul_few<KIND, NW, PARTS, CONV, XT, RW, KW, true><<<grid, 512, p.lds, a.stream>>>(a, p);       \
    else                                                                                             \
        matmul_few<KIND, NW, PARTS, CONV, XT, RW, KW, false><<<grid, 512, p.lds, a.stream>>>(a, p);      \
    break;
    case 2: FP4Q_FEW(4, 2)
    case 4: FP4Q_FEW(2, 4)
    default:
        if constexpr (XT == 1) { // eight steps of more than 16 rows do not fit
            FP4Q_FEW(1, 8)
        }
#undef FP4Q_FEW
    }
}

template <Kind KIND, int NW, int XM, int PARTS>
void many_tiles(const MatmulArgs& a, const MatmulPlan& p)
{
    const uint32_t tiles = (uint32_t)((a.n + p.rows - 1) / p.rows * ((a.m + p.tokens - 1) / p.tokens));
    const dim3 grid(tiles, 1, (uint32_t)p.splits);
    if (scales_together(a))
        matmul_many<KIND, NW, XM, PARTS, true><<<grid, 64 * WN, 0, a.stream>>>(a, p);
    else
        matmul_many<KIND, NW, XM, PARTS, false><<<grid, 64 * WN, 0, a.stream>>>(a, p);
    if (p.splits > 1)
        matmul_join<KIND, NW, XM><<<tiles * (WN * XM * TN / NW), 256, 0, a.stream>>>(a, p);
}

template <Kind KIND, int NW>
hipError_t launch_weights(const MatmulArgs& a, const MatmulPlan& p)
{
    if (p.prepared) {
        const int64_t all = (a.m * (a.k / (KIND == kMx ? 32 : 16)) + 255) / 256;
        const dim3 cover((uint32_t)(all < 1 ? 1 : (all < 65536 ? all : 65536)));
        matmul_parts<KIND><<<cover, 256, 0, a.stream>>>(a);
    }
    if (!p.many) {
        if (p.parts == 1 && p.tokens == 32)
            few_form<KIND, NW, 1, false, 2>(a, p);
        else if (p.parts == 1)
            few_form<KIND, NW, 1, false>(a, p);
        else if (p.prepared)
            few_form<KIND, NW, kParts, false>(a, p);
        else
            few_form<KIND, NW, kParts, true>(a, p);
    } else if (p.tokens == 32) {
        if (p.parts == 1)
            many_tiles<KIND, NW, 1, 1>(a, p);
        else
            many_tiles<KIND, NW, 1, kParts>(a, p);
    } else if (p.tokens == 64) {
        many_tiles<KIND, NW, 2, 1>(a, p);
    } else {
        many_tiles<KIND, NW, 4, 1>(a, p);
    }
    return hipGetLastError();
}

} // namespace
} // namespace fp4q
