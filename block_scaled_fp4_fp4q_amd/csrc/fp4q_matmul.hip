// fp4q_matmul.hip -- products of activations with 4-bit weights.
//
//   y_mn = S sum_k x_mk v_nk s_n(k)        (v a code's value, s its block's scale)
//
// and, of two weights, act(x W0^T) * (x W1^T).  A code times its E4M3 scale has
// at most six significant bits and a code times 2^e two, so dequantized weights
// enter the matrix cores exactly as bf16, and so does x of bf16; the global scale
// is one binary32 factor of the sum.  A weight that is stored rotated is never
// rotated back: x W^T = (x H)(W H)^T with H the orthonormal block Hadamard, so x is
// rotated, in binary32.
//
// Parts.  Where x is not exact in bf16 it is given as a sum of bf16 parts, one
// matrix product each: binary32 in three, which hold its 24 bits; rotated bf16 in
// two, 16 bits, 2^8 finer than the rounding of a bf16 result.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "fp4q_device.h"
#include "fp4q_matmul_launch.h"

namespace fp4q {

namespace {

typedef __bf16 b16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mfma16(u32x4 x, u32x4 y, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b16x8, x), __builtin_bit_cast(b16x8, y), c, 0, 0, 0);
}

// ---- weights -------------------------------------------------------------------

// Two codes of a word times their block's scale s, as bf16: the product has six
// bits, so cutting binary32 to its upper half loses nothing.
template <int SEL>
__device__ __forceinline__ uint32_t nv_pair(uint32_t w, float s)
{
    float a, b;
    fp4_unpack2<SEL>(w, a, b);
    return __builtin_amdgcn_perm(__float_as_uint(b * s), __float_as_uint(a * s), 0x07060302u);
}

template <int SEL>
__device__ __forceinline__ uint32_t mx_pair(uint32_t w, float step)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, step, SEL));
}

// the eight codes of a word; s is the value of an E4M3 byte, or a power of two
template <bool MX>
__device__ __forceinline__ u32x4 expand(uint32_t w, float s)
{
    if constexpr (MX)
        return u32x4{mx_pair<0>(w, s), mx_pair<1>(w, s), mx_pair<2>(w, s), mx_pair<3>(w, s)};
    else
        return u32x4{nv_pair<0>(w, s), nv_pair<1>(w, s), nv_pair<2>(w, s), nv_pair<3>(w, s)};
}

// a lane's scales of 32 values: two E4M3 bytes, or one E8M0 byte whose exponent
// the conversions apply (255 stands for NaN)
struct Scales {
    float lo, hi;
};

// as loaded; the two of NVFP4 are put together where they are used, so that nothing
// waits for them before
template <bool MX>
struct Bytes {
    uint32_t b[MX ? 1 : 2];
};

template <bool MX>
__device__ __forceinline__ Scales scales_of(const Bytes<MX>& s)
{
    if constexpr (MX) {
        const float x = __uint_as_float(s.b[0] << 23);
        return Scales{x, x};
    } else {
        const auto t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(s.b[0] | (s.b[1] << 8), 1.0f, false);
        return Scales{t[0], t[1]};
    }
}

// Raw buffer resource over `bytes` bytes from p (uniform): a load past the end
// gives zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const uint8_t* p, int bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, __builtin_amdgcn_readfirstlane(bytes), 0x00027000);
}

// OR-ed to an offset, past every buffer's end (a select would become a branch
// around the load)
constexpr int kPast = 0x7FFFFFFF;

// the scale bytes of 32 values of a row from value k on, as scales_of takes them;
// `past` as above.  NVFP4: of two blocks; a row may end after the first, and the
// second's scale is then zero.
template <bool MX>
__device__ __forceinline__ Bytes<MX> load_scales(__amdgpu_buffer_rsrc_t scales, int at, int k, int cols, int past)
{
    Bytes<MX> r;
    r.b[0] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(scales, at | past, 0, 0);
    if constexpr (!MX)
        r.b[1] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(scales, (at + 1) | (k + 16 < cols ? past : kPast), 0, 0);
    return r;
}

// ---- activations ------------------------------------------------------------------

// x as a sum of PARTS bf16 values, their bits in the upper halves of h: cut, the
// remainder cut again, and for the last part rounded to nearest even (with three
// parts it is exact).  A value that is not finite is its first part alone.
template <int PARTS>
__device__ __forceinline__ void parts_of(float x, uint32_t* h)
{
    if constexpr (PARTS == 1) {
        h[0] = f32_to_bf16(x) << 16;
    } else {
        const bool finite = __builtin_fabsf(x) < __builtin_huge_valf();
        h[0] = finite ? __float_as_uint(x) & 0xFFFF0000u : f32_to_bf16(x) << 16;
        float rest = finite ? x - __uint_as_float(h[0]) : 0.0f;
        if constexpr (PARTS == 3) {
            h[1] = __float_as_uint(rest) & 0xFFFF0000u;
            rest -= __uint_as_float(h[1]);
        }
        h[PARTS - 1] = f32_to_bf16(rest) << 16;
    }
}

// the N values of x from element `at` on, widened
template <int N, bool BF16>
__device__ __forceinline__ void load_x(const void* x, int64_t at, float* v)
{
    load_block<N, BF16, false>(static_cast<const char*>(x) + at * (BF16 ? 2 : 4), 0, v);
}

// ---- results --------------------------------------------------------------------------

__device__ __forceinline__ float activation(int act, float g)
{
    if (act == kActSilu)
        return g / (1.0f + expf(-g));
    if (act == kActGelu)
        return 0.5f * g * (1.0f + erff(g * 0.70710678118654752f));
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
template <bool MX, int NW>
__device__ __forceinline__ f32x4 finish4(const MatmulArgs& a, const f32x4* sum)
{
    f32x4 r = sum[0];
    if constexpr (!MX)
        r *= *a.global[0];
    if constexpr (NW == 2) {
        f32x4 u = sum[1];
        if constexpr (!MX)
            u *= *a.global[1];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = activation(a.act, r[i]) * u[i];
    }
    return r;
}

// partial sums of split s: [weight][m][n, padded to four]
__device__ __forceinline__ f32x4* partial_of(const MatmulArgs& a, const MatmulPlan& p, int s, int w, int64_t m, int64_t n)
{
    const int64_t wide = (a.n + 3) & ~(int64_t)3;
    float* sums = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + p.partials);
    return reinterpret_cast<f32x4*>(sums + (((int64_t)s * a.weights + w) * a.m + m) * wide + n);
}

// ---- few rows of x ------------------------------------------------------------------
//
// A workgroup of RW x KW waves takes 16 RT RW rows of the weight and up to
// 16 MT rows of x; RW waves share the rows, KW the long axis, 128 values
// a step.  W is the first operand of 16x16x32 products: lane n + 16 g loads the
// 16 bytes of row n that hold values 32 g .. 32 g + 31 of a step, whole
// blocks, and gives them to four products, eight at a time; x comes from LDS,
// where it was put, rotated and in parts, by the whole workgroup.  The codes of
// the next AHEAD steps are on their way while a step is computed.
constexpr int kAhead = 4;

template <bool MX, int RT>
struct Codes {
    u32x4 c[RT];
    Bytes<MX> s[RT];
};

template <bool MX, int NW, int PARTS, int RT, int RW, int KW, int MT>
__global__ __launch_bounds__(64 * RW * KW) void matmul_few(const MatmulArgs a, const MatmulPlan p)
{
    constexpr int B = MX ? 32 : 16;
    constexpr int T = 64 * RW * KW;
    constexpr int ROWS = 16 * RT; // of a wave
    extern __shared__ u32x4 lds[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int r = lane & 15, g = lane >> 4;
    const int rw = wave % RW, kw = wave / RW;
    const int64_t n0 = (int64_t)blockIdx.x * p.rows, m0 = (int64_t)blockIdx.y * p.tokens;
    const int split = blockIdx.z;
    const int64_t m_left = a.m - m0;
    const int mt = (int)(m_left < 16 * MT ? m_left : 16 * MT);
    const int steps = (int)((a.k + kStepK - 1) / kStepK);
    const int s0 = split * p.split_steps;
    const int s1 = s0 + p.split_steps < steps ? s0 + p.split_steps : steps;

    // this wave's rows of each weight, from its first one on
    const int64_t nw = n0 + rw * ROWS;
    const int64_t left = a.n - nw;
    const int live = left <= 0 ? 0 : (int)(left < ROWS ? left : ROWS);
    const int crow = (int)(a.k / 2), srow = (int)(a.k / B);
    __amdgpu_buffer_rsrc_t codes[NW], scales[NW];
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const int64_t first = live > 0 ? nw : 0;
        codes[w] = buffer_of(a.codes[w] + first * crow, live * crow);
        scales[w] = buffer_of(a.scales[w] + first * srow, live * srow);
    }
    auto load = [&](int step, Codes<MX, RT * NW>& t) {
        const int k = step * kStepK + 32 * g;
        const int past = step < s1 && k < (int)a.k ? 0 : kPast;
#pragma unroll
        for (int w = 0; w < NW; ++w)
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const int row = 16 * i + r;
                t.c[w * RT + i] = __builtin_amdgcn_raw_buffer_load_b128(codes[w], (row * crow + k / 2) | past, 0, 0);
                t.s[w * RT + i] = load_scales<MX>(scales[w], row * srow + k / B, k, (int)a.k, past);
            }
    };

    Codes<MX, RT * NW> ring[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        load(s0 + kw + KW * i, ring[i]);

    // x of chunk_steps steps from step `from` on: [part][row][value], rows padded
    // by 16 bytes so that 16 rows meet all banks
    const int stride = p.chunk_steps * (kStepK / 8) + 1;
    auto fill = [&](int from) {
        const int per = p.chunk_steps * (kStepK / B); // blocks of a row
        for (int u = threadIdx.x; u < mt * per; u += T) {
            const int row = u / per, b = u - row * per;
            const int64_t k = (int64_t)from * kStepK + b * B;
            u32x4* to = lds + row * stride + b * (B / 8);
            if (k >= a.k) {
#pragma unroll
                for (int q = 0; q < PARTS; ++q)
#pragma unroll
                    for (int i = 0; i < B / 8; ++i)
                        to[q * mt * stride + i] = u32x4{0u, 0u, 0u, 0u};
                continue;
            }
            const int64_t at = (m0 + row) * a.x_row + k;
            if constexpr (PARTS == 1) { // bf16, as it is
                const u32x4* x = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.x) + at);
#pragma unroll
                for (int i = 0; i < B / 8; ++i)
                    to[i] = x[i];
            } else {
                float v[B];
                if constexpr (PARTS == 2)
                    load_x<B, true>(a.x, at, v);
                else
                    load_x<B, false>(a.x, at, v);
                if (PARTS == 2 || a.rotate)
                    fwht<B>(v);
#pragma unroll
                for (int i = 0; i < B / 8; ++i) {
                    uint32_t h[8][PARTS];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        parts_of<PARTS>(v[8 * i + j], h[j]);
#pragma unroll
                    for (int q = 0; q < PARTS; ++q)
                        to[q * mt * stride + i] =
                            u32x4{h[0][q] >> 16 | h[1][q], h[2][q] >> 16 | h[3][q], h[4][q] >> 16 | h[5][q], h[6][q] >> 16 | h[7][q]};
                }
            }
        }
    };

    f32x4 acc[RT * NW][MT];
#pragma unroll
    for (int i = 0; i < RT * NW; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
            acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    int x_row[MT]; // places of this lane's rows of x; those past the last repeat it
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        const int row = 16 * j + r;
        x_row[j] = (row < mt ? row : mt - 1) * stride + 4 * g;
    }

    const int turns = p.chunk_steps / KW; // of this wave in a chunk
    const int all = (s1 - s0 + KW - 1) / KW; // the same for every wave of the workgroup
    int in_chunk = turns;
    for (int base = 0; base < all; base += kAhead) {
#pragma unroll
        for (int d = 0; d < kAhead; ++d) {
            const int i = base + d;
            if (i >= all)
                break;
            if (in_chunk == turns) {
                if (i != 0)
                    __syncthreads();
                fill(s0 + i * KW);
                __syncthreads();
                in_chunk = 0;
            }
            const u32x4* x = lds + (in_chunk * KW + kw) * (kStepK / 8);
            Codes<MX, RT * NW>& t = ring[d];
            Scales sc[RT * NW];
#pragma unroll
            for (int w = 0; w < RT * NW; ++w)
                sc[w] = scales_of<MX>(t.s[w]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                u32x4 xv[MT][PARTS];
#pragma unroll
                for (int y = 0; y < MT; ++y)
#pragma unroll
                    for (int q = 0; q < PARTS; ++q)
                        xv[y][q] = x[x_row[y] + q * mt * stride + j];
#pragma unroll
                for (int w = 0; w < RT * NW; ++w) {
                    const u32x4 wv = expand<MX>(t.c[w][j], j < 2 ? sc[w].lo : sc[w].hi);
#pragma unroll
                    for (int y = 0; y < MT; ++y)
#pragma unroll
                        for (int q = PARTS - 1; q >= 0; --q) // small parts first
                            acc[w][y] = mfma16(wv, xv[y][q], acc[w][y]);
                }
            }
            load(s0 + kw + KW * (i + kAhead), t);
            ++in_chunk;
        }
    }

    // join the waves that share rows, in order
    __syncthreads();
    f32x4* red = reinterpret_cast<f32x4*>(lds);
#pragma unroll
    for (int w = 0; w < RT * NW; ++w)
#pragma unroll
        for (int y = 0; y < MT; ++y)
            red[((wave * RT * NW + w) * MT + y) * 64 + lane] = acc[w][y];
    __syncthreads();
    for (int u = threadIdx.x; u < RW * RT * MT * 64; u += T) {
        const int l = u & 63;
        int rest = u >> 6;
        const int y = rest % MT;
        rest /= MT;
        const int i = rest % RT, part = rest / RT;
        const int64_t n = n0 + part * ROWS + 16 * i + 4 * (l >> 4), m = m0 + 16 * y + (l & 15);
        if (n >= a.n || m >= a.m)
            continue;
        f32x4 sum[NW];
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            sum[w] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < KW; ++k)
                sum[w] += red[(((k * RW + part) * RT * NW + w * RT + i) * MT + y) * 64 + l];
        }
        if (p.splits == 1) {
            store4(a, m, n, finish4<MX, NW>(a, sum));
        } else {
#pragma unroll
            for (int w = 0; w < NW; ++w)
                *partial_of(a, p, split, w, m, n) = sum[w];
        }
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
// last ones' are those of the next step.
typedef __attribute__((address_space(3))) void lds_void;
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16 mfma32(u32x4 x, u32x4 y, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b16x8, x), __builtin_bit_cast(b16x8, y), c, 0, 0, 0);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of_x(const void* p, int64_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, __builtin_amdgcn_readfirstlane((int)bytes), 0x00027000);
}

// 64 values of a row of the weight: codes, and scale bytes as they came: in ONE load, or
// each in one of its own, put together where they are used, so that nothing waits for
// them before.
template <bool MX, bool ONE>
struct Wide {
    static constexpr int NS = ONE ? 1 : (MX ? 2 : 4);
    u32x4 c[2];
    uint32_t s[NS];
};

template <bool MX, bool ONE>
__device__ __forceinline__ uint32_t scale_word(const Wide<MX, ONE>& w)
{
    if constexpr (ONE)
        return w.s[0];
    else if constexpr (MX)
        return w.s[0] | (w.s[1] << 8);
    else
        return w.s[0] | (w.s[1] << 8) | (w.s[2] << 16) | (w.s[3] << 24);
}

// the factor of values 8 j .. 8 j + 7 of 64
template <bool MX>
__device__ __forceinline__ float factor_of(uint32_t word, int j)
{
    if constexpr (MX)
        return __uint_as_float((j < 4 ? word & 0xFFu : word >> 8) << 23);
    const auto t = j < 4 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(word, 1.0f, false)
                         : __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(word, 1.0f, true);
    return t[(j >> 1) & 1];
}

template <bool MX, int NW, int TM, int WN, bool ONE>
__global__ __launch_bounds__(64 * WN, 2) void matmul_many(const MatmulArgs a, const MatmulPlan p)
{
    constexpr int B = MX ? 32 : 16;
    constexpr int BM = 32 * TM;
    constexpr int BN = 64 * WN / NW; // columns of y
    constexpr int WC = 64 / NW;      // of a wave
    constexpr int U = kStepK / 8;    // 16-byte units of a row of x
    __shared__ u32x4 xbuf[2][BM * U];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int n = lane & 31, h = lane >> 5;

    // workgroups of one XCD (every eighth) take neighbouring tiles: kGroup rows of tiles at a
    // time, the rows of tiles fastest
    const uint32_t tiles_m = (uint32_t)((a.m + BM - 1) / BM), tiles_n = (uint32_t)((a.n + BN - 1) / BN);
    const uint32_t all = tiles_m * tiles_n;
    uint32_t id = blockIdx.x;
    {
        const uint32_t xcd = id % 8, per = all / 8, more = all % 8;
        id = xcd * per + (xcd < more ? xcd : more) + id / 8;
    }
    constexpr uint32_t kGroup = 8;
    const uint32_t band = id / (kGroup * tiles_n), first = band * kGroup;
    const uint32_t high = tiles_m - first < kGroup ? tiles_m - first : kGroup;
    const uint32_t in = id - band * kGroup * tiles_n;
    const int64_t m0 = (int64_t)(first + in % high) * BM, n0 = (int64_t)(in / high) * BN;

    const int cols = (int)a.k;
    const int steps = (cols + kStepK - 1) / kStepK;
    const int s0 = (int)blockIdx.z * p.split_steps;
    const int s1 = s0 + p.split_steps < steps ? s0 + p.split_steps : steps;
    const int turns = (s1 - s0) * p.parts; // a step for each part of x, the small ones first
    // Offsets are a lane's own (in a vector register) and a uniform part that never passes
    // the buffer's end, where the check against it would wrap: rows of a tile that do not
    // exist are replaced by others, whose results are not stored.

    // x, or its parts: plane q, row m
    const int64_t m_left = a.m - m0;
    const int rows = (int)(m_left < BM ? m_left : BM);
    const int x_row = (int)(p.parts == 1 ? a.x_row : a.k) * 2; // bytes
    const char* x = (p.parts == 1 ? static_cast<const char*>(a.x) : static_cast<const char*>(a.workspace)) + m0 * x_row;
    const int64_t plane = a.m * a.k * 2;
    constexpr int LOADS = BM / (4 * WN); // of a wave: four rows each
    static_assert(LOADS % 4 == 0, "the exchange of units repeats every four loads");
    const int quad = lane >> 4; // row of the four
    int x_unit[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x_unit[i] = (lane & 15) ^ (4 * i + quad);
    auto load_x_tile = [&](int step, int part, int to) {
        const auto src = buffer_of_x(x + part * plane, (int64_t)(rows - 1) * x_row + cols * 2);
        const bool whole = (step + 1) * kStepK <= cols;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int row = (wave * LOADS + i) * 4;
            int at = quad * x_row + x_unit[i % 4] * 16;
            if (!whole) // values past the row's end are zeros
                at |= step * kStepK + x_unit[i % 4] * 8 < cols ? 0 : kPast;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (lds_void*)(&xbuf[to][(wave * LOADS + i) * 64]), 16, at,
                                                     __builtin_amdgcn_readfirstlane((row < rows ? row : 0) * x_row + step * (kStepK * 2)), 0, 0);
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
    const int w_row = 16 * ((n >> 2) & 1) + 4 * (n >> 3) + (n & 3);
    const int c_at = w_row * crow + 32 * h, s_at = w_row * srow + 64 * h / B;
    constexpr int SB = 64 / B; // scale bytes of 64 values
    auto load_w = [&](int step, Wide<MX, ONE> (&t)[2]) {
        const int k = step * kStepK + 64 * h;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int w = NW == 2 ? i : 0, row = NW == 2 ? 0 : 32 * i, up = row < live ? row : 0;
#pragma unroll
            for (int c = 0; c < 2; ++c) // past the row's end: any codes, with scales of zero
                t[i].c[c] = __builtin_amdgcn_raw_buffer_load_b128(codes[w], (c_at + 16 * c) | (k + 32 * c < cols ? 0 : kPast),
                                                                  __builtin_amdgcn_readfirstlane(up * crow + step * (kStepK / 2)), 0);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int w = NW == 2 ? i : 0, row = NW == 2 ? 0 : 32 * i, up = row < live ? row : 0;
            const int to = __builtin_amdgcn_readfirstlane(up * srow + step * (kStepK / B));
            if constexpr (ONE) {
                const int past = k < cols ? 0 : kPast;
                t[i].s[0] = MX ? (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(scales[w], s_at | past, to, 0)
                               : __builtin_amdgcn_raw_buffer_load_b32(scales[w], s_at | past, to, 0);
            } else {
#pragma unroll
                for (int q = 0; q < SB; ++q)
                    t[i].s[q] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(scales[w], (s_at + q) | (k + q * B < cols ? 0 : kPast), to, 0);
            }
        }
    };

    f32x16 acc[TM][2];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                acc[i][j][e] = 0.0f;

    Wide<MX, ONE> now[2], next[2];
    u32x4 wv[2][2];
    uint32_t word[2];
    auto expand_tile = [&](const Wide<MX, ONE>& from_w, int j, int i) {
        if (j == 0)
            word[i] = scale_word<MX, ONE>(from_w);
        wv[j & 1][i] = expand<MX>(from_w.c[j >> 2][j & 3], factor_of<MX>(word[i], j));
    };
    int step = s0, part = p.parts - 1; // of the next loads
    auto advance = [&]() {
        if (part == 0) {
            part = p.parts;
            ++step;
        }
        --part;
    };
    if (turns > 0) {
        load_w(step, now);
        load_x_tile(step, part, 0);
        advance();
        expand_tile(now[0], 0, 0);
        expand_tile(now[1], 0, 1);
    }
    for (int turn = 0; turn < turns; ++turn) {
        const int at = turn & 1;
        __builtin_amdgcn_s_waitcnt(0x0F70); // vmcnt(0): this wave's part of the step's x has arrived
        __syncthreads();                    // everybody's has, and the other buffer is free
        if (turn + 1 < turns) {
            load_w(step, next);
            load_x_tile(step, part, at ^ 1);
            advance();
        }
        auto read_x = [&](int i) { // the i-th of the step's reads
            const int row = 32 * (i % TM) + n;
            return xbuf[at][row * U + ((8 * h + i / TM) ^ (n & 15))];
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
                // the order of these is kept: a read for later, a part of the expansion, the products
                __builtin_amdgcn_sched_barrier(0);
                const u32x4 mine = xv[x_turn % kReadAhead];
                if (x_turn + kReadAhead < 8 * TM)
                    xv[x_turn % kReadAhead] = read_x(x_turn + kReadAhead);
                if (i == 0 || i == TM / 2)
                    expand_tile(j < 7 ? now[i != 0] : next[i != 0], (j + 1) & 7, i != 0);
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    acc[i][t] = mfma32(wv[j & 1][t], mine, acc[i][t]);
            }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            now[i] = next[i];
    }

#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int64_t m = m0 + 32 * i + n;
        if (m >= a.m)
            continue;
#pragma unroll
        for (int t = 0; t < 2 / NW; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t col = nw + 32 * t + 16 * h + 4 * q;
                if (col >= a.n)
                    continue;
                f32x4 sum[NW];
#pragma unroll
                for (int w = 0; w < NW; ++w)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sum[w][e] = acc[i][NW == 2 ? w : t][4 * q + e];
                if (p.splits == 1) {
                    store4(a, m, col, finish4<MX, NW>(a, sum));
                } else {
#pragma unroll
                    for (int w = 0; w < NW; ++w)
                        *partial_of(a, p, (int)blockIdx.z, w, m, col) = sum[w];
                }
            }
    }
}

// the parts of x, rotated: [part][m][k] bf16 in the workspace, a block of values a thread
template <int B, int PARTS>
__global__ __launch_bounds__(256) void matmul_parts(const MatmulArgs a)
{
    const int64_t blocks = a.k / B, all = a.m * blocks, plane = a.m * a.k;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < all; u += (int64_t)gridDim.x * 256) {
        const int64_t row = u / blocks, b = u - row * blocks;
        float v[B];
        load_x<B, PARTS == 2>(a.x, row * a.x_row + b * B, v);
        if (PARTS == 2 || a.rotate)
            fwht<B>(v);
        uint16_t* to = static_cast<uint16_t*>(a.workspace) + u * B;
#pragma unroll
        for (int i = 0; i < B / 8; ++i) {
            uint32_t h[8][PARTS];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                parts_of<PARTS>(v[8 * i + j], h[j]);
#pragma unroll
            for (int q = 0; q < PARTS; ++q)
                *reinterpret_cast<u32x4*>(to + q * plane + 8 * i) =
                    u32x4{h[0][q] >> 16 | h[1][q], h[2][q] >> 16 | h[3][q], h[4][q] >> 16 | h[5][q], h[6][q] >> 16 | h[7][q]};
        }
    }
}

// the sums of all splits, in order, and the results
template <bool MX, int NW>
__global__ __launch_bounds__(256) void matmul_join(const MatmulArgs a, const MatmulPlan p)
{
    const int64_t n = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, m = (int64_t)blockIdx.z * 65535 + blockIdx.y;
    if (n >= a.n || m >= a.m)
        return;
    f32x4 sum[NW];
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        sum[w] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int s = 0; s < p.splits; ++s)
            sum[w] += *partial_of(a, p, s, w, m, n);
    }
    store4(a, m, n, finish4<MX, NW>(a, sum));
}

enum { kFew1 = 0, kFew16 = 1, kFew32 = 2, kFew64 = 3, kMany = 4 };

int parts_for(const MatmulArgs& a) { return !a.bf16 ? 3 : (a.rotate ? 2 : 1); }

template <bool MX, int NW, int PARTS>
void launch_few(const MatmulArgs& a, const MatmulPlan& p, dim3 grid)
{
    switch (p.form) {
    case kFew1: matmul_few<MX, NW, PARTS, 1, 1, 8, 1><<<grid, 512, p.lds, a.stream>>>(a, p); break;
    case kFew16: matmul_few<MX, NW, PARTS, 2, 1, 8, 1><<<grid, 512, p.lds, a.stream>>>(a, p); break;
    case kFew32: matmul_few<MX, NW, PARTS, 1, 4, 2, 2><<<grid, 512, p.lds, a.stream>>>(a, p); break;
    default:
        if constexpr (PARTS < 3)
            matmul_few<MX, NW, PARTS, 1, 4, 2, 4><<<grid, 512, p.lds, a.stream>>>(a, p);
        break;
    }
}

template <bool MX, int NW>
hipError_t launch_weights(const MatmulArgs& a, const MatmulPlan& p)
{
    const uint32_t tiles_n = (uint32_t)((a.n + p.rows - 1) / p.rows), tiles_m = (uint32_t)((a.m + p.tokens - 1) / p.tokens);
    if (p.form == kMany) {
        if (p.parts > 1) {
            constexpr int B = MX ? 32 : 16;
            const int64_t all = (a.m * (a.k / B) + 255) / 256;
            const dim3 cover((uint32_t)(all < 65536 ? all : 65536));
            if (p.parts == 2)
                matmul_parts<B, 2><<<cover, 256, 0, a.stream>>>(a);
            else
                matmul_parts<B, 3><<<cover, 256, 0, a.stream>>>(a);
        }
        const dim3 grid(tiles_n * tiles_m, 1, (uint32_t)p.splits);
        // the scale bytes of 64 values in one load, where every row's begin so that they can be
        uintptr_t places = (uintptr_t)(a.k / (MX ? 32 : 16));
        for (int w = 0; w < NW; ++w)
            places |= reinterpret_cast<uintptr_t>(a.scales[w]);
        if (places % (MX ? 2 : 4) == 0)
            matmul_many<MX, NW, 4, 4, true><<<grid, 256, 0, a.stream>>>(a, p);
        else
            matmul_many<MX, NW, 4, 4, false><<<grid, 256, 0, a.stream>>>(a, p);
    } else {
        const dim3 grid(tiles_n, tiles_m, (uint32_t)p.splits);
        switch (p.parts) {
        case 1: launch_few<MX, NW, 1>(a, p, grid); break;
        case 2: launch_few<MX, NW, 2>(a, p, grid); break;
        default: launch_few<MX, NW, 3>(a, p, grid); break;
        }
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1)
        return e;
    const dim3 cover((uint32_t)((a.n + 1023) / 1024), (uint32_t)(a.m < 65535 ? a.m : 65535), (uint32_t)((a.m + 65534) / 65535));
    matmul_join<MX, NW><<<cover, 256, 0, a.stream>>>(a, p);
    return hipGetLastError();
}

} // namespace

MatmulPlan plan_matmul(const MatmulArgs& a)
{
    MatmulPlan p{};
    const int parts = p.parts = parts_for(a);
    const int64_t steps = (a.k + kStepK - 1) / kStepK;
    p.splits = 1;
    p.split_steps = (int)steps;
    if (a.m > 64 && a.k < ((int64_t)1 << 22) && a.x_row < ((int64_t)1 << 22)) {
        p.form = kMany;
        p.rows = 256 / a.weights;
        p.tokens = 128;
        p.partials = parts == 1 ? 0 : (size_t)parts * a.m * a.k * 2;
        p.partials = (p.partials + 255) & ~(size_t)255;
        p.workspace = p.partials;
        const int64_t tiles_n = (a.n + p.rows - 1) / p.rows, tiles_m = (a.m + p.tokens - 1) / p.tokens;
        p.refused = tiles_n > 0x7FFFFF / tiles_m;
        return p;
    }
    int kw, rt, mt, rw;
    if (a.m <= 4) {
        p.form = kFew1, rt = 1, rw = 1, kw = 8, mt = 1;
    } else if (a.m <= 16) {
        p.form = kFew16, rt = 2, rw = 1, kw = 8, mt = 1;
    } else if (a.m <= 32 || parts == 3) {
        p.form = kFew32, rt = 1, rw = 4, kw = 2, mt = 2;
    } else {
        p.form = kFew64, rt = 1, rw = 4, kw = 2, mt = 4;
    }
    p.rows = 16 * rt * rw;
    p.tokens = 16 * mt;
    const int rows = (int)(a.m < p.tokens ? a.m : p.tokens);
    const int whole = (int)(steps + kw - 1) / kw * kw; // steps, filled up to the waves' number
    p.chunk_steps = whole;
    while (p.chunk_steps > kw && (size_t)rows * parts * (p.chunk_steps * 256 + 16) > 56 * 1024)
        p.chunk_steps = (p.chunk_steps / 2 + kw - 1) / kw * kw;
    const size_t x = (size_t)rows * parts * (p.chunk_steps * 256 + 16);
    const size_t red = (size_t)rw * kw * rt * a.weights * mt * 1024;
    p.lds = x > red ? x : red;
    const int64_t tiles_n = (a.n + p.rows - 1) / p.rows, tiles_m = (a.m + p.tokens - 1) / p.tokens;
    p.refused = tiles_n > 0x7FFFFF || tiles_m > 65535;
    return p;
}

hipError_t launch_matmul(const MatmulArgs& a, const MatmulPlan& p)
{
    if (a.mx)
        return a.weights == 2 ? launch_weights<true, 2>(a, p) : launch_weights<true, 1>(a, p);
    return a.weights == 2 ? launch_weights<false, 2>(a, p) : launch_weights<false, 1>(a, p);
}

} // namespace fp4q
