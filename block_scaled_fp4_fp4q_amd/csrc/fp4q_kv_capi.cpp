// fp4q_kv_capi.cpp -- the 4-bit KV cache's part of the C ABI (include/fp4q.h).
//
// As in fp4q_capi.cpp, every argument that the host can see is validated
// before anything reaches the HIP runtime.  Slots, lengths and page numbers
// lie on the device and are checked by the kernels.
#include "fp4q.h"

#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>

#include "fp4q_kv_launch.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMostTokenStride = 1 << 20; // 16 rows stay within 32-bit offsets
constexpr int64_t kMostStride = (int64_t)1 << 46;

fp4q_status check_spec(const fp4q_spec* s)
{
    if (!s)
        return FP4Q_E_NULL;
    if (s->format < FP4Q_NVFP4 || s->format > FP4Q_IF6)
        return FP4Q_E_ARG;
    if (s->format != FP4Q_NVFP4 && s->format != FP4Q_MXFP4)
        return FP4Q_E_UNSUPPORTED;
    if (s->block != (s->format == FP4Q_MXFP4 ? 32 : 16))
        return FP4Q_E_UNSUPPORTED;
    if (s->rotate != 0 && s->rotate != s->block)
        return FP4Q_E_ARG;
    return FP4Q_OK;
}

// shapes, strides and pointers of a cache
fp4q_status check_cache(const fp4q_spec* s, const fp4q_kv_cache* c, fp4q::KvView& v)
{
    if (!c)
        return FP4Q_E_NULL;
    if (c->reserved != 0)
        return FP4Q_E_ARG;
    if (c->num_pages < 0 || c->kv_heads < 1 || c->page_size < 1)
        return FP4Q_E_SHAPE;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return FP4Q_E_UNSUPPORTED;
    const int64_t strides[6] = {c->code_page, c->code_head, c->code_token,
                                c->scale_page, c->scale_head, c->scale_token};
    for (int64_t st : strides)
        if (st < 0 || st > kMostStride)
            return FP4Q_E_SHAPE;
    if (c->code_token > kMostTokenStride || c->scale_token > kMostTokenStride)
        return FP4Q_E_SHAPE;
    // a byte offset into a cache fits in 63 bits
    const int64_t far = (c->code_page > c->scale_page ? c->code_page : c->scale_page);
    const int64_t wide = (c->code_head > c->scale_head ? c->code_head : c->scale_head);
    if ((far != 0 && c->num_pages > (INT64_MAX >> 2) / far) || (wide != 0 && c->kv_heads > (INT64_MAX >> 2) / wide))
        return FP4Q_E_SHAPE;
    if (c->num_pages > (INT64_MAX >> 2) / c->page_size)
        return FP4Q_E_SHAPE;
    const bool mx = s->format == FP4Q_MXFP4;
    const uintptr_t sa = mx && c->head_dim == 64 ? 2 : 4;
    if (c->num_pages != 0) {
        if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales)
            return FP4Q_E_NULL;
    }
    if (!mx && (!c->k_global || !c->v_global))
        return FP4Q_E_NULL;
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, sa) ||
        !aligned(c->v_scales, sa) || (!mx && (!aligned(c->k_global, 4) || !aligned(c->v_global, 4))))
        return FP4Q_E_ALIGN;
    for (int i = 0; i < 6; ++i)
        if (strides[i] % (int64_t)(i < 3 ? 16 : sa) != 0)
            return FP4Q_E_ALIGN;
    v.codes[0] = c->k_codes;
    v.codes[1] = c->v_codes;
    v.scales[0] = c->k_scales;
    v.scales[1] = c->v_scales;
    v.global[0] = mx ? nullptr : c->k_global;
    v.global[1] = mx ? nullptr : c->v_global;
    v.num_pages = c->num_pages;
    v.heads = c->kv_heads;
    v.page_size = c->page_size;
    v.head_dim = c->head_dim;
    v.mx = mx;
    v.c_page = c->code_page;
    v.c_head = c->code_head;
    v.c_token = c->code_token;
    v.s_page = c->scale_page;
    v.s_head = c->scale_head;
    v.s_token = c->scale_token;
    return FP4Q_OK;
}

bool valid_dtype(int32_t d) { return d == FP4Q_F32 || d == FP4Q_BF16; }

// rows of head_dim values: 16-byte aligned base, strides in elements
bool rows_aligned(const void* p, int64_t stride1, int64_t stride2, int32_t dtype)
{
    const int64_t step = dtype == FP4Q_BF16 ? 8 : 4;
    return aligned(p, 16) && stride1 % step == 0 && stride2 % step == 0;
}

bool stride_ok(int64_t s) { return s >= 0 && s <= kMostStride; }

// Whether rows of `row` units, counts[i] of them strides[i] apart in each of N
// dimensions, share no unit: in order of their strides, each dimension steps
// past all that the ones before it cover (every view of a tensor does whose
// elements are its own).  Counts and strides are such that extents fit 63 bits.
template <int N>
bool rows_apart(const int64_t (&counts)[N], const int64_t (&strides)[N], int64_t row)
{
    int64_t covered = row;
    bool used[N] = {};
    for (int turn = 0; turn < N; ++turn) {
        int next = -1;
        for (int i = 0; i < N; ++i) {
            if (counts[i] == 0)
                return true;
            if (!used[i] && (next < 0 || strides[i] < strides[next] ||
                             (strides[i] == strides[next] && counts[i] < counts[next])))
                next = i;
        }
        used[next] = true;
        if (counts[next] == 1)
            continue;
        if (strides[next] < covered)
            return false;
        covered += (counts[next] - 1) * strides[next];
    }
    return true;
}

fp4q_status check_attend(const fp4q_spec* spec, const fp4q_kv_cache* cache,
                         const fp4q_attention* c, fp4q::AttendArgs& a)
{
    fp4q_status st = check_spec(spec);
    if (st != FP4Q_OK)
        return st;
    if ((st = check_cache(spec, cache, a.kv)) != FP4Q_OK)
        return st;
    if (!c)
        return FP4Q_E_NULL;
    if (!valid_dtype(c->dtype) || (c->causal != 0 && c->causal != 1) || c->window < 0 ||
        (c->window != 0 && !c->causal) || c->reserved != 0 || !std::isfinite(c->scale))
        return FP4Q_E_ARG;
    if (c->batch < 0 || c->total_q < 0 || c->max_q < 0 || c->max_kv < 0 || c->q_heads < 1 ||
        c->q_heads % cache->kv_heads != 0 || c->table_len < 0 || c->table_stride < 0)
        return FP4Q_E_SHAPE;
    if (!stride_ok(c->q_row_stride) || !stride_ok(c->q_head_stride) ||
        !stride_ok(c->out_row_stride) || !stride_ok(c->out_head_stride))
        return FP4Q_E_SHAPE;
    const int64_t most = c->q_row_stride > c->out_row_stride ? c->q_row_stride : c->out_row_stride;
    const int64_t wide = c->q_head_stride > c->out_head_stride ? c->q_head_stride : c->out_head_stride;
    if ((most != 0 && c->total_q > (INT64_MAX >> 4) / most) || (wide != 0 && c->q_heads > (INT64_MAX >> 4) / wide))
        return FP4Q_E_SHAPE;
    if (c->total_q > (INT64_MAX >> 4) / c->q_heads)
        return FP4Q_E_SHAPE;
    // grids and row numbers within a sequence stay in 31 bits
    const int group = c->q_heads / cache->kv_heads;
    if ((int64_t)c->max_q * group > INT_MAX - 1024 || c->max_kv > INT_MAX - 8192 ||
        c->window > INT_MAX - 8192 || c->max_q > INT_MAX - 8192)
        return FP4Q_E_SHAPE;
    if (!c->q_starts && (int64_t)c->batch * c->max_q != c->total_q)
        return FP4Q_E_SHAPE;
    if (c->block_table && cache->page_size % 16 != 0)
        return FP4Q_E_UNSUPPORTED;
    if (c->batch > 1 && c->block_table && c->table_stride < c->table_len)
        return FP4Q_E_SHAPE;
    const bool empty = c->total_q == 0 || c->batch == 0 || c->max_q == 0;
    if (!empty && (!c->q || !c->out || !c->kv_lens))
        return FP4Q_E_NULL;
    if (!rows_aligned(c->q, c->q_row_stride, c->q_head_stride, c->dtype) ||
        !rows_aligned(c->out, c->out_row_stride, c->out_head_stride, c->dtype) ||
        !aligned(c->lse, 4) || !aligned(c->q_starts, 4) || !aligned(c->kv_lens, 4) ||
        !aligned(c->block_table, 4))
        return FP4Q_E_ALIGN;
    if (!empty && !rows_apart<2>({c->total_q, c->q_heads}, {c->out_row_stride, c->out_head_stride}, cache->head_dim))
        return FP4Q_E_SHAPE;
    a.rotate = spec->rotate;
    a.bf16 = c->dtype == FP4Q_BF16;
    a.causal = c->causal != 0;
    a.batch = empty ? 0 : c->batch;
    a.max_q = c->max_q;
    a.max_kv = c->max_kv;
    a.q_heads = c->q_heads;
    a.group = group;
    a.window = c->window;
    a.total_q = c->total_q;
    a.scale = c->scale;
    a.q = c->q;
    a.q_row = c->q_row_stride;
    a.q_head = c->q_head_stride;
    a.out = c->out;
    a.o_row = c->out_row_stride;
    a.o_head = c->out_head_stride;
    a.lse = c->lse;
    a.q_starts = c->q_starts;
    a.kv_lens = c->kv_lens;
    a.table = c->block_table;
    a.table_stride = c->table_stride;
    a.table_len = c->table_len;
    return FP4Q_OK;
}

} // namespace

extern "C" {

fp4q_status fp4q_kv_write(const fp4q_spec* spec, const fp4q_kv_cache* cache, const void* k,
                          const void* v, int32_t dtype, int64_t tokens, int64_t k_token_stride,
                          int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                          const int64_t* slots, void* stream)
{
    fp4q::KvWriteArgs a{};
    fp4q_status st = check_spec(spec);
    if (st != FP4Q_OK)
        return st;
    if (spec->scale_rule != FP4Q_SCALE_ABSMAX && spec->scale_rule != FP4Q_SCALE_SWEEP &&
        spec->scale_rule != FP4Q_SCALE_FOUR_OVER_SIX)
        return FP4Q_E_ARG;
    if (spec->objective != FP4Q_OBJ_MSE && spec->objective != FP4Q_OBJ_WMSE)
        return FP4Q_E_ARG;
    if (spec->objective != FP4Q_OBJ_MSE ||
        (spec->scale_rule == FP4Q_SCALE_FOUR_OVER_SIX && spec->format != FP4Q_NVFP4))
        return FP4Q_E_UNSUPPORTED;
    if (spec->format == FP4Q_NVFP4 && spec->global_scale_given != 1)
        return FP4Q_E_ARG;
    if (spec->scale_rule == FP4Q_SCALE_SWEEP &&
        (spec->sweep_lo > spec->sweep_hi || spec->sweep_lo < -126 || spec->sweep_hi > 126))
        return FP4Q_E_ARG;
    if ((st = check_cache(spec, cache, a.kv)) != FP4Q_OK)
        return st;
    if (!valid_dtype(dtype))
        return FP4Q_E_ARG;
    if (tokens < 0 || !stride_ok(k_token_stride) || !stride_ok(k_head_stride) ||
        !stride_ok(v_token_stride) || !stride_ok(v_head_stride))
        return FP4Q_E_SHAPE;
    const int64_t most = k_token_stride > v_token_stride ? k_token_stride : v_token_stride;
    const int64_t wide = k_head_stride > v_head_stride ? k_head_stride : v_head_stride;
    if ((most != 0 && tokens > (INT64_MAX >> 4) / most) || (wide != 0 && cache->kv_heads > (INT64_MAX >> 4) / wide) ||
        tokens > (INT64_MAX >> 4) / ((int64_t)cache->kv_heads * cache->head_dim))
        return FP4Q_E_SHAPE;
    if (tokens != 0 && (!k || !v || !slots))
        return FP4Q_E_NULL;
    if (!rows_aligned(k, k_token_stride, k_head_stride, dtype) ||
        !rows_aligned(v, v_token_stride, v_head_stride, dtype) || !aligned(slots, 8))
        return FP4Q_E_ALIGN;
    // rows that share bytes would be written at once
    const int64_t counts[3] = {cache->num_pages, cache->kv_heads, cache->page_size};
    if (!rows_apart<3>(counts, {cache->code_page, cache->code_head, cache->code_token}, cache->head_dim / 2) ||
        !rows_apart<3>(counts, {cache->scale_page, cache->scale_head, cache->scale_token},
                       cache->head_dim / spec->block) ||
        (cache->num_pages != 0 && (cache->k_codes == cache->v_codes || cache->k_scales == cache->v_scales)))
        return FP4Q_E_SHAPE;
    if (tokens == 0)
        return FP4Q_OK;
    a.rule = spec->scale_rule;
    a.lo = spec->sweep_lo;
    a.hi = spec->sweep_hi;
    a.rotate = spec->rotate;
    a.bf16 = dtype == FP4Q_BF16;
    a.x[0] = k;
    a.x[1] = v;
    a.x_token[0] = k_token_stride;
    a.x_token[1] = v_token_stride;
    a.x_head[0] = k_head_stride;
    a.x_head[1] = v_head_stride;
    a.slots = slots;
    a.tokens = tokens;
    a.stream = static_cast<hipStream_t>(stream);
    return fp4q::launch_kv_write(a) == hipSuccess ? FP4Q_OK : FP4Q_E_HIP;
}

fp4q_status fp4q_kv_read(const fp4q_spec* spec, const fp4q_kv_cache* cache, const int64_t* slots,
                         int64_t tokens, void* k, void* v, int32_t dtype, void* stream)
{
    fp4q::KvReadArgs a{};
    fp4q_status st = check_spec(spec);
    if (st != FP4Q_OK)
        return st;
    if ((st = check_cache(spec, cache, a.kv)) != FP4Q_OK)
        return st;
    if (!valid_dtype(dtype))
        return FP4Q_E_ARG;
    if (tokens < 0 || tokens > (INT64_MAX >> 4) / ((int64_t)cache->kv_heads * cache->head_dim))
        return FP4Q_E_SHAPE;
    if (tokens != 0 && (!k || !v || !slots))
        return FP4Q_E_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8))
        return FP4Q_E_ALIGN;
    if (tokens == 0)
        return FP4Q_OK;
    a.rotate = spec->rotate;
    a.bf16 = dtype == FP4Q_BF16;
    a.slots = slots;
    a.tokens = tokens;
    a.y[0] = k;
    a.y[1] = v;
    a.stream = static_cast<hipStream_t>(stream);
    return fp4q::launch_kv_read(a) == hipSuccess ? FP4Q_OK : FP4Q_E_HIP;
}

size_t fp4q_attend_workspace_bytes(const fp4q_spec* spec, const fp4q_kv_cache* cache,
                                   const fp4q_attention* call)
{
    fp4q::AttendArgs a{};
    if (check_attend(spec, cache, call, a) != FP4Q_OK || a.batch == 0)
        return 0;
    return fp4q::plan_attend(a).workspace;
}

fp4q_status fp4q_attend(const fp4q_spec* spec, const fp4q_kv_cache* cache,
                        const fp4q_attention* call, void* workspace, size_t ws_bytes, void* stream)
{
    fp4q::AttendArgs a{};
    const fp4q_status st = check_attend(spec, cache, call, a);
    if (st != FP4Q_OK)
        return st;
    if (a.batch == 0)
        return FP4Q_OK;
    const fp4q::AttendPlan p = fp4q::plan_attend(a);
    if (p.groups == 0)
        return FP4Q_E_SHAPE; // more workgroups than a launch holds
    if (p.workspace != 0) {
        if (!workspace)
            return FP4Q_E_NULL;
        if (ws_bytes < p.workspace)
            return FP4Q_E_ARG;
        if (!aligned(workspace, 256))
            return FP4Q_E_ALIGN;
    }
    a.workspace = workspace;
    a.stream = static_cast<hipStream_t>(stream);
    return fp4q::launch_attend(a, p) == hipSuccess ? FP4Q_OK : FP4Q_E_HIP;
}

} // extern "C"
