// fp4q_matmul_capi.cpp -- the products with 4-bit weights of the C ABI
// (include/fp4q.h).  Every argument is validated on the host before anything
// reaches the HIP runtime.
#include "fp4q.h"

#include <hip/hip_runtime.h>

#include <climits>

#include "fp4q_matmul_launch.h"
#include "fp4q_matmul_plan.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMostCols = (int64_t)1 << 22; // 128 rows stay within 32-bit offsets
constexpr int64_t kMostRows = (int64_t)1 << 36; // and a weight within 63 bits
constexpr int64_t kMostStride = (int64_t)1 << 46;
constexpr int64_t kMostRowStride = (int64_t)1 << 22; // of x

// Whether a row of x and one of y share a byte: `rows` of each, strides and widths in bytes.
bool share(uintptr_t x, int64_t x_step, int64_t x_wide, uintptr_t y, int64_t y_step, int64_t y_wide, int64_t rows)
{
    const int64_t apart = (int64_t)(y - x); // of the first rows
    if (apart >= (rows - 1) * x_step + x_wide || -apart >= (rows - 1) * y_step + y_wide)
        return false;
    if (x_step == y_step && x_step >= x_wide && x_step >= y_wide) { // as two columns of one array
        const int64_t at = ((apart % x_step) + x_step) % x_step;
        return at < x_wide || at + y_wide > x_step;
    }
    for (int64_t i = 0; i < rows; ++i) {
        const int64_t at = apart + i * y_step; // of y's row, from x's first one
        if (at + y_wide <= 0)
            continue;
        int64_t row = x_step == 0 ? 0 : (at + y_wide - 1) / x_step; // the last one that begins before its end
        row = row < rows ? row : rows - 1;
        if (row * x_step + x_wide > at)
            return true;
    }
    return false;
}

fp4q_status check_weight(const fp4q_spec* s, const fp4q_weight* w)
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
    if (!w)
        return FP4Q_E_NULL;
    if (w->rows < 0 || w->cols < 0 || w->cols % s->block != 0 || w->cols > kMostCols || w->rows > kMostRows)
        return FP4Q_E_SHAPE;
    const bool mx = s->format == FP4Q_MXFP4;
    if (w->rows != 0 && ((w->cols != 0 && (!w->codes || !w->scales)) || (!mx && !w->global_scale)))
        return FP4Q_E_NULL;
    if (!aligned(w->codes, mx ? 16 : 8) || (!mx && !aligned(w->global_scale, 4)))
        return FP4Q_E_ALIGN;
    return FP4Q_OK;
}

fp4q_status check_sizes(const fp4q_spec* s, const fp4q_weight* w, int64_t tokens, int32_t dtype, fp4q::MatmulArgs& a)
{
    if (dtype != FP4Q_F32 && dtype != FP4Q_BF16)
        return FP4Q_E_ARG;
    if (tokens < 0 || tokens > INT_MAX)
        return FP4Q_E_SHAPE;
    a.mx = s->format == FP4Q_MXFP4;
    a.rotate = s->rotate;
    a.bf16 = dtype == FP4Q_BF16;
    a.n = w->rows;
    a.k = w->cols;
    a.m = tokens;
    return FP4Q_OK;
}

size_t workspace_bytes(const fp4q_spec* spec, const fp4q_weight* w, int weights, int64_t tokens, int32_t dtype)
{
    fp4q::MatmulArgs a{};
    a.weights = weights;
    if (check_weight(spec, w) != FP4Q_OK || check_sizes(spec, w, tokens, dtype, a) != FP4Q_OK || a.n == 0 || a.m == 0)
        return 0;
    const fp4q::MatmulPlan p = fp4q::plan_of(a);
    return p.refused ? 0 : p.workspace;
}

fp4q_status run(const fp4q_spec* spec, const fp4q_weight* const* w, int weights, int32_t act, const void* x, int32_t dtype,
                int64_t tokens, int64_t x_stride, void* y, int64_t y_stride, void* workspace, size_t ws_bytes, void* stream)
{
    fp4q::MatmulArgs a{};
    a.weights = weights;
    a.act = act;
    fp4q_status st;
    for (int i = 0; i < weights; ++i)
        if ((st = check_weight(spec, w[i])) != FP4Q_OK)
            return st;
    if (weights == 2 && (w[0]->rows != w[1]->rows || w[0]->cols != w[1]->cols))
        return FP4Q_E_SHAPE;
    if ((st = check_sizes(spec, w[0], tokens, dtype, a)) != FP4Q_OK)
        return st;
    if (x_stride < 0 || x_stride > kMostRowStride || y_stride < 0 || y_stride > kMostStride ||
        (x_stride != 0 && tokens > (INT64_MAX >> 4) / x_stride) || (y_stride != 0 && tokens > (INT64_MAX >> 4) / y_stride))
        return FP4Q_E_SHAPE;
    if (tokens > 1 && y_stride < a.n)
        return FP4Q_E_SHAPE; // rows of y would share elements
    if (a.n != 0 && a.m != 0 && (!y || (a.k != 0 && !x)))
        return FP4Q_E_NULL;
    const int64_t step = a.bf16 ? 8 : 4;
    if (!aligned(x, 16) || x_stride % step != 0 || !aligned(y, a.bf16 ? 2 : 4))
        return FP4Q_E_ALIGN;
    if (a.n == 0 || a.m == 0)
        return FP4Q_OK;
    const int64_t size = a.bf16 ? 2 : 4;
    if (a.k != 0 && share((uintptr_t)x, x_stride * size, a.k * size, (uintptr_t)y, y_stride * size, a.n * size, a.m))
        return FP4Q_E_SHAPE; // x would be overwritten while it is read
    for (int i = 0; i < weights; ++i) {
        a.codes[i] = w[i]->codes;
        a.scales[i] = w[i]->scales;
        a.global[i] = a.mx ? nullptr : w[i]->global_scale;
    }
    a.x = x;
    a.x_row = x_stride;
    a.y = y;
    a.y_row = y_stride;
    a.y_wide = aligned(y, a.bf16 ? 8 : 16) && y_stride % 4 == 0;
    a.stream = static_cast<hipStream_t>(stream);
    const fp4q::MatmulPlan p = fp4q::plan_of(a);
    if (p.refused)
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
    return (a.mx ? fp4q::launch_matmul_mx(a, p) : fp4q::launch_matmul_nv(a, p)) == hipSuccess ? FP4Q_OK : FP4Q_E_HIP;
}

} // namespace

extern "C" {

size_t fp4q_matmul_workspace_bytes(const fp4q_spec* spec, const fp4q_weight* w, int64_t tokens, int32_t dtype)
{
    return workspace_bytes(spec, w, 1, tokens, dtype);
}

fp4q_status fp4q_matmul(const fp4q_spec* spec, const fp4q_weight* w, const void* x, int32_t dtype, int64_t tokens,
                        int64_t x_stride, void* y, int64_t y_stride, void* workspace, size_t ws_bytes, void* stream)
{
    return run(spec, &w, 1, 0, x, dtype, tokens, x_stride, y, y_stride, workspace, ws_bytes, stream);
}

size_t fp4q_gated_workspace_bytes(const fp4q_spec* spec, const fp4q_weight* gate, int64_t tokens, int32_t dtype)
{
    return workspace_bytes(spec, gate, 2, tokens, dtype);
}

fp4q_status fp4q_gated(const fp4q_spec* spec, const fp4q_weight* gate, const fp4q_weight* up, int32_t activation,
                       const void* x, int32_t dtype, int64_t tokens, int64_t x_stride, void* y, int64_t y_stride,
                       void* workspace, size_t ws_bytes, void* stream)
{
    if (activation != FP4Q_ACT_SILU && activation != FP4Q_ACT_GELU && activation != FP4Q_ACT_GELU_TANH)
        return FP4Q_E_ARG;
    const fp4q_weight* w[2] = {gate, up};
    return run(spec, w, 2, activation, x, dtype, tokens, x_stride, y, y_stride, workspace, ws_bytes, stream);
}

} // extern "C"
