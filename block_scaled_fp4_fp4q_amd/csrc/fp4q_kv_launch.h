// fp4q_kv_launch.h -- internal interface between the C ABI of the 4-bit KV
// cache (fp4q_kv_capi.cpp) and its kernel launchers (fp4q_kv.hip,
// fp4q_attend.hip).  Not installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4q {

// one cache, as the kernels see it; strides in bytes
struct KvView {
    uint8_t* codes[2];  // K, V
    uint8_t* scales[2];
    const float* global[2];
    int64_t num_pages;
    int heads, page_size, head_dim, mx; // mx: MXFP4 (else NVFP4)
    int64_t c_page, c_head, c_token;
    int64_t s_page, s_head, s_token;
};

struct KvWriteArgs {
    KvView kv;
    int rule, lo, hi, rotate;
    bool bf16;
    const void* x[2];
    int64_t x_token[2], x_head[2]; // strides in elements
    const int64_t* slots;
    int64_t tokens;
    hipStream_t stream;
};

struct KvReadArgs {
    KvView kv;
    int rotate;
    bool bf16;
    const int64_t* slots;
    int64_t tokens;
    void* y[2]; // [tokens, heads, head_dim]
    hipStream_t stream;
};

struct AttendArgs {
    KvView kv;
    int rotate;
    bool bf16, causal;
    int batch, max_q, max_kv, q_heads, group, window;
    int64_t total_q;
    float scale;
    const void* q;
    int64_t q_row, q_head; // strides in elements
    void* out;
    int64_t o_row, o_head;
    float* lse; // [total_q, q_heads] or null
    const int32_t* q_starts; // [batch + 1] or null
    const int32_t* kv_lens;  // [batch]
    const int32_t* table;    // [batch, table_len] or null
    int64_t table_stride;
    int table_len;
    void* workspace;
    hipStream_t stream;
};

// How one attention call is cut into workgroups, from its sizes alone.
struct AttendPlan {
    bool many;         // the kernel for many queries (else the one for few)
    int rows_per_tile; // query rows of one workgroup
    int tiles;         // row tiles per sequence and KV head
    int groups;        // workgroups (0: more than a launch holds)
    int parts;         // few: workgroups that run at once (0: one workgroup per pair)
    int chunk;         // many: keys of one workgroup
    int chunks;        // many: key chunks per row tile; few: 2 where there are partial results
    size_t workspace;  // bytes of partial results (0 where chunks == 1)
};

// keys that one row tile can see at most, counted from the 32-key boundary
// at or below its first visible key
inline int64_t attend_span(const AttendArgs& a)
{
    const int64_t all = (int64_t)a.max_kv;
    if (a.window == 0)
        return all;
    const int64_t most = (int64_t)a.window + a.max_q - 1 + 31;
    return most < all ? most : all;
}

AttendPlan plan_attend(const AttendArgs& a);

hipError_t launch_kv_write(const KvWriteArgs& a);
hipError_t launch_kv_read(const KvReadArgs& a);
hipError_t launch_attend(const AttendArgs& a, const AttendPlan& p);

} // namespace fp4q
