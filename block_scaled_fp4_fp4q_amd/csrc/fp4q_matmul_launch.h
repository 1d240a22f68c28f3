// fp4q_matmul_launch.h -- internal interface between the C ABI of the products
// with 4-bit weights (fp4q_matmul_capi.cpp) and their kernel launchers
// (fp4q_matmul_nv.hip, fp4q_matmul_mx.hip).  Not installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4q {

enum { kActSilu = 0, kActGelu = 1, kActGeluTanh = 2 };

// y [m, n] = x [m, k] W^T of one weight, or act(x W0^T) * (x W1^T) of two
struct MatmulArgs {
    const uint8_t* codes[2];
    const uint8_t* scales[2];
    const float* global[2]; // null for MXFP4
    int weights;            // 1 or 2
    int mx, rotate, act;
    bool bf16;
    bool y_wide; // four values of a row of y can be stored at once
    int64_t n, k, m;
    const void* x;
    int64_t x_row; // in elements
    void* y;
    int64_t y_row;
    void* workspace;
    hipStream_t stream;
};

constexpr int kStepK = 128;   // values of the long axis in one step of a workgroup of many rows
constexpr int kFewStep = 256; // and of a wave of few
constexpr int kCus = 256;

// How one call is cut into workgroups, from its sizes and types alone.
struct MatmulPlan {
    bool many;       // the kernel for many rows of x (else the one for few)
    bool prepared;   // x is taken from the workspace, in parts
    bool refused;    // more workgroups than a launch holds
    int parts;       // bf16 parts of x: 1 or 3
    int rows;        // weight rows of a workgroup
    int tokens;      // rows of x of a workgroup
    int waves_k;     // few: waves that share the long axis
    int chunk_steps; // few: steps whose x is held in LDS at once
    int splits;      // many: workgroups that share a tile's long axis
    int split_steps; // many: steps of each
    size_t lds;      // few
    size_t partials;  // where the partial sums begin
    size_t workspace; // bytes
};

hipError_t launch_matmul_nv(const MatmulArgs& a, const MatmulPlan& p);
hipError_t launch_matmul_mx(const MatmulArgs& a, const MatmulPlan& p);

} // namespace fp4q
