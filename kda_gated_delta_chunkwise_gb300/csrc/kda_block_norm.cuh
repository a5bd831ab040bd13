// The norms around a block: of every head with a gate, behind a recurrence or
// an attention, and of the residual stream, behind the block.
#pragma once

#include "kda_internal.cuh"
#include "kda_linear.cuh"

namespace kda {

// Blocks of the backwards' persistent grids at most: two of 256 threads (gated),
// one of 512 (residual) on each of the 152 SMs.
constexpr int kGatedBwdBlocks = 152 * 2;
constexpr int kResidualBwdBlocks = 152;
constexpr int kResidualMaxWidth = 8192;

struct GatedArgs {
    kda_dtype_t dt;
    const void *x, *gate, *dy;   // token strides in elements, heads contiguous; dy contiguous
    int64_t x_stride, g_stride;
    const float *w;              // [d], nullable
    void *y, *dx, *dgate;        // contiguous
    float *dw, *partial;         // backward: [d], nullable together
    int norm, act, h, d;
    int64_t tokens;
    float eps;
    FastDiv by_heads;
};
cudaError_t launch_gated_norm(const GatedArgs &p, bool back, cudaStream_t s);

struct ResidualArgs {
    kda_dtype_t stream_dt, dt;   // of the residual stream, of the branch and the output
    const void *x, *b;           // residual (backward: the stored sum), branch
    const void *dy, *dh;         // backward; dh nullable
    const float *w, *wb, *c;     // [D], nullable
    void *h, *y;                 // h may be x, y may be b
    void *dx, *db;               // backward
    float *dw, *dwb, *dc;        // backward: [D], nullable
    float *partial;              // [blocks][3][D], null when none of them is wanted
    int branch_norm, D;
    int64_t tokens;
    float scale, eps;
};
cudaError_t launch_residual_norm(const ResidualArgs &p, bool back, cudaStream_t s);
cudaError_t read_block_error(int *out, bool reset);

}  // namespace kda
