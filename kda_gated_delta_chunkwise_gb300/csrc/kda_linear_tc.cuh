// Launchers of the tensor-core steps of linear attention (bf16, d_k = d_v = 128).
#pragma once

#include "kda_linear.cuh"

namespace kda {

constexpr int kLinMaxBlock = 256;  // tokens per block at most (two 128-row tiles, see lin_attend_tc_kernel)

// Every block's own state: out [block][head][128][128] fp32; total and total_rev
// [block][head]: its decay_total as the forward and as the reverse scan use it
// (forward only, nullable).
cudaError_t launch_state_tc(const LinGeom &geo, bool rev, const void *x, int64_t xs, const void *y, int64_t ys,
                            int64_t tokens, const float *log_decay, int decay, float *out, float *total,
                            float *total_rev, Launches &l);
// The scan over the blocks: own states -> three bf16 arrays, part_stride
// elements apart, of the states before (reverse: the gradients after) each
// block; the last state to sT. Reverse: also <S, G> of every block, S in `other`.
cudaError_t launch_scan_tc(const LinGeom &geo, bool rev, const float *own, const float *total,
                           const float *s0, float *sT, float c, void *out, int64_t part_stride, const void *other,
                           float *inner, Launches &l);
constexpr int kScanPartials = 128;  // partial sums of <S, G> per block and head

// out = c_state f x S + c_intra (D o x y^T) z; state_t: S is read transposed.
// With `dot`, S comes in three parts and the row dots with w are written too.
struct AttendTc {
    LinGeom geo;
    bool rev, state_t;
    const void *x, *y, *z, *w;
    int64_t x_stride, y_stride, z_stride, w_stride;
    const void *states;
    int64_t tokens;
    const float *log_decay;
    int decay;
    void *out;
    float c_state, c_intra;
    float *dot, *dot_state;  // [2][tokens][H], the sums of two column halves, nullable
};
cudaError_t launch_attend_tc(const AttendTc &a, Launches &l);
// The same over blocks of any length with the state carried along inside:
// states holds every block's first state (reverse: the gradient after its last
// token) in fp32; c_roll multiplies what the block's tokens add to it.
struct RollTc {
    LinGeom geo;
    bool rev, state_t;
    const void *x, *y, *z;
    int64_t x_stride, y_stride, z_stride;
    const float *states;
    int64_t tokens;
    const float *log_decay;
    int decay;
    void *out;
    float c_state, c_intra, c_roll;
};
cudaError_t launch_roll_tc(const RollTc &a, Launches &l);
// Reads (and optionally clears) the error word of these kernels' waits.
cudaError_t read_linear_error(int *out, bool reset);

}  // namespace kda
