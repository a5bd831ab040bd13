// Launchers of window attention on the tensor cores (bf16).
#pragma once

#include "kda_window.cuh"

namespace kda {

cudaError_t launch_window_forward_tc(const WinGeom &geo, const WinArgs &a, cudaStream_t s);
// dq, dk and dv, but for those of sinks that far queries see, whose near and far
// parts win_far_sum_kernel adds up; room for lse2, delta [hq][tokens].
cudaError_t launch_window_backward_tc(const WinGeom &geo, const WinArgs &a, float *lse2, float *delta, float *part,
                                      float *near, Launches &l);
// Reads (and optionally clears) the error word of these kernels' waits.
cudaError_t read_window_error(int *out, bool reset);

}  // namespace kda
