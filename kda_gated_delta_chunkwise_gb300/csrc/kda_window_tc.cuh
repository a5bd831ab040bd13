// Launchers of window attention on the tensor cores (bf16).
#pragma once

#include "kda_window.cuh"

namespace kda {

cudaError_t launch_window_forward_tc(const WinGeom &geo, const WinArgs &a, cudaStream_t s);
// dq, and dk and dv of the near pairs with the far ones' `sums` added (nullable);
// lse2, delta [hq][tokens].
cudaError_t launch_window_backward_tc(const WinGeom &geo, const WinArgs &a, const float *lse2, const float *delta,
                                      const float *sums, cudaStream_t s);
// Reads (and optionally clears) the error word of these kernels' waits.
cudaError_t read_window_error(int *out, bool reset);

}  // namespace kda
