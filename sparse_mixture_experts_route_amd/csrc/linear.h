// Launchers of the dense projection and its gradients (linear.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe_train.h"

namespace moe {

// C [M, N] = A B over K: A [M, K] or (TN) [K, M], B [K, N] or (NT) [N, K]
enum DenseForm { DENSE_NN, DENSE_NT, DENSE_TN };

struct DensePlan {
  int tile;    // 0: 256 x 256, 1: 128 x 128, 2: 32 x 32, K over the waves
  int splits;  // along K
  int m_tiles, n_tiles, nk, grid;
};
DensePlan dense_plan(DenseForm form, int64_t M, int64_t N, int64_t K);
size_t dense_partials_bytes(DenseForm form, int64_t M, int64_t N, int64_t K);
hipError_t launch_dense(DenseForm form, const void* A, const void* B, int64_t M, int64_t N, int64_t K, const void* bias,
                        int act, const void* residual, void* u, void* y, float* partials, hipStream_t s);
// dU = dy act'(u) to `du` (may be null) and the sums of its columns to `dbias` (may be
// null; `sums`: slope_parts(T, N) * N float32)
int64_t slope_parts(int64_t T, int N);
hipError_t launch_slope(const void* dy, const void* u, int act, void* du, void* dbias, float* sums, int64_t T, int N,
                        hipStream_t s);

}  // namespace moe
