// Launch arguments of the layer norm kernels (validated by the C ABI layer).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "bounds.cuh"

namespace ql {

struct NormArgs {
    const void* x;
    bool x_bf16;
    int64_t m, n, sx;          // rows contiguous, row stride sx
    const void *w, *b;         // or null
    bool w_bf16;
    float eps;
    void* y;
    bool y_bf16;
    int64_t sy;
    float *mean, *rstd;        // or null
    Bounds bnd;                // x, w, b, y, mean, rstd
};

// dx, and the sums over the rows of dy * h and of dy (null: none)
struct NormBackArgs {
    const void* dy;
    bool dy_bf16;
    int64_t sdy;
    const void* x;
    bool x_bf16;
    int64_t m, n, sx;
    const float *mean, *rstd;
    const void* w;             // or null
    bool w_bf16;
    void* dx;                  // x's type
    int64_t sdx;
    float *dw, *db;            // [n], or both null
    float* part;               // workspace: sums of some rows each, [parts][2][n]
    BoundsOf<9> bnd;           // dy, x, mean, rstd, w, dx, workspace, dw, db
};

size_t norm_back_workspace(int64_t m, int64_t n);
cudaError_t launch_norm(const NormArgs& a, cudaStream_t st, int num_sms);
cudaError_t launch_norm_back(const NormBackArgs& a, cudaStream_t st, int num_sms);

}  // namespace ql
