// Launch arguments of the routing and exchange kernels (validated by the C ABI
// layer): which experts a token goes to, the order of its slots (token, j) by
// expert, and the rows' way there and back.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "bounds.cuh"

namespace ql {

constexpr int kRouteMaxExperts = 512;
constexpr int kRouteMaxK = 32;
constexpr int kRouteMaxGroups = 32;

struct RouteArgs {
    const void* logits;
    bool bf16;
    int64_t m, sl;
    int experts;
    const float* bias;         // or null
    int k, groups, kept, group_best;
    bool sigmoid, renormalise;
    float scale;
    float* weights;            // [m][k]
    int32_t* chosen;           // [m][k]
    Bounds bnd;                // logits, bias, weights, chosen
};

struct RouteBackArgs {
    const float* dweights;     // [m][k]
    const void* logits;
    bool bf16;
    int64_t m, sl;
    int experts;
    const int32_t* chosen;     // [m][k]
    int k;
    bool sigmoid, renormalise;
    float scale;
    void* dlogits;             // the logits' type
    int64_t sd;
    Bounds bnd;                // dweights, logits, chosen, dlogits
};

struct PlanArgs {
    const int32_t* chosen;     // [slots]
    int64_t slots;
    int experts;
    int32_t* offsets;          // [experts + 1]
    int32_t* rows;             // [slots]
    int32_t* counts;           // workspace [chunks][experts], or null
    int64_t chunk;             // slots per chunk
    uint32_t* dev_status;
    Bounds bnd;                // chosen, offsets, rows, counts
};

// Rows of x [m][n] to the places that `rows` [m][k] gives, zeros from offsets[experts] on.
struct DispatchArgs {
    const void* x;
    int64_t m, n, sx;          // n, sx in elements
    int es;
    const int32_t* rows;
    const int32_t* offsets;
    int experts, k;
    void* xs;                  // [m * k][n]
    int64_t sxs;
    Bounds bnd;                // x, rows, offsets, xs
};

// y[t] = add[t] + sum_j weights[t][j] ys[rows[t][j]]
struct CombineArgs {
    const void* ys;
    bool bf16;                 // ys, add and y
    int64_t m, n, sys;
    int k;
    const int32_t* rows;
    const float* weights;      // or null: 1
    const void* add;           // or null
    int64_t sadd;
    void* y;
    int64_t sy;
    Bounds bnd;                // ys, rows, weights, add, y
};

// dys[rows[t][j]] = weights[t][j] dy[t] (zeros from offsets[experts] on),
// dweights[t][j] = dy[t] . ys[rows[t][j]]
struct CombineBackArgs {
    const void* dy;
    bool bf16;                 // dy, ys and dys
    int64_t m, n, sdy;
    const void* ys;
    int64_t sys;
    int k;
    const int32_t* rows;
    const int32_t* offsets;
    int experts;
    const float* weights;
    void* dys;
    int64_t sdys;
    float* dweights;
    BoundsOf<7> bnd;           // dy, ys, rows, offsets, weights, dys, dweights
};

int64_t plan_chunk(int64_t slots);
size_t plan_workspace(int64_t slots, int experts);
cudaError_t launch_route(const RouteArgs& a, cudaStream_t st);
cudaError_t launch_route_back(const RouteBackArgs& a, cudaStream_t st);
cudaError_t launch_plan(const PlanArgs& a, cudaStream_t st);
cudaError_t launch_dispatch(const DispatchArgs& a, cudaStream_t st);
cudaError_t launch_combine(const CombineArgs& a, cudaStream_t st, int num_sms);
cudaError_t launch_combine_back(const CombineBackArgs& a, cudaStream_t st, int num_sms);

}  // namespace ql
