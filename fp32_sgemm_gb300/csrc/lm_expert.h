// Kernels of routing by expert: the router's choice, rows sorted by expert and
// back (lm_route.cu, lm_expert.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace sg {

constexpr int kRouteMaxExperts = 1024, kRouteMaxK = 32;

struct RouteArgs {
    const void *logits;
    int64_t ldl;
    int T, E, k;
    int normalize;
    float *weights;             // [T][k]
    int64_t *experts;           // [T][k]
    const int64_t *chosen;      // gradient: [T][k]
    const float *dweights;      // gradient: [T][k]
    void *dlogits;
    int64_t ldd;
};
// type: sgemmDataType_t.
cudaError_t route_launch(int type, bool grad, const RouteArgs &p, cudaStream_t s);

// Rows; pitches in bytes.
struct ExpertRows {
    int64_t T;
    int k;
    int64_t D, elem;            // elements of a row, bytes of one
    const void *x;              // dispatch: tokens; combine: rows; gradient: dy
    int64_t ldx;                // bytes
    const int32_t *slots;       // [T][k]
    const float *weights;       // [T][k] or NULL
    void *out;                  // dispatch: rows; combine: tokens; gradient: drows or NULL
    int64_t ldo;                // bytes
    const void *rows;           // gradient: rows, or NULL if dweights is not wanted
    int64_t ldr;                // bytes
    float *dweights;            // gradient: [T][k] or NULL
    int32_t *owner;             // gradient: [T k] for the choice that names each row, or NULL
};
// Writes slots (p.slots) and ends[G] as well.
cudaError_t expert_dispatch_launch(const ExpertRows &p, const int64_t *experts, int G, int32_t *slots, int32_t *ends,
                                   cudaStream_t s);
cudaError_t expert_combine_launch(int type, const ExpertRows &p, cudaStream_t s);
cudaError_t expert_combine_grad_launch(int type, const ExpertRows &p, cudaStream_t s);

}  // namespace sg
