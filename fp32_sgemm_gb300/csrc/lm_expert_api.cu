// C ABI of routing by expert (declared in include/sgemm_gb300_lm.h): argument
// checks and launches.
#include "lm_expert.h"
#include "lm_host.h"

namespace {

using namespace sg::host;

sgemmStatus_t status(cudaError_t e) { return e == cudaSuccess ? SGEMM_STATUS_SUCCESS : SGEMM_STATUS_LAUNCH_FAILED; }

sgemmStatus_t check_route(int type, int64_t T, int64_t E, int64_t k, const void *logits, int64_t ldl) {
    if (!type_ok(type) || T < 0 || E < 1 || k < 1 || k > E) return SGEMM_STATUS_INVALID_VALUE;
    if (E > sg::kRouteMaxExperts || k > sg::kRouteMaxK || T > kMaxDim / k) return SGEMM_STATUS_NOT_SUPPORTED;
    return check_matrix(logits, T, E, ldl, type, T > 0);
}

// T tokens of D elements, k choices of each.
sgemmStatus_t check_rows(int type, int64_t T, int64_t D, int64_t k) {
    if (!type_ok(type) || T < 0 || D < 0 || k < 0) return SGEMM_STATUS_INVALID_VALUE;
    if (T > kMaxDim || D > kMaxDim || k > kMaxDim || T * k > kMaxDim) return SGEMM_STATUS_NOT_SUPPORTED;
    return SGEMM_STATUS_SUCCESS;
}

}  // namespace

extern "C" {

sgemmStatus_t sgemmRouteTopK(sgemmHandle_t h, sgemmDataType_t type, int64_t T, int64_t E, int64_t k, int normalize,
                             const void *logits, int64_t ldl, float *weights, int64_t *experts, cudaStream_t stream) {
    sgemmStatus_t st = check_route(type, T, E, k, logits, ldl);
    if (st != SGEMM_STATUS_SUCCESS || T == 0) return st;
    if ((st = check_vector(weights, 4)) != SGEMM_STATUS_SUCCESS || (st = check_vector(experts, 8)) != SGEMM_STATUS_SUCCESS)
        return st;
    if (h == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    if ((st = check_device(h)) != SGEMM_STATUS_SUCCESS) return st;
    sg::RouteArgs p{};
    p.logits = logits;
    p.ldl = ldl;
    p.T = int(T);
    p.E = int(E);
    p.k = int(k);
    p.normalize = normalize != 0;
    p.weights = weights;
    p.experts = experts;
    return status(sg::route_launch(type, false, p, stream));
}

sgemmStatus_t sgemmRouteTopKGrad(sgemmHandle_t h, sgemmDataType_t type, int64_t T, int64_t E, int64_t k, int normalize,
                                 const void *logits, int64_t ldl, const int64_t *experts, const float *dweights,
                                 void *dlogits, int64_t ldd, cudaStream_t stream) {
    sgemmStatus_t st = check_route(type, T, E, k, logits, ldl);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    if ((st = check_matrix(dlogits, T, E, ldd, type, T > 0)) != SGEMM_STATUS_SUCCESS || T == 0) return st;
    if ((st = check_vector(experts, 8)) != SGEMM_STATUS_SUCCESS || (st = check_vector(dweights, 4)) != SGEMM_STATUS_SUCCESS)
        return st;
    if (h == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    if ((st = check_device(h)) != SGEMM_STATUS_SUCCESS) return st;
    sg::RouteArgs p{};
    p.logits = logits;
    p.ldl = ldl;
    p.T = int(T);
    p.E = int(E);
    p.k = int(k);
    p.normalize = normalize != 0;
    p.chosen = experts;
    p.dweights = dweights;
    p.dlogits = dlogits;
    p.ldd = ldd;
    return status(sg::route_launch(type, true, p, stream));
}

sgemmStatus_t sgemmExpertDispatch(sgemmHandle_t h, sgemmDataType_t type, int64_t T, int64_t D, int64_t k, int64_t G,
                                  const void *X, int64_t ldx, const int64_t *experts, void *rows, int64_t ldr,
                                  int32_t *slots, int32_t *groupEnds, cudaStream_t stream) {
    sgemmStatus_t st = check_rows(type, T, D, k);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    if (G < 0) return SGEMM_STATUS_INVALID_VALUE;
    if (G > SGEMM_MAX_GROUPS) return SGEMM_STATUS_NOT_SUPPORTED;
    const bool any = T * k > 0;
    if ((st = check_matrix(X, T, D, ldx, type, any && D > 0)) != SGEMM_STATUS_SUCCESS ||
        (st = check_matrix(rows, T * k, D, ldr, type, any && D > 0)) != SGEMM_STATUS_SUCCESS ||
        (any && (st = check_vector(experts, 8)) != SGEMM_STATUS_SUCCESS) ||
        (any && (st = check_vector(slots, 4)) != SGEMM_STATUS_SUCCESS) ||
        (G > 0 && (st = check_vector(groupEnds, 4)) != SGEMM_STATUS_SUCCESS))
        return st;
    if (!any && G == 0) return SGEMM_STATUS_SUCCESS;
    if (h == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    if ((st = check_device(h)) != SGEMM_STATUS_SUCCESS) return st;
    sg::ExpertRows p{};
    p.T = T;
    p.k = int(k);
    p.D = D;
    p.elem = type_size(type);
    p.x = X;
    p.ldx = ldx * p.elem;
    p.slots = slots;
    p.out = rows;
    p.ldo = ldr * p.elem;
    return status(sg::expert_dispatch_launch(p, experts, int(G), slots, groupEnds, stream));
}

sgemmStatus_t sgemmExpertCombine(sgemmHandle_t h, sgemmDataType_t type, int64_t T, int64_t D, int64_t k,
                                 const void *rows, int64_t ldr, const int32_t *slots, const float *weights, void *Y,
                                 int64_t ldy, cudaStream_t stream) {
    sgemmStatus_t st = check_rows(type, T, D, k);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    const bool any = T > 0 && D > 0, used = any && k > 0;
    if ((st = check_matrix(rows, T * k, D, ldr, type, used)) != SGEMM_STATUS_SUCCESS ||
        (st = check_matrix(Y, T, D, ldy, type, any)) != SGEMM_STATUS_SUCCESS ||
        (used && (st = check_vector(slots, 4)) != SGEMM_STATUS_SUCCESS))
        return st;
    if (weights != nullptr && !aligned(weights, 4)) return SGEMM_STATUS_MISALIGNED;
    if (!any) return SGEMM_STATUS_SUCCESS;
    if (h == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    if ((st = check_device(h)) != SGEMM_STATUS_SUCCESS) return st;
    sg::ExpertRows p{};
    p.T = T;
    p.k = int(k);
    p.D = D;
    p.elem = type_size(type);
    p.x = rows;
    p.ldx = ldr * p.elem;
    p.slots = slots;
    p.weights = weights;
    p.out = Y;
    p.ldo = ldy * p.elem;
    return status(sg::expert_combine_launch(type, p, stream));
}

sgemmStatus_t sgemmExpertCombineGradEx(sgemmHandle_t h, sgemmDataType_t type, int64_t T, int64_t D, int64_t k,
                                       const void *dY, int64_t lddy, const void *rows, int64_t ldr,
                                       const int32_t *slots, const float *weights, void *dRows, int64_t lddr,
                                       float *dWeights, int32_t *owners, cudaStream_t stream) {
    sgemmStatus_t st = check_rows(type, T, D, k);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    const bool any = T * k > 0, used = any && D > 0;
    if ((st = check_matrix(dY, T, D, lddy, type, used)) != SGEMM_STATUS_SUCCESS ||
        ((rows != nullptr || dWeights != nullptr) &&
         (st = check_matrix(rows, T * k, D, ldr, type, used && dWeights != nullptr)) != SGEMM_STATUS_SUCCESS) ||
        (dRows != nullptr && (st = check_matrix(dRows, T * k, D, lddr, type, used)) != SGEMM_STATUS_SUCCESS) ||
        (any && (st = check_vector(slots, 4)) != SGEMM_STATUS_SUCCESS))
        return st;
    if (!aligned(weights, 4) || !aligned(dWeights, 4) || !aligned(owners, 4)) return SGEMM_STATUS_MISALIGNED;
    if (!any || (dWeights == nullptr && (dRows == nullptr || D == 0))) return SGEMM_STATUS_SUCCESS;
    if (h == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    if ((st = check_device(h)) != SGEMM_STATUS_SUCCESS) return st;
    sg::ExpertRows p{};
    p.T = T;
    p.k = int(k);
    p.D = D;
    p.elem = type_size(type);
    p.x = dY;
    p.ldx = lddy * p.elem;
    p.slots = slots;
    p.weights = weights;
    p.out = D > 0 ? dRows : nullptr;
    p.ldo = lddr * p.elem;
    p.rows = rows;
    p.ldr = ldr * p.elem;
    p.dweights = dWeights;
    p.owner = owners;
    return status(sg::expert_combine_grad_launch(type, p, stream));
}

sgemmStatus_t sgemmExpertCombineGrad(sgemmHandle_t h, sgemmDataType_t type, int64_t T, int64_t D, int64_t k,
                                     const void *dY, int64_t lddy, const void *rows, int64_t ldr, const int32_t *slots,
                                     const float *weights, void *dRows, int64_t lddr, float *dWeights,
                                     cudaStream_t stream) {
    return sgemmExpertCombineGradEx(h, type, T, D, k, dY, lddy, rows, ldr, slots, weights, dRows, lddr, dWeights,
                                    nullptr, stream);
}

}  // extern "C"
