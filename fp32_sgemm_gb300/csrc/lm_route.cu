// The router's choice and its gradient.  With p = softmax(l) over a token's E
// logits, the k largest are chosen, the lower index among equals:
//
//   w_j = p[e_j]                      (normalize: divided by the sum of the chosen p)
//   dl_e = p_e ([e chosen] g_e - sum_j p[e_j] g_j)    (normalize: of the chosen alone,
//                                                      with w in the place of p)
//
// One warp a token, the logits in registers (element lane + 32 i), read once: the
// choice takes k rounds of "the largest key, then the lowest index that has
// it" (two warp reductions of integers each), on the bits of the logits made to
// grow with their values.  Sums are FP32, in an order that E alone decides.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "../../include/sgemm_gb300_lm.h"
#include "lm_expert.h"
#include "lm_launch.cuh"
#include "lm_ptx.cuh"

namespace sg {
namespace {

constexpr int kThreads = 256;

template <class T> __device__ __forceinline__ float load_f(const T *p) { return (float)*p; }
template <class T> __device__ __forceinline__ T to_type(float x) { return (T)x; }
template <> __device__ __forceinline__ __half to_type<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 to_type<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Grows with x; both zeros alike, NaN above all, -inf the least that is not 0.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t u = x == 0.f ? 0u : __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, d));
    return v;
}

template <class T, int V>
__global__ void __launch_bounds__(kThreads)
lm_route_kernel(const RouteArgs p) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = blockIdx.x * (int64_t)(kThreads / 32) + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const T *row = static_cast<const T *>(p.logits) + t * p.ldl;
    float l[V];
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 32 * i;
        l[i] = e < p.E ? load_f(row + e) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = lane + 32 * i < p.E ? order_key(l[i]) : 0u;
    // Lane j holds choice j.
    float mine = -INFINITY;
    int expert = -1;
    for (int j = 0; j < p.k; ++j) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint32_t top = __reduce_max_sync(~0u, best);
        if (top <= order_key(-INFINITY)) break;               // masked, or none left
        const uint32_t e = __reduce_min_sync(~0u, best == top ? (uint32_t)(lane + 32 * at) : ~0u);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if ((uint32_t)(lane + 32 * i) == e) key[i] = 0u;
        if (lane == j) {
            expert = (int)e;
            mine = __uint_as_float(top & 0x80000000u ? top & 0x7FFFFFFFu : ~top);
        }
    }
    const float most = __shfl_sync(~0u, mine, 0);
    // (No choice at all: weights of 0.  A NaN, chosen first, makes all NaN.)
    const float ref = most == -INFINITY ? 0.f : most;
    const float power = expert < 0 ? 0.f : expf(mine - ref);
    float sum;
    if (p.normalize) {
        sum = warp_sum(lane < p.k ? power : 0.f);
    } else {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 32 * i < p.E) sum += expf(l[i] - ref);
        sum = warp_sum(sum);
    }
    if (lane < p.k) {
        p.weights[t * p.k + lane] = expert < 0 ? 0.f : power / sum;
        p.experts[t * p.k + lane] = expert;
    }
}

template <class T, int V>
__global__ void __launch_bounds__(kThreads)
lm_route_grad_kernel(const RouteArgs p) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = blockIdx.x * (int64_t)(kThreads / 32) + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const T *row = static_cast<const T *>(p.logits) + t * p.ldl;
    // Lane j holds choice j.
    int expert = -1;
    float g = 0.f, logit = -INFINITY;
    if (lane < p.k) {
        const int64_t e = p.chosen[t * p.k + lane];
        if (e >= 0 && e < p.E) {
            expert = (int)e;
            g = p.dweights[t * p.k + lane];
            logit = load_f(row + e);
        }
    }
    float l[V];
    float most = logit, sum;
    if (!p.normalize) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            l[i] = e < p.E ? load_f(row + e) : -INFINITY;
            most = fmaxf(most, l[i]);
        }
    }
    most = warp_max(most);
    const float ref = most == -INFINITY ? 0.f : most;
    const float power = expert < 0 ? 0.f : expf(logit - ref);
    if (p.normalize) {
        sum = warp_sum(power);
    } else {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            l[i] = lane + 32 * i < p.E ? expf(l[i] - ref) : 0.f;
            sum += l[i];
        }
        sum = warp_sum(sum);
    }
    const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
    const float w = power * inv;
    const float mean = warp_sum(w * g);
    const float add = p.normalize ? w * (g - mean) : w * g;
    float d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = p.normalize ? 0.f : -l[i] * inv * mean;
    for (int j = 0; j < p.k; ++j) {
        const int e = __shfl_sync(~0u, expert, j);
        const float a = __shfl_sync(~0u, add, j);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 32 * i == e) d[i] += a;
    }
    T *out = static_cast<T *>(p.dlogits) + t * p.ldd;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (lane + 32 * i < p.E) out[lane + 32 * i] = to_type<T>(d[i]);
}

template <class T, int V>
cudaError_t run(bool grad, const RouteArgs &p, cudaStream_t s) {
    const int64_t blocks = (p.T + (int64_t)kThreads / 32 - 1) / (kThreads / 32);
    return grad ? launch(lm_route_grad_kernel<T, V>, blocks, kThreads, s, p)
                : launch(lm_route_kernel<T, V>, blocks, kThreads, s, p);
}

template <class T>
cudaError_t by_width(bool grad, const RouteArgs &p, cudaStream_t s) {
    if (p.E <= 32) return run<T, 1>(grad, p, s);
    if (p.E <= 64) return run<T, 2>(grad, p, s);
    if (p.E <= 128) return run<T, 4>(grad, p, s);
    if (p.E <= 256) return run<T, 8>(grad, p, s);
    if (p.E <= 512) return run<T, 16>(grad, p, s);
    return run<T, 32>(grad, p, s);
}

}  // namespace

cudaError_t route_launch(int type, bool grad, const RouteArgs &p, cudaStream_t s) {
    if (type == SGEMM_TYPE_F32) return by_width<float>(grad, p, s);
    if (type == SGEMM_TYPE_F16) return by_width<__half>(grad, p, s);
    return by_width<__nv_bfloat16>(grad, p, s);
}

}  // namespace sg
