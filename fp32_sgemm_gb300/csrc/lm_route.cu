// The router's choice and its gradient.  With p = softmax(l) over a token's E
// logits, the k largest are chosen, the lower index among equals:
//
//   w_j = p[e_j]                      (normalize: divided by the sum of the chosen p)
//   dl_e = p_e ([e chosen] g_e - sum_j p[e_j] g_j)    (normalize: of the chosen alone,
//                                                      with w in the place of p)
//
// One warp a token, the logits in registers (element lane + 32 i), read once: the
// choice takes k rounds of "the largest key, then the lowest index that has
// it" (warp reductions of integers), on the bits of the logits made to grow with
// their values.  Sums are FP32, in an order that E alone decides.
//
// On the device (one GB300): 32768 tokens, 8 of 256 experts, bf16, 14.5 us, gradient
// 11.0 (3.3 TB/s); 65536 tokens, 2 of 8, FP32, 9.6 and 11.2; 16 tokens, 2 of 64, 1.3 and
// 1.6.  What bounds the choice is integer operations, some 300 a warp and token.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

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

// Grows with x; both zeros alike, NaN above all, -inf the least.  (x + 0 makes -0 0
// and any NaN the one with all bits set but the sign.)
__device__ __forceinline__ uint32_t order_key(float x) {
    const int u = __float_as_int(__fadd_rn(x, 0.f));
    return (uint32_t)(u ^ ((u >> 31) | (int)0x80000000));
}
constexpr uint32_t kMasked = 0x007FFFFFu;              // of -inf
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

// V logits of a lane: neighbours, in vector loads (VEC: the row is aligned for them
// and E a multiple of V), or 32 apart.
template <class T, int V, bool VEC>
struct Logits {
    static __device__ __forceinline__ int expert(int lane, int i) { return VEC ? lane * V + i : lane + 32 * i; }
    static __device__ __forceinline__ void load(const T *row, int E, int lane, float (&l)[V]) {
        if constexpr (VEC) {
            constexpr int BYTES = V * (int)sizeof(T), WORD = BYTES >= 16 ? 16 : BYTES;
            using W = std::conditional_t<WORD == 16, uint4, std::conditional_t<WORD == 8, uint2, std::conditional_t<WORD == 4, uint32_t, uint16_t>>>;
            union U {
                W w[BYTES / WORD];
                T e[V];
                __device__ U() {}
            } u;
            const bool in = lane * V < E;
#pragma unroll
            for (int i = 0; i < BYTES / WORD; ++i)
                if (in) u.w[i] = reinterpret_cast<const W *>(row + lane * V)[i];
#pragma unroll
            for (int i = 0; i < V; ++i) l[i] = in ? load_f(&u.e[i]) : -INFINITY;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) l[i] = lane + 32 * i < E ? load_f(row + lane + 32 * i) : -INFINITY;
        }
    }
    static __device__ __forceinline__ void store(T *row, int E, int lane, const float (&d)[V]) {
        if constexpr (VEC) {
            constexpr int BYTES = V * (int)sizeof(T), WORD = BYTES >= 16 ? 16 : BYTES;
            using W = std::conditional_t<WORD == 16, uint4, std::conditional_t<WORD == 8, uint2, std::conditional_t<WORD == 4, uint32_t, uint16_t>>>;
            union U {
                W w[BYTES / WORD];
                T e[V];
                __device__ U() {}
            } u;
#pragma unroll
            for (int i = 0; i < V; ++i) u.e[i] = to_type<T>(d[i]);
            if (lane * V < E)
#pragma unroll
                for (int i = 0; i < BYTES / WORD; ++i) reinterpret_cast<W *>(row + lane * V)[i] = u.w[i];
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane + 32 * i < E) row[lane + 32 * i] = to_type<T>(d[i]);
        }
    }
};

// key falling, by a network of exchanges (odd-even merges).
template <int V>
__device__ __forceinline__ void sort_falling(uint32_t (&key)[V]) {
#pragma unroll
    for (int p = 1; p < V; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t a = key[i + j], b = key[i + j + k];
                        key[i + j] = max(a, b);
                        key[i + j + k] = min(a, b);
                    }
}

template <class T, int V, bool VEC>
__global__ void __launch_bounds__(kThreads)
lm_route_kernel(const RouteArgs p) {
    using L = Logits<T, V, VEC>;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = blockIdx.x * (int64_t)(kThreads / 32) + (threadIdx.x >> 5);
    if (t >= p.T) return;
    float l[V];
    L::load(static_cast<const T *>(p.logits) + t * p.ldl, p.E, lane, l);
    // 16-bit logits have no bits below the 13th: there the key holds 1023 less the
    // expert, so that one reduction finds the largest and among equals the first.
    // FP32: two.
    constexpr bool PACKED = sizeof(T) == 2;
    constexpr uint32_t VALUE = PACKED ? 0xFFFFE000u : 0xFFFFFFFFu;
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        key[i] = order_key(l[i]);                             // (of what is not there, too: -inf)
        if (PACKED) key[i] = (key[i] & VALUE) | (uint32_t)(1023 - L::expert(lane, i));
    }
    // Lane j holds choice j.
    float mine = -INFINITY;
    int expert = -1;
    auto take = [&](int j, uint32_t top, uint32_t e) {
        if (lane == j) {
            expert = (int)e;
            mine = __uint_as_float((top & 0x80000000u ? top & 0x7FFFFFFFu : ~top) & VALUE);
        }
    };
    // A lane's keys are sorted first where that is fewer operations than looking
    // through them once for each choice (32768 tokens, 8 of 256 experts, bf16:
    // 14.5 us, 17.3 without).
    constexpr int LEAST = V <= 4 ? 2 : V <= 8 ? 3 : V <= 16 ? 4 : 6;
    if (PACKED && V > 1 && p.k >= LEAST) {
        sort_falling(key);
        for (int j = 0; j < p.k; ++j) {
            const uint32_t top = __reduce_max_sync(~0u, key[0]);
            if ((top & VALUE) <= kMasked) break;              // masked, or none left
            const bool won = key[0] == top;
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = won ? (i + 1 < V ? key[i + 1] : 0u) : key[i];
            take(j, top, 1023u - (top & ~VALUE));
        }
    } else {
        for (int j = 0; j < p.k; ++j) {
            uint32_t best = key[0];
#pragma unroll
            for (int i = 1; i < V; ++i) best = max(best, key[i]);
            const uint32_t top = __reduce_max_sync(~0u, best);
            if ((top & VALUE) <= kMasked) break;
            uint32_t e;
            if constexpr (PACKED) {
                e = 1023u - (top & ~VALUE);
#pragma unroll
                for (int i = 0; i < V; ++i) key[i] = key[i] == top ? 0u : key[i];
            } else {
                uint32_t at = ~0u;
#pragma unroll
                for (int i = V - 1; i >= 0; --i)
                    if (key[i] == top) at = (uint32_t)L::expert(lane, i);
                e = __reduce_min_sync(~0u, at);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if ((uint32_t)L::expert(lane, i) == e) key[i] = 0u;
            }
            take(j, top, e);
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
            if (L::expert(lane, i) < p.E) sum += expf(l[i] - ref);
        sum = warp_sum(sum);
    }
    if (lane < p.k) {
        p.weights[t * p.k + lane] = expert < 0 ? 0.f : power / sum;
        p.experts[t * p.k + lane] = expert;
    }
}

template <class T, int V, bool VEC>
__global__ void __launch_bounds__(kThreads)
lm_route_grad_kernel(const RouteArgs p) {
    using L = Logits<T, V, VEC>;
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
        L::load(row, p.E, lane, l);
#pragma unroll
        for (int i = 0; i < V; ++i) most = fmaxf(most, l[i]);
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
            l[i] = L::expert(lane, i) < p.E ? expf(l[i] - ref) : 0.f;
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
            if (L::expert(lane, i) == e) d[i] += a;
    }
    L::store(static_cast<T *>(p.dlogits) + t * p.ldd, p.E, lane, d);
}

template <class T, int V>
cudaError_t run(bool grad, const RouteArgs &p, cudaStream_t s) {
    const int64_t blocks = (p.T + (int64_t)kThreads / 32 - 1) / (kThreads / 32);
    constexpr int64_t BYTES = std::min<int64_t>(16, V * (int64_t)sizeof(T)), ELEM = sizeof(T);
    auto whole = [&](const void *q, int64_t ld) {
        return reinterpret_cast<uintptr_t>(q) % BYTES == 0 && (p.T == 1 || ld * ELEM % BYTES == 0);
    };
    const bool vec = V > 1 && p.E % V == 0 && whole(p.logits, p.ldl) && (!grad || whole(p.dlogits, p.ldd));
    if (grad) return launch(vec ? lm_route_grad_kernel<T, V, true> : lm_route_grad_kernel<T, V, false>, blocks, kThreads, s, p);
    return launch(vec ? lm_route_kernel<T, V, true> : lm_route_kernel<T, V, false>, blocks, kThreads, s, p);
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
