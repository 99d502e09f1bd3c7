// Rows of numbers as 8-bit integers with a scale each:
//
//   s = max |x| / 127 (rounded to FP32, at least 2^-126 unless all are 0)
//   q = x / s rounded to the nearest integer, ties to even
//
// The quotient's rounding is exact: r = rint(x * (1 / s)) is at most one off, and
// x - r s, which one fused operation gives without rounding (it is a multiple of
// half a unit of s and no larger than s), says whether a neighbour is nearer.  A
// row with an infinity or a NaN has scale NaN and integers 0, so that products
// with it are NaN.
//
// One CTA a row, 8 neighbours a thread and step; two steps stay in registers
// (a row of 16384), more are read again.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "../../include/sgemm_gb300_lm.h"
#include "lm_int8.h"
#include "lm_launch.cuh"
#include "lm_ptx.cuh"

namespace sg {
namespace {

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_float(int8_t x) { return (float)x; }

template <class T>
__device__ __forceinline__ void load8(const T *row, int64_t c, int64_t K, bool vec, float (&v)[8]) {
    if (vec && c + 8 <= K) {
        alignas(16) T e[8];
        if constexpr (sizeof(T) == 1) {
            *reinterpret_cast<uint2 *>(e) = *reinterpret_cast<const uint2 *>(row + c);
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i)
                reinterpret_cast<uint4 *>(e)[i] = reinterpret_cast<const uint4 *>(row + c)[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = as_float(e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < K ? as_float(row[c + i]) : 0.f;
    }
}

__device__ __forceinline__ int nearest(float x, float s, float inv) {
    float r = rintf(x * inv);
    const float rest = fmaf(-r, s, x);
    const float twice = 2.f * fabsf(rest);
    if (twice > s || (twice == s && ((int)r & 1))) r += copysignf(1.f, rest);
    return (int)fminf(fmaxf(r, -127.f), 127.f);
}

// (In f16 the rows are always those of a workspace: aligned, whole chunks.)
template <bool OUT16>
__device__ __forceinline__ void store8(void *out, int64_t at, const int (&q)[8], int n) {
    if constexpr (OUT16) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __halves2half2(__int2half_rn(q[2 * i]), __int2half_rn(q[2 * i + 1]));
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(static_cast<__half *>(out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if (n < 8) {
        for (int i = 0; i < n; ++i) static_cast<int8_t *>(out)[at + i] = (int8_t)q[i];
    } else {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = (q[4 * i] & 0xFF) | (q[4 * i + 1] & 0xFF) << 8 | (q[4 * i + 2] & 0xFF) << 16 |
                   (uint32_t)q[4 * i + 3] << 24;
        *reinterpret_cast<uint2 *>(static_cast<int8_t *>(out) + at) = make_uint2(w[0], w[1]);
    }
}

constexpr int kHeld = 2;

// T8: X holds integers already.  The kernel lets the next one begin only when it
// has waited itself (chained): what comes behind may then read everything but
// this kernel's outputs at once.
template <class T, bool OUT16>
__global__ void __launch_bounds__(1024)
lm_int8_quantize_kernel(const T *x, int64_t ldx, int64_t K, bool vec, void *out, int64_t ldo, int64_t cols,
                        bool out_vec, float *scales, bool chained) {
    if (!chained) griddep_launch_dependents();
    griddep_wait();
    if (chained) griddep_launch_dependents();
    const T *row = x + blockIdx.x * ldx;
    const int64_t chunks = (cols + 7) / 8, to = blockIdx.x * ldo;
    float v[kHeld][8];
    float s = 1.f, inv = 1.f;
    bool good = true;
    if constexpr (sizeof(T) == 1) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int64_t c = threadIdx.x + i * (int64_t)blockDim.x;
            if (c < chunks) load8(row, c * 8, K, vec, v[i]);
        }
    } else {
        // The largest |x| by its bits: infinities and NaN come out on top.
        uint32_t most = 0;
        for (int64_t c = threadIdx.x, i = 0; c < chunks; c += blockDim.x, ++i) {
            float u[8];
            load8(row, c * 8, K, vec, u);
#pragma unroll
            for (int e = 0; e < 8; ++e) most = max(most, __float_as_uint(u[e]) & 0x7FFFFFFFu);
#pragma unroll
            for (int h = 0; h < kHeld; ++h)
                if (i == h)
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[h][e] = u[e];
        }
        __shared__ uint32_t part[32];
        most = __reduce_max_sync(~0u, most);
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = most;
        __syncthreads();
        most = 0;
        for (int w = 0; w < (int)blockDim.x / 32; ++w) most = max(most, part[w]);
        good = most < 0x7F800000u;
        s = most == 0u ? 0.f : fmaxf(__uint_as_float(most) / 127.f, 1.17549435e-38f);
        if (!good) s = __uint_as_float(0x7FC00000u);
        inv = s > 0.f ? 1.f / s : 0.f;
        if (threadIdx.x == 0) scales[blockIdx.x] = s;
    }
    for (int64_t c = threadIdx.x, i = 0; c < chunks; c += blockDim.x, ++i) {
        float u[8];
        if (i >= kHeld) load8(row, c * 8, K, vec, u);
#pragma unroll
        for (int h = 0; h < kHeld; ++h)
            if (i == h)
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = v[h][e];
        int q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            q[e] = sizeof(T) == 1 ? (int)u[e] : good ? nearest(u[e], s, inv) : 0;
        const int n = (int)min((int64_t)8, cols - c * 8);
        if (out_vec || n < 8) {
            store8<OUT16>(out, to + c * 8, q, n);
        } else {
            for (int e = 0; e < 8; ++e) static_cast<int8_t *>(out)[to + c * 8 + e] = (int8_t)q[e];
        }
    }
}

template <class T>
cudaError_t quantize(const void *x, int64_t ldx, int64_t rows, int64_t K, void *out, int64_t ldo, int64_t cols,
                     bool out16, float *scales, bool chained, cudaStream_t s) {
    const int64_t bytes = sizeof(T) == 1 ? 8 : 16;
    const bool vec = reinterpret_cast<uintptr_t>(x) % bytes == 0 && ldx * (int64_t)sizeof(T) % bytes == 0;
    const bool out_vec = reinterpret_cast<uintptr_t>(out) % 8 == 0 && ldo % 8 == 0;
    const int threads = (int)std::min<int64_t>(1024, std::max<int64_t>(32, ((cols + 7) / 8 + 31) / 32 * 32));
    return launch(out16 ? lm_int8_quantize_kernel<T, true> : lm_int8_quantize_kernel<T, false>, rows, threads, s,
                  static_cast<const T *>(x), ldx, K, vec, out, ldo, cols, out_vec, scales, chained);
}

// ------------------------------------------------------------------- join

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads)
lm_int8_join_kernel(const int32_t *part, int64_t ld, int64_t plane, int splits, const int32_t *row_group,
                    const float *x_scales, const float *scales, int64_t rows, int64_t cols, void *out, int64_t ldo,
                    int out_type) {
    griddep_launch_dependents();
    griddep_wait();
    const int64_t total = rows * cols;
    for (int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x; i < total; i += gridDim.x * (int64_t)kThreads) {
        const int64_t r = total <= 0xFFFFFFFFll ? (uint32_t)i / (uint32_t)cols : i / cols, c = i - r * cols;
        const int g = row_group[r];
        float y = 0.f;
        if (g >= 0) {
            int32_t sum = 0;
            for (int z = 0; z < splits; ++z) sum += part[z * plane + r * ld + c];
            y = (float)sum * x_scales[r] * scales[g * cols + c];
        }
        if (out_type == kOutF32) static_cast<float *>(out)[r * ldo + c] = y;
        else if (out_type == kOutF16) static_cast<__half *>(out)[r * ldo + c] = __float2half_rn(y);
        else static_cast<__nv_bfloat16 *>(out)[r * ldo + c] = __float2bfloat16_rn(y);
    }
}

// 16 bytes a thread; the aligned words that hold them are loaded whole and
// shifted, unless they reach beyond the operand.
__global__ void __launch_bounds__(kThreads)
lm_int8_copy_kernel(const int8_t *w, int64_t ldw, int64_t stride, int64_t rows, int64_t cols, int64_t batch, int8_t *out,
                    int64_t ldo, const int32_t *ends) {
    griddep_launch_dependents();
    griddep_wait();
    const int64_t per_row = ldo / 16, total = per_row * rows * batch;
    const int64_t bytes = (batch - 1) * stride + (rows - 1) * ldw + cols;
    for (int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x; i < total; i += gridDim.x * (int64_t)kThreads) {
        const int64_t r = i / per_row, b = r / rows, c = (i - r * per_row) * 16;
        if (ends != nullptr && ends[b] <= (b > 0 ? ends[b - 1] : 0)) continue;
        const int64_t at = b * stride + (r - b * rows) * ldw + c;
        const int skip = (int)(reinterpret_cast<uintptr_t>(w + at) & 3);
        const int n = (int)min((int64_t)16, cols - c);
        uint32_t v[5] = {0, 0, 0, 0, 0};
        if (n == 16 && at >= skip && at - skip + 20 <= bytes) {
            const uint32_t *from = reinterpret_cast<const uint32_t *>(w + at - skip);
#pragma unroll
            for (int e = 0; e < 5; ++e) v[e] = from[e];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __funnelshift_r(v[e], v[e + 1], 8 * skip);
        } else {
            for (int e = 0; e < n; ++e) v[e / 4] |= (uint32_t)(uint8_t)w[at + e] << (8 * (e % 4));
        }
        *reinterpret_cast<uint4 *>(out + r * ldo + c) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

}  // namespace

cudaError_t int8_quantize_launch(int from, const void *x, int64_t ldx, int64_t T, int64_t K, void *out, int64_t ldo,
                                 int64_t cols, bool out16, float *scales, bool chained, cudaStream_t s) {
    if (from == SGEMM_TYPE_F32) return quantize<float>(x, ldx, T, K, out, ldo, cols, out16, scales, chained, s);
    if (from == SGEMM_TYPE_F16) return quantize<__half>(x, ldx, T, K, out, ldo, cols, out16, scales, chained, s);
    if (from == SGEMM_TYPE_BF16) return quantize<__nv_bfloat16>(x, ldx, T, K, out, ldo, cols, out16, scales, chained, s);
    return quantize<int8_t>(x, ldx, T, K, out, ldo, cols, out16, scales, chained, s);
}

cudaError_t int8_join_launch(const int32_t *part, int64_t ld_part, int64_t plane, int splits, const int32_t *row_group,
                             const float *x_scales, const float *scales, int64_t rows, int64_t cols, void *out,
                             int64_t ldo, int out_type, cudaStream_t s) {
    const int64_t blocks = std::min<int64_t>((rows * cols + kThreads - 1) / kThreads, 152 * 16);
    return launch(lm_int8_join_kernel, blocks, kThreads, s, part, ld_part, plane, splits, row_group, x_scales, scales,
                  rows, cols, out, ldo, out_type);
}

cudaError_t int8_copy_launch(const int8_t *w, int64_t ldw, int64_t stride, int64_t rows, int64_t cols, int64_t batch,
                             int8_t *out, int64_t ldo, const int32_t *ends, cudaStream_t s) {
    const int64_t blocks = std::min<int64_t>((ldo / 16 * rows * batch + kThreads - 1) / kThreads, 152 * 16);
    return launch(lm_int8_copy_kernel, blocks, kThreads, s, w, ldw, stride, rows, cols, batch, out, ldo, ends);
}

}  // namespace sg
