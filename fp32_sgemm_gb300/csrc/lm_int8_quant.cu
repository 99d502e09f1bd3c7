// Rows of numbers as 8-bit integers with a scale each (lm_int8_round.cuh has the
// rounding).
//
// One CTA a row, 8 neighbours a thread and step; what a thread has in its first
// one or four steps stays in registers, more is read again.  8192 rows of 4096 bf16 to
// bytes: 25 us, where the bytes alone take 15.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "../../include/sgemm_gb300_lm.h"
#include "lm_int8.h"
#include "lm_int8_round.cuh"
#include "lm_launch.cuh"
#include "lm_ptx.cuh"

namespace sg {
namespace {

// T8: X holds integers already.  The kernel lets the next one begin only when it
// has waited itself (chained): what comes behind may then read everything but
// this kernel's outputs at once.
template <class T, bool OUT16, int HELD>
__global__ void __launch_bounds__(HELD == 1 ? 1024 : 256, HELD == 1 ? 1 : 3)
lm_int8_quantize_kernel(const T *x, int64_t ldx, int64_t rows, int64_t K, bool vec, void *out, int64_t ldo, int64_t cols,
                        bool out_vec, float *scales, bool chained) {
    if (!chained) griddep_launch_dependents();
    griddep_wait();
    if (chained) griddep_launch_dependents();
    __shared__ uint32_t part[2][32];
    const int64_t chunks = (cols + 7) / 8;
    const int warps = (int)blockDim.x / 32, lane = threadIdx.x & 31;
    Eight<T> next[HELD];
    auto load = [&](int64_t r) {
#pragma unroll
        for (int h = 0; h < HELD; ++h) {
            const int64_t c = threadIdx.x + h * (int64_t)blockDim.x;
            next[h].load(x + r * ldx + c * 8, K - c * 8, vec);
        }
    };
    // (Rows of one warp each: several in a CTA, blockDim.y of them.)
    const int64_t first = blockIdx.x * (int64_t)blockDim.y + threadIdx.y, step = gridDim.x * (int64_t)blockDim.y;
    int turn = 0;
    if (first < rows) load(first);
    for (int64_t r = first; r < rows; r += step, turn ^= 1) {
        const T *row = x + r * ldx;
        Eight<T> v[HELD];
#pragma unroll
        for (int h = 0; h < HELD; ++h) v[h] = next[h];
        if (r + step < rows) load(r + step);
        float s = 1.f, inv = 1.f;
        bool zero = false;
        if constexpr (sizeof(T) != 1) {
            uint32_t most = 0;
#pragma unroll
            for (int h = 0; h < HELD; ++h) most = max(most, v[h].most());
            for (int64_t c = threadIdx.x + HELD * (int64_t)blockDim.x; c < chunks; c += blockDim.x) {
                Eight<T> u;
                u.load(row + c * 8, K - c * 8, vec);
                most = max(most, u.most());
            }
            most = __reduce_max_sync(~0u, most);
            if (warps > 1) {                       // (two tables: a warp may be one row ahead)
                if (lane == 0) part[turn][threadIdx.x >> 5] = most;
                __syncthreads();
                most = __reduce_max_sync(~0u, lane < warps ? part[turn][lane] : 0u);
            }
            const RowScale of(most);
            s = of.s;
            inv = of.inv;
            if (threadIdx.x == 0) scales[r] = of.scale;
            if (!of.finite) {
#pragma unroll
                for (int h = 0; h < HELD; ++h) v[h].clear();
                zero = true;
            }
        }
        auto put = [&](const Eight<T> &u, int64_t c) {
            // (Integers already: by themselves.  A row that is not finite: zeros.)
            const Rounded q = nearest(u.e, s, inv);
            const int n = (int)min((int64_t)8, cols - c * 8);
            store8<OUT16>(out, r * ldo + c * 8, q, n, out_vec);
        };
#pragma unroll
        for (int h = 0; h < HELD; ++h) {
            const int64_t c = threadIdx.x + h * (int64_t)blockDim.x;
            if (c < chunks) put(v[h], c);
        }
        for (int64_t c = threadIdx.x + HELD * (int64_t)blockDim.x; c < chunks; c += blockDim.x) {
            Eight<T> u;
            u.load(row + c * 8, zero ? 0 : K - c * 8, vec);
            put(u, c);
        }
    }
}

template <class T>
cudaError_t quantize(const void *x, int64_t ldx, int64_t rows, int64_t K, void *out, int64_t ldo, int64_t cols,
                     bool out16, float *scales, bool chained, cudaStream_t s) {
    const int64_t bytes = sizeof(T) == 1 ? 8 : 16;
    const bool vec = reinterpret_cast<uintptr_t>(x) % bytes == 0 && ldx * (int64_t)sizeof(T) % bytes == 0;
    const bool out_vec = reinterpret_cast<uintptr_t>(out) % 8 == 0 && ldo % 8 == 0;
    const int64_t chunks = (cols + 7) / 8;
    // A thread for every 8 columns of every row while the device holds them all at
    // once; then fewer, each with the loads of its next row on their way (8192
    // rows of 4096, bf16: 41 us, 24.5).
    auto run = [&](auto held, bool all) {
        constexpr int H = decltype(held)::value;
        const int threads = (int)std::min<int64_t>(H == 1 ? 1024 : 256, std::max<int64_t>(32, ((chunks + H - 1) / H + 31) / 32 * 32));
        const int many = threads == 32 && rows > 152 ? 8 : 1;
        const int64_t blocks = all ? rows : 152 * (many > 1 ? 4 : std::max(1, 768 / threads));
        return launch(out16 ? lm_int8_quantize_kernel<T, true, H> : lm_int8_quantize_kernel<T, false, H>,
                      std::min((rows + many - 1) / many, blocks), dim3(unsigned(threads), unsigned(many)), s,
                      static_cast<const T *>(x), ldx, rows, K, vec, out, ldo, cols, out_vec, scales, chained);
    };
    constexpr int HELD = sizeof(T) == 4 ? 2 : 4;
    if (rows * chunks <= 304 * 1024) return run(std::integral_constant<int, 1>(), true);
    return chunks <= 32 ? run(std::integral_constant<int, 1>(), false) : run(std::integral_constant<int, HELD>(), false);
}

// ------------------------------------------------------------------- join

constexpr int kThreads = 256;

// Four columns of one row a thread (the planes' pitch is a multiple of 8), rows dealt
// to blockIdx.y.
template <class T>
__global__ void __launch_bounds__(kThreads)
lm_int8_join_kernel(const int32_t *part, int64_t ld, int64_t plane, int splits, const int32_t *row_group,
                    const float *x_scales, const float *scales, int64_t rows, int64_t cols, T *out, int64_t ldo, bool vec) {
    griddep_launch_dependents();
    griddep_wait();
    const int64_t c = (blockIdx.x * (int64_t)kThreads + threadIdx.x) * 4;
    if (c >= cols) return;
    const int n = (int)min((int64_t)4, cols - c);
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
        const int g = row_group[r];
        float y[4] = {0.f, 0.f, 0.f, 0.f};
        if (g >= 0) {
            int4 sum = make_int4(0, 0, 0, 0);
#pragma unroll 4
            for (int z = 0; z < splits; ++z) {
                const int4 v = *reinterpret_cast<const int4 *>(part + z * plane + r * ld + c);
                sum.x += v.x;
                sum.y += v.y;
                sum.z += v.z;
                sum.w += v.w;
            }
            const float xs = x_scales[r], s[4] = {(float)sum.x, (float)sum.y, (float)sum.z, (float)sum.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) y[i] = s[i] * xs * scales[g * cols + c + i];
        }
        T *to = out + r * ldo + c;
        alignas(16) T v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) v[i] = y[i];
            else if constexpr (std::is_same_v<T, __half>) v[i] = __float2half_rn(y[i]);
            else v[i] = __float2bfloat16_rn(y[i]);
        }
        if (vec && n == 4) {
            if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(v);
            else *reinterpret_cast<uint2 *>(to) = *reinterpret_cast<const uint2 *>(v);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) to[i] = v[i];
        }
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
    const int elem = out_type == kOutF32 ? 4 : 2;
    const bool vec = reinterpret_cast<uintptr_t>(out) % (4 * elem) == 0 && ldo % 4 == 0;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned((cols + 4 * kThreads - 1) / (4 * kThreads)), unsigned(std::min<int64_t>(rows, 65535)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (out_type == kOutF32)
        return cudaLaunchKernelEx(&cfg, lm_int8_join_kernel<float>, part, ld_part, plane, splits, row_group, x_scales,
                                  scales, rows, cols, static_cast<float *>(out), ldo, vec);
    if (out_type == kOutF16)
        return cudaLaunchKernelEx(&cfg, lm_int8_join_kernel<__half>, part, ld_part, plane, splits, row_group, x_scales,
                                  scales, rows, cols, static_cast<__half *>(out), ldo, vec);
    return cudaLaunchKernelEx(&cfg, lm_int8_join_kernel<__nv_bfloat16>, part, ld_part, plane, splits, row_group, x_scales,
                              scales, rows, cols, static_cast<__nv_bfloat16 *>(out), ldo, vec);
}

cudaError_t int8_copy_launch(const int8_t *w, int64_t ldw, int64_t stride, int64_t rows, int64_t cols, int64_t batch,
                             int8_t *out, int64_t ldo, const int32_t *ends, cudaStream_t s) {
    const int64_t blocks = std::min<int64_t>((ldo / 16 * rows * batch + kThreads - 1) / kThreads, 152 * 16);
    return launch(lm_int8_copy_kernel, blocks, kThreads, s, w, ldw, stride, rows, cols, batch, out, ldo, ends);
}

}  // namespace sg
