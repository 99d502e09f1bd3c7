// Small kernels around the tensor-core products of the language-model
// operators: operand copies TMA can address, FP32 split into bf16 planes,
// the joins of partial results.  All are bound by memory, or by being a launch
// of a few microseconds; the copies move 8 neighbouring elements a thread, so
// that writes are whole 16-byte words.  On one GB300 the copy of 50001 x 1001
// f16 to a pitch of 1008 (200 MB moved) adds 35 us to the call that needs it,
// 5.7 TB/s; a copy of little, 1 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "lm_kernels.h"
#include "ptx.cuh"

namespace sg {
namespace {

// A launch that may begin while the kernel before it in the stream ends
// (griddepcontrol.wait orders its memory accesses).
template <class... P, class... A>
cudaError_t launch(void (*fn)(P...), int64_t blocks, int threads, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(std::max<int64_t>(1, blocks)));
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, P(args)...);
}

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = 152 * 16;

// Ends out of order are put in order by the kernel that reads the copy: a
// group that does not end behind the one before it is empty there too.
__device__ __forceinline__ bool unused(const LmCopyFilter &f, int64_t b) {
    return f.ends != nullptr && f.ends[b] <= (b > 0 ? f.ends[b - 1] : 0);
}

__device__ __forceinline__ bool keeps(const LmCopyFilter &f, int64_t row) {
    if (f.target == nullptr) return true;
    const int64_t t = f.target[row];
    return t >= 0 && t < f.vocab && f.grad[row] != 0.f;
}

// x = p0 + p1 + p2, each plane the bf16 nearest to what the ones before it
// leave: |p1| <= 2^-8 and |p2| <= 2^-17 of x's leading bit, so that the plane
// products left out of a product are below 2^-23.9 of it, with either sign.
// (Truncated planes leave up to 2^-21, always on the product's side of zero.)
// The sum is exact for |x| >= 2^-110; below, p2 meets bf16's smallest step,
// 2^-133.  x that would round up to infinity has its p0 truncated.  Values
// that are not finite stay in p0.
__device__ __forceinline__ float bf16_bits(float x, uint16_t &bits) {
    const __nv_bfloat16 h = __float2bfloat16_rn(x);
    bits = *reinterpret_cast<const uint16_t *>(&h);
    return __uint_as_float((uint32_t)bits << 16);
}
__device__ __forceinline__ void split3(float x, uint16_t &a, uint16_t &b, uint16_t &c) {
    const uint32_t u = __float_as_uint(x);
    const bool finite = (u & 0x7F800000u) != 0x7F800000u;
    float h = bf16_bits(x, a);
    if (finite && (a & 0x7F80u) == 0x7F80u) {
        a = (uint16_t)(u >> 16);
        h = __uint_as_float(u & 0xFFFF0000u);
    }
    const float r = finite ? x - h : 0.f;
    bf16_bits(r - bf16_bits(r, b), c);
}

__device__ __forceinline__ void load16(const void *p, uint32_t *w) {
    const uint4 v = *static_cast<const uint4 *>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
}

// Chunk i of a copy: 8 neighbours of one row.
template <bool F32>
__device__ __forceinline__ void copy_chunk(const LmCopy &j, int64_t i) {
    const int64_t per_row = j.ld_dst / 8;
    int64_t r, b;
    if (j.chunks <= 0xFFFFFFFFll) {                 // 32-bit divisions
        r = (uint32_t)i / (uint32_t)per_row;
        b = j.batch == 1 ? 0 : (uint32_t)r / (uint32_t)j.rows;
    } else {
        r = i / per_row;
        b = r / j.rows;
    }
    const int64_t c = (i - r * per_row) * 8;
    if (unused(j.keep, b)) return;
    const bool kept = keeps(j.keep, r);
    const int64_t to = r * j.ld_dst + c;
    constexpr int ELEM = F32 ? 4 : 2, WORDS = 2 * ELEM;        // 32-bit words of 8 elements
    const unsigned char *base = static_cast<const unsigned char *>(j.src);
    const int64_t at = (b * j.stride + (r - b * j.rows) * j.ld + c) * ELEM;
    // Rows of an odd pitch start anywhere in 16 bytes: the aligned words that
    // hold the chunk are loaded whole and shifted, unless they reach beyond
    // the operand.  (Forward pass of 1023 rows, 50001 x 1001 f16, of which 73 us
    // are not the copies: 118 -> 108 us.)
    const int skip = (int)(reinterpret_cast<uintptr_t>(base + at) & 15);
    const int64_t first = at - skip;
    uint32_t w[WORDS];
    if (!kept) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0u;
    } else if (c + 8 <= j.cols && first >= 0 && (skip == 0 || first + WORDS * 4 + 16 <= j.bytes)) {
        uint32_t l[WORDS + 4];
#pragma unroll
        for (int i = 0; i < WORDS; i += 4)
            load16(base + first + 4 * i, l + i);
        if (skip != 0) {
            load16(base + first + 4 * WORDS, l + WORDS);
#pragma unroll
            for (int i = 0; i < WORDS + 2; ++i) l[i] = skip & 8 ? l[i + 2] : l[i];
#pragma unroll
            for (int i = 0; i < WORDS + 1; ++i) l[i] = skip & 4 ? l[i + 1] : l[i];
            if constexpr (!F32) {
#pragma unroll
                for (int i = 0; i < WORDS; ++i) l[i] = __funnelshift_r(l[i], l[i + 1], 8 * (skip & 2));
            }
        }
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = l[i];
    } else if constexpr (F32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = c + e < j.cols ? reinterpret_cast<const uint32_t *>(base + at)[e] : 0u;
    } else {
        const uint16_t *s = reinterpret_cast<const uint16_t *>(base + at);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = (c + 2 * i < j.cols ? s[2 * i] : 0u) | (uint32_t)(c + 2 * i + 1 < j.cols ? s[2 * i + 1] : 0u) << 16;
    }
    uint16_t *dst = static_cast<uint16_t *>(j.dst) + to;
    if constexpr (F32) {
        alignas(16) uint16_t v[3][8];
#pragma unroll
        for (int e = 0; e < 8; ++e) split3(__uint_as_float(w[e]), v[0][e], v[1][e], v[2][e]);
#pragma unroll
        for (int q = 0; q < 3; ++q)
            *reinterpret_cast<uint4 *>(dst + q * j.plane) = *reinterpret_cast<const uint4 *>(v[q]);
    } else {
        *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// One CTA: the largest |grad| of a counted row.
__device__ void grad_scale(const LmGradScale &g) {
    __shared__ float most[kThreads / 32];
    float m = 0.f;
    for (int i = threadIdx.x; i < g.rows; i += kThreads) {
        const int64_t t = g.target[i];
        if (t >= 0 && t < g.vocab) m = fmaxf(m, fabsf(g.grad[i]));
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
    if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, most[w]);
        const bool usable = m > 1.0e-30f && m < 1.0e30f;
        g.scale2[0] = usable ? g.top / m : 1.f;
        g.scale2[1] = usable ? m / g.top : 1.f;
    }
}

template <bool F32>
__global__ void __launch_bounds__(kThreads)
lm_copy_kernel(const __grid_constant__ LmCopy a, const __grid_constant__ LmCopy b,
               const __grid_constant__ LmGradScale scale) {
    griddep_launch_dependents();
    griddep_wait();
    if (blockIdx.x == 0 && scale.scale2 != nullptr) grad_scale(scale);
    const int64_t step = gridDim.x * (int64_t)kThreads;
    int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x;
    for (; i < a.chunks; i += step) copy_chunk<F32>(a, i);
    for (i -= a.chunks; i < b.chunks; i += step) copy_chunk<F32>(b, i);
}

// Joins the slabs' {maximum, sum of exp(l - maximum)} of each row in a fixed
// order: 32 rows per CTA, one per lane (neighbouring rows are neighbours in
// memory), the slabs dealt to 32 warps, 8 of a warp loaded at a time and
// joined to what it has (their maximum first, so that the exponentials do not
// wait for one another).
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(kJoinWarps * 32)
lm_lse_join_kernel(const float2 *part, int slabs, int rows, const float *picked, const int64_t *target,
                   int64_t vocab, float *loss, float *lse) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ float met[kJoinWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = min(blockIdx.x * 32 + lane, rows - 1);
    constexpr int U = 8;                            // loads in flight
    float m = -INFINITY, s = 0.f;
    for (int i = warp; i < slabs; i += U * kJoinWarps) {
        float2 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            v[u] = i + u * kJoinWarps < slabs ? part[(int64_t)(i + u * kJoinWarps) * rows + row]
                                              : make_float2(-INFINITY, 0.f);
        const float before = m;
#pragma unroll
        for (int u = 0; u < U; ++u) m = fmaxf(m, v[u].x);
        const float ref = m == -INFINITY ? 0.f : m;
        s *= expf(before - ref);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u * kJoinWarps < slabs) s += v[u].y * expf(v[u].x - ref);
    }
    met[warp][lane] = m;
    __syncthreads();
    const float own = m;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, met[w][lane]);
    const float ref = m == -INFINITY ? 0.f : m;
    s *= expf(own - ref);
    __syncthreads();
    met[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && (int)blockIdx.x * 32 + lane < rows) {
        s = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) s += met[w][lane];
        const float l = ref + logf(s);
        lse[row] = l;
        const int64_t t = target[row];
        loss[row] = t >= 0 && t < vocab ? l - picked[row] : 0.f;
    }
}

template <class Out> __device__ __forceinline__ Out to_out(float x);
template <> __device__ __forceinline__ float to_out<float>(float x) { return x; }
template <> __device__ __forceinline__ __half to_out<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 to_out<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

template <class Out>
__global__ void __launch_bounds__(kThreads)
lm_join_splits_kernel(const float *part, int64_t ld, int64_t plane, int splits, const float *alpha, int rows,
                      int cols, Out *out, int64_t ldo) {
    griddep_launch_dependents();
    griddep_wait();
    const float a = alpha != nullptr ? *alpha : 1.f;
    const int64_t total = (int64_t)rows * cols;
    for (int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x; i < total; i += gridDim.x * (int64_t)kThreads) {
        const int64_t r = total <= 0xFFFFFFFFll ? (uint32_t)i / (uint32_t)cols : i / cols, c = i - r * cols;
        float s = 0.f;
        for (int z = 0; z < splits; ++z) s += part[z * plane + r * ld + c];
        out[r * ldo + c] = to_out<Out>(a * s);
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads)
lm_zero_kernel(T *p, int64_t ld, int64_t stride, int64_t rows, int64_t cols, int64_t batch) {
    griddep_launch_dependents();
    griddep_wait();
    const int64_t total = rows * cols * batch;
    for (int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x; i < total; i += gridDim.x * (int64_t)kThreads) {
        const int64_t r = i / cols, b = r / rows;
        p[b * stride + (r - b * rows) * ld + (i - r * cols)] = T(0);
    }
}

int64_t blocks_for(int64_t threads) { return std::min<int64_t>((threads + kThreads - 1) / kThreads, kMaxBlocks); }

}  // namespace

cudaError_t lm_launch_copy(bool f32, LmCopy a, LmCopy b, const LmGradScale &scale, cudaStream_t s) {
    for (LmCopy *j : {&a, &b}) {
        if (j->src == nullptr) continue;
        j->chunks = j->ld_dst / 8 * j->rows * j->batch;
        j->bytes = ((j->batch - 1) * j->stride + (j->rows - 1) * j->ld + j->cols) * (f32 ? 4 : 2);
    }
    return launch(f32 ? lm_copy_kernel<true> : lm_copy_kernel<false>, blocks_for(a.chunks + b.chunks), kThreads, s, a,
                  b, scale);
}

cudaError_t lm_launch_lse_join(const float2 *part, int slabs, int rows, const float *picked, const int64_t *target,
                               int64_t vocab, float *loss, float *lse, cudaStream_t s) {
    return launch(lm_lse_join_kernel, (rows + 31) / 32, kJoinWarps * 32, s, part, slabs, rows, picked, target,
                  vocab, loss, lse);
}

cudaError_t lm_launch_join_splits(const float *part, int64_t ld_part, int64_t plane, int splits, const float *alpha,
                                  int rows, int cols, void *out, int64_t ldo, int out_type, cudaStream_t s) {
    const int64_t blocks = blocks_for((int64_t)rows * cols);
    if (out_type == kOutF32)
        return launch(lm_join_splits_kernel<float>, blocks, kThreads, s, part, ld_part, plane, splits, alpha, rows,
                      cols, static_cast<float *>(out), ldo);
    if (out_type == kOutF16)
        return launch(lm_join_splits_kernel<__half>, blocks, kThreads, s, part, ld_part, plane, splits, alpha, rows,
                      cols, static_cast<__half *>(out), ldo);
    return launch(lm_join_splits_kernel<__nv_bfloat16>, blocks, kThreads, s, part, ld_part, plane, splits, alpha,
                  rows, cols, static_cast<__nv_bfloat16 *>(out), ldo);
}

cudaError_t lm_launch_zero(void *p, int64_t ld, int64_t stride, int elem, int64_t rows, int64_t cols, int64_t batch,
                           cudaStream_t s) {
    const int64_t blocks = blocks_for(rows * cols * batch);
    if (elem == 4)
        return launch(lm_zero_kernel<uint32_t>, blocks, kThreads, s, static_cast<uint32_t *>(p), ld, stride, rows,
                      cols, batch);
    return launch(lm_zero_kernel<uint16_t>, blocks, kThreads, s, static_cast<uint16_t *>(p), ld, stride, rows, cols,
                  batch);
}

}  // namespace sg
