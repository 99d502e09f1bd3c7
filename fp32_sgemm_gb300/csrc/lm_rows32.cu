// Grouped products of few FP32 rows a group: y[t, :] = x[t, :] . op(W_g).
//
// W is read once, as it is, and that read bounds the product: on the tensor
// cores FP32 takes three bf16 planes, which would have to be written and read
// again (four times the bytes).  On the FP32 pipes 8 rows cost little more than
// one.  A CTA takes 32 columns of a group for 8 of its rows; its warps share the
// contraction, 16 x 32 elements of W a step (K x N matrices) or 32 x 32 (N x K),
// each lane four neighbours of a row; the x of 2048 columns lie in shared
// memory.  The lanes' and warps' FP32 sums are joined in a fixed order.
//
// Measured, K x N / N x K, beside the tensor cores': 8 groups of 8 rows, 4096 x
// 2048: 104 / 94 us and 175 / 179, of one row 81 / 72 (3.7 TB/s; what bounds it is
// how many loads are on their way between the stagings of x), of 16 186 / 157
// and 176 / 179; one group of one row, 4096 x 4096: 24 / 24 and 48 / 47 (with 256
// threads 40 / 34); 8 rows in each of 7, 1023 x 777: 15 / 14 and 25 / 24 (with 512
// threads 19 / 19).
#include "lm_mma.cuh"

namespace sg {

constexpr int kRowsT = 8, kRowsN = 32, kRowsK = 2048;      // rows, columns, staged part of K

// Four neighbours, n of them in the matrix.
__device__ __forceinline__ float4 load4(const float *p, int64_t n, bool vec) {
    if (vec && n >= 4) return *reinterpret_cast<const float4 *>(p);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (n > 0) v.x = p[0];
    if (n > 1) v.y = p[1];
    if (n > 2) v.z = p[2];
    if (n > 3) v.w = p[3];
    return v;
}
__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
    return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, c))));
}

// THREADS: 256 and two CTAs on an SM, so that one reads while the other stages x
// or joins; 512 where there is not even one tile for each SM.
template <bool TRANS, int THREADS>
__global__ void __launch_bounds__(THREADS, 512 / THREADS)
lm_rows32_kernel(const LmArgs p, const LmRows q) {
    constexpr int WARPS = THREADS / 32;
    extern __shared__ unsigned char smem_raw[];
    float *xs = reinterpret_cast<float *>(smem_raw);                        // [kRowsT][kRowsK]
    float *sums = xs + kRowsT * kRowsK;                                     // [warp][kRowsT][kRowsN]
    int *start = reinterpret_cast<int *>(sums + WARPS * kRowsT * kRowsN);
    uint32_t *prefix = reinterpret_cast<uint32_t *>(start + p.G + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_launch_dependents();
    griddep_wait();
    if (warp == 0) lm_group_tables<LmThin, kRagN>(p, start, prefix, lane);
    __syncthreads();
    const int tiles = (int)prefix[p.G + 1];
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
        int lo = 0, hi = p.G;                   // last g with prefix[g] <= t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= (uint32_t)t) lo = mid;
            else hi = mid - 1;
        }
        // Row chunks of a group side by side: they share W.
        const int local = t - (int)prefix[lo], rows = start[lo + 1] - start[lo], chunks = (rows + kRowsT - 1) / kRowsT;
        const int block = local / chunks, r0 = start[lo] + (local - block * chunks) * kRowsT;
        const int nr = min(kRowsT, start[lo + 1] - r0), n0 = block * kRowsN;
        const int K = lo == p.G ? 0 : q.K;      // rows behind the last end: zeros
        const float *W = q.W + (int64_t)min(lo, p.G - 1) * q.stride;
        constexpr int CN = TRANS ? 8 : 4;       // columns of a lane
        float acc[kRowsT][CN];
#pragma unroll
        for (int r = 0; r < kRowsT; ++r)
#pragma unroll
            for (int c = 0; c < CN; ++c) acc[r][c] = 0.f;

        for (int64_t k0 = 0; k0 < K; k0 += kRowsK) {
            const int nk = (int)min((int64_t)kRowsK, K - k0);
            __syncthreads();
            for (int i = threadIdx.x; i < kRowsT * (kRowsK / 4); i += THREADS) {
                const int r = i / (kRowsK / 4), k = (i % (kRowsK / 4)) * 4;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < nr && k < nk) v = load4(q.X + (int64_t)(r0 + r) * q.ldx + k0 + k, nk - k, q.x_vec);
                *reinterpret_cast<float4 *>(xs + r * kRowsK + k) = v;
            }
            __syncthreads();
            if constexpr (TRANS) {
                // Lane: columns n0 + lane / 8 + 4 j, k 4 (lane % 8) of 32.
                const int n = n0 + (lane >> 3), kl = (lane & 7) * 4;
                for (int k = warp * 32 + kl; k < nk; k += WARPS * 32) {
                    float4 w[CN];
#pragma unroll
                    for (int c = 0; c < CN; ++c)
                        w[c] = load4(W + (int64_t)min(n + 4 * c, p.M - 1) * q.ldw + k0 + k, nk - k, q.w_vec);
#pragma unroll
                    for (int r = 0; r < kRowsT; ++r) {
                        const float4 x = *reinterpret_cast<const float4 *>(xs + r * kRowsK + k);
#pragma unroll
                        for (int c = 0; c < CN; ++c) acc[r][c] = dot4(w[c], x, acc[r][c]);
                    }
                }
            } else {
                // Lane: columns n0 + 4 (lane % 8) and three more, k 4 (lane / 8)
                // and three more of 16.
                const int n = n0 + (lane & 7) * 4;
#pragma unroll 2
                for (int k = warp * 16 + (lane >> 3) * 4; k < nk; k += WARPS * 16) {
                    float4 w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = load4(W + (int64_t)(k0 + min(k + i, nk - 1)) * q.ldw + n, p.M - n, q.w_vec);
#pragma unroll
                    for (int r = 0; r < kRowsT; ++r) {
                        const float4 x = *reinterpret_cast<const float4 *>(xs + r * kRowsK + k);
                        const float xk[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (k + i >= nk) break;         // (what was read twice)
                            acc[r][0] = fmaf(w[i].x, xk[i], acc[r][0]);
                            acc[r][1] = fmaf(w[i].y, xk[i], acc[r][1]);
                            acc[r][2] = fmaf(w[i].z, xk[i], acc[r][2]);
                            acc[r][3] = fmaf(w[i].w, xk[i], acc[r][3]);
                        }
                    }
                }
            }
        }
        // Lanes of the same columns, then warps.
#pragma unroll
        for (int r = 0; r < kRowsT; ++r)
#pragma unroll
            for (int c = 0; c < CN; ++c) {
                float v = acc[r][c];
#pragma unroll
                for (int d = TRANS ? 1 : 8; d < (TRANS ? 8 : 32); d <<= 1) v += __shfl_xor_sync(~0u, v, d);
                if constexpr (TRANS) {
                    if ((lane & 7) == c) sums[(warp * kRowsT + r) * kRowsN + (lane >> 3) + 4 * c] = v;
                } else {
                    if ((lane >> 3) == c) sums[(warp * kRowsT + r) * kRowsN + (lane & 7) * 4 + c] = v;
                }
            }
        __syncthreads();
        if (threadIdx.x < kRowsT * kRowsN) {
            const int r = threadIdx.x / kRowsN, c = threadIdx.x % kRowsN;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) v += sums[(w * kRowsT + r) * kRowsN + c];
            if (r < nr && n0 + c < p.M) static_cast<float *>(p.C)[(int64_t)(r0 + r) * p.ldc + n0 + c] = v;
        }
        __syncthreads();
    }
}

template <int THREADS>
LmKernel rows32_info(bool trans) {
    LmKernel k;
    k.fn = trans ? reinterpret_cast<const void *>(&lm_rows32_kernel<true, THREADS>)
                 : reinterpret_cast<const void *>(&lm_rows32_kernel<false, THREADS>);
    k.threads = THREADS;
    k.smem = (kRowsT * kRowsK + THREADS / 32 * kRowsT * kRowsN) * 4;
    k.tile_m = kRowsN;
    k.bn = kRowsT;
    return k;
}
LmKernel lm_rows32_kernel_info(bool trans, bool few) { return few ? rows32_info<512>(trans) : rows32_info<256>(trans); }

}  // namespace sg
