// Tokens sorted by expert and back.  Choice a = t k + j of token t goes to row
// slots[a] of the sorted rows: choices of expert 0 first, each expert's in the
// order of a, those of no expert behind the last end (row r is then written as
// ~r in slots, and holds zeros), so that slots names every row once.
//
//   dispatch       rows[slots[t, j]] = x[t]
//   combine        y[t] = sum_j w[t, j] rows[slots[t, j]]      (j in order, FP32, rounded once)
//   its gradient   drows[slots[t, j]] = w[t, j] dy[t],  dw[t, j] = dy[t] . rows[slots[t, j]],
//                  drows[r] = 0 for a row r that no slot names
//
// The gradient of a dispatch is a combine without weights.  All three are bound
// by memory and go by token, so that what a token has once (x, y, dy) is moved
// once.  On the device (one GB300): 16384 tokens of two choices, 4096 bf16: dispatch 67
// us, of which the sort is 7 (402 MB, 6 TB/s), combine 66, without weights 62 (6.5
// TB/s), gradients 109 (6.2 TB/s); 8192 of eight, 2048: 57, 52, 92; 8192 of four, 1001
// f16, whose rows lie at odd addresses: 22, 23, 49 (3 TB/s); 16 of two, 1024: 2.5, 2.3,
// 3.6.  Many choices of narrow rows, 65536 of eight, 512 bf16: 154, 102, 187; there the
// sort, which has one cluster, takes 60 us ahead of the copy (bytes alone: 90).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "../../include/sgemm_gb300_lm.h"
#include "lm_expert.h"
#include "lm_launch.cuh"
#include "lm_ptx.cuh"

namespace sg {
namespace {

// ------------------------------------------------------------------- sort
//
// One cluster of up to 8 CTAs of 32 warps.  Each warp has a run of the choices,
// counts it by expert (a histogram of its own in shared memory), the histograms
// are added up over warps and, through distributed shared memory, over CTAs, and
// each warp goes over its run again with the row at which its choices of each
// expert start, 32 choices at a time: the order is that of the choices.
constexpr int kSortThreads = 1024, kSortWarps = 32, kSortCluster = 8, kAhead = 8;

// Bytes of its shared memory, all of it dynamic: what a launch may have without
// asking (48 KB) counts static arrays as well.
constexpr size_t sort_smem(int G) { return (size_t(G + 1) * (kSortWarps + 2) + kSortWarps) * 4; }

__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Choice a's expert, G for none; -1 from n on.
__device__ __forceinline__ int bin_of(const int64_t *experts, int64_t a, int64_t n, int G) {
    if (a >= n) return -1;
    const int64_t e = experts[a];
    return e >= 0 && e < G ? (int)e : G;
}

__global__ void __launch_bounds__(kSortThreads, 1)
lm_expert_sort_kernel(const int64_t *experts, int n, int G, int32_t *slots, int32_t *ends) {
    extern __shared__ uint32_t sm[];
    const int bins = G + 1;
    uint32_t *total = sm;                        // [bins] this CTA's
    uint32_t *first = total + bins;              // [bins] row of this CTA's first
    uint32_t *hist = first + bins;               // [warp][bins]
    uint32_t *sums = hist + kSortWarps * bins;   // [warp]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank(), ctas = (int)gridDim.x, bits = 32 - __clz(G);
    griddep_launch_dependents();
    griddep_wait();
    for (int i = threadIdx.x; i < kSortWarps * bins; i += kSortThreads) hist[i] = 0u;
    __syncthreads();
    const int64_t warps = (int64_t)ctas * kSortWarps;
    const int64_t run = ((n + warps - 1) / warps + 31) / 32 * 32;
    const int64_t a0 = (rank * kSortWarps + warp) * run, a1 = min(a0 + run, (int64_t)n);
    uint32_t *own = hist + warp * bins;
    // (Loads of kAhead steps together; the first are kept for the second time.)
    int kept[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) kept[i] = bin_of(experts, a0 + 32 * i + lane, a1, G);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (kept[i] >= 0) atomicAdd(own + kept[i], 1u);
    for (int64_t a = a0 + 32 * kAhead; a < a1; a += 32 * kAhead) {
        int b[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) b[i] = bin_of(experts, a + 32 * i + lane, a1, G);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (b[i] >= 0) atomicAdd(own + b[i], 1u);
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kSortThreads) {
        uint32_t sum = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t c = hist[w * bins + b];
            hist[w * bins + b] = sum;
            sum += c;
        }
        total[b] = sum;
    }
    cluster_sync();
    // Rows of the experts before, then of the CTAs before.
    uint32_t before = 0;
    for (int b0 = 0; b0 < bins; b0 += kSortThreads) {
        const int b = b0 + (int)threadIdx.x;
        uint32_t all = 0, earlier = 0;
        if (b < bins)
            for (int c = 0; c < ctas; ++c) {
                const uint32_t v = ld_cluster(cluster_addr(total + b, (uint32_t)c));
                all += v;
                if (c < rank) earlier += v;
            }
        uint32_t scan = all;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(~0u, scan, d);
            if (lane >= d) scan += o;
        }
        if (lane == 31) sums[warp] = scan;
        __syncthreads();
        uint32_t of_warps = before;
        for (int w = 0; w < kSortWarps; ++w) {
            if (w < warp) of_warps += sums[w];
            before += sums[w];
        }
        __syncthreads();
        if (b < bins) {
            first[b] = of_warps + scan - all + earlier;
            if (rank == 0 && b < G) ends[b] = (int32_t)(of_warps + scan);
        }
    }
    // (No CTA leaves, or goes on to write, before the others have read.)
    cluster_sync();
    for (int64_t a = a0; a < a1; a += 32 * kAhead) {
        int b[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) b[i] = a == a0 ? kept[i] : bin_of(experts, a + 32 * i + lane, a1, G);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (a + 32 * i >= a1) break;
            // Lanes of the same expert, by the bits of its number (524288 choices of
            // 256 experts: 80 us with __match_any_sync, 60).
            uint32_t same = __ballot_sync(~0u, b[i] >= 0);
            for (int bit = 0; bit < bits; ++bit) {
                const bool set = (b[i] >> bit) & 1;
                const uint32_t with = __ballot_sync(~0u, set);
                same &= set ? with : ~with;
            }
            const uint32_t below = same & ((1u << lane) - 1u);
            if (b[i] >= 0) {
                const int32_t r = (int32_t)(first[b[i]] + own[b[i]] + __popc(below));
                slots[a + 32 * i + lane] = b[i] < G ? r : ~r;
            }
            __syncwarp();
            if (b[i] >= 0 && below == 0u) own[b[i]] += __popc(same);
            __syncwarp();
        }
    }
}

// ------------------------------------------------------------------- rows

// Pieces of a row that one load or store takes: the widest that every row of
// the call is aligned to.
int64_t piece_bytes(std::initializer_list<int64_t> all) {
    int64_t any = 16;
    for (int64_t v : all) any |= v;
    return any & -any;
}
int64_t address(const void *p) { return (int64_t)reinterpret_cast<uintptr_t>(p); }

constexpr int kThreads = 256, kWarps = kThreads / 32;
// CTAs for `tasks` warps, at most `most` times the SMs.
int64_t blocks_for(int64_t tasks, int64_t most) { return std::min((tasks + kWarps - 1) / kWarps, 152 * most); }

// Few choices are not sorted first: each warp counts those that come before its
// token's in shared memory, and CTA 0 the ends as well: one launch in the place of
// two.  Measured on the device, us: 16 tokens, two of 64 experts, 1024 bf16, 3.0,
// sorted first 6.5; 512 of two, 1024, 3.4 / 7.4; 128 of eight, 2048, 6.6 / 9.7; 256 of
// eight, 2048, 9.8 / 10.0; 512 of eight, 2048, 22.5 / 10.2.  A count is n / 32 steps,
// and there are n of them for each part of a row that a warp takes.
constexpr int kFewChoices = 4096;
bool few_choices(int64_t n, int64_t parts) { return n <= kFewChoices && n * n * parts <= 1 << 23; }

// Row of choice a among n, by one warp.
__device__ __forceinline__ int32_t place_of(const uint16_t *bins, int n, int a, int G, int lane) {
    const int b = bins[a];
    uint32_t before = 0;
    for (int i = lane; i < n; i += 32) {
        const int o = bins[i];
        before += o < b || (o == b && i < a);
    }
    const int32_t r = (int32_t)__reduce_add_sync(~0u, before);
    return b < G ? r : ~r;
}

template <class P, int U>
__global__ void __launch_bounds__(kThreads)
lm_expert_dispatch_few_kernel(const ExpertRows p, const int64_t *experts, int G, int32_t *ends, int64_t pieces,
                              int64_t parts) {
    __shared__ uint16_t bins[kFewChoices];
    __shared__ uint32_t count[kRouteMaxExperts + 1];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, n = (int)p.T * p.k;
    for (int i = threadIdx.x; i < n; i += kThreads) bins[i] = (uint16_t)bin_of(experts, i, n, G);
    if (blockIdx.x == 0)
        for (int g = threadIdx.x; g <= G; g += kThreads) count[g] = 0u;
    __syncthreads();
    if (blockIdx.x == 0) {
        for (int i = threadIdx.x; i < n; i += kThreads) atomicAdd(count + bins[i], 1u);
        __syncthreads();
        if (threadIdx.x < 32) {
            uint32_t sum = 0;
            for (int g0 = 0; g0 < G; g0 += 32) {
                uint32_t c = g0 + lane < G ? count[g0 + lane] : 0u;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint32_t o = __shfl_up_sync(~0u, c, d);
                    if (lane >= d) c += o;
                }
                if (g0 + lane < G) ends[g0 + lane] = (int32_t)(sum + c);
                sum += __shfl_sync(~0u, c, 31);
            }
        }
    }
    int32_t *slots = const_cast<int32_t *>(p.slots);
    const int64_t tasks = p.T * parts;
    for (int64_t i = blockIdx.x * (int64_t)kWarps + (threadIdx.x >> 5); i < tasks; i += gridDim.x * (int64_t)kWarps) {
        const int64_t t = i / parts, part = i - t * parts, c0 = part * (U * 32) + lane;
        const P *from = reinterpret_cast<const P *>(static_cast<const char *>(p.x) + t * p.ldx);
        P v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + u * 32 < pieces) v[u] = from[c0 + u * 32];
        for (int j = 0; j < p.k; ++j) {
            const int32_t slot = place_of(bins, n, (int)t * p.k + j, G, lane);
            if (part == 0 && lane == 0) slots[t * p.k + j] = slot;
            P *to = reinterpret_cast<P *>(static_cast<char *>(p.out) + (int64_t)(slot < 0 ? ~slot : slot) * p.ldo);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + u * 32 < pieces) to[c0 + u * 32] = slot < 0 ? P{} : v[u];
        }
    }
}

// A warp takes U * 32 pieces of one token at a time.
template <class P, int U>
__global__ void __launch_bounds__(kThreads)
lm_expert_dispatch_kernel(const ExpertRows p, int64_t pieces, int64_t parts) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t tasks = p.T * parts;
    for (int64_t i = blockIdx.x * (int64_t)kWarps + (threadIdx.x >> 5); i < tasks; i += gridDim.x * (int64_t)kWarps) {
        const int64_t t = i / parts, c0 = (i - t * parts) * (U * 32) + lane;
        const P *from = reinterpret_cast<const P *>(static_cast<const char *>(p.x) + t * p.ldx);
        P v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + u * 32 < pieces) v[u] = from[c0 + u * 32];
        for (int j = 0; j < p.k; ++j) {
            const int32_t slot = p.slots[t * p.k + j];
            P *to = reinterpret_cast<P *>(static_cast<char *>(p.out) + (int64_t)(slot < 0 ? ~slot : slot) * p.ldo);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + u * 32 < pieces) to[c0 + u * 32] = slot < 0 ? P{} : v[u];
        }
    }
}

// Elements of a piece as FP32 and back.
template <class T, class P>
struct Piece {
    static constexpr int N = sizeof(P) / sizeof(T);
    union {
        P p;
        T e[N];
    };
    __device__ __forceinline__ Piece() {}
    __device__ __forceinline__ float get(int i) const { return (float)e[i]; }
    __device__ __forceinline__ void set(int i, float v) {
        if constexpr (std::is_same_v<T, __half>) e[i] = __float2half_rn(v);
        else if constexpr (std::is_same_v<T, __nv_bfloat16>) e[i] = __float2bfloat16_rn(v);
        else e[i] = v;
    }
};

// rows outside [0, T k) are none.
__device__ __forceinline__ bool row_of(const ExpertRows &p, int32_t slot) {
    return slot >= 0 && slot < p.T * p.k;
}

// U pieces of J rows are on their way at once.
template <class T, class P, int U, int J>
__global__ void __launch_bounds__(kThreads, 4)
lm_expert_combine_kernel(const ExpertRows p, int64_t pieces, int64_t parts) {
    griddep_launch_dependents();
    griddep_wait();
    using Pc = Piece<T, P>;
    const int lane = threadIdx.x & 31;
    const int64_t tasks = p.T * parts;
    for (int64_t i = blockIdx.x * (int64_t)kWarps + (threadIdx.x >> 5); i < tasks; i += gridDim.x * (int64_t)kWarps) {
        const int64_t t = i / parts, c0 = (i - t * parts) * (U * 32) + lane;
        float sum[U][Pc::N];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < Pc::N; ++e) sum[u][e] = 0.f;
#pragma unroll J
        for (int j = 0; j < p.k; ++j) {
            const int32_t slot = p.slots[t * p.k + j];
            if (!row_of(p, slot)) continue;
            const float w = p.weights != nullptr ? p.weights[t * p.k + j] : 1.f;
            const P *from = reinterpret_cast<const P *>(static_cast<const char *>(p.x) + slot * p.ldx);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + u * 32 < pieces) {
                    Pc v;
                    v.p = from[c0 + u * 32];
#pragma unroll
                    for (int e = 0; e < Pc::N; ++e) sum[u][e] = fmaf(w, v.get(e), sum[u][e]);
                }
        }
        P *to = reinterpret_cast<P *>(static_cast<char *>(p.out) + t * p.ldo);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + u * 32 < pieces) {
                Pc v;
#pragma unroll
                for (int e = 0; e < Pc::N; ++e) v.set(e, sum[u][e]);
                to[c0 + u * 32] = v.p;
            }
    }
}

// A CTA a token: KC choices at a time, so that dy's pieces meet KC rows, and U
// pieces of each at once.  What counts is how many loads are on their way on an SM,
// so the registers are held down: 16384 tokens of two choices, 4096 bf16, two
// choices at a time 107 us, with two pieces and as many registers as it likes 191;
// 8192 of eight, 2048, 89 and 133, four at a time 116; odd f16 rows, 8192 of four,
// 1001, eight pieces 49, two 64 (without the rows that no slot names, below).
template <class T, class P, int KC, int U>
__global__ void __launch_bounds__(kThreads, sizeof(P) == 16 ? 5 : 3)
lm_expert_combine_grad_kernel(const ExpertRows p, int64_t pieces) {
    griddep_launch_dependents();
    griddep_wait();
    using Pc = Piece<T, P>;
    __shared__ float part[kWarps][KC];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = blockIdx.x;
    const P *dy = reinterpret_cast<const P *>(static_cast<const char *>(p.x) + t * p.ldx);
    for (int j0 = 0; j0 < p.k; j0 += KC) {
        float dot[KC], w[KC];
        bool none[KC];                                      // zeros, whatever dy holds
        const P *row[KC];                                   // NULL: takes no part in dweights
        P *to[KC];                                          // NULL: no row
#pragma unroll
        for (int j = 0; j < KC; ++j) {
            dot[j] = 0.f;
            w[j] = 0.f;
            row[j] = nullptr;
            to[j] = nullptr;
            none[j] = true;
            if (j0 + j < p.k) {
                // (Without owners row ~slot is of no expert.)
                const int32_t slot = p.slots[t * p.k + j0 + j], at = slot < 0 && p.owner == nullptr ? ~slot : slot;
                none[j] = slot < 0;
                if (slot >= 0) w[j] = p.weights != nullptr ? p.weights[t * p.k + j0 + j] : 1.f;
                if (p.dweights != nullptr && row_of(p, slot))
                    row[j] = reinterpret_cast<const P *>(static_cast<const char *>(p.rows) + slot * p.ldr);
                if (p.out != nullptr && row_of(p, at)) {
                    to[j] = reinterpret_cast<P *>(static_cast<char *>(p.out) + at * p.ldo);
                    if (p.owner != nullptr && threadIdx.x == 0) p.owner[at] = (int32_t)(t * p.k + j0 + j);
                }
            }
        }
        for (int64_t c0 = threadIdx.x; c0 < pieces; c0 += (int64_t)blockDim.x * U) {
            Pc g[U], r[KC][U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t c = c0 + u * blockDim.x;
                if (c < pieces) {
                    g[u].p = dy[c];
#pragma unroll
                    for (int j = 0; j < KC; ++j)
                        if (row[j] != nullptr) r[j][u].p = row[j][c];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t c = c0 + u * blockDim.x;
                if (c >= pieces) break;
#pragma unroll
                for (int j = 0; j < KC; ++j) {
                    if (row[j] != nullptr)
#pragma unroll
                        for (int e = 0; e < Pc::N; ++e) dot[j] = fmaf(g[u].get(e), r[j][u].get(e), dot[j]);
                    if (to[j] != nullptr) {
                        Pc v;
#pragma unroll
                        for (int e = 0; e < Pc::N; ++e) v.set(e, none[j] ? 0.f : w[j] * g[u].get(e));
                        to[j][c] = v.p;
                    }
                }
            }
        }
        if (p.dweights != nullptr) {
#pragma unroll
            for (int j = 0; j < KC; ++j)
#pragma unroll
                for (int d = 16; d; d >>= 1) dot[j] += __shfl_xor_sync(~0u, dot[j], d);
            if (lane == 0)
#pragma unroll
                for (int j = 0; j < KC; ++j) part[warp][j] = dot[j];
            __syncthreads();
            if ((int)threadIdx.x < KC && j0 + (int)threadIdx.x < p.k) {
                float sum = 0.f;
                for (int v = 0; v < (int)blockDim.x / 32; ++v) sum += part[v][threadIdx.x];
                p.dweights[t * p.k + j0 + threadIdx.x] = sum;
            }
            __syncthreads();
        }
    }
}

// Zeros for the rows of a gradient that no slot names (and a negative slot names
// none): owner[r] is the choice that names row r, noted where its gradient is written,
// and what lies there otherwise is no choice that names r, whatever it is.  A lane
// looks at a row.  (8192 tokens of eight choices, 2048 bf16, sum and gradients: 146
// us, 143 without it; looked at by the kernel above instead, with the owners noted by
// one before it, 150; zeros written everywhere first would move half as much again.)
template <class P>
__global__ void __launch_bounds__(kThreads)
lm_expert_bare_kernel(const ExpertRows p, int64_t pieces) {
    griddep_launch_dependents();
    griddep_wait();
    // (Rows of no expert are neighbours: a warp's rows are not.)
    const int64_t n = p.T * p.k, warps = gridDim.x * (int64_t)kWarps;
    const int lane = threadIdx.x & 31;
    for (int64_t r0 = blockIdx.x * (int64_t)kWarps + (threadIdx.x >> 5); r0 < n; r0 += 32 * warps) {
        const int64_t r = r0 + lane * warps;
        bool bare = false;
        if (r < n) {
            const int32_t a = p.owner[r];
            bare = a < 0 || a >= n || p.slots[a] != r;
        }
        for (uint32_t left = __ballot_sync(~0u, bare); left; left &= left - 1u) {
            P *to = reinterpret_cast<P *>(static_cast<char *>(p.out) + (r0 + (__ffs(left) - 1) * warps) * p.ldo);
            for (int64_t c = lane; c < pieces; c += 32) to[c] = P{};
        }
    }
}

// Pieces that a lane takes at once: narrow ones (rows of odd bases or pitches) many.
template <class P> constexpr int kPieces = sizeof(P) >= 8 ? 4 : 8;

template <class T, class P>
cudaError_t combine_by_piece(const ExpertRows &p, cudaStream_t s) {
    const int64_t pieces = p.D * p.elem / (int64_t)sizeof(P);
    auto run = [&](auto count, auto rows, int64_t most) {
        constexpr int U = decltype(count)::value, J = decltype(rows)::value;
        const int64_t parts = (pieces + U * 32 - 1) / (U * 32);
        return launch(lm_expert_combine_kernel<T, P, U, J>, blocks_for(p.T * parts, most), kThreads, s, p, pieces, parts);
    };
    // Four pieces of two rows where a row has as many for each lane, else two of four
    // (16384 tokens of two choices, 4096 bf16: 67 us, 69; 65536 of eight, 512: 138, 102).
    if (pieces >= 128) return run(std::integral_constant<int, 4>(), std::integral_constant<int, 2>(), 64);
    return run(std::integral_constant<int, 2>(), std::integral_constant<int, 4>(), 8);
}

template <class T, class P>
cudaError_t grad_by_piece(const ExpertRows &p, cudaStream_t s) {
    const int64_t pieces = p.D * p.elem / (int64_t)sizeof(P);
    auto run = [&](auto choices) {
        constexpr int KC = decltype(choices)::value, U = (sizeof(P) == 16 ? 4 : 16) / KC;
        const int64_t each = (pieces + U - 1) / U;
        const int threads = (int)std::min<int64_t>(kThreads, std::max<int64_t>(32, (each + 31) / 32 * 32));
        return launch(lm_expert_combine_grad_kernel<T, P, KC, U>, p.T, threads, s, p, pieces);
    };
    const cudaError_t e = p.k == 1 ? run(std::integral_constant<int, 1>()) : run(std::integral_constant<int, 2>());
    if (e != cudaSuccess || p.out == nullptr || p.owner == nullptr) return e;
    return launch(lm_expert_bare_kernel<P>, blocks_for(p.T * p.k, 8), kThreads, s, p, pieces);
}

cudaError_t sort_launch(const int64_t *experts, int n, int G, int32_t *slots, int32_t *ends, cudaStream_t s) {
    const size_t smem = sort_smem(G);
    if (smem > 48 * 1024) {                       // (for any number of experts: another call may ask for more)
        const cudaError_t opted = cudaFuncSetAttribute(lm_expert_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       int(sort_smem(SGEMM_MAX_GROUPS)));
        if (opted != cudaSuccess) return opted;
    }
    // A warp has at least 64 choices before there is another CTA.
    int ctas = 1;
    while (ctas < kSortCluster && (int64_t)ctas * kSortWarps * 64 < n) ctas *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(ctas));
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(ctas);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, lm_expert_sort_kernel, experts, n, G, slots, ends);
}

template <class P>
cudaError_t dispatch_by_piece(const ExpertRows &p, const int64_t *experts, int G, int32_t *slots, int32_t *ends,
                              cudaStream_t s) {
    constexpr int U = kPieces<P>;
    const int64_t pieces = p.D * p.elem / (int64_t)sizeof(P), parts = (pieces + U * 32 - 1) / (U * 32);
    const bool any = p.T * p.k > 0 && p.D > 0;
    if (any && few_choices(p.T * p.k, parts))
        return launch(lm_expert_dispatch_few_kernel<P, U>, blocks_for(p.T * parts, 64), kThreads, s, p, experts, G, ends,
                      pieces, parts);
    const cudaError_t e = sort_launch(experts, int(p.T * p.k), G, slots, ends, s);
    if (e != cudaSuccess || !any) return e;
    return launch(lm_expert_dispatch_kernel<P, U>, blocks_for(p.T * parts, 64), kThreads, s, p, pieces, parts);
}

}  // namespace

cudaError_t expert_dispatch_launch(const ExpertRows &p, const int64_t *experts, int G, int32_t *slots, int32_t *ends,
                                   cudaStream_t s) {
    switch (piece_bytes({address(p.x), p.ldx, address(p.out), p.ldo, p.D * p.elem})) {
        case 16: return dispatch_by_piece<uint4>(p, experts, G, slots, ends, s);
        case 8: return dispatch_by_piece<uint2>(p, experts, G, slots, ends, s);
        case 4: return dispatch_by_piece<uint32_t>(p, experts, G, slots, ends, s);
        default: return dispatch_by_piece<uint16_t>(p, experts, G, slots, ends, s);
    }
}

cudaError_t expert_combine_launch(int type, const ExpertRows &p, cudaStream_t s) {
    const int64_t piece = piece_bytes({address(p.x), p.ldx, address(p.out), p.ldo, p.D * p.elem});
    if (type == SGEMM_TYPE_F32)
        return piece == 16 ? combine_by_piece<float, uint4>(p, s) : combine_by_piece<float, uint32_t>(p, s);
    if (type == SGEMM_TYPE_F16)
        return piece == 16 ? combine_by_piece<__half, uint4>(p, s) : combine_by_piece<__half, uint16_t>(p, s);
    return piece == 16 ? combine_by_piece<__nv_bfloat16, uint4>(p, s) : combine_by_piece<__nv_bfloat16, uint16_t>(p, s);
}

cudaError_t expert_combine_grad_launch(int type, const ExpertRows &p, cudaStream_t s) {
    int64_t piece = piece_bytes({address(p.x), p.ldx, p.D * p.elem});
    if (p.out != nullptr) piece = std::min(piece, piece_bytes({address(p.out), p.ldo}));
    if (p.dweights != nullptr) piece = std::min(piece, piece_bytes({address(p.rows), p.ldr}));
    if (type == SGEMM_TYPE_F32)
        return piece == 16 ? grad_by_piece<float, uint4>(p, s) : grad_by_piece<float, uint32_t>(p, s);
    if (type == SGEMM_TYPE_F16)
        return piece == 16 ? grad_by_piece<__half, uint4>(p, s) : grad_by_piece<__half, uint16_t>(p, s);
    return piece == 16 ? grad_by_piece<__nv_bfloat16, uint4>(p, s) : grad_by_piece<__nv_bfloat16, uint16_t>(p, s);
}

}  // namespace sg
