// Tensor-core products behind the language-model operators (grouped
// products, vocabulary cross entropy): 16-bit operands, FP32 accumulation,
// tcgen05.mma kind::f16 with operands staged by TMA.
//
//   D[m, n] = sum_k A[m, k] B[k, n]
//
// One kernel template serves every form; what changes is
//   * how each operand is stored: K contiguous ("K-major") or M / N
//     contiguous ("MN-major").  Both are read as they are (the MMA's
//     descriptors name the layout), so no operand is ever transposed in
//     memory;
//   * which extent is ragged (kRagNone, kRagN: columns of D are rows of a
//     token matrix that belong to groups, kRagK: the contraction runs over
//     the rows of a group);
//   * what the epilogue does with D (Epi).
//
// For kRagN the tokens are put on the MMA's N side and the group's matrix
// on its M side, because N may be any multiple of 16 (32 on an SM pair) per
// instruction: a group of r rows costs ceil(r / 16) * 16 columns of MMA
// time instead of a multiple of 128 or 256 rows.
//
// Structure: persistent CTAs (or SM pairs, cta_group::2: each SM holds half
// of the 256 rows of A and half of B's columns, so that shared memory feeds
// the tensor core 2/3 of the bytes per MMA that one SM alone would).  Warp 0
// is the TMA producer, warp 1 issues the MMAs, the others run the epilogue
// out of TMEM while the next tile is multiplied into the other accumulator.
// Every wait is bounded and reports its site in the handle's error word.
//
// What bounds it, measured on one GB300 (copies 6.69 TB/s, a library's bf16
// product 1915 TFLOP/s in a burst, 1730 sustained), bf16:
//   * many rows: the tensor core.  4096 tokens against 32768 x 4096: the tensor
//     pipe is busy 98.7% of the active cycles of the forward pass, 90% of the
//     kernel of d (its epilogue lasts longer than the two runs of 512 terms the
//     MMAs may be ahead), 97 to 97.7% of the gradient's two products.  8192
//     tokens against 131072 x 4096, loss and gradients: 20.8 to 21.2 ms for 35.2
//     TFLOP, 1660 to 1690 TFLOP/s at the power limit.  32768 rows in 8 groups,
//     4096 x 2048: 288 to 299 us, 1840 to 1910 TFLOP/s forward, 294 to 299 us
//     weight gradient.  With fewer tiles the last round leaves pairs idle (8192
//     rows: 108 and 100 us, 1270 and 1380 TFLOP/s, 256 and 1024 tiles on 76
//     pairs);
//   * few rows: reading the matrices.  19 of 64 groups' 1024 x 2048 (80 MB):
//     19.1 us, 4.2 TB/s, of which the first and last 3.5 us move nothing; 16
//     tokens against 32000 x 1024 (66 MB): 18 us and 3.5 for the join;
//   * FP32: six bf16 products for one, and the three planes of both operands
//     written and read again: 4096 rows in 8 groups, 1024 x 2048, both
//     gradients 219 to 245 us (206 GFLOP of bf16, 108 us).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "lm_kernels.h"
#include "lm_ptx.cuh"

namespace sg {

// ------------------------------------------------------------ PTX wrappers

__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

// MN-major operand stored with the 128-byte swizzle: chunks of 64 elements
// of M (N) by 64 of K, each K row 128 bytes, as a TMA box {64, 64} writes
// them.  Leading offset: from one chunk of 64 to the next (8 KB); stride
// offset: from 8 rows of K to the next 8 (1 KB).  K = 16 advances 2 KB.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(8192u >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

// Instruction descriptor, kind::f16: D f32, A and B both f16 (0) or bf16 (1).
__device__ __forceinline__ uint32_t idesc_f16(uint32_t bf16, bool a_mn, bool b_mn, int M, int N) {
    return (1u << 4) | (bf16 << 7) | (bf16 << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Arrive on an mbarrier of a CTA of the cluster, with nothing to publish.
// (With release semantics the arrival waits for the thread's earlier writes:
// once per stage, that halved the rate of the weight gradients.)
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" :: "r"(cluster_bar) : "memory");
}

__device__ __forceinline__ void fence_proxy_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void tmem_ld_32cols_nowait(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// 32 bytes to a 32-byte aligned address in one store: a whole sector.  (Kept out
// of L1, where it would take the place of what the epilogue has spilled.)
__device__ __forceinline__ void st_global_32B(void *p, const uint32_t *v) {
    asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
                    "r"(v[7]) : "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two FP32 additions in one (each rounded as by itself).
__device__ __forceinline__ void add2(float &a0, float &a1, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tadd.rn.f32x2 a, a, b;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}" : "+f"(a0), "+f"(a1) : "f"(b0), "f"(b1));
}

template <class T> __device__ __forceinline__ T lm_cvt(float x);
template <> __device__ __forceinline__ float lm_cvt<float>(float x) { return x; }
template <> __device__ __forceinline__ __half lm_cvt<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 lm_cvt<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <class T> __device__ __forceinline__ uint32_t lm_pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t lm_pack2<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <> __device__ __forceinline__ uint32_t lm_pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// ----------------------------------------------------------------- tiles

// One output tile: 128 rows of A per SM (256 on a pair) by up to BN columns.
// STG: floats of epilogue staging per warp (0 where the epilogue needs none).
template <int BN_, int STAGES_, bool PAIR_, int STG_ = 32 * 17>
struct LmTile {
    static constexpr bool PAIR = PAIR_;
    static constexpr int BM = 128, BN = BN_, BK = 64, STAGES = STAGES_;
    static constexpr int TILE_M = PAIR ? 256 : 128;
    static constexpr int B_ROWS = PAIR ? BN / 2 : BN;       // columns of B this SM stages
    static constexpr int GRAN = PAIR ? 32 : 16;             // granule of the MMA's N
    static constexpr int A_BYTES = BM * BK * 2, B_BYTES = B_ROWS * BK * 2;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int EPI_WARPS = BN >= 64 ? 8 : 4;
    static constexpr int SLAB = BN / (EPI_WARPS / 4);       // columns per epilogue warp
    static constexpr int TMEM_COLS = 2 * BN <= 64 ? 64 : 2 * BN <= 128 ? 128 : 2 * BN <= 256 ? 256 : 512;
    static constexpr int THREADS = (2 + EPI_WARPS) * 32;
    static constexpr int BARS = 3 * STAGES + 5;
    static constexpr int STG = STG_, STAGING = EPI_WARPS * STG * 4;
    // Ring, barriers (8 bytes each), TMEM address (16), epilogue staging;
    // the group tables of kRagN / kRagK follow.
    static constexpr int FIXED = STAGES * STAGE_BYTES + ((BARS * 8 + 16 + 15) / 16) * 16 + STAGING + 1024;
    static_assert(BN % 32 == 0 && SLAB % 32 == 0 && B_BYTES % 1024 == 0, "tile");
    static_assert(FIXED <= 227 * 1024, "shared memory per CTA");
};

struct LmWork {
    int m0, n0;          // first row, first column of D
    int nmma, nvalid;    // columns multiplied, columns that exist
    int kb0, nkb;        // blocks of 64 of the contraction
    int krow0, klast;    // kRagK: first token row, rows in the last block
    int g, s;            // group, K split
};

// Ends of the groups -> start rows and (kRagN) the running number of tiles,
// by one warp.  Ends that run backwards or past T are pulled into range
// (every access stays inside the operands) and reported (kSiteGroupEnds).
// Entry G is a group of its own, the rows behind the last end, which get zeros.
// EARLY: the kernel has not waited yet, and nothing says that L1 holds no older copy:
// they are read past it.  (128 rows in 1024 groups, 256 x 256, f16: 19.3 us if so,
// 18.5 if not.)
template <class Tile, int RAG, bool EARLY = false>
__device__ __forceinline__ void lm_group_tables(const LmArgs &p, int *start, uint32_t *prefix, int lane) {
    int row = 0;
    uint32_t tiles = 0;
    bool bad = false;
    auto end_of = [&](int g) -> int {
        if (g >= p.G) return p.T;
        return EARLY ? (int)ld_relaxed_gpu(reinterpret_cast<const uint32_t *>(p.ends + g)) : p.ends[g];
    };
    int following = end_of(lane);
    for (int g0 = 0; g0 <= p.G; g0 += 32) {
        const int g = g0 + lane;
        int e = following;
        following = end_of(g + 32);
        bad |= e < 0 || e > p.T;
        e = min(max(e, 0), p.T);
        int top = e;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(~0u, top, d);
            if (lane >= d) top = max(top, o);
        }
        top = max(top, row);
        bad |= top != e;
        int first = __shfl_up_sync(~0u, top, 1);
        if (lane == 0) first = row;
        if (g <= p.G) start[g] = first;
        if (g == p.G) start[p.G + 1] = p.T;
        row = __shfl_sync(~0u, top, 31);
        if constexpr (RAG == kRagN) {
            uint32_t n = g <= p.G ? (uint32_t)((top - first + p.tile_n - 1) / p.tile_n) * (uint32_t)p.tiles_m : 0u;
            uint32_t sum = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t o = __shfl_up_sync(~0u, sum, d);
                if (lane >= d) sum += o;
            }
            if (g <= p.G) prefix[g] = tiles + sum - n;
            tiles += __shfl_sync(~0u, sum, 31);
            if (g == p.G) prefix[p.G + 1] = tiles;
        }
    }
    if (__any_sync(~0u, bad) && lane == 0 && blockIdx.x == 0) record_error(p.err, kSiteGroupEnds);
}

template <class Tile, int RAG>
__device__ __forceinline__ LmWork lm_work(const LmArgs &p, const int *start, const uint32_t *prefix, int t) {
    LmWork w;
    w.s = 0;
    w.kb0 = 0;
    w.krow0 = 0;
    w.klast = 64;
    if constexpr (RAG == kRagN) {
        w.s = t % p.splits;
        t /= p.splits;
        int lo = 0, hi = p.G;                   // last g with prefix[g] <= t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= (uint32_t)t) lo = mid;
            else hi = mid - 1;
        }
        w.g = lo;
        const int local = t - (int)prefix[lo];
        const int r0 = start[lo], rows = start[lo + 1] - r0;
        const int nt = (rows + p.tile_n - 1) / p.tile_n;
        // Columns spread evenly over the group's tiles.
        const int per = ((rows + nt - 1) / nt + Tile::GRAN - 1) / Tile::GRAN * Tile::GRAN;
        const int band = local / (p.group_m * nt), in = local - band * p.group_m * nt;
        const int bw = min(p.group_m, p.tiles_m - band * p.group_m);
        const int tn = in / bw, tm = band * p.group_m + in - tn * bw;
        w.m0 = tm * Tile::TILE_M;
        w.n0 = r0 + tn * per;
        w.nvalid = min(per, rows - tn * per);
        w.nmma = (w.nvalid + Tile::GRAN - 1) / Tile::GRAN * Tile::GRAN;
        w.kb0 = (int)((int64_t)p.kb * w.s / p.splits);
        w.nkb = lo == p.G ? 0 : (int)((int64_t)p.kb * (w.s + 1) / p.splits) - w.kb0;
    } else if constexpr (RAG == kRagK) {
        const int per_g = p.tiles_m * p.tiles_n, at = t / per_g;
        w.g = (int)prefix[at];                  // the groups in their order of work
        const int in = t - at * per_g;
        const int tn = in / p.tiles_m, tm = in - tn * p.tiles_m;
        const int rows = start[w.g + 1] - start[w.g];
        w.m0 = tm * Tile::TILE_M;
        w.n0 = tn * p.tile_n;
        w.nvalid = min(p.tile_n, p.N - w.n0);
        w.nmma = p.tile_n;
        w.krow0 = start[w.g];
        w.nkb = (rows + 63) >> 6;
        w.klast = rows - ((w.nkb - 1) << 6);
    } else {
        w.g = 0;
        const int tile = t / p.splits;
        w.s = t - tile * p.splits;
        const int per_band = p.group_m * p.tiles_n;
        const int band = tile / per_band, in = tile - band * per_band;
        const int bw = min(p.group_m, p.tiles_m - band * p.group_m);
        const int tn = in / bw, tm = band * p.group_m + in - tn * bw;
        w.m0 = tm * Tile::TILE_M;
        w.n0 = tn * p.tile_n;
        w.nvalid = min(p.tile_n, p.N - w.n0);
        w.nmma = p.tile_n;
        w.kb0 = (int)((int64_t)p.kb * w.s / p.splits);
        w.nkb = (int)((int64_t)p.kb * (w.s + 1) / p.splits) - w.kb0;
    }
    return w;
}

// kRagK: the order in which the groups are worked on, largest first (prefix
// holds it): a group's tiles cost what it is long, and what is left over in
// the last round is short.  Empty groups come before all, their zeros are
// written while the first products run.  4096 rows of 1024 x 2048 over 8
// groups, FP32: 135 -> 113, 122 -> 117, 157 -> 138, 127 -> 110 us (four sets of
// sizes); 8192 rows of 2048 x 5632, F16: 127 -> 126, 131 -> 133, 142 -> 139,
// 134 -> 126.  (Dealt out forth and back instead of round by round: up to
// 20% longer.)  The order costs a step per group; of more than 256 groups,
// whose tiles are many and even out, they stay as they are.
constexpr int kLmSortedGroups = 256;
__device__ __forceinline__ void lm_order_groups(const LmArgs &p, const int *start, uint32_t *order) {
    for (int g = threadIdx.x; g < p.G; g += blockDim.x) {
        int at = g;
        if (p.G <= kLmSortedGroups) {
            // (An empty group's size wraps to the largest.)
            const uint32_t rows = (uint32_t)(start[g + 1] - start[g]) - 1u;
            int from = start[0];
            at = 0;
            for (int h = 0; h < p.G; ++h) {
                const int to = start[h + 1];
                const uint32_t n = (uint32_t)(to - from) - 1u;
                at += n > rows || (n == rows && h < g);
                from = to;
            }
        }
        order[at] = (uint32_t)g;
    }
}

// A product of FP32 operands, each held as three bf16 planes (x = p0 + p1 +
// p2, lm_aux.cu): stage i of a block of 64 holds plane i of both, and p_i q_j
// with i + j <= 2 are multiplied, smallest first.
__device__ constexpr int plane_a(int pr) { return (0x046 >> (2 * pr)) & 3; }     // 2 1 0 1 0 0
__device__ constexpr int plane_b(int pr) { return (0x124 >> (2 * pr)) & 3; }     // 0 1 2 0 1 0

// -------------------------------------------------------------- epilogues

// 32 columns of this lane's row of D, as a piece of a row-major matrix (VEC: of
// one whose rows always take vector stores).
template <bool VEC, class Out>
__device__ __forceinline__ void lm_store_rows(const LmArgs &p, Out *base, int row, int row0, int col, int cnt,
                                              const float (&v)[32], float *stg, int lane) {
    if (VEC || p.vec) {
        if (row >= p.M) return;
        Out *c = base + (int64_t)row * p.ldc + col;
        if (cnt == 32) {
            if constexpr (sizeof(Out) == 2) {
                uint32_t u[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) u[i] = lm_pack2<Out>(v[2 * i], v[2 * i + 1]);
                st_global_32B(c, u);
                st_global_32B(c + 16, u + 8);
            } else {
                uint32_t u[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(v[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) st_global_32B(c + 8 * i, u + 8 * i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < cnt) c[i] = lm_cvt<Out>(v[i]);
        }
    } else if constexpr (sizeof(Out) == 2) {
        // Rows that vector stores cannot reach: turned in shared memory, so
        // that a warp writes 32 neighbours of one row at a time (rows 34
        // elements apart there: no bank is met twice).
        uint32_t *words = reinterpret_cast<uint32_t *>(stg);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) words[lane * 17 + i] = lm_pack2<Out>(v[2 * i], v[2 * i + 1]);
        __syncwarp();
        const Out *from = reinterpret_cast<const Out *>(stg) + lane;
        Out *to = base + (int64_t)row0 * p.ldc + col + lane;
        if (lane < cnt) {
            if (row0 + 32 <= p.M) {
#pragma unroll
                for (int r = 0; r < 32; ++r) to[(int64_t)r * p.ldc] = from[r * 34];
            } else {
                for (int r = 0; row0 + r < p.M; ++r) to[(int64_t)r * p.ldc] = from[r * 34];
            }
        }
    } else {
        // The same for FP32, half a warp on 16 neighbours of a row.
        const int c = lane & 15, rr = lane >> 4;
#pragma unroll
        for (int h = 0; h < 32; h += 16) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; ++i) stg[lane * 17 + i] = v[h + i];
            __syncwarp();
            if (h + c < cnt)
#pragma unroll 8
                for (int r = rr; r < 32; r += 2)
                    if (row0 + r < p.M) base[(int64_t)(row0 + r) * p.ldc + col + h + c] = lm_cvt<Out>(stg[r * 17 + c]);
        }
    }
}

// 32 columns of D are 32 token rows of the output; this lane holds output
// column f of each.
template <class Out>
__device__ __forceinline__ void lm_store_cols(const LmArgs &p, Out *base, int f0, int tok, int cnt,
                                              const float (&v)[32], float *stg, int lane) {
    if (sizeof(Out) == 4 || !p.vec) {
        const int f = f0 + lane;
        if (f >= p.M) return;
        Out *c = base + (int64_t)tok * p.ldc + f;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < cnt) c[(int64_t)j * p.ldc] = lm_cvt<Out>(v[j]);
        return;
    }
    if constexpr (sizeof(Out) == 2) {
        // Through shared memory: 16 bytes of one token row per lane.
        Out *s = reinterpret_cast<Out *>(stg);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 32; ++j) s[j * 32 + lane] = lm_cvt<Out>(v[j]);
        __syncwarp();
        const int f = f0 + (lane & 3) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = i * 8 + (lane >> 2);
            if (j >= cnt) continue;
            Out *c = base + (int64_t)(tok + j) * p.ldc + f;
            const Out *src = s + j * 32 + (lane & 3) * 8;
            if (f + 8 <= p.M) {
                *reinterpret_cast<uint4 *>(c) = *reinterpret_cast<const uint4 *>(src);
            } else {
                for (int e = 0; e < 8; ++e)
                    if (f + e < p.M) c[e] = src[e];
            }
        }
    }
}

// A wait that lasts as long as work that goes on (the whole contraction of a
// tile, or tiles without a tail): its limit starts anew while this SM's
// producer issues copies, and it gives up when none was issued for as long as
// the limit.  `issued` only grows, and only as far as there are stages to fill.
// (A fixed limit ran out in correct calls: 1000001 rows in one group, 1 ms.)
template <bool CLUSTER>
__device__ __forceinline__ bool lm_wait_working(uint64_t *bar, uint32_t parity, uint64_t limit,
                                                const volatile uint32_t *issued) {
    uint32_t seen = *issued;
    while (!mbar_wait_bounded<CLUSTER>(bar, parity, limit)) {
        const uint32_t now = *issued;
        if (now == seen) return false;
        seen = now;
    }
    return true;
}

// kRagK, a group's last block of rows: once this SM's copies have landed,
// the warp clears the rows behind the group (they belong to others) up to the
// next multiple of 16, where the MMAs stop; both operands, so that an
// infinity there does not meet a zero.  False if the copies did not land.
template <class Tile>
__device__ __forceinline__ bool lm_clear_tail(unsigned char *stage, uint64_t *landed, uint32_t parity, int rows,
                                              const LmArgs &p, const volatile uint32_t *issued, int lane) {
    // (All tiles since the last tail lie between: those of other groups too.)
    bool ok = lm_wait_working<false>(landed, parity, downstream_limit(p.timeout_ns), issued);
    if (!ok && lane == 0) record_error(p.err, kSiteConsumerFull);
    ok = __all_sync(~0u, ok);
    const int r1 = (rows + 15) & ~15, per = (r1 - rows) * 8;      // 16-byte words per chunk of 64 columns
    constexpr int CHUNKS = Tile::STAGE_BYTES / 8192;
    if (ok)
        for (int i = lane; i < per; i += 32)
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c)
                *reinterpret_cast<uint4 *>(stage + c * 8192 + rows * 128 + i * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
    return ok;
}

// MODE of a kernel: 16-bit operands in one running sum; the same in runs of
// eight blocks, or, where a contraction may be long, of 128; FP32 operands in
// three planes, summed block by block.
constexpr int kPlain = 0, kRuns = 1, kLong = 2, kPlanes = 3;

// ---------------------------------------------------------------- kernel

// Threads of a kernel: kRagK has one more warp, which clears tails.
template <class Tile, int RAG>
constexpr int lm_threads() { return Tile::THREADS + (RAG == kRagK ? 32 : 0); }

template <class Tile, bool A_MN, bool B_MN, int RAG, int EPI, int MODE>
__global__ void __launch_bounds__(lm_threads<Tile, RAG>(), 1)
lm_mma_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const LmArgs p) {
    constexpr bool PAIR = Tile::PAIR;
    constexpr int BN = Tile::BN, STAGES = Tile::STAGES, SLAB = Tile::SLAB;
    constexpr bool CHUNKED = MODE != kPlain;
    constexpr int PLANES = MODE == kPlanes ? 3 : 1, CH = MODE == kRuns ? 8 : MODE == kLong ? 128 : 1;
    static_assert((CH & (CH - 1)) == 0, "");
    static_assert(!B_MN || Tile::B_ROWS % 64 == 0, "MN-major B is staged in chunks of 64 columns");

    extern __shared__ unsigned char smem_raw[];
    const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
    unsigned char *smem = smem_raw + pad;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + STAGES * Tile::STAGE_BYTES);
    uint64_t *full = bars;                  // TMA -> MMA
    uint64_t *empty = bars + STAGES;        // MMA -> TMA
    uint64_t *tfull = bars + 2 * STAGES;    // MMA -> epilogue, per accumulator
    uint64_t *tempty = tfull + 2;           // epilogue -> MMA, per accumulator
    uint64_t *drain = tempty + 2;           // MMA completion before teardown
    uint64_t *tailbar = drain + 1;          // kRagK, per stage: this SM's copies of a group's last block
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + Tile::BARS);
    volatile uint32_t *progress = tmem_slot + 1;    // stages the producer has issued, each time round
    unsigned char *after = reinterpret_cast<unsigned char *>(bars) + ((Tile::BARS * 8 + 16 + 15) / 16) * 16;
    float *staging = reinterpret_cast<float *>(after);
    int *g_start = reinterpret_cast<int *>(after + Tile::STAGING);
    uint32_t *g_prefix = reinterpret_cast<uint32_t *>(g_start + p.G + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_rank() : 0u;

    if (warp == 0) {
        if constexpr (PAIR) tmem_alloc_pair(tmem_slot, Tile::TMEM_COLS);
        else tmem_alloc(tmem_slot, Tile::TMEM_COLS);
    }
    if (threadIdx.x == 32) {
        for (int s = 0; s < STAGES; ++s) {
            // kRagK on a pair: the other SM arrives as well (it may have to
            // clear rows of a group's last block first).
            mbar_init(&full[s], PAIR && RAG == kRagK ? 2 : 1);
            mbar_init(&empty[s], 1);
            mbar_init(&tailbar[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], (PAIR ? 2 : 1) * Tile::EPI_WARPS);
        }
        mbar_init(drain, 1);
        *progress = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
    }
    griddep_launch_dependents();
    griddep_wait();
    if constexpr (RAG != kRagNone)
        if (warp == 2) lm_group_tables<Tile, RAG>(p, g_start, g_prefix, lane);
    if constexpr (RAG == kRagK) {
        __syncthreads();
        lm_order_groups(p, g_start, g_prefix);
    }
    tc_fence_before();
    __syncwarp();               // (the barriers, too, take whole warps)
    if constexpr (PAIR) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(tmem_slot);
    const int slot = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
    const int slots = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;
    const int num_tiles = RAG == kRagN ? (int)g_prefix[p.G + 1] * p.splits : p.num_tiles;

    if (warp == 0) {
        // ---------------- TMA producer (one elected lane issues) ----------------
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        // K-major B is copied in as many rows as a tile may have.
        const uint32_t stage_bytes =
            B_MN ? (uint32_t)Tile::STAGE_BYTES : (uint32_t)(Tile::A_BYTES + p.tile_n / (PAIR ? 2 : 1) * 128);
        const uint32_t full_pair = PAIR ? cluster_addr(&full[0], 0) : 0u;   // rank 0's barriers
        for (int t = slot; ok && t < num_tiles; t += slots) {
            const LmWork w = lm_work<Tile, RAG>(p, g_start, g_prefix, t);
            const int ma = w.m0 + (int)rank * Tile::BM;
            const int nb = w.n0 + (int)rank * (w.nmma >> 1);
            for (int kb = 0; ok && kb < w.nkb; ++kb) {
                // kRagNone: A may have a second plane, which goes over the same B.
                const int again = RAG == kRagNone && w.kb0 + kb >= p.kb_plane ? 1 : 0;
                const int kc = RAG == kRagK ? w.krow0 + kb * 64 : (w.kb0 + kb - again * p.kb_plane) * 64;
                const bool tail = RAG == kRagK && kb == w.nkb - 1 && (w.klast & 15) != 0;
                for (int pl = 0; pl < PLANES; ++pl) {
                    if (p.withhold == kWithholdRefill && issued >= STAGES) { ok = false; break; }
                    if (!mbar_wait_bounded<PAIR>(&empty[stage], phase ^ 1u, p.timeout_ns)) {
                        if (lane == 0) record_error(p.err, kSiteProducerEmpty);
                        ok = false;
                    }
                    ok = __all_sync(~0u, ok);
                    if (!ok) break;
                    unsigned char *sa = smem + stage * Tile::STAGE_BYTES, *sb = sa + Tile::A_BYTES;
                    const int za = RAG == kRagN ? pl * p.G + w.g : pl + again;
                    const uint32_t fb = full_pair + (uint32_t)stage * 8u;
                    // Copies of this stage, completing on the ring's barrier
                    // (rank 0's for a pair) or, for a tail, on a local one.
                    auto load_all = [&](auto &&load) {
                        if constexpr (A_MN) {
                            load(sa, &tmA, ma, kc, za);
                            load(sa + 8192, &tmA, ma + 64, kc, za);
                        } else {
                            load(sa, &tmA, kc, ma, za);
                        }
                        if constexpr (B_MN) {
#pragma unroll
                            for (int c = 0; c < Tile::B_ROWS / 64; ++c)
                                load(sb + c * 8192, &tmB, nb + c * 64, kc, pl);
                        } else {
                            load(sb, &tmB, kc, nb, pl);
                        }
                    };
                    if (!tail) {
                        if (elect_one()) {
                            if constexpr (PAIR) {
                                if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * stage_bytes);
                                else if (RAG == kRagK) mbar_arrive_cluster_relaxed(fb);
                                load_all([&](void *dst, const CUtensorMap *m, int c0, int c1, int c2) {
                                    tma_load_3d_pair(dst, m, fb, c0, c1, c2);
                                });
                            } else {
                                mbar_arrive_expect_tx(&full[stage], stage_bytes);
                                load_all([&](void *dst, const CUtensorMap *m, int c0, int c1, int c2) {
                                    tma_load_3d(dst, m, &full[stage], c0, c1, c2);
                                });
                            }
                        }
                        __syncwarp();
                    } else {
                        // Rows behind the group have to be cleared first: the
                        // copies report to this SM's own barrier, and the
                        // warp that clears (lm_clear_tail) arrives in this
                        // one's place.
                        if (elect_one()) {
                            mbar_arrive_expect_tx(&tailbar[stage], Tile::STAGE_BYTES);
                            load_all([&](void *dst, const CUtensorMap *m, int c0, int c1, int c2) {
                                tma_load_3d(dst, m, &tailbar[stage], c0, c1, c2);
                            });
                        }
                        __syncwarp();
                    }
                    ++issued;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                        // (Each time round, and not by the lane whose arrivals
                        // would wait for it: every stage cost 3%.)
                        if (lane == 31) *progress = (uint32_t)issued;
                    }
                }
            }
        }
        if (!ok) {
            // Let this CTA's own copies land before it can exit (rank 1 of
            // a pair sees them as the release of its stages).
            const int pending = issued < STAGES ? issued : STAGES;
            for (int back = 1; back <= pending; ++back) {
                int s = stage - back;
                uint32_t ph = phase;
                if (s < 0) { s += STAGES; ph ^= 1u; }
                mbar_wait_bounded<PAIR>(rank == 0 ? &full[s] : &empty[s], ph, p.timeout_ns);
            }
        }
    } else if (warp == 1 && rank == 0) {
        // ---------------- MMA issuer (rank 0 of a pair) ----------------
        // The whole warp walks the loop and one elected lane issues: with
        // the control flow uniform, descriptors stay in uniform registers,
        // where the MMA takes them.  (Under a branch on the lane number the
        // issue of a stage's four MMAs took longer than their execution.)
        const uint64_t da0 = A_MN ? smem_desc_mn_sw128(smem_u32(smem)) : smem_desc_k_sw128(smem_u32(smem));
        const uint64_t db0 = B_MN ? smem_desc_mn_sw128(smem_u32(smem) + Tile::A_BYTES)
                                  : smem_desc_k_sw128(smem_u32(smem) + Tile::A_BYTES);
        constexpr uint64_t KA = A_MN ? 2048 >> 4 : 32 >> 4, KB = B_MN ? 2048 >> 4 : 32 >> 4;   // per 16 of K
        int stage = 0, gc = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = slot; ok && t < num_tiles; t += slots) {
            const LmWork w = lm_work<Tile, RAG>(p, g_start, g_prefix, t);
            const uint32_t idesc = idesc_f16(p.bf16, A_MN, B_MN, Tile::TILE_M, w.nmma);
            uint32_t d_tmem = 0;
            // The last block of a group's rows may be short: kept out of the
            // loop, whose instructions have to stay ahead of the tensor core.
            const int whole = RAG == kRagK && w.nkb > 0 && w.klast < 64 ? w.nkb - 1 : w.nkb;
            for (int kb = 0; kb < whole; ++kb) {
                const bool first = CHUNKED ? (kb & (CH - 1)) == 0 : kb == 0;
                const bool last = kb == w.nkb - 1 || (CHUNKED && (kb & (CH - 1)) == CH - 1);
                if (first) {
                    const int ab = gc & 1;
                    if (!mbar_wait_bounded<PAIR>(&tempty[ab], ((uint32_t)(gc >> 1) & 1u) ^ 1u, p.timeout_ns)) {
                        if (lane == 0) record_error(p.err, kSiteConsumerFull);
                        ok = false;
                    }
                    ok = __all_sync(~0u, ok);
                    if (!ok) break;
                    tc_fence_after();
                    d_tmem = tmem_base + (uint32_t)(ab * BN);
                }
                uint64_t da[PLANES], db[PLANES];
                int st[PLANES];
#pragma unroll
                for (int pl = 0; pl < PLANES; ++pl) {
                    if (ok && !mbar_wait_bounded<PAIR>(&full[stage], phase, downstream_limit(p.timeout_ns))) {
                        if (lane == 0) record_error(p.err, kSiteConsumerFull);
                        ok = false;
                    }
                    ok = __all_sync(~0u, ok);
                    da[pl] = da0 + (uint64_t)(stage * (Tile::STAGE_BYTES >> 4));
                    db[pl] = db0 + (uint64_t)(stage * (Tile::STAGE_BYTES >> 4));
                    st[pl] = stage;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int pr = 0; pr < (PLANES == 3 ? 6 : 1); ++pr) {
                        const uint64_t a = da[PLANES == 3 ? plane_a(pr) : 0], b = db[PLANES == 3 ? plane_b(pr) : 0];
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const uint32_t acc = first && pr == 0 && kk == 0 ? 0u : 1u;
                            if constexpr (PAIR) mma_f16_pair(d_tmem, a + kk * KA, b + kk * KB, idesc, acc);
                            else mma_f16(d_tmem, a + kk * KA, b + kk * KB, idesc, acc);
                        }
                    }
                    if (p.withhold != kWithholdRelease) {
#pragma unroll
                        for (int pl = 0; pl < PLANES; ++pl) {
                            if constexpr (PAIR) mma_commit_pair_mc(&empty[st[pl]], 0x3);
                            else mma_commit(&empty[st[pl]]);
                        }
                    }
                    if (last) {
                        if constexpr (PAIR) mma_commit_pair_mc(&tfull[gc & 1], 0x3);
                        else mma_commit(&tfull[gc & 1]);
                    }
                }
                __syncwarp();
                if (!ok) break;
                if (last) ++gc;
            }
            if constexpr (RAG == kRagK) {
                if (ok && whole < w.nkb) {
                    const bool first = CHUNKED ? (whole & (CH - 1)) == 0 : whole == 0;
                    const int steps = (w.klast + 15) >> 4, ab = gc & 1;
                    if (first) {
                        ok = mbar_wait_bounded<PAIR>(&tempty[ab], ((uint32_t)(gc >> 1) & 1u) ^ 1u, p.timeout_ns);
                        if (!ok && lane == 0) record_error(p.err, kSiteConsumerFull);
                        tc_fence_after();
                        d_tmem = tmem_base + (uint32_t)(ab * BN);
                    }
                    uint64_t da[PLANES], db[PLANES];
                    int st[PLANES];
#pragma unroll
                    for (int pl = 0; pl < PLANES; ++pl) {
                        ok = ok && mbar_wait_bounded<PAIR>(&full[stage], phase, 2 * downstream_limit(p.timeout_ns));
                        if (!ok && lane == 0) record_error(p.err, kSiteConsumerFull);
                        ok = __all_sync(~0u, ok);
                        da[pl] = da0 + (uint64_t)(stage * (Tile::STAGE_BYTES >> 4));
                        db[pl] = db0 + (uint64_t)(stage * (Tile::STAGE_BYTES >> 4));
                        st[pl] = stage;
                        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    }
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int pr = 0; pr < (PLANES == 3 ? 6 : 1); ++pr) {
                            const uint64_t a = da[PLANES == 3 ? plane_a(pr) : 0], b = db[PLANES == 3 ? plane_b(pr) : 0];
                            for (int kk = 0; kk < steps; ++kk) {
                                const uint32_t acc = first && pr == 0 && kk == 0 ? 0u : 1u;
                                if constexpr (PAIR) mma_f16_pair(d_tmem, a + kk * KA, b + kk * KB, idesc, acc);
                                else mma_f16(d_tmem, a + kk * KA, b + kk * KB, idesc, acc);
                            }
                        }
                        if (p.withhold != kWithholdRelease) {
#pragma unroll
                            for (int pl = 0; pl < PLANES; ++pl) {
                                if constexpr (PAIR) mma_commit_pair_mc(&empty[st[pl]], 0x3);
                                else mma_commit(&empty[st[pl]]);
                            }
                        }
                        if constexpr (PAIR) mma_commit_pair_mc(&tfull[ab], 0x3);
                        else mma_commit(&tfull[ab]);
                    }
                    __syncwarp();
                    ++gc;
                }
            }
        }
        if (elect_one()) {
            if constexpr (PAIR) mma_commit_pair(drain);
            else mma_commit(drain);
        }
        __syncwarp();
        mbar_wait_bounded(drain, 0u, p.timeout_ns);
    } else if (RAG == kRagK && warp == 2 + Tile::EPI_WARPS) {
        // ---------------- clears the tails, ahead of the MMAs ----------------
        int stage = 0;
        uint32_t phases = 0;                    // of the tail barriers, a bit each
        bool ok = true;
        for (int t = slot; ok && t < num_tiles; t += slots) {
            const LmWork w = lm_work<Tile, RAG>(p, g_start, g_prefix, t);
            const bool tail = w.nkb > 0 && (w.klast & 15) != 0;
            stage = (stage + (w.nkb - (tail ? 1 : 0)) * PLANES) % STAGES;
            for (int pl = 0; tail && ok && pl < PLANES; ++pl) {
                ok = lm_clear_tail<Tile>(smem + stage * Tile::STAGE_BYTES, &tailbar[stage], (phases >> stage) & 1u,
                                         w.klast, p, progress, lane);
                phases ^= 1u << stage;
                if (ok && lane == 0) {
                    if (rank == 0) mbar_arrive(&full[stage]);
                    else mbar_arrive_cluster(cluster_addr(&full[stage], 0));
                }
                stage = stage + 1 == STAGES ? 0 : stage + 1;
            }
        }
    } else if (warp >= 2 && warp < 2 + Tile::EPI_WARPS) {
        // ---------------- epilogue ----------------
        const int quarter = warp & 3, ew = warp - 2;
        const int slab0 = (ew >> 2) * SLAB;
        float *stg = staging + ew * Tile::STG;
        const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16);
        int gc = 0;
        bool ok = true;
        float alpha = 1.f;
        if (EPI == kEpiRows && p.alpha != nullptr) alpha = *p.alpha;
        if (EPI == kEpiDLogits && p.gscale != nullptr) alpha = *p.gscale;
        for (int t = slot; ok && t < num_tiles; t += slots) {
            const LmWork w = lm_work<Tile, RAG>(p, g_start, g_prefix, t);
            float sum[CHUNKED ? SLAB : 1];
            uint32_t taddr = 0;
            auto wait_acc = [&]() {
                ok = __all_sync(~0u, lm_wait_working<PAIR>(&tfull[gc & 1], (uint32_t)(gc >> 1) & 1u,
                                                           downstream_limit(p.timeout_ns), progress));
                if (!ok && lane == 0) record_error(p.err, kSiteConsumerFull);
                tc_fence_after();
                taddr = lane_base + (uint32_t)((gc & 1) * BN + slab0);
            };
            auto release_acc = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    // Only the loads from tensor memory have to come before (they
                    // are complete, and fenced); a release would wait for the
                    // stores of the tile before, too.
                    if constexpr (PAIR) mbar_arrive_cluster_relaxed(cluster_addr(&tempty[gc & 1], 0));
                    else mbar_arrive(&tempty[gc & 1]);
                }
                ++gc;
            };
            const int row0 = w.m0 + (int)rank * Tile::BM + quarter * 32;   // first row of this warp
            const int row = row0 + lane;
            // Per-row state of the loss epilogues.
            float run_max = -INFINITY, run_sum = 0.f, row_lse = 0.f, row_g = 0.f;
            int tgt = -1;
            if constexpr (EPI == kEpiLse || EPI == kEpiDLogits) {
                if (row < p.M) {
                    const int64_t tv = p.target[row];
                    // (All on their way together; of a token that is not
                    // counted they are not used.)
                    float lse = 0.f, grad = 0.f;
                    if constexpr (EPI == kEpiDLogits) {
                        lse = p.lse[row];
                        grad = p.grad[row];
                    }
                    if (tv >= 0 && tv < p.vocab) {
                        const int64_t rel = tv - p.v0;
                        tgt = rel >= 0 && rel < p.N ? (int)rel : -1;
                        row_lse = lse;
                        row_g = grad * alpha;
                    }
                }
            }
            // The tile's columns, out of tensor memory or from `sum`.
            auto store_tile = [&](auto from_sum) {
                uint32_t next[32];
#pragma unroll
                for (int c0 = 0; c0 < SLAB; c0 += 32) {
                    const int col = slab0 + c0;                 // column in the tile
                    if (col < w.nvalid && (EPI == kEpiCols || row0 < p.M)) {
                        float v[32];
                        if constexpr (decltype(from_sum)::value) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = sum[c0 + i];
                        } else if (w.nkb > 0) {
                            // The next 32 columns are on their way while these
                            // are worked on.
                            if (c0 == 0) tmem_ld_32cols_nowait(taddr, next);
                            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(next[i]);
                            if (c0 + 32 < SLAB && col + 32 < w.nvalid)
                                tmem_ld_32cols_nowait(taddr + (uint32_t)(c0 + 32), next);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = 0.f;
                        }
                        const int cnt = min(32, w.nvalid - col);
                        const int n = w.n0 + col;               // column of D
                        if constexpr (EPI == kEpiCols) {
                            if (p.out == kOutF32)
                                lm_store_cols(p, static_cast<float *>(p.C) + w.s * p.stride_c, row0, n, cnt, v, stg, lane);
                            else if (p.out == kOutF16)
                                lm_store_cols(p, static_cast<__half *>(p.C), row0, n, cnt, v, stg, lane);
                            else
                                lm_store_cols(p, static_cast<__nv_bfloat16 *>(p.C), row0, n, cnt, v, stg, lane);
                        } else if constexpr (EPI == kEpiLse) {
                            if (cnt < 32)
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if (i >= cnt) v[i] = -INFINITY;
                            float bm = v[0];
#pragma unroll
                            for (int i = 1; i < 32; ++i) bm = fmaxf(bm, v[i]);
                            const float nm = fmaxf(run_max, bm);
                            const float ref = (nm == -INFINITY ? 0.f : nm) * kLog2E;
                            float s = run_sum * exp2_approx(fmaf(run_max, kLog2E, -ref));
#pragma unroll
                            for (int i = 0; i < 32; ++i) s += exp2_approx(fmaf(v[i], kLog2E, -ref));
                            run_sum = s;
                            run_max = nm;
                            const int rel = tgt - n;
                            if (rel >= 0 && rel < cnt) {
                                float pick = v[0];
#pragma unroll
                                for (int i = 1; i < 32; ++i)
                                    if (i == rel) pick = v[i];
                                p.picked[row] = pick;
                            }
                        } else {
                            if constexpr (EPI == kEpiDLogits) {
                                // exp(x) as the square of exp(x / 2), whose product
                                // keeps results below 2^-126 (gradients of
                                // improbable entries).
                                const int rel = tgt - n;
#pragma unroll
                                for (int i = 0; i < 32; ++i) {
                                    const float h = exp2_approx((v[i] - row_lse) * (0.5f * kLog2E));
                                    v[i] = h * h;
                                }
                                if (rel >= 0 && rel < 32)
#pragma unroll
                                    for (int i = 0; i < 32; ++i)
                                        if (i == rel) v[i] -= 1.f;
#pragma unroll
                                for (int i = 0; i < 32; ++i) v[i] *= row_g;
                                if (row_g == 0.f)
#pragma unroll
                                    for (int i = 0; i < 32; ++i) v[i] = 0.f;
                            } else {
                                if (p.acc_in != nullptr && row < p.M) {
                                    const float *a = p.acc_in + (int64_t)row * p.ld_acc + n;
#pragma unroll
                                    for (int i = 0; i < 32; ++i)
                                        if (i < cnt) v[i] += a[i];
                                }
#pragma unroll
                                for (int i = 0; i < 32; ++i) v[i] *= alpha;
                            }
                            const int64_t z = (int64_t)(RAG == kRagK ? w.g : w.s) * p.stride_c;
                            if (EPI == kEpiDLogits && MODE != kPlanes && !PAIR && p.lo != nullptr) {
                                // What the rounding to 16 bits leaves, in a plane of its own.
                                float rest[32];
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    rest[i] = v[i] - (p.out == kOutF16 ? __half2float(__float2half_rn(v[i]))
                                                                       : __bfloat162float(__float2bfloat16_rn(v[i])));
                                if (p.out == kOutF16)
                                    lm_store_rows<true>(p, static_cast<__half *>(p.lo), row, row0, n, cnt, rest, stg, lane);
                                else
                                    lm_store_rows<true>(p, static_cast<__nv_bfloat16 *>(p.lo), row, row0, n, cnt, rest, stg, lane);
                            }
                            // (d has the operands' type.)
                            if (EPI == kEpiDLogits ? MODE == kPlanes : p.out == kOutF32)
                                lm_store_rows<EPI == kEpiDLogits>(p, static_cast<float *>(p.C) + z, row, row0, n, cnt, v, stg, lane);
                            else if (p.out == kOutF16)
                                lm_store_rows<EPI == kEpiDLogits>(p, static_cast<__half *>(p.C) + z, row, row0, n, cnt, v, stg, lane);
                            else
                                lm_store_rows<EPI == kEpiDLogits>(p, static_cast<__nv_bfloat16 *>(p.C) + z, row, row0, n, cnt, v, stg, lane);
                        }
                        // Lanes without a row or column to store come back early; the
                        // next load from tensor memory takes the warp together.
                        __syncwarp();
                    }
                }
            };
            if (CHUNKED && (MODE != kLong || w.nkb > CH)) {
                // Runs of CH blocks of the contraction are summed in an
                // accumulator of their own and added here in FP32 with rounding
                // to nearest (the tensor core's own running sum truncates).
                // FP32 operands: one block (two doubled the error, at 40003
                // terms to 2^-20 of their magnitudes).  Logits of 16-bit
                // operands: eight (losses at 4096 terms off by 1.5 to 2e-7 of
                // themselves, about a unit in the last place, twice that with
                // sixteen, 1.7e-6 with one sum; gradients of 8192 rows, 32768 x
                // 4096, 3.96 ms, with sixteen 3.80), in the gradient as in the
                // loss: against an lse from other sums all probabilities are off
                // the same way, by 2% at logits of 2330.  Other sums of
                // 16-bit operands that may have more than 16384 terms: 128 (one
                // sum of a million terms of one sign is off by 0.6%, of 65536 by
                // 0.04%, a unit of f16's last place; runs of 8192 by 0.005%); a tile of
                // fewer goes the plain way.
#pragma unroll
                for (int c = 0; c < (CHUNKED ? SLAB : 1); ++c) sum[c] = 0.f;
                for (int kb = 0; ok && kb < w.nkb; kb += CH) {
                    wait_acc();
                    if (!ok) break;
#pragma unroll
                    for (int c0 = 0; c0 < SLAB; c0 += 32) {
                        if (slab0 + c0 < w.nvalid) {
                            uint32_t r[32];
                            tmem_ld_32cols_nowait(taddr + (uint32_t)c0, r);
                            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                            // (In pairs for the loss alone: forward pass of 8192
                            // rows, 32768 x 1024, 287 -> 278 us; with the other
                            // epilogues, whose registers are scarcer, no gain.)
                            if constexpr (EPI == kEpiLse) {
#pragma unroll
                                for (int i = 0; i < 32; i += 2)
                                    add2(sum[c0 + i], sum[c0 + i + 1], __uint_as_float(r[i]), __uint_as_float(r[i + 1]));
                            } else {
#pragma unroll
                                for (int i = 0; i < 32; ++i) sum[CHUNKED ? c0 + i : 0] += __uint_as_float(r[i]);
                            }
                        }
                    }
                    release_acc();
                }
                if (!ok) break;
                store_tile(std::integral_constant<bool, CHUNKED>());
            } else {
                if (w.nkb > 0) wait_acc();
                if (!ok) break;
                store_tile(std::false_type());
                if (w.nkb > 0) release_acc();
            }
            if constexpr (EPI == kEpiLse) {
                if (row < p.M)
                    p.part[(int64_t)((w.n0 / p.tile_n) * (BN / SLAB) + (ew >> 2)) * p.M + row] =
                        make_float2(run_max, run_sum);
            }
        }
    }

    // ---------------- teardown ----------------
    tc_fence_before();
    __syncwarp();               // (the barriers, too, take whole warps)
    if constexpr (PAIR) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    if (warp == 0) {
        if constexpr (PAIR) tmem_dealloc_pair(tmem_base, Tile::TMEM_COLS);
        else tmem_dealloc(tmem_base, Tile::TMEM_COLS);
    }
}

template <class Tile, bool A_MN, bool B_MN, int RAG, int EPI, int MODE>
LmKernel lm_kernel_info() {
    static_assert(MODE != kPlanes || Tile::STAGES >= 6, "two blocks of three planes in flight");
    static_assert(RAG == kRagNone || Tile::FIXED + 8 * (kLmMaxGroups + 2) <= 227 * 1024, "room for the group tables");
    LmKernel k;
    k.fn = reinterpret_cast<const void *>(&lm_mma_kernel<Tile, A_MN, B_MN, RAG, EPI, MODE>);
    k.threads = lm_threads<Tile, RAG>();
    k.smem = Tile::FIXED;
    k.tile_m = Tile::TILE_M;
    k.bn = Tile::BN;
    k.gran = Tile::GRAN;
    k.pair = Tile::PAIR ? 1 : 0;
    k.box_a = Tile::BM;
    k.a_mn = A_MN ? 1 : 0;
    return k;
}

using LmBig = LmTile<256, 6, true>;      // 256 x 256 on an SM pair
using LmBigBare = LmTile<256, 7, true, 0>;   // for epilogues without staging
using LmMid = LmTile<128, 6, false>;     // 128 x 128
using LmWide = LmTile<256, 4, false>;    // 128 x 256, for few rows against a long matrix
using LmThin = LmTile<32, 10, false>;    // 128 x 32, for few tokens

}  // namespace sg
