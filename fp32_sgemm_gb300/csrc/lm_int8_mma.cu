// Products of many rows of 8-bit integers with 8-bit weights, by group or not,
// on the tcgen05 tensor cores:
//
//   y[t, n] = sx[t] sw[n] sum_k x[t, k] w[n, k]
//
// sm_103a's tensor cores take no 8-bit integers, so both operands become f16
// (exactly).  x, which is small or needed by many tiles, is f16 in memory when
// the MMAs begin; the weights are read as the bytes they are and become f16 on
// their way into tensor memory, where the MMA takes its A operand from: a warp's
// lanes load a row of a 128-byte tile each, turn four bytes at a time into two
// pairs of f16 and store them to the lane's columns.  Through shared memory
// instead, the f16 weights would be written and read there beside x: 80 KB for
// 512 cycles of MMAs, which is more than it moves.
//
// Tiles, groups and SM pairs are those of lm_mma.cuh: 256 rows of W by up to 128 or
// 192 tokens (two accumulators, and two slots of converted W: the 512 columns of
// tensor memory).  An accumulator takes 1024 terms, whose sum FP32 holds exactly;
// the epilogue's warps add them up as 32-bit integers.
//
// Warps: 0 copies W, the last one x, 1 issues the MMAs, four or eight from 2 on
// convert, then eight are the epilogue.
//
// What bounds it, measured on one GB300 (quantisation included): the turns of the
// warps' loops, in which each waits for, does and tells little (with blocks of 128
// columns in tiles of 128 tokens a turn takes 900 cycles, its MMAs 512, whether W is
// converted or not), so a block is 256 columns; then the tensor core at the power
// limit: 2048 tokens, 8192 x 28672, 531 us, 1810 TFLOP/s; 8192 tokens, 4096 x 14336,
// 552 us, 1740; 2048 tokens, 4096 x 14336, 152 us (12 rounds of tiles); 256 tokens,
// 8192 x 28672, 80 us.  Few tokens: reading W, 32 tokens, 8192 x 28672, 52 us, 4.6
// TB/s; and beginning and end, 17 tokens, 4096 x 4096, 13 us.
#include <type_traits>

#include "lm_int8.h"
#include "lm_int8_round.cuh"
#include "lm_mma.cuh"

namespace sg {
namespace {

// BN: rows of x in a tile at most; BK: columns of K in a block.
template <int BN_, int BK_, int STAGES_, int CONV_>
struct Int8Tile {
    static constexpr int GRAN = 32, TILE_M = 256, BN = BN_, BK = BK_;
    static constexpr int STAGES = STAGES_, SLOTS = 2;
    static constexpr int W_CHUNK = 128 * 128, W_BYTES = BK / 128 * W_CHUNK, X_CHUNK = BN / 2 * 128, X_BYTES = BK / 64 * X_CHUNK;
    static constexpr int CONV_WARPS = CONV_, EPI_WARPS = 8, SLAB = BN / 2;
    static constexpr int CONV_COLS = BK / (CONV_WARPS / 4);         // of a converting warp (four reach all lanes)
    static constexpr int THREADS = (3 + CONV_WARPS + EPI_WARPS) * 32;
    static constexpr int TMEM_COLS = 512, SLOT0 = 2 * BN, SLOT_COLS = BK / 2;
    static constexpr int BARS = 4 * STAGES + 5;
    static constexpr int STG = 32 * 17, STAGING = EPI_WARPS * STG * 4;
    static constexpr int RING = STAGES * (W_BYTES + X_BYTES);
    static constexpr int FIXED = RING + ((BARS * 8 + 16 + 15) / 16) * 16 + STAGING + 1024;
    static constexpr int RUN_BLOCKS = kInt8Run / BK;
    static_assert(SLOT0 + SLOTS * SLOT_COLS <= TMEM_COLS && X_CHUNK % 1024 == 0 && W_BYTES % 1024 == 0, "");
    static_assert(FIXED + 8 * (kLmMaxGroups + 2) <= 227 * 1024, "room for the group tables");
};
// Few turns of the warps' loops, which bound all but the largest products; and wide
// tiles, which move less through shared memory and L2.  2048 rows, 4096 x 14336:
// 157 us, in wide tiles 196; 8192 rows: 598 and 547.
using Int8Deep = Int8Tile<128, 256, 3, 8>;
using Int8Wide = Int8Tile<192, 128, 5, 4>;

__device__ __forceinline__ void mma_f16_pair_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

// 32 columns of this lane.
__device__ __forceinline__ void tmem_st_32cols(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
           "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
           "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
           "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Tile t as lm_work gives it (kRagN), without its 64-bit divisions: every warp asks
// at every tile, and the MMAs' warp is waited for meanwhile.
template <class Tile>
__device__ __forceinline__ LmWork int8_work(const LmArgs &p, const int *start, const uint32_t *prefix, int tile) {
    LmWork w;
    uint32_t t = (uint32_t)tile;
    w.s = 0;
    w.kb0 = 0;
    w.nkb = p.kb;
    if (p.splits > 1) {
        w.s = (int)(t % (uint32_t)p.splits);
        t /= (uint32_t)p.splits;
        // (p.kb is at most 1024.)
        w.kb0 = (int)((uint32_t)(p.kb * w.s) / (uint32_t)p.splits);
        w.nkb = (int)((uint32_t)(p.kb * (w.s + 1)) / (uint32_t)p.splits) - w.kb0;
    }
    int lo = 0, hi = p.G;                   // last g with prefix[g] <= t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    w.g = lo;
    const uint32_t local = t - prefix[lo], rows = (uint32_t)(start[lo + 1] - start[lo]);
    const uint32_t nt = (rows + (uint32_t)p.tile_n - 1) / (uint32_t)p.tile_n;
    const uint32_t per = ((rows + nt - 1) / nt + Tile::GRAN - 1) / Tile::GRAN * Tile::GRAN;
    const uint32_t wide = (uint32_t)p.group_m * nt, band = local / wide, in = local - band * wide;
    const uint32_t bw = min((uint32_t)p.group_m, (uint32_t)p.tiles_m - band * (uint32_t)p.group_m);
    const uint32_t tn = in / bw, tm = band * (uint32_t)p.group_m + in - tn * bw;
    w.m0 = (int)(tm * Tile::TILE_M);
    w.n0 = start[lo] + (int)(tn * per);
    w.nvalid = (int)min(per, rows - tn * per);
    w.nmma = (w.nvalid + Tile::GRAN - 1) / Tile::GRAN * Tile::GRAN;
    if (lo == p.G) w.nkb = 0;
    w.krow0 = 0;
    w.klast = 64;
    return w;
}

// tmW: bytes {K, N, G}, boxes of 128 x 128.  tmX: f16 {K, T}, boxes of 64 x tile_n / 2.
template <class Tile>
__global__ void __launch_bounds__(Tile::THREADS, 1)
lm_int8_mma_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const __grid_constant__ Int8Args q) {
    constexpr int STAGES = Tile::STAGES, SLOTS = Tile::SLOTS, BN = Tile::BN, SLAB = Tile::SLAB;
    const LmArgs &p = q.lm;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
    unsigned char *smem = smem_raw + pad;
    unsigned char *smem_x = smem + STAGES * Tile::W_BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Tile::RING);
    uint64_t *wfull = bars;                     // this SM's bytes of W have landed
    uint64_t *ready = wfull + STAGES;           // rank 0: both SMs' x has landed and their W is converted
    uint64_t *wempty = ready + STAGES;          // converting warps -> copies of W
    uint64_t *xempty = wempty + STAGES;         // MMAs -> copies of x, and converting warps
    uint64_t *tfull = xempty + STAGES;          // MMAs -> epilogue, per accumulator
    uint64_t *tempty = tfull + 2;               // epilogue -> MMAs
    // (The other SM's threads or MMAs signal all but wfull and wempty: waited for at
    // the cluster's scope.)
    uint64_t *drain = tempty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + Tile::BARS);
    volatile uint32_t *progress = tmem_slot + 1;
    unsigned char *after = reinterpret_cast<unsigned char *>(bars) + ((Tile::BARS * 8 + 16 + 15) / 16) * 16;
    float *staging = reinterpret_cast<float *>(after);
    int *g_start = reinterpret_cast<int *>(after + Tile::STAGING);
    uint32_t *g_prefix = reinterpret_cast<uint32_t *>(g_start + p.G + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();

    if (warp == 0) tmem_alloc_pair(tmem_slot, Tile::TMEM_COLS);
    if (threadIdx.x == 32) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&wfull[s], 1);
            mbar_init(&ready[s], 1 + 2 * Tile::CONV_WARPS);
            mbar_init(&wempty[s], Tile::CONV_WARPS);
            mbar_init(&xempty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 2 * Tile::EPI_WARPS);
        }
        mbar_init(drain, 1);
        *progress = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmX);
    }
    // The kernel before wrote x and its scales, and let this one begin when all
    // before it was done: W's first stages are on their way and converted meanwhile.
    // Waits that have a limit begin behind it, however long it takes, but those for
    // W's first stages, which need nothing of it.
    griddep_launch_dependents();
    if (warp == 2) {
        if (p.ends != nullptr) {
            lm_group_tables<Tile, kRagN, true>(p, g_start, g_prefix, lane);
        } else if (lane == 0) {
            const uint32_t tiles = (uint32_t)((p.T + p.tile_n - 1) / p.tile_n) * (uint32_t)p.tiles_m;
            g_start[0] = 0; g_start[1] = g_start[2] = p.T;
            g_prefix[0] = 0; g_prefix[1] = g_prefix[2] = tiles;
        }
    }
    tc_fence_before();
    __syncwarp();               // (the barriers, too, take whole warps)
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(tmem_slot);
    const int slot0 = (int)(blockIdx.x >> 1), slots = (int)(gridDim.x >> 1);
    const int num_tiles = (int)g_prefix[p.G + 1] * p.splits;

    if (warp == 0 || warp == Tile::THREADS / 32 - 1) {
        // ---------------- copies: W by the first warp, x by the last ----------------
        // (Rings of their own: a stage of W is free once it is converted, long
        // before the MMAs have read the x beside it.)
        const bool of_w = warp == 0;
        if (!of_w) griddep_wait();
        uint64_t *full = of_w ? wfull : ready, *empty = of_w ? wempty : xempty;
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        const uint32_t x_bytes = (uint32_t)(p.tile_n / 2 * 128) * (Tile::BK / 64);      // of this SM
        const uint32_t ready0 = cluster_addr(&ready[0], 0);
        for (int t = slot0; ok && t < num_tiles; t += slots) {
            const LmWork w = int8_work<Tile>(p, g_start, g_prefix, t);
            const int mw = w.m0 + (int)rank * 128;
            const int nx = w.n0 + (int)rank * (w.nmma >> 1);
            for (int kb = 0; kb < w.nkb; ++kb) {
                if (p.withhold == kWithholdRefill && issued >= STAGES) { ok = false; break; }
                if (issued == STAGES) griddep_wait();
                if (!mbar_wait_bounded<true>(&empty[stage], phase ^ 1u, p.timeout_ns)) {
                    if (lane == 0) record_error(p.err, kSiteProducerEmpty);
                    ok = false;
                }
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                const int kc = (w.kb0 + kb) * Tile::BK;
                if (elect_one()) {
                    if (of_w) {
                        mbar_arrive_expect_tx(&wfull[stage], Tile::W_BYTES);
#pragma unroll
                        for (int c = 0; c < Tile::BK / 128; ++c)
                            tma_load_3d(smem + stage * Tile::W_BYTES + c * Tile::W_CHUNK, &tmW, &wfull[stage], kc + c * 128, mw,
                                        w.g);
                    } else {
                        unsigned char *sx = smem_x + stage * Tile::X_BYTES;
                        if (rank == 0) mbar_arrive_expect_tx(&ready[stage], 2 * x_bytes);
#pragma unroll
                        for (int c = 0; c < Tile::BK / 64; ++c)
                            tma_load_3d_pair(sx + c * Tile::X_CHUNK, &tmX, ready0 + (uint32_t)stage * 8u, kc + c * 64, nx, 0);
                    }
                }
                __syncwarp();
                ++issued;
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                    if (of_w && lane == 31) *progress = (uint32_t)issued;
                }
            }
        }
        if (!ok) {
            // Let this CTA's own copies land before it can exit (rank 1 sees
            // those of x as the release of its stages).
            const int pending = issued < STAGES ? issued : STAGES;
            for (int back = 1; back <= pending; ++back) {
                int s = stage - back;
                uint32_t ph = phase;
                if (s < 0) { s += STAGES; ph ^= 1u; }
                mbar_wait_bounded<true>(of_w || rank == 0 ? &full[s] : &empty[s], ph, p.timeout_ns);
            }
        }
    } else if (warp == 1 && rank == 0) {
        // ---------------- MMAs (one elected lane of a uniform warp) ----------------
        griddep_wait();
        const uint64_t db0 = smem_desc_k_sw128(smem_u32(smem_x));
        int stage = 0, gc = 0;
        uint32_t phase = 0, block = 0;
        bool ok = true;
        for (int t = slot0; ok && t < num_tiles; t += slots) {
            const LmWork w = int8_work<Tile>(p, g_start, g_prefix, t);
            const uint32_t idesc = idesc_f16(0, false, false, Tile::TILE_M, w.nmma);
            uint32_t d_tmem = 0;
            for (int kb = 0; kb < w.nkb; ++kb) {
                const bool first = kb % Tile::RUN_BLOCKS == 0;
                const bool last = kb == w.nkb - 1 || kb % Tile::RUN_BLOCKS == Tile::RUN_BLOCKS - 1;
                if (first) {
                    const int ab = gc & 1;
                    if (!mbar_wait_bounded<true>(&tempty[ab], ((uint32_t)(gc >> 1) & 1u) ^ 1u, p.timeout_ns)) {
                        if (lane == 0) record_error(p.err, kSiteConsumerFull);
                        ok = false;
                    }
                    d_tmem = tmem_base + (uint32_t)(ab * BN);
                }
                if (ok && !mbar_wait_bounded<true>(&ready[stage], phase, 3 * downstream_limit(p.timeout_ns))) {
                    if (lane == 0) record_error(p.err, kSiteConsumerFull);
                    ok = false;
                }
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t a = tmem_base + Tile::SLOT0 + block % SLOTS * Tile::SLOT_COLS;
                    const uint64_t b = db0 + (uint64_t)(stage * (Tile::X_BYTES >> 4));
#pragma unroll
                    for (int kk = 0; kk < Tile::BK / 16; ++kk)
                        mma_f16_pair_ts(d_tmem, a + kk * 8, b + (kk >> 2) * (Tile::X_CHUNK >> 4) + (kk & 3) * 2, idesc,
                                        first && kk == 0 ? 0u : 1u);
                    if (p.withhold != kWithholdRelease) mma_commit_pair_mc(&xempty[stage], 0x3);
                    if (last) mma_commit_pair_mc(&tfull[gc & 1], 0x3);
                }
                __syncwarp();
                ++block;
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                if (last) ++gc;
            }
        }
        if (elect_one()) mma_commit_pair(drain);
        __syncwarp();
        mbar_wait_bounded(drain, 0u, p.timeout_ns);
    } else if (warp >= 2 && warp < 2 + Tile::CONV_WARPS) {
        // ---------------- W into tensor memory ----------------
        // (Four warps reach all lanes of tensor memory; the next four, if there are
        // any, take the second half of a block's columns.)
        const int quarter = warp & 3, row = quarter * 32 + lane, col0 = ((warp - 2) >> 2) * Tile::CONV_COLS;
        const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16) + Tile::SLOT0 + col0 / 2;
        const uint32_t ready0 = cluster_addr(&ready[0], 0);
        int stage = 0;
        uint32_t phase = 0, block = 0;
        bool ok = true;
        for (int t = slot0; ok && t < num_tiles; t += slots) {
            const LmWork w = int8_work<Tile>(p, g_start, g_prefix, t);
            for (int kb = 0; kb < w.nkb; ++kb) {
                ok = __all_sync(~0u, mbar_wait_bounded(&wfull[stage], phase, downstream_limit(p.timeout_ns)));
                if (!ok) {
                    if (lane == 0) record_error(p.err, kSiteConsumerFull);
                    break;
                }
                if (block >= SLOTS) {
                    if (block == SLOTS) griddep_wait();
                    // The MMAs of the block that had this slot are done.
                    const uint32_t before = block - SLOTS;
                    ok = mbar_wait_bounded<true>(&xempty[before % STAGES], (before / STAGES) & 1u,
                                                  2 * downstream_limit(p.timeout_ns));
                    ok = __all_sync(~0u, ok);
                    if (!ok) {
                        if (lane == 0) record_error(p.err, kSiteConsumerFull);
                        break;
                    }
                    tc_fence_after();
                }
                const unsigned char *sw = smem + stage * Tile::W_BYTES + col0 / 128 * Tile::W_CHUNK + row * 128;
                static_assert(Tile::CONV_COLS == 128, "one chunk of W for a warp");
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t r[32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(sw + (((h * 4 + c) ^ (row & 7)) << 4));
                        to_f16(v.x, r[8 * c], r[8 * c + 1]);
                        to_f16(v.y, r[8 * c + 2], r[8 * c + 3]);
                        to_f16(v.z, r[8 * c + 4], r[8 * c + 5]);
                        to_f16(v.w, r[8 * c + 6], r[8 * c + 7]);
                    }
                    tmem_st_32cols(lane_base + block % SLOTS * Tile::SLOT_COLS + h * 32, r);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&wempty[stage]);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                // What this publishes is in tensor memory alone, and complete.  The
                // fence above and the one behind the MMAs' wait order it: as the PTX
                // ISA describes tcgen05.fence, a relaxed signal between the two is
                // enough (its example has st.relaxed and ld.relaxed), at a scope that
                // holds both threads, here the cluster.  (A release waits for more:
                // 8192 rows, 14336 x 4096, 1157 us in the place of 591; 2048 rows, 242
                // and 160; 64 groups of 128 rows, 2048 x 1024, 67 and 52.)
                if (lane == 0) mbar_arrive_cluster_relaxed(ready0 + (uint32_t)stage * 8u);
                ++block;
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            }
        }
    } else if (warp >= 2 + Tile::CONV_WARPS && warp < 2 + Tile::CONV_WARPS + Tile::EPI_WARPS) {
        // ---------------- epilogue ----------------
        const int quarter = warp & 3, ew = warp - 2 - Tile::CONV_WARPS;
        const int slab0 = (ew >> 2) * SLAB;
        float *stg = staging + ew * Tile::STG;
        griddep_wait();
        const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16);
        int gc = 0;
        bool ok = true;
        for (int t = slot0; ok && t < num_tiles; t += slots) {
            const LmWork w = int8_work<Tile>(p, g_start, g_prefix, t);
            const int row0 = w.m0 + (int)rank * 128 + quarter * 32;       // first channel of this warp
            int sum[SLAB];
#pragma unroll
            for (int c = 0; c < SLAB; ++c) sum[c] = 0;
            for (int kb = 0; kb < w.nkb; kb += Tile::RUN_BLOCKS) {
                ok = __all_sync(~0u, lm_wait_working<true>(&tfull[gc & 1], (uint32_t)(gc >> 1) & 1u,
                                                           downstream_limit(p.timeout_ns), progress));
                if (!ok) {
                    if (lane == 0) record_error(p.err, kSiteConsumerFull);
                    break;
                }
                tc_fence_after();
                const uint32_t taddr = lane_base + (uint32_t)((gc & 1) * BN + slab0);
#pragma unroll
                for (int c0 = 0; c0 < SLAB; c0 += 16) {
                    if (slab0 + c0 < w.nvalid) {
                        float r[16];
                        tmem_ld_16cols(taddr + (uint32_t)c0, r);
#pragma unroll
                        for (int i = 0; i < 16; ++i) sum[c0 + i] += __float2int_rn(r[i]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(cluster_addr(&tempty[gc & 1], 0));
                ++gc;
            }
            if (!ok) break;
            const int f = min(row0 + lane, p.M - 1);
            const float ws = w.g < p.G && p.splits == 1 ? q.scales[(int64_t)w.g * p.M + f] : 0.f;
#pragma unroll
            for (int c0 = 0; c0 < SLAB; c0 += 32) {
                const int col = slab0 + c0;
                if (col < w.nvalid && row0 < p.M) {
                    const int cnt = min(32, w.nvalid - col), n = w.n0 + col;
                    float v[32];
                    if (p.splits > 1) {
                        // (Bits of the integers: the store does not look at them.)
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __int_as_float(sum[c0 + i]);
                        lm_store_cols(p, static_cast<float *>(p.C) + w.s * p.stride_c, row0, n, cnt, v, stg, lane);
                        if (w.s == 0 && row0 == 0 && lane < cnt) q.row_group[n + lane] = w.g < p.G ? w.g : -1;
                    } else {
                        const float xs = w.g < p.G && lane < cnt ? q.x_scales[n + lane] : 0.f;
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = (float)sum[c0 + i] * __shfl_sync(~0u, xs, i) * ws;
                        if (p.out == kOutF32) lm_store_cols(p, static_cast<float *>(p.C), row0, n, cnt, v, stg, lane);
                        else if (p.out == kOutF16) lm_store_cols(p, static_cast<__half *>(p.C), row0, n, cnt, v, stg, lane);
                        else lm_store_cols(p, static_cast<__nv_bfloat16 *>(p.C), row0, n, cnt, v, stg, lane);
                    }
                    __syncwarp();
                }
            }
        }
    }

    // ---------------- teardown ----------------
    tc_fence_before();
    __syncwarp();
    cluster_sync();
    tc_fence_after();
    if (warp == 0) tmem_dealloc_pair(tmem_base, Tile::TMEM_COLS);
}

}  // namespace

template <class Tile>
LmKernel mma_kernel_info() {
    LmKernel k;
    k.fn = reinterpret_cast<const void *>(&lm_int8_mma_kernel<Tile>);
    k.threads = Tile::THREADS;
    k.smem = Tile::FIXED;
    k.tile_m = Tile::TILE_M;
    k.bn = Tile::BN;
    k.gran = Tile::BK;
    k.pair = 1;
    k.box_a = 128;
    return k;
}
LmKernel int8_mma_kernel(bool wide) { return wide ? mma_kernel_info<Int8Wide>() : mma_kernel_info<Int8Deep>(); }

}  // namespace sg
