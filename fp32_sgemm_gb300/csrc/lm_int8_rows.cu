// Products of a few rows of 8-bit integers with 8-bit weights, by group or not:
//
//   y[t, n] = sx[t] sw[n] sum_k x[t, k] w[n, k]
//
// The weights are read once, straight into registers, and that read bounds the
// product.  sm_103a has no tensor instruction for 8-bit integers beyond
// mma.sync at the rate of the integer pipes (151 TOPS measured, 592 TFLOP/s in
// f16), so they become f16 on the way, exactly: a byte less 128 under the
// leading bits of 1024, and 1152 less.  FP32 accumulators hold sums of 1024
// terms exactly; these are added as 32-bit integers, so a result does not
// depend on how the contraction is cut.
//
// A warp takes 16 rows of W for 8 NB tokens, KS of them share the contraction, and
// a CTA's other warps the rows that follow.  A lane loads 16 neighbouring bytes of a row (four lanes 64 of them) and
// multiplies them with the same 16 columns of x, which lie in shared memory as
// f16 (rows 16 bytes off a multiple of 128: no bank is met twice): the order of
// k within a product is free as long as both operands agree.  Loads run one
// step ahead, also from one tile to the next.
#include <type_traits>

#include "../../include/sgemm_gb300_lm.h"
#include "lm_int8.h"
#include "lm_int8_round.cuh"
#include "lm_mma.cuh"

namespace sg {
namespace {

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four integers as two pairs of f16: bytes 0 1 and 2 3.
__device__ __forceinline__ void to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    w ^= 0x80808080u;
    const uint32_t magic = 0x64646464u, less = 0x64806480u;             // 1024 + u - 1152
    const uint32_t l = __byte_perm(w, magic, 0x4140), h = __byte_perm(w, magic, 0x4342);
    const __half2 dl = __hsub2(*reinterpret_cast<const __half2 *>(&l), *reinterpret_cast<const __half2 *>(&less));
    const __half2 dh = __hsub2(*reinterpret_cast<const __half2 *>(&h), *reinterpret_cast<const __half2 *>(&less));
    lo = *reinterpret_cast<const uint32_t *>(&dl);
    hi = *reinterpret_cast<const uint32_t *>(&dh);
}

// 16 bytes at p, n of them in the row (the others 0).
__device__ __forceinline__ uint4 load16(const int8_t *p, int n, bool vec) {
    if (n <= 0) return make_uint4(0, 0, 0, 0);
    if (vec && n >= 16) {
        // (Read once: kept out of L1.)
        uint4 w;
        asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "l"(p));
        return w;
    }
    uint32_t v[5] = {0, 0, 0, 0, 0};
    const int skip = (int)(reinterpret_cast<uintptr_t>(p) & 3);
    if (n >= 20 && skip != 0) {
        // The aligned words that hold them (all in the row: n - 16 more follow).
        const uint32_t *from = reinterpret_cast<const uint32_t *>(p + 4 - skip);
        uint32_t head = 0;
        for (int e = 0; e < 4 - skip; ++e) head |= (uint32_t)(uint8_t)p[e] << (8 * (skip + e));
        v[0] = head;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e + 1] = from[e];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __funnelshift_r(v[e], v[e + 1], 8 * skip);
    } else if (n >= 16 && skip == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = reinterpret_cast<const uint32_t *>(p)[e];
    } else {
        for (int e = 0; e < min(n, 16); ++e) v[e / 4] |= (uint32_t)(uint8_t)p[e] << (8 * (e % 4));
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// Tokens t0 .. t0 + nt of numbers, quantised as lm_int8_quant.cu does: columns
// k_begin .. k_end as f16 in xs (to `width` columns, 0 behind k_end).  The warps
// are dealt to the tokens, a power of two to each.
template <class T, int WARPS>
__device__ __forceinline__ void stage_typed(const Int8Args &q, int64_t t0, int nt, int k_begin, int k_end, int width,
                                            unsigned char *xs, uint32_t *most_of, float *scale_of) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int share = WARPS;                                  // warps of a token
    while (share > 1 && share * nt > WARPS) share >>= 1;
    const int side = WARPS / share, part = warp % share, in = part * 32 + lane;
    for (int r0 = 0; r0 < nt; r0 += side) {
        const int r = r0 + warp / share;
        const T *row = static_cast<const T *>(q.x) + (t0 + min(r, nt - 1)) * q.ldx;
        uint32_t most = 0;
#pragma unroll 4
        for (int c = in * 8; c < q.K; c += share * 256) {
            Eight<T> v;
            v.load(row + c, q.K - c, q.x_vec);
            most = max(most, v.most());
        }
        most = __reduce_max_sync(~0u, most);
        if (share > 1) {
            __syncthreads();
            if (lane == 0) most_of[warp] = most;
            __syncthreads();
            most = 0;
            for (int u = 0; u < share; ++u) most = max(most, most_of[warp / share * share + u]);
        }
        const RowScale s(most);
        if (r < nt) {
            if (in == 0) scale_of[r] = s.scale;
#pragma unroll 4
            for (int c = in * 8; c < width; c += share * 256) {
                Eight<T> v;
                v.load(row + k_begin + c, s.finite ? k_end - k_begin - c : 0, q.x_vec);
                store8<true>(xs + r * q.x_pitch, c, nearest(v.e, s.s, s.inv), 8, true);
            }
        }
    }
}
template <int WARPS>
__device__ __forceinline__ void stage_numbers(const Int8Args &q, int64_t t0, int nt, int k_begin, int k_end, int width,
                                              unsigned char *xs, uint32_t *most_of, float *scale_of) {
    if (q.from == SGEMM_TYPE_F32) stage_typed<float, WARPS>(q, t0, nt, k_begin, k_end, width, xs, most_of, scale_of);
    else if (q.from == SGEMM_TYPE_F16) stage_typed<__half, WARPS>(q, t0, nt, k_begin, k_end, width, xs, most_of, scale_of);
    else stage_typed<__nv_bfloat16, WARPS>(q, t0, nt, k_begin, k_end, width, xs, most_of, scale_of);
}

// Columns of k in one step of a warp: a lane has 16 of every 64 of two rows.
constexpr int kStep = 256, kLoads = kStep / 64;

template <int NB, int WARPS, int KS>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS)
lm_int8_rows_kernel(const Int8Args q) {
    constexpr int TOKENS = NB * 8, THREADS = WARPS * 32, HIGH = 16 * (WARPS / KS);
    const LmArgs &p = q.lm;
    extern __shared__ unsigned char smem_raw[];
    uint32_t *most_of = reinterpret_cast<uint32_t *>(smem_raw);             // [16]
    float *scale_of = reinterpret_cast<float *>(most_of + 16);              // [16]
    int *red = reinterpret_cast<int *>(scale_of + 16);                           // [2][warp][NB * 4][32]
    int *start = red + 2 * WARPS * NB * 128;
    uint32_t *prefix = reinterpret_cast<uint32_t *>(start + p.G + 2);
    unsigned char *xs = smem_raw + ((32 + 2 * WARPS * NB * 128 + 2 * (p.G + 2)) * 4 + 15) / 16 * 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kw = warp % KS, rw = warp / KS;
    const int g = lane >> 2, c4 = lane & 3;
    const int k_begin = blockIdx.y * q.k_slice, k_end = min(q.K, k_begin + q.k_slice);
    // This warp's steps of the contraction: every KS-th, so that a CTA reads
    // neighbouring pieces of its rows at a time.
    const int steps = (k_end - k_begin + kStep - 1) / kStep;
    const int per = steps > kw ? (steps - 1 - kw) / KS + 1 : 0;

    griddep_launch_dependents();
    if (!q.early) griddep_wait();
    if (warp == 0) {
        if (p.ends != nullptr) {
            lm_group_tables<LmThin, kRagN>(p, start, prefix, lane);
        } else if (lane == 0) {
            const uint32_t tiles = (uint32_t)((p.T + p.tile_n - 1) / p.tile_n) * (uint32_t)p.tiles_m;
            start[0] = 0; start[1] = start[2] = p.T;
            prefix[0] = 0; prefix[1] = prefix[2] = tiles;
        }
    }
    __syncthreads();
    const int tiles = (int)prefix[p.G + 1];

    struct Tile {
        int g, t0, nt, n0;
    };
    auto tile_of = [&](int t) {
        int lo = 0, hi = p.G;                   // last g with prefix[g] <= t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= (uint32_t)t) lo = mid;
            else hi = mid - 1;
        }
        // Blocks of W one after another for the same tokens.
        const int local = t - (int)prefix[lo], chunk = local / p.tiles_m;
        Tile w;
        w.g = lo;
        w.n0 = (local - chunk * p.tiles_m) * HIGH;
        w.t0 = start[lo] + chunk * TOKENS;
        w.nt = min(TOKENS, start[lo + 1] - w.t0);
        return w;
    };
    // A CTA's tiles are neighbours, so that x is staged as seldom as it can be.
    const int first = (int)((int64_t)tiles * blockIdx.x / gridDim.x);
    const int last = (int)((int64_t)tiles * (blockIdx.x + 1) / gridDim.x);

    // The loads of one step, and the place of the next one.
    uint4 wa[kLoads], wb[kLoads];
    Tile nt{};
    int l_tile = first, l_step = 0;
    const int8_t *pa = nullptr, *pb = nullptr;
    bool l_live = false;
    auto point = [&]() {
        if (l_tile >= last) {
            l_live = false;
            return;
        }
        nt = tile_of(l_tile);
        l_live = nt.g < p.G;                     // (rows behind the last end have no W)
        const int8_t *base = q.w + (int64_t)min(nt.g, p.G - 1) * q.stride_w;
        pa = base + (int64_t)min(nt.n0 + rw * 16 + g, p.M - 1) * q.ldw;
        pb = base + (int64_t)min(nt.n0 + rw * 16 + g + 8, p.M - 1) * q.ldw;
    };
    auto load = [&](uint4 (&a)[kLoads], uint4 (&b)[kLoads]) {
        if (l_live) {
            const int k = k_begin + (kw + l_step * KS) * kStep + c4 * 16;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                a[i] = load16(pa + k + i * 64, k_end - k - i * 64, q.w_vec);
                b[i] = load16(pb + k + i * 64, k_end - k - i * 64, q.w_vec);
            }
        }
        if (++l_step == per) {
            l_step = 0;
            ++l_tile;
            point();
        }
    };
    point();
    if (per > 0 && first < last) load(wa, wb);
    if (q.early) griddep_wait();

    int staged_g = -1, staged_t = -1;
    const unsigned char *x_lane[NB];
    for (int t = first; t < last; ++t) {
        const Tile w = tile_of(t);
        if (w.g < p.G && (w.g != staged_g || w.t0 != staged_t)) {
            // x of this tile's tokens as f16; columns behind K become 0.
            __syncthreads();
            if (q.from != SGEMM_TYPE_S8) {
                stage_numbers<WARPS>(q, w.t0, w.nt, k_begin, k_end, steps * kStep, xs, most_of, scale_of);
            } else {
                const int chunks = steps * (kStep / 16), total = chunks * w.nt;
                for (int i = threadIdx.x; i < total; i += THREADS) {
                    const int r = i / chunks, c = i - r * chunks;
                    const uint4 v = load16(static_cast<const int8_t *>(q.x) + (int64_t)(w.t0 + r) * q.ldx + k_begin + c * 16,
                                           k_end - k_begin - c * 16, true);
                    uint32_t h[8];
                    to_f16(v.x, h[0], h[1]);
                    to_f16(v.y, h[2], h[3]);
                    to_f16(v.z, h[4], h[5]);
                    to_f16(v.w, h[6], h[7]);
                    uint4 *to = reinterpret_cast<uint4 *>(xs + r * q.x_pitch + c * 32);
                    to[0] = make_uint4(h[0], h[1], h[2], h[3]);
                    to[1] = make_uint4(h[4], h[5], h[6], h[7]);
                }
            }
            __syncthreads();
            staged_g = w.g;
            staged_t = w.t0;
        }
        // (Columns of tokens that are not there take the last one's x; their sums go nowhere.)
#pragma unroll
        for (int n = 0; n < NB; ++n) x_lane[n] = xs + min(n * 8 + g, w.nt - 1) * q.x_pitch + (kw * kStep + c4 * 16) * 2;
        int sum[NB][4];
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[n][i] = 0;
        if (w.g < p.G) {
            float acc[2][NB][4];
            for (int s = 0; s < per; ++s) {
                uint4 a[kLoads], b[kLoads];
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    a[i] = wa[i];
                    b[i] = wb[i];
                }
                load(wa, wb);
                // Two accumulators in turn, each of at most kInt8Run terms.
                constexpr int FLUSH = 2 * kInt8Run / kStep;
                if (s % FLUSH == 0)
#pragma unroll
                    for (int z = 0; z < 2; ++z)
#pragma unroll
                        for (int n = 0; n < NB; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[z][n][i] = 0.f;
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    uint32_t ha[8], hb[8];
                    to_f16(a[i].x, ha[0], ha[1]);
                    to_f16(a[i].y, ha[2], ha[3]);
                    to_f16(a[i].z, ha[4], ha[5]);
                    to_f16(a[i].w, ha[6], ha[7]);
                    to_f16(b[i].x, hb[0], hb[1]);
                    to_f16(b[i].y, hb[2], hb[3]);
                    to_f16(b[i].z, hb[4], hb[5]);
                    to_f16(b[i].w, hb[6], hb[7]);
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        const uint4 *x = reinterpret_cast<const uint4 *>(x_lane[n] + (s * (KS * kStep) + i * 64) * 2);
                        const uint4 u = x[0], v = x[1];
                        mma16816(acc[0][n], ha[0], hb[0], ha[1], hb[1], u.x, u.y);
                        mma16816(acc[1][n], ha[2], hb[2], ha[3], hb[3], u.z, u.w);
                        mma16816(acc[0][n], ha[4], hb[4], ha[5], hb[5], v.x, v.y);
                        mma16816(acc[1][n], ha[6], hb[6], ha[7], hb[7], v.z, v.w);
                    }
                }
                if (s % FLUSH == FLUSH - 1 || s == per - 1)
#pragma unroll
                    for (int z = 0; z < 2; ++z)
#pragma unroll
                        for (int n = 0; n < NB; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i) sum[n][i] += __float2int_rn(acc[z][n][i]);
            }
        } else {
            for (int s = 0; s < per; ++s) load(wa, wb);         // (moves on to the next tile)
        }
        // Join the sums of the KS warps (two buffers: a warp may be one tile ahead).
        int *buf = red + (t & 1) * (WARPS * NB * 128);
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) buf[(warp * NB * 4 + n * 4 + i) * 32 + lane] = sum[n][i];
        if constexpr (KS == 1) __syncwarp();
        else __syncthreads();
        const int own = KS == 1 ? lane : (int)threadIdx.x, all = KS == 1 ? 16 * w.nt : HIGH * w.nt;
        for (int o = own; o < all; o += KS == 1 ? 32 : THREADS) {
            // Column `col` of the MMA's row r sits in lane (r % 8) * 4 + (col % 8) / 2,
            // register (r / 8) * 2 + col % 2 of block col / 8.
            const int col = KS == 1 ? o >> 4 : o / HIGH, high = KS == 1 ? rw * 16 + (o & 15) : o % HIGH, r = high & 15;
            const int at = ((col >> 3) * 4 + (r >> 3) * 2 + (col & 1)) * 32 + (r & 7) * 4 + ((col & 7) >> 1);
            const int *of = buf + (high >> 4) * (KS * NB * 128);
            int v = 0;
#pragma unroll
            for (int u = 0; u < KS; ++u) v += of[u * NB * 128 + at];
            const int n = w.n0 + high;
            const int64_t row = w.t0 + col;
            if (n < p.M) {
                if (p.splits > 1) {
                    static_cast<int *>(p.C)[blockIdx.y * p.stride_c + row * p.ldc + n] = v;
                    if (n == 0 && blockIdx.y == 0) q.row_group[row] = w.g < p.G ? w.g : -1;
                } else {
                    const float xs_of = q.from == SGEMM_TYPE_S8 ? q.x_scales[row] : scale_of[col];
                    const float y = w.g < p.G ? (float)v * xs_of * q.scales[(int64_t)w.g * p.M + n] : 0.f;
                    if (p.out == kOutF32) static_cast<float *>(p.C)[row * p.ldc + n] = y;
                    else if (p.out == kOutF16) static_cast<__half *>(p.C)[row * p.ldc + n] = __float2half_rn(y);
                    else static_cast<__nv_bfloat16 *>(p.C)[row * p.ldc + n] = __float2bfloat16_rn(y);
                }
            }
        }
    }
}

template <int NB, int WARPS, int KS>
const void *rows_kernel() {
    return reinterpret_cast<const void *>(&lm_int8_rows_kernel<NB, WARPS, KS>);
}
template <int NB>
const void *rows_kernel(int warps, int ks) {
    if (warps == 16) return ks == 16 ? rows_kernel<NB, 16, 16>() : ks == 8 ? rows_kernel<NB, 16, 8>() : rows_kernel<NB, 16, 4>();
    return ks == 8 ? rows_kernel<NB, 8, 8>() : ks == 4 ? rows_kernel<NB, 8, 4>() : rows_kernel<NB, 8, 1>();
}

}  // namespace

LmKernel int8_rows_kernel(int tokens, int warps, int ks) {
    LmKernel k;
    k.fn = tokens <= 8 ? rows_kernel<1>(warps, ks) : rows_kernel<2>(warps, ks);
    k.threads = warps * 32;
    k.bn = tokens <= 8 ? 8 : 16;
    k.tile_m = 16 * (warps / ks);
    return k;
}
int64_t int8_rows_smem(int tokens, int warps, int64_t x_pitch, int64_t G) {
    const int64_t nb = tokens <= 8 ? 1 : 2;
    return ((32 + 2 * warps * nb * 128 + 2 * (G + 2)) * 4 + 15) / 16 * 16 + std::min<int64_t>(tokens, nb * 8) * x_pitch;
}

}  // namespace sg
