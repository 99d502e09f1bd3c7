// Products of a few rows of 8-bit integers with 8-bit weights, by group or not:
//
//   y[t, n] = sx[t] sw[n] sum_k x[t, k] w[n, k]
//
// The weights are read once, straight into registers, one step ahead (also from
// one tile to the next), and that read should bound the product; what does bound
// it is the instructions beside it, so they are few:
//   * up to four tokens: __dp4a, one instruction for four products, x as bytes;
//   * more: mma.sync in f16.  (In 8-bit integers it runs at __dp4a's rate: 151 TOPS
//     measured, 592 TFLOP/s in f16.)  The bytes become f16 on the way, exactly: a
//     byte plus 128 under the leading bits of 1024, and 1152 less.  FP32
//     accumulators hold sums of 1024 terms exactly; these are added as 32-bit
//     integers.
// Either way the sum is exact, so a result does not depend on how the contraction
// is cut.
//
// A warp takes 16 rows of W, KS of them share the contraction, and a CTA's other
// warps the rows that follow.  A lane loads 16 neighbouring bytes of a row (four
// lanes 64 of them) and multiplies them with the same 16 columns of x, which lie
// in shared memory (f16 rows 16 bytes off a multiple of 128: no bank is met twice):
// the order of k within a product is free as long as both operands agree.
//
// Measured (one GB300, f16 x, quantisation included; reading alone takes 34.6, 8.7
// and 2.5 us): 28672 x 8192, one token 41.8 us (5.6 TB/s; 38.4 where calls follow one
// another), four 41.8, eight 46.4; 14336 x 4096, one 13.6, seven (14335) 17.2; 4096 x
// 4096, one 6.9, eight 10.2; 64 groups of 2048 x 1024, 32 tokens 18.3, 128 tokens
// 30.3 (4.5 TB/s).  A ring of TMA copies in the place of the registers kept more
// bytes on their way and took longer (one token, 28672 x 8192: 48 us), as did loads
// of 512 columns a step (eight tokens: 57 us): the instructions bound it, and the
// registers, not the loads.  W that is not 16-byte aligned or of a pitch
// that is no multiple of 16 is put together from words: 4096 x 4095, one token, 15 us.
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

// W may be read before the kernel has waited, where nothing says that L1 holds no
// older copy: rows that are aligned go past it (relaxed loads at the device's scope),
// whole pieces and the bytes of a row's end alike.  (Read once: kept out of L1, too.)
__device__ __forceinline__ uint4 load_whole(const int8_t *p) {
    uint4 w;
    asm volatile("ld.relaxed.gpu.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "l"(p));
    return w;
}
__device__ __forceinline__ uint32_t load_byte(const int8_t *p) {
    uint32_t b;
    asm volatile("ld.relaxed.gpu.global.u8 %0, [%1];" : "=r"(b) : "l"(p));
    return b;
}
// 16 bytes at p, n of them in the row (the others 0).
__device__ __noinline__ uint4 load_some(const int8_t *p, int n) {
    const int skip = (int)(reinterpret_cast<uintptr_t>(p) & 3);
    if (n >= 16 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) return load_whole(p);
    uint32_t v[5] = {0, 0, 0, 0, 0};
    if (n >= 20) {
        // (A row that is not aligned: the kernel has waited.)  The aligned words that
        // hold them, all in the row: n - 16 more follow.
        const uint32_t *from = reinterpret_cast<const uint32_t *>(p + 4 - skip);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < 4 - skip) v[0] |= (uint32_t)(uint8_t)p[e] << (8 * (skip + e));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e + 1] = from[e];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __funnelshift_r(v[e], v[e + 1], 8 * skip);
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (e < n) v[e / 4] |= load_byte(p + e) << (8 * (e % 4));
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// Tokens t0 .. t0 + nt of numbers, quantised as lm_int8_quant.cu does: columns
// k_begin .. k_end as f16 or bytes in xs (to `width` columns, 0 behind k_end).  The warps
// are dealt to the tokens, a power of two to each.
template <class T, int WARPS, bool F16>
__device__ __forceinline__ void stage_typed(const Int8Args &q, int64_t t0, int nt, int k_end, int width,
                                            unsigned char *xs, uint32_t *most_of, float *scale_of) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int share = WARPS;                                  // warps of a token
    while (share > 1 && share * nt > WARPS) share >>= 1;
    const int side = WARPS / share, part = warp % share, in = part * 32 + lane;
    for (int r0 = 0; r0 < nt; r0 += side) {
        const int r = r0 + warp / share;
        const T *row = static_cast<const T *>(q.x) + (t0 + min(r, nt - 1)) * q.ldx;
        // (The first pieces are kept.)
        constexpr int HELD = 4;
        Eight<T> held[HELD];
        uint32_t most = 0;
#pragma unroll
        for (int h = 0; h < HELD; ++h) held[h].load(row + in * 8 + h * share * 256, q.K - in * 8 - h * share * 256, q.x_vec);
#pragma unroll
        for (int h = 0; h < HELD; ++h) most = max(most, held[h].most());
        for (int c = in * 8 + HELD * share * 256; c < q.K; c += share * 256) {
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
            // (k_begin is 0 here: a row that a CTA quantises itself is not cut.)
#pragma unroll
            for (int h = 0; h < HELD; ++h) {
                const int c = in * 8 + h * share * 256;
                if (!s.finite) held[h].clear();
                if (c < width) store8<F16>(xs + r * q.x_pitch, c, nearest(held[h].e, s.s, s.inv), 8, true);
            }
            for (int c = in * 8 + HELD * share * 256; c < width; c += share * 256) {
                Eight<T> v;
                v.load(row + c, s.finite ? k_end - c : 0, q.x_vec);
                store8<F16>(xs + r * q.x_pitch, c, nearest(v.e, s.s, s.inv), 8, true);
            }
        }
    }
}
template <int WARPS, bool F16>
__device__ __forceinline__ void stage_numbers(const Int8Args &q, int64_t t0, int nt, int k_end, int width,
                                              unsigned char *xs, uint32_t *most_of, float *scale_of) {
    if (q.from == SGEMM_TYPE_F32) stage_typed<float, WARPS, F16>(q, t0, nt, k_end, width, xs, most_of, scale_of);
    else if (q.from == SGEMM_TYPE_F16) stage_typed<__half, WARPS, F16>(q, t0, nt, k_end, width, xs, most_of, scale_of);
    else stage_typed<__nv_bfloat16, WARPS, F16>(q, t0, nt, k_end, width, xs, most_of, scale_of);
}

// Columns of k in one step of a warp: a lane has 16 of every 64 of two rows.
constexpr int kStep = 256, kLoads = kStep / 64;

// TOKENS: 1, 2 or 4 by __dp4a, 8 by mma.sync.
template <int TOKENS, int WARPS, int KS>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS)
lm_int8_rows_kernel(const __grid_constant__ Int8Args q) {
    constexpr bool DOT = TOKENS <= 4;
    constexpr int THREADS = WARPS * 32, HIGH = 16 * (WARPS / KS);
    constexpr int SUMS = 16 * TOKENS;                                       // of one warp
    const LmArgs &p = q.lm;
    extern __shared__ unsigned char smem_raw[];
    uint32_t *most_of = reinterpret_cast<uint32_t *>(smem_raw);             // [16]
    float *scale_of = reinterpret_cast<float *>(most_of + 16);              // [16]
    int *red = reinterpret_cast<int *>(scale_of + 16);                      // [2][warp][SUMS]
    int *start = red + 2 * WARPS * SUMS;
    uint32_t *prefix = reinterpret_cast<uint32_t *>(start + p.G + 2);
    unsigned char *xs = smem_raw + ((32 + 2 * WARPS * SUMS + 2 * (p.G + 2)) * 4 + 15) / 16 * 16;
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
            lm_group_tables<LmThin, kRagN, true>(p, start, prefix, lane);
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
    int l_tile = first, l_step = 0, l_k = 0;
    const int8_t *pa = nullptr, *pb = nullptr;
    bool l_live = false;
    auto point = [&]() {
        // (Rows behind the last end, which have no W, are the last tiles.)
        l_live = false;
        if (l_tile >= last) return;
        const Tile nt = tile_of(l_tile);
        l_live = nt.g < p.G;
        l_k = k_begin + kw * kStep + c4 * 16;
        const int8_t *base = q.w + (int64_t)min(nt.g, p.G - 1) * q.stride_w + l_k;
        pa = base + (int64_t)min(nt.n0 + rw * 16 + g, p.M - 1) * q.ldw;
        pb = base + (int64_t)min(nt.n0 + rw * 16 + g + 8, p.M - 1) * q.ldw;
    };
    auto load = [&]() {
        if (!l_live) return;
        if (q.w_vec && l_k + kStep - 48 <= k_end) {                 // (all lanes alike, or nearly)
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                wa[i] = load_whole(pa + i * 64);
                wb[i] = load_whole(pb + i * 64);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                wa[i] = load_some(pa + i * 64, k_end - l_k - i * 64);
                wb[i] = load_some(pb + i * 64, k_end - l_k - i * 64);
            }
        }
        l_k += KS * kStep;
        pa += KS * kStep;
        pb += KS * kStep;
        if (++l_step == per) {
            l_step = 0;
            ++l_tile;
            point();
        }
    };
    point();
    if (per > 0) load();
    if (q.early) griddep_wait();

    int staged_g = -1, staged_t = -1;
    for (int t = first; t < last; ++t) {
        const Tile w = tile_of(t);
        if (w.g < p.G && (w.g != staged_g || w.t0 != staged_t)) {
            // x of this tile's tokens; columns behind K become 0.
            __syncthreads();
            if (q.from != SGEMM_TYPE_S8) {
                stage_numbers<WARPS, !DOT>(q, w.t0, w.nt, k_end, steps * kStep, xs, most_of, scale_of);
            } else {
                const int chunks = steps * (kStep / 16), total = chunks * w.nt;
                for (int i = threadIdx.x; i < total; i += THREADS) {
                    const int r = i / chunks, c = i - r * chunks;
                    const int8_t *from = static_cast<const int8_t *>(q.x) + (int64_t)(w.t0 + r) * q.ldx + k_begin + c * 16;
                    const int n = k_end - k_begin - c * 16;
                    const uint4 v = n >= 16 ? *reinterpret_cast<const uint4 *>(from) : load_some(from, n);
                    if constexpr (DOT) {
                        *reinterpret_cast<uint4 *>(xs + r * q.x_pitch + c * 16) = v;
                    } else {
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
            }
            __syncthreads();
            staged_g = w.g;
            staged_t = w.t0;
        }
        // Two buffers: a warp may be one tile ahead.
        int *own = red + ((t & 1) * WARPS + warp) * SUMS;                   // [token][row]
        if constexpr (DOT) {
            // (Tokens that are not there take the last one's x; their sums go nowhere.)
            const unsigned char *x_lane[TOKENS];
#pragma unroll
            for (int n = 0; n < TOKENS; ++n) x_lane[n] = xs + min(n, w.nt - 1) * q.x_pitch + kw * kStep + c4 * 16;
            int sum[2][TOKENS];
#pragma unroll
            for (int n = 0; n < TOKENS; ++n) sum[0][n] = sum[1][n] = 0;
            if (w.g < p.G)
                for (int s = 0; s < per; ++s) {
                    uint4 a[kLoads], b[kLoads];
#pragma unroll
                    for (int i = 0; i < kLoads; ++i) {
                        a[i] = wa[i];
                        b[i] = wb[i];
                    }
                    load();
#pragma unroll
                    for (int i = 0; i < kLoads; ++i)
#pragma unroll
                        for (int n = 0; n < TOKENS; ++n) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(x_lane[n] + i * 64);
                            sum[0][n] = __dp4a((int)a[i].x, (int)x.x, sum[0][n]);
                            sum[1][n] = __dp4a((int)b[i].x, (int)x.x, sum[1][n]);
                            sum[0][n] = __dp4a((int)a[i].y, (int)x.y, sum[0][n]);
                            sum[1][n] = __dp4a((int)b[i].y, (int)x.y, sum[1][n]);
                            sum[0][n] = __dp4a((int)a[i].z, (int)x.z, sum[0][n]);
                            sum[1][n] = __dp4a((int)b[i].z, (int)x.z, sum[1][n]);
                            sum[0][n] = __dp4a((int)a[i].w, (int)x.w, sum[0][n]);
                            sum[1][n] = __dp4a((int)b[i].w, (int)x.w, sum[1][n]);
                        }
#pragma unroll
                    for (int n = 0; n < TOKENS; ++n) x_lane[n] += KS * kStep;
                }
#pragma unroll
            for (int n = 0; n < TOKENS; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    int v = sum[h][n];
                    v += __shfl_xor_sync(~0u, v, 1);
                    v += __shfl_xor_sync(~0u, v, 2);
                    if (c4 == 0) own[n * 16 + h * 8 + g] = v;
                }
        } else {
            const unsigned char *x_lane = xs + min(g, w.nt - 1) * q.x_pitch + (kw * kStep + c4 * 16) * 2;
            int sum[4];
            float acc[2][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sum[i] = 0;
                acc[0][i] = acc[1][i] = 0.f;
            }
            if (w.g < p.G)
                for (int s = 0; s < per; ++s) {
                    uint4 a[kLoads], b[kLoads];
#pragma unroll
                    for (int i = 0; i < kLoads; ++i) {
                        a[i] = wa[i];
                        b[i] = wb[i];
                    }
                    load();
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
                        const uint4 *x = reinterpret_cast<const uint4 *>(x_lane + i * 128);
                        const uint4 u = x[0], v = x[1];
                        mma16816(acc[0], ha[0], hb[0], ha[1], hb[1], u.x, u.y);
                        mma16816(acc[1], ha[2], hb[2], ha[3], hb[3], u.z, u.w);
                        mma16816(acc[0], ha[4], hb[4], ha[5], hb[5], v.x, v.y);
                        mma16816(acc[1], ha[6], hb[6], ha[7], hb[7], v.z, v.w);
                    }
                    x_lane += KS * kStep * 2;
                    // Two accumulators in turn, each of at most kInt8Run terms.
                    constexpr int FLUSH = 2 * kInt8Run / kStep;
                    if (s % FLUSH == FLUSH - 1 || s == per - 1)
#pragma unroll
                        for (int z = 0; z < 2; ++z)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                sum[i] += __float2int_rn(acc[z][i]);
                                acc[z][i] = 0.f;
                            }
                }
            // Register i: row lane / 4 + 8 (i / 2), token 2 (lane % 4) + i % 2.
#pragma unroll
            for (int i = 0; i < 4; ++i) own[(c4 * 2 + (i & 1)) * 16 + g + (i >> 1) * 8] = sum[i];
        }
        // Join the sums of the KS warps.
        if constexpr (KS == 1) __syncwarp();
        else __syncthreads();
        const int all = KS == 1 ? 16 * w.nt : HIGH * w.nt;
        for (int o = KS == 1 ? lane : (int)threadIdx.x; o < all; o += KS == 1 ? 32 : THREADS) {
            const int col = KS == 1 ? o >> 4 : o / HIGH, high = KS == 1 ? rw * 16 + (o & 15) : o % HIGH;
            const int *of = red + ((t & 1) * WARPS + (high >> 4) * KS) * SUMS + col * 16 + (high & 15);
            int v = 0;
#pragma unroll
            for (int u = 0; u < KS; ++u) v += of[u * SUMS];
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

template <int TOKENS, int WARPS, int KS>
const void *rows_kernel() {
    return reinterpret_cast<const void *>(&lm_int8_rows_kernel<TOKENS, WARPS, KS>);
}
template <int TOKENS>
const void *rows_kernel(int warps, int ks) {
    if (warps == 16)
        return ks == 16 ? rows_kernel<TOKENS, 16, 16>() : ks == 8 ? rows_kernel<TOKENS, 16, 8>() : rows_kernel<TOKENS, 16, 4>();
    return ks == 8 ? rows_kernel<TOKENS, 8, 8>() : ks == 4 ? rows_kernel<TOKENS, 8, 4>() : rows_kernel<TOKENS, 8, 1>();
}

}  // namespace

LmKernel int8_rows_kernel(int tokens, int warps, int ks) {
    LmKernel k;
    k.fn = tokens == 1   ? rows_kernel<1>(warps, ks)
           : tokens == 2 ? rows_kernel<2>(warps, ks)
           : tokens == 4 ? rows_kernel<4>(warps, ks)
                         : rows_kernel<8>(warps, ks);
    k.threads = warps * 32;
    k.bn = tokens;
    k.tile_m = 16 * (warps / ks);
    return k;
}
int64_t int8_rows_pitch(int tokens, int64_t k_slice) { return tokens <= 4 ? k_slice : k_slice * 2 + 16; }
int64_t int8_rows_smem(int tokens, int rows, int warps, int64_t k_slice, int64_t G) {
    return ((32 + 2 * warps * 16 * tokens + 2 * (G + 2)) * 4 + 15) / 16 * 16 + rows * int8_rows_pitch(tokens, k_slice);
}

}  // namespace sg
