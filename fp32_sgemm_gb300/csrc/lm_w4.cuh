// Products of a few rows with 4-bit weights and group scales:
//
//   y[t, n] = sum_g s[n, g] sum_{k in g} (q[n, k] - z[n, g]) x[t, k]
//
// The weights are read once (half a byte each) and that read bounds the
// product, so everything else is kept off its way:
//   * each warp streams 16 weight rows, 256 columns (2 KB) at a time, through
//     its own ring of TMA copies;
//   * q - z is an integer of magnitude below 256 (z is any byte), exact in
//     f16 and bf16, so the weights meet x in the tensor core unscaled
//     (mma.sync m16n8k16, the rows of W on the M side, 8 tokens on the N side)
//     and the scale is applied to the FP32 sum of its group: no weight is ever
//     rounded.  A nibble becomes a float by one logic operation (its bits under
//     those of 128 or 1024) and one subtraction, for two weights at a time;
//   * the order of k inside a group is free as long as both operands agree.
//     A lane multiplies the 8 weights of a 32-bit word with the 8 x values
//     of the same columns, kept in shared memory in the order in which the
//     nibbles come out; which word a lane takes is chosen so that it reads
//     as many neighbouring words at once as the group allows (16, 8 or 4
//     bytes for groups of 128, 64, 32);
//   * FP32 x is held as three bf16 planes (exactly for |x| >= 2^-110), as three tokens.
// The warps of a CTA share 16 rows and split K; their sums are joined in a
// fixed order through shared memory.
//
// Measured (one GB300; reading alone takes 18.1, 1.3 and 5.2 us): 28672 x 8192,
// f16, groups of 128, one row 26.8 us, 4.5 TB/s; 4096 x 4096, bf16, one row 4.9
// us, most of it the launch and one pass through the memory; 14335 x 4096
// with zero points, groups of 32, bf16, seven rows 13.9 us, 2.5 TB/s.  The long
// ones are at no unit's limit: instructions issue in 59% of the active cycles,
// DRAM is at 54%, the matrix pipe at 24%.  What is left is latency: a group's
// products are a chain of up to eight dependent mma.sync, about 26 cycles each
// whatever the number of rows, with four warps on a quarter of an SM.  The same
// on the FP32 pipes took 33.5 us, on tcgen05 with the unpacked weights in tensor
// memory 44.8.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "lm_ptx.cuh"
#include "lm_w4.h"

namespace sg {

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
    if constexpr (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%10, %11, %12, %13};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%10, %11, %12, %13};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// (w & mask) ^ magic in one operation, with both constants in registers.
__device__ __forceinline__ uint32_t and_xor(uint32_t w, uint32_t mask, uint32_t magic) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(w), "r"(mask), "r"(magic));
    return r;
}
__device__ __forceinline__ uint32_t in_register(uint32_t v) {
    uint32_t r;
    asm volatile("mov.b32 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// What the unpacking subtracts for one zero point z, twice in a register each.
// Any byte is a zero point: q - z is in [-255, 15], exact in both types.
//   f16: 1024 + z, and 64 + z for the nibbles four bits higher.
//   bf16 holds 128 + q beside a nibble, and 128 + z exactly only for z < 128;
//   from 128 on the nibble is complemented and the sign set, which makes it
//   -(128 + 15 - q) = q - 143, and z - 143 is subtracted.  `other` is what the
//   masked nibble is combined with (and_xor) to get there.  As that takes five
//   operations more, a step none of whose zero points is above 127 (ANY false)
//   goes without (14335 x 4096, groups of 32, seven rows: 14.8 us with it in
//   every step).
struct W4Zero {
    uint32_t zero, other;
};
// Byte `at` of z.
template <bool BF16, bool ANY>
__device__ __forceinline__ W4Zero w4_zero(uint32_t z, int at, uint32_t magic) {
    if constexpr (BF16 && !ANY) {
        return {__byte_perm(z, 0x43434343u, 0x4040u | (uint32_t)at * 0x101u), magic};
    } else if constexpr (BF16) {
        const uint32_t u = __byte_perm(z, 0x4B000000u, 0x7440u | (uint32_t)at);       // 2^23 + z
        const bool high = (u & 0x80u) != 0;
        const float c = __uint_as_float(u) - (high ? 8388608.f + 143.f : 8388608.f - 128.f);
        return {__byte_perm(__float_as_uint(c), 0u, 0x3232u), high ? 0xC30FC30Fu : 0x43004300u};
    } else {
        const uint32_t u = __byte_perm(z, 0x64646464u, 0x4040u | (uint32_t)at * 0x101u);
        const uint32_t sub = 0x63806380u;                                             // 960 twice
        const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&u), *reinterpret_cast<const __half2 *>(&sub));
        return {u, *reinterpret_cast<const uint32_t *>(&d)};
    }
}

// The constants of the unpacking, kept in registers.
template <bool BF16>
struct W4Unpack {
    uint32_t mask, magic, mask4, sixteenth;
    __device__ __forceinline__ W4Unpack() {
        mask = in_register(0x000F000Fu);
        magic = in_register(BF16 ? 0x43004300u : 0x64006400u);
        mask4 = in_register(0x00F000F0u);
        sixteenth = 0x2C002C00u;     // 1 / 16 twice, f16
    }
    // A zero point of 8.
    __device__ __forceinline__ W4Zero eight() const {
        if constexpr (BF16) return {0x43084308u, magic};
        else return {0x64086408u, 0x54805480u};
    }
    // The 8 nibbles of w as four pairs (0,4) (1,5) (2,6) (3,7) of q - z: each
    // nibble in the low bits of a float whose unit there is one, less that
    // float and z (a published conversion: Kim et al., 2022).  f16 has room
    // for the nibble four bits higher, as 1024 + 16 q, which one fused
    // operation brings to q - z: two shifts fewer.
    __device__ __forceinline__ void operator()(uint32_t w, const W4Zero &zero, uint32_t (&o)[4]) const {
        if constexpr (BF16) {
            const __nv_bfloat162 z = *reinterpret_cast<const __nv_bfloat162 *>(&zero.zero);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t v = and_xor(w >> (4 * i), mask, zero.other);
                const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), z);
                o[i] = *reinterpret_cast<const uint32_t *>(&d);
            }
        } else {
            const __half2 z = *reinterpret_cast<const __half2 *>(&zero.zero);
            const __half2 z4 = *reinterpret_cast<const __half2 *>(&zero.other);
            const __half2 s = *reinterpret_cast<const __half2 *>(&sixteenth);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t u = i ? w >> 8 : w;
                const uint32_t v = and_xor(u, mask, magic), v4 = and_xor(u, mask4, magic);
                const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&v), z);
                const __half2 d4 = __hfma2(*reinterpret_cast<const __half2 *>(&v4), s, __hneg2(z4));
                o[2 * i] = *reinterpret_cast<const uint32_t *>(&d);
                o[2 * i + 1] = *reinterpret_cast<const uint32_t *>(&d4);
            }
        }
    }
};

// N scales of one row (raw bits; 16-bit ones two to a register) and N zero
// points (bytes), by vector loads where the rows are aligned for them.
template <int TYPE, int N, bool ZEROS>
struct W4Meta {
    static constexpr int REGS = TYPE == 0 ? N : N / 2;
    uint32_t s[REGS];
    uint32_t z[(N + 3) / 4];

    // n of them exist (N but for the last step of a row).
    __device__ __forceinline__ void load(const W4Args &p, const unsigned char *scales, const uint8_t *zeros, int n) {
        if (p.s_vec && n == N) {
            const uint32_t *src = reinterpret_cast<const uint32_t *>(scales);
            if constexpr (REGS == 1) {
                s[0] = *src;
            } else if constexpr (REGS == 2) {
                const uint2 v = *reinterpret_cast<const uint2 *>(src);
                s[0] = v.x; s[1] = v.y;
            } else {
#pragma unroll
                for (int i = 0; i < REGS; i += 4) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(src + i);
                    s[i] = v.x; s[i + 1] = v.y; s[i + 2] = v.z; s[i + 3] = v.w;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < REGS; ++i) s[i] = 0u;
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (j < n) {
                    if constexpr (TYPE == 0) s[j] = reinterpret_cast<const uint32_t *>(scales)[j];
                    else s[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(scales)[j] << (16 * (j & 1));
                }
        }
        if constexpr (ZEROS) {
            if (p.z_vec && n == N) {
                if constexpr (N == 2) z[0] = *reinterpret_cast<const uint16_t *>(zeros);
                else if constexpr (N == 4) z[0] = *reinterpret_cast<const uint32_t *>(zeros);
                else {
                    const uint2 v = *reinterpret_cast<const uint2 *>(zeros);
                    z[0] = v.x; z[1] = v.y;
                }
            } else {
#pragma unroll
                for (int i = 0; i < (N + 3) / 4; ++i) z[i] = 0u;
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (j < n) z[j / 4] |= (uint32_t)zeros[j] << (8 * (j & 3));
            }
        }
    }
    __device__ __forceinline__ float scale(int j) const {
        if constexpr (TYPE == 0) return __uint_as_float(s[j]);
        else if constexpr (TYPE == 2) return __uint_as_float((j & 1) ? s[j / 2] & 0xFFFF0000u : s[j / 2] << 16);
        else {
            const __half2 h = *reinterpret_cast<const __half2 *>(&s[j / 2]);
            return (j & 1) ? __high2float(h) : __low2float(h);
        }
    }
    template <bool ANY>
    __device__ __forceinline__ W4Zero zero(const W4Unpack<TYPE != 1> &unpack, int j) const {
        if constexpr (!ZEROS) return unpack.eight();
        else return w4_zero<TYPE != 1, ANY>(z[j / 4], j & 3, unpack.magic);
    }
    // Whether a zero point is above 127.
    __device__ __forceinline__ bool high() const {
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < (N + 3) / 4; ++i) any |= z[i];
        return (any & 0x80808080u) != 0;
    }
};

// TYPE: 0 FP32, 1 f16, 2 bf16.  8 * NB columns on the N side.
// Eight warps share 16 rows and split K.  TEAMS: two such teams in one CTA
// where x takes most of shared memory (one for 32 columns: more registers);
// otherwise one, and two CTAs on an SM (4096 x 4096, one row: 5.5 us, with two
// teams in one CTA 6.2; 28672 x 8192, bf16: 31.5 and 30.3).
template <int TYPE, int GROUP, int NB, bool ZEROS, int TEAMS, int MIN_CTAS>
__global__ void __launch_bounds__(TEAMS * 256, MIN_CTAS)
lm_w4_kernel(const __grid_constant__ CUtensorMap tmQ, const W4Args p) {
    constexpr bool BF16 = TYPE != 1;
    constexpr int PLANES = TYPE == 0 ? 3 : 1;
    constexpr int SLOTS = GROUP / 32;                     // words a lane takes of a group and row
    constexpr int NG = 256 / GROUP;                       // groups per step
    constexpr int STAGES = kW4Stages;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char *ring = smem;
    constexpr int WARPS = 8, THREADS = TEAMS * 256;
    float *red = reinterpret_cast<float *>(smem + TEAMS * WARPS * STAGES * 2048);   // [team][2][warp][NB * 4][32]
    uint64_t *bars = reinterpret_cast<uint64_t *>(red + TEAMS * 2 * WARPS * NB * 128);
    unsigned char *xs = reinterpret_cast<unsigned char *>(bars + TEAMS * WARPS * STAGES);   // [column][x_pitch]

    const int lane = threadIdx.x & 31, team = TEAMS == 1 ? 0 : (int)(threadIdx.x >> 8);
    const int warp = (int)(threadIdx.x >> 5) & 7, thread = (int)threadIdx.x & 255;     // of the team
    const int slot = (int)blockIdx.x * TEAMS + team, slots = (int)gridDim.x * TEAMS;
    red += team * (2 * WARPS * NB * 128);
    // The MMA's row lane / 4 (and + 8) is weight row g (and g + 8), in an
    // order in which the rows a shared-memory phase reads meet different
    // banks: rows 0 4 | 1 5 | .. for 16-byte reads, 0 2 4 6 | .. for 8-byte ones.
    const int m = lane >> 2, q = lane & 3;
    const int g = GROUP == 128 ? (m >> 1) | (m & 1) << 2 : GROUP == 64 ? (m >> 2) | (m & 3) << 1 : m;
    // This CTA's slice of K and this warp's steps in it.
    const int k_begin = blockIdx.y * p.k_slice, k_end = min(p.K, k_begin + p.k_slice);
    const int steps = (k_end - k_begin + 255) >> 8;
    const int s0 = steps * warp / WARPS, per = steps * (warp + 1) / WARPS - s0;
    const int k_warp = k_begin + s0 * 256;
    const int blocks = (p.N + 15) >> 4;
    const int mine = blocks > slot ? (blocks - 1 - slot) / slots + 1 : 0;

    // Per warp: a ring of 2 KB stages filled by TMA (16 rows of 128 bytes,
    // 128-byte swizzle: 16-byte piece c of row r sits at c ^ (r % 8); rows
    // past N and columns past K arrive as zeros).
    unsigned char *ring_w = ring + (team * WARPS + warp) * (STAGES * 2048);
    uint64_t *full = bars + (team * WARPS + warp) * STAGES;
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < STAGES; ++i) mbar_init(&full[i], 1);
        fence_barrier_init();
    }
    __syncwarp();
    griddep_launch_dependents();
    griddep_wait();
    int ld_row = slot << 4, ld_s = 0, ld_stage = 0;
    auto issue = [&]() {
        if (ld_row < p.N && per > 0) {
            if (elect_one()) {
                mbar_arrive_expect_tx(&full[ld_stage], 2048);
                tma_load_2d(ring_w + ld_stage * 2048, &tmQ, &full[ld_stage], (k_warp >> 1) + ld_s * 128, ld_row);
            }
            __syncwarp();
            ld_stage = ld_stage == STAGES - 1 ? 0 : ld_stage + 1;
            if (++ld_s == per) {
                ld_s = 0;
                ld_row += slots << 4;
            }
        }
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) issue();

    // x in nibble order (within 8 columns 0 4 1 5 2 6 3 7), the 16 chunks of
    // 128 columns in the order in which the lanes q = 0..3 take them.
    {
        const int chunks = steps * 32, total = chunks * p.tokens;      // chunks of 8 columns
        // Chunk c is word `slot` of lane `lq`; see the loop below.
        auto place = [&](int c) {
            const int in = c & 15;
            const int lq = GROUP == 128 ? in >> 2 : GROUP == 64 ? (in >> 1) & 3 : in & 3;
            const int slot = GROUP == 128 ? in & 3 : GROUP == 64 ? (in >> 3) * 2 + (in & 1) : in >> 2;
            return xs + ((c & ~15) + slot * 4 + lq) * 16;
        };
        auto ordered = [](const uint16_t *v) {
            return make_uint4(v[0] | (uint32_t)v[4] << 16, v[1] | (uint32_t)v[5] << 16,
                              v[2] | (uint32_t)v[6] << 16, v[3] | (uint32_t)v[7] << 16);
        };
        if (TYPE != 0 && p.x_vec && k_end - k_begin == steps * 256) {
            // Whole chunks: several loads on their way at a time.
            constexpr int U = 8;
            for (int i0 = threadIdx.x; i0 < total; i0 += U * THREADS) {
                uint4 v[U];
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int i = min(i0 + j * THREADS, total - 1), t = i / chunks, c = i - t * chunks;
                    v[j] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.X) +
                                                            (int64_t)t * p.ldx + k_begin + c * 8);
                }
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int i = i0 + j * THREADS, t = i / chunks, c = i - t * chunks;
                    if (i < total)
                        *reinterpret_cast<uint4 *>(place(c) + t * p.x_pitch) =
                            make_uint4(__byte_perm(v[j].x, v[j].z, 0x5410), __byte_perm(v[j].x, v[j].z, 0x7632),
                                       __byte_perm(v[j].y, v[j].w, 0x5410), __byte_perm(v[j].y, v[j].w, 0x7632));
                }
            }
        } else {
            for (int i = threadIdx.x; i < total; i += THREADS) {
                const int t = i / chunks, c = i - t * chunks, k = k_begin + c * 8;
                unsigned char *at = place(c);
                if constexpr (TYPE == 0) {
                    const float *sx = static_cast<const float *>(p.X) + (int64_t)t * p.ldx + k;
                    uint16_t v[3][8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float f = k + e < k_end ? sx[e] : 0.f;
                        const uint32_t u = __float_as_uint(f);
                        const bool odd = (u & 0x7F800000u) == 0x7F800000u;
                        const uint32_t h = odd && (u & 0x7FFFFFu) ? 0x7FC00000u : u & 0xFFFF0000u;
                        const float r1 = odd ? 0.f : f - __uint_as_float(h);
                        const uint32_t m = __float_as_uint(r1) & 0xFFFF0000u;
                        v[0][e] = (uint16_t)(h >> 16);
                        v[1][e] = (uint16_t)(m >> 16);
                        v[2][e] = (uint16_t)(__float_as_uint(r1 - __uint_as_float(m)) >> 16);
                    }
#pragma unroll
                    for (int pl = 0; pl < 3; ++pl)
                        *reinterpret_cast<uint4 *>(at + (t * 3 + pl) * p.x_pitch) = ordered(v[pl]);
                } else {
                    const uint16_t *sx = static_cast<const uint16_t *>(p.X) + (int64_t)t * p.ldx + k;
                    uint16_t v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = k + e < k_end ? sx[e] : (uint16_t)0;
                    *reinterpret_cast<uint4 *>(at + t * p.x_pitch) = ordered(v);
                }
            }
        }
    }

    // Scales and zero points come one step ahead of their use.
    W4Meta<TYPE, NG, ZEROS> ma, mb, na, nb;
    constexpr int SB = TYPE == 0 ? 4 : 2;                 // bytes of a scale
    const unsigned char *sa = nullptr, *sb = nullptr;
    const uint8_t *za = nullptr, *zb = nullptr;
    auto point_meta = [&](int row0) {
        const int64_t ra = min(row0 + g, p.N - 1), rb = min(row0 + g + 8, p.N - 1);
        const unsigned char *base = static_cast<const unsigned char *>(p.scales) + (k_warp / GROUP) * SB;
        sa = base + ra * p.lds * SB;
        sb = base + rb * p.lds * SB;
        if constexpr (ZEROS) {
            za = p.zeros + ra * p.ldz + k_warp / GROUP;
            zb = p.zeros + rb * p.ldz + k_warp / GROUP;
        }
    };
    const int n_last = (k_end - k_warp - (per - 1) * 256) / GROUP;     // groups in this warp's last step
    auto load_meta = [&](int s) {
        const int n = s == per - 1 ? min(NG, n_last) : NG;
        na.load(p, sa, za, n);
        nb.load(p, sb, zb, n);
        sa += NG * SB;
        sb += NG * SB;
        if constexpr (ZEROS) {
            za += NG;
            zb += NG;
        }
    };
    if (per > 0 && mine > 0) {
        point_meta(slot << 4);
        load_meta(0);
    }
    __syncthreads();

    const W4Unpack<BF16> unpack;
    // Columns beyond the last take its x: their products go nowhere.
    const int cols = p.tokens * PLANES;
    const unsigned char *x_lane[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) x_lane[n] = xs + (s0 * 32 + q) * 16 + min(n * 8 + m, cols - 1) * p.x_pitch;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int b = 0; b < mine; ++b) {
        const int row0 = (slot + b * slots) << 4;
        float sum[NB][4];
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[n][i] = 0.f;
        for (int s = 0; s < per; ++s) {
            ma = na;
            mb = nb;
            if (s + 1 < per) {
                load_meta(s + 1);
            } else if (b + 1 < mine) {
                point_meta(row0 + (slots << 4));
                load_meta(0);
            }
            const bool landed = ok && mbar_wait_bounded(&full[stage], phase, p.timeout_ns);
            const unsigned char *st = ring_w + stage * 2048 + g * 128;
            uint32_t wa[8], wb[8];
            if constexpr (GROUP == 128) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(st + (((h * 4 + q) ^ g) << 4));
                    const uint4 v = *reinterpret_cast<const uint4 *>(st + 1024 + (((h * 4 + q) ^ g) << 4));
                    wa[4 * h] = u.x; wa[4 * h + 1] = u.y; wa[4 * h + 2] = u.z; wa[4 * h + 3] = u.w;
                    wb[4 * h] = v.x; wb[4 * h + 1] = v.y; wb[4 * h + 2] = v.z; wb[4 * h + 3] = v.w;
                }
            } else if constexpr (GROUP == 64) {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int at = (((h * 2 + (q >> 1)) ^ g) << 4) + (q & 1) * 8;
                    const uint2 u = *reinterpret_cast<const uint2 *>(st + at);
                    const uint2 v = *reinterpret_cast<const uint2 *>(st + 1024 + at);
                    wa[2 * h] = u.x; wa[2 * h + 1] = u.y;
                    wb[2 * h] = v.x; wb[2 * h + 1] = v.y;
                }
            } else {
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    const int at = ((h ^ g) << 4) + q * 4;
                    wa[h] = *reinterpret_cast<const uint32_t *>(st + at);
                    wb[h] = *reinterpret_cast<const uint32_t *>(st + 1024 + at);
                }
            }
            __syncwarp();
            // One answer for the warp: where a wait ran out no copy may be issued
            // into a stage that has one in flight.  (Asked for behind the reads:
            // 28672 x 8192, one row, 26.8 us, ahead of them 27.5.)
            if (__all_sync(~0u, landed)) {
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                if (p.withhold != kWithholdRefill) issue();
            } else {
                if (ok && lane == 0) record_error(p.err, kSiteConsumerFull);
                ok = false;
            }
            // Past the end of K the words are 0 and x is 0: they add nothing.
            auto multiply = [&](auto any) {
                float c[NB][4];
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    const int j = w / SLOTS;
                    const bool first = w % SLOTS == 0;
                    uint32_t a[4], d[4];
                    unpack(wa[w], ma.template zero<decltype(any)::value>(unpack, j), a);
                    unpack(wb[w], mb.template zero<decltype(any)::value>(unpack, j), d);
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(x_lane[n] + s * 512 + w * 64);
                        if (first) mma16816<BF16>(c[n], a[0], d[0], a[1], d[1], x.x, x.y, 0.f, 0.f, 0.f, 0.f);
                        else mma16816<BF16>(c[n], a[0], d[0], a[1], d[1], x.x, x.y, c[n][0], c[n][1], c[n][2], c[n][3]);
                        mma16816<BF16>(c[n], a[2], d[2], a[3], d[3], x.z, x.w, c[n][0], c[n][1], c[n][2], c[n][3]);
                    }
                    if (w % SLOTS == SLOTS - 1) {
                        const float f0 = ma.scale(j), f1 = mb.scale(j);
#pragma unroll
                        for (int n = 0; n < NB; ++n) {
                            sum[n][0] = fmaf(f0, c[n][0], sum[n][0]);
                            sum[n][1] = fmaf(f0, c[n][1], sum[n][1]);
                            sum[n][2] = fmaf(f1, c[n][2], sum[n][2]);
                            sum[n][3] = fmaf(f1, c[n][3], sum[n][3]);
                        }
                    }
                }
            };
            bool high = false;
            if constexpr (ZEROS && BF16) high = __any_sync(~0u, ma.high() || mb.high());
            if (ZEROS && BF16 && high) multiply(std::true_type());
            else multiply(std::false_type());
        }
        // Join the warps' sums (two buffers: a warp may be one block ahead).
        float *buf = red + (b & 1) * (WARPS * NB * 128);
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) buf[(warp * NB * 4 + n * 4 + i) * 32 + lane] = sum[n][i];
        if constexpr (TEAMS == 1) __syncthreads();
        else asm volatile("bar.sync %0, 256;" :: "r"(1 + team) : "memory");
        for (int o = thread; o < 16 * p.tokens; o += 256) {
            const int t = o >> 4, r = o & 15;
            float y = 0.f;
#pragma unroll
            for (int pl = PLANES - 1; pl >= 0; --pl) {
                // Column col of the MMA's row r sits in lane (r % 8) * 4 + (col % 8) / 2,
                // register (r / 8) * 2 + col % 2 of block col / 8.
                const int col = t * PLANES + pl;
                const int r7 = r & 7;                     // row -> the MMA's row
                const int mr = GROUP == 128 ? (r7 & 3) << 1 | r7 >> 2 : GROUP == 64 ? (r7 & 1) << 2 | r7 >> 1 : r7;
                const int at = ((col >> 3) * 4 + (r >> 3) * 2 + (col & 1)) * 32 + mr * 4 + ((col & 7) >> 1);
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) v += buf[w * NB * 128 + at];
                y += v;
            }
            const int n = row0 + r;
            if (n < p.N) {
                if (p.part != nullptr) {
                    p.part[((int64_t)blockIdx.y * p.tokens + t) * p.ld_part + n] = y;
                } else if constexpr (TYPE == 0) {
                    static_cast<float *>(p.Y)[(int64_t)t * p.ldy + n] = y;
                } else if constexpr (TYPE == 1) {
                    static_cast<__half *>(p.Y)[(int64_t)t * p.ldy + n] = __float2half_rn(y);
                } else {
                    static_cast<__nv_bfloat16 *>(p.Y)[(int64_t)t * p.ldy + n] = __float2bfloat16_rn(y);
                }
            }
        }
    }
    // After a wait ran out: the copies still in flight (the stage waited for and
    // those issued behind it) have to land before the CTA may exit.
    if (!ok)
        while (stage != ld_stage) {
            mbar_wait_bounded(&full[stage], phase, p.timeout_ns);
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
}

template <int TYPE, int GROUP, bool ZEROS>
const void *w4_kernel_by_size(int nb, bool alone) {
    if (nb == 1)
        return alone ? reinterpret_cast<const void *>(&lm_w4_kernel<TYPE, GROUP, 1, ZEROS, 2, 1>)
                     : reinterpret_cast<const void *>(&lm_w4_kernel<TYPE, GROUP, 1, ZEROS, 1, 2>);
    if (nb == 2)
        return alone ? reinterpret_cast<const void *>(&lm_w4_kernel<TYPE, GROUP, 2, ZEROS, 2, 1>)
                     : reinterpret_cast<const void *>(&lm_w4_kernel<TYPE, GROUP, 2, ZEROS, 1, 2>);
    return reinterpret_cast<const void *>(&lm_w4_kernel<TYPE, GROUP, 4, ZEROS, 1, 1>);
}
template <int TYPE, bool ZEROS>
const void *w4_kernel_by_group(int group, int nb, bool alone) {
    return group == 32 ? w4_kernel_by_size<TYPE, 32, ZEROS>(nb, alone)
         : group == 64 ? w4_kernel_by_size<TYPE, 64, ZEROS>(nb, alone)
                       : w4_kernel_by_size<TYPE, 128, ZEROS>(nb, alone);
}

}  // namespace sg
