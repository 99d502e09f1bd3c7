// Products of a few rows with 4-bit weights and group scales:
//
//   y[t, n] = sum_g s[n, g] sum_{k in g} (q[n, k] - z[n, g]) x[t, k]
//
// The weights are read once (half a byte each) and that read bounds the
// product, so everything else is kept off its way:
//   * each warp streams 16 weight rows, 128 columns (1 KB) at a time, through
//     its own ring of asynchronous copies;
//   * q - z is an integer of at most 5 bits, exact in f16 and bf16, so the
//     weights meet x in the tensor core unscaled (mma.sync m16n8k16, the rows
//     of W on the M side, 8 tokens on the N side) and the scale is applied to
//     the FP32 sum of its group: no weight is ever rounded.  A nibble becomes
//     a float by one logic operation (its bits under those of 128 or 1024)
//     and one subtraction, for two weights at a time;
//   * the order of k inside a group is free as long as both operands agree:
//     the lane that unpacks a 32-bit word (8 weights) multiplies it with the
//     8 x values of the same columns, kept in shared memory in the order in
//     which the nibbles come out;
//   * FP32 x is held as three bf16 planes (exactly), as three tokens.
// The eight warps of a CTA share 16 rows and split K; their sums are joined
// in a fixed order through shared memory.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "lm_w4.h"
#include "ptx.cuh"

namespace sg {

constexpr int kW4Warps = 8, kW4Stages = 5;
constexpr int kW4RowBytes = 80;                          // 64 bytes of a row, padded off bank conflicts
constexpr int kW4StageBytes = 16 * kW4RowBytes;
constexpr int kW4RingBytes = kW4Warps * kW4Stages * kW4StageBytes;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    const uint32_t n = valid ? 16u : 0u;
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two nibbles (bits 0-3 and 16-19 of w) -> two 16-bit floats q - z; `zero`
// holds 128 + z (bf16) or 1024 + z (f16) twice.
template <bool BF16>
__device__ __forceinline__ uint32_t unpack2(uint32_t w, uint32_t zero) {
    const uint32_t magic = BF16 ? 0x43004300u : 0x64006400u;
    const uint32_t v = (w & 0x000F000Fu) | magic;
    uint32_t r;
    if constexpr (BF16) {
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v),
                                         *reinterpret_cast<const __nv_bfloat162 *>(&zero));
        r = *reinterpret_cast<const uint32_t *>(&d);
    } else {
        const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&v), *reinterpret_cast<const __half2 *>(&zero));
        r = *reinterpret_cast<const uint32_t *>(&d);
    }
    return r;
}

template <int TYPE>
__device__ __forceinline__ float w4_scale(const void *scales, int64_t i) {
    if constexpr (TYPE == 0) return static_cast<const float *>(scales)[i];
    else if constexpr (TYPE == 1) return __half2float(static_cast<const __half *>(scales)[i]);
    else return __bfloat162float(static_cast<const __nv_bfloat16 *>(scales)[i]);
}

// TYPE: 0 FP32, 1 f16, 2 bf16.  COLS = 8 * NB columns on the N side.
template <int TYPE, int GROUP, int NB>
__global__ void __launch_bounds__(kW4Warps * 32)
lm_w4_kernel(const W4Args p) {
    constexpr bool BF16 = TYPE != 1;
    constexpr int PLANES = TYPE == 0 ? 3 : 1;
    constexpr int SLOTS = GROUP / 32;                     // 32-column slots per group
    constexpr int NG = 4 / SLOTS;                         // groups per step of 128
    extern __shared__ __align__(128) unsigned char smem_raw[];
    unsigned char *ring = smem_raw;
    float *red = reinterpret_cast<float *>(smem_raw + kW4RingBytes);          // [2][warp][NB * 4][32]
    unsigned char *xs = smem_raw + kW4RingBytes + 2 * kW4Warps * NB * 512;    // [column][x_pitch bytes]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, q = lane & 3;
    // This CTA's slice of K and this warp's steps in it.
    const int k_begin = blockIdx.y * p.k_slice, k_end = min(p.K, k_begin + p.k_slice);
    const int steps = (k_end - k_begin + 127) >> 7;
    const int s0 = steps * warp / kW4Warps, s1 = steps * (warp + 1) / kW4Warps;
    const int per = s1 - s0;
    const int blocks = (p.N + 15) >> 4;
    const int mine = blocks > (int)blockIdx.x ? (blocks - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;

    griddep_launch_dependents();
    griddep_wait();

    const uint32_t ring_w = smem_u32(ring) + warp * (kW4Stages * kW4StageBytes);
    // Copies of step i (of this warp's sequence) into stage i % kW4Stages.
    int ld_b = 0, ld_s = 0, ld_stage = 0;
    auto issue = [&]() {
        if (ld_b < mine) {
            const int row0 = ((int)blockIdx.x + ld_b * (int)gridDim.x) << 4;
            const int k0 = k_begin + (s0 + ld_s) * 128;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int id = lane + 32 * i, r = id >> 2, piece = id & 3;
                const int row = min(row0 + r, p.N - 1);
                const bool valid = k0 + piece * 32 < k_end;
                const uint8_t *src = p.Q + (int64_t)row * p.ldq + ((valid ? k0 + piece * 32 : k_begin) >> 1);
                cp_async16(ring_w + ld_stage * kW4StageBytes + r * kW4RowBytes + piece * 16, src, valid);
            }
            if (++ld_s == per) { ld_s = 0; ++ld_b; }
            if (++ld_stage == kW4Stages) ld_stage = 0;
        }
        cp_async_commit();
    };
    if (per > 0)
#pragma unroll
        for (int i = 0; i < kW4Stages - 1; ++i) issue();

    // x in nibble order: within 8 columns, 0 4 1 5 2 6 3 7.
    {
        const int chunks = steps * 16;                    // of 8 columns
        for (int i = threadIdx.x; i < chunks * p.tokens; i += kW4Warps * 32) {
            const int t = i / chunks, c = i - t * chunks, k = k_begin + c * 8;
            if constexpr (TYPE == 0) {
                const float *src = static_cast<const float *>(p.X) + (int64_t)t * p.ldx + k;
                uint16_t v[3][8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float f = k + e < k_end ? src[e] : 0.f;
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
                for (int pl = 0; pl < 3; ++pl) {
                    uint4 o;
                    o.x = v[pl][0] | (uint32_t)v[pl][4] << 16;
                    o.y = v[pl][1] | (uint32_t)v[pl][5] << 16;
                    o.z = v[pl][2] | (uint32_t)v[pl][6] << 16;
                    o.w = v[pl][3] | (uint32_t)v[pl][7] << 16;
                    *reinterpret_cast<uint4 *>(xs + (int64_t)(t * 3 + pl) * p.x_pitch + c * 16) = o;
                }
            } else {
                const uint16_t *src = static_cast<const uint16_t *>(p.X) + (int64_t)t * p.ldx + k;
                uint16_t v[8];
                if (p.x_vec && k + 8 <= k_end) {
                    *reinterpret_cast<uint4 *>(v) = *reinterpret_cast<const uint4 *>(src);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = k + e < k_end ? src[e] : (uint16_t)0;
                }
                uint4 o;
                o.x = v[0] | (uint32_t)v[4] << 16;
                o.y = v[1] | (uint32_t)v[5] << 16;
                o.z = v[2] | (uint32_t)v[6] << 16;
                o.w = v[3] | (uint32_t)v[7] << 16;
                *reinterpret_cast<uint4 *>(xs + (int64_t)t * p.x_pitch + c * 16) = o;
            }
        }
    }
    __syncthreads();

    const int cols = p.tokens * PLANES;
    const uint32_t zsym = BF16 ? 0x43084308u : 0x64086408u;
    int stage = 0;
    for (int b = 0; b < mine; ++b) {
        const int row0 = ((int)blockIdx.x + b * (int)gridDim.x) << 4;
        const int ra = min(row0 + g, p.N - 1), rb = min(row0 + g + 8, p.N - 1);
        float sum[NB][4];
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[n][i] = 0.f;
        for (int s = 0; s < per; ++s) {
            const int k0 = k_begin + (s0 + s) * 128;
            const int live = min(4, (k_end - k0 + 31) >> 5);      // slots that exist
            // Scales and zero points of this step's groups.
            float sc[NG][2];
            uint32_t zc[NG][2];
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const int64_t gi = (k0 / GROUP) + j;
                const bool in = j * SLOTS < live;
                sc[j][0] = in ? w4_scale<TYPE>(p.scales, ra * p.lds + gi) : 0.f;
                sc[j][1] = in ? w4_scale<TYPE>(p.scales, rb * p.lds + gi) : 0.f;
                zc[j][0] = zc[j][1] = zsym;
                if (p.zeros != nullptr && in) {
                    const uint32_t base = BF16 ? 0x4300u : 0x6400u;
                    zc[j][0] = (base | (p.zeros[ra * p.ldz + gi] & 15u)) * 0x10001u;
                    zc[j][1] = (base | (p.zeros[rb * p.ldz + gi] & 15u)) * 0x10001u;
                }
            }
            cp_async_wait<kW4Stages - 2>();
            __syncwarp();
            const unsigned char *st = ring + warp * (kW4Stages * kW4StageBytes) + stage * kW4StageBytes;
            uint32_t wa[4], wb[4];
#pragma unroll
            for (int slot = 0; slot < 4; ++slot) {
                wa[slot] = *reinterpret_cast<const uint32_t *>(st + g * kW4RowBytes + slot * 16 + q * 4);
                wb[slot] = *reinterpret_cast<const uint32_t *>(st + (g + 8) * kW4RowBytes + slot * 16 + q * 4);
            }
            __syncwarp();
            issue();
            if (++stage == kW4Stages) stage = 0;
            float c[NB][4];
#pragma unroll
            for (int slot = 0; slot < 4; ++slot) {
                const int j = slot / SLOTS;
                if (slot % SLOTS == 0) {
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) c[n][i] = 0.f;
                }
                if (GROUP == 128 || slot < live) {
                    uint32_t a[4], d[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        a[i] = unpack2<BF16>(wa[slot] >> (4 * i), zc[j][0]);
                        d[i] = unpack2<BF16>(wb[slot] >> (4 * i), zc[j][1]);
                    }
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        const int col = n * 8 + g;
                        uint4 x = make_uint4(0, 0, 0, 0);
                        if (col < cols)
                            x = *reinterpret_cast<const uint4 *>(xs + (int64_t)col * p.x_pitch +
                                                                 ((s0 + s) * 16 + slot * 4 + q) * 16);
                        mma16816<BF16>(c[n], a[0], d[0], a[1], d[1], x.x, x.y);
                        mma16816<BF16>(c[n], a[2], d[2], a[3], d[3], x.z, x.w);
                    }
                }
                if (slot % SLOTS == SLOTS - 1) {
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        sum[n][0] = fmaf(sc[j][0], c[n][0], sum[n][0]);
                        sum[n][1] = fmaf(sc[j][0], c[n][1], sum[n][1]);
                        sum[n][2] = fmaf(sc[j][1], c[n][2], sum[n][2]);
                        sum[n][3] = fmaf(sc[j][1], c[n][3], sum[n][3]);
                    }
                }
            }
        }
        // Join the warps' sums (two buffers: a warp may be one block ahead).
        float *buf = red + (b & 1) * (kW4Warps * NB * 128);
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) buf[(warp * NB * 4 + n * 4 + i) * 32 + lane] = sum[n][i];
        __syncthreads();
        for (int o = threadIdx.x; o < 16 * p.tokens; o += kW4Warps * 32) {
            const int t = o >> 4, r = o & 15;
            float y = 0.f;
#pragma unroll
            for (int pl = PLANES - 1; pl >= 0; --pl) {
                // Column col of row r sits in lane (r % 8) * 4 + (col % 8) / 2,
                // register (r / 8) * 2 + col % 2 of block col / 8.
                const int col = t * PLANES + pl;
                const int at = ((col >> 3) * 4 + (r >> 3) * 2 + (col & 1)) * 32 + (r & 7) * 4 + ((col & 7) >> 1);
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kW4Warps; ++w) v += buf[w * NB * 128 + at];
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
}

template <int TYPE>
const void *w4_kernel_of(int group, int nb) {
    if (group == 32) {
        if (nb == 1) return reinterpret_cast<const void *>(&lm_w4_kernel<TYPE, 32, 1>);
        if (nb == 2) return reinterpret_cast<const void *>(&lm_w4_kernel<TYPE, 32, 2>);
        return reinterpret_cast<const void *>(&lm_w4_kernel<TYPE, 32, 4>);
    }
    if (group == 64) {
        if (nb == 1) return reinterpret_cast<const void *>(&lm_w4_kernel<TYPE, 64, 1>);
        if (nb == 2) return reinterpret_cast<const void *>(&lm_w4_kernel<TYPE, 64, 2>);
        return reinterpret_cast<const void *>(&lm_w4_kernel<TYPE, 64, 4>);
    }
    if (nb == 1) return reinterpret_cast<const void *>(&lm_w4_kernel<TYPE, 128, 1>);
    if (nb == 2) return reinterpret_cast<const void *>(&lm_w4_kernel<TYPE, 128, 2>);
    return reinterpret_cast<const void *>(&lm_w4_kernel<TYPE, 128, 4>);
}

}  // namespace sg
