// Arithmetic of the 8-bit products.  Rows of numbers as 8-bit integers with a scale
// each:
//
//   s = max |x| / 127 (rounded to FP32, at least 2^-126 unless all are 0)
//   q = x / s rounded to the nearest integer, ties to even
//
// The quotient's rounding is exact: r = rint(x * (1 / s)) is at most one off, and
// x - r s, which one fused operation gives without rounding (it is a multiple of
// half a unit of s and no larger than s), says whether a neighbour is nearer.  A
// row with an infinity or a NaN has scale NaN and integers 0, so that products
// with it are NaN.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace sg {

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_float(int8_t x) { return (float)x; }

// Eight neighbours as they are stored, those from n on as 0.
template <class T>
struct Eight {
    alignas(sizeof(T) == 1 ? 8 : 16) T e[8];
    __device__ __forceinline__ void load(const T *p, int64_t n, bool vec) {
        if (vec && n >= 8) {
            if constexpr (sizeof(T) == 1) {
                *reinterpret_cast<uint2 *>(e) = *reinterpret_cast<const uint2 *>(p);
            } else {
#pragma unroll
                for (int i = 0; i < (int)sizeof(T) / 2; ++i)
                    reinterpret_cast<uint4 *>(e)[i] = reinterpret_cast<const uint4 *>(p)[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i < n) e[i] = p[i];
                else e[i] = T(0);
            }
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = T(0);
    }
    // The bits of the largest |x|: infinities and NaN come out on top.
    __device__ __forceinline__ uint32_t most() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(as_float(e[i])) & 0x7FFFFFFFu);
        return m;
    }
};

// Eight numbers as integers: adding 1.5 * 2^23 rounds to the nearest one, ties to
// even, with the integer in the low bits (`t`); r is the same as a float.
struct Rounded {
    float t[8], r[8];
    __device__ __forceinline__ int integer(int i) const { return __float_as_int(t[i]); }        // its low byte
};
constexpr float kMagic = 12582912.f;
template <class T>
__device__ __forceinline__ Rounded nearest(const T (&x)[8], float s, float inv) {
    Rounded q;
    float off = 0.f;
    const float half = 0.5f * s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        q.t[i] = fmaf(as_float(x[i]), inv, kMagic);
        q.r[i] = q.t[i] - kMagic;
        off = fmaxf(off, fabsf(fmaf(-q.r[i], s, as_float(x[i]))));
    }
    if (off >= half) {                  // (seldom) a tie, or a neighbour is nearer
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float rest = fmaf(-q.r[i], s, as_float(x[i])), a = fabsf(rest);
            if (a > half || (a == half && (__float_as_int(q.t[i]) & 1))) {
                q.t[i] += copysignf(1.f, rest);
                q.r[i] = q.t[i] - kMagic;
            }
        }
    }
    return q;
}

// (In f16 the rows are always those of a workspace: aligned, whole chunks.)
template <bool OUT16>
__device__ __forceinline__ void store8(void *out, int64_t at, const Rounded &q, int n, bool vec) {
    if constexpr (OUT16) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(q.r[2 * i], q.r[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(static_cast<__half *>(out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if (n < 8 || !vec) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) static_cast<int8_t *>(out)[at + i] = (int8_t)q.integer(i);
    } else {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = __byte_perm(__byte_perm(q.integer(4 * i), q.integer(4 * i + 1), 0x0040),
                               __byte_perm(q.integer(4 * i + 2), q.integer(4 * i + 3), 0x0040), 0x5410);
        *reinterpret_cast<uint2 *>(static_cast<int8_t *>(out) + at) = make_uint2(w[0], w[1]);
    }
}

// The scale of a row whose largest |x| has the bits `most`.
struct RowScale {
    bool finite;
    float s, inv, scale;                // for the rounding; what the row's scale reads as
    __device__ __forceinline__ explicit RowScale(uint32_t most) {
        finite = most < 0x7F800000u;
        s = most == 0u ? 0.f : fmaxf(__uint_as_float(most) / 127.f, 1.17549435e-38f);
        inv = s > 0.f ? 1.f / s : 0.f;
        scale = finite ? s : __uint_as_float(0x7FC00000u);
    }
};

// Four integers as two pairs of f16: a byte plus 128 under the leading bits of
// 1024, less 1152 (bytes 0 1 and 2 3; a published conversion: Kim et al., 2022).
__device__ __forceinline__ void to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    w ^= 0x80808080u;
    const uint32_t magic = 0x64646464u, less = 0x64806480u;
    const uint32_t l = __byte_perm(w, magic, 0x4140), h = __byte_perm(w, magic, 0x4342);
    const __half2 dl = __hsub2(*reinterpret_cast<const __half2 *>(&l), *reinterpret_cast<const __half2 *>(&less));
    const __half2 dh = __hsub2(*reinterpret_cast<const __half2 *>(&h), *reinterpret_cast<const __half2 *>(&less));
    lo = *reinterpret_cast<const uint32_t *>(&dl);
    hi = *reinterpret_cast<const uint32_t *>(&dh);
}

}  // namespace sg
