// 8-bit integer operands with a scale for each row: the row of a matrix of
// activations is a token, that of a weight matrix an output channel.
//   s = max(fl(amax / 127), 2^-100),  r = fl(1 / s),  q = clamp(rint(fl(x r)), -127, 127)
// A row that holds an infinity or a NaN has the scale NaN and codes 0.
// Codes: rows x s8_codes_ld(K) bytes (K up to whole 16 bytes), 0 behind K.
#pragma once
#include <cuda_fp16.h>

#include "fp4_common.cuh"
#include "qg_ptx.cuh"

namespace qg {

constexpr float kRowScaleFloor = 0x1p-100f;

__host__ __device__ inline int64_t s8_codes_ld(int64_t K) { return (K + 15) / 16 * 16; }

// |x| as bits: unsigned numbers that order like the magnitudes, infinity and NaN above all.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ bool bits_finite(uint32_t amax_bits) { return amax_bits < 0x7f800000u; }

// Scale of values whose largest magnitude is `amax_bits`, at least `least`.
__device__ __forceinline__ float s8_scale(uint32_t amax_bits, float least) {
    return bits_finite(amax_bits) ? fmaxf(__fdiv_rn(__uint_as_float(amax_bits), 127.f), least)
                                  : __uint_as_float(0x7fc00000u);
}
// r; 0 for a scale that is NaN, so that every code is 0 (x r is NaN for a NaN, code 0 as well).
__device__ __forceinline__ float s8_inverse(float scale) { return scale == scale ? __fdiv_rn(1.f, scale) : 0.f; }
// fl(x r) rounded to a whole number, ties to even, by adding 1.5 * 2^23: the sum's unit is 1, its
// low byte the code (conversions to integers run at an eighth of this rate).  No clamp is needed:
// |x| <= 127 s (1 + 2^-24), so |fl(x r)| < 127.5.  Not for r = 0, where x may be infinite or NaN.
__device__ __forceinline__ float s8_shifted(float x, float r) { return __fadd_rn(__fmul_rn(x, r), 12582912.f); }
// Codes in a word, the first in the low byte; 0 for r = 0.
__device__ __forceinline__ uint32_t s8_pack(const float* x, float r) {
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __float_as_uint(s8_shifted(x[i], r));
    return r == 0.f ? 0u : __byte_perm(__byte_perm(y[0], y[1], 0x0040), __byte_perm(y[2], y[3], 0x0040), 0x5410);
}
// The code as a number.
__device__ __forceinline__ float s8_number(float x, float r) {
    return r == 0.f ? 0.f : __fadd_rn(s8_shifted(x, r), -12582912.f);
}

// sum sa sb + bias, the scale of the smaller magnitude first: fl(sum) times the larger one alone can
// be infinite where the result is not.  Scales that are NaN stay.
__device__ __forceinline__ float s8_scaled(int sum, float sa, float sb, float bias) {
    const bool less = fabsf(sa) < fabsf(sb);
    return fmaf(static_cast<float>(sum) * (less ? sa : sb), less ? sb : sa, bias);
}

// Four whole numbers' low bytes in a word, the first in the low byte.
__device__ __forceinline__ uint32_t pack_s8(int a, int b, int c, int d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// The four codes of a word as fp16 pairs, exact: the byte XOR 0x80 (offset binary)
// under the exponent of 1024 is 1024 + q + 128, and 1152 less is q.
__device__ __forceinline__ void s8_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const __half2 c1152 = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    w ^= 0x80808080u;
    const uint32_t l = __byte_perm(w, 0x64646464u, 0x4140), h = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&l), c1152);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&h), c1152);
    lo = *reinterpret_cast<const uint32_t*>(&a);
    hi = *reinterpret_cast<const uint32_t*>(&b);
}

// Eight values of a row as they lie in memory, 0 from the n-th on.
template <class T>
struct S8Piece {
    static constexpr int WORDS = 2 * static_cast<int>(sizeof(T));
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const T* p, int n, bool aligned) {
        if (aligned && n >= 8) {
#pragma unroll
            for (int i = 0; i < WORDS / 4; ++i) {
                const uint4 v = reinterpret_cast<const uint4*>(p)[i];
                w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
            }
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = i < n ? __float_as_uint(p[i]) : 0u;
        } else {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = (2 * i < n ? h[2 * i] : 0u) | (2 * i + 1 < n ? static_cast<uint32_t>(h[2 * i + 1]) << 16 : 0u);
        }
    }
    __device__ __forceinline__ void values(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            if constexpr (sizeof(T) == 4) {
                x[i] = __uint_as_float(w[i]);
            } else {
                const float2 f = unpack2<T>(w[i]);
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            }
        }
    }
    // The running maximum of the magnitudes' bits, of 16-bit types in either half of the word
    // (half the work of doing it behind the conversion), and its fp32 bits.
    __device__ __forceinline__ uint32_t largest(uint32_t m) const {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            if constexpr (sizeof(T) == 4)
                m = max(m, w[i] & 0x7fffffffu);
            else
                m = __vmaxu2(m, w[i] & 0x7fff7fffu);
        }
        return m;
    }
    __device__ __forceinline__ static uint32_t bits(uint32_t m) {
        if constexpr (sizeof(T) == 4) {
            return m;
        } else {
            const float2 f = unpack2<T>(m);
            return max(abs_bits(f.x), abs_bits(f.y));
        }
    }
};

__device__ __forceinline__ uint32_t warp_max_u32(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

// D += A . B of 16 x 16 by 16 x 8 fp16 values.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

}  // namespace qg
