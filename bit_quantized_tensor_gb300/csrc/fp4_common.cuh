// Microscaled 4-bit floating point: formats, packed layout and conversions
// shared by the quantizers, the products and the norm that feeds them.
//
// A value is e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and negatives) times the scale
// of its block along the reduction axis, times a scale of the whole tensor:
//   nv: blocks of 16, e4m3 block scale  s = e4m3(fl(amax / fl(6 ts))), at most
//       448, tensor scale ts (fp32);
//   mx: blocks of 32, e8m0 block scale  s = 2^(floor(log2 amax) - 2), no
//       tensor scale (1).
// With d = fl(s ts) and r = fl(1 / d), at most the largest fp32 number, the code of x
// is fl(x r) rounded to e2m1, ties to even, saturated at +-6; a block whose scale is 0
// gets codes 0.
// A block that holds an infinity or a NaN gets the format's NaN scale.
//
// Packed layout of a rows x K operand:
//   codes  : rows of codes_ld(K) bytes, the even position in the low nibble,
//            zero behind K;
//   scales : 512-byte tiles of 128 rows x 4 blocks, row-block major; row r,
//            block c of a tile at byte 16 (r % 32) + 4 (r / 32) + c.  This is
//            the order in which tcgen05.cp 32x128b puts scales into tensor
//            memory (lane r % 32, column r / 32, byte c), so a tile moves from
//            global memory to the tensor core untouched.
#pragma once
#include <atomic>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "qg_internal.h"

namespace qg {

constexpr int kNv = QG_FP4_NV, kMx = QG_FP4_MX;

__host__ __device__ constexpr int fp4_block(int fmt) { return fmt == kNv ? 16 : 32; }
__host__ __device__ inline int64_t fp4_codes_ld(int64_t K) { return (K + 31) / 32 * 16; }
__host__ __device__ inline int64_t fp4_col_tiles(int fmt, int64_t K) {
    const int64_t b = fp4_block(fmt);
    return ((K + b - 1) / b + 3) / 4;
}
__host__ __device__ inline int64_t fp4_scale_bytes(int fmt, int64_t rows, int64_t K) {
    return (rows + 127) / 128 * fp4_col_tiles(fmt, K) * 512;
}
// Byte of the scale of (row, block) among `col_tiles` tiles a row-block.
__host__ __device__ inline int64_t fp4_scale_offset(int64_t row, int64_t blk, int64_t col_tiles) {
    return ((row >> 7) * col_tiles + (blk >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (blk & 3);
}

// ------------------------------------------------------- element types

template <class T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Two values from / to one 32-bit word of a 16-bit type.
template <class T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// N consecutive values; p is 16-byte aligned and all N exist.
template <class T, int N>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[N]) {
    if constexpr (sizeof(T) == 4) {
        static_assert(N % 4 == 0, "16-byte pieces");
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + i);
            x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
        }
    } else {
        static_assert(N % 8 == 0, "16-byte pieces");
#pragma unroll
        for (int i = 0; i < N; i += 8) {
            const uint4 v = *reinterpret_cast<const uint4*>(p + i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = unpack2<T>(w[j]);
                x[i + 2 * j] = f.x;
                x[i + 2 * j + 1] = f.y;
            }
        }
    }
}

template <class T, int N>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[N]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 8)
            *reinterpret_cast<uint4*>(p + i) =
                make_uint4(pack2<T>(x[i], x[i + 1]), pack2<T>(x[i + 2], x[i + 3]),
                           pack2<T>(x[i + 4], x[i + 5]), pack2<T>(x[i + 6], x[i + 7]));
    }
}

// 16 values in whole 32-byte sectors (p 32-byte aligned), one store a sector.
template <class T>
__device__ __forceinline__ void store_sectors(T* p, const float (&x)[16]) {
    constexpr int PER = 32 / static_cast<int>(sizeof(T));
#pragma unroll
    for (int i = 0; i < 16; i += PER) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (sizeof(T) == 4)
                w[j] = __float_as_uint(x[i + j]);
            else
                w[j] = pack2<T>(x[i + 2 * j], x[i + 2 * j + 1]);
        }
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + i), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    }
}

// N consecutive values of which the first `n` exist (the rest read as 0).
template <class T, int N>
__device__ __forceinline__ void load_some(const T* p, int n, bool aligned, float (&x)[N]) {
    if (aligned && n >= N) {
        load_vec<T, N>(p, x);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = i < n ? to_f32<T>(p[i]) : 0.f;
    }
}

template <class T, int N>
__device__ __forceinline__ void store_some(T* p, int n, bool aligned, const float (&x)[N]) {
    if (aligned && n >= N) {
        store_vec<T, N>(p, x);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) p[i] = from_f32<T>(x[i]);
    }
}

// ------------------------------------------------------- scales and codes

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3);
    return __half2float(__half(h));
}

__device__ __forceinline__ float e8m0_value(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23);
}

template <int FMT>
__device__ __forceinline__ float scale_value(uint32_t byte) {
    return FMT == kNv ? e4m3_value(byte) : e8m0_value(byte);
}

// Scale byte of a block and the factor r its values are multiplied by.
// `amax_bits` is the largest |x| of the block as bits: as unsigned numbers
// they order like the magnitudes, with infinity and NaN above all others.
struct BlockScale {
    uint32_t byte;
    float r;
};

// e4m3(fl(amax / six_ts)).  The product with inv_six = fl(1 / six_ts) is within
// 2^-22 of the quotient, so both round to the same e4m3 number unless it lies
// within 4 units of the last place of the middle between two of them, or
// below 2^-6, where they lie closer: then the division itself is done.
__device__ __forceinline__ uint32_t nv_scale_byte(uint32_t amax_bits, float six_ts, float inv_six) {
    float q = __fmul_rn(__uint_as_float(amax_bits), inv_six);
    const uint32_t low = (__float_as_uint(q) & 0xfffffu) - 0x7fffcu;  // distance from the middle, + 4
    if (low <= 8u || !(q >= 0x1p-6f)) q = __fdiv_rn(__uint_as_float(amax_bits), six_ts);
    return __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
}

// What a kernel needs of the tensor scale.  inv_six is 0 where 1 / six is no normal
// number (ts below 2^-130 or above 2^123): then every block takes the division.
struct TensorScale {
    float ts, six, inv_six;
};
__device__ __forceinline__ TensorScale tensor_scale(const float* ts) {
    TensorScale t;
    t.ts = ts ? *ts : 1.f;
    t.six = __fmul_rn(6.f, t.ts);
    t.inv_six = __frcp_rn(t.six);
    if (!(t.inv_six >= 0x1p-126f && t.inv_six <= 0x1.fffffep+127f)) t.inv_six = 0.f;
    return t;
}

// r of every e4m3 byte (128 of them); at most the largest number, since 0 times an
// infinity would not be 0.
__device__ __forceinline__ float nv_factor(uint32_t byte, float ts) {
    return byte && byte < 127 ? fminf(__frcp_rn(__fmul_rn(e4m3_value(byte), ts)), 0x1.fffffep+127f) : 0.f;
}

template <int FMT>
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits, const TensorScale& t) {
    BlockScale b;
    if constexpr (FMT == kNv) {
        b.byte = amax_bits >= 0x7f800000u ? 0x7fu : nv_scale_byte(amax_bits, t.six, t.inv_six);
        b.r = nv_factor(b.byte, t.ts);
    } else {
        const uint32_t e = amax_bits >> 23;  // floor(log2) + 127; 0 below 2^-126
        b.byte = e > 2 ? e - 2 : 0;
        // 2^(127 - byte): bits (254 - byte) << 23; byte <= 252, so it is normal
        b.r = __uint_as_float((254u - b.byte) << 23);
        if (amax_bits >= 0x7f800000u) b = {0xffu, 0.f};
    }
    return b;
}

// The same with the factors of all bytes in shared memory (128 floats, nv).
__device__ __forceinline__ void fill_factors(float* table, float ts) {
    for (int i = threadIdx.x; i < 128; i += blockDim.x) table[i] = nv_factor(i, ts);
}
template <int FMT>
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits, const TensorScale& t, const float* table) {
    if constexpr (FMT == kNv) {
        const uint32_t byte = amax_bits >= 0x7f800000u ? 0x7fu : nv_scale_byte(amax_bits, t.six, t.inv_six);
        return {byte, table[byte]};
    } else {
        return block_scale<FMT>(amax_bits, t);
    }
}

// Eight values to eight e2m1 codes (round to nearest, ties to even, saturated
// at 6), value i in nibble i.
__device__ __forceinline__ uint32_t e2m1x8(const float* x) {
    uint32_t r;
    asm("{\n.reg .b8 b0, b1, b2, b3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        "mov.b32 %0, {b0, b1, b2, b3};\n}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

// Eight codes to eight values, exact.
__device__ __forceinline__ void e2m1x8_values(uint32_t w, float (&x)[8]) {
    uint32_t h[4];
    asm("{\n.reg .b8 b0, b1, b2, b3;\n"
        "mov.b32 {b0, b1, b2, b3}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<__half>(h[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <int N>
__device__ __forceinline__ uint32_t absmax_bits(const float (&x)[N]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    return m;
}

// The codes of 8 values times r.
__device__ __forceinline__ uint32_t scaled_codes8(const float* x, float r) {
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        uint64_t p, f;
        asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x[j]), "f"(x[j + 1]));
        asm("mov.b64 %0, {%1, %1};" : "=l"(f) : "f"(r));
        asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(p) : "l"(f));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(y[j]), "=f"(y[j + 1]) : "l"(p));
    }
    return e2m1x8(y);
}

// One block of a row: its codes (BLOCK / 8 words) and its scale byte.
template <int FMT>
__device__ __forceinline__ uint32_t quantize_block(const float (&x)[fp4_block(FMT)], const TensorScale& t,
                                                   uint32_t (&codes)[fp4_block(FMT) / 8]) {
    constexpr int B = fp4_block(FMT);
    const BlockScale s = block_scale<FMT>(absmax_bits<B>(x), t);
#pragma unroll
    for (int i = 0; i < B; i += 8) codes[i / 8] = scaled_codes8(x + i, s.r);
    return s.byte;
}

// The same for a block that is still packed in words of T (two 16-bit values
// each): the maximum is found on the packed words.
template <class T>
__device__ __forceinline__ uint32_t packed_amax_bits(uint32_t m) {  // the larger half of m, as fp32 bits
    const uint32_t h = max(m & 0xffffu, m >> 16);
    if constexpr (std::is_same<T, __half>::value)
        return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(h))));
    else
        return h << 16;
}
template <int FMT, class T, int WORDS>
__device__ __forceinline__ uint32_t quantize_words(const uint32_t (&w)[WORDS], const TensorScale& t,
                                                   const float* table, uint32_t (&codes)[fp4_block(FMT) / 8]) {
    constexpr int B = fp4_block(FMT);
    static_assert(WORDS * 4 == B * static_cast<int>(sizeof(T)), "one block");
    if constexpr (sizeof(T) == 4) {
        float x[B];
#pragma unroll
        for (int i = 0; i < B; ++i) x[i] = __uint_as_float(w[i]);
        const BlockScale s = block_scale<FMT>(absmax_bits<B>(x), t, table);
#pragma unroll
        for (int i = 0; i < B; i += 8) codes[i / 8] = scaled_codes8(x + i, s.r);
        return s.byte;
    } else {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
        const BlockScale s = block_scale<FMT>(packed_amax_bits<T>(m), t, table);
#pragma unroll
        for (int i = 0; i < WORDS; i += 4) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = unpack2<T>(w[i + j]);
                x[2 * j] = f.x;
                x[2 * j + 1] = f.y;
            }
            codes[i / 4] = scaled_codes8(x, s.r);
        }
        return s.byte;
    }
}

// N values as they lie in memory, the first n of them existing (the rest 0).
template <class T, int N>
__device__ __forceinline__ void load_words(const T* p, int n, bool aligned, uint32_t (&w)[N * sizeof(T) / 4]) {
    constexpr int W = N * static_cast<int>(sizeof(T)) / 4;
    if (aligned && n >= N) {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
            w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
        }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = i < n ? reinterpret_cast<const uint32_t*>(p)[i] : 0u;
    } else {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < W; ++i)
            w[i] = (2 * i < n ? h[2 * i] : 0u) | (2 * i + 1 < n ? static_cast<uint32_t>(h[2 * i + 1]) << 16 : 0u);
    }
}

// ------------------------------------------------------- host

constexpr int64_t kMaxGridY = 65535;  // of a grid's y and z

inline size_t dtype_bytes(int dtype) { return dtype == QG_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == QG_F16 || dtype == QG_BF16 || dtype == QG_F32; }
inline bool fmt_ok(int fmt) { return fmt == kNv || fmt == kMx; }

// Launches with programmatic stream serialization: the kernel may be set up
// while the one before it on the stream drains.  Every kernel launched this
// way begins with pdl_wait_prior_grid() before it reads or writes memory that
// an earlier call may use, and lets its own successor start only after that.
// Inputs may thus be written while it already runs: its parameters are not
// `const ... __restrict__` and nothing is read with __ldg, which promise the opposite.
template <class F, class... Args>
int launch_serialized(F* kernel, dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream,
                      Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return map_cuda(cudaLaunchKernelEx(&cfg, kernel, args...));
}

// Lifts the kernel's limit of dynamic shared memory to all that a CTA can have, once per
// device; each kernel is called with a type of its own as TAG, which keeps its flags.
// The limit of a call's own size would not do: another thread's launch, with less, could
// lower it again between the two calls.
template <class TAG, class F>
int raise_smem(F* kernel) {
    static std::atomic<bool> done[64] = {};
    const int dev = current_device();
    if (dev < 0 || dev >= 64) return QG_ERR_CUDA;
    if (done[dev].load(std::memory_order_acquire)) return QG_OK;
    cudaFuncAttributes a;
    cudaError_t e = cudaFuncGetAttributes(&a, kernel);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 232448 - static_cast<int>(a.sharedSizeBytes));
    if (e != cudaSuccess) return map_cuda(e);
    done[dev].store(true, std::memory_order_release);
    return QG_OK;
}

// Calls f with a value of the C++ type of `dtype`.
template <class F>
int by_dtype(int dtype, F&& f) {
    if (dtype == QG_F16) return f(__half{});
    if (dtype == QG_BF16) return f(__nv_bfloat16{});
    return f(float{});
}

// Quantizers (qg_fp4_quant.cu); arguments already checked.
int fp4_quantize_run(int fmt, int dtype, int64_t M, int64_t K, const void* X, int64_t ldx, const float* ts,
                     uint8_t* Xq, uint8_t* Xs, bool zero_pad, cudaStream_t s);
int fp4_quantize_both_run(int fmt, int dtype, int64_t M, int64_t K, const void* X, int64_t ldx, const float* ts,
                          uint8_t* Xq, uint8_t* Xs, uint8_t* Tq, uint8_t* Ts, float* colsum, float* partial,
                          cudaStream_t s);

// Adds `parts` rows of n partial sums, in order, into out (qg_norm.cu).
int sum_partials_run(const float* partial, int64_t parts, int64_t n, float* out, cudaStream_t s);

}  // namespace qg
