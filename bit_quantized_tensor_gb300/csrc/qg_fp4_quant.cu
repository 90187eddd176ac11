// Microscaled 4-bit quantizers: along the rows (fp4_quantize), along rows and
// columns in one pass (fp4_quantize_both), the tensor scale they may use
// (fp4_tensor_scale), and the way back to values (fp4_dequantize).  Formats,
// layout and the rounding rules: fp4_common.cuh.
#include "fp4_common.cuh"
#include "qg_ptx.cuh"

namespace qg {

// ------------------------------------------------------- along the rows
//
// One thread quantizes one block: its 16 or 32 values come in 16-byte loads,
// the maximum and the codes stay in its registers, and the scale bytes of the
// four blocks of a scale tile's row go out as one word through two shuffles.
// Bound by memory: 2 or 4 bytes in and 0.56 (nv) or 0.53 (mx) out per value.
constexpr int kQuantThreads = 256;

template <int FMT, class T>
__global__ void __launch_bounds__(kQuantThreads)
    k_fp4_quantize(int64_t M, int64_t rows, int64_t K, const T* __restrict__ X, int64_t ldx, bool aligned,
                   const float* __restrict__ tscale, uint8_t* __restrict__ Xq, uint8_t* __restrict__ Xs) {
    constexpr int B = fp4_block(FMT);
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int64_t tiles = fp4_col_tiles(FMT, K);
    const int64_t per_row = 4 * tiles;  // blocks of a row, up to whole scale words
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kQuantThreads + threadIdx.x;
    const int64_t row = item / per_row, blk = item - row * per_row;
    if (row >= rows) return;  // per_row is a multiple of 4: groups of 4 lanes leave together
    const float ts = FMT == kNv && tscale ? *tscale : 1.f;
    const float six_ts = __fmul_rn(6.f, ts);
    uint32_t byte = 0;
    const int64_t k0 = blk * B, ld = fp4_codes_ld(K);
    if (row < M && k0 < 2 * ld) {
        uint32_t codes[B / 8];
        if (k0 < K) {
            float x[B];
            load_some<T, B>(X + row * ldx + k0, static_cast<int>(min(K - k0, int64_t(B))), aligned, x);
            byte = quantize_block<FMT>(x, ts, six_ts, codes);
        } else {
#pragma unroll
            for (int i = 0; i < B / 8; ++i) codes[i] = 0;
        }
        uint8_t* q = Xq + row * ld + k0 / 2;
        if constexpr (B == 16)
            *reinterpret_cast<uint2*>(q) = make_uint2(codes[0], codes[1]);
        else
            *reinterpret_cast<uint4*>(q) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
    }
    const uint32_t quad = 0xfu << (threadIdx.x & 28);
    uint32_t word = byte << (8 * (threadIdx.x & 3));
    word |= __shfl_xor_sync(quad, word, 1);
    word |= __shfl_xor_sync(quad, word, 2);
    if ((threadIdx.x & 3) == 0) *reinterpret_cast<uint32_t*>(Xs + fp4_scale_offset(row, blk, tiles)) = word;
}

// ------------------------------------------------------- rows and columns
//
// A CTA takes a tile of 128 x 128 values through shared memory once and
// quantizes it along both axes: X (blocks along a row) and X^T (blocks along
// a column), as a training step needs an operand once for each of its two
// products.  The tile also gives the column sums (the bias gradient).
constexpr int kBothThreads = 256;
constexpr int kTile = 128;

template <class T>
struct BothSmem {
    // 4-byte words a row: odd, so that a warp walking down a column as well as
    // along a row meets distinct banks
    static constexpr int PITCH = kTile * static_cast<int>(sizeof(T)) / 4 + 1;
    static constexpr int BYTES = kTile * PITCH * 4;
};

template <class T>
__device__ __forceinline__ float tile_at(const uint32_t* tile, int m, int k) {
    return to_f32<T>(reinterpret_cast<const T*>(tile + m * BothSmem<T>::PITCH)[k]);
}

template <int FMT, class T>
__global__ void __launch_bounds__(kBothThreads)
    k_fp4_quantize_both(int64_t M, int64_t K, const T* __restrict__ X, int64_t ldx, bool aligned,
                        const float* __restrict__ tscale, uint8_t* __restrict__ Xq, uint8_t* __restrict__ Xs,
                        uint8_t* __restrict__ Tq, uint8_t* __restrict__ Ts, float* __restrict__ partial) {
    constexpr int B = fp4_block(FMT);
    constexpr int NB = kTile / B;  // blocks along an axis of the tile
    constexpr int PITCH = BothSmem<T>::PITCH;
    extern __shared__ uint32_t tile[];
    __shared__ float colsum[kBothThreads / kTile][kTile];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTile, k0 = static_cast<int64_t>(blockIdx.x) * kTile;
    const float ts = FMT == kNv && tscale ? *tscale : 1.f;
    const float six_ts = __fmul_rn(6.f, ts);

    // the tile, zero outside X
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    for (int i = threadIdx.x; i < kTile * (kTile / V); i += kBothThreads) {
        const int m = i / (kTile / V), k = (i % (kTile / V)) * V;
        uint32_t w[4] = {0, 0, 0, 0};
        const int64_t left = K - (k0 + k);
        if (m0 + m < M && left > 0) {
            const T* p = X + (m0 + m) * ldx + k0 + k;
            if (aligned && left >= V) {
                const uint4 v = *reinterpret_cast<const uint4*>(p);
                w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
            } else {
                T e[V];
#pragma unroll
                for (int j = 0; j < V; ++j) e[j] = j < left ? p[j] : from_f32<T>(0.f);
                memcpy(w, e, 16);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) tile[m * PITCH + k * static_cast<int>(sizeof(T)) / 4 + j] = w[j];
    }
    __syncthreads();

    if (Xq) {
        const int64_t ld = fp4_codes_ld(K), tiles = fp4_col_tiles(FMT, K);
        for (int i = threadIdx.x; i < kTile * NB; i += kBothThreads) {
            // a warp's lanes on 32 rows of the same block
            const int m = i % kTile, b = i / kTile;
            const int64_t k = k0 + b * B;
            if (k >= 2 * ld) continue;  // uniform over the CTA's threads of a block
            float x[B];
            uint32_t codes[B / 8];
#pragma unroll
            for (int j = 0; j < B; ++j) x[j] = tile_at<T>(tile, m, b * B + j);
            const uint32_t byte = quantize_block<FMT>(x, ts, six_ts, codes);
            if (m0 + m < M) {
                uint8_t* q = Xq + (m0 + m) * ld + k / 2;
                if constexpr (B == 16)
                    *reinterpret_cast<uint2*>(q) = make_uint2(codes[0], codes[1]);
                else
                    *reinterpret_cast<uint4*>(q) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
            }
            Xs[fp4_scale_offset(m0 + m, k / B, tiles)] = static_cast<uint8_t>(m0 + m < M ? byte : 0);
        }
        // blocks between ld and the end of the last scale word
        for (int i = threadIdx.x; i < kTile * NB; i += kBothThreads) {
            const int m = i % kTile, b = i / kTile;
            const int64_t k = k0 + b * B;
            if (k >= 2 * ld && k / B < 4 * tiles) Xs[fp4_scale_offset(m0 + m, k / B, tiles)] = 0;
        }
    }
    if (Tq) {
        const int64_t ld = fp4_codes_ld(M), tiles = fp4_col_tiles(FMT, M);
        for (int i = threadIdx.x; i < kTile * NB; i += kBothThreads) {
            const int k = i % kTile, b = i / kTile;
            const int64_t m = m0 + b * B;
            if (m >= 2 * ld) continue;
            float x[B];
            uint32_t codes[B / 8];
#pragma unroll
            for (int j = 0; j < B; ++j) x[j] = tile_at<T>(tile, b * B + j, k);
            const uint32_t byte = quantize_block<FMT>(x, ts, six_ts, codes);
            if (k0 + k < K) {
                uint8_t* q = Tq + (k0 + k) * ld + m / 2;
                if constexpr (B == 16)
                    *reinterpret_cast<uint2*>(q) = make_uint2(codes[0], codes[1]);
                else
                    *reinterpret_cast<uint4*>(q) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
            }
            Ts[fp4_scale_offset(k0 + k, m / B, tiles)] = static_cast<uint8_t>(k0 + k < K ? byte : 0);
        }
        for (int i = threadIdx.x; i < kTile * NB; i += kBothThreads) {
            const int k = i % kTile, b = i / kTile;
            const int64_t m = m0 + b * B;
            if (m >= 2 * ld && m / B < 4 * tiles) Ts[fp4_scale_offset(k0 + k, m / B, tiles)] = 0;
        }
    }
    if (partial) {
        const int k = threadIdx.x % kTile, part = threadIdx.x / kTile;
        constexpr int ROWS = kTile / (kBothThreads / kTile);
        float sum = 0.f;
#pragma unroll 8
        for (int m = 0; m < ROWS; ++m) sum += tile_at<T>(tile, part * ROWS + m, k);
        colsum[part][k] = sum;
        __syncthreads();
        if (part == 0 && k0 + k < K) partial[blockIdx.y * K + k0 + k] = colsum[0][k] + colsum[1][k];
    }
}

// ------------------------------------------------------- tensor scale
//
// ts = max(fl(amax fl(1 / 2688)), 2^-100) over the finite values, 1 where all are 0:
// 2688 = 6 * 448, so the largest value of the tensor lands on the largest
// code times the largest block scale.  Each CTA leaves its maximum in the
// workspace and one more warp joins them (a maximum does not depend on the
// order); bound by reading X once.
constexpr int kAmaxThreads = 512;
constexpr int kAmaxMaxCtas = 1024;

__device__ __forceinline__ uint32_t finite_abs_bits(float v) {
    const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
    return b >= 0x7f800000u ? 0u : b;
}

template <class T>
__global__ void __launch_bounds__(kAmaxThreads)
    k_fp4_amax(int64_t M, int64_t K, const T* __restrict__ X, int64_t ldx, bool aligned,
               uint32_t* __restrict__ part) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int64_t per_row = (K + V - 1) / V;
    const int64_t items = M * per_row, step = static_cast<int64_t>(gridDim.x) * kAmaxThreads;
    uint32_t m = 0;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kAmaxThreads + threadIdx.x; i < items; i += step) {
        const int64_t row = i / per_row, k = (i - row * per_row) * V;
        float x[V];
        load_some<T, V>(X + row * ldx + k, static_cast<int>(min(K - k, int64_t(V))), aligned, x);
#pragma unroll
        for (int j = 0; j < V; ++j) m = max(m, finite_abs_bits(x[j]));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    __shared__ uint32_t wm[kAmaxThreads / 32];
    if ((threadIdx.x & 31) == 0) wm[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x < 32) {
        m = threadIdx.x < kAmaxThreads / 32 ? wm[threadIdx.x] : 0u;
        m = __reduce_max_sync(0xffffffffu, m);
        if (threadIdx.x == 0) part[blockIdx.x] = m;
    }
}

__global__ void __launch_bounds__(32) k_fp4_scale_join(const uint32_t* __restrict__ part, int parts,
                                                       float* __restrict__ scale) {
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    uint32_t m = 0;
    for (int i = threadIdx.x; i < parts; i += 32) m = max(m, part[i]);
    m = __reduce_max_sync(0xffffffffu, m);
    if (threadIdx.x == 0)
        *scale = m ? fmaxf(__fmul_rn(__uint_as_float(m), 1.f / 2688.f), 0x1p-100f) : 1.f;
}

// ------------------------------------------------------- back to values

constexpr int kDequantThreads = 256;

template <int FMT, class T>
__global__ void __launch_bounds__(kDequantThreads)
    k_fp4_dequantize(int64_t M, int64_t K, const uint8_t* __restrict__ Xq, const uint8_t* __restrict__ Xs,
                     const float* __restrict__ tscale, T* __restrict__ Y, int64_t ldy, bool aligned) {
    constexpr int B = fp4_block(FMT);
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int64_t per_row = (K + 15) / 16;  // one thread takes 16 values
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kDequantThreads + threadIdx.x;
    const int64_t row = item / per_row, k = (item - row * per_row) * 16;
    if (row >= M) return;
    const float ts = FMT == kNv && tscale ? *tscale : 1.f;
    const uint2 q = *reinterpret_cast<const uint2*>(Xq + row * fp4_codes_ld(K) + k / 2);
    const uint32_t byte = Xs[fp4_scale_offset(row, k / B, fp4_col_tiles(FMT, K))];
    const float d = __fmul_rn(scale_value<FMT>(byte), ts);
    float lo[8], hi[8], x[16];
    e2m1x8_values(q.x, lo);
    e2m1x8_values(q.y, hi);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = __fmul_rn(lo[i], d);
        x[8 + i] = __fmul_rn(hi[i], d);
    }
    store_some<T, 16>(Y + row * ldy + k, static_cast<int>(min(K - k, int64_t(16))), aligned, x);
}

// ------------------------------------------------------- host side

static bool rows_aligned(const void* p, int64_t ld, size_t elem, int64_t rows) {
    return aligned16(p) && (rows <= 1 || (static_cast<size_t>(ld) * elem) % 16 == 0);
}

int fp4_quantize_run(int fmt, int dtype, int64_t M, int64_t K, const void* X, int64_t ldx, const float* ts,
                     uint8_t* Xq, uint8_t* Xs, bool zero_pad, cudaStream_t s) {
    const int64_t rows = zero_pad ? (M + 127) / 128 * 128 : M;
    const int64_t items = rows * 4 * fp4_col_tiles(fmt, K);
    const int64_t ctas = (items + kQuantThreads - 1) / kQuantThreads;
    if (ctas == 0) return QG_OK;
    if (ctas > INT32_MAX) return QG_ERR_UNSUPPORTED;
    return by_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        const bool al = rows_aligned(X, ldx, sizeof(T), M);
        auto* f = fmt == kNv ? k_fp4_quantize<kNv, T> : k_fp4_quantize<kMx, T>;
        return launch_serialized(f, dim3(static_cast<unsigned>(ctas)), kQuantThreads, 0, 1, s, M, rows, K,
                                 static_cast<const T*>(X), ldx, al, ts, Xq, Xs);
    });
}

int fp4_quantize_both_run(int fmt, int dtype, int64_t M, int64_t K, const void* X, int64_t ldx, const float* ts,
                          uint8_t* Xq, uint8_t* Xs, uint8_t* Tq, uint8_t* Ts, float* colsum, float* partial,
                          cudaStream_t s) {
    const int64_t gx = (K + kTile - 1) / kTile, gy = (M + kTile - 1) / kTile;
    if (gy > 65535 || gx > INT32_MAX) return QG_ERR_UNSUPPORTED;
    int rc = QG_OK;
    if (gx && gy)
        rc = by_dtype(dtype, [&](auto t) {
            using T = decltype(t);
            const bool al = rows_aligned(X, ldx, sizeof(T), M);
            auto* f = fmt == kNv ? k_fp4_quantize_both<kNv, T> : k_fp4_quantize_both<kMx, T>;
            if constexpr (BothSmem<T>::BYTES > 48 * 1024) {
                const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                           BothSmem<T>::BYTES);
                if (e != cudaSuccess) return map_cuda(e);
            }
            return launch_serialized(f, dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), kBothThreads,
                                     BothSmem<T>::BYTES, 1, s, M, K, static_cast<const T*>(X), ldx, al, ts, Xq,
                                     Xs, Tq, Ts, colsum ? partial : nullptr);
        });
    if (rc || !colsum) return rc;
    return sum_partials_run(partial, gy, K, colsum, s);
}

static int amax_ctas(int64_t M, int64_t K) {
    const int64_t n = (M * ((K + 7) / 8) + kAmaxThreads - 1) / kAmaxThreads;
    return static_cast<int>(n < 1 ? 1 : n > kAmaxMaxCtas ? kAmaxMaxCtas : n);
}

#define QG_FP4_BUDGETS(T, NAME)                                                                              \
    QG_BLOCK_KERNEL_BUDGET("k_fp4_quantize<nv," NAME ">", reinterpret_cast<const void*>(k_fp4_quantize<kNv, T>), \
                           kQuantThreads, 0, 0, 1, 4);                                                       \
    QG_BLOCK_KERNEL_BUDGET("k_fp4_quantize<mx," NAME ">", reinterpret_cast<const void*>(k_fp4_quantize<kMx, T>), \
                           kQuantThreads, 0, 0, 1, 4);                                                       \
    QG_BLOCK_KERNEL_BUDGET("k_fp4_quantize_both<nv," NAME ">",                                               \
                           reinterpret_cast<const void*>(k_fp4_quantize_both<kNv, T>), kBothThreads,         \
                           BothSmem<T>::BYTES, 0, 1, 2);                                                     \
    QG_BLOCK_KERNEL_BUDGET("k_fp4_quantize_both<mx," NAME ">",                                               \
                           reinterpret_cast<const void*>(k_fp4_quantize_both<kMx, T>), kBothThreads,         \
                           BothSmem<T>::BYTES, 0, 1, 2);                                                     \
    QG_BLOCK_KERNEL_BUDGET("k_fp4_amax<" NAME ">", reinterpret_cast<const void*>(k_fp4_amax<T>), kAmaxThreads, \
                           0, 0, 1, 2);                                                                      \
    QG_BLOCK_KERNEL_BUDGET("k_fp4_dequantize<nv," NAME ">",                                                  \
                           reinterpret_cast<const void*>(k_fp4_dequantize<kNv, T>), kDequantThreads, 0, 0, 1, 4); \
    QG_BLOCK_KERNEL_BUDGET("k_fp4_dequantize<mx," NAME ">",                                                  \
                           reinterpret_cast<const void*>(k_fp4_dequantize<kMx, T>), kDequantThreads, 0, 0, 1, 4)
QG_FP4_BUDGETS(__half, "f16");
QG_FP4_BUDGETS(__nv_bfloat16, "bf16");
QG_FP4_BUDGETS(float, "f32");
QG_BLOCK_KERNEL_BUDGET("k_fp4_scale_join", reinterpret_cast<const void*>(k_fp4_scale_join), 32, 0, 0, 1, 1);

}  // namespace qg

using namespace qg;

// Checks shared by the calls that read a rows x K matrix of floating type.
static int check_matrix(int fmt, int dtype, int64_t M, int64_t K, const void* X, int64_t ldx) {
    if (!fmt_ok(fmt) || !dtype_ok(dtype)) return QG_ERR_UNSUPPORTED;
    if (M < 0 || K < 0 || M > INT32_MAX || K > INT32_MAX) return QG_ERR_INVALID_ARG;
    if (M && K && !X) return QG_ERR_INVALID_ARG;
    if (M > 1 && ldx < K) return QG_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(X) % dtype_bytes(dtype)) return QG_ERR_MISALIGNED;
    return QG_OK;
}

static int check_scale(int fmt, const float* ts) {
    if (ts && fmt == kMx) return QG_ERR_UNSUPPORTED;  // the power-of-two format has no tensor scale
    if (reinterpret_cast<uintptr_t>(ts) % 4) return QG_ERR_MISALIGNED;
    return QG_OK;
}

extern "C" {

int64_t qg_fp4_codes_ld(int64_t K) { return K > 0 ? fp4_codes_ld(K) : 0; }

size_t qg_fp4_scale_bytes(int fmt, int64_t rows, int64_t K) {
    if (!fmt_ok(fmt) || rows <= 0 || K <= 0) return 0;
    return static_cast<size_t>(fp4_scale_bytes(fmt, rows, K));
}

int fp4_tensor_scale(int dtype, int64_t M, int64_t K, const void* X, int64_t ldx, float* scale, void* ws,
                     size_t ws_bytes, void* stream) {
    const NvtxRange nvtx_range("fp4_tensor_scale");
    int rc = check_matrix(kNv, dtype, M, K, X, ldx);
    if (rc) return rc;
    if (!scale) return QG_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(scale) % 4) return QG_ERR_MISALIGNED;
    if (!ws || ws_bytes < qg_workspace_size(QG_OP_FP4_TENSOR_SCALE, 1, 1, 1)) return QG_ERR_WORKSPACE;
    if (!aligned16(ws)) return QG_ERR_MISALIGNED;
    if (current_device() < 0) return QG_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int64_t m = M, k = K;
    if (ldx == K || M <= 1) {  // rows end to end: one long row
        k = M * K;
        m = k ? 1 : 0;
    }
    const int ctas = amax_ctas(m, k);
    uint32_t* part = static_cast<uint32_t*>(ws);
    rc = by_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        return launch_serialized(k_fp4_amax<T>, dim3(static_cast<unsigned>(ctas)), kAmaxThreads, 0, 1, s, m, k,
                                 static_cast<const T*>(X), ldx, rows_aligned(X, ldx, sizeof(T), m), part);
    });
    if (rc) return rc;
    return launch_serialized(k_fp4_scale_join, dim3(1), 32, 0, 1, s, part, ctas, scale);
}

int fp4_quantize(int fmt, int dtype, int64_t M, int64_t K, const void* X, int64_t ldx, const float* tscale,
                 uint8_t* Xq, uint8_t* Xs, void* stream) {
    const NvtxRange nvtx_range("fp4_quantize");
    int rc = check_matrix(fmt, dtype, M, K, X, ldx);
    if (!rc) rc = check_scale(fmt, tscale);
    if (rc) return rc;
    if (M == 0 || K == 0) return QG_OK;
    if (!Xq || !Xs) return QG_ERR_INVALID_ARG;
    if (!aligned16(Xq) || !aligned16(Xs)) return QG_ERR_MISALIGNED;
    if (current_device() < 0) return QG_ERR_CUDA;
    return fp4_quantize_run(fmt, dtype, M, K, X, ldx, tscale, Xq, Xs, true, static_cast<cudaStream_t>(stream));
}

int fp4_quantize_both(int fmt, int dtype, int64_t M, int64_t K, const void* X, int64_t ldx, const float* tscale,
                      uint8_t* Xq, uint8_t* Xs, uint8_t* Tq, uint8_t* Ts, void* stream) {
    const NvtxRange nvtx_range("fp4_quantize_both");
    int rc = check_matrix(fmt, dtype, M, K, X, ldx);
    if (!rc) rc = check_scale(fmt, tscale);
    if (rc) return rc;
    if ((Xq == nullptr) != (Xs == nullptr)) return QG_ERR_INVALID_ARG;
    if (M == 0 || K == 0) return QG_OK;
    if (!Tq || !Ts) return QG_ERR_INVALID_ARG;
    if (!aligned16(Xq) || !aligned16(Xs) || !aligned16(Tq) || !aligned16(Ts)) return QG_ERR_MISALIGNED;
    if (current_device() < 0) return QG_ERR_CUDA;
    return fp4_quantize_both_run(fmt, dtype, M, K, X, ldx, tscale, Xq, Xs, Tq, Ts, nullptr, nullptr,
                                 static_cast<cudaStream_t>(stream));
}

int fp4_dequantize(int fmt, int dtype, int64_t M, int64_t K, const uint8_t* Xq, const uint8_t* Xs,
                   const float* tscale, void* Y, int64_t ldy, void* stream) {
    const NvtxRange nvtx_range("fp4_dequantize");
    int rc = check_matrix(fmt, dtype, M, K, Y, ldy);
    if (!rc) rc = check_scale(fmt, tscale);
    if (rc) return rc;
    if (M == 0 || K == 0) return QG_OK;
    if (!Xq || !Xs) return QG_ERR_INVALID_ARG;
    if (!aligned16(Xq) || !aligned16(Xs)) return QG_ERR_MISALIGNED;
    if (current_device() < 0) return QG_ERR_CUDA;
    const int64_t items = M * ((K + 15) / 16), ctas = (items + kDequantThreads - 1) / kDequantThreads;
    if (ctas > INT32_MAX) return QG_ERR_UNSUPPORTED;
    return by_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        auto* f = fmt == kNv ? k_fp4_dequantize<kNv, T> : k_fp4_dequantize<kMx, T>;
        return launch_serialized(f, dim3(static_cast<unsigned>(ctas)), kDequantThreads, 0, 1,
                                 static_cast<cudaStream_t>(stream), M, K, Xq, Xs, tscale, static_cast<T*>(Y), ldy,
                                 rows_aligned(Y, ldy, sizeof(T), M));
    });
}

}  // extern "C"
